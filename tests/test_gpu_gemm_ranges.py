"""Batched products with a trellis-coded matrix whose parts lie far from 1: tables of tiny
and of huge entries, activations, scales and entries of opposite powers, entries that are not finite.

Tolerances: tests/gemm_reference.py (product_bound), then half a step of the output's
type.  Powers of two change no rounding, so the bounds are those of matrices near 1."""
import numpy as np
import pytest

from trellis_coded_weight_tcq_b200 import tcq

pytestmark = pytest.mark.gpu


def _coded(rng, L, k, T, rows, cols, table, scale, device):
    """(arguments of tcq.gemm up to cols, W in float64) for a given numpy table and
    per-block scales (or None)."""
    import torch
    from oracle import oracle_decode

    nb = rows * (cols // T)
    W = tcq.tcq_words_per_block(k, T)
    bits = rng.integers(0, 2**32, size=(nb, W), dtype=np.uint64).astype(np.uint32)
    used = T * k - 32 * (W - 1)
    if used < 32:
        bits[:, -1] &= np.uint32(((1 << used) - 1) << (32 - used))
    start = rng.integers(0, 2**32, size=nb, dtype=np.uint64).astype(np.uint32)
    values = oracle_decode(bits, start, table, L, k, T).reshape(rows, cols)
    if scale is not None:
        values = values * np.repeat(scale.astype(np.float64).reshape(rows, -1), T, axis=1)
        scale = torch.from_numpy(scale).to(device)
    return (torch.from_numpy(bits.view(np.int32)).to(device), torch.from_numpy(start.view(np.int32)).to(device), scale,
            torch.from_numpy(table).to(device), L, k, T, rows, cols), torch.from_numpy(values).to(device)


def _table(rng, L, code, power):
    """Normal entries of standard deviation 2^power."""
    return (rng.standard_normal(1 << L) * 2.0**power).astype(np.float16 if code == "f16" else np.float32)


def _check_dgrad(args, w, dz, what):
    import torch
    from tests import gemm_reference as ref
    from tests.test_gpu_gemm import _check

    dx = tcq.gemm_dgrad(*args, dz)
    d = dz.double()
    want = d @ w
    half = ref.weight_half_step(dz.shape[0], dz.dtype, args[2] is None and args[3].dtype == torch.float16)
    bound = ref.product_bound(d, w.T.contiguous(), half) + 1e-300
    bound = bound + 2.0**-24 * (d.abs() @ w.abs().amax(1, keepdim=True))
    _check(dx, want, bound + ref.half_step(dz.dtype) * (want.abs() + bound) +
           (2.0**-25 if dz.dtype == torch.float16 else 0), what)


@pytest.mark.parametrize("n", [1, 24, 600])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T", [64, 100])  # decoded inside the product, and ahead of it
@pytest.mark.parametrize("code,power,scaled,xpower", [
    ("f32", -24, True, 0), ("f32", -24, False, 8), ("f32", 20, True, 0), ("f32", 20, False, -13),
    ("f16", -18, True, 0), ("f16", 13, True, 0), ("f16", 13, False, -8), ("f16", -18, False, 6)])
def test_tables_far_from_one(code, power, scaled, xpower, T, dtype, n, cuda_device):
    """Entries of about 6e-8 and 1e6 (binary32), of 4e-6 (steps of binary16's subnormals) and
    of 8192 (binary16), with scales that bring the weights to about 0.02, and without."""
    import torch
    from tests.test_gpu_gemm import check_gemm

    rng = np.random.default_rng(n + T + power + 100)
    rows, cols, L = 130, 6 * T, 16 if code == "f16" else 12
    scale = (rng.lognormal(-4.0, 0.5, rows * 6) * 2.0**-power).astype(np.float32) if scaled else None
    args, w = _coded(rng, L, 2, T, rows, cols, _table(rng, L, code, power), scale, cuda_device)
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    x = torch.from_numpy(rng.standard_normal((n, cols)) * 2.0**xpower).to(cuda_device).to(dt)
    check_gemm(args, w, x, tcq.gemm(*args, x))
    dz = torch.from_numpy(rng.standard_normal((n, rows)) * 2.0**xpower).to(cuda_device).to(dt)
    _check_dgrad(args, w, dz, "dgrad")


@pytest.mark.parametrize("n", [1, 24, 600])
@pytest.mark.parametrize("T", [64, 100])
@pytest.mark.parametrize("xpower,spower,tpower", [(120, -118, 0), (-122, 110, 0), (60, 90, -100), (-60, -90, 100),
                                                  (110, 0, -100), (-110, 0, 100)])
def test_opposite_powers(xpower, spower, tpower, T, n, cuda_device):
    """Activations, scales and table entries whose powers nearly cancel, while two of the
    three together pass the ends of fp32's range."""
    import torch
    from tests.test_gpu_gemm import check_gemm

    rng = np.random.default_rng(n + T + xpower + 200)
    rows, cols, L = 130, 5 * T, 12
    scale = (rng.lognormal(0.0, 0.5, rows * 5) * 2.0**spower).astype(np.float32) if spower else None
    args, w = _coded(rng, L, 2, T, rows, cols, _table(rng, L, "f32", tpower), scale, cuda_device)
    x = torch.from_numpy(rng.standard_normal((n, cols)) * 2.0**xpower).to(cuda_device).to(torch.bfloat16)
    check_gemm(args, w, x, tcq.gemm(*args, x))
    dz = torch.from_numpy(rng.standard_normal((n, rows)) * 2.0**xpower).to(cuda_device).to(torch.bfloat16)
    _check_dgrad(args, w, dz, "dgrad")


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("n", [1, 24, 600])
@pytest.mark.parametrize("T,nb", [(64, 3), (100, 3)])
def test_table_entry_that_is_not_finite(T, nb, n, scaled, bad, cuda_device):
    """The outputs of rows that never decode to it are what they are with any other entry
    there, behind the last column, too."""
    import torch

    rng = np.random.default_rng(T + n)
    rows, cols = 20, T * nb
    table = _table(rng, 16, "f16", 0)
    scale = rng.lognormal(-4.0, 0.5, rows * nb).astype(np.float32) if scaled else None
    state = rng.bit_generator.state
    args, w = _coded(rng, 16, 2, T, rows, cols, table, scale, cuda_device)
    table[0] = bad
    rng.bit_generator.state = state
    args2, w2 = _coded(rng, 16, 2, T, rows, cols, table, scale, cuda_device)
    keep = torch.isfinite(w2).all(1)
    assert torch.equal(args[0], args2[0]) and int(keep.sum()) >= 10
    x = torch.from_numpy(rng.standard_normal((n, cols))).to(cuda_device).to(torch.bfloat16)
    y, y2 = tcq.gemm(*args, x), tcq.gemm(*args2, x)
    assert torch.isfinite(y2[:, keep]).all()
    assert torch.equal(y2[:, keep], y[:, keep])


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [4, 64])
def test_small_elements_beside_a_large_one(T, dtype, scaled, cuda_device):
    """Rows brought to binary16 by a power of two are exact down to 2^-31 of their largest
    element (bfloat16) or 2^-28 (binary16, rows that are not aligned), and within 2^-39 of
    it below.  The identity, in codes of one symbol per weight, shows every element."""
    import torch

    k = L = 4
    size = 64
    if dtype == "bf16":
        dt, pad, top, least, eps = torch.bfloat16, 0, 1.0, 2.0**-31, 2.0**-7
        small = [2.0**-20 * (1 + eps), least, least * (1 + eps), least * (2 - eps), least / 2 * (1 + eps), 2.0**-36 * 1.25,
                 2.0**-60]
    else:
        dt, pad, top, least, eps = torch.float16, 1, 2.0**15, 2.0**-13, 2.0**-10
        small = [1 + eps, least, least * (1 + eps), least * (2 - eps), least / 2 * (1 + eps), 2.0**-24]
    table = np.zeros(16, dtype=np.float16)
    table[1] = 1.0
    blocks = np.eye(size, dtype=np.uint64).reshape(-1, T)
    words = np.zeros((blocks.shape[0], max(1, T * k // 32)), dtype=np.uint64)
    for t in range(T):
        words[:, t * k // 32] |= blocks[:, t] << np.uint64(32 - k - t * k % 32)
    bits = torch.from_numpy(words.astype(np.uint32).view(np.int32)).to(cuda_device)
    start = torch.zeros(blocks.shape[0], dtype=torch.int32, device=cuda_device)
    times = 0.5 if scaled else 1.0
    scale = torch.full((blocks.shape[0],), times, device=cuda_device) if scaled else None
    x = torch.zeros((2, size + 2 * pad), dtype=dt, device=cuda_device)[:, pad:pad + size]
    for i, v in enumerate(small):
        x[0, 5 * i + 1] = v
        assert float(x[0, 5 * i + 1]) == v
    x[0, 0] = top
    args = (bits, start, scale, torch.from_numpy(table).to(cuda_device), L, k, T, size, size)
    for y in (tcq.gemm(*args, x), tcq.gemm_dgrad(*args, x)):
        for i, v in enumerate(small):
            got = float(y[0, 5 * i + 1])
            if v >= least and (dtype == "bf16" or v * times >= 2.0**-13):
                assert got == v * times
            else:  # and the output's own half step
                off = 2.0**-39 * top * times
                assert abs(got - v * times) <= off + max(eps / 2 * (v * times + off), 2.0**-25 if dtype == "f16" else 0)
        assert float(y[0, 0]) == top * times and bool((y[1] == 0).all())


@pytest.mark.parametrize("n", [1, 24, 300])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T", [64, 100])
@pytest.mark.parametrize("code", ["f16", "f32", "mad"])
def test_blocks_of_unequal_scale(code, T, dtype, n, cuda_device):
    """A row's blocks of scales 2^20 apart, met by activations as much larger: the small
    block's weights keep their bits, in its columns of the input gradient, too.  The bound has
    a half step of each weight and nothing relative to the row's largest."""
    import torch
    from tests import gemm_reference as ref
    from tests.test_gpu_gemm import _check

    rng = np.random.default_rng(T + n + len(code))
    rows, nb, L = 130, 4, 12
    size = np.where(np.arange(nb) % 2 == 0, 1.0, 2.0**-20)
    scale = (rng.lognormal(-2.0, 0.3, (rows, nb)) * size).astype(np.float32).reshape(-1)
    if code == "mad":
        args, w = ref.random_matrix(rng, L, 2, T, rows, nb * T, "mad", False, cuda_device)
        w = w * torch.from_numpy(np.repeat(scale.astype(np.float64).reshape(rows, nb), T, axis=1)).to(cuda_device)
        args = (*args[:2], torch.from_numpy(scale).to(cuda_device), *args[3:])
    else:
        args, w = _coded(rng, L, 2, T, rows, nb * T, _table(rng, L, code, 0), scale, cuda_device)
    dt = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    reach = torch.from_numpy(np.repeat(np.where(size == 1, 2.0**-10, 2.0**10), T)).to(cuda_device)
    x = (torch.from_numpy(rng.standard_normal((n, nb * T))).to(cuda_device) * reach).to(dt)
    dz = torch.from_numpy(rng.standard_normal((n, rows)) * 2.0**8).to(cuda_device).to(dt)
    half = ref.weight_half_step(n, dt, False)
    for got, a, b in ((tcq.gemm(*args, x), x.double(), w), (tcq.gemm_dgrad(*args, dz), dz.double(), w.T.contiguous())):
        want = a @ b.T
        bound = (a.shape[1] / 16 + 2) * 2.0**-22 * (a.abs() @ b.abs().T) + 8 * half * ((a * a) @ (b * b).T).sqrt()
        _check(got, want, bound + ref.half_step(dt) * (want.abs() + bound) + (2.0**-25 if dtype == "f16" else 0), "unequal blocks")
