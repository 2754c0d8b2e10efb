"""Batched products with a trellis-coded matrix (tcq_gemm, tcq_gemm_dgrad) and the
weight gradient from an 8-bit checkpoint (tcq_wgrad8) against float64.

Tolerances: tests/gemm_reference.py (product_bound, act_error), then half a step of
the output's type."""
import numpy as np
import pytest

from trellis_coded_weight_tcq_b200 import tcq

pytestmark = pytest.mark.gpu


def _x(rng, n, cols, dtype, device, std=1.0, pad=0):
    import torch

    wide = rng.standard_normal((n, cols + pad)) * std
    wide[:, :: 37] *= 20  # a few wide columns
    return torch.from_numpy(wide).to(device).to(dtype)[:, pad // 2: pad // 2 + cols]


def _dtype(name):
    import torch

    return {"f16": torch.float16, "bf16": torch.bfloat16}[name]


def _check(got, want, bound, what):
    import torch

    assert got.shape == want.shape
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), what
    worst = float((err / bound).max())
    assert worst <= 1, f"{what}: {worst:.3g} times its bound"


def check_gemm(args, w, x, y, act="none", bias=None, residual=None, checkpoint=None, tokens=None):
    # tokens: of the call, where x and y are a part of it
    import torch
    from tests import gemm_reference as ref

    xd = x.double()
    z = xd @ w.T
    exact = args[2] is None and (args[3] is tcq.MAD or args[3].dtype == torch.float16)
    bz = ref.product_bound(xd, w, ref.weight_half_step(tokens or x.shape[0], x.dtype, exact))
    if bias is not None:
        z = z + bias.double()
    bz = bz + 2.0**-23 * z.abs() + 1e-300
    want = ref.act(z, act)
    bound = 1.13 * bz + (ref.act_error(z) * (1 + z.abs()) if act not in ("none", "relu") else 0)
    if residual is not None:
        want = want + residual.double()
    bound = bound + ref.half_step(y.dtype) * (want.abs() + bound) + (2.0**-25 if y.dtype == torch.float16 else 0)
    _check(y, want, bound, f"gemm {args[4:]} n={x.shape[0]}")
    if checkpoint is not None:
        # every value within its quantisation step (half a unit of the group, or half an
        # e4m3 step) and the product's error of z, a step of the scale included
        v = ref.packed_values(checkpoint)
        top = torch.nn.functional.pad(z.abs() + bz, (0, -z.shape[1] % 32)).view(z.shape[0], -1, 32).amax(2)
        top = top.repeat_interleave(32, 1)[:, :z.shape[1]]
        unit = top / (64 if checkpoint.format == "int8" else 224)  # the scale is at most this
        step = unit / 2 if checkpoint.format == "int8" else torch.maximum(z.abs() * 2.0**-4, unit * 2.0**-10)
        _check(v, z, step * (1 + 2.0**-8) + 1.1 * bz, "checkpoint of z")


SHAPES = [  # L, k, T, rows, blocks per row, code, scaled, n, dtype
    (16, 2, 256, 256, 4, "f16", False, 256, "f16"),
    (16, 2, 256, 300, 3, "f16", True, 257, "bf16"),     # ragged rows and tokens
    (16, 2, 256, 1, 1, "f16", True, 1, "bf16"),         # one row, one block, one token
    (16, 2, 64, 129, 5, "mad", True, 17, "f16"),
    (16, 3, 256, 520, 2, "mad", False, 130, "bf16"),
    (16, 4, 128, 77, 3, "f16", True, 33, "bf16"),
    (12, 2, 256, 257, 2, "f32", True, 64, "f16"),
    (14, 1, 32, 40, 7, "f32", False, 5, "bf16"),
    (8, 2, 100, 65, 3, "f16", True, 9, "bf16"),         # blocks of no whole 8 columns
    (5, 3, 4, 9, 3, "f32", True, 3, "f16"),             # tiny blocks: every window meets the start state
    (16, 4, 12, 50, 5, "mad", True, 21, "f16"),
    (3, 3, 8, 33, 1, "f16", False, 40, "bf16"),         # an eight-entry table, eight columns
    (16, 2, 256, 2048, 16, "f16", True, 512, "bf16"),   # several tiles in every direction
    (12, 3, 64, 4099, 3, "f16", True, 2, "f16"),
    (16, 2, 256, 3000, 6, "f16", True, 100, "f16"),     # runs of stages that cut tiles, a ring of three
    (16, 2, 128, 1500, 24, "mad", True, 1000, "bf16"),
    (14, 1, 64, 2500, 9, "f32", True, 200, "f16"),
    (16, 4, 256, 20000, 1, "f16", False, 20, "bf16"),   # more row tiles than SMs, few stages each
    (8, 3, 64, 130, 1, "mad", True, 256, "f16"),        # one stage per tile
    (16, 2, 256, 520, 8, "f16", True, 1025, "bf16"),
    (16, 2, 256, 520, 8, "mad", True, 256, "f16"),      # the largest count decoded as it goes
    (16, 2, 256, 520, 8, "mad", True, 257, "bf16"),     # the first that decodes ahead
    (12, 2, 100, 300, 20, "f32", True, 9, "f16"),       # decoded ahead, few tiles: a cut reduction
    (16, 3, 20, 270, 130, "mad", True, 300, "bf16"),
]


@pytest.mark.parametrize("L,k,T,rows,nb,code,scaled,n,dtype", SHAPES)
def test_gemm(L, k, T, rows, nb, code, scaled, n, dtype, cuda_device):
    from tests import gemm_reference as ref

    rng = np.random.default_rng(rows * 31 + n + L)
    args, w = ref.random_matrix(rng, L, k, T, rows, nb * T, code, scaled, cuda_device)
    x = _x(rng, n, nb * T, _dtype(dtype), cuda_device)
    check_gemm(args, w, x, tcq.gemm(*args, x))


@pytest.mark.parametrize("L,k,T,rows,nb,code,scaled,n,dtype", SHAPES)
def test_gemm_dgrad(L, k, T, rows, nb, code, scaled, n, dtype, cuda_device):
    import torch
    from tests import gemm_reference as ref

    rng = np.random.default_rng(rows * 17 + n + k)
    args, w = ref.random_matrix(rng, L, k, T, rows, nb * T, code, scaled, cuda_device)
    dz = _x(rng, n, rows, _dtype(dtype), cuda_device, std=1e-3)
    dx = tcq.gemm_dgrad(*args, dz)
    d = dz.double()
    want = d @ w
    half = ref.weight_half_step(n, dz.dtype, not scaled and code != "f32")
    bound = ref.product_bound(d, w.T.contiguous(), half) + 1e-300
    if scaled:  # a weight's subnormal error is relative to its row's power
        bound = bound + 2.0**-24 * (d.abs() @ w.abs().amax(1, keepdim=True))
    bound = bound + ref.half_step(dz.dtype) * (want.abs() + bound) + (2.0**-25 if dz.dtype == torch.float16 else 0)
    _check(dx, want, bound, "dgrad")


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("n,rows,dtype,fmt", [(70, 300, "bf16", "int8"), (3, 64, "f16", "e4m3"),
                                              (257, 33, "f16", "int8"), (300, 513, "bf16", "e4m3")])
def test_gemm_epilogue(act, n, rows, dtype, fmt, cuda_device):
    """Bias, activation, residual (the output's own buffer, too) and the 8-bit
    pre-activation, together and alone."""
    import torch
    from tests import gemm_reference as ref

    rng = np.random.default_rng(n + rows)
    args, w = ref.random_matrix(rng, 16, 2, 256, rows, 512, "f16", True, cuda_device)
    x = _x(rng, n, 512, _dtype(dtype), cuda_device, std=3.0)
    bias = torch.from_numpy(rng.standard_normal(rows).astype(np.float32)).to(cuda_device)
    res = _x(rng, n, rows, _dtype(dtype), cuda_device)
    ck = tcq.Packed8(torch.empty((n, rows), dtype=torch.int8, device=cuda_device),
                     torch.empty((n, -(-rows // 32)), dtype=torch.uint8, device=cuda_device), fmt)
    y = tcq.gemm(*args, x, bias=bias, act=act, residual=res, checkpoint=ck)
    check_gemm(args, w, x, y, act, bias, res, ck)
    check_gemm(args, w, x, tcq.gemm(*args, x, act=act), act)
    buf = res.clone()
    y2 = tcq.gemm(*args, x, bias=bias, act=act, residual=buf, out=buf)
    assert y2.data_ptr() == buf.data_ptr() and torch.equal(y2, y)


@pytest.mark.parametrize("dtype,fmt", [("bf16", "e4m3"), ("f16", "int8")])
def test_gemm_epilogue_of_a_cut_reduction(dtype, fmt, cuda_device):
    """The epilogue on sums of pieces: bias, activation, residual and the 8-bit
    pre-activation, ragged rows, an output that only 2-byte stores can reach."""
    import torch
    from tests import gemm_reference as ref

    rng = np.random.default_rng(60)
    for rows in (301, 512):
        args, w = ref.random_matrix(rng, 12, 2, 100, rows, 2000, "f16", True, cuda_device)
        x = _x(rng, 33, 2000, _dtype(dtype), cuda_device)
        bias = torch.from_numpy(rng.standard_normal(rows).astype(np.float32)).to(cuda_device)
        res = _x(rng, 33, rows, _dtype(dtype), cuda_device, pad=1)
        ck = tcq.Packed8(torch.empty((33, rows), dtype=torch.int8, device=cuda_device),
                         torch.empty((33, -(-rows // 32)), dtype=torch.uint8, device=cuda_device), fmt)
        buf = torch.full((33, rows + 3), 7.0, dtype=x.dtype, device=cuda_device)
        y = tcq.gemm(*args, x, bias=bias, act="gelu", residual=res, checkpoint=ck, out=buf[:, 1:rows + 1])
        check_gemm(args, w, x, y, "gelu", bias, res, ck)
        assert (buf[:, :1] == 7).all() and (buf[:, rows + 1:] == 7).all()
        assert torch.equal(tcq.gemm(*args, x, bias=bias, act="gelu", residual=res), y)


def test_gemm_strides_and_alignment(cuda_device):
    """Odd row strides and bases that no 16-byte access may touch, in and out; what lies
    between the rows stays as it was."""
    import torch
    from tests import gemm_reference as ref

    rng = np.random.default_rng(5)
    args, w = ref.random_matrix(rng, 16, 2, 256, 200, 256, "f16", True, cuda_device)
    for dtype in ("f16", "bf16"):
        for pad in (1, 2, 8, 15):
            x = _x(rng, 40, 256, _dtype(dtype), cuda_device, pad=pad)
            buf = torch.full((40, 200 + pad), 7.0, dtype=x.dtype, device=cuda_device)
            out = buf[:, pad // 2: pad // 2 + 200]
            res = _x(rng, 40, 200, x.dtype, cuda_device, pad=pad)
            tcq.gemm(*args, x, residual=res, out=out)
            check_gemm(args, w, x, out, residual=res)
            assert (buf[:, :pad // 2] == 7).all() and (buf[:, pad // 2 + 200:] == 7).all()
            dz = _x(rng, 40, 200, x.dtype, cuda_device, pad=pad)
            gbuf = torch.full((40, 256 + pad), 7.0, dtype=x.dtype, device=cuda_device)
            tcq.gemm_dgrad(*args, dz, out=gbuf[:, pad // 2: pad // 2 + 256])
            assert torch.equal(gbuf[:, pad // 2: pad // 2 + 256], tcq.gemm_dgrad(*args, dz.contiguous()))
            assert (gbuf[:, :pad // 2] == 7).all() and (gbuf[:, pad // 2 + 256:] == 7).all()


def test_gemm_extreme_ranges(cuda_device):
    """Rows of very different size, zeros, scales far below binary16's range, and rows
    with infinities or NaN, which touch no other row."""
    import torch
    from tests import gemm_reference as ref

    rng = np.random.default_rng(11)
    args, w = ref.random_matrix(rng, 16, 2, 256, 130, 512, "f16", True, cuda_device, small_scales=True)
    x = _x(rng, 12, 512, torch.bfloat16, cuda_device)
    x[1] *= 2.0**60
    x[2] *= 2.0**-50
    x[3] = 0
    x[4, 5:] = 0
    x[5] *= 2.0**66
    check_gemm(args, w, x, tcq.gemm(*args, x))
    dz = _x(rng, 12, 130, torch.bfloat16, cuda_device)
    dz[1] *= 2.0**50
    dz[2] = 0
    got = tcq.gemm_dgrad(*args, dz).double()
    want = dz.double() @ w
    rel = (got - want).norm(dim=1) / want.norm(dim=1).clamp_min(1e-300)
    # rms: the output's rounding (at most 2^-9 each) and the weights' (2^-11)
    assert float(rel.max()) <= 2.0**-9 + 2.0**-11
    ok = tcq.gemm(*args, x)
    bad = x.clone()
    bad[0, 3] = float("nan")
    bad[6, 7] = float("inf")
    bad[7, 0], bad[7, 1] = float("inf"), float("-inf")
    y = tcq.gemm(*args, bad)
    keep = [i for i in range(12) if i not in (0, 6, 7)]
    assert torch.equal(y[keep], ok[keep])
    assert torch.isnan(y[0]).all() and not torch.isfinite(y[6]).any() and not torch.isfinite(y[7]).any()


@pytest.mark.parametrize("n", [1, 24, 600])
@pytest.mark.parametrize("code,L,T", [("f16", 16, 256), ("f32", 12, 64), ("mad", 16, 100)])
def test_matrix_arrays_at_element_alignment(code, L, T, n, cuda_device):
    """Arrays of the matrix and the bias that start one element past any larger alignment,
    and activations of an odd stride, with many tokens, too."""
    import torch
    from tests import gemm_reference as ref

    def shifted(t):
        return None if t is None else torch.cat([t.reshape(-1)[:1], t.reshape(-1)])[1:].view(t.shape)

    rng = np.random.default_rng(L + T + n)
    rows, cols = 270, 10 * T
    args, w = ref.random_matrix(rng, L, 2, T, rows, cols, code, True, cuda_device)
    odd = (shifted(args[0]), shifted(args[1]), shifted(args[2]), args[3] if code == "mad" else shifted(args[3]), *args[4:])
    bias = shifted(torch.from_numpy(rng.standard_normal(rows)).float().to(cuda_device))
    x = _x(rng, n, cols, torch.bfloat16, cuda_device, pad=3)
    res = _x(rng, n, rows, torch.bfloat16, cuda_device, pad=5)
    check_gemm(odd, w, x, tcq.gemm(*odd, x, bias=bias, act="gelu", residual=res), "gelu", bias, res)
    dz = _x(rng, n, rows, torch.bfloat16, cuda_device, pad=7)
    assert torch.equal(tcq.gemm_dgrad(*odd, dz), tcq.gemm_dgrad(*args, dz))


@pytest.mark.parametrize("n", [1, 5, 300])
def test_activations_of_extreme_values(n, cuda_device):
    """Pre-activations of any size, infinite and NaN (through the bias)."""
    import torch
    from tests import gemm_reference as ref

    inf = float("inf")
    rng = np.random.default_rng(4)
    args, _ = ref.random_matrix(rng, 16, 2, 256, 64, 256, "f16", True, cuda_device)
    big = torch.tensor([inf, -inf, float("nan"), 3e38, -3e38, 1e20, -1e20, 3e4, -3e4, 200.0, -200.0, 20.0, -20.0, 0.0, -0.0],
                       device=cuda_device)
    bias = torch.zeros(64, device=cuda_device)
    bias[:15] = big
    x = torch.zeros((n, 256), dtype=torch.bfloat16, device=cuda_device)
    for act in ("none", "relu", "silu", "gelu", "gelu_tanh"):
        z = big.double()
        want = torch.where(z == -inf, torch.zeros_like(z), ref.act(z.clamp(-1e30, 1e30), act)) if act != "none" else z
        want = torch.where(z == inf, z, want)
        want = torch.where((z.abs() > 1e30) & torch.isfinite(z), z if act == "none" else z.clamp_min(0), want)
        got = tcq.gemm(*args, x, bias=bias, act=act)[:, :15]
        want = want.float().to(torch.bfloat16)
        assert torch.isnan(got[:, 2]).all()
        keep = [i for i in range(15) if i != 2]
        # a step of bfloat16, and what a vanishing slope leaves of an fp32 exponential
        err = (got[:, keep].double() - want[keep].double()).abs()
        err = torch.where(got[:, keep] == want[keep], torch.zeros_like(err), err)
        assert (err <= 2.0**-7 * want[keep].double().abs() + 2.0**-20).all(), (act, got[0], want)


def test_gemm_zero_and_one(cuda_device):
    import torch
    from tests import gemm_reference as ref

    rng = np.random.default_rng(2)
    args, w = ref.random_matrix(rng, 16, 2, 256, 40, 256, "f16", False, cuda_device)
    x = _x(rng, 0, 256, torch.float16, cuda_device)
    assert tcq.gemm(*args, x).shape == (0, 40)
    assert tcq.gemm_dgrad(*args, x[:, :40]).shape == (0, 256)
    none = (args[0][:0], args[1][:0], None, args[3], 16, 2, 256, 0, 256)
    assert tcq.gemm(*none, _x(rng, 3, 256, torch.float16, cuda_device)).shape == (3, 0)
    dx = tcq.gemm_dgrad(*none, torch.empty((3, 0), dtype=torch.float16, device=cuda_device),
                        out=torch.ones((3, 256), dtype=torch.float16, device=cuda_device))
    assert (dx == 0).all()


def test_gemm_repeats_bit_for_bit_and_matches_the_matvec(cuda_device):
    import torch
    from tests import gemm_reference as ref

    rng = np.random.default_rng(3)
    args, w = ref.random_matrix(rng, 16, 2, 256, 700, 4096, "f16", True, cuda_device)
    x = _x(rng, 30, 4096, torch.float16, cuda_device)
    y = tcq.gemm(*args, x)
    for _ in range(3):
        assert torch.equal(tcq.gemm(*args, x), y)
    check_gemm(args, w, x, y)
    v = tcq.gemv(*args, x[4].float().contiguous())
    check_gemm(args, w, x[4:5], v.to(torch.float16)[None])  # the two kernels meet the same bound


@pytest.mark.parametrize("n,rows,cols,dtype,fmt,pad", [
    (256, 256, 256, "bf16", "int8", 0), (1, 1, 1, "f16", "int8", 0), (77, 300, 200, "bf16", "e4m3", 0),
    (1000, 513, 100, "f16", "e4m3", 0), (65, 64, 1025, "f16", "int8", 8), (129, 37, 43, "bf16", "int8", 3),
    (4099, 260, 520, "bf16", "int8", 0)])
def test_wgrad8(n, rows, cols, dtype, fmt, pad, cuda_device):
    import torch
    from tests import gemm_reference as ref

    rng = np.random.default_rng(n + rows + cols)
    dz = _x(rng, n, rows, _dtype(dtype), cuda_device, std=1e-3, pad=pad)
    packed = tcq.pack8(_x(rng, n, cols, _dtype(dtype), cuda_device), fmt)
    xv = ref.packed_values(packed)
    want = dz.double().T @ xv
    bound = (n / 16 + 2) * 2.0**-22 * (dz.double().abs().T @ xv.abs()) + 2.0**-24 * want.abs() + 1e-300
    dw = tcq.wgrad8(dz, packed)
    _check(dw, want, bound, "wgrad8")
    # added to what is there, in a strided buffer; what lies between the rows stays
    buf = torch.full((rows, cols + 5), 2.0, device=cuda_device)
    tcq.wgrad8(dz, packed, out=buf[:, :cols], accumulate=True)
    _check(buf[:, :cols], want + 2, bound + 2.0**-23 * (want.abs() + 2), "wgrad8 accumulate")
    assert (buf[:, cols:] == 2).all()
    tcq.wgrad8(dz, packed, out=buf[:, :cols])
    assert torch.equal(buf[:, :cols], dw)


@pytest.mark.parametrize("dtype,rows", [("bf16", 1801), ("f16", 1800)])
def test_cut_last_round(dtype, rows, cuda_device):
    """More tiles than the device takes at a time and a few left over: whole tiles and cut
    ones in one product (74 pairs of multiprocessors take 88 and 90 tiles in two rounds)."""
    import torch
    from tests import gemm_reference as ref

    rng = np.random.default_rng(rows)
    n = 2600
    args, w = ref.random_matrix(rng, 16, 2, 256, rows, 2560, "f16", True, cuda_device)
    x = _x(rng, n, 2560, _dtype(dtype), cuda_device)
    bias = torch.from_numpy(rng.standard_normal(rows)).float().to(cuda_device)
    residual = _x(rng, n, rows, _dtype(dtype), cuda_device)
    ck = tcq.Packed8(torch.empty((n, rows), dtype=torch.int8, device=cuda_device),
                     torch.empty((n, -(-rows // 32)), dtype=torch.uint8, device=cuda_device))
    y = tcq.gemm(*args, x, bias=bias, act="silu", residual=residual, checkpoint=ck)
    check_gemm(args, w, x, y, "silu", bias, residual, ck)
    dz = _x(rng, n, rows + 310, _dtype(dtype), cuda_device, std=1e-3)
    packed = tcq.pack8(x[:, :2500].contiguous())
    xv = ref.packed_values(packed)
    want = dz.double().T @ xv
    bound = (n / 16 + 2) * 2.0**-22 * (dz.double().abs().T @ xv.abs()) + 2.0**-24 * want.abs() + 1e-300
    dw = tcq.wgrad8(dz, packed)
    _check(dw, want, bound, "wgrad8")
    tcq.wgrad8(dz, packed, out=dw, accumulate=True)
    _check(dw, 2 * want, 2 * bound + 2.0**-23 * 2 * want.abs(), "wgrad8 accumulate")


@pytest.mark.parametrize("cols", [320, 448])
def test_dgrad_narrow_last_tiles(cols, cuda_device):
    """Tiles of one and of three column blocks, a single stage each and many per
    multiprocessor: a store may still read its box when the next tile's outputs come."""
    from tests import gemm_reference as ref

    rng = np.random.default_rng(cols)
    rows, n = 60, 60000
    args, w = ref.random_matrix(rng, 12, 2, 64, rows, cols, "f16", False, cuda_device)
    dz = _x(rng, n, rows, _dtype("f16"), cuda_device)
    d = dz.double()
    want = d @ w
    bound = ref.product_bound(d, w.T.contiguous(), 0.0) + 1e-300
    bound = bound + ref.half_step(dz.dtype) * (want.abs() + bound) + 2.0**-25
    for _ in range(5):
        _check(tcq.gemm_dgrad(*args, dz), want, bound, "dgrad")


@pytest.mark.parametrize("rows,nb,n", [(2603, 8, 2600), (14336, 9, 2100)])
def test_dgrad_cut_last_round(rows, nb, n, cuda_device):
    """The same for the input gradient; the longer one goes through its tiles in bands, the
    last of them one tile wide."""
    from tests import gemm_reference as ref

    rng = np.random.default_rng(rows + n)
    args, w = ref.random_matrix(rng, 16, 2, 256, rows, nb * 256, "mad", False, cuda_device)
    dz = _x(rng, n, rows, _dtype("f16"), cuda_device, std=1e-3)
    dx = tcq.gemm_dgrad(*args, dz)
    d = dz.double()
    want = d @ w
    bound = ref.product_bound(d, w.T.contiguous(), ref.weight_half_step(n, dz.dtype, True)) + 1e-300
    _check(dx, want, bound + ref.half_step(dz.dtype) * (want.abs() + bound) + 2.0**-25, "dgrad")


def test_wgrad8_without_tokens(cuda_device):
    import torch

    empty = tcq.Packed8(torch.empty((0, 40), dtype=torch.int8, device=cuda_device),
                        torch.empty((0, 2), dtype=torch.uint8, device=cuda_device))
    dz = torch.empty((0, 30), dtype=torch.bfloat16, device=cuda_device)
    buf = torch.full((30, 44), 3.0, device=cuda_device)
    tcq.wgrad8(dz, empty, out=buf[:, :40], accumulate=True)
    assert (buf == 3).all()
    tcq.wgrad8(dz, empty, out=buf[:, :40])
    assert (buf[:, :40] == 0).all() and (buf[:, 40:] == 3).all()
