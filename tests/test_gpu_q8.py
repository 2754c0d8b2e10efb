"""8-bit activation checkpoints (tcq_pack8, tcq_unpack8) byte for byte against a
float64 restatement, and the gradient through an activation (tcq_act_grad8)."""
import numpy as np
import pytest

from trellis_coded_weight_tcq_b200 import tcq

pytestmark = pytest.mark.gpu


def _dtype(name):
    import torch

    return {"f16": torch.float16, "bf16": torch.bfloat16}[name]


def _rows(rng, n, cols, dtype, device, pad=0):
    import torch

    wide = rng.standard_normal((n, cols + pad)) * np.exp2(rng.integers(-12, 12, (n, 1)))
    return torch.from_numpy(wide).to(device).to(dtype)[:, pad // 2: pad // 2 + cols]


def _check_pack(x, fmt):
    import torch
    from tests import gemm_reference as ref

    p = tcq.pack8(x, fmt)
    codes, scales, values = ref.quantised(x.double().cpu().numpy(), fmt)
    np.testing.assert_array_equal(p.scales.cpu().numpy(), scales)
    one = tcq.Packed8(p.codes, torch.full_like(p.scales, 127), fmt)
    np.testing.assert_array_equal(ref.packed_values(one).cpu().numpy(), codes)
    for dtype in (torch.bfloat16, torch.float16):
        want = torch.from_numpy(values).to(dtype)  # numpy rounds float64 once, to nearest even
        if dtype == torch.float16:
            want = torch.where(torch.isinf(want), torch.full_like(want, 65504.0).copysign(want), want)
        got = tcq.unpack8(p, dtype).cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    return p


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,cols,pad", [(1, 1, 0), (1, 32, 0), (3, 33, 0), (5, 31, 1), (7, 40, 8), (9, 64, 3),
                                        (130, 4097, 0), (64, 4096, 0), (33, 1000, 16), (2, 8, 0)])
def test_pack_and_unpack(fmt, dtype, n, cols, pad, cuda_device):
    _check_pack(_rows(np.random.default_rng(n * cols), n, cols, _dtype(dtype), cuda_device, pad), fmt)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("cols", [64, 65])  # the vector and the element kernels
def test_special_values(fmt, cols, cuda_device):
    """Zeros of both signs, subnormals, the types' largest numbers, magnitudes on either
    side of each scale, exact ties; a NaN or an infinity spoils its group and no other."""
    import torch

    for dtype in (torch.bfloat16, torch.float16):
        x = torch.zeros((12, cols), dtype=dtype, device=cuda_device)
        tiny = torch.finfo(dtype).smallest_normal
        x[1] = -0.0
        x[2, ::3] = tiny / 4
        x[3] = torch.finfo(dtype).max
        x[3, ::2] = -torch.finfo(dtype).max
        x[4] = torch.arange(cols, device=cuda_device).to(dtype) + 0.5       # ties of int8
        x[5, 0], x[5, 1:] = 127.0, 0.5
        x[6, 0], x[6, 1:] = 127.5, 0.25
        x[7, 0], x[7, 1:] = 448.0, 0.0009765625
        x[8, 0], x[8, 1:] = 450.0, 17.0
        x[9, 40] = float("nan")
        x[9, 0] = 1
        x[10, 3] = float("-inf")
        x[10, 33:] = 2
        x[11] = torch.linspace(-2, 2, cols, device=cuda_device).to(dtype)
        p = _check_pack(x, fmt)
        assert int(p.scales[9, 1]) == 255 and int(p.scales[9, 0]) != 255
        assert int(p.scales[10, 0]) == 255 and int(p.scales[10, 1]) != 255


def test_unpack_into_a_strided_buffer(cuda_device):
    import torch

    x = _rows(np.random.default_rng(1), 20, 96, torch.bfloat16, cuda_device)
    p = tcq.pack8(x)
    for pad in (1, 8):
        buf = torch.full((20, 96 + pad), 9.0, dtype=torch.bfloat16, device=cuda_device)
        tcq.unpack8(p, out=buf[:, :96])
        assert torch.equal(buf[:, :96], tcq.unpack8(p)) and (buf[:, 96:] == 9).all()


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("n,rows,dtype,fmt,pad", [(1, 1, "f16", "int8", 0), (3, 40, "bf16", "e4m3", 0),
                                                  (257, 300, "bf16", "int8", 8), (100, 4099, "f16", "e4m3", 1),
                                                  (2000, 264, "bf16", "int8", 0)])
def test_act_grad(act, n, rows, dtype, fmt, pad, cuda_device):
    import torch
    from tests import gemm_reference as ref

    rng = np.random.default_rng(n + rows)
    dy = _rows(rng, n, rows, _dtype(dtype), cuda_device, pad)
    z = torch.from_numpy(rng.standard_normal((n, rows)) * 3).to(cuda_device).to(_dtype(dtype))
    p = tcq.pack8(z, fmt)
    zv = ref.packed_values(p)
    dz, db = tcq.act_grad8(dy, None if act == "none" else p, act)
    term = dy.double() * ref.act_slope(zv, act)
    off = dy.double().abs() * (ref.act_error(zv) * (1 + zv.abs()) if act not in ("none", "relu") else 0)
    bound = off + ref.half_step(dz.dtype) * (term.abs() + off) + (2.0**-25 if dz.dtype == torch.float16 else 2.0**-134)
    assert ((dz.double() - term).abs() <= bound).all()
    # sums: every term's error, and n additions
    sb = off.sum(0) + (n + 2) * 2.0**-24 * term.abs().sum(0) + 1e-300
    assert ((db.double() - term.sum(0)).abs() <= sb).all()
    # the slope against central differences of the activation
    h = 1e-6
    diff = (ref.act(zv + h, act) - ref.act(zv - h, act)) / (2 * h)
    smooth = zv.abs() > 2 * h if act == "relu" else torch.ones_like(zv, dtype=torch.bool)
    assert ((dz.double() - dy.double() * diff).abs() <= bound + 1e-8 * dy.double().abs())[smooth].all()
    # no sums wanted, and in place
    buf = dy.clone()
    dz2, none = tcq.act_grad8(buf, None if act == "none" else p, act, dbias=False, out=buf)
    assert none is None and torch.equal(dz2, dz) and dz2.data_ptr() == buf.data_ptr()
    dz3, db3 = tcq.act_grad8(dy, None if act == "none" else p, act)
    assert torch.equal(dz3, dz) and torch.equal(db3, db)


def test_act_grad_large_and_missing_values(cuda_device):
    """Pre-activations far out give slopes of 0 and 1 (no NaN); a NaN group gives NaN."""
    import torch

    z = torch.zeros((2, 64), dtype=torch.bfloat16, device=cuda_device)
    z[0, :32] = torch.tensor([1e30, -1e30, 3e38, -3e38] * 8)
    z[0, 32:] = 100.0
    z[1, 0] = float("nan")
    dy = torch.full((2, 64), 2.0, dtype=torch.bfloat16, device=cuda_device)
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        dz, _ = tcq.act_grad8(dy, tcq.pack8(z), act)
        # the int8 group of 3e38 holds 1e30 as 0
        v = tcq.unpack8(tcq.pack8(z))[0].float()
        mid = 0.0 if act == "relu" else 0.5
        want = torch.where(v > 0, torch.full_like(v, 2.0), torch.where(v < 0, torch.zeros_like(v), 2 * mid))
        assert torch.equal(dz[0].float(), want), act
        assert torch.isnan(dz[1, :32]).all() and (dz[1, 32:].float() == 2 * mid).all()


def test_act_grad_without_tokens(cuda_device):
    import torch

    dy = torch.empty((0, 70), dtype=torch.float16, device=cuda_device)
    dz, db = tcq.act_grad8(dy, None, "none")
    assert dz.shape == (0, 70) and (db == 0).all()
