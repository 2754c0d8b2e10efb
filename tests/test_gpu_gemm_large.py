"""Offsets past 32 bits in the batched products and the 8-bit checkpoints: outputs and
inputs of more than 2^31 elements, checked at both ends."""
import numpy as np
import pytest

from trellis_coded_weight_tcq_b200 import tcq

pytestmark = pytest.mark.gpu


def _needs(gib):
    import torch

    if torch.cuda.get_device_properties(0).total_memory < gib * 2**30:
        pytest.skip(f"needs {gib} GiB")


def test_products_past_32_bits(cuda_device):
    import torch
    from tests import gemm_reference as ref
    from tests.test_gpu_gemm import check_gemm

    _needs(60)
    rng = np.random.default_rng(1)
    rows, n = 16500, 131100  # 2.16e9 outputs
    args, w = ref.random_matrix(rng, 8, 2, 64, rows, 64, "f16", True, cuda_device)
    x = torch.randn(n, 64, device=cuda_device).to(torch.float16)
    y = tcq.gemm(*args, x)
    for part in (slice(0, 300), slice(n // 2, n // 2 + 300), slice(n - 300, n)):
        check_gemm(args, w, x[part], y[part])
    dx = tcq.gemm_dgrad(*args, y)  # 2.16e9 inputs
    for part in (slice(0, 40), slice(n - 40, n)):
        want = y[part].double() @ w
        err = (dx[part].double() - want).norm() / want.norm()
        assert float(err) < 2.0**-10  # the output's and the weights' half steps, 2^-11 each
    del x, dx
    ck = tcq.pack8(y, "int8")
    codes, scales, values = ref.quantised(y[-3:].double().cpu().numpy(), "int8")
    np.testing.assert_array_equal(ck.scales[-3:].cpu().numpy(), scales)
    np.testing.assert_array_equal(ck.codes[-3:].cpu().numpy(), codes)
    dz, db = tcq.act_grad8(y, ck, "silu")
    v = ref.packed_values(tcq.Packed8(ck.codes[-3:], ck.scales[-3:]))
    term = y[-3:].double() * ref.act_slope(v, "silu")
    off = y[-3:].double().abs() * ref.act_error(v) * (1 + v.abs())
    assert ((dz[-3:].double() - term).abs() <= off + 2.0**-11 * (term.abs() + off) + 2.0**-25).all()
    back = tcq.unpack8(ck, torch.float16, out=dz)
    assert torch.equal(back[-3:].double().cpu(), torch.from_numpy(values).to(torch.float16).double())


def test_weight_gradient_past_32_bits(cuda_device):
    import torch
    from tests import gemm_reference as ref

    _needs(60)
    rows, cols, n = 47000, 46000, 17
    dz = torch.randn(n, rows, device=cuda_device).to(torch.bfloat16)
    p = tcq.pack8(torch.randn(n, cols, device=cuda_device).to(torch.bfloat16))
    dw = tcq.wgrad8(dz, p)
    v = ref.packed_values(p)
    for part in (slice(0, 100), slice(rows - 100, rows)):
        want = dz[:, part].double().T @ v
        bound = 4 * 2.0**-22 * (dz[:, part].double().abs().T @ v.abs()) + 1e-30
        assert ((dw[part].double() - want).abs() <= bound).all()
