"""A block's gradients, tight enough to tell a missing or a wrong one: every step's element
by element on the step's own inputs, and the whole chain's against float64 autograd.

The chain's tolerance: each rounding's half step, taken as its standard deviation (a rounding
error spread evenly over its step has half a step over sqrt 3), carried through the
products in squares, since the errors of different elements are independent.  It has to be
below a tenth of the gradient's own norm."""
import numpy as np
import pytest

from trellis_coded_weight_tcq_b200 import tcq

pytestmark = pytest.mark.gpu


def _half_steps(packed, cols):
    """Half a step of every element of an int8 checkpoint."""
    import torch

    return torch.exp2(packed.scales.double() - 128).repeat_interleave(32, 1)[:, :cols]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 33, 300, 2000])
def test_block_gradients(n, dtype, cuda_device):
    import torch
    from tests import gemm_reference as ref
    from tests.test_gpu_gemm import _check
    from tests.test_gpu_layer import _block

    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    up, down, x, g = _block(np.random.default_rng(500 + n), cuda_device, n, dt)
    h = up.forward(x)
    down.forward(h, residual=x)
    dh = down.backward(g)
    dx = up.backward(dh)
    half, u = ref.weight_half_step(n, dt, False), ref.half_step(dt)

    # each step
    for got, d, w in ((dh, g, down.w), (dx, up.dz, up.w)):
        dd = d.double()
        want = dd @ w
        bound = ref.product_bound(dd, w.T.contiguous(), half) + 2.0**-24 * (dd.abs() @ w.abs().amax(1, keepdim=True)) + 1e-300
        bound = bound + u * (want.abs() + bound) + (2.0**-25 if dtype == "f16" else 0)
        _check(got, want, bound, "input gradient")
        assert float((bound**2).sum().sqrt()) < 0.1 * float(want.norm())
    z = ref.packed_values(up.z8)
    term = dh.double() * ref.act_slope(z, "silu")
    off = dh.double().abs() * ref.act_error(z) * (1 + z.abs())
    assert ((up.dz.double() - term).abs() <= off + u * (term.abs() + off) + (2.0**-25 if dtype == "f16" else 0)).all()
    assert ((up.db.double() - term.sum(0)).abs() <= off.sum(0) + (n + 2) * 2.0**-24 * term.abs().sum(0) + 1e-300).all()

    # the chain: loss = sum(g y), y = silu(x Wu^T + bu) Wd^T + bd + x, without the residual's share of dx
    xd, bu = x.double().requires_grad_(), up.bias.double().requires_grad_()
    wu, wd = up.w.clone().requires_grad_(), down.w.clone().requires_grad_()
    zd = xd @ wu.T + bu
    hd = ref.act(zd, "silu")
    (g.double() * (hd @ wd.T)).sum().backward()
    zd, hd, gd, xv = zd.detach(), hd.detach(), g.double(), x.double()
    dhd = gd @ down.w
    dzd = dhd * ref.act_slope(zd, "silu")
    w2u, w2d = up.w**2, down.w**2
    z_off2 = _half_steps(up.z8, 1024)**2 + half**2 * (xv**2 @ w2u.T)
    dh_off2 = half**2 * (gd**2 @ w2d) + (u * dhd)**2
    term_off2 = (0.5 * dhd)**2 * z_off2 + 1.1**2 * dh_off2   # the slope's slope is at most 1/2, the slope 1.1
    dz_off2 = term_off2 + (u * dzd)**2 + (2.0**-50 if dtype == "f16" else 0)
    h_off2 = 1.1**2 * half**2 * (xv**2 @ w2u.T) + (u * hd)**2 + _half_steps(down.x8, 1024)**2
    x_off2 = _half_steps(up.x8, 512)**2
    checks = [(dx, xd.grad, dz_off2 @ w2u + half**2 * (dzd**2 @ w2u) + (u * xd.grad)**2),
              (up.db, bu.grad, term_off2.sum(0)),
              (up.dw, wu.grad, dz_off2.T @ xv**2 + (dzd**2).T @ x_off2),
              (down.dw, wd.grad, (gd**2).T @ h_off2),
              (down.db, gd.sum(0), 2.0**-40 * (gd**2).sum(0))]
    for i, (got, want, off2) in enumerate(checks):
        allowed, size = float(off2.sum().sqrt()), float(want.norm())
        assert allowed < 0.1 * size, (i, allowed, size)
        assert float((got.double() - want).norm()) <= allowed, i
