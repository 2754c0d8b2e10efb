"""Outputs that share elements with an input that the call still reads are refused; rows
that interleave in one buffer, and the residual's or the gradient's own place, are not."""
import numpy as np
import pytest

from trellis_coded_weight_tcq_b200 import tcq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 30, 600])
def test_outputs_over_inputs(n, cuda_device):
    import torch
    from tests import gemm_reference as ref

    rng = np.random.default_rng(n)
    size = 256
    args, _ = ref.random_matrix(rng, 16, 2, 256, size, size, "f16", True, cuda_device)
    x = torch.from_numpy(rng.standard_normal((n, size))).to(cuda_device).to(torch.bfloat16)
    y, dx = tcq.gemm(*args, x), tcq.gemm_dgrad(*args, x)

    flat = torch.zeros(2 * n * size + size, dtype=torch.bfloat16, device=cuda_device)
    place = flat[:n * size].view(n, size)
    place.copy_(x)
    for at in (0, 1, 8, size - 8, (n - 1) * size + 8):  # itself, a few elements and rows further
        out = flat[at:at + n * size].view(n, size)
        for call in (lambda: tcq.gemm(*args, place, out=out), lambda: tcq.gemm_dgrad(*args, place, out=out)):
            with pytest.raises(ValueError, match="overlaps"):
                call()
        if at:
            with pytest.raises(ValueError, match="overlaps"):
                tcq.gemm(*args, x, residual=place, out=out)
            with pytest.raises(ValueError, match="overlaps"):
                tcq.act_grad8(place, None, "none", out=out)
    assert torch.equal(place, x)
    assert torch.equal(tcq.gemm(*args, place, out=flat[n * size:2 * n * size].view(n, size)), y)  # next to it

    wide = torch.zeros((n, 2 * size + 16), dtype=torch.bfloat16, device=cuda_device)
    left, right = wide[:, :size], wide[:, size:2 * size]
    for source, target in ((left, right), (right, left)):
        source.copy_(x)
        assert torch.equal(tcq.gemm(*args, source, out=target), y)
        assert torch.equal(tcq.gemm_dgrad(*args, source, out=target), dx)
        assert torch.equal(source, x)
    if n > 1:
        with pytest.raises(ValueError, match="overlaps"):
            tcq.gemm(*args, left, out=wide[:, size - 1:2 * size - 1])
    right.copy_(x)
    assert torch.equal(tcq.gemm(*args, x, residual=right, out=right), tcq.gemm(*args, x, residual=x))
    right.copy_(x)
    dz, _ = tcq.act_grad8(right, None, "none", out=right)
    assert torch.equal(dz, x)
