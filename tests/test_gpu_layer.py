"""The batched operators together, as a model uses them: a two-layer block with coded
weights run forward and backward with 8-bit checkpoints, under graph capture, on
another stream, with given outputs and workspaces."""
import numpy as np
import pytest

from trellis_coded_weight_tcq_b200 import tcq

pytestmark = pytest.mark.gpu


class Layer:
    """y = act(x W^T + b) (+ residual), keeping x and the pre-activation in 8 bits."""

    def __init__(self, rng, rows, cols, act, device):
        import torch
        from tests import gemm_reference as ref

        self.matrix, self.w = ref.random_matrix(rng, 16, 2, 256, rows, cols, "f16", True, device)
        self.bias = torch.from_numpy(0.1 * rng.standard_normal(rows).astype(np.float32)).to(device)
        self.act, self.rows = act, rows

    def forward(self, x, residual=None):
        import torch

        n = x.shape[0]
        self.x8 = tcq.pack8(x)
        self.z8 = tcq.Packed8(torch.empty((n, self.rows), dtype=torch.int8, device=x.device),
                              torch.empty((n, -(-self.rows // 32)), dtype=torch.uint8, device=x.device))
        return tcq.gemm(*self.matrix, x, bias=self.bias, act=self.act, residual=residual, checkpoint=self.z8)

    def backward(self, dy):
        dz, self.db = tcq.act_grad8(dy, self.z8, self.act)
        self.dw = tcq.wgrad8(dz, self.x8)
        self.dz = dz
        return tcq.gemm_dgrad(*self.matrix, dz)


def _block(rng, device, n, dtype):
    import torch

    up, down = Layer(rng, 1024, 512, "silu", device), Layer(rng, 512, 1024, "none", device)
    x = torch.from_numpy(rng.standard_normal((n, 512))).to(device).to(dtype)
    g = torch.from_numpy(1e-2 * rng.standard_normal((n, 512))).to(device).to(dtype)
    return up, down, x, g


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 33, 300, 2000])
def test_block_forward_and_backward(n, dtype, cuda_device):
    """Every step against float64 on the step's own inputs, and the whole block's
    gradients against float64 differences of its loss sum(g y)."""
    import torch
    from tests import gemm_reference as ref
    from tests.test_gpu_gemm import check_gemm

    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    up, down, x, g = _block(np.random.default_rng(n), cuda_device, n, dt)
    h = up.forward(x)
    y = down.forward(h, residual=x)
    check_gemm(up.matrix, up.w, x, h, "silu", up.bias, None, up.z8)
    check_gemm(down.matrix, down.w, h, y, "none", down.bias, x, down.z8)
    dh = down.backward(g)
    dx = up.backward(dh)
    assert torch.equal(down.dz, g)  # no activation
    for layer, d in ((down, g), (up, up.dz)):
        want = d.double().T @ ref.packed_values(layer.x8)
        bound = (n / 16 + 2) * 2.0**-22 * (d.double().abs().T @ ref.packed_values(layer.x8).abs()) + 1e-30
        assert ((layer.dw.double() - want).abs() <= bound + 2.0**-24 * want.abs()).all()
    # the loss in float64 from (x, b of up): differences along one random direction each
    rng = np.random.default_rng(n + 1)

    def loss(xv, bv):
        hv = ref.act(xv @ up.w.T + bv, "silu")
        return float((g.double() * (hv @ down.w.T + down.bias.double() + x.double())).sum())

    xd, bd = x.double(), up.bias.double()
    vx = torch.from_numpy(rng.standard_normal(x.shape)).to(cuda_device)
    vb = torch.from_numpy(rng.standard_normal(up.bias.shape)).to(cuda_device)
    e = 1e-4
    along_x = (loss(xd + e * vx, bd) - loss(xd - e * vx, bd)) / (2 * e)
    along_b = (loss(xd, bd + e * vb) - loss(xd, bd - e * vb)) / (2 * e)
    # dh is off by half a step and its weights' rounding, the slope by the 8-bit z: the
    # slope of silu changes by at most 1/2 per unit, z by half a step of its group
    # (amax / 128), then rounding of dz, its weights and dx (each half a step or less)
    dhd = g.double() @ down.w
    step = ref.packed_values(up.z8).abs().amax(1, keepdim=True) / 126
    u = 2.0**-8 if dtype == "bf16" else 2.0**-11
    half = ref.weight_half_step(n, dt, False)
    dz_off = dhd.abs() * (0.5 * step + 1.1 * 2 * u) + 1.1 * 8 * half * dhd.norm(dim=1, keepdim=True) / 16
    dx_off = dz_off @ up.w.abs()
    dx_off = dx_off + 2 * u * dx.double().abs() + half * (dhd.abs() @ up.w.abs())
    # the errors of different elements are independent of vx: 6 standard deviations
    off_x = 6 * float((dx_off * vx).norm())
    off_b = 6 * float((dz_off * vb).norm())
    assert abs(float((dx.double() * vx).sum()) - along_x) <= off_x + 1e-6 * abs(along_x) + 1e-7
    assert abs(float((up.db.double() * vb).sum()) - along_b) <= off_b + 1e-6 * abs(along_b) + 1e-7


def test_given_outputs_and_workspaces(cuda_device):
    import torch

    up, _, x, g = _block(np.random.default_rng(8), cuda_device, 50, torch.bfloat16)
    n, rows, cols = 50, 1024, 512
    y = tcq.gemm(*up.matrix, x)
    ws = torch.empty(tcq.tcq_gemm_workspace_bytes(16, 2, 256, rows, cols, n, tcq.TCQ_F16), dtype=torch.uint8,
                     device=cuda_device).fill_(255)
    out = torch.empty_like(y)
    assert tcq.gemm(*up.matrix, x, out=out, workspace=ws) is out and torch.equal(out, y)
    with pytest.raises(tcq.TCQError) as e:
        tcq.gemm(*up.matrix, x, workspace=ws[:-256])
    assert e.value.status == tcq.TCQ_ERR_WORKSPACE
    for wrong in (dict(out=out[:49]), dict(out=out.float()), dict(residual=g), dict(bias=up.bias[:5]),
                  dict(act="tanh"), dict(workspace=ws.float()),
                  dict(checkpoint=tcq.Packed8(up.bias, up.bias, "int8"))):
        with pytest.raises(ValueError):
            tcq.gemm(*up.matrix, x, **wrong)
    with pytest.raises(ValueError):
        tcq.gemm(*up.matrix, x[:, :256])
    with pytest.raises(TypeError):
        tcq.gemm(*up.matrix, x.float())
    with pytest.raises(ValueError):
        tcq.gemm(*up.matrix, x.t().contiguous().t())
    with pytest.raises(ValueError):
        tcq.act_grad8(y, None, "silu")
    with pytest.raises(ValueError):
        tcq.wgrad8(y, tcq.pack8(x), accumulate=True)
    with pytest.raises(ValueError):
        tcq.wgrad8(y, tcq.pack8(x[:49]))


def test_other_stream(cuda_device):
    """Launched on the current stream, or on the one given."""
    import torch

    up, _, x, _ = _block(np.random.default_rng(9), cuda_device, 40, torch.float16)
    want = tcq.gemm(*up.matrix, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = tcq.gemm(*up.matrix, x)
    b, ws = torch.empty_like(want), torch.empty(1 << 24, dtype=torch.uint8, device=cuda_device)
    s.wait_stream(torch.cuda.current_stream())
    tcq.gemm(*up.matrix, x, out=b, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


def test_given_stream_owns_what_a_call_allocates(cuda_device):
    """A stream that is given is not ordered after the current one: its results and its
    scratch are not memory that the current stream still writes, nor may the current
    stream get that scratch while the call has yet to run."""
    import torch

    up, _, x, g = _block(np.random.default_rng(10), cuda_device, 500, torch.bfloat16)
    rows, cols = 1024, 512
    nbytes = tcq.tcq_gemm_workspace_bytes(16, 2, 256, rows, cols, 500, tcq.TCQ_F16)
    want, packed = tcq.gemm(*up.matrix, x), tcq.pack8(x)
    grad = tcq.wgrad8(want, packed)
    calls = [(lambda s: tcq.gemm(*up.matrix, x, stream=s), want),
             (lambda s: tcq.gemm_dgrad(*up.matrix, want, stream=s), tcq.gemm_dgrad(*up.matrix, want)),
             (lambda s: tcq.pack8(x, stream=s).codes, packed.codes),
             (lambda s: tcq.unpack8(packed, stream=s), tcq.unpack8(packed)),
             (lambda s: tcq.act_grad8(x, packed, "silu", stream=s)[0], tcq.act_grad8(x, packed, "silu")[0]),
             (lambda s: tcq.wgrad8(want, packed, stream=s), grad)]
    s = torch.cuda.Stream()
    for call, expected in calls:
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        held = torch.empty_like(expected)  # the current stream writes it when the call is long over
        torch.cuda._sleep(50_000_000)
        held.fill_(1)
        del held
        got = call(s)
        torch.cuda.synchronize()
        assert torch.equal(got, expected)
    torch.cuda.empty_cache()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
    got = calls[0][0](s)
    other = torch.empty(nbytes, dtype=torch.uint8, device=cuda_device).fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and bool((other == 255).all())


def test_calls_side_by_side(cuda_device):
    """Blocks of different sizes on four streams at once, each several times, and a captured
    one replayed among them, give the bits of the same calls alone."""
    import torch

    sizes = (1, 40, 300, 2000)
    blocks = [_block(np.random.default_rng(60 + n), cuda_device, n, torch.bfloat16) for n in sizes]

    def step(up, down, x, g):
        h = up.forward(x)
        y = down.forward(h, residual=x)
        dx = up.backward(down.backward(g))
        return y, dx, up.dw, up.db, down.dw, down.db

    want = [[t.clone() for t in step(*b)] for b in blocks]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(*blocks[2])
    streams = [torch.cuda.Stream() for _ in sizes]
    got = [[] for _ in sizes]
    for _ in range(6):
        for i, (s, b) in enumerate(zip(streams, blocks)):
            with torch.cuda.stream(s):
                got[i].append(step(*b))
        graph.replay()
    torch.cuda.synchronize()
    for runs, expected in zip(got, want):
        for run in runs:
            assert all(torch.equal(a, b) for a, b in zip(run, expected))
    assert all(torch.equal(a, b) for a, b in zip(captured, want[2]))
    del graph


@pytest.mark.parametrize("n", [1, 40, 700])
def test_capture_and_replay(n, cuda_device):
    """The block's forward and backward captured once and replayed on new inputs gives
    the bits of direct calls; a direct call in between does not disturb the graph."""
    import torch

    rng = np.random.default_rng(77)
    up, down, x, g = _block(rng, cuda_device, n, torch.bfloat16)
    xs, gs = x.clone(), g.clone()

    def step(a, b):
        h = up.forward(a)
        y = down.forward(h, residual=a)
        dx = up.backward(down.backward(b))
        return y, dx, up.dw, up.db, down.dw, down.db

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(xs, gs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(xs, gs)
    for seed in (1, 2):
        r = np.random.default_rng(seed)
        xs.copy_(torch.from_numpy(r.standard_normal(x.shape)))
        gs.copy_(torch.from_numpy(1e-2 * r.standard_normal(g.shape)))
        want = [t.clone() for t in step(xs.clone(), gs.clone())]
        graph.replay()
        step(x, g)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    del graph


def test_leaves_the_error_word_clear(cuda_device):
    assert tcq.device_errors() == 0
