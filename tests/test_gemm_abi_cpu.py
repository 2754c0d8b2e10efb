"""Host-side checks of the batched products and the 8-bit checkpoints that need no
GPU: every refusal comes before any CUDA call, sizes are as documented."""
import ctypes

import pytest

from trellis_coded_weight_tcq_b200 import tcq

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call below ends on the host
ODD = ctypes.c_void_p(0x10001)
BIG = 1 << 40
OK, INVALID, UNSUPPORTED, WORKSPACE = (tcq.TCQ_OK, tcq.TCQ_ERR_INVALID_ARG, tcq.TCQ_ERR_UNSUPPORTED,
                                       tcq.TCQ_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def lib():
    from trellis_coded_weight_tcq_b200 import build

    build.build()
    return tcq.load_library()


def _gemm(**over):
    v = dict(bits=FAKE, st=FAKE, sc=None, cb=FAKE, dt=tcq.TCQ_F16, L=16, k=2, T=256, rows=64, cols=512, x=FAKE,
             xt=tcq.TCQ_X_BF16, ldx=512, n=4, bias=None, act=0, res=None, ldr=0, y=FAKE, ldy=64, zc=None, zs=None,
             zf=0, ws=FAKE, wsb=BIG)
    v.update(over)
    return tcq.tcq_gemm(v["bits"], v["st"], v["sc"], v["cb"], v["dt"], v["L"], v["k"], v["T"], v["rows"], v["cols"],
                        v["x"], v["xt"], v["ldx"], v["n"], v["bias"], v["act"], v["res"], v["ldr"], v["y"], v["ldy"],
                        v["zc"], v["zs"], v["zf"], v["ws"], v["wsb"], None)


MATRIX_REFUSALS = [
    (dict(dt=3), INVALID), (dict(rows=-1), INVALID), (dict(cols=-256), INVALID), (dict(cols=500), INVALID),
    (dict(rows=1 << 31), INVALID), (dict(L=17), UNSUPPORTED), (dict(k=5), UNSUPPORTED), (dict(k=0), UNSUPPORTED),
    (dict(T=255, cols=510), UNSUPPORTED), (dict(T=0), UNSUPPORTED), (dict(dt=tcq.TCQ_F32), UNSUPPORTED),
    (dict(bits=None), INVALID), (dict(st=None), INVALID), (dict(cb=None), INVALID), (dict(cb=ODD), INVALID),
    (dict(bits=ctypes.c_void_p(0x10002)), INVALID), (dict(sc=ctypes.c_void_p(0x10002)), INVALID),
    (dict(ws=None), INVALID), (dict(ws=ctypes.c_void_p(0x10080)), INVALID), (dict(wsb=0), WORKSPACE),
    (dict(n=-1), INVALID), (dict(n=1 << 31), INVALID), (dict(xt=2), INVALID),
]


@pytest.mark.parametrize("over,status", MATRIX_REFUSALS + [
    (dict(x=None), INVALID), (dict(x=ODD), INVALID), (dict(ldx=511), INVALID), (dict(y=None), INVALID),
    (dict(ldy=63), INVALID), (dict(res=ODD, ldr=64), INVALID), (dict(res=FAKE, ldr=63), INVALID),
    (dict(bias=ctypes.c_void_p(0x10002)), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID),
    (dict(zf=2), INVALID), (dict(zc=FAKE), INVALID), (dict(zs=FAKE), INVALID), (dict(cols=0), INVALID)])
def test_gemm_refusals(over, status):
    assert _gemm(**over) == status


def test_gemm_single_token_needs_no_workspace():
    import torch

    if torch.cuda.is_available():
        pytest.skip("passes the checks: with a GPU there it would run on the made-up addresses")
    assert _gemm(n=1, ws=None, wsb=0) not in (INVALID, WORKSPACE)
    assert _gemm(n=1, ws=None, wsb=0, zc=FAKE, zs=FAKE) == INVALID


def test_gemm_without_work():
    assert _gemm(n=0, x=None, y=None, ws=None, wsb=0) == OK
    assert _gemm(rows=0, bits=None, st=None, x=None, y=None, ws=None, wsb=0) == OK


def _dgrad(**over):
    v = dict(bits=FAKE, st=FAKE, sc=None, cb=FAKE, dt=tcq.TCQ_F16, L=16, k=2, T=256, rows=64, cols=512, dz=FAKE,
             xt=tcq.TCQ_X_F16, lddz=64, n=4, dx=FAKE, lddx=512, ws=FAKE, wsb=BIG)
    v.update(over)
    return tcq.tcq_gemm_dgrad(v["bits"], v["st"], v["sc"], v["cb"], v["dt"], v["L"], v["k"], v["T"], v["rows"],
                              v["cols"], v["dz"], v["xt"], v["lddz"], v["n"], v["dx"], v["lddx"], v["ws"], v["wsb"],
                              None)


@pytest.mark.parametrize("over,status", MATRIX_REFUSALS + [
    (dict(dz=None), INVALID), (dict(lddz=63), INVALID), (dict(dx=None), INVALID), (dict(lddx=511), INVALID),
    (dict(dx=ODD), INVALID)])
def test_gemm_dgrad_refusals(over, status):
    assert _dgrad(**over) == status
    assert _dgrad(n=0, dz=None, dx=None, ws=None) == OK


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), INVALID), (dict(rows=-1), INVALID), (dict(cols=1 << 31), INVALID), (dict(xt=2), INVALID),
    (dict(fmt=2), INVALID), (dict(dz=None), INVALID), (dict(lddz=63), INVALID), (dict(codes=None), INVALID),
    (dict(scales=None), INVALID), (dict(dw=None), INVALID), (dict(dw=ctypes.c_void_p(0x10002)), INVALID),
    (dict(lddw=95), INVALID), (dict(ws=None), INVALID), (dict(wsb=100), WORKSPACE), (dict(rows=0, dw=None), OK),
    (dict(cols=0, dw=None), OK), (dict(n=0, acc=1, dz=None, codes=None), OK)])
def test_wgrad8_refusals(over, status):
    v = dict(dz=FAKE, xt=0, lddz=64, codes=FAKE, scales=FAKE, fmt=0, n=4, rows=64, cols=96, dw=FAKE, lddw=96, acc=0,
             ws=FAKE, wsb=BIG)
    v.update(over)
    assert tcq.tcq_wgrad8(v["dz"], v["xt"], v["lddz"], v["codes"], v["scales"], v["fmt"], v["n"], v["rows"],
                          v["cols"], v["dw"], v["lddw"], v["acc"], v["ws"], v["wsb"], None) == status


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), INVALID), (dict(cols=-1), INVALID), (dict(xt=2), INVALID), (dict(fmt=-1), INVALID),
    (dict(x=None), INVALID), (dict(x=ODD), INVALID), (dict(ldx=39), INVALID), (dict(codes=None), INVALID),
    (dict(scales=None), INVALID), (dict(n=0, x=None), OK), (dict(cols=0, x=None), OK)])
def test_pack8_refusals(over, status):
    v = dict(x=FAKE, xt=1, ldx=40, n=3, cols=40, fmt=1, codes=FAKE, scales=FAKE)
    v.update(over)
    assert tcq.tcq_pack8(v["x"], v["xt"], v["ldx"], v["n"], v["cols"], v["fmt"], v["codes"], v["scales"],
                         None) == status
    assert tcq.tcq_unpack8(v["codes"], v["scales"], v["fmt"], v["n"], v["cols"], v["x"], v["xt"], v["ldx"],
                           None) == status


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), INVALID), (dict(rows=-1), INVALID), (dict(xt=2), INVALID), (dict(zf=2), INVALID),
    (dict(act=5), INVALID), (dict(dy=None), INVALID), (dict(dz=None), INVALID), (dict(lddy=39), INVALID),
    (dict(lddz=39), INVALID), (dict(zc=None), INVALID), (dict(zs=None), INVALID), (dict(db=ODD), INVALID),
    (dict(ws=None), INVALID), (dict(wsb=0), WORKSPACE), (dict(rows=0, dy=None), OK), (dict(n=0, db=None, dy=None), OK)])
def test_act_grad8_refusals(over, status):
    v = dict(dy=FAKE, xt=0, lddy=40, zc=FAKE, zs=FAKE, zf=0, act=2, n=3, rows=40, dz=FAKE, lddz=40, db=FAKE, ws=FAKE,
             wsb=BIG)
    v.update(over)
    assert tcq.tcq_act_grad8(v["dy"], v["xt"], v["lddy"], v["zc"], v["zs"], v["zf"], v["act"], v["n"], v["rows"],
                             v["dz"], v["lddz"], v["db"], v["ws"], v["wsb"], None) == status


def test_workspace_queries():
    F16 = tcq.TCQ_F16
    assert tcq.tcq_gemm_workspace_bytes(16, 2, 256, 64, 512, 0, F16) == 0
    assert tcq.tcq_gemm_workspace_bytes(16, 2, 256, 64, 500, 4, F16) == 0
    assert tcq.tcq_gemm_workspace_bytes(17, 2, 256, 64, 512, 4, F16) == 0
    for n in (1, 3, 300, 5000):
        assert tcq.tcq_gemm_workspace_bytes(16, 2, 256, 64, 512, n, F16) > 0
        assert tcq.tcq_gemm_dgrad_workspace_bytes(16, 2, 256, 64, 512, n, F16) > 0
        assert tcq.tcq_wgrad8_workspace_bytes(64, 96, n) >= 2 * n * 96
        assert tcq.tcq_act_grad8_workspace_bytes(n, 40) >= 160
    assert tcq.tcq_wgrad8_workspace_bytes(64, 96, 0) == 0 and tcq.tcq_act_grad8_workspace_bytes(0, 40) == 0


def test_binding_refusals():
    """The Python functions refuse CPU tensors, wrong types and wrong shapes themselves."""
    import torch

    cb = torch.zeros(1 << 16, dtype=torch.float16)
    bits, start = torch.zeros((8, 16), dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    x = torch.zeros((3, 512), dtype=torch.bfloat16)
    for call in (lambda: tcq.gemm(bits, start, None, cb, 16, 2, 256, 4, 512, x),
                 lambda: tcq.gemm_dgrad(bits, start, None, cb, 16, 2, 256, 4, 512, x[:, :4]),
                 lambda: tcq.pack8(x), lambda: tcq.act_grad8(x, None, "none"),
                 lambda: tcq.wgrad8(x, tcq.Packed8(x.to(torch.int8), torch.zeros((3, 16), dtype=torch.uint8)))):
        with pytest.raises(ValueError):
            call()
