"""C-ABI and binding checks of the gated delta rule that need no GPU: every case fails validation (or has nothing to do)
before anything would be enqueued."""
import ctypes

import pytest
import torch

fc = pytest.importorskip("long_fft_convolution_amd")

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def _ints(*v):
    return (ctypes.c_int64 * len(v))(*v)


def _fwd(**kw):
    a = dict(q=0x10000000, k=0x20000000, v=0x30000000, g=0x51000000, b=0x52000000, out=0x40000000, st=None, s0=None, s1=None,
             sl=None, ns=0, cu=None, B=1, N=100, H=4, Hk=2, Dk=64, Dv=64, scale=1.0, dt=2, ws=0x70000000, wsb=1 << 40)
    a.update(kw)
    return fc.lib().fftconv_delta_fwd(a["q"], a["k"], a["v"], a["g"], a["b"], a["out"], a["st"], a["s0"], a["s1"], a["sl"],
                                      a["ns"], a["cu"], a["B"], a["N"], a["H"], a["Hk"], a["Dk"], a["Dv"], a["scale"],
                                      a["dt"], a["ws"], a["wsb"], None)


COMMON = [
    (dict(dt=7), UNSUPPORTED, "dtype"), (dict(B=-1), INVALID, "B=-1"), (dict(N=-1), INVALID, "N=-1"),
    (dict(Hk=3), INVALID, "multiple"), (dict(Hk=0), INVALID, "multiple"), (dict(Dk=0), UNSUPPORTED, "Dk=0"),
    (dict(Dv=257), UNSUPPORTED, "Dv=257"), (dict(H=1 << 17, Hk=1), UNSUPPORTED, "H="),
    (dict(N=1 << 31), UNSUPPORTED, "too many"), (dict(N=1 << 30, H=64, Hk=1), UNSUPPORTED, "too many"),
    (dict(B=1 << 20, N=1, H=4, Hk=1), UNSUPPORTED, "too many"), (dict(scale=float("inf")), INVALID, "scale"),
    (dict(q=None), INVALID, "q must"), (dict(v=None), INVALID, "v must"), (dict(g=None), INVALID, "log_decay must"),
    (dict(b=None), INVALID, "beta must"), (dict(k=0x20000001), INVALID, "aligned"), (dict(g=0x51000002), INVALID, "aligned"),
    (dict(s0=0x50000002), INVALID, "aligned"), (dict(cu=0x60000002), INVALID, "aligned"),
    (dict(ws=None), WORKSPACE, "needs"), (dict(wsb=100), WORKSPACE, "needs"), (dict(ws=0x70000004), INVALID, "aligned"),
    (dict(ws=0x20000000), INVALID, "overlaps"),
]


@pytest.mark.parametrize("kw,status,text", COMMON + [
    (dict(ns=-1), INVALID, "n_slots"), (dict(out=None), INVALID, "out must"),
    (dict(st=_ints(12800, -128, 64, 12800, 128, 64, 25600, 256, 64, 25600, 256, 64)), INVALID, "negative"),
    (dict(st=_ints(12800, 128, 64, 12800, 128, 64, 25600, 256, 64, 25600, 0, 64)), INVALID, "share memory"),
    (dict(st=_ints(12800, 1 << 23, 64, 12800, 128, 64, 25600, 256, 64, 25600, 256, 64)), UNSUPPORTED, "token stride"),
    (dict(out=0x30000080), INVALID, "overlaps v"), (dict(out=0x52000000), INVALID, "overlaps beta"),
    (dict(s1=0x10000080), INVALID, "overlaps"), (dict(s0=0x60000000, s1=0x60000100), INVALID, "without being it"),
    (dict(s0=0x40000000), INVALID, "overlaps state_in"),
])
def test_prompt_refusals(kw, status, text):
    assert _fwd(**kw) == status
    assert text in fc.fftconv_last_error()


def test_nothing_to_do():
    assert _fwd(B=0) == 0 and _fwd(H=0, Hk=0) == 0 and _fwd(N=0, q=None, k=None, v=None, g=None, b=None, out=None) == 0
    assert _step(B=0) == 0
    assert _bwd(B=0) == 0 and _bwd(N=0, q=None, k=None, v=None, g=None, b=None, do=None) == 0


def _step(**kw):
    a = dict(q=0x10000000, k=0x20000000, v=0x30000000, g=0x51000000, b=0x52000000, s=0x60000000, out=0x40000000, st=None,
             sl=None, ns=0, B=3, H=4, Hk=2, Dk=64, Dv=64, scale=1.0, dt=1)
    a.update(kw)
    return fc.lib().fftconv_delta_step(a["q"], a["k"], a["v"], a["g"], a["b"], a["s"], a["out"], a["st"], a["sl"], a["ns"],
                                       a["B"], a["H"], a["Hk"], a["Dk"], a["Dv"], a["scale"], a["dt"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dt=5), UNSUPPORTED, "dtype"), (dict(Hk=3), INVALID, "multiple"), (dict(s=None), INVALID, "state must"),
    (dict(g=None), INVALID, "log_decay must"), (dict(s=0x60000002), INVALID, "aligned"), (dict(sl=0x61000001, ns=9), INVALID, "aligned"),
    (dict(out=0x30000000), INVALID, "overlaps v"), (dict(s=0x10000000), INVALID, "state overlaps"),
    (dict(out=0x60000000), INVALID, "overlaps"), (dict(st=_ints(256, 64, 128, 64, 256, 64, 0, 64)), INVALID, "share memory"),
])
def test_step_refusals(kw, status, text):
    assert _step(**kw) == status
    assert text in fc.fftconv_last_error()


def _bwd(**kw):
    a = dict(do=0x08000000, q=0x10000000, k=0x20000000, v=0x30000000, g=0x51000000, b=0x52000000, dq=0x11000000, dk=0x21000000,
             dv=0x31000000, dg=0x53000000, db=0x54000000, st=None, s0=None, ds1=None, ds0=None, cu=None, B=1, N=100, H=4, Hk=2,
             Dk=64, Dv=64, scale=1.0, dt=2, ws=0x70000000, wsb=1 << 40)
    a.update(kw)
    return fc.lib().fftconv_delta_bwd(a["do"], a["q"], a["k"], a["v"], a["g"], a["b"], a["dq"], a["dk"], a["dv"], a["dg"],
                                      a["db"], a["st"], a["s0"], a["ds1"], a["ds0"], a["cu"], a["B"], a["N"], a["H"],
                                      a["Hk"], a["Dk"], a["Dv"], a["scale"], a["dt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status,text", COMMON + [
    (dict(do=None), INVALID, "dout must"), (dict(dq=0x10000000), INVALID, "dq overlaps q"),
    (dict(dk=0x11000000), INVALID, "dk overlaps dq"), (dict(dg=0x52000000), INVALID, "dlog_decay overlaps beta"),
    (dict(db=0x53000000), INVALID, "dbeta overlaps dlog_decay"), (dict(dv=0x31000001), INVALID, "aligned"),
    (dict(s0=0x61000000, ds0=0x61000000), INVALID, "dstate_in overlaps state_in"),
])
def test_backward_refusals(kw, status, text):
    assert _bwd(**kw) == status
    assert text in fc.fftconv_last_error()


def test_workspace_sizes():
    f, b = fc.fftconv_delta_fwd_workspace_bytes, fc.fftconv_delta_bwd_workspace_bytes
    assert f(0, 17, 4, 2, 64, 64, 2) == 0 and f(1, 17, 4, 2, 64, 64, 9) == 0 and f(1, 17, 4, 2, 257, 64, 2) == 0
    assert f(1, 17, 4, 2, 64, 64, 2) >= 4 * 28 * 1024          # a record a (chunk, head)
    assert f(1, 131072, 20, 20, 128, 128, 2) >= 2048 * 20 * 28 * 1024 + 12 * 20 * 3 * 65536      # and segments' matrices
    assert b(1, 100, 4, 4, 64, 64, 2) >= 2 * 4 * (52 * 1024 + 2 * 64 * 64 * 4 + 2 * 64 * 64 * 4)
    assert b(1, 100, 4, 2, 64, 64, 2) >= b(1, 100, 4, 4, 64, 64, 2) + 2 * 100 * 4 * 64 * 4       # parts of shared heads


def test_binding_refuses_what_does_not_fit():
    q, v, g = torch.zeros(1, 5, 2, 8), torch.zeros(1, 5, 4, 8), torch.zeros(1, 5, 4)
    with pytest.raises(ValueError, match="device tensor"):
        fc.delta_attention(q, q, v, g, g)
    with pytest.raises(ValueError, match="dimensions"):
        fc.delta_attention(q[0], q, v, g, g)
    with pytest.raises(ValueError, match="dimensions"):
        fc.fftconv_delta_step(q, q, v, g, g, g, v, 1.0)
