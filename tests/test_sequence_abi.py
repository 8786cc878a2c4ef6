"""C-ABI checks of decay attention and the linear product that need no GPU: every case here fails validation (or has
nothing to do) before anything would be enqueued."""
import ctypes

import pytest

fc = pytest.importorskip("long_fft_convolution_amd")

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def _ints(*v):
    return (ctypes.c_int64 * len(v))(*v)


def _fwd(**kw):
    a = dict(q=0x10000000, k=0x20000000, v=0x30000000, ld=0x1000, out=0x40000000, st=None, s0=None, s1=None, sl=None, ns=0,
             cu=None, B=1, N=100, H=4, Hk=2, Dk=64, Dv=64, scale=1.0, dt=2, ws=0x70000000, wsb=1 << 40)
    a.update(kw)
    return fc.lib().fftconv_decay_fwd(a["q"], a["k"], a["v"], a["ld"], a["out"], a["st"], a["s0"], a["s1"], a["sl"], a["ns"],
                                      a["cu"], a["B"], a["N"], a["H"], a["Hk"], a["Dk"], a["Dv"], a["scale"], a["dt"],
                                      a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dt=7), UNSUPPORTED, "dtype"), (dict(B=-1), INVALID, "B=-1"), (dict(N=-1), INVALID, "N=-1"),
    (dict(Hk=3), INVALID, "multiple"), (dict(Hk=0), INVALID, "multiple"), (dict(Dk=0), UNSUPPORTED, "Dk=0"),
    (dict(Dv=257), UNSUPPORTED, "Dv=257"), (dict(H=1 << 17, Hk=1), UNSUPPORTED, "H="),
    (dict(N=1 << 31), UNSUPPORTED, "too many"), (dict(scale=float("nan")), INVALID, "scale"),
    (dict(ns=-1), INVALID, "n_slots"), (dict(q=None), INVALID, "q must"), (dict(out=None), INVALID, "out must"),
    (dict(ld=None), INVALID, "log_decay"), (dict(k=0x20000001), INVALID, "aligned"), (dict(s0=0x50000002), INVALID, "aligned"),
    (dict(cu=0x60000002), INVALID, "aligned"),
    (dict(st=_ints(25600, -256, 64, 12800, 128, 64, 12800, 128, 64, 25600, 256, 64)), INVALID, "negative"),
    (dict(st=_ints(25600, 256, 64, 12800, 128, 64, 12800, 128, 64, 25600, 0, 64)), INVALID, "share memory"),
    (dict(st=_ints(25600, 1 << 60, 64, 12800, 128, 64, 12800, 128, 64, 25600, 256, 64)), INVALID, "stride"),
    (dict(out=0x10000080), INVALID, "overlaps q"), (dict(s1=0x10000080), INVALID, "overlaps"),
    (dict(s0=0x50000000, s1=0x50000100), INVALID, "without being it"), (dict(s0=0x40000000), INVALID, "overlaps state_in"),
    (dict(N=100000, ws=None), WORKSPACE, "needs"), (dict(N=100000, wsb=100), WORKSPACE, "needs"),
    (dict(N=100000, ws=0x70000004), INVALID, "aligned"), (dict(N=100000, ws=0x20000000), INVALID, "overlaps"),
])
def test_prompt_refusals(kw, status, text):
    assert _fwd(**kw) == status
    assert text in fc.fftconv_last_error()


def test_prompt_with_nothing_to_do():
    assert _fwd(B=0) == 0 and _fwd(H=0, Hk=0) == 0 and _fwd(N=0, q=None, k=None, v=None, out=None) == 0
    assert fc.fftconv_last_error() == ""


def test_workspace_sizes():
    # few (sequence, head) pairs over a long sequence are cut into segments, many are not
    f = fc.fftconv_decay_fwd_workspace_bytes
    assert f(1, 17, 12, 64, 64, 1) == 0 and f(0, 17, 12, 64, 64, 1) == 0 and f(1, 17, 12, 64, 64, 9) == 0
    assert f(1, 131072, 20, 128, 128, 2) >= 20 * 128 * 128 * 4 * 2
    assert fc.fftconv_decay_bwd_workspace_bytes(1, 100, 4, 2, 64, 32, 2) >= 100 * 4 * 64 * 4   # shared heads' parts
    assert fc.fftconv_decay_bwd_workspace_bytes(1, 100, 4, 4, 64, 32, 2) == 0
    assert fc.fftconv_linear_fwd_workspace_bytes(1, 10240, 2560, 2) == 0
    assert fc.fftconv_linear_bwd_workspace_bytes(100, 64, 64, 2) >= 100 * 64 * 2
    assert fc.fftconv_linear_bwd_workspace_bytes(100, 64, 64, 9) == 0


def _step(**kw):
    a = dict(q=0x10000000, k=0x20000000, v=0x30000000, ld=0x1000, state=0x50000000, out=0x40000000, st=None, sl=None, ns=0,
             B=2, H=4, Hk=2, Dk=64, Dv=64, scale=1.0, dt=2)
    a.update(kw)
    return fc.lib().fftconv_decay_step(a["q"], a["k"], a["v"], a["ld"], a["state"], a["out"], a["st"], a["sl"], a["ns"],
                                       a["B"], a["H"], a["Hk"], a["Dk"], a["Dv"], a["scale"], a["dt"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dt=3), UNSUPPORTED, "dtype"), (dict(Hk=3), INVALID, "multiple"), (dict(Dk=300), UNSUPPORTED, "Dk=300"),
    (dict(state=None), INVALID, "state"), (dict(v=None), INVALID, "v must"), (dict(state=0x50000001), INVALID, "aligned"),
    (dict(out=0x50000100), INVALID, "overlaps"), (dict(state=0x10000040), INVALID, "overlaps"),
    (dict(st=_ints(256, 64, 128, 64, 128, 64, 256, 0)), INVALID, "share memory"), (dict(ns=-3), INVALID, "n_slots"),
])
def test_step_refusals(kw, status, text):
    assert _step(**kw) == status
    assert text in fc.fftconv_last_error()


def _bwd(**kw):
    a = dict(do=0x8000000, q=0x10000000, k=0x20000000, v=0x30000000, ld=0x1000, dq=0x40000000, dk=0x48000000, dv=0x50000000,
             st=None, s0=None, ds1=None, ds0=None, cu=None, B=1, N=100, H=4, Hk=2, Dk=64, Dv=64, scale=1.0, dt=2,
             ws=0x70000000, wsb=1 << 24)
    a.update(kw)
    return fc.lib().fftconv_decay_bwd(a["do"], a["q"], a["k"], a["v"], a["ld"], a["dq"], a["dk"], a["dv"], a["st"], a["s0"],
                                      a["ds1"], a["ds0"], a["cu"], a["B"], a["N"], a["H"], a["Hk"], a["Dk"], a["Dv"],
                                      a["scale"], a["dt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dt=3), UNSUPPORTED, "dtype"), (dict(do=None), INVALID, "dout must"), (dict(ld=None), INVALID, "log_decay"),
    (dict(dq=0x10000100), INVALID, "dq overlaps q"), (dict(dk=0x40000100), INVALID, "dk overlaps dq"),
    (dict(ds0=0x30000000), INVALID, "dstate_in overlaps"), (dict(ds1=0x8000, ds0=0x8000), INVALID, "overlaps dstate_out"),
    (dict(ws=None), WORKSPACE, "needs"), (dict(wsb=64), WORKSPACE, "needs"), (dict(ws=0x40000000), INVALID, "overlaps"),
])
def test_backward_refusals(kw, status, text):
    assert _bwd(**kw) == status
    assert text in fc.fftconv_last_error()


def _lin(**kw):
    a = dict(x=0x10000000, W=0x20000000, b=0x1000, r=0x30000000, out=0x40000000, pre=0x50000000, st=None, M=100, N=64, K=96,
             act=2, dt=2, ws=0x70000000, wsb=1 << 30)
    a.update(kw)
    return fc.lib().fftconv_linear_fwd(a["x"], a["W"], a["b"], a["r"], a["out"], a["pre"], a["st"], a["M"], a["N"], a["K"],
                                       a["act"], a["dt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dt=3), UNSUPPORTED, "dtype"), (dict(act=5), UNSUPPORTED, "activation"), (dict(act=-1), UNSUPPORTED, "activation"),
    (dict(M=-1), INVALID, "M=-1"), (dict(K=1 << 31), INVALID, "K="), (dict(x=None), INVALID, "x must"),
    (dict(W=None), INVALID, "W must"), (dict(out=None), INVALID, "out must"), (dict(out=0x40000001), INVALID, "aligned"),
    (dict(st=_ints(96, 96, 64, 32, 64)), INVALID, "share memory"), (dict(st=_ints(-96, 96, 64, 64, 64)), INVALID, "negative"),
    (dict(out=0x10000040), INVALID, "overlaps x"), (dict(pre=0x40000040), INVALID, "overlaps out"),
    (dict(r=0x40000080), INVALID, "without being it"), (dict(pre=0x30000040), INVALID, "overlaps residual"),
    (dict(M=128, N=128, K=8192, ws=None), WORKSPACE, "needs"), (dict(M=128, N=128, K=8192, wsb=8), WORKSPACE, "needs"),
])
def test_linear_refusals(kw, status, text):
    assert _lin(**kw) == status
    assert text in fc.fftconv_last_error()


def test_linear_with_nothing_to_do():
    assert _lin(M=0) == 0 and _lin(N=0, W=None, b=None) == 0


def _linb(**kw):
    a = dict(do=0x8000000, x=0x10000000, W=0x20000000, pre=0x30000000, dx=0x40000000, dW=0x48000000, db=0x50000000, st=None,
             M=100, N=64, K=96, act=2, dt=2, ws=0x70000000, wsb=1 << 30)
    a.update(kw)
    return fc.lib().fftconv_linear_bwd(a["do"], a["x"], a["W"], a["pre"], a["dx"], a["dW"], a["db"], a["st"], a["M"], a["N"],
                                       a["K"], a["act"], a["dt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dt=3), UNSUPPORTED, "dtype"), (dict(act=9), UNSUPPORTED, "activation"), (dict(pre=None), INVALID, "pre must"),
    (dict(x=None), INVALID, "x must"), (dict(W=None), INVALID, "W must"), (dict(do=None), INVALID, "dout must"),
    (dict(dx=0x8000040), INVALID, "dx overlaps dout"), (dict(dW=0x40000040), INVALID, "dW overlaps dx"),
    (dict(ws=None), WORKSPACE, "needs"), (dict(wsb=8), WORKSPACE, "needs"), (dict(ws=0x70000008), INVALID, "aligned"),
])
def test_linear_backward_refusals(kw, status, text):
    assert _linb(**kw) == status
    assert text in fc.fftconv_last_error()


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import torch
    t = torch.zeros((1, 4, 2, 8))
    with pytest.raises(ValueError, match="device"):
        fc.decay_attention(t, t, t, torch.zeros(2))
    with pytest.raises(ValueError, match="device"):
        fc.linear_act(torch.zeros(2, 3), torch.zeros(4, 3))


def test_refuses_launches_past_the_grid():
    # a launch holds fewer than 2^32 threads
    assert _fwd(B=1 << 22, N=1, H=4, Hk=4, Dk=1, Dv=1) == UNSUPPORTED and "too many" in fc.fftconv_last_error()
    assert _lin(M=1, N=1 << 28, K=1) == UNSUPPORTED and "too large" in fc.fftconv_last_error()
    assert _lin(M=1 << 30, N=1 << 20, K=8, ws=None) == UNSUPPORTED and "too large" in fc.fftconv_last_error()
    assert _linb(M=8, N=1 << 28, K=8) == UNSUPPORTED and "too large" in fc.fftconv_last_error()


def test_refuses_token_strides_past_a_chunk_offset():
    wide = 1 << 24      # elements of 2 bytes: 32 MiB
    st = _ints(0, wide, 64, 12800, 128, 64, 12800, 128, 64, 25600, 256, 64)
    assert _fwd(st=st) == UNSUPPORTED and "q has a token stride" in fc.fftconv_last_error()
