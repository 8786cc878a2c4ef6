"""C-ABI and binding checks of the root-mean-square norm that need no GPU: every case fails validation or has nothing to do."""
import ctypes

import pytest
import torch

fc = pytest.importorskip("long_fft_convolution_amd")

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def _ints(*v):
    return (ctypes.c_int64 * len(v))(*v)


def _fwd(**kw):
    a = dict(x=0x10000000, r=None, w=None, out=0x20000000, sum=None, sc=None, st=None, M=100, G=4, D=64, eps=1e-6, dt=2)
    a.update(kw)
    return fc.lib().fftconv_norm_fwd(a["x"], a["r"], a["w"], a["out"], a["sum"], a["sc"], a["st"], a["M"], a["G"], a["D"],
                                     a["eps"], a["dt"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dt=9), UNSUPPORTED, "dtype"), (dict(M=-1), INVALID, "M=-1"), (dict(G=-2), INVALID, "G=-2"),
    (dict(D=0), UNSUPPORTED, "D=0"), (dict(D=(1 << 20) + 1), UNSUPPORTED, "D="), (dict(M=1 << 31, G=1), UNSUPPORTED, "rows"),
    (dict(M=1 << 20, G=1 << 11), UNSUPPORTED, "rows"), (dict(eps=-1.0), INVALID, "eps"), (dict(eps=float("nan")), INVALID, "eps"),
    (dict(x=None), INVALID, "x must"), (dict(out=None), INVALID, "out must"), (dict(x=0x10000001), INVALID, "aligned"),
    (dict(w=0x30000001), INVALID, "weight must be aligned"), (dict(sc=0x30000002), INVALID, "scales must be aligned"),
    (dict(out=0x10000040), INVALID, "overlaps x"), (dict(out=0x10000000), INVALID, "overlaps x"),
    (dict(r=0x30000000, out=0x30000000), INVALID, "overlaps residual"), (dict(w=0x20000000), INVALID, "out overlaps weight"),
    (dict(r=0x30000000, sum=0x30000080), INVALID, "sum overlaps residual"), (dict(sum=0x10000080), INVALID, "sum overlaps x"),
    (dict(sum=0x20000000), INVALID, "sum overlaps out"), (dict(sc=0x20000000), INVALID, "scales overlaps out"),
    (dict(st=_ints(256, -64, 0, 0, 256, 64, 0, 0)), INVALID, "negative"),
    (dict(st=_ints(256, 64, 0, 0, 256, 0, 0, 0)), INVALID, "share memory"),
    # in place with another stride
    (dict(r=0x30000000, sum=0x30000000, st=_ints(256, 64, 512, 64, 256, 64, 256, 64)), INVALID, "sum overlaps residual"),
])
def test_forward_refusals(kw, status, text):
    assert _fwd(**kw) == status
    assert text in fc.fftconv_last_error()


def test_nothing_to_do():
    assert _fwd(M=0) == 0 and _fwd(G=0) == 0 and _fwd(M=0, x=None, out=None) == 0


def _bwd(**kw):
    a = dict(dy=0x10000000, x=0x20000000, w=None, ds=None, dx=0x30000000, dw=0x40000000, st=None, M=100, G=4, D=64, eps=1e-6,
             dt=2, ws=0x70000000, wsb=1 << 30)
    a.update(kw)
    return fc.lib().fftconv_norm_bwd(a["dy"], a["x"], a["w"], a["ds"], a["dx"], a["dw"], a["st"], a["M"], a["G"], a["D"],
                                     a["eps"], a["dt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dt=-1), UNSUPPORTED, "dtype"), (dict(M=-1), INVALID, "M=-1"), (dict(D=0), UNSUPPORTED, "D=0"),
    (dict(dy=None), INVALID, "dout must"), (dict(x=None), INVALID, "x must"), (dict(ds=0x50000001), INVALID, "aligned"),
    (dict(ws=None), WORKSPACE, "needs"), (dict(wsb=64), WORKSPACE, "needs"), (dict(ws=0x70000004), INVALID, "aligned"),
    (dict(ws=0x20000000), INVALID, "overlaps"), (dict(dx=0x20000000), INVALID, "dx overlaps x"),
    (dict(dx=0x10000000), INVALID, "dx overlaps dout"), (dict(ds=0x30000080), INVALID, "dx overlaps dsum"),
    (dict(dw=0x30000000), INVALID, "dweight overlaps dx"), (dict(ds=0x40000000), INVALID, "dweight overlaps dsum"),
])
def test_backward_refusals(kw, status, text):
    assert _bwd(**kw) == status
    assert text in fc.fftconv_last_error()


def test_workspace_sizes():
    f = fc.fftconv_norm_bwd_workspace_bytes
    assert f(0, 64) == 0 and f(10, 0) == 0 and f(10, (1 << 20) + 1) == 0 and f(1 << 31, 64) == 0
    assert f(3, 64) == 768 + 24 and f(100000, 64) == 512 * 64 * 4 + 800000


def test_rows_of_views():
    base = torch.zeros(4, 6, 5, 8)
    g = fc._row_groups
    assert g((4, 6, 5, 8), (base, None)) == (120, 1, 8, None)
    wide = torch.zeros(4, 6, 15, 8)[:, :, 5:10]
    M, G, D, st = g(wide.shape, (wide, base, None, None))
    assert (M, G, D, list(st)) == (24, 5, 8, [120, 8, 40, 8, 0, 0, 0, 0])
    steps = torch.zeros(4, 1, 5, 16)[..., :8]
    M, G, D, st = g(steps.shape, (steps, None, None, None))
    assert M * G == 20 and st[1] == 16 and (M == 1 or st[0] == 80)
    with pytest.raises(ValueError, match="fold"):
        g((4, 6, 5, 8), (torch.zeros(4, 7, 15, 8)[:, :6, 5:10], base, None, None))


def test_binding_refuses_host_tensors():
    x = torch.zeros(3, 64)
    with pytest.raises(ValueError, match="device tensor"):
        fc.rms_norm(x, torch.ones(64))
    with pytest.raises(ValueError, match="device tensor"):
        fc.rms_norm_bwd(x, x)
