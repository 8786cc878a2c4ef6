"""The norm over more rows than a launch has workgroups, and at the row counts where the threads of a row change: against
float64 on the device, with the tolerances of the parity tests (one half unit of a 16-bit result and 2^-6 of it, e4m3
2^-4 and 2^-14, gradients one half unit of their norm and 2^-18 for fp32 steps)."""
import pytest
import torch

import long_fft_convolution_amd as fc

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _rows(M, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((M, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)] + [
        torch.randn((D,), generator=g, device="cuda").to(torch.bfloat16)]


@pytest.mark.parametrize("M,D", [(16500, 2560), (65600, 768), (600000, 24), (2048, 1000), (2049, 1000), (16400, 1100)])
def test_forward(M, D):
    print(f"[case] norm {M} x {D}", flush=True)
    x, res, w = _rows(M, D, M)
    out, total = fc.rms_norm(x, w, EPS, residual=res)
    small, scales, total8 = fc.rms_norm(x, w, EPS, residual=res, eight_bits=True)
    assert torch.equal(total, total8)
    for i in range(0, M, 16384):
        t = x[i:i + 16384].double() + res[i:i + 16384].double()
        assert ((total[i:i + 16384].double() - t).abs() <= 2.0 ** -8 * (1 + 2.0 ** -10) * t.abs()).all()
        y = t / (t.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
        assert ((out[i:i + 16384].double() - y).abs() <= 2.0 ** -8 * (1 + 2.0 ** -6) * y.abs()).all()
        s = scales[i:i + 16384].double()[:, None]
        assert ((s - y.abs().amax(-1, keepdim=True) / 448).abs() <= 2.0 ** -15 * s).all()
        z = small[i:i + 16384].float().double() * s
        assert ((z - y).abs() <= (2.0 ** -4 + 2.0 ** -14) * y.abs() + 2.0 ** -10 * s * (1 + 2.0 ** -4)).all()


@pytest.mark.parametrize("M,D", [(256, 768), (257, 768), (5000, 768), (5000, 129), (1600, 4096), (1600, 2560), (600, 2568), (70000, 24)])
def test_gradients(M, D):
    print(f"[case] norm gradients {M} x {D}", flush=True)
    x, dy, w = _rows(M, D, M + 1)
    ds = x.flip(0).contiguous()
    dx, dw = fc.rms_norm_bwd(dy, x, w, EPS, dsum=ds)
    t, g = x.double(), dy.double()
    r = 1 / (t.square().mean(-1, keepdim=True) + EPS).sqrt()
    u = g * w.double()
    want = r * (u - t * r * r * (u * t).mean(-1, keepdim=True)) + ds.double()
    for got, ref in ((dx, want), (dw, (g * t * r).sum(0))):
        assert float((got.double() - ref).norm()) <= (2.0 ** -8 + 2.0 ** -18) * float(ref.norm())
    again = fc.rms_norm_bwd(dy, x, w, EPS, dsum=ds)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
