"""GPU parity of the root-mean-square norm (storage type and 8 bits, gradients) with its definition in float64 on the
rounded inputs.

Tolerances, with u the storage type's half unit in the last place (2^-24, 2^-11, 2^-8) relative to the value:
* sum: the fp32 sum of two values (exact to 2^-24) rounded once: u (1 + 2^-10) for 16 bits, 2 * 2^-24 for fp32, per element;
* out: squares summed in fp32 (relative error below 2^-24 times the additions of one thread, 64, and the steps of the
  tree, 10), a root and a division: below 40 * 2^-24 on the factor, three more roundings, then one of u: per element
  u (1 + 2^-6) for 16 bits (43 * 2^-24 is less than 2^-6 of 2^-11), 2^-18 for fp32;
* fp16 results below 2^-14 are subnormal, their steps 2^-24: half of one, 2^-25, whatever the value;
* rows read again (wide ones): one thread adds D / 256 squares, at most 400 here: 420 * 2^-24 / 2 < 2^-15 of the factor;
* 8 bits: scales 2^-15 relative; values half a step of e4m3, 2^-4 relative for normal numbers (from 2^-6) and half of
  2^-9 below, of a quotient with that error: 2^-4 + 2^-14;
* gradients, relative to the tensor's norm (their terms cancel): u for 16 bits and 2^-18 for what fp32 adds.
"""
import pytest
import torch

import long_fft_convolution_amd as fc

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
EPS = 1e-6


def _say(msg):
    print(f"[case] {msg}", flush=True)


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale).to(dtype)


def _norm64(t, w):
    y = t / (t.square().mean(-1, keepdim=True) + EPS).sqrt()
    return y if w is None else y * w


def _within(got, want, tol, name, least=0.0):
    got = got.double().cpu()
    off = (got - want).abs()
    bad = off > tol * want.abs() + least
    assert torch.isfinite(got).all() and not bad.any(), \
        f"{name}: {float((off / want.abs().clamp(min=1e-30))[bad].max()):.3e} off at {int(bad.sum())} places"


def _factor_tol(dtype, D):
    wide = 2.0 ** -15 if D > 8192 else 0.0
    return (2.0 ** -18 if dtype == "f32" else U[dtype] * (1 + 2.0 ** -6)) + wide


# one value, less and more than a piece, parts of a wave, odd widths (value by value), a wave, a workgroup, wider
WIDTHS = [1, 7, 8, 33, 64, 65, 128, 192, 256, 320, 768, 1000, 1001, 2560, 4096, 4104, 10240, 16384, 16392, 20001]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_rows(D, dtype):
    for M, residual, weighted in ((1, True, True), (3, False, True), (130, True, False)):
        _say(f"norm {dtype} {M} x {D} residual={residual} weight={weighted}")
        x = _rand((M, D), DT[dtype], D + M, 2.0)
        r = _rand((M, D), DT[dtype], D + M + 1, 3.0) if residual else None
        w = _rand((D,), DT[dtype], D + 2) if weighted else None
        got = fc.rms_norm(x.cuda(), None if w is None else w.cuda(), EPS, None if r is None else r.cuda())
        t = x.double() if r is None else x.double() + r.double()
        want = _norm64(t, None if w is None else w.double())
        # a sum that cancels has an error relative to its terms, not to itself
        least = 2.0 ** -24 * 20.0 if residual else 0.0
        if residual:
            _within(got[1], t, U[dtype] * (1 + 2.0 ** -10) + 2.0 ** -24, "sum", 1e-30)
            got = got[0]
        _within(got, want, _factor_tol(dtype, D), "out", least + (2.0 ** -25 if dtype == "f16" else 0.0))


def test_many_rows():
    # more rows than workgroups meet at once, and rows that leave the last workgroup part empty
    for M, D in ((16384 * 4 + 3, 512), (16384 * 16 * 2 + 5, 128), (2049, 1536), (16390, 2056)):
        _say(f"norm many rows {M} x {D}")
        x = torch.randn((M, D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(D)).to(torch.bfloat16)
        got = fc.rms_norm(x)
        want = _norm64(x.double(), None)
        assert ((got.double() - want).abs() <= _factor_tol("bf16", D) * want.abs()).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [1, 33, 64, 100, 128, 768, 2560, 5000, 16384, 16392, 20001])
def test_eight_bits(D, dtype):
    for M, residual in ((5, True), (2100, False)):
        if M * D > 1 << 24:
            M = 300
        _say(f"norm in 8 bits {dtype} {M} x {D}")
        x, w = _rand((M, D), DT[dtype], D, 2.0), _rand((D,), DT[dtype], 2)
        r = _rand((M, D), DT[dtype], 3) if residual else None
        out, scales, *rest = fc.rms_norm(x.cuda(), w.cuda(), EPS, None if r is None else r.cuda(), eight_bits=True)
        assert out.dtype == torch.float8_e4m3fn and scales.shape == (M,) and len(rest) == residual
        t = x.double() if r is None else x.double() + r.double()
        y = _norm64(t, w.double())
        want = y.abs().amax(-1) / 448
        _within(scales, want, 2.0 ** -15, "scales")
        v = y / scales.double().cpu()[:, None]
        _within(out.float(), v, 2.0 ** -4 + 2.0 ** -14, "8 bits", 2.0 ** -10 + 2.0 ** -14)
        assert float(out.float().abs().max()) == 448


def test_eight_bits_of_rows_without_values():
    # a zero row, one whose result lies below fp32's normal numbers, one with a NaN, one with an infinity
    x = torch.zeros((4, 256))
    x[1] = 1e-30
    x[2, 3] = float("nan")
    x[3, 5] = float("inf")
    w = torch.ones(256)
    for eps in (1e-6, 0.0):
        xs = x[1:] if eps == 0.0 else x
        out, scales = fc.rms_norm(xs.cuda(), w.cuda(), eps, eight_bits=True)
        out, scales = out.float().cpu(), scales.cpu()
        nan = 2 if eps else 1
        assert torch.isnan(scales[nan]) and torch.isnan(out[nan]).all()
        assert torch.isnan(out[nan + 1, 5])
        if eps:
            assert (out[0] == 0).all() and scales[0] == 2.0 ** -126
            assert torch.allclose(out[1] * scales[1], torch.full((256,), 1e-27), rtol=2.0 ** -4)


def _heads_of(M, H, D, dtype, seed):
    """(M, H, D) inside wider rows, as a projection leaves it."""
    wide = _rand((M, 3 * H * D), dtype, seed).cuda()
    return wide[:, H * D:2 * H * D].unflatten(1, (H, D)), wide


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,H,D", [(1, 1, 64), (5, 20, 128), (33, 12, 64), (7, 3, 33), (100, 2, 256), (4, 3, 20000)])
def test_heads_inside_rows(M, H, D, dtype):
    _say(f"norm of heads {dtype} {M} x {H} x {D}")
    x, wide = _heads_of(M, H, D, DT[dtype], 4)
    kept = wide.clone()
    want = _norm64(x.double().cpu(), None)
    least = 2.0 ** -25 if dtype == "f16" else 0.0
    _within(fc.rms_norm(x), want, _factor_tol(dtype, D), "out", least)
    # back into the rows' last third; nothing else of them changes
    into = wide[:, 2 * H * D:].unflatten(1, (H, D))
    fc.fftconv_norm_fwd(x, None, into, EPS)
    _within(into, want, _factor_tol(dtype, D), "out in place of the values", least)
    assert torch.equal(wide[:, :2 * H * D], kept[:, :2 * H * D])
    dy = _rand((M, H, D), DT[dtype], 8).cuda()
    dx, _ = fc.rms_norm_bwd(dy, x)
    wx, _ = _grads64(dy.double().cpu(), x.double().cpu(), None)
    _norm_close(dx, wx, dtype, "dx")


def test_sum_in_place():
    for D in (768, 20001):
        x, r = _rand((9, D), torch.bfloat16, 1).cuda(), _rand((9, D), torch.bfloat16, 2).cuda()
        out, total = fc.rms_norm(x, residual=r)
        out8, scales, _ = fc.rms_norm(x, residual=r, eight_bits=True)
        for place in (0, 1):
            a, b = x.clone(), r.clone()
            got = torch.empty_like(out)
            fc.fftconv_norm_fwd(a, None, got, EPS, residual=b, sum=(a, b)[place])
            assert torch.equal(got, out) and torch.equal((a, b)[place], total) and torch.equal((b, a)[place], (r, x)[place])
        b, got, s = r.clone(), torch.empty_like(out8), torch.empty_like(scales)
        fc.fftconv_norm_fwd(x, None, got, EPS, residual=b, sum=b, scales=s)
        assert torch.equal(got.view(torch.uint8), out8.view(torch.uint8)) and torch.equal(s, scales) and torch.equal(b, total)


def _grads64(dy, x, w, dsum=None):
    r = 1 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
    u = dy if w is None else dy * w
    dx = r * (u - x * r * r * (u * x).mean(-1, keepdim=True))
    return (dx if dsum is None else dx + dsum), (dy * x * r).flatten(0, -2).sum(0)


def _norm_close(got, want, dtype, name):
    off = float((got.double().cpu() - want).norm() / want.norm().clamp(min=1e-300))
    assert torch.isfinite(got).all() and off <= (U[dtype] if dtype != "f32" else 0.0) + 2.0 ** -18, f"{name}: {off:.3e}"


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", WIDTHS[1:])
def test_gradients(D, dtype):
    for M, more in ((1, False), (6, True), (1500, False)):
        if M * D > 1 << 23:
            M = 100
        _say(f"norm gradients {dtype} {M} x {D} dsum={more}")
        x, dy, w = _rand((M, D), DT[dtype], D, 2.0), _rand((M, D), DT[dtype], D + 1), _rand((D,), DT[dtype], D + 2)
        ds = _rand((M, D), DT[dtype], 4) if more else None
        dx, dw = fc.rms_norm_bwd(dy.cuda(), x.cuda(), w.cuda(), EPS, None if ds is None else ds.cuda())
        wx, ww = _grads64(dy.double(), x.double(), w.double(), None if ds is None else ds.double())
        _norm_close(dx, wx, dtype, "dx")
        _norm_close(dw, ww, dtype, "dweight")
        again = fc.rms_norm_bwd(dy.cuda(), x.cuda(), w.cuda(), EPS, None if ds is None else ds.cuda())
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_gradients_against_differences():
    # the fp32 forward's differences, h = 2^-6: third-order terms (h^2 / 6 of a value of size 1) and the roundings
    # (2^-22 of a sum of size 1, over h) both stay below 2^-10
    M, D, h = 3, 40, 2.0 ** -6
    x, dy, w = _rand((M, D), torch.float32, 1), _rand((M, D), torch.float32, 2), _rand((D,), torch.float32, 3)
    dx, dw = fc.rms_norm_bwd(dy.cuda(), x.cuda(), w.cuda())

    def loss(x, w):
        return float((fc.rms_norm(x.cuda(), w.cuda()).double().cpu() * dy.double()).sum())

    for i in (0, 7, 39):
        e = torch.zeros_like(x)
        e[1, i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - float(dx[1, i])) < 2.0 ** -10
        assert abs((loss(x, w + e[1]) - loss(x, w - e[1])) / (2 * h) - float(dw[i])) < 2.0 ** -10


def test_single_gradients_and_in_place():
    x, dy, w = (t.cuda() for t in (_rand((50, 768), torch.float16, 1), _rand((50, 768), torch.float16, 2), _rand((768,), torch.float16, 3)))
    ds = _rand((50, 768), torch.float16, 4).cuda()
    dx, dw = fc.rms_norm_bwd(dy, x, w, EPS, ds)
    ws = torch.empty(fc.fftconv_norm_bwd_workspace_bytes(50, 768), dtype=torch.uint8, device="cuda")
    only = torch.empty_like(dw)
    fc.fftconv_norm_bwd(dy, x, w, None, only, EPS, workspace=ws)
    assert torch.equal(only, dw)
    place = ds.clone()
    fc.fftconv_norm_bwd(dy, x, w, place, None, EPS, dsum=place, workspace=ws)
    assert torch.equal(place, dx)


def test_no_rows():
    w = _rand((64,), torch.float32, 1).cuda()
    x = torch.empty((0, 64), device="cuda")
    assert fc.rms_norm(x, w).shape == (0, 64)
    dx, dw = fc.rms_norm_bwd(x, x, w)
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros_like(w))


def test_graph_and_stream():
    x, w = _rand((64, 2560), torch.bfloat16, 1).cuda(), _rand((2560,), torch.bfloat16, 2).cuda()
    dy, r = _rand((64, 2560), torch.bfloat16, 3).cuda(), _rand((64, 2560), torch.bfloat16, 4).cuda()
    out, total, dx = (torch.empty_like(x) for _ in range(3))
    dw = torch.empty_like(w)
    ws = torch.empty(fc.fftconv_norm_bwd_workspace_bytes(64, 2560), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        fc.fftconv_norm_fwd(x, w, out, EPS, residual=r, sum=total)
        fc.fftconv_norm_bwd(dy, total, w, dx, dw, EPS, workspace=ws)
    for seed in range(3):
        x.copy_(_rand((64, 2560), torch.bfloat16, 10 + seed))
        for t in (out, total, dx, dw):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        want, wt = fc.rms_norm(x, w, EPS, r)
        wdx, wdw = fc.rms_norm_bwd(dy, wt, w, EPS)
        for a, b in ((out, want), (total, wt), (dx, wdx), (dw, wdw)):
            assert torch.equal(a, b)
    other = torch.cuda.Stream()
    got = fc.rms_norm(x, w, EPS, r, stream=other)
    other.synchronize()
    assert torch.equal(got[0], want)
