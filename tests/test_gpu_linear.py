"""GPU parity of the linear product (bias, activation, residual; gradients) with the float64 oracle on the rounded inputs.

Tolerances, relative L2 per tensor, with u the storage type's half unit in the last place (2^-24, 2^-11, 2^-8):
results are rounded once from fp32 sums (u), gradients meet dz rounded as well (sqrt(2) u): 2 u for fp16 and bf16.
fp32: sums of up to K terms in fp32, relative error at most about sqrt(K) 2^-24 of the terms' norm: 5e-6 at K <= 4096.
"""
import sys

import numpy as np
import pytest
import torch

import long_fft_convolution_amd as fc
from oracle import sequence as seq

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TOL = {"f32": 5e-6, "f16": 2 * 2.0 ** -11, "bf16": 2 * 2.0 ** -8}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def _say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale).to(dtype)


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _cuda(t):
    return None if t is None else t.cuda()


def _close(got, want, tol, name):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape and np.isfinite(got).all(), name
    norm, err = np.linalg.norm(want), np.linalg.norm(got - want)
    assert err <= tol * norm, f"{name}: relL2 {err / max(norm, 1e-300):.3e} > {tol:.1e}"


SIZES = [
    # M, N, K: the few-rows kernel, its edges, odd sizes, every tile, split products, K below and above a step
    (1, 1, 1), (1, 48, 64), (1, 1000, 2560), (3, 17, 33), (16, 64, 96), (17, 65, 64), (33, 256, 512), (64, 128, 7),
    (65, 64, 64), (65, 33, 31), (100, 200, 72), (128, 128, 2048), (300, 77, 130), (130, 2304, 768), (513, 257, 65),
    (512, 6400, 64), (200, 100, 4096), (1111, 999, 333), (4000, 3400, 40),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward(M, N, K, dtype):
    act = ACTS[(M + N + K) % 5]
    bias, res = (M + N) % 3 != 0, (M + K) % 2 == 0
    _say(f"linear {dtype} {M}x{N}x{K} {act} bias={bias} residual={res}")
    x, W = _rand((M, K), DT[dtype], 1), _rand((N, K), DT[dtype], 2, K ** -0.5)
    b = _rand((N,), DT[dtype], 3) if bias else None
    r = _rand((M, N), DT[dtype], 4) if res else None
    out, pre = fc.linear_act(x.cuda(), W.cuda(), _cuda(b), _cuda(r), act, keep_pre=True)
    want, want_pre = seq.linear_fwd(_f64(x), _f64(W), _f64(b), _f64(r), act)
    _close(out, want, TOL[dtype], "out")
    _close(pre, want_pre, TOL[dtype], "pre")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gradients(M, N, K, dtype):
    act = ACTS[(M + N + 2 * K) % 5]
    _say(f"linear gradients {dtype} {M}x{N}x{K} {act}")
    x, W, dout = _rand((M, K), DT[dtype], 1), _rand((N, K), DT[dtype], 2), _rand((M, N), DT[dtype], 3)
    pre = None if act == "none" else _rand((M, N), DT[dtype], 4, 2.0)
    got = fc.linear_act_bwd(dout.cuda(), x.cuda(), W.cuda(), _cuda(pre), act)
    for name, g, w in zip(("dx", "dW", "dbias"), got, seq.linear_bwd(_f64(dout), _f64(x), _f64(W), _f64(pre), act)):
        _close(g, w, TOL[dtype], name)


@pytest.mark.parametrize("act", ACTS)
def test_activations_each(act):
    x, W = _rand((70, 64), torch.float32, 1, 3.0), _rand((96, 64), torch.float32, 2)
    b, dout = _rand((96,), torch.float32, 3), _rand((70, 96), torch.float32, 4)
    out, pre = fc.linear_act(x.cuda(), W.cuda(), b.cuda(), None, act, keep_pre=True)
    want, want_pre = seq.linear_fwd(_f64(x), _f64(W), _f64(b), None, act)
    _close(out, want, TOL["f32"], "out")
    got = fc.linear_act_bwd(dout.cuda(), x.cuda(), W.cuda(), pre, act)
    for name, g, w in zip(("dx", "dW", "dbias"), got, seq.linear_bwd(_f64(dout), _f64(x), _f64(W), _f64(pre), act)):
        _close(g, w, TOL["f32"], name)


@pytest.mark.parametrize("act", ACTS)
def test_activations_at_large_arguments(act):
    # identity product: out = act(x); no overflow on the way to act's limits, slopes 0 and 1
    z = torch.tensor([[-3e38, -1e20, -1e4, -100.0, 0.0, 100.0, 1e4, 1e20]])
    x = torch.cat([z, z.flip(1)])
    out = fc.linear_act(x.cuda(), torch.eye(8).cuda(), None, None, act)
    np.testing.assert_allclose(_f64(out), _f64(x) if act == "none" else np.maximum(_f64(x), 0), rtol=1e-6, atol=1e-30)
    if act != "none":
        dx, _, db = fc.linear_act_bwd(torch.ones_like(x).cuda(), x.cuda(), torch.eye(8).cuda(), x.cuda(), act)
        want = seq.act_slope(np.clip(_f64(x), -1e4, 1e4), act)
        np.testing.assert_allclose(_f64(dx), want, rtol=1e-6, atol=1e-30)


def test_empty_sizes():
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")
    assert fc.linear_act(e(0, 8), e(4, 8)).shape == (0, 4)
    b, r = _rand((4,), torch.bfloat16, 1).cuda(), _rand((3, 4), torch.bfloat16, 2).cuda()
    assert torch.equal(fc.linear_act(e(3, 0), e(4, 0), b, r), (b.float() + r.float()).to(torch.bfloat16))
    out = fc.linear_act(e(100, 0), e(4, 0), b)
    assert torch.equal(out, b.expand(100, 4))
    dx, dW, db = fc.linear_act_bwd(e(0, 4), e(0, 8), e(4, 8))
    assert dx.shape == (0, 8) and (dW == 0).all() and (db == 0).all()
    dx, dW, db = fc.linear_act_bwd(e(5, 0), e(5, 8), e(0, 8))
    assert (dx == 0).all() and dW.shape == (0, 8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_and_in_place(dtype):
    # column blocks of wider matrices, rows at odd addresses, the residual updated in place
    dt = DT[dtype]
    for M, off, wide in ((5, 0, 200), (5, 3, 201), (300, 8, 208), (300, 1, 203)):
        _say(f"strided {dtype} M={M} offset {off} of {wide}")
        K, N = 96, 72
        big = [_rand((rows, wide), dt, s).cuda() for s, rows in enumerate((M, N, M, M, M))]
        x, W, r, dout, pre = (t[:, off:off + w] for t, w in zip(big, (K, K, N, N, N)))
        want, _ = seq.linear_fwd(_f64(x), _f64(W), None, _f64(r), "gelu")
        ws = lambda f: torch.empty(max(1, f(M, N, K, dt)), dtype=torch.uint8, device="cuda")
        grads = [torch.zeros((n, wide), dtype=dt, device="cuda") for n in (M, N)]
        dx, dW = (g[:, off:off + K] for g in grads)
        fc.fftconv_linear_bwd(dout, x, W, pre, dx, dW, None, "silu", ws(fc.fftconv_linear_bwd_workspace_bytes))
        for g, w in zip((dx, dW), seq.linear_bwd(_f64(dout), _f64(x), _f64(W), _f64(pre), "silu")):
            _close(g, w, TOL[dtype], "gradient")
        assert all((g[:, :off] == 0).all() and (g[:, off + K:] == 0).all() for g in grads)
        edges = big[2].clone()
        fc.fftconv_linear_fwd(x, W, None, r, r, None, "gelu", ws(fc.fftconv_linear_fwd_workspace_bytes))
        _close(r, want, TOL[dtype], "in place")
        assert torch.equal(big[2][:, :off], edges[:, :off]) and torch.equal(big[2][:, off + N:], edges[:, off + N:])


def test_rows_past_the_edge_do_not_leak():
    # NaN outside the operands (neighbouring rows and columns) never reaches a result
    dt = torch.bfloat16
    M, N, K = 200, 90, 72
    x = torch.full((M + 60, K + 8), float("nan"), dtype=dt, device="cuda")
    W = torch.full((N + 60, K + 8), float("nan"), dtype=dt, device="cuda")
    dout = torch.full((M + 60, N + 6), float("nan"), dtype=dt, device="cuda")
    x[:M, :K], W[:N, :K], dout[:M, :N] = 1.0, 2.0, 1.0
    out = fc.linear_act(x[:M, :K], W[:N, :K])
    assert (out == 2.0 * K).all()
    dx, dW, db = fc.linear_act_bwd(dout[:M, :N], x[:M, :K], W[:N, :K])
    assert (dx == 2.0 * N).all() and (dW == M).all() and (db == M).all()
    one = fc.linear_act(x[:1, :K], W[:N, :K])
    assert (one == 2.0 * K).all()


def test_repeatable_and_on_another_stream():
    x, W = _rand((300, 4096), torch.bfloat16, 1).cuda(), _rand((100, 4096), torch.bfloat16, 2).cuda()
    a = fc.linear_act(x, W)                 # a split product: joined in a fixed order
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = fc.linear_act(x, W)
    s.synchronize()
    assert torch.equal(a, b)


WHOLE_AND_SPLIT = [
    # more tiles than compute units with a rest that is split along K, of each tile width; rows of the few-rows kernel
    (1000, 2304, 768), (4100, 4400, 640), (1030, 9000, 260), (2, 333, 4095), (4, 50, 31), (4, 1030, 768),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K", WHOLE_AND_SPLIT)
def test_whole_and_split_tiles(M, N, K, dtype):
    test_forward(M, N, K, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,apart", [(80, 1 << 26), (4200, 1 << 20)])      # bytes
def test_rows_past_four_gibibytes(M, apart, dtype):
    N, K, ld = 72, 96, apart // (2 if dtype == "bf16" else 4)
    _say(f"linear {dtype}, {M} rows {ld} elements apart")
    x, W, d = _rand((M, K), DT[dtype], 1), _rand((N, K), DT[dtype], 2, 0.1), _rand((M, N), DT[dtype], 3)
    xv, dv, ov = (torch.empty((M, ld), dtype=DT[dtype], device="cuda")[:, :n] for n in (K, N, N))
    xv.copy_(x), dv.copy_(d)
    fc.fftconv_linear_fwd(xv, W.cuda(), None, None, ov, None, "none",
                          torch.empty(max(1, fc.fftconv_linear_fwd_workspace_bytes(M, N, K, DT[dtype])), dtype=torch.uint8,
                                      device="cuda"))
    _close(ov, seq.linear_fwd(_f64(x), _f64(W), None, None, "none")[0], TOL[dtype], "out")
    dx, dW, db = fc.linear_act_bwd(dv, xv, W.cuda())
    for name, got, want in zip(("dx", "dW", "dbias"), (dx, dW, db), seq.linear_bwd(_f64(d), _f64(x), _f64(W), None, "none")):
        _close(got, want, TOL[dtype], name)


def test_graph_replays_equal_eager_calls():
    M, N, K = 200, 300, 2048
    x, W, b = (_rand(s, torch.bfloat16, i, 0.1).cuda() for i, s in enumerate(((M, K), (N, K), (N,))))
    d = _rand((M, N), torch.bfloat16, 9).cuda()
    out, pre = fc.linear_act(x, W, b, None, "gelu", keep_pre=True)      # loads the kernels
    grads = fc.linear_act_bwd(d, x, W, pre, "gelu")
    size = max(fc.fftconv_linear_fwd_workspace_bytes(M, N, K, x.dtype), fc.fftconv_linear_bwd_workspace_bytes(M, N, K, x.dtype))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fc.fftconv_linear_fwd(x, W, b, None, out, pre, "gelu", ws)
        fc.fftconv_linear_bwd(d, x, W, pre, *grads, "gelu", ws)
    for seed in (20, 21, 22):
        x.copy_(_rand((M, K), torch.bfloat16, seed, 0.1))
        graph.replay()
        torch.cuda.synchronize()
        want, want_pre = fc.linear_act(x, W, b, None, "gelu", keep_pre=True)
        assert torch.equal(out, want) and torch.equal(pre, want_pre)
        for got, w in zip(grads, fc.linear_act_bwd(d, x, W, want_pre, "gelu")):
            assert torch.equal(got, w)
