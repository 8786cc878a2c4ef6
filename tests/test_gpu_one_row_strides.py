"""Strides of dimensions that hold one element lead nowhere: sequences of one token and matrices of one row whose views
carry any nominal stride there (as a transposed (1, B, F) tensor does) give the results of dense ones, bit for bit."""
import pytest
import torch

import long_fft_convolution_amd as fc

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _rand(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype]).cuda()


def _nominal(t, dim, stride):
    """The same view with another stride along a dimension of one element."""
    assert t.shape[dim] == 1
    strides = list(t.stride())
    strides[dim] = stride
    return t.as_strided(t.shape, strides)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("H,Hk,D", [(4, 4, 64), (4, 2, 64), (2, 1, 40), (1, 1, 33)])
@pytest.mark.parametrize("stride", [1 << 26, 1 << 27, (1 << 36) + 8, 7])
def test_sequences_of_one_token(stride, H, Hk, D, dtype):
    print(f"[case] one token {dtype} H={H}/{Hk} D={D} stride {stride}", flush=True)
    B, F = 3, H + 2 * Hk
    a = torch.full((H,), -0.1, device="cuda")
    qkv, dout = _rand((B, 1, F, D), dtype, 1), _rand((B, 1, 2 * H, D), dtype, 2)[:, :, :H]
    parts = [slice(0, H), slice(H, H + Hk), slice(H + Hk, F)]
    q, k, v = (qkv[:, :, p] for p in parts)
    want, want_S = fc.decay_attention(q, k, v, a, 0.5)
    want_g = fc.decay_attention_bwd(q, k, v, a, dout, 0.5)
    far = [_nominal(t, 1, stride) for t in (q, k, v, dout)]
    out, S = fc.decay_attention(*far[:3], a, 0.5)
    assert torch.equal(out, want) and torch.equal(S, want_S)
    outs = [torch.full((B, 1, 2 * n, D), 5.0, dtype=DT[dtype], device="cuda") for n in (H, Hk, Hk)]
    grads = [_nominal(o[:, :, :o.shape[2] // 2], 1, stride) for o in outs]
    ws = torch.empty(max(16, fc.fftconv_decay_bwd_workspace_bytes(B, B, H, Hk, D, D, DT[dtype])), dtype=torch.uint8, device="cuda")
    fc.fftconv_decay_bwd(far[3], *far[:3], a, *grads, 0.5, workspace=ws)
    for g, w in zip(grads, want_g):
        assert torch.equal(g, w)
    assert all((o[:, :, o.shape[2] // 2:] == 5.0).all() for o in outs)


def test_packed_buffer_of_one_token():
    H, D = 2, 64
    a, cu = torch.full((H,), -0.1, device="cuda"), torch.tensor([0, 0, 1, 1], dtype=torch.int32, device="cuda")
    qkv = _rand((1, 3 * H, D), "bf16", 1)
    q, k, v = qkv[:, :H], qkv[:, H:2 * H], qkv[:, 2 * H:]
    dout = _rand((1, H, D), "bf16", 2)
    want = fc.decay_attention_bwd(q, k, v, a, dout, cu_seqlens=cu)[:3]
    # one dimension that is not dense makes the binding pass every stride
    heads = [_rand((1, 2 * H, D), "bf16", 3)[:, ::2] for _ in range(3)]
    for h, t in zip(heads, (q, k, v)):
        h.copy_(t)
    got = fc.decay_attention_bwd(*(_nominal(t, 0, 1 << 27) for t in heads), a, dout, cu_seqlens=cu)[:3]
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_products_of_one_row(dtype):
    K, N = 96, 72
    x, W, r, d = _rand((1, K), dtype, 1), _rand((N, 2 * K), dtype, 2)[:, :K], _rand((1, N), dtype, 3), _rand((1, N), dtype, 4)
    want = fc.linear_act(x, W, None, r, "gelu")
    want_g = fc.linear_act_bwd(d, x, W, bias=False)
    out = r.clone()         # the residual updated in place, its two views with nominal strides of their own
    ws = lambda f: torch.empty(max(16, f(1, N, K, DT[dtype])), dtype=torch.uint8, device="cuda")
    fc.fftconv_linear_fwd(_nominal(x, 0, 1 << 33), W, None, _nominal(out, 0, 5), _nominal(out, 0, 1 << 30), None, "gelu",
                          ws(fc.fftconv_linear_fwd_workspace_bytes))
    assert torch.equal(out, want)
    dx, dW = torch.empty_like(x), torch.empty((N, K), dtype=DT[dtype], device="cuda")
    fc.fftconv_linear_bwd(_nominal(d, 0, 1 << 33), _nominal(x, 0, 1 << 34), W, None, _nominal(dx, 0, 3), dW, None, "none",
                          ws(fc.fftconv_linear_bwd_workspace_bytes))
    assert torch.equal(dx, want_g[0]) and torch.equal(dW, want_g[1])
