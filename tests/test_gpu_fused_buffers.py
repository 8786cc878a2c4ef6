"""Results written beside other tensors of the call into one buffer: dq, dk and dv as blocks of a fused buffer, outputs as
column blocks of a matrix that also holds inputs.  Results equal those of separate tensors bit for bit, everything
else in the buffer stays."""
import pytest
import torch

import long_fft_convolution_amd as fc

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _rand(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype]).cuda()


def _scratch(nbytes):
    return torch.empty(max(16, nbytes), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk,D", [(4, 4, 64), (4, 2, 64), (3, 1, 40)])
@pytest.mark.parametrize("packed", [False, True])
def test_gradients_in_one_buffer(packed, H, Hk, D, dtype):
    lead = (330,) if packed else (2, 165)
    cu = torch.tensor([0, 100, 330], dtype=torch.int32, device="cuda") if packed else None
    F = H + 2 * Hk
    qkv = _rand((*lead, F + 1, D), dtype, 1)                    # inputs as views of one buffer, too
    q, k, v = qkv[..., :H, :], qkv[..., H:H + Hk, :], qkv[..., H + Hk:F, :]
    dout, a = _rand((*lead, H, D), dtype, 2), torch.full((H,), -0.01, device="cuda")
    want = fc.decay_attention_bwd(q, k, v, a, dout, 0.2, cu_seqlens=cu)
    buf = torch.full((*lead, F + 1, D), 5.0, dtype=DT[dtype], device="cuda")
    parts = buf[..., :H, :], buf[..., H:H + Hk, :], buf[..., H + Hk:F, :]
    ws = _scratch(fc.fftconv_decay_bwd_workspace_bytes(2, 330, H, Hk, D, D, DT[dtype]))
    fc.fftconv_decay_bwd(dout, q, k, v, a, *parts, 0.2, cu_seqlens=cu, workspace=ws)
    for name, got, w in zip(("dq", "dk", "dv"), parts, want):
        assert torch.equal(got, w), name
    assert (buf[..., F, :] == 5.0).all()


def test_heads_in_turn():
    # q, k, v, out of each head side by side, for a prompt and for single tokens
    B, N, H, D = 2, 100, 3, 64
    buf = _rand((B, N, H, 4, D), "f16", 3)
    q, k, v, out = (buf[..., i, :] for i in range(4))
    a = torch.full((H,), -0.01, device="cuda")
    before = buf.clone()
    want, _ = fc.decay_attention(q, k, v, a, 0.2)
    fc.fftconv_decay_fwd(q, k, v, a, out, 0.2, workspace=_scratch(fc.fftconv_decay_fwd_workspace_bytes(B, B * N, H, D, D, q.dtype)))
    assert torch.equal(out, want) and torch.equal(buf[..., :3, :], before[..., :3, :])
    tokens = [t[:, 7] for t in (q, k, v, out)]
    state, want_state = torch.zeros((B, H, D, D), device="cuda"), torch.zeros((B, H, D, D), device="cuda")
    want = torch.empty((B, H, D), dtype=torch.float16, device="cuda")
    fc.fftconv_decay_step(*tokens[:3], a, want_state, want, 0.2)
    fc.fftconv_decay_step(*tokens[:3], a, state, tokens[3], 0.2)
    assert torch.equal(tokens[3], want) and torch.equal(state, want_state)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", [(3, 96, 72), (200, 96, 72), (130, 33, 31)])
def test_product_beside_its_input(M, K, N, dtype):
    W, b = _rand((N, K), dtype, 1), _rand((N,), dtype, 2)
    buf = _rand((M, K + 3 * N + 1), dtype, 3)
    before = buf.clone()
    x, r, out, pre = buf[:, :K], buf[:, K:K + N], buf[:, K + N:K + 2 * N], buf[:, K + 2 * N:K + 3 * N]
    want, want_pre = fc.linear_act(x, W, b, r, "silu", keep_pre=True)
    fc.fftconv_linear_fwd(x, W, b, r, out, pre, "silu", _scratch(fc.fftconv_linear_fwd_workspace_bytes(M, N, K, DT[dtype])))
    assert torch.equal(out, want) and torch.equal(pre, want_pre)
    assert torch.equal(buf[:, :K + N], before[:, :K + N]) and torch.equal(buf[:, -1], before[:, -1])
    d = _rand((M, N), dtype, 4)
    want = fc.linear_act_bwd(d, x, W, pre, "silu")
    buf2 = torch.full((M, K + 2 * N), 3.0, dtype=DT[dtype], device="cuda")
    dx, dout, p = buf2[:, :K], buf2[:, K:K + N], buf2[:, K + N:]
    dout.copy_(d), p.copy_(pre)
    dW, db = torch.empty_like(W), torch.empty_like(b)
    fc.fftconv_linear_bwd(dout, x, W, p, dx, dW, db, "silu", _scratch(fc.fftconv_linear_bwd_workspace_bytes(M, N, K, DT[dtype])))
    assert all(torch.equal(g, w) for g, w in zip((dx, dW, db), want))
    assert torch.equal(dout, d) and torch.equal(p, pre)
