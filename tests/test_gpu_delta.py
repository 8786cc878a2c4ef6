"""GPU parity of the gated delta rule (prompts, gradients, single tokens) with the float64 oracle on the rounded inputs.

Tolerances, relative L2 per tensor, with u the storage type's half unit in the last place (2^-24, 2^-11, 2^-8):
* results in 16 bits: the result's rounding (u) and, in bf16, that of the products q k^T (another u; 2^-16 in fp16),
  in quadrature below sqrt(2) u, and terms of 2^-16: 1.5 u;
* fp32 results (states, gates' gradients, fp32 storage): products of exact terms accumulated in fp32.  A chunk of 64
  tokens adds sums of at most 256 products (64 half units at worst, a few in the mean), the inverse's and the update's
  chains of 64 more, over at most 40 chunks whose errors the decay forgets or which add like a random walk (6 times
  that of one): 5e-6, which is 84 half units.
A tensor whose oracle value is zero must be zero.
"""
import numpy as np
import pytest
import torch

import long_fft_convolution_amd as fc
from oracle import sequence as seq

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TOL = {"f32": 5e-6, "f16": 1.5 * 2.0 ** -11, "bf16": 1.5 * 2.0 ** -8}
FP32 = 5e-6


def _say(msg):
    print(f"[case] {msg}", flush=True)


def _close(got, want, tol, name):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, name
    assert np.isfinite(got).all(), name
    norm = np.linalg.norm(want)
    err = np.linalg.norm(got - want)
    assert err <= tol * norm, f"{name}: relL2 {err / max(norm, 1e-300):.3e} > {tol:.1e}"


def _rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale).to(dtype)


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _inputs(lead, H, Hk, Dk, Dv, dtype, seed):
    """q, k (of norm 1), v, log_decay, beta; heads that do not decay and that forget at once among them."""
    dt = DT[dtype]
    k = _rand((*lead, Hk, Dk), torch.float64, seed + 1)
    k = (k / k.norm(dim=-1, keepdim=True).clamp(min=1e-6)).to(dt)
    g = torch.Generator().manual_seed(seed + 77)
    rate = torch.exp(torch.rand(H, generator=g) * np.log(1e3) + np.log(1e-4))
    if H > 2:
        rate[0], rate[1] = 0.0, 20.0
    a = -rate * torch.rand((*lead, H), generator=g)
    beta = torch.rand((*lead, H), generator=g) * 1.5
    return _rand((*lead, Hk, Dk), dt, seed), k, _rand((*lead, H, Dv), dt, seed + 2), a.float(), beta.float()


def _gpu(*ts):
    return [None if t is None else t.cuda() for t in ts]


PROMPTS = [
    # B, N, H, Hk, Dk, Dv: one token, a chunk less and more one, odd widths, wide and uneven heads, segments
    (1, 1, 1, 1, 64, 64), (2, 17, 3, 3, 64, 64), (1, 63, 2, 1, 64, 128), (2, 64, 4, 2, 128, 64), (1, 65, 3, 1, 128, 128),
    (3, 130, 2, 2, 40, 72), (1, 200, 1, 1, 7, 5), (1, 129, 2, 2, 96, 33), (1, 150, 2, 1, 256, 200), (2, 97, 1, 1, 160, 256),
    (1, 1030, 3, 3, 64, 64), (1, 2100, 2, 1, 128, 128), (1, 2307, 2, 2, 33, 65), (1, 2049, 1, 1, 256, 72),
    (70, 66, 3, 3, 64, 128), (44, 70, 3, 3, 128, 136),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("B,N,H,Hk,Dk,Dv", PROMPTS)
def test_prompt(B, N, H, Hk, Dk, Dv, dtype):
    _say(f"prompt {dtype} B={B} N={N} H={H}/{Hk} Dk={Dk} Dv={Dv}")
    ins = _inputs((B, N), H, Hk, Dk, Dv, dtype, N + H)
    S0 = _rand((B, H, Dk, Dv), torch.float32, 5) if N % 2 else None
    out, S = fc.delta_attention(*_gpu(*ins), scale=0.25, state_in=None if S0 is None else S0.cuda())
    for b in range(0, B, max(1, B // 3)):
        want, ws = seq.delta_fwd(*(_f64(t[b]) for t in ins), 0.25, None if S0 is None else _f64(S0[b]))
        _close(out[b], want, TOL[dtype], f"out[{b}]")
        _close(S[b], ws, FP32, f"state[{b}]")


NAMES = ("dq", "dk", "dv", "dlog_decay", "dbeta")


def _grads_close(got, want, dtype, where):
    for name, x, y in zip(NAMES, got, want):
        # 16 bits: the result's own rounding, everything before it is fp32
        _close(x, y, FP32 if x.dtype == torch.float32 else TOL[dtype], f"{name}{where}")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("B,N,H,Hk,Dk,Dv", PROMPTS)
def test_gradients(B, N, H, Hk, Dk, Dv, dtype):
    _say(f"gradients {dtype} B={B} N={N} H={H}/{Hk} Dk={Dk} Dv={Dv}")
    ins = _inputs((B, N), H, Hk, Dk, Dv, dtype, N + H)
    dout = _rand((B, N, H, Dv), DT[dtype], 9)
    S0, dS = (_rand((B, H, Dk, Dv), torch.float32, s) if N % 2 else None for s in (5, 6))
    got = fc.delta_attention_bwd(*_gpu(*ins, dout), scale=0.25, state_in=None if S0 is None else S0.cuda(),
                                 dstate_out=None if dS is None else dS.cuda())
    for b in range(0, B, max(1, B // 3)):
        want = seq.delta_bwd(_f64(dout[b]), *(_f64(t[b]) for t in ins), 0.25, None if S0 is None else _f64(S0[b]),
                             None if dS is None else _f64(dS[b]))
        _grads_close([t[b] for t in got[:5]], want, dtype, f"[{b}]")
        if S0 is not None:
            _close(got[5][b], want[5], FP32, f"dstate_in[{b}]")


LENGTHS = [(0,), (1,), (0, 1, 63, 64, 65, 0), (5, 700, 0, 300, 1), (0, 0, 0), tuple(range(1, 40)), (300,) + (1,) * 300,
           (2500, 3)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("lens", LENGTHS)
def test_packed(lens, dtype):
    _say(f"packed {dtype} lengths {str(lens)[:60]}")
    H, Hk, Dk, Dv, B, T = 4, 2, 64, 96, len(lens), sum(lens)
    if T == 2503:
        H, Hk, Dk, Dv = 1, 1, 128, 64
    lead, behind = 3, 2          # tokens of no sequence around them
    ins = _inputs((lead + T + behind,), H, Hk, Dk, Dv, dtype, T)
    ends = lead + np.concatenate([[0], np.cumsum(lens)])
    cu = torch.tensor(ends, dtype=torch.int32).cuda()
    S0 = _rand((B, H, Dk, Dv), torch.float32, 5)
    q, k, v, a, beta = _gpu(*ins)
    out = torch.full_like(v, 7.0)
    S = torch.empty((B, H, Dk, Dv), device="cuda")
    ws = torch.empty(max(1, fc.fftconv_delta_fwd_workspace_bytes(B, lead + T + behind, H, Hk, Dk, Dv, q.dtype)), dtype=torch.uint8,
                     device="cuda")
    fc.fftconv_delta_fwd(q, k, v, a, beta, out, 0.25, S0.cuda(), S, cu_seqlens=cu, workspace=ws)
    assert (out[:lead] == 7).all() and (out[lead + T:] == 7).all()
    for b, (x, y) in enumerate(zip(ends, ends[1:])):
        if b > 12 and b < B - 2:
            continue
        want, ws_ = seq.delta_fwd(*(_f64(t[x:y]) for t in ins), 0.25, _f64(S0[b]))
        _close(out[x:y], want, TOL[dtype], f"out[{b}]")
        _close(S[b], ws_, FP32, f"state[{b}]")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("lens", LENGTHS)
def test_packed_gradients(lens, dtype):
    _say(f"packed gradients {dtype} lengths {str(lens)[:60]}")
    H, Hk, Dk, Dv, B, T = 4, 2, 64, 96, len(lens), sum(lens)
    lead, behind = 3, 2
    ins = _inputs((lead + T + behind,), H, Hk, Dk, Dv, dtype, T)
    ends = lead + np.concatenate([[0], np.cumsum(lens)])
    cu = torch.tensor(ends, dtype=torch.int32).cuda()
    S0, dS = _rand((B, H, Dk, Dv), torch.float32, 5), _rand((B, H, Dk, Dv), torch.float32, 6)
    dout = _rand(ins[2].shape, DT[dtype], 9)
    q, k, v, a, beta, do = _gpu(*ins, dout)
    grads = [torch.full_like(t, 7.0) for t in (q, k, v, a, beta)]
    dS0 = torch.empty((B, H, Dk, Dv), device="cuda")
    ws = torch.empty(max(1, fc.fftconv_delta_bwd_workspace_bytes(B, lead + T + behind, H, Hk, Dk, Dv, q.dtype)), dtype=torch.uint8,
                     device="cuda")
    fc.fftconv_delta_bwd(do, q, k, v, a, beta, *grads, 0.25, S0.cuda(), dS.cuda(), dS0, cu, ws)
    for t in grads:
        assert (t[:lead] == 7).all() and (t[lead + T:] == 7).all()
    for b, (x, y) in enumerate(zip(ends, ends[1:])):
        if b > 12 and b < B - 2:
            continue
        want = seq.delta_bwd(_f64(dout[x:y]), *(_f64(t[x:y]) for t in ins), 0.25, _f64(S0[b]), _f64(dS[b]))
        _grads_close([t[x:y] for t in grads], want, dtype, f"[{b}]")
        _close(dS0[b], want[5], FP32, f"dstate_in[{b}]")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,Dk,Dv", [(1, 1, 1, 64, 64), (3, 4, 2, 128, 128), (2, 3, 3, 40, 72), (5, 2, 1, 33, 65), (2, 2, 2, 256, 200),
                                          (1, 1, 1, 5, 3), (130, 4, 4, 128, 128), (90, 4, 2, 200, 256), (200, 3, 3, 64, 64)])
def test_step(B, H, Hk, Dk, Dv, dtype):
    _say(f"step {dtype} B={B} H={H}/{Hk} Dk={Dk} Dv={Dv}")
    ins = _inputs((B,), H, Hk, Dk, Dv, dtype, B + H)
    n = B + 4
    pool = _rand((n, H, Dk, Dv), torch.float32, 3)
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, n
    q, k, v, a, beta = _gpu(*ins)
    state, out = pool.cuda(), torch.full((B, H, Dv), 9.0, dtype=DT[dtype], device="cuda")
    fc.fftconv_delta_step(q, k, v, a, beta, state, out, 0.25, slots.cuda())
    got, kept = state.cpu(), set(range(n))
    for b in range(B):
        s = int(slots[b])
        if not 0 <= s < n:
            assert (out[b] == 0).all()
            continue
        kept.discard(s)
        want, ws = seq.delta_fwd(*(_f64(t[b:b + 1]) for t in ins), 0.25, _f64(pool[s]))
        _close(out[b:b + 1], want, TOL[dtype], f"out[{b}]")
        _close(got[s], ws, FP32, f"state[{b}]")
    for s in kept:
        assert torch.equal(got[s], pool[s])


def test_tokens_after_a_prompt():
    """The prompt form, and the last tokens by themselves from the state that the rest leaves."""
    B, N, H, Hk, D = 3, 200, 4, 2, 64
    q, k, v, a, beta = _gpu(*_inputs((B, N), H, Hk, D, D, "bf16", 4))
    out, S = fc.delta_attention(q, k, v, a, beta)
    _, part = fc.delta_attention(*(t[:, :N - 3].contiguous() for t in (q, k, v, a, beta)))
    got = torch.empty((B, H, D), dtype=q.dtype, device="cuda")
    for t in range(N - 3, N):
        fc.fftconv_delta_step(q[:, t], k[:, t], v[:, t], a[:, t].contiguous(), beta[:, t].contiguous(), part, got, D ** -0.5)
        # one rounding each and one of the products on the prompt's side: sqrt(3) u
        _close(got, out[:, t].double().cpu().numpy(), 2 * 2.0 ** -8, f"token {t}")
    _close(part, S.double().cpu().numpy(), FP32, "state")
