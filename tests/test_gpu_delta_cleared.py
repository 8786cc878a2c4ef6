"""Gated delta rule behind tokens that clear the state.

Tolerances, relative L2 against the float64 oracle on the rounded inputs: 16-bit results 1.5 half units of their type (2^-11,
2^-8), fp32 results 5e-6 (products of exact terms accumulated in fp32 over at most 40 chunks of 64 tokens)."""
import numpy as np
import pytest
import torch

import long_fft_convolution_amd as fc
from oracle import sequence as seq

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TOL = {"f32": 5e-6, "f16": 1.5 * 2.0 ** -11, "bf16": 1.5 * 2.0 ** -8}
FP32 = 5e-6
CLEAR = [float("-inf"), -200.0, -105.0]


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _close(got, want, tol, name):
    got = _f64(got)
    assert got.shape == want.shape and np.isfinite(got).all(), name
    err, norm = np.linalg.norm(got - want), np.linalg.norm(want)
    assert err <= tol * norm, f"{name}: relL2 {err / max(norm, 1e-300):.3e} > {tol:.1e}"


def _inputs(lead, H, Hk, Dk, Dv, dtype, seed):
    """q, k (of norm 1), v, log_decay, beta on the GPU."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    k = r(*lead, Hk, Dk)
    k = k / k.norm(dim=-1, keepdim=True)
    a = -torch.exp(r(*lead, H) - 3)
    return [t.to(d).cuda() for t, d in ((r(*lead, Hk, Dk), DT[dtype]), (k, DT[dtype]), (r(*lead, H, Dv), DT[dtype]),
                                        (a, torch.float32), (torch.sigmoid(r(*lead, H)), torch.float32))]


def _spoilt(*shape):
    """States with what a slot may hold from before: NaN, infinities, the largest values."""
    S = torch.randn(shape, generator=torch.Generator().manual_seed(2))
    flat = S.view(-1)
    flat[::7], flat[1::7], flat[2::7], flat[3::7] = float("nan"), float("inf"), float("-inf"), torch.finfo(torch.float32).max
    return S.cuda()


@pytest.mark.parametrize("clear", CLEAR)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,N,H,Dk,Dv", [(2, 1, 2, 64, 64), (2, 130, 2, 40, 72), (1, 2100, 2, 128, 64)])
def test_a_first_token_clears_a_spoilt_state(B, N, H, Dk, Dv, dtype, clear):
    """Prompt (cut at 2100 tokens) and gradients equal those without a state; the state's own gradient is zero."""
    print(f"[case] cleared {dtype} B={B} N={N} H={H} {Dk} {Dv} by {clear}", flush=True)
    ins = _inputs((B, N), H, H, Dk, Dv, dtype, N)
    ins[3][:, 0] = clear
    S0, dout = _spoilt(B, H, Dk, Dv), torch.randn((B, N, H, Dv), device="cuda").to(DT[dtype])
    out, S = fc.delta_attention(*ins, state_in=S0)
    none = fc.delta_attention(*ins)
    assert torch.equal(out, none[0]) and torch.equal(S, none[1])
    want, wS = seq.delta_fwd(*(_f64(t[0]) for t in ins), Dk ** -0.5)
    _close(out[0], want, TOL[dtype], "out")
    _close(S[0], wS, FP32, "state")
    grads, plain = fc.delta_attention_bwd(*ins, dout, state_in=S0), fc.delta_attention_bwd(*ins, dout)
    for x, y in zip(grads[:5], plain[:5]):
        assert torch.equal(x, y)
    assert (grads[5] == 0).all()


@pytest.mark.parametrize("clear", CLEAR)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,Dk,Dv", [(3, 128, 128), (2, 33, 65), (1, 256, 40)])
def test_a_token_clears_a_spoilt_slot(H, Dk, Dv, dtype, clear):
    B, n = 4, 6
    q, k, v, a, beta = _inputs((B,), H, H, Dk, Dv, dtype, 5)
    a[1:] = clear
    pool = _spoilt(n, H, Dk, Dv)
    pool[4] = torch.randn((H, Dk, Dv), generator=torch.Generator().manual_seed(9)).cuda()
    kept, slots = pool.clone(), [4, 0, 5, 2]
    out = torch.empty((B, H, Dv), dtype=DT[dtype], device="cuda")
    fc.fftconv_delta_step(q, k, v, a, beta, pool, out, 0.25, torch.tensor(slots, dtype=torch.int32, device="cuda"))
    for b, s in enumerate(slots):
        want, wS = seq.delta_fwd(*(_f64(t[b:b + 1]) for t in (q, k, v, a, beta)), 0.25, _f64(kept[s]) if b == 0 else None)
        _close(out[b:b + 1], want, TOL[dtype], f"out[{b}]")
        _close(pool[s], wS, FP32, f"state[{b}]")
    for s in (1, 3):
        assert torch.equal(pool[s].view(torch.int32), kept[s].view(torch.int32))


@pytest.mark.parametrize("lens", [(0, 5, 200, 1, 0), (0, 2600, 0, 2500, 2100, 70)])
def test_packed_sequences_keep_or_clear_each_their_own_state(lens):
    """Odd sequences start with a token that clears a spoilt state; an empty one passes on what it got, whatever it is."""
    B, T, H, D, lead = len(lens), sum(lens), 2, 64, 3
    ends = lead + np.concatenate([[0], np.cumsum(lens)])
    cu = torch.tensor(ends, dtype=torch.int32).cuda()
    ins = _inputs((lead + T,), H, H, D, D, "bf16", T)
    S0 = torch.randn((B, H, D, D), generator=torch.Generator().manual_seed(8)).cuda()
    for b in range(B):
        if b % 2 or lens[b] == 0:
            S0[b] = _spoilt(H, D, D)
        if b % 2 and lens[b]:
            ins[3][ends[b]] = float("-inf")
    out, S = fc.delta_attention(*ins, scale=0.25, state_in=S0, cu_seqlens=cu)
    for b, (x, y) in enumerate(zip(ends, ends[1:])):
        if x == y:
            assert torch.equal(S[b].view(torch.int32), S0[b].view(torch.int32))
            continue
        want, wS = seq.delta_fwd(*(_f64(t[x:y]) for t in ins), 0.25, None if b % 2 else _f64(S0[b]))
        _close(out[x:y], want, TOL["bf16"], f"out[{b}]")
        _close(S[b], wS, FP32, f"state[{b}]")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_gradients_of_decays_of_any_size(dtype):
    """Each head, from one that forgets nothing to one that forgets all, by itself.

    dlog_decay_t is formed as the sum over the tokens i >= t of t's block of 64 of q_i dq_i - v_i dv_i and of <G, S> behind the
    block.  Its terms are fp32 values from products of exact terms, each off by at most 5e-6 of the sum of its products'
    magnitudes (the tolerance of fp32 results), and so is the whole of the sum of all those.  A token that clears the state has
    the gradient 0."""
    N, H, D, scale = 200, 7, 64, 0.3
    ins = _inputs((1, N), H, H, D, D, dtype, 21)
    a = ins[3]
    for h, x in enumerate([0.0, -1e-3, -2.0, -12.0, -40.0, -100.0]):
        a[..., h] = x
    a[..., 6] = -0.1
    a[0, ::9, 6], a[0, 4::9, 6], a[0, 7::9, 6] = CLEAR
    dout = torch.randn((1, N, H, D), generator=torch.Generator().manual_seed(3)).cuda().to(DT[dtype])
    S0, dS = (torch.randn((1, H, D, D), generator=torch.Generator().manual_seed(s)).cuda() for s in (4, 5))
    got = _f64(fc.delta_attention_bwd(*ins, dout, scale=scale, state_in=S0, dstate_out=dS)[3][0])
    q, k, v, g, b, do = (_f64(t[0]) for t in (*ins, dout))
    want = seq.delta_bwd(do, q, k, v, g, b, scale, _f64(S0[0]), _f64(dS[0]))
    each = np.abs(q * want[0]).sum(-1) + np.abs(v * want[2]).sum(-1)
    S = _f64(S0[0])
    for t0 in range(0, N, 64):
        t1 = min(N, t0 + 64)
        S = seq.delta_fwd(*(t[t0:t1] for t in (q, k, v, g, b)), scale, S)[1]
        G = seq.delta_bwd(*(t[t1:] for t in (do, q, k, v, g, b)), scale, S, _f64(dS[0]))[5] if t1 < N else _f64(dS[0])
        terms = each[t0:t1][::-1].cumsum(0)[::-1] + np.abs(G * S).sum((1, 2))
        off = np.abs(got[t0:t1] - want[3][t0:t1]) / terms
        assert off.max() <= FP32, f"{off.max():.2e} at token, head {np.unravel_index(off.argmax(), off.shape)} of {t0}"
    cleared = _f64(a[0]) < -104
    assert cleared[:, 6].sum() > 60 and not cleared[:, :6].any() and (got[cleared] == 0).all()
