"""GPU parity of decay attention (prompt form, gradients, single tokens) with the float64 oracle on the rounded inputs.

Tolerances, relative L2 per tensor, with u the storage type's half unit in the last place (2^-24, 2^-11, 2^-8):
* results in the storage type: three independent roundings of at most u each meet in them (the products q k^T, the
  state, the result; the kernels accumulate in fp32), sqrt(3) u < 2 u; gradients of shared heads add fp32 terms
  and round once more, the same bound;
* fp32 results (states, fp32 storage): 5e-6, which is 84 half units: exp of a product rounded in fp32 and chains of
  up to 64-token sums, each a few half units, over at most 40 chunks.
A tensor whose oracle value is zero must be zero.
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
STATE_TOL = 5e-6


def _say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


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
    return t.double().cpu().numpy()


def _decays(H, seed):
    g = torch.Generator().manual_seed(seed + 77)
    a = -torch.exp(torch.rand(H, generator=g) * np.log(1e3) + np.log(1e-4))
    if H > 2:
        a[0] = 0.0                  # no decay
        a[1] = -30.0                # forgets at once
    return a.float()


def _inputs(lead, H, Hk, Dk, Dv, dtype, seed):
    dt = DT[dtype]
    return (_rand((*lead, H, Dk), dt, seed), _rand((*lead, Hk, Dk), dt, seed + 1), _rand((*lead, Hk, Dv), dt, seed + 2),
            _decays(H, seed))


def _gpu(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _sequences(lens):
    ends = np.concatenate([[0], np.cumsum(lens)])
    return [(int(a), int(b)) for a, b in zip(ends, ends[1:])]


PROMPTS = [
    # B, N, H, Hk, Dk, Dv: one token, a chunk less and more one, odd widths, wide and uneven heads, segments
    (1, 1, 1, 1, 64, 64), (2, 17, 3, 3, 64, 64), (1, 63, 2, 1, 64, 128), (2, 64, 4, 2, 128, 64), (1, 65, 3, 1, 128, 128),
    (3, 130, 2, 2, 40, 72), (1, 200, 1, 1, 7, 5), (1, 129, 2, 2, 96, 33), (1, 150, 2, 1, 256, 200), (2, 97, 1, 1, 160, 256),
    (1, 1030, 3, 3, 64, 64), (1, 2100, 2, 1, 128, 128),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("B,N,H,Hk,Dk,Dv", PROMPTS)
def test_prompt(B, N, H, Hk, Dk, Dv, dtype):
    _say(f"prompt {dtype} B={B} N={N} H={H}/{Hk} Dk={Dk} Dv={Dv}")
    q, k, v, a = _inputs((B, N), H, Hk, Dk, Dv, dtype, N + H)
    S0 = _rand((B, H, Dk, Dv), torch.float32, 5) if N % 2 else None
    out, S = fc.decay_attention(*_gpu(q, k, v, a), scale=0.25, state_in=None if S0 is None else S0.cuda())
    for b in range(B):
        want, ws = seq.decay_fwd(_f64(q[b]), _f64(k[b]), _f64(v[b]), _f64(a), 0.25, None if S0 is None else _f64(S0[b]))
        _close(out[b], want, TOL[dtype], f"out[{b}]")
        _close(S[b], ws, STATE_TOL, f"state[{b}]")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("B,N,H,Hk,Dk,Dv", PROMPTS)
def test_gradients(B, N, H, Hk, Dk, Dv, dtype):
    _say(f"gradients {dtype} B={B} N={N} H={H}/{Hk} Dk={Dk} Dv={Dv}")
    q, k, v, a = _inputs((B, N), H, Hk, Dk, Dv, dtype, N + H)
    dout = _rand((B, N, H, Dv), DT[dtype], 9)
    S0, dS = (_rand((B, H, Dk, Dv), torch.float32, s) if N % 2 else None for s in (5, 6))
    got = fc.decay_attention_bwd(*_gpu(q, k, v, a, dout), scale=0.25, state_in=None if S0 is None else S0.cuda(),
                                 dstate_out=None if dS is None else dS.cuda())
    for b in range(B):
        want = seq.decay_bwd(_f64(dout[b]), _f64(q[b]), _f64(k[b]), _f64(v[b]), _f64(a), 0.25,
                             None if S0 is None else _f64(S0[b]), None if dS is None else _f64(dS[b]))
        for name, x, y in zip(("dq", "dk", "dv"), got, want):
            _close(x[b], y, TOL[dtype], f"{name}[{b}]")
        if S0 is not None:
            _close(got[3][b], want[3], STATE_TOL, f"dstate_in[{b}]")


LENGTHS = [(0,), (1,), (0, 1, 63, 64, 65, 0), (5, 700, 0, 300, 1), (0, 0, 0), tuple(range(1, 40)), (300,) + (1,) * 300]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("lens", LENGTHS)
def test_packed(lens, dtype):
    _say(f"packed {dtype} lengths {str(lens)[:60]}")
    H, Hk, Dk, Dv, B, T = 4, 2, 64, 96, len(lens), sum(lens)
    q, k, v, a = _inputs((T,), H, Hk, Dk, Dv, dtype, 3)
    dout = _rand((T, H, Dv), DT[dtype], 9)
    S0, dS = (_rand((B, H, Dk, Dv), torch.float32, s) for s in (5, 6))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    qg, kg, vg, ag, dg, S0g, dSg = _gpu(q, k, v, a, dout, S0, dS)
    out, S = fc.decay_attention(qg, kg, vg, ag, scale=0.2, state_in=S0g, cu_seqlens=cu)
    grads = fc.decay_attention_bwd(qg, kg, vg, ag, dg, scale=0.2, state_in=S0g, dstate_out=dSg, cu_seqlens=cu)
    for b, (i, j) in enumerate(_sequences(lens)):
        part = [_f64(t[i:j]) for t in (q, k, v)]
        want, ws = seq.decay_fwd(*part, _f64(a), 0.2, _f64(S0[b]))
        _close(out[i:j], want, TOL[dtype], f"out[{b}]")
        _close(S[b], ws, STATE_TOL, f"state[{b}]")
        want = seq.decay_bwd(_f64(dout[i:j]), *part, _f64(a), 0.2, _f64(S0[b]), _f64(dS[b]))
        for name, x, y in zip(("dq", "dk", "dv"), grads, want):
            _close(x[i:j], y, TOL[dtype], f"{name}[{b}]")
        _close(grads[3][b], want[3], STATE_TOL, f"dstate_in[{b}]")


def test_packed_neighbours_and_gaps_are_apart():
    # NaN in one sequence stays there; tokens of no sequence are not written; bounds past the end are clamped
    T, H, D = 300, 2, 64
    q, k, v, a = _inputs((T,), H, H, D, D, "bf16", 8)
    bad = v.clone()
    bad[100:170] = float("nan")
    cu = torch.tensor([10, 100, 170, 9999], dtype=torch.int32).cuda()
    qg, kg, vg, bg, ag = _gpu(q, k, v, bad, a)
    outs = []
    for val in (vg, bg):
        out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        fc.fftconv_decay_fwd(qg, kg, val, ag, out, 0.1, cu_seqlens=cu, workspace=torch.empty(
            fc.fftconv_decay_fwd_workspace_bytes(3, T, H, D, D, torch.bfloat16), dtype=torch.uint8, device="cuda"))
        outs.append(out)
    good, withnan = outs
    assert (good[:10] == 7.0).all() and (withnan[:10] == 7.0).all()
    assert torch.equal(good[10:100], withnan[10:100]) and torch.equal(good[170:], withnan[170:])
    assert withnan[100:170].isnan().all()
    want, _ = seq.decay_fwd(*(_f64(t[170:]) for t in (q, k, v)), _f64(a), 0.1)
    _close(good[170:], want, TOL["bf16"], "last sequence")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,Dk,Dv", [(1, 1, 1, 64, 64), (3, 4, 2, 128, 128), (2, 3, 1, 7, 5), (70, 8, 8, 64, 128),
                                          (2, 2, 2, 256, 250), (5, 2, 1, 33, 256)])
def test_tokens_one_by_one(B, H, Hk, Dk, Dv, dtype):
    # three single-token steps on a pool with slots in any order, two of them padding
    _say(f"step {dtype} B={B} H={H}/{Hk} Dk={Dk} Dv={Dv}")
    q, k, v, a = _inputs((3, B), H, Hk, Dk, Dv, dtype, B)
    n_slots = B + 3
    pool = _rand((n_slots, H, Dk, Dv), torch.float32, 6)
    slots = torch.randperm(n_slots, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, n_slots
    state, sg, ag = pool.cuda(), slots.cuda(), a.cuda()
    outs = []
    for t in range(3):
        out = torch.full((B, H, Dv), float("nan"), dtype=DT[dtype], device="cuda")
        fc.fftconv_decay_step(*_gpu(q[t], k[t], v[t]), ag, state, out, 0.3, sg)
        outs.append(out)
    want_pool = _f64(pool)
    for b in range(B):
        s = int(slots[b])
        if not 0 <= s < n_slots:
            assert all((o[b] == 0).all() for o in outs)
            continue
        want, want_pool[s] = seq.decay_fwd(*(_f64(t[:, b]) for t in (q, k, v)), _f64(a), 0.3, _f64(pool[s]))
        for t in range(3):
            _close(outs[t][b], want[t], TOL[dtype], f"out[{b}] of token {t}")
    _close(state, want_pool, STATE_TOL, "pool")


def test_prompt_then_tokens_is_the_longer_prompt():
    # prompt in two parts through a pool, then single tokens: the oracle of the whole sequence
    H, Hk, D, N = 3, 1, 64, 150
    q, k, v, a = _inputs((1, N), H, Hk, D, D, "f16", 4)
    pool = torch.zeros((4, H, D, D), device="cuda")
    slot = torch.tensor([2], dtype=torch.int32, device="cuda")
    qg, kg, vg, ag = _gpu(q, k, v, a)
    out = torch.empty((1, N, H, D), dtype=torch.float16, device="cuda")
    for i, j in ((0, 70), (70, 147)):
        fc.fftconv_decay_fwd(qg[:, i:j], kg[:, i:j], vg[:, i:j], ag, out[:, i:j], 0.125, pool, pool, slot)
    for t in range(147, N):
        fc.fftconv_decay_step(qg[:, t], kg[:, t], vg[:, t], ag, pool, out[:, t], 0.125, slot)
    want, S = seq.decay_fwd(*(_f64(t[0]) for t in (q, k, v)), _f64(a), 0.125)
    _close(out[0], want, TOL["f16"], "out")
    _close(pool[2], S, STATE_TOL, "state")
    assert (pool[[0, 1, 3]] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_views(dtype):
    # q, k, v as views of one projection's output, heads first in memory, rows at odd addresses, broadcast k
    B, N, H, D = 2, 90, 3, 64
    a = _decays(H, 1).cuda()
    qkv = _rand((B, N, 3, H, D), DT[dtype], 2).cuda()
    odd = torch.empty((B * H * N * (D + 1) + 1,), dtype=DT[dtype], device="cuda")[1:].view(B, H, N, D + 1)[..., :D]
    odd.copy_(qkv[:, :, 0].transpose(1, 2))
    shared = qkv[:1, :, 1].expand(B, N, H, D)
    for name, q, k, v in (("fused", qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]),
                          ("odd", odd.transpose(1, 2), qkv[:, :, 1], qkv[:, :, 2]),
                          ("broadcast", qkv[:, :, 0], shared, qkv[:, :, 2])):
        _say(f"strided {name} {dtype}")
        store = torch.zeros((B, H, N, D + 1), dtype=DT[dtype], device="cuda")
        out = store[..., :D].transpose(1, 2)
        fc.fftconv_decay_fwd(q, k, v, a, out, 0.2)
        grads = fc.decay_attention_bwd(q, k, v, a, out, scale=0.2)
        assert (store[..., D] == 0).all()
        for b in range(B):
            x = [_f64(t[b]) for t in (q, k, v)]
            _close(out[b], seq.decay_fwd(*x, _f64(a), 0.2)[0], TOL[dtype], f"{name} out")
            for n, g, w in zip(("dq", "dk", "dv"), grads, seq.decay_bwd(_f64(out[b]), *x, _f64(a), 0.2)):
                _close(g[b], w, TOL[dtype], f"{name} {n}")


def test_decay_of_minus_infinity_and_zero_scale():
    q, k, v, _ = _inputs((1, 70), 2, 2, 64, 64, "bf16", 1)
    a = torch.tensor([float("-inf"), 0.0])
    qg, kg, vg, ag = _gpu(q, k, v, a)
    out, S = fc.decay_attention(qg, kg, vg, ag, scale=0.5)
    want, ws = seq.decay_fwd(*(_f64(t[0]) for t in (q, k, v)), _f64(a), 0.5)
    _close(out[0], want, TOL["bf16"], "out")
    _close(S[0], ws, STATE_TOL, "state")
    dS = _rand((1, 2, 64, 64), torch.float32, 3)
    got = fc.decay_attention_bwd(qg, kg, vg, ag, torch.ones_like(qg), scale=0.0, state_in=torch.zeros_like(dS).cuda(),
                                 dstate_out=dS.cuda())
    want = seq.decay_bwd(np.ones((70, 2, 64)), *(_f64(t[0]) for t in (q, k, v)), _f64(a), 0.0, None, _f64(dS[0]))
    for n, g, w in zip(("dq", "dk", "dv"), got, want):
        _close(g[0], w, TOL["bf16"], n)
    _close(got[3][0], want[3], STATE_TOL, "dstate_in")


def test_single_gradients_equal_the_joint_call():
    q, k, v, a = _inputs((2, 300), 4, 2, 64, 64, "bf16", 1)
    dout = _rand((2, 300, 4, 64), torch.bfloat16, 2)
    qg, kg, vg, ag, dg = _gpu(q, k, v, a, dout)
    S0, dS = (_rand((2, 4, 64, 64), torch.float32, s).cuda() for s in (3, 4))
    ws = torch.empty(fc.fftconv_decay_bwd_workspace_bytes(2, 600, 4, 2, 64, 64, torch.bfloat16), dtype=torch.uint8,
                     device="cuda")
    all_four = fc.decay_attention_bwd(qg, kg, vg, ag, dg, 0.2, S0, dS)
    for i in range(4):
        want = [torch.full_like(t, 5.0) if j == i else None for j, t in enumerate(all_four)]
        fc.fftconv_decay_bwd(dg, qg, kg, vg, ag, *want[:3], 0.2, S0, dS, want[3], workspace=ws)
        assert torch.equal(want[i], all_four[i]), i


def test_another_stream_and_graph_replay():
    B, N, H, D = 1, 1500, 2, 64
    q, k, v, a = _inputs((B, N), H, H, D, D, "bf16", 1)
    qg, kg, vg, ag = _gpu(q, k, v, a)
    want, want_S = fc.decay_attention(qg, kg, vg, ag, scale=0.2)
    out, S = torch.zeros_like(want), torch.zeros_like(want_S)
    ws = torch.empty(max(1, fc.fftconv_decay_fwd_workspace_bytes(B, N, H, D, D, torch.bfloat16)), dtype=torch.uint8,
                     device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    fc.fftconv_decay_fwd(qg, kg, vg, ag, out, 0.2, None, S, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(S, want_S)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fc.fftconv_decay_fwd(qg, kg, vg, ag, out, 0.2, None, S, workspace=ws)
    for seed in (5, 6, 7):
        vg.copy_(_rand((B, N, H, D), torch.bfloat16, seed))
        graph.replay()
        torch.cuda.synchronize()
        want, want_S = fc.decay_attention(qg, kg, vg, ag, scale=0.2)
        assert torch.equal(out, want) and torch.equal(S, want_S)


@pytest.mark.parametrize("H,Hk,Dk,Dv", [(1, 1, 128, 128), (2, 1, 72, 40), (1, 1, 200, 136)])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_packed_in_segments_of_several_parts(H, Hk, Dk, Dv, dtype):
    lens = (1500, 0, 1000, 64)
    _say(f"packed in segments {dtype} H={H}/{Hk} Dk={Dk} Dv={Dv}")
    B, T = len(lens), sum(lens)
    q, k, v, a = _inputs((T,), H, Hk, Dk, Dv, dtype, 11)
    a[0] = -0.003
    dout = _rand((T, H, Dv), DT[dtype], 9)
    S0, dS = (_rand((B, H, Dk, Dv), torch.float32, s) for s in (5, 6))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()
    qg, kg, vg, ag, dg, S0g, dSg = _gpu(q, k, v, a, dout, S0, dS)
    out, S = fc.decay_attention(qg, kg, vg, ag, scale=0.2, state_in=S0g, cu_seqlens=cu)
    grads = fc.decay_attention_bwd(qg, kg, vg, ag, dg, scale=0.2, state_in=S0g, dstate_out=dSg, cu_seqlens=cu)
    want, want_S = np.zeros(out.shape), np.zeros(S.shape)
    want_g = [np.zeros(g.shape) for g in grads]
    for b, (i, j) in enumerate(_sequences(lens)):
        part = [_f64(t[i:j]) for t in (q, k, v)]
        want[i:j], want_S[b] = seq.decay_fwd(*part, _f64(a), 0.2, _f64(S0[b]))
        g = seq.decay_bwd(_f64(dout[i:j]), *part, _f64(a), 0.2, _f64(S0[b]), _f64(dS[b]))
        for n in range(3):
            want_g[n][i:j] = g[n]
        want_g[3][b] = g[3]
    _close(out, want, TOL[dtype], "out")
    _close(S, want_S, STATE_TOL, "state")
    for name, x, y in zip(("dq", "dk", "dv"), grads, want_g):
        _close(x, y, TOL[dtype], name)
    _close(grads[3], want_g[3], STATE_TOL, "dstate_in")


def test_tokens_and_states_past_four_gibibytes():
    # rows 16 MiB apart and the last states of a pool of 4.3 GiB
    N, H, D, ld = 300, 1, 128, 1 << 23
    slots, n_slots = (65800, 3), 65801
    _say(f"tokens {ld} elements apart, pool of {n_slots} states")
    q, k, v, a = _inputs((N,), H, H, D, D, "bf16", 21)
    a[0] = -0.01
    views = [torch.empty((N, ld), dtype=torch.bfloat16, device="cuda")[:, :D].unsqueeze(1) for i in range(4)]
    for view, t in zip(views, (q, k, v)):
        view.copy_(t)
    pool = torch.empty((n_slots, H, D, D), device="cuda")
    S0 = _rand((2, H, D, D), torch.float32, 5)
    for i, slot in enumerate(slots):
        pool[slot] = S0[i].cuda()
    cu = torch.tensor([0, 200, N], dtype=torch.int32).cuda()
    at = torch.tensor(slots, dtype=torch.int32).cuda()
    ws = torch.empty(max(1, fc.fftconv_decay_fwd_workspace_bytes(2, N, H, D, D, torch.bfloat16)), dtype=torch.uint8,
                     device="cuda")
    fc.fftconv_decay_fwd(*views[:3], a.cuda(), views[3], 0.2, pool, pool, at, cu, ws)
    states = []
    for b, (i, j) in enumerate(((0, 200), (200, N))):
        want, S = seq.decay_fwd(_f64(q[i:j]), _f64(k[i:j]), _f64(v[i:j]), _f64(a), 0.2, _f64(S0[b]))
        _close(views[3][i:j], want, TOL["bf16"], f"out[{b}]")
        _close(pool[slots[b]], S, STATE_TOL, f"state[{b}]")
        states.append(S)
    tok = [t[:2].contiguous() for t in (q, k, v)]
    out = torch.empty((2, H, D), dtype=torch.bfloat16, device="cuda")
    fc.fftconv_decay_step(*_gpu(*tok), a.cuda(), pool, out, 0.2, at)
    for b in range(2):
        want, S = seq.decay_fwd(*(_f64(t[b:b + 1]) for t in tok), _f64(a), 0.2, states[b])
        _close(out[b:b + 1], want, TOL["bf16"], f"token[{b}]")
        _close(pool[slots[b]], S, STATE_TOL, f"state after the token[{b}]")


def test_graph_replays_of_gradients_and_tokens():
    B, N, H, Hk, D = 2, 700, 4, 2, 64
    q, k, v, a = _inputs((B, N), H, Hk, D, D, "bf16", 1)
    qg, kg, vg, ag, dg = _gpu(q, k, v, a, _rand((B, N, H, D), torch.bfloat16, 2))
    grads = fc.decay_attention_bwd(qg, kg, vg, ag, dg, 0.2)[:3]
    ws = torch.empty(fc.fftconv_decay_bwd_workspace_bytes(B, B * N, H, Hk, D, D, torch.bfloat16), dtype=torch.uint8,
                     device="cuda")
    S = torch.zeros((B, H, D, D), device="cuda")
    out = torch.empty((B, H, D), dtype=torch.bfloat16, device="cuda")
    tok = [t[:, 0].contiguous() for t in (qg, kg, vg)]
    fc.fftconv_decay_step(*tok, ag, S, out, 0.2)
    S.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fc.fftconv_decay_bwd(dg, qg, kg, vg, ag, *grads, 0.2, workspace=ws)
        fc.fftconv_decay_step(*tok, ag, S, out, 0.2)
    eager_S, eager_out = torch.zeros_like(S), torch.empty_like(out)
    for seed in (5, 6, 7):
        dg.copy_(_rand((B, N, H, D), torch.bfloat16, seed))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(grads, fc.decay_attention_bwd(qg, kg, vg, ag, dg, 0.2)):
            assert torch.equal(got, want)
        fc.fftconv_decay_step(*tok, ag, eager_S, eager_out, 0.2)
        assert torch.equal(S, eager_S) and torch.equal(out, eager_out)
