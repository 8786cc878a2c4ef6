"""Gated delta rule where it can go wrong: views of fused buffers, gates that clear or keep the state, keys that repeat,
values that are no numbers, state pools, places past 4 GiB, workspaces of garbage, graphs, streams, parts of the gradients.

Tolerances as in the parity tests: 1.5 half units of a 16-bit result (its rounding and that of q k^T in bf16), 5e-6 for
fp32 results (sums of up to 256 exact products and chains of 64, over at most 40 chunks); the oracle is float64 on the
rounded inputs."""
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


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _close(got, want, tol, name):
    got = _f64(got)
    assert got.shape == want.shape and np.isfinite(got).all(), name
    err, norm = np.linalg.norm(got - want), np.linalg.norm(want)
    assert err <= tol * norm, f"{name}: relL2 {err / max(norm, 1e-300):.3e} > {tol:.1e}"


def _inputs(lead, H, Hk, Dk, Dv, dtype, seed, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    k = r(*lead, Hk, Dk)
    k = k / k.norm(dim=-1, keepdim=True)
    a = -torch.exp(r(*lead, H) - 3)
    return [t.to(d).to(device) for t, d in ((r(*lead, Hk, Dk), DT[dtype]), (k, DT[dtype]), (r(*lead, H, Dv), DT[dtype]),
                                           (a, torch.float32), (torch.sigmoid(r(*lead, H)), torch.float32))]


def _all(ins, dout, scale=0.3, S0=None, dS=None):
    """out, state, gradients from the library."""
    out, S = fc.delta_attention(*ins, scale=scale, state_in=S0)
    return (out, S, *fc.delta_attention_bwd(*ins, dout, scale=scale, state_in=S0, dstate_out=dS))


def _check(ins, dout, got, dtype, scale=0.3, S0=None, dS=None, skip=()):
    want_out, want_S = seq.delta_fwd(*(_f64(t[0]) for t in ins), scale, None if S0 is None else _f64(S0[0]))
    want = (want_out, want_S, *seq.delta_bwd(_f64(dout[0]), *(_f64(t[0]) for t in ins), scale, None if S0 is None else _f64(S0[0]),
                                             None if dS is None else _f64(dS[0])))
    for name, x, y in zip(("out", "state", "dq", "dk", "dv", "dlog_decay", "dbeta", "dstate_in"), got, want):
        if x is not None and name not in skip:
            _close(x[0], y, FP32 if x.dtype == torch.float32 else TOL[dtype], name)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H,Hk,Dk,Dv", [(4, 2, 64, 64), (3, 1, 40, 72), (2, 2, 33, 7), (2, 1, 128, 128)])
def test_views_of_fused_rows(H, Hk, Dk, Dv, dtype):
    """q, k, v and their gradients side by side in the rows of one matrix, out inside another."""
    _say(f"views {dtype} {H}/{Hk} {Dk} {Dv}")
    N = 150
    q, k, v, a, b = _inputs((1, N), H, Hk, Dk, Dv, dtype, 3)
    sizes = [Hk * Dk, Hk * Dk, H * Dv]

    def fused(fill):
        wide = torch.full((1, N, sum(sizes) + 5), fill, dtype=q.dtype, device="cuda")
        return wide, [t.unflatten(2, (-1, d)) for t, d in zip(wide[..., :sum(sizes)].split(sizes, dim=2), (Dk, Dk, Dv))]

    wide, views = fused(9.0)
    for t, x in zip(views, (q, k, v)):
        t.copy_(x)
    gwide, gviews = fused(9.0)
    dout = torch.randn((1, N, H, Dv), device="cuda").to(q.dtype)
    want = _all((q, k, v, a, b), dout)
    out_wide = torch.full((1, N, H, Dv + 3), 9.0, dtype=q.dtype, device="cuda")
    out, S = out_wide[..., :Dv], torch.empty_like(want[1])
    ws = torch.empty(max(fc.fftconv_delta_fwd_workspace_bytes(1, N, H, Hk, Dk, Dv, q.dtype),
                         fc.fftconv_delta_bwd_workspace_bytes(1, N, H, Hk, Dk, Dv, q.dtype)), dtype=torch.uint8, device="cuda")
    fc.fftconv_delta_fwd(*views, a, b, out, 0.3, state_out=S, workspace=ws)
    da, db = torch.empty_like(a), torch.empty_like(b)
    fc.fftconv_delta_bwd(dout, *views, a, b, *gviews, da, db, 0.3, workspace=ws)
    for x, y in zip((out, S, *gviews, da, db), want):
        # the same sums in the same order, whatever the rows' alignment
        assert torch.equal(x, y)
    assert (out_wide[..., Dv:] == 9).all() and (gwide[..., sum(sizes):] == 9).all()
    one, oneS = torch.empty((1, H, Dv), dtype=q.dtype, device="cuda"), want[1].clone()
    two, twoS = torch.empty_like(one), want[1].clone()
    fc.fftconv_delta_step(*(t[:, 5] for t in views), a[:, 5].contiguous(), b[:, 5].contiguous(), oneS, one, 0.3)
    fc.fftconv_delta_step(*(t[:, 5].contiguous() for t in (q, k, v)), a[:, 5].contiguous(), b[:, 5].contiguous(), twoS, two, 0.3)
    assert torch.equal(one, two) and torch.equal(oneS, twoS)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_at_their_limits(dtype):
    """Tokens that clear the state (-inf, -200, -90), that keep all of it, that write nothing or the whole of a value."""
    H, D, N = 4, 64, 200
    ins = _inputs((1, N), H, H, D, D, dtype, 5)
    a, b = ins[3], ins[4]
    a[0, ::7, 0] = float("-inf")
    a[0, 3::5, 1] = -200.0
    a[0, ::2, 2] = -90.0
    a[..., 3] = 0.0
    b[0, ::3, 3] = 0.0
    b[0, 1::3, 3] = 1.0
    b[..., 0] = 2.0
    dout = torch.randn((1, N, H, D), device="cuda").to(ins[0].dtype)
    S0, dS = torch.randn((1, H, D, D), device="cuda"), torch.randn((1, H, D, D), device="cuda")
    _check(ins, dout, _all(ins, dout, S0=S0, dS=dS), dtype, S0=S0, dS=dS)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_repeated_keys(dtype):
    """One key for a whole sequence, written whole each time and never forgotten: the system's matrix is full of ones."""
    H, D, N = 2, 64, 130
    ins = _inputs((1, N), H, H, D, D, dtype, 6)
    ins[1].zero_()
    ins[1][..., 0] = 1.0
    ins[3].zero_()
    ins[4].fill_(1.0)
    dout = torch.randn((1, N, H, D), device="cuda").to(ins[0].dtype)
    got = _all(ins, dout)
    _check(ins, dout, got, dtype, skip=("dlog_decay",))
    # a whole write leaves nothing of the state behind along the key, so a gate's gradient is exactly 0. It is formed as
    # sum over i >= t of q_i dq_i - v_i dv_i, terms that are not 0 and cancel: what is left is their roundings, of the size
    # of each term and independent, so of the root of the sum of squares behind t
    dq, dv = _f64(got[2][0]), _f64(got[4][0])
    terms = (_f64(ins[0][0]) * dq).sum(-1) ** 2 + (_f64(ins[2][0]) * dv).sum(-1) ** 2
    behind = np.sqrt(np.cumsum(terms[::-1], axis=0)[::-1])
    assert np.linalg.norm(_f64(got[5][0])) <= FP32 * np.linalg.norm(behind)


@pytest.mark.parametrize("dtype,scale", [("f16", 1e-4), ("f16", 200.0), ("bf16", 1e12), ("f32", 1e-12)])
def test_values_of_any_size(dtype, scale):
    """Values (and with them states and outputs) far from 1; keys keep their norm."""
    ins = _inputs((1, 200), 2, 2, 64, 64, dtype, 7)
    ins[2] = (ins[2].double() * scale).to(DT[dtype])
    out, S = fc.delta_attention(*ins, scale=0.3)
    want, wS = seq.delta_fwd(*(_f64(t[0]) for t in ins), 0.3)
    # fp16 results near 1e-5 are subnormal: half a step of 2^-24 each, beside the relative error
    err = np.linalg.norm(_f64(out[0]) - want)
    least = 2.0 ** -25 * np.sqrt(want.size) if dtype == "f16" else 0.0
    assert err <= TOL[dtype] * np.linalg.norm(want) + least
    _close(S[0], wS, FP32, "state")


def test_not_a_number_stays_in_its_sequence_and_head():
    H, Hk, D = 4, 2, 64
    lens = [70, 33, 65, 10]
    cu = torch.tensor([0, 70, 103, 168, 178], dtype=torch.int32, device="cuda")
    ins = _inputs((178,), H, Hk, D, D, "bf16", 8)
    dout = torch.randn((178, H, D), device="cuda").to(torch.bfloat16)
    want = (*fc.delta_attention(*ins, cu_seqlens=cu), *fc.delta_attention_bwd(*ins, dout, cu_seqlens=cu)[:5])
    v = ins[2].clone()
    v[80, 1] = float("nan")             # sequence 1, head 1
    v[120, 3] = float("inf")            # sequence 2, head 3
    bad = (ins[0], ins[1], v, ins[3], ins[4])
    got = (*fc.delta_attention(*bad, cu_seqlens=cu), *fc.delta_attention_bwd(*bad, dout, cu_seqlens=cu)[:5])
    hit = torch.zeros(178, H, dtype=torch.bool, device="cuda")
    hit[70:103, 1] = hit[103:168, 3] = True
    for name, x, y in zip(("out", "state", "dq", "dk", "dv", "dg", "db"), got, want):
        if name == "state":
            states = torch.ones(4, H, dtype=torch.bool, device="cuda")
            states[1, 1] = states[2, 3] = False
            assert torch.equal(x[states], y[states])
            continue
        clean = ~hit if x.shape[1] == H else ~(hit.unflatten(1, (Hk, H // Hk)).any(2))
        assert torch.equal(x[clean], y[clean]), name
    assert torch.isnan(got[0][80, 1]).all() and len(lens) == 4


@pytest.mark.parametrize("N", [150, 2100])
def test_state_pool_in_place(N):
    """Prompts that continue states of a pool, one of them with no slot; 2100 tokens are cut into segments."""
    B, H, D, slots = 3, 1, 64, 7
    ins = _inputs((B, N), H, H, D, D, "bf16", 9)
    pool = torch.randn((slots, H, D, D), device="cuda")
    kept = pool.clone()
    where = torch.tensor([5, -1, 2], dtype=torch.int32, device="cuda")
    out = torch.empty_like(ins[2])
    ws = torch.full((fc.fftconv_delta_fwd_workspace_bytes(B, B * N, H, H, D, D, torch.bfloat16),), 255, dtype=torch.uint8, device="cuda")
    fc.fftconv_delta_fwd(*ins, out, 0.3, state_in=pool, state_out=pool, state_slots=where, workspace=ws)
    for b, s in enumerate((5, None, 2)):
        want, wS = seq.delta_fwd(*(_f64(t[b]) for t in ins), 0.3, None if s is None else _f64(kept[s]))
        _close(out[b], want, TOL["bf16"], f"out[{b}]")
        if s is not None:
            _close(pool[s], wS, FP32, f"state[{b}]")
    others = [s for s in range(slots) if s not in (5, 2)]
    assert torch.equal(pool[others], kept[others])


def test_places_past_four_gib():
    """Rows 8 MiB apart (700 tokens: 5.6 GB) and a pool whose last state lies past 4 GiB."""
    N, D = 700, 64
    q, k, v, a, b = _inputs((1, N), 1, 1, D, D, "bf16", 10)
    want, S = fc.delta_attention(q, k, v, a, b, scale=0.3)
    step = (8 << 20) // 2
    wide = torch.empty((N, step), dtype=torch.bfloat16, device="cuda")
    views = [wide[:, i * D:(i + 1) * D].view(1, N, 1, D) for i in range(4)]
    for t, x in zip(views, (q, k, v)):
        t.copy_(x)
    ws = torch.empty(fc.fftconv_delta_fwd_workspace_bytes(1, N, 1, 1, D, D, torch.bfloat16), dtype=torch.uint8, device="cuda")
    got = torch.empty_like(S)
    fc.fftconv_delta_fwd(*views[:3], a, b, views[3], 0.3, state_out=got, workspace=ws)
    assert torch.equal(views[3], want) and torch.equal(got, S)
    del wide, views
    slots = 300000
    pool = torch.zeros((slots, 1, D, D), device="cuda")
    where = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
    pool[slots - 1] = S[0]
    one, two, state = torch.empty((1, 1, D), dtype=q.dtype, device="cuda"), torch.empty((1, 1, D), dtype=q.dtype, device="cuda"), S.clone()
    fc.fftconv_delta_step(q[:, 0], k[:, 0], v[:, 0], a[:, 0], b[:, 0], pool, one, 0.3, where)
    fc.fftconv_delta_step(q[:, 0], k[:, 0], v[:, 0], a[:, 0], b[:, 0], state, two, 0.3)
    assert torch.equal(one, two) and torch.equal(pool[slots - 1], state[0]) and (pool[:slots - 1] == 0).all()


@pytest.mark.parametrize("N,H,Hk", [(150, 4, 2), (1100, 2, 2)])
def test_graph_replays(N, H, Hk):
    """Prompt, gradients and a token in one graph, replayed with other inputs and eager work in between."""
    D = 64
    ins = _inputs((2, N), H, Hk, D, D, "bf16", 11)
    dout = torch.randn((2, N, H, D), device="cuda").to(torch.bfloat16)
    out, S = torch.empty_like(ins[2]), torch.empty((2, H, D, D), device="cuda")
    grads = [torch.empty_like(t) for t in ins]
    token = torch.empty((2, H, D), dtype=torch.bfloat16, device="cuda")
    f = torch.full((fc.fftconv_delta_fwd_workspace_bytes(2, 2 * N, H, Hk, D, D, torch.bfloat16),), 255, dtype=torch.uint8, device="cuda")
    w = torch.full((fc.fftconv_delta_bwd_workspace_bytes(2, 2 * N, H, Hk, D, D, torch.bfloat16),), 255, dtype=torch.uint8, device="cuda")
    a0, b0 = ins[3][:, 0].contiguous(), ins[4][:, 0].contiguous()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        fc.fftconv_delta_fwd(*ins, out, 0.3, state_out=S, workspace=f)
        fc.fftconv_delta_bwd(dout, *ins, *grads, 0.3, workspace=w)
        fc.fftconv_delta_step(ins[0][:, 0], ins[1][:, 0], ins[2][:, 0], a0, b0, S, token, 0.3)
    for seed in range(3):
        for t, x in zip(ins, _inputs((2, N), H, Hk, D, D, "bf16", 20 + seed)):
            t.copy_(x)
        a0.copy_(ins[3][:, 0])
        b0.copy_(ins[4][:, 0])
        for t in (out, S, *grads, token):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        want = _all(ins, dout)
        last = want[1].clone()
        one = torch.empty_like(token)
        fc.fftconv_delta_step(ins[0][:, 0], ins[1][:, 0], ins[2][:, 0], a0, b0, last, one, 0.3)
        for x, y in zip((out, *grads, S, token), (want[0], *want[2:7], last, one)):
            assert torch.equal(x, y)


def test_another_stream():
    ins = _inputs((1, 3000), 2, 2, 64, 64, "bf16", 12)
    dout = torch.randn((1, 3000, 2, 64), device="cuda").to(torch.bfloat16)
    want = (*fc.delta_attention(*ins), *fc.delta_attention_bwd(*ins, dout)[:5])
    work = torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(4):
            work = torch.nn.functional.normalize(work @ work)
    got = (*fc.delta_attention(*ins, stream=s), *fc.delta_attention_bwd(*ins, dout, stream=s)[:5])
    taken = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 18, 1 << 20, 1 << 22, 1 << 24) for _ in range(4)]
    torch.cuda.synchronize()
    assert len(taken) == 16
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("H,Hk,Dk,Dv", [(2, 2, 64, 64), (4, 2, 128, 128), (2, 1, 256, 33)])
def test_parts_of_the_gradients(H, Hk, Dk, Dv):
    """Each gradient by itself equals that of the whole call, which repeats bit by bit; the workspace may hold anything."""
    N = 140
    ins = _inputs((2, N), H, Hk, Dk, Dv, "bf16", 13)
    dout = torch.randn((2, N, H, Dv), device="cuda").to(torch.bfloat16)
    S0, dS = torch.randn((2, H, Dk, Dv), device="cuda"), torch.randn((2, H, Dk, Dv), device="cuda")
    want = fc.delta_attention_bwd(*ins, dout, scale=0.3, state_in=S0, dstate_out=dS)
    ws = torch.full((fc.fftconv_delta_bwd_workspace_bytes(2, 2 * N, H, Hk, Dk, Dv, torch.bfloat16),), 255, dtype=torch.uint8, device="cuda")
    for i in range(6):
        some = [torch.empty_like(t) if j == i else None for j, t in enumerate((*ins, S0))]
        fc.fftconv_delta_bwd(dout, *ins, *some[:5], 0.3, state_in=S0, dstate_out=dS, dstate_in=some[5], workspace=ws)
        assert torch.equal(some[i], want[i]), i


def test_gradients_against_differences():
    """The fp32 forward's differences along random directions, h = 2^-7: third-order terms of h^2 / 6 of values of size 1
    and roundings of 2^-20 of the loss over h, both below 2^-9 of the directions' sizes."""
    ins = _inputs((1, 90), 2, 1, 32, 40, "f32", 14)
    dout = torch.randn((1, 90, 2, 40), device="cuda")
    S0 = torch.randn((1, 2, 32, 40), device="cuda")
    grads = fc.delta_attention_bwd(*ins, dout, scale=0.3, state_in=S0)
    args = [*ins, S0]

    def loss(args):
        return float((fc.delta_attention(*args[:5], scale=0.3, state_in=args[5])[0].double() * dout.double()).sum())

    h = 2.0 ** -7
    for i, g in enumerate(grads):
        step = torch.randn(args[i].shape, device="cuda")
        step /= step.norm()
        up, down = ([*args[:i], args[i] + s * h * step, *args[i + 1:]] for s in (1, -1))
        want = (loss(up) - loss(down)) / (2 * h)
        assert abs(want - float((g.double() * step.double()).sum())) < 2.0 ** -9 * max(1.0, float(g.norm())), i
