"""Cases that measure the operators of a gated delta rule block beside the long convolution and decay attention: the
rule itself (prompt, backward, single token) and the root-mean-square norm with the residual's addition and an output
in 8 bits (forward, backward).

Plain form, per sequence and head with a_t = exp(log_decay_t) <= 1, beta_t and an fp32 state S (Dk x Dv):

    u_t = beta_t (v_t - a_t S_{t-1}^T k_t),   S_t = a_t S_{t-1} + k_t u_t^T,   out_t = scale * S_t^T q_t
    s = x + residual,   y = s / sqrt(mean(s^2) + eps) * weight,   8 bits: y ~ out * max|y| / 448

Widths are 768 = 12 x 64 and 2560 = 20 x 128, lengths from one token to 131072; keys have norm 1.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FP8 = torch.float8_e4m3fn
EPS = 1e-6
MOST_STATE = 131072 * 20 * 128     # tokens x heads x head width of the largest prompt


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a short prompt of odd length, as an interactive user sends it: latency
        dict(name="delta prompt 17", op="delta_fwd", dtype="f16", B=1, N=17, lengths="", H=12, Hk=12, Dk=64, Dv=64,
             state=False),
        # prompts of different lengths packed into one call, query/key heads shared by five value heads, each with the
        # state of its earlier part; empty and one-token members
        dict(name="delta prompt packed", op="delta_fwd", dtype="bf16", B=12, N=0,
             lengths="0,1,63,64,65,257,1000,1023,1777,2048,4096,6001", H=20, Hk=4, Dk=128, Dv=128, state=True),
        # one long document (genome-scale context)
        dict(name="delta prompt 131072", op="delta_fwd", dtype="bf16", B=1, N=131072, lengths="", H=20, Hk=20, Dk=128,
             Dv=128, state=False),
        # training step of the 2560-wide model
        dict(name="delta backward 4x4096", op="delta_bwd", dtype="bf16", B=4, N=4096, lengths="", H=20, Hk=20, Dk=128,
             Dv=128, state=False),
        # training step of the 768-wide model, odd length, shared query/key heads, gradients of the carried state
        dict(name="delta backward 8x1000", op="delta_bwd", dtype="f16", B=8, N=1000, lengths="", H=12, Hk=4, Dk=64,
             Dv=64, state=True),
        # one user's next token: latency
        dict(name="delta token 1", op="delta_step", dtype="bf16", B=1, H=20, Hk=20, Dk=128, Dv=128),
        # the next token of a full serving batch
        dict(name="delta token 256", op="delta_step", dtype="bf16", B=256, H=20, Hk=20, Dk=128, Dv=128),
        # one user's next token, the residual stream's addition fused: latency
        dict(name="norm 1x2560", op="norm_fwd", dtype="bf16", M=1, G=1, D=2560, residual=True, eight=False, inside=0),
        # a prompt batch's rows for a product in 8 bits
        dict(name="norm 16384x2560 8 bits", op="norm_fwd", dtype="bf16", M=16384, G=1, D=2560, residual=True, eight=True,
             inside=0),
        # the keys of 16384 tokens, 20 heads, as they lie between queries and values in the projection's rows
        dict(name="norm heads 16384x20x128", op="norm_fwd", dtype="f16", M=16384, G=20, D=128, residual=False, eight=False,
             inside=7680),
        # training step of the 2560-wide model, with the residual stream's own gradient
        dict(name="norm backward 16384x2560", op="norm_bwd", dtype="bf16", M=16384, G=1, D=2560, residual=True),
        # a few odd rows in fp32
        dict(name="norm backward 1000x768", op="norm_bwd", dtype="f32", M=1000, G=1, D=768, residual=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_bwd", "delta_step", "norm_fwd", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op.startswith("norm"):
        D = rng.choice([64, 128, 768, 1536, 2560, _log_int(rng, 33, 10240), 8 * _log_int(rng, 8, 1280)])
        G = rng.choice([1, 1, 4, 20]) if D <= 256 else 1
        case = dict(op=op, dtype=dtype, M=_log_int(rng, 1, max(2, 16384 * 2560 // (G * D))), G=G, D=D,
                    residual=rng.random() < 0.5)
        if op == "norm_fwd":
            case.update(eight=rng.random() < 0.3, inside=3 * G * D if not case["residual"] and rng.random() < 0.5 else 0)
        return case
    Dk, Dv = rng.choice([(64, 64), (128, 128), (64, 128), (128, 64), (96, 96), (32, 64), (40, 72), (33, 65), (192, 256)])
    Hk = rng.choice([1, 2, 3, 4, 5, 8, 12, 20])
    H = Hk * rng.choice([1, 1, 1, 2, 4])
    if op == "delta_step":
        return dict(op=op, dtype=dtype, B=_log_int(rng, 1, 256 if max(Dk, Dv) <= 128 else 64), H=H, Hk=Hk, Dk=Dk, Dv=Dv)
    most = MOST_STATE if op == "delta_fwd" else 4 * 4096 * 20 * 128
    total = _log_int(rng, 16, max(32, min(131072, most // (H * max(Dk, Dv)))))
    if dtype == "f32":
        total = min(total, 16384)
    B = min(total, _log_int(rng, 1, 32))
    case = dict(op=op, dtype=dtype, B=B, N=max(1, total // B), lengths="", H=H, Hk=Hk, Dk=Dk, Dv=Dv,
                state=rng.random() < 0.5)
    if rng.random() < 0.4:
        parts = sorted(rng.randint(0, total) for _ in range(B - 1))
        ends = [0] + parts + [total]
        case.update(N=0, lengths=",".join(str(b - a) for a, b in zip(ends, ends[1:])))
    return case


def _lengths(case):
    return [int(s) for s in case["lengths"].split(",")] if case["lengths"] else [case["N"]] * case["B"]


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("norm"):
        n = case["M"] * case["G"] * case["D"]
        w = case["D"] * e
        if case["op"] == "norm_bwd":
            return dict(bytes=n * e * (4 if case["residual"] else 3) + 2 * w, flops=10 * n)
        out = n + 4 * case["M"] * case["G"] if case["eight"] else n * e
        return dict(bytes=n * e * (3 if case["residual"] else 1) + out + w, flops=5 * n)
    H, Hk, Dk, Dv = (case[x] for x in ("H", "Hk", "Dk", "Dv"))
    if case["op"] == "delta_step":
        B = case["B"]
        return dict(bytes=B * (8 * H * Dk * Dv + e * (2 * H * Dv + 2 * Hk * Dk) + 8 * H), flops=7 * B * H * Dk * Dv)
    T, S = sum(_lengths(case)), case["B"] * H * Dk * Dv * 4
    qk, vo, gates = 2 * T * Hk * Dk * e, 2 * T * H * Dv * e, 8 * T * H
    if case["op"] == "delta_fwd":
        return dict(bytes=qk + vo + gates + S * (2 if case["state"] else 1), flops=7 * T * H * Dk * Dv)
    return dict(bytes=2 * qk + vo + T * H * Dv * e + 2 * gates + S * (3 if case["state"] else 0),
                flops=18 * T * H * Dk * Dv)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def randn(*shape, dtype=dt, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32) * scale).to(dtype)

    s = dict(case=dict(case))
    if case["op"].startswith("norm"):
        M, G, D = case["M"], case["G"], case["D"]
        s["weight"] = (1 + randn(D, dtype=torch.float32, scale=0.2)).to(dt)
        if case["op"] == "norm_bwd":
            s["dout"], s["x"] = randn(M, G, D), randn(M, G, D, scale=2.0)
            s["dsum"] = randn(M, G, D) if case["residual"] else None
            s["dx"], s["dweight"] = torch.empty_like(s["x"]), torch.empty_like(s["weight"])
            return s
        if case["inside"]:      # columns G D .. 2 G D of wider rows
            s["x"] = randn(M, case["inside"], scale=2.0)[:, G * D:2 * G * D].unflatten(1, (G, D))
        else:
            s["x"] = randn(M, G, D, scale=2.0)
        if case["residual"]:
            s["residual"], s["sum"] = randn(M, G, D, scale=3.0), torch.empty((M, G, D), dtype=dt, device=DEVICE)
        s["out"] = torch.empty((M, G, D), dtype=FP8 if case["eight"] else dt, device=DEVICE)
        if case["eight"]:
            s["scales"] = torch.empty((M, G), dtype=torch.float32, device=DEVICE)
        return s
    B, H, Hk, Dk, Dv = (case[x] for x in ("B", "H", "Hk", "Dk", "Dv"))
    s["scale"] = Dk ** -0.5
    if case["op"] == "delta_step":
        lead = (B,)
        slots = B + 3           # a pool with a few free slots, its sequences in any order
        s["slots"] = torch.randperm(slots, generator=g, device=DEVICE)[:B].to(torch.int32)
        s["state"] = randn(slots, H, Dk, Dv, dtype=torch.float32)
    elif case["lengths"]:
        lens = _lengths(case)
        lead = (sum(lens),)
        s["cu_seqlens"] = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEVICE)
    else:
        lead = (B, case["N"])
    # each head forgets at its own rate, each token by its own share of it; how much of a value is written is a sigmoid
    rate = torch.exp(math.log(1e-4) + torch.rand((H,), generator=g, device=DEVICE) * math.log(1e3))
    s["log_decay"] = -rate * torch.nn.functional.softplus(randn(*lead, H, dtype=torch.float32) + 0.5)
    s["beta"] = torch.sigmoid(randn(*lead, H, dtype=torch.float32))
    k = randn(*lead, Hk, Dk, dtype=torch.float32)
    s["k"] = (k / k.square().sum(-1, keepdim=True).sqrt()).to(dt)
    s["q"], s["v"] = randn(*lead, Hk, Dk), randn(*lead, H, Dv)
    if case["op"] != "delta_bwd":
        s["out"] = torch.empty((*lead, H, Dv), dtype=dt, device=DEVICE)
    if case["op"] == "delta_fwd":
        s["state_out"] = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=DEVICE)
    if case["op"] == "delta_bwd":
        s["dout"] = randn(*lead, H, Dv)
        for x in ("q", "k", "v", "log_decay", "beta"):
            s["d" + x] = torch.empty_like(s[x])
    if case.get("state"):
        s["state_in"] = randn(B, H, Dk, Dv, dtype=torch.float32)
        if case["op"] == "delta_bwd":
            s["dstate_out"] = randn(B, H, Dk, Dv, dtype=torch.float32)
            s["dstate_in"] = torch.empty_like(s["dstate_out"])
    return s


# ---------------------------------------------------------------- plain forms (32 bits, rounded once)
CHUNK = 64


def _chunked(t, state):
    """(B, heads, chunks, CHUNK, D) in 32 bits, zeros behind each sequence's end."""
    t = t.float()
    cu = state.get("cu_seqlens")
    if cu is not None:
        lens = _lengths(state["case"])
        at = cu[:-1, None].long() + torch.arange(max(lens), device=t.device)
        inside = at < cu[1:, None].long()
        t = t[at.clamp(max=t.shape[0] - 1)] * inside.reshape(*inside.shape, *[1] * (t.dim() - 1))
    t = t.unsqueeze(-1) if t.dim() == 3 else t
    t = torch.nn.functional.pad(t.transpose(1, 2), (0, 0, 0, -t.shape[1] % CHUNK))
    return t.unflatten(2, (-1, CHUNK))


def _unchunked(t, state, dtype, gate=False):
    """(B, heads, chunks, CHUNK, D) -> the caller's layout and type."""
    t = t.flatten(2, 3).transpose(1, 2)
    t = t[..., 0] if gate else t
    cu = state.get("cu_seqlens")
    if cu is None:
        return t[:, :state["case"]["N"]].to(dtype)
    inside = torch.arange(t.shape[1], device=t.device) < (cu[1:] - cu[:-1])[:, None]
    return t[inside].to(dtype)


def _t(m):
    return m.transpose(-1, -2).contiguous()


def _rule(s):
    """What both directions need of the chunks: everything that no state goes into."""
    share = s["case"]["H"] // s["case"]["Hk"]
    q, k, v = (_chunked(s[x], s) for x in ("q", "k", "v"))
    q, k = (t.repeat_interleave(share, 1) for t in (q, k))
    beta = _chunked(s["beta"], s)
    G = _chunked(s["log_decay"], s).double().cumsum(-2)              # (..., CHUNK, 1)
    D = torch.exp(torch.tril(G - G.transpose(-1, -2))).float().tril()
    A = (beta * D * (k @ _t(k))).tril(-1)
    P = (D * (q @ _t(k))) * s["scale"]
    # (I + A)^-1 = (I - A)(I + A^2)(I + A^4) ..., A^CHUNK = 0
    eye = torch.eye(CHUNK, device=q.device)
    T, power = eye - A, A @ A
    for _ in range(CHUNK.bit_length() - 3):
        T, power = T @ (eye + power), power @ power
    T = T @ (eye + power)
    first, last = torch.exp(G).float(), torch.exp(G[..., -1:, :] - G).float()
    return dict(q=q, k=k, v=v, beta=beta, A=A, P=P, D=D, T=T, first=first, last=last, end=first[..., -1:, :],
                W=T @ (beta * first * k), U0=T @ (beta * v), kT=_t(last * k))


def _forward_states(c, first):
    """States before each chunk, u of each chunk and the last state: the recurrence, chunk by chunk."""
    n = c["q"].shape[2]
    S = torch.zeros((*c["q"].shape[:2], c["q"].shape[-1], c["v"].shape[-1]), device=c["q"].device) if first is None \
        else first
    states, us = [], []
    for i in range(n):
        states.append(S)
        us.append(c["U0"][:, :, i] - c["W"][:, :, i] @ S)
        S = c["end"][:, :, i] * S + c["kT"][:, :, i] @ us[-1]
    return torch.stack(states, 2), torch.stack(us, 2), S


def _plain_delta(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    share = case["H"] // case["Hk"]
    if case["op"] == "delta_step":
        at = s["slots"].long()
        q, k = (s[x].float().repeat_interleave(share, 1) for x in ("q", "k"))
        S = s["state"][at] * torch.exp(s["log_decay"])[..., None, None]
        u = s["beta"][..., None] * (s["v"].float() - (k[..., None, :] @ S)[..., 0, :])
        S = S + k[..., :, None] * u[..., None, :]
        s["state"][at] = S
        return dict(out=((q[..., None, :] @ S)[..., 0, :] * s["scale"]).to(dt), state=s["state"])
    c = _rule(s)
    S0, U, last = _forward_states(c, s.get("state_in"))
    if case["op"] == "delta_fwd":
        out = (s["scale"] * c["first"] * c["q"]) @ S0 + c["P"] @ U
        return dict(out=_unchunked(out, s, dt), state_out=last)
    do = _chunked(s["dout"], s)
    # dU = P^T dO + last (K G), dR = T^T dU; G before the chunk from G behind it
    dU0, TT = _t(c["P"]) @ do, _t(c["T"])
    own_part = _t(s["scale"] * c["first"] * c["q"]) @ do
    kbT = _t(c["beta"] * c["first"] * c["k"])
    ke = c["last"] * c["k"]
    G = s["dstate_out"] if "dstate_out" in s else torch.zeros_like(last)
    Gs, dRs = [], []
    for i in reversed(range(do.shape[2])):
        Gs.append(G)
        dRs.append(TT[:, :, i] @ (dU0[:, :, i] + ke[:, :, i] @ G))
        G = c["end"][:, :, i] * G + own_part[:, :, i] - kbT[:, :, i] @ dRs[-1]
    G1, dR = torch.stack(Gs[::-1], 2), torch.stack(dRs[::-1], 2)
    dv = c["beta"] * dR
    S0T, GT = _t(S0), _t(G1)
    dP = (do @ _t(U)).tril() * c["D"] * s["scale"]
    dB = -(dR @ _t(U)).tril(-1) * c["D"] * c["beta"]        # gradient of k k^T
    dq = s["scale"] * c["first"] * (do @ S0T) + dP @ c["k"]
    dk = _t(dP) @ c["q"] + c["last"] * (U @ GT) + (dB + _t(dB)) @ c["k"] - c["first"] * (dv @ S0T)
    wrong = c["v"] - c["first"] * (c["k"] @ S0) - (c["D"].tril(-1) * (c["k"] @ _t(c["k"]))) @ U
    dbeta = (dR * wrong).sum(-1, keepdim=True)
    # the gradient of the summed logarithms is q dq - v dv at a token, and that of the state behind the chunk
    behind = S0[:, :, 1:]
    S1 = torch.cat([behind, last[:, :, None]], 2)
    each = ((c["q"] * dq).sum(-1, keepdim=True) - (c["v"] * dv).sum(-1, keepdim=True)).double()
    dg = each.flip(-2).cumsum(-2).flip(-2) + (G1.double() * S1).sum((-1, -2))[..., None, None]
    shared = (case["Hk"], share)
    dq, dk = (t.unflatten(1, shared).sum(2) for t in (dq, dk))
    r = dict(dq=_unchunked(dq, s, dt), dk=_unchunked(dk, s, dt), dv=_unchunked(dv, s, dt),
             dlog_decay=_unchunked(dg, s, torch.float32, True), dbeta=_unchunked(dbeta, s, torch.float32, True))
    return dict(r, dstate_in=G) if case["state"] else r


def _plain_norm(s):
    """Outputs not yet rounded."""
    case = s["case"]
    x, w = s["x"].float(), s["weight"].float()
    if case["op"] == "norm_fwd":
        t = x + s["residual"].float() if case["residual"] else x
        y = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * w
        r = dict(sum=t) if case["residual"] else {}
        if not case["eight"]:
            return dict(r, out=y)
        scales = y.abs().amax(-1) / 448
        return dict(r, out=y / scales[..., None], scales=scales)
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    dy, xh = s["dout"].float(), x * rstd
    dxh = dy * w
    dx = rstd * (dxh - xh * (dxh * xh).mean(-1, keepdim=True))
    if case["residual"]:
        dx = dx + s["dsum"].float()
    return dict(dx=dx, dweight=(dy * xh).sum((0, 1)))


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return _own_run(state)
    if state["case"]["op"].startswith("delta"):
        return _plain_delta(state)
    dt = DTYPES[state["case"]["dtype"]]
    r = {k: v if k == "scales" else v.to(dt) if not (k == "out" and state["case"]["eight"]) else v
         for k, v in _plain_norm(state).items()}
    if state["case"].get("eight"):
        r["out"] = r["out"].clamp(-448, 448).to(FP8)
    return r


def _own_run(s):
    import long_fft_convolution_amd as fc

    case, op = s["case"], s["case"]["op"]
    if op == "norm_fwd":
        fc.fftconv_norm_fwd(s["x"], s["weight"], s["out"], EPS, residual=s.get("residual"), sum=s.get("sum"),
                            scales=s.get("scales"))
        return {k: s[k] for k in ("out", "sum", "scales") if k in s}
    if op == "norm_bwd":
        if "workspace" not in s:
            _workspace(s, fc.fftconv_norm_bwd_workspace_bytes(case["M"] * case["G"], case["D"]))
        fc.fftconv_norm_bwd(s["dout"], s["x"], s["weight"], s["dx"], s["dweight"], EPS, dsum=s["dsum"],
                            workspace=s["workspace"])
        return dict(dx=s["dx"], dweight=s["dweight"])
    if op == "delta_step":
        fc.fftconv_delta_step(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["state"], s["out"], s["scale"],
                              s["slots"])
        return dict(out=s["out"], state=s["state"])
    sizes = (case["B"], s["v"].numel() // (case["H"] * case["Dv"]), case["H"], case["Hk"], case["Dk"], case["Dv"],
             s["q"].dtype)
    if op == "delta_fwd":
        if "workspace" not in s:
            _workspace(s, fc.fftconv_delta_fwd_workspace_bytes(*sizes))
        fc.fftconv_delta_fwd(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["out"], s["scale"],
                             state_in=s.get("state_in"), state_out=s["state_out"], cu_seqlens=s.get("cu_seqlens"),
                             workspace=s["workspace"])
        return dict(out=s["out"], state_out=s["state_out"])
    if "workspace" not in s:
        _workspace(s, fc.fftconv_delta_bwd_workspace_bytes(*sizes))
    fc.fftconv_delta_bwd(s["dout"], s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["dq"], s["dk"], s["dv"],
                         s["dlog_decay"], s["dbeta"], s["scale"], state_in=s.get("state_in"),
                         dstate_out=s.get("dstate_out"), dstate_in=s.get("dstate_in"), cu_seqlens=s.get("cu_seqlens"),
                         workspace=s["workspace"])
    names = ("dq", "dk", "dv", "dlog_decay", "dbeta") + (("dstate_in",) if case["state"] else ())
    return {k: s[k] for k in names}


def _exact_norm(s):
    """In 64 bits; values in 8 bits as they are before that rounding, in units of their scale."""
    case = s["case"]
    t, w = s["x"].double(), s["weight"].double()
    r = {}
    if case["op"] == "norm_fwd" and case["residual"]:
        t = r["sum"] = t + s["residual"].double()
    length = ((t * t).sum(-1, keepdim=True) / case["D"] + EPS).sqrt()
    unit = t / length
    if case["op"] == "norm_fwd":
        r["out"] = unit * w
        if case["eight"]:
            r["scales"] = r["out"].abs().max(-1).values / 448
            r["out"] = r["out"] / r["scales"].unsqueeze(-1)
        return r
    # y = unit w: the part of w dy that is along the row's direction changes only its length
    wdy = w * s["dout"].double()
    along = (wdy * unit).sum(-1, keepdim=True) / case["D"]
    r["dx"] = (wdy - along * unit) / length
    if case["residual"]:
        r["dx"] = r["dx"] + s["dsum"].double()
    r["dweight"] = (unit * s["dout"].double()).flatten(0, 1).sum(0)
    return r


def _workspace(state, nbytes):
    """The call's scratch, kept with the state as a program keeps it."""
    state["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device=DEVICE) if nbytes else None


# ---------------------------------------------------------------- 64 bits, token by token
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s)
    H, Dk, Dv = case["H"], case["Dk"], case["Dv"]
    share = H // case["Hk"]
    if case["op"] == "delta_step":
        state = s["state"].double()
        out = torch.empty((case["B"], H, Dv), dtype=torch.float64, device=DEVICE)
        for b, slot in enumerate(s["slots"].tolist()):
            k, q = (s[x][b].double().repeat_interleave(share, 0)[:, :, None] for x in ("k", "q"))
            S = state[slot] * torch.exp(s["log_decay"][b].double())[:, None, None]
            u = s["beta"][b].double()[:, None] * (s["v"][b].double() - (k * S).sum(1))
            state[slot] = S + k * u[:, None, :]
            out[b] = s["scale"] * (q * state[slot]).sum(1)
        return dict(out=out, state=state)
    lens = _lengths(case)
    backward = case["op"] == "delta_bwd"
    # (sequences walked together) x (tokens walked one by one)
    groups = [(list(range(case["B"])), None)] if not case["lengths"] else [([b], b) for b in range(case["B"])]
    steps = case["N"] if not case["lengths"] else sum(lens)
    each = (case["B"] if not case["lengths"] else 1) * H * Dk * Dv * 8 * 8 / 2e12
    if steps * (80e-6 + each) * (4 if backward else 1) > 20:
        return None
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    got = {}
    for bs, b in groups:
        def part(name):
            t = s[name].double()
            t = t if b is None else t[ends[b]:ends[b + 1]][None]
            return t.repeat_interleave(share, 2) if name in ("q", "k") else t

        def carried(name):
            return s[name][bs].double() if s.get(name) is not None else \
                torch.zeros((len(bs), H, Dk, Dv), dtype=torch.float64, device=DEVICE)

        q, k, v, beta, a = part("q"), part("k"), part("v"), part("beta"), torch.exp(part("log_decay"))
        n = q.shape[1]

        def step(S, t):
            """State behind token t, the decayed one before its write, and what was wrong with the value there."""
            decayed = a[:, t, :, None, None] * S
            wrong = v[:, t] - (k[:, t, :, None, :] @ decayed)[:, :, 0]
            return decayed + k[:, t, :, :, None] * (beta[:, t, :, None] * wrong)[:, :, None, :], decayed, wrong

        S = carried("state_in")
        if not backward:
            out = torch.empty((len(bs), n, H, Dv), dtype=torch.float64, device=DEVICE)
            for t in range(n):
                S = step(S, t)[0]
                out[:, t] = s["scale"] * (q[:, t, :, None, :] @ S)[:, :, 0]
            got.setdefault("out", []).append(out)
            got.setdefault("state_out", []).append(S)
            continue
        do = part("dout")
        block, kept = 64, []
        for t in range(n):
            if t % block == 0:
                kept.append(S)
            S = step(S, t)[0]
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dg, db = torch.empty_like(beta), torch.empty_like(beta)
        G = carried("dstate_out")
        for first in reversed(range(0, n, block)):
            S, inner = kept.pop(), []
            for t in range(first, min(n, first + block)):
                inner.append(step(S, t))
                S = inner[-1][0]
            for t in reversed(range(first, min(n, first + block))):
                S, decayed, wrong = inner.pop()
                kt, bt = k[:, t], beta[:, t, :, None]
                dq[:, t] = s["scale"] * (S @ do[:, t, :, :, None])[..., 0]
                G = G + s["scale"] * q[:, t, :, :, None] * do[:, t, :, None, :]
                du = (kt[:, :, None, :] @ G)[:, :, 0]
                db[:, t] = (du * wrong).sum(-1)
                dv[:, t] = bt * du
                dk[:, t] = (G @ (bt * wrong)[..., None] - decayed @ dv[:, t, :, :, None])[..., 0]
                G = G - kt[..., :, None] * dv[:, t, :, None, :]
                dg[:, t] = (G * decayed).sum((-1, -2))
                G = a[:, t, :, None, None] * G
        for name, t in (("dq", dq), ("dk", dk)):
            got.setdefault(name, []).append(t.unflatten(2, (case["Hk"], share)).sum(3))
        for name, t in (("dv", dv), ("dlog_decay", dg), ("dbeta", db)):
            got.setdefault(name, []).append(t)
        if case["state"]:
            got.setdefault("dstate_in", []).append(G)
    packed = bool(case["lengths"])
    return {k: (torch.cat([x[0] for x in t]) if packed and not k.startswith(("state", "dstate")) else torch.cat(t))
            for k, t in got.items()}
