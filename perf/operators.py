"""Cases that measure the sequence-model operators next to the convolution: linear attention with a decay for
each head (prompt, backward, single token) and the matrix product with bias, activation and residual (forward,
backward).

Plain form, per sequence and head with decay d = exp(log_decay) <= 1 and an fp32 state S (Dk x Dv):

    S_t = d S_{t-1} + k_t v_t^T,   out_t = scale * S_t^T q_t
    out = act(x W^T + bias) + residual

Widths are 768 = 12 x 64 and 2560 = 20 x 128 (the gated configurations' H), sequence lengths go from one token
to 131072; decays are exp(-alpha_h), alpha_h log-uniform in [1e-4, 1e-1] like the repository's filters.
"""
import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
MOST_STATE = 131072 * 20 * 128     # tokens x heads x head width of the largest prompt


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a short prompt of odd length, as an interactive user sends it: latency
        dict(name="decay prompt 17", op="decay_fwd", dtype="f16", B=1, N=17, lengths="", H=12, Hk=12, Dk=64, Dv=64,
             state=False),
        # prompts of different lengths packed into one call, shared key/value heads, each with the state of its
        # earlier part (continued prefill); empty and one-token members
        dict(name="decay prompt packed", op="decay_fwd", dtype="bf16", B=12, N=0,
             lengths="0,1,63,64,65,257,1000,1023,1777,2048,4096,6001", H=20, Hk=4, Dk=128, Dv=128, state=True),
        # one long document (genome-scale context)
        dict(name="decay prompt 131072", op="decay_fwd", dtype="bf16", B=1, N=131072, lengths="", H=20, Hk=20, Dk=128,
             Dv=128, state=False),
        # training step of the 2560-wide model
        dict(name="decay backward 4x4096", op="decay_bwd", dtype="bf16", B=4, N=4096, lengths="", H=20, Hk=20, Dk=128,
             Dv=128, state=False),
        # training step of the 768-wide model, odd length, shared key/value heads, gradients of the carried state
        dict(name="decay backward 8x1000", op="decay_bwd", dtype="f16", B=8, N=1000, lengths="", H=12, Hk=4, Dk=64,
             Dv=64, state=True),
        # one user's next token: latency
        dict(name="decay token 1", op="decay_step", dtype="bf16", B=1, H=20, Hk=20, Dk=128, Dv=128),
        # the next token of a full serving batch
        dict(name="decay token 256", op="decay_step", dtype="bf16", B=256, H=20, Hk=20, Dk=128, Dv=128),
        # MLP input product for one user's next token: latency, the weights' bytes
        dict(name="linear 1x2560", op="linear_fwd", dtype="bf16", M=1, K=2560, N=10240, act="gelu", residual=False),
        # in-projection of a few odd prompts in fp32
        dict(name="linear 1000x768 f32", op="linear_fwd", dtype="f32", M=1000, K=768, N=2304, act="silu", residual=True),
        # MLP input product of a training batch
        dict(name="linear 16384x2560", op="linear_fwd", dtype="bf16", M=16384, K=2560, N=10240, act="gelu",
             residual=False),
        # training step of the 768-wide model's out-projection
        dict(name="linear backward 4096x768", op="linear_bwd", dtype="f16", M=4096, K=768, N=768, act="none"),
        # MLP input product of the 2560-wide model, backward
        dict(name="linear backward 8192x2560", op="linear_bwd", dtype="bf16", M=8192, K=2560, N=10240, act="gelu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decay_fwd", "decay_fwd", "decay_bwd", "decay_step", "linear_fwd", "linear_fwd", "linear_bwd"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    if op.startswith("decay"):
        Dk, Dv = rng.choice([(64, 64), (128, 128), (64, 128), (128, 64), (96, 96), (32, 64), (40, 72)])
        Hk = rng.choice([1, 2, 3, 4, 5, 8, 12, 20])
        H = Hk * rng.choice([1, 1, 1, 2, 4])
        if op == "decay_step":
            return dict(op=op, dtype=dtype, B=_log_int(rng, 1, 256), H=H, Hk=Hk, Dk=Dk, Dv=Dv)
        most = MOST_STATE if op == "decay_fwd" else 4 * 4096 * 20 * 128
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
    K = rng.choice([768, 1536, 2560, _log_int(rng, 64, 4096), 8 * _log_int(rng, 8, 512)])
    N = rng.choice([768, 2304, 2560, 10240, _log_int(rng, 64, 10240), 8 * _log_int(rng, 8, 1280)])
    M = _log_int(rng, 1, 16384 if dtype != "f32" else 2048) if op == "linear_fwd" else \
        _log_int(rng, 64, 8192 if dtype != "f32" else 1024)
    case = dict(op=op, dtype=dtype, M=M, K=K, N=N, act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]))
    if op == "linear_fwd":
        case["residual"] = rng.random() < 0.5
    return case


def _lengths(case):
    return [int(s) for s in case["lengths"].split(",")] if case["lengths"] else [case["N"]] * case["B"]


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("decay"):
        H, Hk, Dk, Dv = (case[x] for x in ("H", "Hk", "Dk", "Dv"))
        if case["op"] == "decay_step":
            B = case["B"]
            return dict(bytes=B * (8 * H * Dk * Dv + e * (H * (Dk + Dv) + Hk * (Dk + Dv))), flops=5 * B * H * Dk * Dv)
        T, S = sum(_lengths(case)), case["B"] * H * Dk * Dv * 4
        qo, kv = T * H * (Dk + Dv) * e, T * Hk * (Dk + Dv) * e
        if case["op"] == "decay_fwd":
            return dict(bytes=qo + kv + S * (2 if case["state"] else 1), flops=4 * T * H * Dk * Dv)
        return dict(bytes=qo + T * H * Dk * e + 2 * kv + S * (3 if case["state"] else 0), flops=10 * T * H * Dk * Dv)
    M, K, N = case["M"], case["K"], case["N"]
    if case["op"] == "linear_fwd":
        return dict(bytes=e * (M * K + N * K + N + M * N * (2 if case["residual"] else 1)), flops=2 * M * N * K)
    n_pre = 0 if case["act"] == "none" else 1
    return dict(bytes=e * (2 * M * K + 2 * N * K + N + M * N * (1 + n_pre)), flops=4 * M * N * K)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def randn(*shape, dtype=dt, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32) * scale).to(dtype)

    s = dict(case=dict(case))
    if case["op"].startswith("decay"):
        B, H, Hk, Dk, Dv = (case[x] for x in ("B", "H", "Hk", "Dk", "Dv"))
        u = torch.rand((H,), generator=g, device=DEVICE, dtype=torch.float32)
        s["log_decay"] = -torch.exp(math.log(1e-4) + u * (math.log(1e-1) - math.log(1e-4)))
        s["scale"] = Dk ** -0.5
        if case["op"] == "decay_step":
            lead = (B,)
            slots = B + 3   # a pool with a few free slots, its sequences in any order
            s["slots"] = torch.randperm(slots, generator=g, device=DEVICE)[:B].to(torch.int32)
            s["state"] = randn(slots, H, Dk, Dv, dtype=torch.float32, scale=4.0)
        elif case["lengths"]:
            lens = _lengths(case)
            lead = (sum(lens),)
            s["cu_seqlens"] = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEVICE)
        else:
            lead = (B, case["N"])
        s["q"], s["k"], s["v"] = randn(*lead, H, Dk), randn(*lead, Hk, Dk), randn(*lead, Hk, Dv)
        if case["op"] != "decay_bwd":
            s["out"] = torch.empty((*lead, H, Dv), dtype=dt, device=DEVICE)
        if case["op"] == "decay_fwd":
            s["state_out"] = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=DEVICE)
        if case["op"] == "decay_bwd":
            s["dout"] = randn(*lead, H, Dv)
            s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in ("q", "k", "v"))
        if case.get("state"):
            s["state_in"] = randn(B, H, Dk, Dv, dtype=torch.float32, scale=4.0)
            if case["op"] == "decay_bwd":
                s["dstate_out"] = randn(B, H, Dk, Dv, dtype=torch.float32)
                s["dstate_in"] = torch.empty_like(s["dstate_out"])
        return s
    M, K, N = case["M"], case["K"], case["N"]
    s["x"], s["W"] = randn(M, K), randn(N, K, scale=K ** -0.5)
    if case["op"] == "linear_fwd":
        s["bias"] = randn(N, scale=0.5)
        s["out"] = torch.empty((M, N), dtype=dt, device=DEVICE)
        if case["residual"]:
            s["residual"] = randn(M, N)
    else:
        s["dout"] = randn(M, N)
        s["pre"] = None if case["act"] == "none" else randn(M, N)
        s["dx"], s["dW"] = torch.empty_like(s["x"]), torch.empty_like(s["W"])
        s["dbias"] = torch.empty((N,), dtype=dt, device=DEVICE)
    return s


# ---------------------------------------------------------------- plain forms (32 bits, rounded once)
CHUNK = 128


def _padded(t, state):
    """(B, Hx, N', D) in 32 bits with N' a multiple of CHUNK, zeros behind each sequence's end."""
    t = t.float()
    cu = state.get("cu_seqlens")
    if cu is not None:
        lens = _lengths(state["case"])
        n = max(lens)
        at = cu[:-1, None].long() + torch.arange(n, device=t.device)
        inside = at < cu[1:, None].long()
        t = t[at.clamp(max=max(0, t.shape[0] - 1))] * inside[:, :, None, None]
    t = t.transpose(1, 2)
    return torch.nn.functional.pad(t, (0, 0, 0, -t.shape[2] % CHUNK))


def _unpadded(t, state, dtype):
    """(B, H, N', D) -> the caller's layout and type."""
    t = t.transpose(1, 2)
    cu = state.get("cu_seqlens")
    if cu is None:
        return t[:, :state["case"]["N"]].to(dtype)
    inside = torch.arange(t.shape[1], device=t.device) < (cu[1:] - cu[:-1])[:, None]
    return t[inside].to(dtype)


def _span(t, H):
    """Key/value heads repeated for the heads that share them."""
    return t.repeat_interleave(H // t.shape[1], dim=1)


def _chunks(t):
    return t.reshape(*t.shape[:2], -1, CHUNK, t.shape[-1])


def _power(log_decay, steps):
    """decay^steps, 0 where steps < 0; (H, ...) for steps (...)."""
    p = torch.exp(log_decay.reshape(-1, *[1] * steps.dim()) * steps.clamp(min=0))
    return torch.where(steps < 0, torch.zeros_like(p), p)


def _states_before(U, first, a):
    """State before each chunk from each chunk's own sum U (B, H, n, Dk, Dv): a triangular product over chunks."""
    B, H, n, Dk, Dv = U.shape
    c = torch.arange(n, device=U.device, dtype=torch.float32)
    W = _power(a, CHUNK * (c[:, None] - c[None, :] - 1))                       # (H, n, n)
    S = (W @ U.reshape(B, H, n, Dk * Dv)).reshape(U.shape)
    return S if first is None else S + _power(a, CHUNK * c)[:, :, None, None] * first[:, :, None]


def _plain_decay(x, y, z, a, first, inclusive_from):
    """sum_{j<=i} d^(i-j) (x_i.y_j) z_j + d^(i+inclusive_from) x_i^T first, over (B, H, N', D)."""
    x, y, z = _chunks(x), _chunks(y), _chunks(z)
    i = torch.arange(CHUNK, device=x.device, dtype=torch.float32)
    P = (x @ y.transpose(-1, -2)) * _power(a, i[:, None] - i[None, :])[:, None]
    U = y.transpose(-1, -2) @ (z * _power(a, CHUNK - 1 - i)[:, None, :, None])
    if inclusive_from == 0 and first is not None:
        first = first * torch.exp(-a)[:, None, None]
    S = _states_before(U, first, a)
    o = P @ z + (x * _power(a, i + 1)[:, None, :, None]) @ S
    return o.reshape(*o.shape[:2], -1, o.shape[-1])


def _final_state(k, v, a, first, lens):
    n = torch.arange(k.shape[2], device=k.device, dtype=torch.float32)
    left = lens[:, None] - 1 - n                                                # (B, N')
    w = _power(a, left).transpose(0, 1)                                         # (B, H, N')
    S = (k * w[..., None]).transpose(-1, -2) @ v
    return S if first is None else S + torch.exp(a[None, :] * lens[:, None])[..., None, None] * first


def _plain_decay_run(s):
    case, a, scale = s["case"], s["log_decay"], s["scale"]
    H = case["H"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "decay_step":
        at = s["slots"].long()
        k, v = (_span(s[x].float(), H) for x in ("k", "v"))
        S = s["state"][at] * torch.exp(a)[:, None, None] + k[..., :, None] * v[..., None, :]
        s["state"][at] = S
        out = (s["q"].float()[..., None, :] @ S)[..., 0, :] * scale
        return dict(out=out.to(dt), state=s["state"])
    lens = torch.tensor(_lengths(case), dtype=torch.float32, device=a.device)
    q, k, v = _padded(s["q"], s), _span(_padded(s["k"], s), H), _span(_padded(s["v"], s), H)
    first = s.get("state_in")
    if case["op"] == "decay_fwd":
        out = _unpadded(_plain_decay(q, k, v, a, first, 1) * scale, s, dt)
        return dict(out=out, state_out=_final_state(k, v, a, first, lens))
    do = _padded(s["dout"], s)
    firstT = None if first is None else first.transpose(-1, -2)
    dq = _plain_decay(do, v, k, a, firstT, 1) * scale
    # the gradient of the state runs backwards: the same sums over each sequence read from its end
    n = torch.arange(q.shape[2], device=q.device)
    back = lens[:, None].long() - 1 - n
    rev = back.clamp(min=0)[:, None, :, None]
    live = (back >= 0)[:, None, :, None]

    def turned(t):
        return torch.gather(t, 2, rev.expand(*t.shape[:2], -1, t.shape[3])) * live

    G = s.get("dstate_out")
    GT = None if G is None else G.transpose(-1, -2)
    qr, kr, vr, dor = turned(q * scale), turned(k), turned(v), turned(do)
    dk = turned(_plain_decay(vr, dor, qr, a, GT, 0))
    dv = turned(_plain_decay(kr, qr, dor, a, G, 0))
    shared = (case["Hk"], H // case["Hk"])
    dk, dv = (t.unflatten(1, shared).sum(2) for t in (dk, dv))
    r = dict(dq=_unpadded(dq, s, dt), dk=_unpadded(dk, s, dt), dv=_unpadded(dv, s, dt))
    if case["state"]:
        up = _power(a, n + 1.0) * 1.0
        w = (up[None] * (n < lens[:, None].long())[:, None])[..., None]
        r["dstate_in"] = (q * scale * w).transpose(-1, -2) @ do + \
            torch.exp(a[None, :] * lens[:, None])[..., None, None] * G
    return r


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _linear_run(s, real):
    """The linear operators in `real` arithmetic (float32, or float64 for exact())."""
    case = s["case"]
    x, W = s["x"].to(real), s["W"].to(real)
    if case["op"] == "linear_fwd":
        z = _act(x @ W.T + s["bias"].to(real), case["act"])
        return dict(out=z + s["residual"].to(real) if case["residual"] else z)
    dz = s["dout"].to(real)
    if case["act"] != "none":
        dz = dz * _act_slope(s["pre"].to(real), case["act"])
    return dict(dx=dz @ W, dW=dz.T @ x, dbias=dz.sum(0))


# ---------------------------------------------------------------- one pass
def run(state):
    if own:
        return _own_run(state)
    if state["case"]["op"].startswith("decay"):
        return _plain_decay_run(state)
    dt = DTYPES[state["case"]["dtype"]]
    return {k: v.to(dt) for k, v in _linear_run(state, torch.float32).items()}


def _workspace(state, nbytes):
    """The call's scratch, kept with the state as a program keeps it."""
    if "workspace" not in state:
        state["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device=DEVICE) if nbytes else None
    return state["workspace"]


def _own_run(s):
    import long_fft_convolution_amd as fc

    case, op = s["case"], s["case"]["op"]
    if op == "decay_step":
        fc.fftconv_decay_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["out"], s["scale"], s["slots"])
        return dict(out=s["out"], state=s["state"])
    if op == "decay_fwd":
        if "workspace" not in s:
            _workspace(s, fc.fftconv_decay_fwd_workspace_bytes(
                case["B"], s["q"].numel() // (case["H"] * case["Dk"]), case["H"], case["Dk"], case["Dv"],
                s["q"].dtype))
        fc.fftconv_decay_fwd(s["q"], s["k"], s["v"], s["log_decay"], s["out"], s["scale"],
                             state_in=s.get("state_in"), state_out=s["state_out"], cu_seqlens=s.get("cu_seqlens"),
                             workspace=s["workspace"])
        return dict(out=s["out"], state_out=s["state_out"])
    if op == "decay_bwd":
        if "workspace" not in s:
            _workspace(s, fc.fftconv_decay_bwd_workspace_bytes(
                case["B"], s["q"].numel() // (case["H"] * case["Dk"]), case["H"], case["Hk"], case["Dk"],
                case["Dv"], s["q"].dtype))
        fc.fftconv_decay_bwd(s["dout"], s["q"], s["k"], s["v"], s["log_decay"], s["dq"], s["dk"], s["dv"], s["scale"],
                             state_in=s.get("state_in"), dstate_out=s.get("dstate_out"),
                             dstate_in=s.get("dstate_in"), cu_seqlens=s.get("cu_seqlens"), workspace=s["workspace"])
        r = dict(dq=s["dq"], dk=s["dk"], dv=s["dv"])
        return dict(r, dstate_in=s["dstate_in"]) if case["state"] else r
    if op == "linear_fwd":
        if "workspace" not in s:
            _workspace(s, fc.fftconv_linear_fwd_workspace_bytes(case["M"], case["N"], case["K"], s["x"].dtype))
        fc.fftconv_linear_fwd(s["x"], s["W"], s["bias"], s.get("residual"), s["out"], activation=case["act"],
                              workspace=s["workspace"])
        return dict(out=s["out"])
    if "workspace" not in s:
        _workspace(s, fc.fftconv_linear_bwd_workspace_bytes(case["M"], case["N"], case["K"], s["x"].dtype))
    fc.fftconv_linear_bwd(s["dout"], s["x"], s["W"], s["pre"], s["dx"], s["dW"], s["dbias"], activation=case["act"],
                          workspace=s["workspace"])
    return dict(dx=s["dx"], dW=s["dW"], dbias=s["dbias"])


# ---------------------------------------------------------------- 64 bits, token by token
def exact(case, seed):
    if not case["op"].startswith("decay"):
        if case["M"] * case["K"] * case["N"] > 5e11:
            return None
        return _linear_run(prepare(case, seed), torch.float64)
    s = prepare(case, seed)
    H, Dk, Dv = case["H"], case["Dk"], case["Dv"]
    share = H // case["Hk"]
    d = torch.exp(s["log_decay"].double())[:, None, None]
    if case["op"] == "decay_step":
        state = s["state"].double()
        out = torch.empty((case["B"], H, Dv), dtype=torch.float64, device=DEVICE)
        for b, slot in enumerate(s["slots"].tolist()):
            kv = s["k"][b].double()[:, :, None] * s["v"][b].double()[:, None, :]
            state[slot] = d * state[slot] + kv.repeat_interleave(share, 0)
            out[b] = s["scale"] * (s["q"][b].double()[:, :, None] * state[slot]).sum(1)
        return dict(out=out, state=state)
    lens = _lengths(case)
    # (sequences walked together) x (tokens walked one by one)
    groups = [(list(range(case["B"])), None)] if not case["lengths"] else [([b], b) for b in range(case["B"])]
    steps = case["N"] if not case["lengths"] else sum(lens)
    each = case["B"] * H * Dk * Dv * 16e-12 if not case["lengths"] else H * Dk * Dv * 16e-12
    if steps * (60e-6 + each) * (3 if case["op"] == "decay_bwd" else 1) > 20:
        return None
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    backward = case["op"] == "decay_bwd"
    got = {}
    for bs, b in groups:
        def part(name):
            t = s[name].double()
            t = t if b is None else t[ends[b]:ends[b + 1]][None]
            return t.repeat_interleave(share, 2) if name in ("k", "v") else t

        def carried(name):
            return s[name][bs].double() if s.get(name) is not None else \
                torch.zeros((len(bs), H, Dk, Dv), dtype=torch.float64, device=DEVICE)

        q, k, v = part("q"), part("k"), part("v")
        S, n = carried("state_in"), q.shape[1]
        if not backward:
            out = torch.empty((len(bs), n, H, Dv), dtype=torch.float64, device=DEVICE)
            for t in range(n):
                S = d * S + k[:, t, :, :, None] * v[:, t, :, None, :]
                out[:, t] = s["scale"] * (q[:, t, :, None, :] @ S)[:, :, 0]
            got.setdefault("out", []).append(out)
            got.setdefault("state_out", []).append(S)
            continue
        do = part("dout")
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        for t in range(n):
            S = d * S + k[:, t, :, :, None] * v[:, t, :, None, :]
            dq[:, t] = s["scale"] * (S @ do[:, t, :, :, None])[..., 0]
        G = carried("dstate_out")
        for t in reversed(range(n)):
            G = G + s["scale"] * q[:, t, :, :, None] * do[:, t, :, None, :]
            dk[:, t] = (G @ v[:, t, :, :, None])[..., 0]
            dv[:, t] = (k[:, t, :, None, :] @ G)[:, :, 0]
            G = d * G
        got.setdefault("dq", []).append(dq)
        for name, t in (("dk", dk), ("dv", dv)):
            got.setdefault(name, []).append(t.unflatten(2, (case["Hk"], share)).sum(3))
        if case["state"]:
            got.setdefault("dstate_in", []).append(G)
    packed = bool(case["lengths"])
    return {k: (torch.cat([x[0] for x in t]) if packed and not k.startswith(("state", "dstate")) else torch.cat(t))
            for k, t in got.items()}
