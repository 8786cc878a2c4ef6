"""Prompts of the gated delta rule that are cut into segments: key widths that leave columns of a segment's map without a
key, whatever the workspace holds, and states of a pool that is updated in place.

Tolerances, relative L2 against the float64 oracle on the rounded inputs: 16-bit results 1.5 half units of their type (2^-11,
2^-8: the result's rounding and, below it, those of its operands), fp32 results 5e-6 (products of exact terms accumulated in
fp32 over at most 80 chunks of 64 tokens, whose errors the decay forgets)."""
import numpy as np
import pytest
import torch

import long_fft_convolution_amd as fc
from oracle import sequence as seq

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TOL = {"f32": 5e-6, "f16": 1.5 * 2.0 ** -11, "bf16": 1.5 * 2.0 ** -8}
FP32 = 5e-6


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


def _garbage(n):
    """Workspace of NaNs."""
    return torch.full((max(1, n),), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("Dk,Dv", [(129, 40), (160, 64), (192, 256), (193, 72), (100, 64), (40, 96)])
def test_widths_between_the_padded_ones(Dk, Dv, dtype):
    """2100 tokens are cut in four; a map has rows of 64, 128 or 256 columns, of which Dk are of keys."""
    print(f"[case] cut {dtype} Dk={Dk} Dv={Dv}", flush=True)
    B, N, H = 1, 2100, 2
    ins = _inputs((B, N), H, 1, Dk, Dv, dtype, Dk)
    S0 = torch.randn((B, H, Dk, Dv), generator=torch.Generator().manual_seed(5)).cuda()
    out, S = torch.empty_like(ins[2]), torch.empty_like(S0)
    ws = _garbage(fc.fftconv_delta_fwd_workspace_bytes(B, N, H, 1, Dk, Dv, DT[dtype]))
    fc.fftconv_delta_fwd(*ins, out, 0.25, S0, S, workspace=ws)
    want, wS = seq.delta_fwd(*(_f64(t[0]) for t in ins), 0.25, _f64(S0[0]))
    _close(out[0], want, TOL[dtype], "out")
    _close(S[0], wS, FP32, "state")


@pytest.mark.parametrize("lens", [(2624,) * 9, (2600, 900, 5000, 64, 1, 3333, 2624, 4095, 5002), (0, 9000, 513, 2049, 3000, 2600, 2600, 2600, 1)])
@pytest.mark.parametrize("H,D", [(4, 128), (7, 64)])
def test_a_pool_in_place_as_one_beside(lens, H, D):
    """More segments than CUs, other work on the chip: where the last segment of a sequence ends before the first one starts,
    the first one still starts from the state that the caller gave."""
    print(f"[case] in place {lens} H={H} D={D}", flush=True)
    B, T = len(lens), sum(lens)
    cu = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32).cuda()
    ins = _inputs((T,), H, H, D, D, "bf16", T)
    pool = torch.randn((B + 2, H, D, D), generator=torch.Generator().manual_seed(3)).cuda()
    slots = torch.randperm(B + 2, generator=torch.Generator().manual_seed(4))[:B].to(torch.int32)
    slots[6] = -1
    where, ws = slots.cuda(), _garbage(fc.fftconv_delta_fwd_workspace_bytes(B, T, H, H, D, D, torch.bfloat16))
    want, after = torch.empty_like(ins[2]), pool.clone()
    fc.fftconv_delta_fwd(*ins, want, 0.25, pool, after, where, cu, ws)
    out, inplace = torch.empty_like(want), [pool.clone() for _ in range(4)]
    work, other = torch.randn((2048, 2048), device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        for _ in range(8):
            work = torch.nn.functional.normalize(work @ work)
    for p in inplace:
        fc.fftconv_delta_fwd(*ins, out, 0.25, p, p, where, cu, ws)
        assert torch.equal(out, want) and torch.equal(p, after)
    for b in (0, 2):      # (cut in several)
        x, y = int(cu[b]), int(cu[b + 1])
        ref, wS = seq.delta_fwd(*(_f64(t[x:y]) for t in ins), 0.25, _f64(pool[int(slots[b])]))
        _close(want[x:y], ref, TOL["bf16"], f"out[{b}]")
        _close(after[int(slots[b])], wS, FP32, f"state[{b}]")
