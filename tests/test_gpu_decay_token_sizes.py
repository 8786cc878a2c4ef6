"""Decay attention where tokens of one chunk differ in size: the fp16 walks scale a chunk's terms by the largest of all of
its tokens.  Float64 oracle on the rounded inputs; q k^T and the states stay inside the normal numbers of fp16.

Tolerances, relative L2 per tensor, u half a unit of the storage type (2^-11, 2^-8): three roundings of at most u each meet
in a result, sqrt(3) u < 2 u; states, fp32, 5e-6 (exp of a product rounded in fp32, sums of up to 130 tokens).
"""
import numpy as np
import pytest
import torch

import long_fft_convolution_amd as fc
from oracle import sequence as seq

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
TOL = {"f16": 2 * 2.0 ** -11, "bf16": 2 * 2.0 ** -8}
STATE_TOL = 5e-6


def _f64(t):
    return t.double().cpu().numpy()


def _close(got, want, tol, name):
    got = _f64(got)
    err = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert err <= tol, f"{name}: relL2 {err:.3e} > {tol:.1e}"


def _sizes(pattern, N):
    """A factor for each token."""
    if pattern == "eights":          # groups of 8 tokens
        return torch.tensor([1.0, 8.0, 64.0, 0.125]).repeat_interleave(8).repeat(N // 32 + 1)[:N]
    if pattern == "one":             # one large token a chunk, at another place in each
        s = torch.ones(N)
        s[torch.arange(0, N, 37)] = 100.0
        return s
    return torch.exp2(torch.randint(-3, 7, (N,), generator=torch.Generator().manual_seed(N)).float())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("pattern", ["eights", "one", "random"])
@pytest.mark.parametrize("N,H,D", [(24, 2, 64), (130, 3, 64), (100, 2, 128), (70, 2, 33)])
def test_prompt_and_gradients(N, H, D, pattern, dtype):
    print(f"[case] token sizes {pattern} {dtype} N={N} H={H} D={D}", flush=True)
    g = torch.Generator().manual_seed(5)
    q, k, v, dout = (torch.randn((1, N, H, D), generator=g) for _ in range(4))
    s = _sizes(pattern, N)[None, :, None, None] / 16         # results below 65504
    a = -torch.tensor([0.003, 0.1, 0.6])[:H]
    q, k, v, dout = (t.to(DT[dtype]) for t in (q * s, k, v * s, dout * s))
    out, S = fc.decay_attention(q.cuda(), k.cuda(), v.cuda(), a.cuda(), scale=0.125)
    x = [_f64(t[0]) for t in (q, k, v)]
    want, ws = seq.decay_fwd(*x, _f64(a), 0.125)
    _close(out[0], want, TOL[dtype], "out")
    for h in range(H):
        _close(S[0, h], ws[h], STATE_TOL, f"state of head {h}")
    want = seq.decay_bwd(_f64(dout[0]), *x, _f64(a), 0.125)
    for name, got, w in zip(("dq", "dk", "dv"), fc.decay_attention_bwd(q.cuda(), k.cuda(), v.cuda(), a.cuda(), dout.cuda(), 0.125), want):
        _close(got[0], w, TOL[dtype], name)
