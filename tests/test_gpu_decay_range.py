"""Decay attention where q k^T or the states are far from 1: small or large enough to leave the range of fp16, with
results well inside it.  Float64 oracle on the rounded inputs.

Tolerances, relative L2 per tensor, u half a unit of the storage type (2^-11, 2^-8): three roundings of at most u each meet
in a result (q k^T, the state, the result), sqrt(3) u < 2 u -- none of which may depend on the size of the
values.  States, fp32: 5e-6, exp of a product rounded in fp32 and sums of up to 64 tokens, over up to 66 chunks.
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
    assert np.isfinite(got).all(), name
    assert np.sqrt((want * want).mean()) > 1e-4, f"{name}: the oracle's values are no fp16 results"
    err = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert err <= tol, f"{name}: relL2 {err:.3e} > {tol:.1e}"


def _rand(shape, size, dtype, seed):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * size).to(DT[dtype])


SHAPES = [
    # N, H, Hk, Dk, Dv: several chunks, segments with sums of their own, rows that are not whole 16-byte pieces
    (200, 3, 3, 64, 64), (2100, 2, 1, 128, 128), (150, 2, 2, 40, 33),
]

PROMPTS = [
    # sizes of q, k, v and scale: states of 1e-6, states of 1e-8, q k^T of 1e-6, states and q k^T beyond 65504
    (30.0, 1e-3, 1e-3, 1.0), (1000.0, 1e-4, 1e-4, 1.0), (1e-3, 1e-3, 1000.0, 0.125), (1e-4, 300.0, 3000.0, 0.125),
    (300.0, 300.0, 1e-3, 0.125),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("sizes", PROMPTS)
@pytest.mark.parametrize("N,H,Hk,Dk,Dv", SHAPES)
def test_prompt(N, H, Hk, Dk, Dv, sizes, dtype):
    print(f"[case] prompt {dtype} N={N} H={H}/{Hk} Dk={Dk} Dv={Dv} sizes {sizes}", flush=True)
    sq, sk, sv, scale = sizes
    q, k, v = _rand((1, N, H, Dk), sq, dtype, 1), _rand((1, N, Hk, Dk), sk, dtype, 2), _rand((1, N, Hk, Dv), sv, dtype, 3)
    a = -torch.tensor([0.003, 0.1, 0.6])[:H].float()
    S0 = torch.randn((1, H, Dk, Dv), generator=torch.Generator().manual_seed(4)) * (sk * sv)
    out, S = fc.decay_attention(q.cuda(), k.cuda(), v.cuda(), a.cuda(), scale=scale, state_in=S0.cuda())
    want, ws = seq.decay_fwd(_f64(q[0]), _f64(k[0]), _f64(v[0]), _f64(a), scale, _f64(S0[0]))
    _close(out[0], want, TOL[dtype], "out")
    S, ws = _f64(S[0]) / (sk * sv), ws / (sk * sv)
    assert np.linalg.norm(S - ws) <= STATE_TOL * np.linalg.norm(ws)


GRADIENTS = [
    # sizes of dout, q, k, v and scale: state gradients of 1e-6, dout v^T of 1e-6, state gradients beyond 65504
    (1e-4, 0.1, 30.0, 30.0, 0.125), (1e-4, 100.0, 100.0, 1e-2, 0.125), (100.0, 1000.0, 3e-4, 3e-4, 1.0),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("sizes", GRADIENTS)
@pytest.mark.parametrize("N,H,Hk,Dk,Dv", SHAPES)
def test_gradients(N, H, Hk, Dk, Dv, sizes, dtype):
    print(f"[case] gradients {dtype} N={N} H={H}/{Hk} Dk={Dk} Dv={Dv} sizes {sizes}", flush=True)
    sd, sq, sk, sv, scale = sizes
    q, k, v = _rand((1, N, H, Dk), sq, dtype, 1), _rand((1, N, Hk, Dk), sk, dtype, 2), _rand((1, N, Hk, Dv), sv, dtype, 3)
    dout = _rand((1, N, H, Dv), sd, dtype, 5)
    a = -torch.tensor([0.003, 0.1, 0.6])[:H].float()
    grads = fc.decay_attention_bwd(q.cuda(), k.cuda(), v.cuda(), a.cuda(), dout.cuda(), scale=scale)
    want = seq.decay_bwd(_f64(dout[0]), _f64(q[0]), _f64(k[0]), _f64(v[0]), _f64(a), scale)
    for name, g, w in zip(("dq", "dk", "dv"), grads, want):
        _close(g[0], w, TOL[dtype], name)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [0.05, 1e-3])
def test_columns_of_different_size(size, dtype):
    # the columns of v, and so of the states and outputs, fall from 1 to 2^-9: each is as good as the largest
    N, D = 200, 64
    q, k, v = _rand((1, N, 1, D), 30.0, dtype, 1), _rand((1, N, 1, D), size, dtype, 2), _rand((1, N, 1, D), 1.0, dtype, 3)
    v = v * torch.exp2(-(torch.arange(D) % 10).float()).to(DT[dtype])
    a = torch.tensor([-0.003])
    out, _ = fc.decay_attention(q.cuda(), k.cuda(), v.cuda(), a.cuda(), scale=1.0)
    want, _ = seq.decay_fwd(_f64(q[0]), _f64(k[0]), _f64(v[0]), _f64(a), 1.0)
    for i in range(D):
        _close(out[0, :, 0, i], want[:, 0, i], TOL[dtype], f"column {i}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("N", [32, 25, 96])
def test_state_of_tokens_long_decayed(N, dtype):
    # only a chunk's first token adds to the state, which has forgotten 24 or 31 times exp(-0.75) when it is returned;
    # 5e-6: exp of a product of up to 24, which is rounded in fp32 (2.5 2^-24 of it)
    q, k, v = (_rand((1, N, 1, 64), 1.0, dtype, s) for s in (1, 2, 3))
    first = N - (N % 32 or 32)
    v[:, :first], v[:, first + 1:] = 0, 0
    a = torch.tensor([-0.75])
    _, S = fc.decay_attention(q.cuda(), k.cuda(), v.cuda(), a.cuda(), scale=1.0)
    _, ws = seq.decay_fwd(_f64(q[0]), _f64(k[0]), _f64(v[0]), _f64(a), 1.0)
    S = _f64(S[0])
    assert np.linalg.norm(ws) > 0 and np.linalg.norm(S - ws) <= STATE_TOL * np.linalg.norm(ws)
