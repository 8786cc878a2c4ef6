"""Gradients of packed sequences that do not fill their buffer: tokens of no sequence keep what they held, whatever the
workspace holds, with and without shared key/value heads; the others equal the float64 oracle.

Tolerance, relative L2 per tensor: three roundings of at most half a unit u of the storage type (2^-24, 2^-11, 2^-8) meet
in a result, sqrt(3) u < 2 u; fp32 storage 5e-6 (exp of a product rounded in fp32, sums of up to 90 tokens).
"""
import numpy as np
import pytest
import torch

import long_fft_convolution_amd as fc
from oracle import sequence as seq

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TOL = {"f32": 5e-6, "f16": 2 * 2.0 ** -11, "bf16": 2 * 2.0 ** -8}
T, MARK = 300, 7.0


def _f64(t):
    return t.double().cpu().numpy()


def _gradients(cu, H, Hk, Dk, Dv, dtype):
    """Inputs on the CPU and dq, dk, dv that held MARK before the call, with a workspace of NaN."""
    g = torch.Generator().manual_seed(H + Dk)
    q, k, v, dout = (torch.randn(s, generator=g).to(DT[dtype]) for s in ((T, H, Dk), (T, Hk, Dk), (T, Hk, Dv), (T, H, Dv)))
    a = -torch.rand(H, generator=g) * 0.1
    grads = [torch.full(t.shape, MARK, dtype=DT[dtype], device="cuda") for t in (q, k, v)]
    B = len(cu) - 1
    ws = torch.full((max(16, fc.fftconv_decay_bwd_workspace_bytes(B, T, H, Hk, Dk, Dv, DT[dtype])),), 255, dtype=torch.uint8,
                    device="cuda")
    fc.fftconv_decay_bwd(dout.cuda(), q.cuda(), k.cuda(), v.cuda(), a.cuda(), *grads, 0.2,
                         cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), workspace=ws)
    return (dout, q, k, v), a, grads


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("H,Hk,Dk,Dv", [(4, 2, 64, 64), (3, 1, 33, 40), (2, 2, 64, 64)])
@pytest.mark.parametrize("cu", [(10, 100, 100, 170, 260), (0, 90, 299), (1, 300), (200, 999), (-5, 60)])
def test_tokens_of_no_sequence_keep_their_gradients(cu, H, Hk, Dk, Dv, dtype):
    print(f"[case] gaps {dtype} H={H}/{Hk} Dk={Dk} Dv={Dv} bounds {cu}", flush=True)
    tensors, a, grads = _gradients(cu, H, Hk, Dk, Dv, dtype)
    bounds = [min(max(c, 0), T) for c in cu]
    for g in grads:
        assert (g[:bounds[0]] == MARK).all() and (g[bounds[-1]:] == MARK).all()
    want = [np.zeros(tuple(g.shape)) for g in grads]
    for i, j in zip(bounds, bounds[1:]):
        for w, part in zip(want, seq.decay_bwd(*(_f64(t[i:j]) for t in tensors), _f64(a), 0.2)):
            w[i:j] = part
    for name, g, w in zip(("dq", "dk", "dv"), grads, want):
        got, w = _f64(g)[bounds[0]:bounds[-1]], w[bounds[0]:bounds[-1]]
        assert np.linalg.norm(got - w) <= TOL[dtype] * np.linalg.norm(w), name


@pytest.mark.parametrize("cu", [(20, 20, 20), (300, 300), (0, 0)])
def test_empty_sequences_write_no_gradient(cu):
    _, _, grads = _gradients(cu, 4, 2, 64, 64, "bf16")
    assert all((g == MARK).all() for g in grads)
