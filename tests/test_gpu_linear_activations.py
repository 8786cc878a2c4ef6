"""Activations of the linear product and their slopes value by value, through an identity product (exact), against float64.

Bounds, as the header states them.  fp32 storage: relative error 2^-20 of GELU and SiLU (exp and reciprocal of the hardware
an ulp or two each, the fit of the normal distribution's tail 3e-7, a handful of fp32 roundings); of the tanh form
2^-20 and 2^-22 more for each unit of the logistic function's argument, which is rounded.  16-bit storage: 2^-15
and the one rounding to the storage type.  A slope's error is of the size of its two summands.  Smallest numbers:
half of fp16's last subnormal place, 2^-126 elsewhere.
"""
import numpy as np
import pytest
import torch
from scipy.special import erfc, expit

import long_fft_convolution_amd as fc

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}
FAR = {"gelu": 12.0, "gelu_tanh": 8.0, "silu": 80.0}
C = np.sqrt(2 / np.pi)


def _arguments(act, dtype):
    z = np.concatenate([np.linspace(-FAR[act], FAR[act], 4096), np.linspace(-4, 4, 2048), [0.0, -0.75, 0.75, 1e-3, -1e-3] + [0.0] * 59])
    return torch.from_numpy(z).to(DT[dtype]).view(-1, 64)


def _parts(z, act):
    """The factor p of the value z p, and the slope's second summand."""
    if act == "gelu":
        return 0.5 * erfc(-z / np.sqrt(2)), z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    if act == "silu":
        return expit(z), z * expit(z) * expit(-z)
    w = 2 * C * (z + 0.044715 * z ** 3)
    return expit(w), z * expit(w) * expit(-w) * 2 * C * (1 + 3 * 0.044715 * z * z)


def _relative(z, act, dtype):
    if dtype != "f32":
        return 2.0 ** -15
    return 2.0 ** -20 + (np.abs(2 * C * (z + 0.044715 * z ** 3)) * 2.0 ** -22 if act == "gelu_tanh" else 0)


def _check(got, want, size, rel, dtype):
    got = got.double().cpu().numpy()
    over = np.abs(got - want) - (U[dtype] * np.abs(want) + (1 + U[dtype]) * rel * size + TINY[dtype])
    i = np.unravel_index(np.argmax(over), over.shape)
    assert (over <= 0).all(), f"worst at {i}: {got[i]!r} for {want[i]!r}, beyond by {over[i]:.2e} ({(over > 0).mean():.1%} of values)"


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_values(act, dtype):
    x = _arguments(act, dtype)
    z = x.double().numpy()
    eye = torch.eye(64, dtype=DT[dtype]).cuda()
    p, _ = _parts(z, act)
    want, rel = z * p, _relative(z, act, dtype)
    _check(fc.linear_act(x.cuda(), eye, None, None, act), want, np.abs(want), rel, dtype)
    _check(fc.linear_act(x[:2].cuda(), eye, None, None, act), want[:2], np.abs(want[:2]), rel if np.isscalar(rel) else rel[:2], dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_slopes(act, dtype):
    x = _arguments(act, dtype)
    z = x.double().numpy()
    eye, ones = torch.eye(64, dtype=DT[dtype]).cuda(), torch.ones_like(x).cuda()
    dx, _, _ = fc.linear_act_bwd(ones, x.cuda(), eye, x.cuda(), act)
    p, n = _parts(z, act)
    _check(dx, p + n, p + np.abs(n), _relative(z, act, dtype), dtype)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_nan_and_infinity(act):
    x = torch.tensor([[float("nan"), float("inf"), 1.0, -1.0]])
    out = fc.linear_act(torch.ones((1, 1)).cuda(), torch.ones((4, 1)).cuda(), (x[0] - 1.0).cuda(), None, act).cpu()[0]
    assert out[0].isnan() and out[1] == float("inf") and out[2:].isfinite().all()
    if act in ("gelu", "gelu_tanh", "silu"):
        _, _, db = fc.linear_act_bwd(torch.ones((1, 4)).cuda(), torch.ones((1, 1)).cuda(), torch.ones((4, 1)).cuda(), x.cuda(), act)
        assert db.cpu()[0].isnan() and db.cpu()[1] == 1.0
