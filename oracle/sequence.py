"""Float64 oracle of the sequence operators next to the convolution: decay attention (its recurrence, token by
token) and the linear product with activation and residual, each with its gradients.

Plain definitions in numpy, sharing no code with the HIP path:

    S_t = d S_{t-1} + k_t v_t^T,   out_t = scale S_t^T q_t,   d = exp(log_decay)
    out = act(x W^T + bias) + residual
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def _heads(t, H):
    """Key/value heads repeated for the heads that share them: (N, Hk, D) -> (N, H, D)."""
    return np.repeat(t, H // t.shape[1], axis=1)


def _decay(log_decay):
    with np.errstate(over="ignore"):
        return np.exp(np.asarray(log_decay, dtype=np.float64))[:, None, None]


def decay_fwd(q, k, v, log_decay, scale, state=None):
    """One sequence: q (N, H, Dk), k (N, Hk, Dk), v (N, Hk, Dv) -> out (N, H, Dv), final state (H, Dk, Dv)."""
    N, H, Dk = q.shape
    k, v, d = _heads(k, H), _heads(v, H), _decay(log_decay)
    S = np.zeros((H, Dk, v.shape[2])) if state is None else np.array(state, dtype=np.float64)
    out = np.zeros((N, H, v.shape[2]))
    for t in range(N):
        S = d * S + k[t][:, :, None] * v[t][:, None, :]
        out[t] = scale * np.einsum("hk,hkv->hv", q[t], S)
    return out, S


def decay_bwd(dout, q, k, v, log_decay, scale, state=None, dstate=None):
    """Gradients of sum(dout * out) + sum(dstate * final state): dq, dk, dv, dstate_in."""
    N, H, Dk = q.shape
    Hk, Dv = k.shape[1], v.shape[2]
    kh, vh, d = _heads(k, H), _heads(v, H), _decay(log_decay)
    S = np.zeros((H, Dk, Dv)) if state is None else np.array(state, dtype=np.float64)
    dq, dk, dv = np.zeros((N, H, Dk)), np.zeros((N, H, Dk)), np.zeros((N, H, Dv))
    for t in range(N):
        S = d * S + kh[t][:, :, None] * vh[t][:, None, :]
        dq[t] = scale * np.einsum("hkv,hv->hk", S, dout[t])
    G = np.zeros((H, Dk, Dv)) if dstate is None else np.array(dstate, dtype=np.float64)
    for t in reversed(range(N)):
        G = G + scale * q[t][:, :, None] * dout[t][:, None, :]
        dk[t] = np.einsum("hkv,hv->hk", G, vh[t])
        dv[t] = np.einsum("hkv,hk->hv", G, kh[t])
        G = d * G
    shared = H // Hk
    return dq, dk.reshape(N, Hk, shared, Dk).sum(2), dv.reshape(N, Hk, shared, Dv).sum(2), G


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0)
    if name == "gelu":
        return 0.5 * z * (1 + _erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * 0.5 * (1 + np.tanh(0.5 * z))
    return np.array(z)


def act_slope(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * (1 + _erf(z / math.sqrt(2))) + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = 0.5 * (1 + np.tanh(0.5 * z))
        return p * (1 + z * (1 - p))
    return np.ones_like(z)


def linear_fwd(x, W, bias=None, residual=None, activation="none"):
    """(out, pre)."""
    pre = x @ W.T
    if bias is not None:
        pre = pre + bias
    out = act(pre, activation)
    return (out if residual is None else out + residual), pre


def linear_bwd(dout, x, W, pre=None, activation="none"):
    """(dx, dW, dbias)."""
    dz = dout if activation == "none" else dout * act_slope(pre, activation)
    return dz @ W, dz.T @ x, dz.sum(0)
