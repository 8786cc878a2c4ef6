"""Float64 oracle of the sequence operators next to the convolution: decay attention and the gated delta rule (their
recurrences, token by token) and the linear product with activation and residual, each with its gradients, and the
root-mean-square norm.

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


def delta_fwd(q, k, v, log_decay, beta, scale, state=None):
    """Gated delta rule over one sequence: q, k (N, Hk, Dk), v (N, H, Dv), log_decay, beta (N, H) -> out, final state.

    u_t = beta_t (v_t - a_t S_{t-1}^T k_t),  S_t = a_t S_{t-1} + k_t u_t^T,  out_t = scale S_t^T q_t,  a = exp(log_decay)
    """
    N, H, Dv = v.shape
    q, k = _heads(q, H), _heads(k, H)
    S = np.zeros((H, q.shape[2], Dv)) if state is None else np.array(state, dtype=np.float64)
    out = np.zeros((N, H, Dv))
    for t in range(N):
        S = np.exp(log_decay[t])[:, None, None] * S
        u = beta[t][:, None] * (v[t] - (S * k[t][:, :, None]).sum(1))
        S = S + k[t][:, :, None] * u[:, None, :]
        out[t] = scale * (S * q[t][:, :, None]).sum(1)
    return out, S


def delta_bwd(dout, q, k, v, log_decay, beta, scale, state=None, dstate=None):
    """Gradients of sum(dout * out) + sum(dstate * final state): dq, dk, dv, dlog_decay, dbeta, dstate_in."""
    N, H, Dv = v.shape
    Hk, Dk = q.shape[1:]
    qh, kh = _heads(q, H), _heads(k, H)
    S = np.zeros((H, Dk, Dv)) if state is None else np.array(state, dtype=np.float64)
    decayed, wrong, after = [], [], []
    for t in range(N):
        D = np.exp(log_decay[t])[:, None, None] * S
        w = v[t] - (D * kh[t][:, :, None]).sum(1)
        S = D + kh[t][:, :, None] * (beta[t][:, None] * w)[:, None, :]
        decayed.append(D), wrong.append(w), after.append(S)
    dq, dk, dv = np.zeros((N, H, Dk)), np.zeros((N, H, Dk)), np.zeros((N, H, Dv))
    dg, db = np.zeros((N, H)), np.zeros((N, H))
    G = np.zeros((H, Dk, Dv)) if dstate is None else np.array(dstate, dtype=np.float64)
    for t in reversed(range(N)):
        dq[t] = scale * (after[t] * dout[t][:, None, :]).sum(2)
        G = G + scale * qh[t][:, :, None] * dout[t][:, None, :]
        du = (G * kh[t][:, :, None]).sum(1)
        db[t] = (du * wrong[t]).sum(1)
        dv[t] = beta[t][:, None] * du
        dk[t] = (G * (beta[t][:, None] * wrong[t])[:, None, :]).sum(2) - (decayed[t] * dv[t][:, None, :]).sum(2)
        G = G - kh[t][:, :, None] * dv[t][:, None, :]
        dg[t] = (G * decayed[t]).sum((1, 2))
        G = np.exp(log_decay[t])[:, None, None] * G
    share = H // Hk
    return dq.reshape(N, Hk, share, Dk).sum(2), dk.reshape(N, Hk, share, Dk).sum(2), dv, dg, db, G


def rms_norm(x, weight=None, eps=1e-6, residual=None):
    """(x + residual) / sqrt(mean of its squares + eps) * weight over the last dimension, and x + residual."""
    t = x if residual is None else x + residual
    y = t / np.sqrt((t * t).mean(-1, keepdims=True) + eps)
    return (y if weight is None else y * weight), t
