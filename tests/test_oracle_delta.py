"""The float64 oracle of the gated delta rule: its limits, the closed form of one chunk, and its gradients against
differences of its forward pass (CPU)."""
import numpy as np
import pytest

from oracle import sequence as seq


def _inputs(N, H, Hk, Dk, Dv, seed):
    r = np.random.default_rng(seed)
    k = r.standard_normal((N, Hk, Dk))
    return (r.standard_normal((N, Hk, Dk)), k / np.linalg.norm(k, axis=-1, keepdims=True), r.standard_normal((N, H, Dv)),
            -np.exp(r.uniform(-4, 0, (N, H))), r.uniform(0, 1.5, (N, H)), r.standard_normal((H, Dk, Dv)))


def test_without_decay_a_written_key_returns_its_value():
    q, k, v, a, b, S0 = _inputs(5, 2, 2, 4, 3, 1)
    out, S = seq.delta_fwd(k, k, v, 0 * a, 1 + 0 * b, 1.0, S0)
    np.testing.assert_allclose(out, v, atol=1e-12)          # beta 1, |k| = 1: S_t^T k_t = v_t


def test_a_cleared_state_sees_its_token_alone():
    q, k, v, a, b, S0 = _inputs(4, 4, 2, 3, 3, 2)
    out, S = seq.delta_fwd(q, k, v, np.full_like(a, -np.inf), b, 0.5, S0)
    q4, k4 = (np.repeat(t, 2, axis=1) for t in (q, k))
    np.testing.assert_allclose(out, 0.5 * (q4 * k4).sum(-1, keepdims=True) * b[..., None] * v, rtol=1e-12)


def test_linear_system_of_a_chunk():
    N, H = 7, 2
    q, k, v, a, b, S0 = _inputs(N, H, H, 5, 4, 3)
    out, S = seq.delta_fwd(q, k, v, a, b, 0.7, S0)
    for h in range(H):
        G = np.cumsum(a[:, h])
        D = np.exp(G[:, None] - G[None, :])
        C = np.tril(D * (k[:, h] @ k[:, h].T), -1)
        w = np.linalg.solve(np.eye(N) + C * b[:, h], v[:, h] - np.exp(G)[:, None] * (k[:, h] @ S0[h]))
        u = b[:, h, None] * w
        want = 0.7 * (np.exp(G)[:, None] * (q[:, h] @ S0[h]) + np.tril(D * (q[:, h] @ k[:, h].T)) @ u)
        np.testing.assert_allclose(out[:, h], want, rtol=1e-10, atol=1e-12)
        np.testing.assert_allclose(S[h], np.exp(G[-1]) * S0[h] + (np.exp(G[-1] - G)[:, None] * k[:, h]).T @ u, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2), (3, 1)])
def test_gradients_against_differences(H, Hk):
    N, Dk, Dv, scale, eps = 6, 3, 4, 0.7, 1e-5
    q, k, v, a, b, S0 = _inputs(N, H, Hk, Dk, Dv, 3)
    r = np.random.default_rng(4)
    dout, dS = r.standard_normal((N, H, Dv)), r.standard_normal((H, Dk, Dv))
    grads = seq.delta_bwd(dout, q, k, v, a, b, scale, S0, dS)

    def loss():
        out, S = seq.delta_fwd(q, k, v, a, b, scale, S0)
        return (out * dout).sum() + (S * dS).sum()

    for t, g in zip((q, k, v, a, b, S0), grads):
        assert g.shape == t.shape
        for i in range(0, t.size, max(1, t.size // 11)):
            old = t.flat[i]
            t.flat[i] = old + eps
            up = loss()
            t.flat[i] = old - eps
            down = loss()
            t.flat[i] = old
            # central difference: eps^2 of a third derivative of size some tens, and 1e-16 / eps of the loss
            assert abs((up - down) / (2 * eps) - g.flat[i]) < 1e-7 * (1 + abs(up))
