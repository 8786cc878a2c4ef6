"""The float64 oracle of decay attention and the linear product: closed forms, and its gradients against
differences of its forward pass (CPU)."""
import numpy as np
import pytest

from oracle import sequence as seq


def _inputs(N, H, Hk, Dk, Dv, seed):
    r = np.random.default_rng(seed)
    return (r.standard_normal((N, H, Dk)), r.standard_normal((N, Hk, Dk)), r.standard_normal((N, Hk, Dv)),
            -np.exp(r.uniform(-4, 0, H)), r.standard_normal((H, Dk, Dv)))


def test_recurrence_is_the_masked_sum():
    N, H, Hk, Dk, Dv = 9, 4, 2, 5, 3
    q, k, v, a, S0 = _inputs(N, H, Hk, Dk, Dv, 1)
    out, S = seq.decay_fwd(q, k, v, a, 0.3, S0)
    for h in range(H):
        kv = h // 2
        for t in range(N):
            want = sum(np.exp(a[h] * (t - j)) * (q[t, h] @ k[j, kv]) * v[j, kv] for j in range(t + 1))
            want = 0.3 * (want + np.exp(a[h] * (t + 1)) * q[t, h] @ S0[h])
            np.testing.assert_allclose(out[t, h], want, rtol=1e-12, atol=1e-12)
        want = np.exp(a[h] * N) * S0[h] + sum(np.exp(a[h] * (N - 1 - j)) * np.outer(k[j, kv], v[j, kv]) for j in range(N))
        np.testing.assert_allclose(S[h], want, rtol=1e-12, atol=1e-12)


def test_empty_sequence_and_limits_of_the_decay():
    q, k, v, a, S0 = _inputs(4, 2, 2, 3, 3, 2)
    out, S = seq.decay_fwd(q[:0], k[:0], v[:0], a, 1.0, S0)
    assert out.shape == (0, 2, 3) and np.array_equal(S, S0)
    out, _ = seq.decay_fwd(q, k, v, np.full(2, -np.inf), 1.0, S0)       # d = 0: each token sees itself alone
    np.testing.assert_allclose(out, (q * k).sum(-1, keepdims=True) * v, rtol=1e-12)
    out, S = seq.decay_fwd(q, k, v, np.zeros(2), 1.0)                    # d = 1: plain running sums
    np.testing.assert_allclose(S, np.einsum("nhk,nhv->hkv", k, v), rtol=1e-12)


@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2), (3, 1)])
def test_decay_gradients_against_differences(H, Hk):
    N, Dk, Dv, scale, eps = 6, 3, 4, 0.7, 1e-5
    q, k, v, a, S0 = _inputs(N, H, Hk, Dk, Dv, 3)
    r = np.random.default_rng(4)
    dout, dS = r.standard_normal((N, H, Dv)), r.standard_normal((H, Dk, Dv))
    grads = seq.decay_bwd(dout, q, k, v, a, scale, S0, dS)

    def loss():
        out, S = seq.decay_fwd(q, k, v, a, scale, S0)
        return (out * dout).sum() + (S * dS).sum()

    for t, g in zip((q, k, v, S0), grads):
        for i in range(0, t.size, max(1, t.size // 11)):
            old = t.flat[i]
            t.flat[i] = old + eps
            up = loss()
            t.flat[i] = old - eps
            down = loss()
            t.flat[i] = old
            # central difference of a quadratic form: exact up to 1e-16 / eps of the loss's size
            assert abs((up - down) / (2 * eps) - g.flat[i]) < 1e-8 * (1 + abs(up))


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_linear_gradients_against_differences(name):
    r = np.random.default_rng(5)
    x, W, b, res, dout = (r.standard_normal(s) for s in ((5, 4), (3, 4), (3,), (5, 3), (5, 3)))
    out, pre = seq.linear_fwd(x, W, b, res, name)
    np.testing.assert_allclose(out - res, seq.act(pre, name), rtol=1e-12, atol=1e-12)
    grads = seq.linear_bwd(dout, x, W, pre, name)
    eps = 1e-5
    for t, g in zip((x, W, b), grads):
        for i in range(t.size):
            old = t.flat[i]
            t.flat[i] = old + eps
            up = (seq.linear_fwd(x, W, b, res, name)[0] * dout).sum()
            t.flat[i] = old - eps
            down = (seq.linear_fwd(x, W, b, res, name)[0] * dout).sum()
            t.flat[i] = old
            # eps^2 of the third derivative plus 1e-16 / eps of the loss
            assert abs((up - down) / (2 * eps) - g.flat[i]) < 1e-7 * (1 + abs(up))


def test_activations_at_large_arguments():
    z = np.array([-1e4, -50.0, 0.0, 50.0, 1e4])
    for name in ("relu", "gelu", "gelu_tanh", "silu"):
        np.testing.assert_allclose(seq.act(z, name), np.maximum(z, 0), atol=1e-15)
        s = seq.act_slope(z, name)
        assert np.isfinite(s).all() and s[0] == 0 and abs(s[-1] - 1) < 1e-12
