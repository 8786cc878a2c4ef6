"""What the gated delta rule's results see beside their own rounding, element by element."""
import numpy as np
import pytest
import torch

import long_fft_convolution_amd as fc

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
LEAST = {"f16": 2.0 ** -25, "bf16": 0.0}


def _f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("N,D", [(64, 128), (64, 64), (37, 40), (1, 128)])
def test_products_of_queries_and_keys_are_not_rounded_to_the_storage_type(N, D, dtype):
    """A prompt of one chunk without a state takes all of its output through P_ij = scale exp(G_i - G_j) q_i . k_j and u.

    Each value is off by the result's rounding (at most half a step, 2^-8 or 2^-11 of it) and by d_i = sum over j of |P_ij u_j|
    times what two terms leave: the first term cuts off at 8 bits (rest below 2^-7), the second is rounded (2^-8 of the rest,
    2^-15 in all) for each of P and u, and the product of the two second terms (2^-14) is left out, 2^-13 together; fp32 sums
    of up to 128 products and the inverse's chains of 64 are below 2^-16.  2^-12 covers both.  fp16 results below 2^-14 have
    steps of 2^-24, whatever their size: half of one, 2^-25, is allowed beside the relative half step."""
    H = 3
    g = torch.Generator().manual_seed(N + D)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    k = r(1, N, H, D)
    q, k, v = (t.to(DT[dtype]) for t in (r(1, N, H, D), k / k.norm(dim=-1, keepdim=True), r(1, N, H, D)))
    a, beta = (-torch.exp(r(1, N, H) - 3)).float(), torch.sigmoid(r(1, N, H)).float()
    out, _ = fc.delta_attention(q.cuda(), k.cuda(), v.cuda(), a.cuda(), beta.cuda(), scale=0.25)
    got = _f64(out[0])
    Q, K, V, A, b = (_f64(t[0]) for t in (q, k, v, a, beta))
    for h in range(H):
        G = np.cumsum(A[:, h])
        decay = np.tril(np.exp(np.minimum(G[:, None] - G[None, :], 0)))
        kk, P = decay * (K[:, h] @ K[:, h].T), 0.25 * decay * (Q[:, h] @ K[:, h].T)
        u = np.zeros((N, D))
        for t in range(N):
            u[t] = b[t, h] * (V[t, h] - kk[t, :t] @ u[:t])
        want, d = P @ u, 2.0 ** -12 * (np.abs(P) @ np.abs(u))
        over = np.abs(got[:, h] - want) - (HALF[dtype] * (np.abs(want) + d) + d + LEAST[dtype])
        i = np.unravel_index(over.argmax(), over.shape)
        assert over[i] <= 0, f"head {h}, token {i[0]}, value {i[1]}: {got[:, h][i]!r}, not {want[i]!r}, {(over > 0).sum()} such"
