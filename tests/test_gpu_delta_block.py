"""The example block (norms, projections, gated delta rule, MLP) as a whole: its single-token form against its prompt
form, and its gradients against differences of the same block in float64 on the CPU."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import sequence as seq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_block_runs_and_its_forms_agree():
    import delta_block
    assert delta_block.main() < 2e-2


def test_block_against_the_oracle():
    import delta_block
    b = delta_block.DeltaBlock(width=128, heads=4, qk_heads=2, dtype=torch.float32, seed=3)
    lengths, H, Hk, D = [40, 0, 85], 4, 2, 32
    T = sum(lengths)
    cu = torch.tensor([0, 40, 40, T], dtype=torch.int32, device="cuda")
    x = torch.randn((T, 128), generator=torch.Generator().manual_seed(2))
    dout = torch.randn((T, 128), generator=torch.Generator().manual_seed(4))
    out, _, kept = b.prompt(x.cuda(), cu, keep=True)
    grads = b.backward(dout.cuda(), kept, cu)
    w = {k: getattr(b, k).double().cpu().numpy() for k in grads if k != "x"}
    n_k, rate = b.n_k.double().cpu().numpy(), b.rate.double().cpu().numpy()

    def forward(x, w):
        proj, _ = seq.linear_fwd(seq.rms_norm(x, w["n_in"])[0], w["w_proj"], w["b_proj"])
        q, k, v, a, g = np.split(proj, np.cumsum(b.sizes)[:-1], axis=1)
        q, k, v = q.reshape(T, Hk, D), k.reshape(T, Hk, D), v.reshape(T, H, D)
        q, k = seq.rms_norm(q, w["n_q"])[0], seq.rms_norm(k, n_k)[0]
        log_decay, beta = -rate * np.logaddexp(0, a), 1 / (1 + np.exp(-g))
        mixed, at = [], 0
        for n in lengths:
            mixed.append(seq.delta_fwd(*(t[at:at + n] for t in (q, k, v, log_decay, beta)), D ** -0.5)[0])
            at += n
        normed = seq.rms_norm(np.concatenate(mixed), w["n_mix"])[0].reshape(T, H * D)
        y, _ = seq.linear_fwd(normed, w["w_out"], None)
        n2, h = seq.rms_norm(y, w["n_mlp"], residual=x)
        act, _ = seq.linear_fwd(n2, w["w_in"], w["b_in"], None, "gelu")
        return seq.linear_fwd(act, w["w_mlp"], None, h)[0]

    x64, d64 = x.double().numpy(), dout.double().numpy()
    want = forward(x64, w)
    # four products, four norms, the rule and two sums in fp32, each a few 2^-24 of its size; a head norm divides by
    # the mixer's outputs, whose size is some tenth of a value's
    assert np.linalg.norm(out.double().cpu().numpy() - want) < 2e-5 * np.linalg.norm(want)
    r = np.random.default_rng(1)
    for name in ("x", *w):
        base = x64 if name == "x" else w[name]
        step = r.standard_normal(base.shape)
        eps = 1e-6
        up, down = (forward(base + s * eps * step, w) if name == "x" else forward(x64, dict(w, **{name: base + s * eps * step}))
                    for s in (1, -1))
        want = ((up - down) * d64).sum() / (2 * eps)
        got = float((grads[name].double().cpu().numpy() * step).sum())
        size = np.linalg.norm(grads[name].double().cpu().numpy()) * np.linalg.norm(step)
        # the gradient's fp32 errors (2e-5 of its norm at most, by the chain above), along a random direction, and the
        # difference's own: eps^2 of third derivatives and 1e-16 / eps of the loss
        assert abs(got - want) < 1e-4 * size, name
