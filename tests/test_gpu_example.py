"""The example block (projections, decay attention, MLP) as a whole: its single-token form against its prompt form, and
its gradients against differences of the same block in float64 on the CPU."""
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
    import decay_block
    assert decay_block.main() < 2e-2


def test_block_against_the_oracle():
    import decay_block
    b = decay_block.DecayBlock(width=128, heads=4, kv_heads=2, dtype=torch.float32, seed=3)
    lengths = [40, 0, 25]
    cu = torch.tensor([0, 40, 40, 65], dtype=torch.int32, device="cuda")
    x = torch.randn((65, 128), generator=torch.Generator().manual_seed(2))
    dout = torch.randn((65, 128), generator=torch.Generator().manual_seed(4))
    out, _, kept = b.prompt(x.cuda(), cu, keep=True)
    grads = b.backward(dout.cuda(), kept, cu)
    w = {k: getattr(b, k).double().cpu().numpy() for k in ("w_qkv", "b_qkv", "w_out", "w_in", "b_in", "w_mlp")}
    a, H, Hk, D = b.log_decay.double().cpu().numpy(), 4, 2, 32

    def forward(x, w):
        qkv, _ = seq.linear_fwd(x, w["w_qkv"], w["b_qkv"])
        mixed, at = [], 0
        for n in lengths:
            q, k, v = np.split(qkv[at:at + n], [H * D, (H + Hk) * D], axis=1)
            mixed.append(seq.decay_fwd(q.reshape(n, H, D), k.reshape(n, Hk, D), v.reshape(n, Hk, D), a, D ** -0.5)[0].reshape(n, H * D))
            at += n
        h, _ = seq.linear_fwd(np.concatenate(mixed), w["w_out"], None, x)
        act, _ = seq.linear_fwd(h, w["w_in"], w["b_in"], None, "gelu")
        return seq.linear_fwd(act, w["w_mlp"], None, h)[0]

    x64, d64 = x.double().numpy(), dout.double().numpy()
    want = forward(x64, w)
    # five products and two sums in fp32, each a few 2^-24 of its size
    assert np.linalg.norm(out.double().cpu().numpy() - want) < 2e-5 * np.linalg.norm(want)
    r = np.random.default_rng(1)
    for name in ("x", *w):
        base = x64 if name == "x" else w[name]
        step = r.standard_normal(base.shape)
        eps = 1e-5
        up, down = (forward(base + s * eps * step, w) if name == "x" else forward(x64, dict(w, **{name: base + s * eps * step}))
                    for s in (1, -1))
        want = ((up - down) * d64).sum() / (2 * eps)
        got = float((grads[name].double().cpu().numpy() * step).sum())
        size = np.linalg.norm(grads[name].double().cpu().numpy()) * np.linalg.norm(step)
        # fp32 gradients against a central difference: 1e-5 of the two vectors' sizes
        assert abs(got - want) < 1e-5 * size, (name, got, want)
