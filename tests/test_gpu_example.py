"""The example block (projections, decay attention, MLP) as a whole: its single-token form against its prompt form, and
its gradients against differences of the same block in float64 on the CPU."""
import os
import sys

import numpy as np
import pytest
import torch

import long_fft_convolution_amd as fc
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


def test_scratch_memory_belongs_to_the_stream_given():
    # behind work on that stream the calls run late; the current stream meanwhile takes and fills memory of its own
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(3)
    q, k, v, d = (torch.randn((1, 3000, 2, 64), generator=g, device=dev).to(torch.bfloat16) for _ in range(4))
    a = -torch.rand(2, generator=g, device=dev) * 0.01
    x, W = (torch.randn((n, 4096), generator=g, device=dev).to(torch.bfloat16) for n in (200, 100))
    y = torch.randn((200, 100), generator=g, device=dev).to(torch.bfloat16)
    work = torch.randn((4096, 4096), generator=g, device=dev)

    def calls(stream):
        return (*fc.decay_attention(q, k, v, a, stream=stream), *fc.decay_attention_bwd(q, k, v, a, d, stream=stream)[:3],
                fc.linear_act(x, W, stream=stream), *fc.linear_act_bwd(y, x, W, stream=stream))

    want = calls(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(4):
            work = torch.nn.functional.normalize(work @ work)
    got = calls(s)
    taken = [torch.full((n,), 255, dtype=torch.uint8, device=dev) for n in (1 << 18, 1 << 20, 1 << 22, 1 << 24) for _ in range(4)]
    torch.cuda.synchronize()
    assert len(taken) == 16
    for i, (w, t) in enumerate(zip(want, got)):
        assert torch.equal(w, t), i
