"""A sequence-model block of the library's operators: projections, decay attention, MLP.

    h   = x + out_proj(decay_attention(qkv_proj(x)))
    out = h + mlp_out(gelu(mlp_in(h)))

run three ways on one set of weights -- a packed batch of prompts, one token at a time from the states the prompts
left, and a training step's gradients -- so that the prompt form, the single-token form and the backward pass meet as
they do in a model.  The block's token mixer could as well be the gated long convolution (causal_conv).

    python examples/decay_block.py            # needs the built library and a GPU; prints how far the forms differ
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import long_fft_convolution_amd as fc  # noqa: E402


class DecayBlock:
    """Weights (torch tensors) and the three passes.  heads x dim query heads, kv_heads shared key/value heads."""

    def __init__(self, width=768, heads=12, kv_heads=4, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.H, self.Hk, self.D = heads, kv_heads, width // heads

        def weight(rows, cols):
            return (torch.randn((rows, cols), generator=g, device=device) * cols ** -0.5).to(dtype)

        self.w_qkv = weight((heads + 2 * kv_heads) * self.D, width)
        self.b_qkv = torch.zeros(self.w_qkv.shape[0], dtype=dtype, device=device)
        self.w_out, self.w_in, self.w_mlp = weight(width, width), weight(2 * width, width), weight(width, 2 * width)
        self.b_in = torch.zeros(2 * width, dtype=dtype, device=device)
        # each head forgets at its own rate: half-lives from 8 to 4096 tokens
        half_lives = torch.logspace(3, 12, heads, base=2.0, device=device)
        self.log_decay = -torch.log(torch.tensor(2.0, device=device)) / half_lives

    def _split(self, qkv):
        """q, k, v as views of the projection's rows: (tokens, heads, dim)."""
        q, k, v = qkv.split([self.H * self.D, self.Hk * self.D, self.Hk * self.D], dim=1)
        return tuple(t.unflatten(1, (-1, self.D)) for t in (q, k, v))

    def prompt(self, x, cu_seqlens, keep=False):
        """Packed prompts x (tokens, width), sequence b = tokens cu_seqlens[b] .. cu_seqlens[b + 1]; (out, states)."""
        qkv = fc.linear_act(x, self.w_qkv, self.b_qkv)
        q, k, v = self._split(qkv)
        mixed, states = fc.decay_attention(q, k, v, self.log_decay, cu_seqlens=cu_seqlens)
        mixed = mixed.flatten(1)
        h = fc.linear_act(mixed, self.w_out, residual=x)
        a, pre = fc.linear_act(h, self.w_in, self.b_in, activation="gelu", keep_pre=True)
        out = fc.linear_act(a, self.w_mlp, residual=h)
        return (out, states, (x, qkv, mixed, h, a, pre)) if keep else (out, states)

    def token(self, x, states):
        """The next token of every sequence, x (sequences, width); states are updated in place."""
        q, k, v = self._split(fc.linear_act(x, self.w_qkv, self.b_qkv))
        mixed = torch.empty((x.shape[0], self.H, self.D), dtype=x.dtype, device=x.device)
        fc.fftconv_decay_step(q, k, v, self.log_decay, states, mixed, self.D ** -0.5)
        h = fc.linear_act(mixed.flatten(1), self.w_out, residual=x)
        return fc.linear_act(fc.linear_act(h, self.w_in, self.b_in, activation="gelu"), self.w_mlp, residual=h)

    def backward(self, dout, kept, cu_seqlens):
        """Gradients of sum(dout * out): of x and of every weight."""
        x, qkv, mixed, h, a, pre = kept
        q, k, v = self._split(qkv)
        da, dw_mlp, _ = fc.linear_act_bwd(dout, a, self.w_mlp, bias=False)
        dh, dw_in, db_in = fc.linear_act_bwd(da, h, self.w_in, pre, "gelu")
        dh += dout                                              # the MLP's residual
        dmixed, dw_out, _ = fc.linear_act_bwd(dh, mixed, self.w_out, bias=False)
        dqkv = torch.empty_like(qkv)                            # dq, dk and dv into one buffer, as the projection takes it
        scratch = torch.empty(fc.fftconv_decay_bwd_workspace_bytes(
            cu_seqlens.numel() - 1, x.shape[0], self.H, self.Hk, self.D, self.D, x.dtype), dtype=torch.uint8, device=x.device)
        fc.fftconv_decay_bwd(dmixed.unflatten(1, (self.H, self.D)), q, k, v, self.log_decay, *self._split(dqkv), self.D ** -0.5,
                             cu_seqlens=cu_seqlens, workspace=scratch)
        dx, dw_qkv, db_qkv = fc.linear_act_bwd(dqkv, x, self.w_qkv)
        return dict(x=dx + dh, w_qkv=dw_qkv, b_qkv=db_qkv, w_out=dw_out, w_in=dw_in, b_in=db_in, w_mlp=dw_mlp)


def main():
    dev, lengths = "cuda", [700, 1, 333]
    block = DecayBlock(device=dev)
    total = sum(lengths)
    x = torch.randn((total, 768), generator=torch.Generator(device=dev).manual_seed(1), device=dev).to(torch.bfloat16)
    cu = torch.tensor([0] + lengths, device=dev).cumsum(0).to(torch.int32)
    out, _, kept = block.prompt(x, cu, keep=True)
    # all but the last token of each sequence as a prompt, then the last one by itself
    last = (cu[1:] - 1).long()
    first = torch.ones(total, dtype=torch.bool, device=dev)
    first[last] = False
    shorter = (cu - torch.arange(len(cu), device=dev)).to(torch.int32)
    _, states = block.prompt(x[first], shorter)
    tokens = block.token(x[last], states)
    err = float((tokens.float() - out[last].float()).norm() / out[last].float().norm())
    print(f"single tokens after a prompt against the longer prompt: relative L2 {err:.2e}")
    grads = block.backward(torch.ones_like(out), kept, cu)
    print("gradient norms:", {k: round(float(g.float().norm()), 2) for k, g in grads.items()})
    return err


if __name__ == "__main__":
    if not main() < 2e-2:      # a few bfloat16 roundings (2^-8 each) on the way through the block
        raise SystemExit("the forms differ")
