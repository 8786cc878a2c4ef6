"""A pre-norm block of the library's operators around the gated delta rule:

    q, k, v, gates = in_proj(norm(x))
    h   = x + out_proj(head_norm(delta_attention(head_norm(q), head_norm(k), v, log_decay(gates), beta(gates))))
    out = h + mlp_out(gelu(mlp_in(norm(h))))

run three ways on one set of weights -- a packed batch of prompts, one token at a time from the states the prompts
left, and a training step's gradients.  The residual's addition before the second norm is the norm's own.

    python examples/delta_block.py            # needs the built library and a GPU; prints how far the forms differ
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import long_fft_convolution_amd as fc  # noqa: E402


class DeltaBlock:
    """Weights (torch tensors) and the three passes.  heads value heads of width / heads, qk_heads shared query/key heads."""

    def __init__(self, width=768, heads=12, qk_heads=4, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.H, self.Hk, self.D = heads, qk_heads, width // heads

        def weight(rows, cols):
            return (torch.randn((rows, cols), generator=g, device=device) * cols ** -0.5).to(dtype)

        def ones(n):
            return (1 + 0.1 * torch.randn((n,), generator=g, device=device)).to(dtype)

        self.sizes = [self.Hk * self.D, self.Hk * self.D, heads * self.D, heads, heads]      # q, k, v, decay, write
        self.w_proj = weight(sum(self.sizes), width)
        self.b_proj = torch.zeros(sum(self.sizes), dtype=dtype, device=device)
        self.w_out, self.w_in, self.w_mlp = weight(width, width), weight(2 * width, width), weight(width, 2 * width)
        self.b_in = torch.zeros(2 * width, dtype=dtype, device=device)
        self.n_in, self.n_mlp, self.n_q, self.n_mix = ones(width), ones(width), ones(self.D), ones(self.D)
        self.n_k = torch.full((self.D,), self.D ** -0.5, dtype=dtype, device=device)     # keys of norm 1
        # each head forgets at its own rate: half-lives around 8 to 4096 tokens
        self.rate = torch.log(torch.tensor(2.0, device=device)) / torch.logspace(3, 12, heads, base=2.0, device=device)

    def _split(self, proj):
        """q, k, v as views of the projection's rows (tokens, heads, dim), and the gates' columns in fp32."""
        q, k, v, a, b = proj.split(self.sizes, dim=1)
        return (*(t.unflatten(1, (-1, self.D)) for t in (q, k, v)), a.float(), b.float())

    def _gates(self, a, b):
        return -self.rate * torch.nn.functional.softplus(a), torch.sigmoid(b)

    def _behind(self, mixed, x):
        """What follows the mixer: head norm, projection, the residual's addition with the second norm, the MLP."""
        normed = fc.rms_norm(mixed, self.n_mix)
        y = fc.linear_act(normed.flatten(1), self.w_out)
        n, h = fc.rms_norm(y, self.n_mlp, residual=x)
        act, pre = fc.linear_act(n, self.w_in, self.b_in, activation="gelu", keep_pre=True)
        return fc.linear_act(act, self.w_mlp, residual=h), (normed, n, h, act, pre)

    def prompt(self, x, cu_seqlens, keep=False):
        """Packed prompts x (tokens, width), sequence b = tokens cu_seqlens[b] .. cu_seqlens[b + 1]; (out, states)."""
        n = fc.rms_norm(x, self.n_in)
        proj = fc.linear_act(n, self.w_proj, self.b_proj)
        q, k, v, a, b = self._split(proj)
        log_decay, beta = self._gates(a, b)
        qn, kn = fc.rms_norm(q, self.n_q), fc.rms_norm(k, self.n_k)
        mixed, states = fc.delta_attention(qn, kn, v, log_decay, beta, cu_seqlens=cu_seqlens)
        out, kept = self._behind(mixed, x)
        return (out, states, (x, n, proj, qn, kn, log_decay, beta, mixed, *kept)) if keep else (out, states)

    def token(self, x, states):
        """The next token of every sequence, x (sequences, width); states are updated in place."""
        q, k, v, a, b = self._split(fc.linear_act(fc.rms_norm(x, self.n_in), self.w_proj, self.b_proj))
        log_decay, beta = self._gates(a, b)
        mixed = torch.empty((x.shape[0], self.H, self.D), dtype=x.dtype, device=x.device)
        fc.fftconv_delta_step(fc.rms_norm(q, self.n_q), fc.rms_norm(k, self.n_k), v, log_decay, beta, states, mixed, self.D ** -0.5)
        return self._behind(mixed, x)[0]

    def backward(self, dout, kept, cu_seqlens):
        """Gradients of sum(dout * out): of x and of every weight (of n_k, a constant, none)."""
        x, n, proj, qn, kn, log_decay, beta, mixed, normed, n2, h, act, pre = kept
        q, k, v, a, b = self._split(proj)
        dact, dw_mlp, _ = fc.linear_act_bwd(dout, act, self.w_mlp, bias=False)
        dn2, dw_in, db_in = fc.linear_act_bwd(dact, n2, self.w_in, pre, "gelu")
        dh, dn_mlp = fc.rms_norm_bwd(dn2, h, self.n_mlp, dsum=dout)              # with the MLP's residual
        dnormed, dw_out, _ = fc.linear_act_bwd(dh, normed.flatten(1), self.w_out, bias=False)
        dmixed, dn_mix = fc.rms_norm_bwd(dnormed.unflatten(1, (self.H, self.D)), mixed, self.n_mix)
        dqn, dkn, dv, da, db, _ = fc.delta_attention_bwd(qn, kn, v, log_decay, beta, dmixed, cu_seqlens=cu_seqlens)
        dq, dn_q = fc.rms_norm_bwd(dqn, q, self.n_q)
        dk, _ = fc.rms_norm_bwd(dkn, k, self.n_k)
        dproj = torch.cat([dq.flatten(1), dk.flatten(1), dv.flatten(1), (-da * self.rate * torch.sigmoid(a)).to(x.dtype),
                           (db * beta * (1 - beta)).to(x.dtype)], dim=1)
        dn, dw_proj, db_proj = fc.linear_act_bwd(dproj, n, self.w_proj)
        dx, dn_in = fc.rms_norm_bwd(dn, x, self.n_in, dsum=dh)                   # with the mixer's residual
        return dict(x=dx, w_proj=dw_proj, b_proj=db_proj, w_out=dw_out, w_in=dw_in, b_in=db_in, w_mlp=dw_mlp, n_in=dn_in,
                    n_mlp=dn_mlp, n_q=dn_q, n_mix=dn_mix)


def main():
    dev, lengths = "cuda", [700, 1, 333]
    block = DeltaBlock(device=dev)
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
