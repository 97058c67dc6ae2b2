"""A Mixture-of-Experts block of many experts, served in 8-bit integers, from the block operators.

    p       = RMSNorm(x)                                   norm before the block
    r       = top-k of sigmoid(p W_r^T) + balance bias     routing by groups, dispatch order
    h       = silu(p W1_e^T) * (p W3_e^T)                  gated projections in 8-bit integers
    y       = combine(h W2_e^T)                            down projection, gate-weighted sum
    x1, p1  = x + block_scale * RMSNorm(y), RMSNorm(x1)    norm after it, residual, the next block's norm

    python examples/moe_block.py            # builds random weights, runs a batch and one token, prints errors

`gradients` shows the backward passes that a training step of the norms and the router takes, with the
experts frozen.
"""
from __future__ import annotations

import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from mixture_experts_gemm_gb300 import ops  # noqa: E402


class Block:
    """Weights of one block: full precision kept for comparison, experts quantised once."""

    def __init__(self, d=2048, f=1408, experts=64, top_k=6, groups=8, top_groups=4, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.d, self.f, self.top_k = d, f, top_k
        self.routing = dict(score="sigmoid", groups=groups, top_groups=top_groups, group_top=2, renormalize=True, scale=1.0)
        self.bias = 0.02 * rn(experts)
        self.norm_in, self.norm_out, self.norm_next = (1 + 0.1 * rn(d) for _ in range(3))
        self.w_router = rn(experts, d) / d ** 0.5
        self.w1, self.w3 = (rn(experts, f, d) / d ** 0.5 for _ in range(2))
        self.w2 = rn(experts, d, f) / f ** 0.5
        self.q1, self.q3, self.q2 = (ops.int8_quantize(w) for w in (self.w1, self.w3, self.w2))

    def choose(self, x):
        """The experts' input p and its routing."""
        p = ops.pre_norm(x, self.norm_in)
        return p, ops.route(p.float() @ self.w_router.t(), self.top_k, bias=self.bias, **self.routing)

    def forward(self, x):
        """x [T, d] bf16 -> (x1, the next block's input), both bf16."""
        p, r = self.choose(x)
        h = ops.int8_experts(p, *self.q1, r.offsets, rows=r.token_of_row, w3=self.q3[0], w3_scale=self.q3[1])
        y = ops.combine(ops.int8_experts(h, *self.q2, r.offsets), r.row_of, r.gate, out_dtype=torch.float32)
        return ops.block_norm(x, y, after="rms", after_weight=self.norm_out, before="rms", before_weight=self.norm_next,
                              block_scale=0.5)

    def reference(self, x, idx=None):
        """The same block in fp32 from the unquantised weights, expert by expert; with idx [T, k], by those experts
        (a token whose choice is a close call may have others here)."""
        rms = lambda v, w: v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
        x = x.float()
        p = rms(x, self.norm_in).bfloat16().float()
        s = torch.sigmoid(p @ self.w_router.t())
        idx = self.best(s) if idx is None else idx.long()
        gate = s.gather(1, idx)
        gate = gate / gate.sum(1, keepdim=True)
        y = torch.zeros_like(x)
        for e in range(self.w_router.shape[0]):
            t, slot = (idx == e).nonzero(as_tuple=True)
            if len(t):
                h = torch.nn.functional.silu(p[t] @ self.w1[e].t()) * (p[t] @ self.w3[e].t())
                y.index_add_(0, t, gate[t, slot, None] * (h @ self.w2[e].t()))
        x1 = x + 0.5 * rms(y, self.norm_out)
        return x1, rms(x1, self.norm_next)

    def best(self, s):
        """The experts that scores s [T, E] choose, in plain form."""
        key = (s + self.bias).view(s.shape[0], self.routing["groups"], -1)
        worth = key.topk(2, -1).values.sum(-1)
        keep = torch.zeros_like(worth).scatter_(1, worth.topk(self.routing["top_groups"], 1).indices, 1.0).bool()
        return key.masked_fill(~keep[:, :, None], -1e9).flatten(1).topk(self.top_k, 1).indices

    def gradients(self, x1, y, logits, idx, d_x1, d_p1, d_gate):
        """Gradients of the norms' inputs and vectors, and of the router's logits."""
        norms = ops.block_norm_backward(d_x1, d_p1, x1, y, after="rms", after_weight=self.norm_out, before="rms",
                                        before_weight=self.norm_next, block_scale=0.5)
        routing = {k: self.routing[k] for k in ("score", "renormalize", "scale")}
        return norms, ops.route_backward(logits, idx, d_gate, **routing)


def error_of(block, x):
    """Largest |x1 - reference| over the reference's root mean square, and of the next input."""
    out, want = block.forward(x), block.reference(x, block.choose(x)[1].idx)
    return [float((a.float() - b).abs().max() / b.square().mean().sqrt()) for a, b in zip(out, want)]


def main():
    block = Block()
    for T in (1, 1024):
        x = torch.randn(T, block.d, device="cuda").bfloat16()
        errors = error_of(block, x)
        torch.cuda.synchronize()
        n, t = 20, time.perf_counter()
        for _ in range(n):
            block.forward(x)
        torch.cuda.synchronize()
        print(f"T={T}: {1e6 * (time.perf_counter() - t) / n:.0f} us a block, largest error / RMS: "
              f"x1 {errors[0]:.3f}, next {errors[1]:.3f}")


if __name__ == "__main__":
    main()
