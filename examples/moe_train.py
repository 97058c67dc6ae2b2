"""A training step of a Mixture-of-Experts layer whose experts run in 8-bit floating point, from the block operators.

    r       = top-k of softmax(x W_r^T)                    routing; or the order of a choice that is replayed
    u, v    = x W1_e^T, x W3_e^T                           e4m3, a scale for every block of 128
    h       = silu(u) * v
    out     = combine(h W2_e^T)
    and back: gradients of the gates and of the experts' results, of the three products (rows and weights), of the
    activation, of the rows' tokens and of the router

    python examples/moe_train.py            # random weights, one step, errors against fp32 and the time of a step

Weights are kept in fp32 and quantised once a step; the optimiser is the caller's.
"""
from __future__ import annotations

import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from mixture_experts_gemm_gb300 import ops  # noqa: E402


class Layer:
    """Weights of one layer, in fp32 and (after `quantise`) in e4m3."""

    def __init__(self, d=2048, f=1408, experts=16, top_k=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.experts, self.top_k = experts, top_k
        self.weights = dict(router=rn(experts, d) / d ** 0.5, w1=rn(experts, f, d) / d ** 0.5,
                            w3=rn(experts, f, d) / d ** 0.5, w2=rn(experts, d, f) / f ** 0.5)
        self.quantise()

    def quantise(self):
        self.q = {n: ops.fp8_quantize(self.weights[n], square=True) for n in ("w1", "w3", "w2")}

    def forward(self, x, idx=None):
        """x [T, d] bf16 -> (out [T, d], what the backward pass needs).  With idx [T, k] that choice of experts is
        replayed, a slot of -1 being dropped; the gates are the router's scores of the chosen experts."""
        logits = x.float() @ self.weights["router"].t()
        if idx is None:
            r = ops.route(logits, self.top_k, renormalize=False)
            idx, gate = r.idx, r.gate
        else:
            r = ops.dispatch_order(idx, self.experts)
            gate = torch.softmax(logits, 1).gather(1, idx.long().clamp(min=0)) * (idx >= 0)
        rows = ops.dispatch(x, r.token_of_row)
        u, v = (ops.fp8_experts(rows, *self.q[n], r.offsets) for n in ("w1", "w3"))
        h = ops.gated(u, v)
        y = ops.fp8_experts(h, *self.q["w2"], r.offsets)
        return ops.combine(y, r.row_of, gate), (x, rows, logits, idx, gate, r, u, v, h, y)

    def backward(self, d_out, saved):
        """Gradients of x and of the weights, as a dict."""
        x, rows, logits, idx, gate, r, u, v, h, y = saved
        d_y, d_gate = ops.combine_backward(d_out, y, r.row_of, gate, r.token_of_row)
        d_h, d_w2 = ops.fp8_experts_backward(d_y, h, *self.q["w2"], r.offsets)
        d_u, d_v = ops.gated_backward(d_h, u, v)
        d_rows, d_w1 = ops.fp8_experts_backward(d_u, rows, *self.q["w1"], r.offsets)
        d_rows3, d_w3 = ops.fp8_experts_backward(d_v, rows, *self.q["w3"], r.offsets)
        d_logits = ops.route_backward(logits, idx, d_gate, renormalize=False)
        d_x = sum(ops.dispatch_backward(g, r.row_of, out_dtype=torch.float32) for g in (d_rows, d_rows3))
        return dict(x=(d_x + d_logits @ self.weights["router"]).to(x.dtype), router=d_logits.t() @ x.float(), w1=d_w1, w3=d_w3,
                    w2=d_w2)

    def reference(self, x, idx, d_out):
        """out and the gradients in fp32 by autograd, expert by expert, for the same choice."""
        x = x.float().requires_grad_(True)
        w = {n: t.detach().clone().requires_grad_(True) for n, t in self.weights.items()}
        with torch.enable_grad():
            scores = torch.softmax(x @ w["router"].t(), 1)
            out = torch.zeros_like(x)
            for e in range(self.experts):
                t, _ = (idx == e).nonzero(as_tuple=True)
                h = torch.nn.functional.silu(x[t] @ w["w1"][e].t()) * (x[t] @ w["w3"][e].t())
                out = out.index_add(0, t, scores[t, e, None] * (h @ w["w2"][e].t()))
            out.backward(d_out.float())
        return out.detach(), dict(x=x.grad, **{n: t.grad for n, t in w.items()})


def errors_of(layer, x, d_out, idx=None):
    """Relative errors (2-norms) of the result and of every gradient against fp32."""
    out, saved = layer.forward(x, idx)
    got = dict(out=out, **layer.backward(d_out, saved))
    want_out, want = layer.reference(x, saved[3], d_out)
    want["out"] = want_out
    return {n: float((got[n].float() - want[n]).norm() / want[n].norm()) for n in got}


def main():
    layer = Layer()
    x, d_out = (torch.randn(4096, 2048, device="cuda").bfloat16() for _ in range(2))
    print({n: round(e, 3) for n, e in errors_of(layer, x, d_out).items()})
    torch.cuda.synchronize()
    n, t = 20, time.perf_counter()
    for _ in range(n):
        layer.quantise()
        layer.backward(d_out, layer.forward(x)[1])
    torch.cuda.synchronize()
    print(f"{1e6 * (time.perf_counter() - t) / n:.0f} us a step")


if __name__ == "__main__":
    main()
