"""A mixture-of-experts layer on the library's own operators.

    python examples/expert_layer.py [--tokens 512] [--experts 32] [--k 4] [--hidden 1024] [--inner 2048]

Serving: the router's choice (moe_route), the expert order (moe_plan), the tokens' rows
quantised into that order (int8_quantize), the experts' two INT8 products
(grouped_int8_gemm) around the gated activation, and the weighted sum (moe_combine).
Training: the same routing and order around one BF16 product an expert (grouped_bf16_gemm),
and the gradients of the weighted sum and of the router.
Both are checked against plain FP32 products of the same weights.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_mma_gb300 as bs  # noqa: E402


class Int8Experts:
    """Experts y = W2 (silu(Wg x) * (Wu x)) with INT8 weights, a scale for each channel."""

    def __init__(self, w_in, w_out):
        # weights are quantised by channel: the same operator, their rows as its rows
        self.w_in, self.s_in = self._quantize(w_in)       # [E, 2 F, H]: gate rows, then up rows
        self.w_out, self.s_out = self._quantize(w_out)    # [E, H, F]

    @staticmethod
    def _quantize(w):
        E, N, K = w.shape
        codes, scales = bs.int8_quantize(w.reshape(E * N, K))
        return codes.view(E, N, K), scales.view(E, N)

    def __call__(self, x, logits, k, **router):
        E = self.w_in.shape[0]
        ids, weights = bs.moe_route(logits, k, **router)
        m_sizes, src, pos = bs.moe_plan(ids, E)
        rows, scales = bs.int8_quantize(x, src=src, k=k)
        gate, up = bs.grouped_int8_gemm(rows, scales, self.w_in, self.s_in, m_sizes).chunk(2, 1)
        inner, scales = bs.int8_quantize(torch.nn.functional.silu(gate) * up)
        y = bs.grouped_int8_gemm(inner, scales, self.w_out, self.s_out, m_sizes)
        return bs.moe_combine(y, pos, weights)


def plain_experts(x, logits, k, w_in, w_out):
    """The same layer in FP32, expert by expert (softmax scores, renormalised)."""
    p, ids = torch.softmax(logits.float(), -1).topk(k)
    p = p / p.sum(-1, keepdim=True)
    out = torch.zeros_like(x, dtype=torch.float32)
    for e in range(w_in.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        gate, up = (x[t].float() @ w_in[e].float().T).chunk(2, 1)
        out[t] += p[t, j, None] * ((torch.nn.functional.silu(gate) * up) @ w_out[e].float().T)
    return out


def train_step(x, logits, k, w, dout):
    """out = sum_j weight_j W[e_j] x and the gradients of its rows and of the router."""
    E = w.shape[0]
    ids, weights = bs.moe_route(logits, k)
    m_sizes, src, pos = bs.moe_plan(ids, E)
    # a padding token (all its logits -inf) leaves rows that no expert owns, and this product
    # wants every row owned: the last expert takes them, and nothing reads what it makes of them
    owned = m_sizes.clone()
    owned[-1] += src.numel() - m_sizes.sum()
    y = bs.grouped_bf16_gemm(x[src.long().clamp_min(0) // k], w, owned)
    out = bs.moe_combine(y, pos, weights)
    dy, dweights = bs.moe_combine_backward(dout, y, src, pos, weights)
    return out, dy, bs.moe_route_backward(logits, ids, dweights)


def main(argv=None):
    ap = argparse.ArgumentParser()
    for name, v in (("tokens", 512), ("experts", 32), ("k", 4), ("hidden", 1024), ("inner", 2048)):
        ap.add_argument("--" + name, type=int, default=v)
    a = ap.parse_args(argv)
    bs.build()
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, logits = rnd(a.tokens, a.hidden), rnd(a.tokens, a.experts)
    w_in = rnd(a.experts, 2 * a.inner, a.hidden) / a.hidden ** 0.5
    w_out = rnd(a.experts, a.hidden, a.inner) / a.inner ** 0.5

    out = Int8Experts(w_in, w_out)(x, logits, a.k)
    want = plain_experts(x, logits, a.k, w_in, w_out)
    off = ((out.float() - want).norm() / want.norm()).item()
    print(f"serving: {a.tokens} tokens, relative difference from FP32 weights {off:.4f}")

    w, dout = rnd(a.experts, a.hidden, a.hidden) / a.hidden ** 0.5, rnd(a.tokens, a.hidden)
    out, dy, dlogits = train_step(x, logits, a.k, w, dout)
    leaf = logits.float().requires_grad_()
    p, ids = torch.softmax(leaf, -1).topk(a.k)
    p = p / p.sum(-1, keepdim=True)
    rows = torch.stack([x.float() @ w[e].float().T for e in range(a.experts)], 1)
    ref = (rows.gather(1, ids[..., None].expand(-1, -1, a.hidden)) * p[..., None]).sum(1)
    ref.backward(dout.float())
    errors = [((u.float() - v).norm() / v.norm()).item() for u, v in ((out, ref), (dlogits, leaf.grad))]
    print(f"training: relative difference of the output {errors[0]:.4f}, of the router's gradient {errors[1]:.4f}")
    status = bs.device_status()
    # a row's largest of a few thousand normal values is about 3.5 sigma, so a step of 1 / 127 of
    # it leaves 0.8% noise in each of the four INT8 operands, 1.6% together, and the gate about
    # doubles its share; BF16 outputs are within 2^-9 of FP32 ones
    if status or off > 0.05 or max(errors) > 0.01:
        raise SystemExit(f"expert layer: out of tolerance (status {bs.status_string(status)})")


if __name__ == "__main__":
    main()
