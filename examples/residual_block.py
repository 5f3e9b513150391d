"""A residual block on the library's own operators: a decoding step and a training step.

    python examples/residual_block.py [--tokens 4] [--rows 2048] [--experts 32] [--k 4] [--hidden 1024] [--inner 2048]

Decoding: the norm before the block (branch_enter), the router's choice (moe_route), the experts of a
few tokens in E4M3 (moe_step), and the step after it -- norm, gate, residual and the next
block's norm, made into the next product's MXFP8 operand on the way (branch_leave, mx_gemm).
Training: the same norms around one BF16 product (grouped_bf16_gemm with one group), dropout in
the residual, and every gradient, with the mask made again from its seed.
Both are checked against the same layers in FP32.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_mma_gb300 as bs  # noqa: E402


def decode_step(x, p, k):
    """(the stream after the block, the next block's first product) for a few tokens x [T, H]."""
    h = bs.branch_enter(x, p["norm"])
    ids, weights = bs.moe_route(h @ p["router"].T, k)
    y = bs.moe_step(h, ids, weights, p["w_in"], p["w_out"], s_in=p["s_in"], s_out=p["s_out"], fmt="e4m3")
    out, codes, scales = bs.branch_leave(x, y, p["post"], norm="rms", gate=p["gate"], next_norm="rms",
                                         next_weight=p["next"], fmt="e4m3")
    return out, bs.mx_gemm(codes, scales, p["w_next"], p["s_next"], "NT")


def rms(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w


def plain_decode(x, p, k, w_in, w_out, w_next):
    """The same in FP32, weights w_in [E, 2F, H], w_out [E, H, F] and w_next as their codes stand."""
    x = x.float()
    h = rms(x, p["norm"]).bfloat16().float()
    probs, ids = torch.softmax((h.bfloat16() @ p["router"].T).float(), -1).topk(k)
    probs = probs / probs.sum(-1, keepdim=True)
    y = torch.zeros_like(x)
    for t in range(len(x)):
        for j in range(k):
            gate, up = (w_in[ids[t, j]] @ h[t]).chunk(2)
            y[t] += probs[t, j] * (w_out[ids[t, j]] @ (torch.nn.functional.silu(gate) * up))
    out = x + p["gate"].float() * rms(y, p["post"])
    return out, rms(out, p["next"]) @ w_next.T


def train_step(x, p, dout, rng, drop):
    """out = x + gate * dropout(norm(W norm(x))) and its gradients in x and the parameters."""
    rows = p["m_sizes"]     # of the one group, on the device
    form = dict(norm="rms", gate=p["gate"], gate_rows=p["rows"], p=drop, rng=rng)
    h = bs.branch_enter(x, p["norm"])
    y = bs.grouped_bf16_gemm(h, p["w"][None], rows)
    out = bs.branch_leave(x, y, p["post"], **form)
    dy, dx, dpost, _, dgate = bs.branch_leave_backward(dout, y, p["post"], **form)
    dh = bs.grouped_bf16_gemm(dy, p["w"].T.contiguous()[None], rows)
    dw = dy.T @ h
    dx, dnorm, _ = bs.branch_enter_backward(dh, x, p["norm"], dres=dx)
    return out, {"x": dx, "w": dw, "norm": dnorm, "post": dpost, "gate": dgate}


def plain_train(x, p, dout, keep):
    """The same by autograd in FP32, keep: 0 or 1 / (1 - drop) for each value."""
    leaf = {k: v.float().requires_grad_() for k, v in {**p, "x": x}.items() if k not in ("rows", "m_sizes")}
    gate = leaf["gate"].repeat_interleave(p["rows"], 0)[:len(x)]
    out = leaf["x"] + gate * keep * rms(rms(leaf["x"], leaf["norm"]) @ leaf["w"].T, leaf["post"])
    out.backward(dout.float())
    return out.detach(), {k: v.grad for k, v in leaf.items()}


def off(got, want):
    return ((got.float() - want).norm() / want.norm()).item()


def values(codes, scales):
    """What E4M3 codes with a scale for 32 stand for."""
    return codes.view(torch.float8_e4m3fn).float() * torch.exp2(scales.float() - 127).repeat_interleave(32, -1)


def main(argv=None):
    ap = argparse.ArgumentParser()
    for name, v in (("tokens", 4), ("rows", 2048), ("experts", 32), ("k", 4), ("hidden", 1024), ("inner", 2048)):
        ap.add_argument("--" + name, type=int, default=v)
    a = ap.parse_args(argv)
    bs.build()
    g = torch.Generator(device="cuda").manual_seed(0)
    H, F, E = a.hidden, a.inner, a.experts
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731

    def mx(*shape):
        codes, scales = bs.mx_quantize((rnd(*shape) / shape[-1] ** 0.5).view(-1, shape[-1]))
        return codes.view(shape), scales.view(*shape[:-1], -1)

    p = {"norm": 1 + 0.1 * rnd(H), "post": 1 + 0.1 * rnd(H), "next": 1 + 0.1 * rnd(H),
         "gate": (0.5 * rnd(1, H)).bfloat16(), "router": (rnd(E, H) / H ** 0.5).bfloat16()}
    (p["w_in"], p["s_in"]), (p["w_out"], p["s_out"]) = mx(E, 2 * F, H), mx(E, H, F)
    p["w_next"], p["s_next"] = mx(2 * H, H)
    x = rnd(a.tokens, H).bfloat16()
    got = decode_step(x, p, a.k)
    want = plain_decode(x, p, a.k, *(values(p[n], p["s" + n[1:]]) for n in ("w_in", "w_out", "w_next")))
    served = [off(u, v) for u, v in zip(got, want)]
    print(f"decoding: {a.tokens} tokens, relative difference from FP32 {served[0]:.4f}, of the next product "
          f"from E4M3 rows {served[1]:.4f}")

    p = {"norm": 1 + 0.1 * rnd(H), "post": 1 + 0.1 * rnd(H), "rows": 512,
         "m_sizes": torch.tensor([a.rows], device="cuda"), "w": (rnd(H, H) / H ** 0.5).bfloat16(),
         "gate": (0.5 * rnd(-(-a.rows // 512), H)).bfloat16()}
    x, dout = rnd(a.rows, H).bfloat16(), rnd(a.rows, H).bfloat16()
    rng = torch.tensor([17, 0], device="cuda")
    out, grads = train_step(x, p, dout, rng, 0.1)
    keep = bs.dropout(torch.ones(a.rows, H, device="cuda"), 0.1, rng)
    want_out, want = plain_train(x, p, dout, keep)
    errors = {"out": off(out, want_out), **{k: off(v, want[k]) for k, v in grads.items()}}
    print("training: relative differences " + ", ".join(f"{k} {v:.4f}" for k, v in errors.items()))
    status = bs.device_status()
    # BF16 rows are within 2^-9 of FP32 ones, a few of them in a row; E4M3 rows (two in the next
    # product, three significant bits each: 2^-5 / sqrt(3) or so) leave 2.5% each
    if status or served[0] > 0.01 or served[1] > 0.06 or max(errors.values()) > 0.015:
        raise SystemExit(f"residual block: out of tolerance (status {bs.status_string(status)})")


if __name__ == "__main__":
    main()
