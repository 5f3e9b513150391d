"""The residual branch's operators and the decoding step's expert layer from their definitions,
in 64 bits on the CPU (not a test module)."""
from __future__ import annotations

import math

import numpy as np
import torch

M32 = np.uint64(0xFFFFFFFF)


def philox(counter, key):
    """Philox4x32-10 of counters [n, 4] and a key [2] (Salmon et al., SC 2011) -> [n, 4]."""
    c = [counter[:, i].astype(np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    for _ in range(10):
        u, v = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(v >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), v & M32,
             (u >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), u & M32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1)


def threshold(p):
    return min(int(np.rint(np.float64(np.float32(p)) * 65536)), 65535)


def mask(n, p, seed, offset, first=0):
    """0 or 1 / (1 - p) for values first .. first + n - 1 (first a multiple of 8)."""
    at = np.arange(first // 8, first // 8 + (n + 7) // 8, dtype=np.uint64)
    seed, offset = seed & (2 ** 64 - 1), offset & (2 ** 64 - 1)
    full = lambda v: np.full_like(at, v)  # noqa: E731
    ctr = np.stack([at & M32, at >> np.uint64(32), full(offset & 0xFFFFFFFF), full(offset >> 32)], 1)
    w = philox(ctr, (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], 2).reshape(-1)[:n]
    drop = threshold(p)
    return torch.from_numpy((bits >= drop).astype(np.float64) * (65536 / (65536 - drop)))


def stats(v, norm, eps):
    """mean (0 for rms), 1 / standard deviation, columns [T, 1]."""
    mean = v.mean(1, keepdim=True) if norm == "layer" else torch.zeros_like(v[:, :1])
    var = ((v - mean) ** 2).mean(1, keepdim=True)
    return mean, 1 / (var + eps).sqrt()


def norm(v, kind, weight=None, bias=None, eps=1e-6):
    """n(v) * weight + bias."""
    if kind != "none":
        mean, r = stats(v, kind, eps)
        v = (v - mean) * r
    v = v if weight is None else v * weight
    return v if bias is None else v + bias


def gate_of(gate, rows, T):
    return 1.0 if gate is None else gate[torch.arange(T) // rows]


def leave(x, y, kind, weight=None, bias=None, gate=None, rows=1, xs=1.0, ys=1.0, keep=1.0, eps=1e-6):
    return xs * x + ys * gate_of(gate, rows, len(x)) * keep * norm(y, kind, weight, bias, eps)


def norm_grad(dz, v, kind, weight=None, eps=1e-6):
    """(gradient in v, sum_rows dz n, sum_rows dz, size of dv's terms, sums of their terms' sizes)."""
    if kind == "none":
        return dz, None, None, dz.abs(), None, None
    mean, r = stats(v, kind, eps)
    n = (v - mean) * r
    q = dz if weight is None else dz * weight
    qm = q.mean(1, keepdim=True) if kind == "layer" else 0.0
    dv = r * (q - qm - n * (q * n).mean(1, keepdim=True))
    # n's own error grows with the mean that was taken off
    far = 1 + mean.abs() * r
    size = r * (q.abs() + q.abs().mean(1, keepdim=True)
                + n.abs() * (q.abs() * (n.abs() + far)).mean(1, keepdim=True)
                + far * (q * n).abs().mean(1, keepdim=True)) * far
    return dv, (dz * n).sum(0), dz.sum(0), size, (dz.abs() * (n.abs() + far)).sum(0), dz.abs().sum(0)


E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def weights(codes, scales, fmt):
    """The values of expert weights [..., rows, K] in 64 bits."""
    if fmt == "bf16":
        return codes.double()
    if fmt == "int8":
        return codes.double() * scales.double()[..., None]
    if fmt == "e2m1":
        v = E2M1[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    else:
        v = codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).double()
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def act(x, kind):
    if kind == "silu":
        return x * torch.sigmoid(x)
    if kind == "gelu":
        return x * torch.special.erfc(-x / math.sqrt(2)) / 2
    return x.clamp_min(0) if kind == "relu" else x


def moe_step(x, ids, weight, w_in, w_out, kind):
    """out [T, H], and the size of its terms with each inner value's own."""
    T, H = x.shape
    out, size = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    F = w_in.shape[1] // 2
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < len(w_in):
                continue
            u = w_in[e] @ x[t]
            a = w_in[e].abs() @ x[t].abs()
            g, up = u[:F], u[F:]
            inner = act(g, kind) * up
            # activations are at most |x|, and change by at most 1.2 of what x does
            big = 1.2 * a[:F] * up.abs() + act(g, kind).abs() * a[F:]
            out[t] += weight[t, j] * (w_out[e] @ inner)
            size[t] += weight[t, j].abs() * (w_out[e].abs() @ torch.stack([inner.abs(), big], 1)) @ torch.tensor(
                [2.0 ** -8, 2.0 ** -16], dtype=torch.float64)
    return out, size
