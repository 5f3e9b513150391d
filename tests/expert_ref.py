"""The expert layer's operators from their definitions, in 64 bits (not a test module)."""
from __future__ import annotations

import numpy as np


def scores(x, score):
    """Scores of logits x [T, E] (float64, -inf closed): softmax of each row, or the sigmoid."""
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1 / (1 + np.exp(-x))
        m = x.max(1, keepdims=True)
        e = np.exp(x - np.where(np.isneginf(m), 0, m))
        s = e.sum(1, keepdims=True)
        return e / np.where(s == 0, 1, s)


def clean(x):
    x = np.asarray(x, dtype=np.float64).copy()
    x[np.isnan(x)] = -np.inf
    return np.minimum(x, float(np.finfo(np.float32).max))


def keys(x, score, bias, groups, topk_groups, group_top):
    """Selection keys [T, E], closed groups at -inf, and the groups' values (or None)."""
    x = clean(x)
    s = scores(x, score)
    key = x.copy()
    if bias is not None:
        with np.errstate(invalid="ignore"):
            key = s + np.asarray(bias, dtype=np.float64)
        key[np.isneginf(x) | np.isnan(key)] = -np.inf
    if topk_groups >= groups:
        return key, None
    by = np.where(np.isneginf(x), -np.inf, s) if bias is None and group_top > 1 else key
    by = -np.sort(-by.reshape(len(x), groups, -1), axis=2)[:, :, :group_top]
    value = np.where(np.isneginf(by[:, :, 0]), -np.inf, np.where(np.isneginf(by), 0, by).sum(2))
    key = key.copy()
    for t in range(len(x)):
        first = sorted(range(groups), key=lambda g: (-value[t, g], g))[:topk_groups]
        for g in set(range(groups)) - set(first):
            key[t, g * by_size(key, groups):(g + 1) * by_size(key, groups)] = -np.inf
    return key, value


def by_size(key, groups):
    return key.shape[1] // groups


def route(x, k, score, bias=None, groups=1, topk_groups=1, group_top=1, renormalize=True, scale=1.0):
    key, _ = keys(x, score, bias, groups, topk_groups, group_top)
    s = scores(clean(x), score)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    used = ~np.isneginf(np.take_along_axis(key, ids, 1))
    p = np.where(used, np.take_along_axis(s, ids, 1), 0)
    return np.where(used, ids, -1).astype(np.int32), weights_of(p, renormalize, scale)


def weights_of(p, renormalize, scale):
    if renormalize:
        total = p.sum(1, keepdims=True)
        p = p / np.where(total == 0, 1, total)
    return p * scale


def route_weights(x, ids, score, renormalize, scale):
    """The weights as a function of the logits, the choice held fixed."""
    s = scores(clean(x), score)
    p = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0)
    return weights_of(p, renormalize, scale)


def route_backward(x, ids, dw, score, renormalize, scale):
    """From the Jacobians: of the weights in the scores, then of the scores in the logits."""
    s = scores(clean(x), score)
    T, E = s.shape
    dx = np.zeros((T, E))
    for t in range(T):
        sel = ids[t][ids[t] >= 0]
        g = dw[t][ids[t] >= 0].astype(np.float64) * scale
        p = s[t, sel]
        ds = np.zeros(E)
        if renormalize:
            if p.sum() > 0:
                J = np.eye(len(sel)) / p.sum() - np.outer(p, np.ones(len(sel))) / p.sum() ** 2
                ds[sel] = J.T @ g
        else:
            ds[sel] = g
        if score == "softmax":
            dx[t] = s[t] * ds - s[t] * (s[t] @ ds)
        else:
            dx[t] = s[t] * (1 - s[t]) * ds
    return dx


def plan(ids, E):
    flat = np.asarray(ids).reshape(-1)
    m = np.zeros(E, dtype=np.int64)
    rows = []
    for e in range(E):
        at = np.nonzero(flat == e)[0]
        m[e] = len(at)
        rows.append(at)
    rows = np.concatenate(rows)
    src = np.full(flat.size, -1, dtype=np.int32)
    src[:len(rows)] = rows
    pos = np.full(flat.size, -1, dtype=np.int32)
    pos[rows] = np.arange(len(rows))
    return m, src, pos.reshape(np.asarray(ids).shape)


def combine(y, pos, w):
    out = np.zeros((pos.shape[0], y.shape[1]))
    for t in range(pos.shape[0]):
        for j in range(pos.shape[1]):
            if 0 <= pos[t, j] < len(y):
                out[t] += (1.0 if w is None else float(w[t, j])) * y[pos[t, j]]
    return out


def combine_backward(dout, y, pos, w):
    dy = np.zeros((pos.size, dout.shape[1]))
    dw = np.zeros(pos.shape)
    for t in range(pos.shape[0]):
        for j in range(pos.shape[1]):
            if pos[t, j] >= 0:
                dy[pos[t, j]] = (1.0 if w is None else float(w[t, j])) * dout[t]
                if y is not None:
                    dw[t, j] = dout[t] @ y[pos[t, j]]
    return dy, dw


def int8_quantize(x, src=None, k=1):
    """x float32 [rows, K] -> codes, scales by the FP32 steps of the definition."""
    x = np.asarray(x, dtype=np.float32)
    if src is not None:
        tok = np.where(src < 0, -1, src // k)
        x = np.where(((tok >= 0) & (tok < len(x)))[:, None], x[np.clip(tok, 0, max(len(x) - 1, 0))],
                     np.float32(0))
    s = np.abs(x).max(1) * (np.float32(1) / np.float32(127))
    s[s == 0] = 1
    q = (x / s[:, None]).astype(np.float32)
    return np.clip(np.rint(q), -127, 127).astype(np.int8), s


def int8_gemm(a, sa, b, sb, bias=None):
    """The integer product exactly, the scales in 64 bits."""
    d = (a.astype(np.float64) @ b.astype(np.float64).T) * np.outer(sa.astype(np.float64),
                                                                  sb.astype(np.float64))
    return d if bias is None else d + bias.astype(np.float64)
