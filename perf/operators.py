"""Cases of the expert-layer operators: routing, the expert order, INT8 quantisation of
(gathered) rows, INT8 products and the weighted sum of the experts' outputs.

``own`` false: plain elementary torch operations in FP32.  ``own`` true: the calls a user
makes of block_scaled_precision_mma_gb300.
"""
import math

import torch

own = False


def _bs():
    import block_scaled_precision_mma_gb300 as bs
    bs.build()
    return bs


DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of 32 sequences: sigmoid scores, a balancing bias, 4 of 8 groups
        {"name": "route_step", "op": "route", "T": 32, "E": 256, "k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "topk_groups": 4, "group_top": 2, "renorm": True,
         "scale": 2.5, "dtype": "f32", "masked": False, "grad": False},
        # a training step's router: softmax, renormalised, forward and backward
        {"name": "route_train", "op": "route", "T": 65536, "E": 128, "k": 8, "score": "softmax",
         "bias": False, "groups": 1, "topk_groups": 1, "group_top": 1, "renorm": True,
         "scale": 1.0, "dtype": "bf16", "masked": True, "grad": True},
        # the expert order of that decoding step
        {"name": "plan_step", "op": "plan", "T": 32, "E": 256, "k": 8, "masked": False},
        # ... and of a long batch of prompts with padding tokens
        {"name": "plan_prompt", "op": "plan", "T": 131072, "E": 128, "k": 8, "masked": True},
        # the decoding step's rows in expert order, quantised on the way
        {"name": "quantize_step", "op": "quantize", "T": 32, "k": 8, "K": 7168, "dtype": "bf16",
         "gather": True, "masked": False},
        # a prompt's activations quantised before a dense layer
        {"name": "quantize_prompt", "op": "quantize", "T": 16384, "k": 1, "K": 7168,
         "dtype": "bf16", "gather": False, "masked": False},
        # a dense layer with a bias, one decoding step of four sequences
        {"name": "int8_step", "op": "dense", "M": 4, "N": 14336, "K": 4096, "bias": True,
         "dtype": "bf16"},
        # the same layer over a prompt
        {"name": "int8_prompt", "op": "dense", "M": 4096, "N": 14336, "K": 4096, "bias": False,
         "dtype": "bf16"},
        # experts of a decoding step: every expert's weights read for a row or a few
        {"name": "experts_step", "op": "grouped", "total": 256, "G": 64, "N": 2048, "K": 7168,
         "dtype": "bf16"},
        # experts of a long prompt
        {"name": "experts_prompt", "op": "grouped", "total": 16384, "G": 8, "N": 7168, "K": 2304,
         "dtype": "bf16"},
        # the weighted sum of a decoding step
        {"name": "combine_step", "op": "combine", "T": 32, "k": 8, "H": 7168, "dtype": "bf16",
         "masked": False, "grad": False},
        # a training step's weighted sum, forward and backward
        {"name": "combine_train", "op": "combine", "T": 8192, "k": 8, "H": 4096, "dtype": "bf16",
         "masked": True, "grad": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "plan", "quantize", "dense", "grouped", "combine"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op == "route":
        grouped = flag()
        groups = rng.choice([2, 4, 8, 16]) if grouped else 1
        per = _log(rng, 3, 1024 // groups) if grouped else _log(rng, 2, 1024)
        if per * groups > 512 and flag():
            per = max(2, per // 3)
        E = per * groups
        take = rng.randint(1, groups)
        k = rng.randint(1, min(16, take * per))
        case = {"op": op, "T": _log(rng, 1, 65536 * 128 / E), "E": E, "k": k,
                "score": rng.choice(["softmax", "sigmoid"]), "bias": flag(), "groups": groups,
                "topk_groups": take, "group_top": min(rng.choice([1, 2]), per), "renorm": flag(),
                "scale": rng.choice([1.0, 2.5]), "dtype": rng.choice(["bf16", "f32"]),
                "masked": flag(), "grad": flag()}
        case["T"] = min(case["T"], 65536)
        return case
    if op == "plan":
        return {"op": op, "T": _log(rng, 1, 131072), "E": _log(rng, 2, 1024),
                "k": rng.randint(1, 8), "masked": flag()}
    if op == "quantize":
        k = rng.choice([1, 2, 4, 8])
        K = 16 * _log(rng, 4, 1024)
        return {"op": op, "T": min(_log(rng, 1, 16384 * 7168 / K / k / 2), 65536), "k": k, "K": K,
                "dtype": rng.choice(["bf16", "f32"]), "gather": k > 1 or flag(), "masked": flag()}
    if op == "dense":
        N, K = _log(rng, 64, 16384), 16 * _log(rng, 4, 896)
        return {"op": op, "M": min(_log(rng, 1, 8192), max(1, int(4096 * 14336 * 4096 / N / K))),
                "N": N, "K": K, "bias": flag(), "dtype": rng.choice(["bf16", "f32"])}
    if op == "grouped":
        G, K = _log(rng, 1, 256), 16 * _log(rng, 8, 448)
        N = _log(rng, 64, max(64, min(16384, (1 << 30) // (G * K))))
        total = min(_log(rng, 1, 16384), max(1, int(16384 * 7168 * 2304 / N / K)))
        return {"op": op, "total": total, "G": G, "N": N, "K": K,
                "dtype": rng.choice(["bf16", "f32"])}
    k = rng.randint(1, 8)
    dtype = rng.choice(["bf16", "f32"])
    H = 8 * _log(rng, 8, 1024)
    most = 8192 * 8 * 4096 * 2 // (H * k * SIZE[dtype])
    return {"op": op, "T": min(_log(rng, 1, max(1, most)), 65536), "k": k, "H": H, "dtype": dtype,
            "masked": flag(), "grad": flag()}


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k, s = case["T"], case["E"], case["k"], SIZE[case["dtype"]]
        b = T * E * s + 8 * T * k + (4 * E if case["bias"] else 0)
        if case["grad"]:
            b += T * E * s + 4 * T * k
        return {"bytes": b, "flops": T * E * (8 if case["grad"] else 4)}
    if op == "plan":
        return {"bytes": 12 * case["T"] * case["k"] + 8 * case["E"], "flops": 0}
    if op == "quantize":
        rows = case["T"] * case["k"]
        b = case["T"] * case["K"] * SIZE[case["dtype"]] + rows * (case["K"] + 4)
        return {"bytes": b + (4 * rows if case["gather"] else 0), "flops": 3 * rows * case["K"]}
    if op == "dense":
        M, N, K = case["M"], case["N"], case["K"]
        b = M * K + N * K + 4 * (M + N) + (2 * N if case["bias"] else 0) + M * N * SIZE[case["dtype"]]
        return {"bytes": b, "flops": 2 * M * N * K}
    if op == "grouped":
        M, N, K = case["total"], case["N"], case["K"]
        busy = sum(m > 0 for m in _sizes(case, 0))
        b = M * K + busy * N * (K + 4) + 4 * M + M * N * SIZE[case["dtype"]] + 8 * case["G"]
        return {"bytes": b, "flops": 2 * M * N * K}
    T, k, H, s = case["T"], case["k"], case["H"], SIZE[case["dtype"]]
    b = T * k * H * s + T * H * s + 8 * T * k
    if case["grad"]:   # the rows and the weights are needed again, but need not be read again
        b += T * H * s + T * k * H * s + 4 * T * k
    return {"bytes": b, "flops": 2 * T * k * H * (3 if case["grad"] else 1)}


# ------------------------------------------------------------------------------- the inputs

def _sizes(case, seed):
    """Rows of each expert: a skewed load, some experts without rows."""
    import numpy as np
    rng = np.random.default_rng([11, seed, case["total"], case["G"]])
    p = rng.gamma(1.5, size=case["G"]) + 1e-9
    if case["G"] >= 4:
        p[rng.permutation(case["G"])[:case["G"] // 8]] = 0
    return [int(m) for m in rng.multinomial(case["total"], p / p.sum())]


def _choice(x, bias, case):
    """Scores and selection keys (those of closed groups at -inf) of a batch of logits, and
    the groups' values, in x's type."""
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    dead = x == -math.inf
    if case["score"] == "softmax":
        top = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
        s = e / e.sum(-1, keepdim=True).clamp_min(1e-30)
    else:
        s = 1 / (1 + torch.exp(-x))
    key = x if bias is None else torch.where(dead, x, s + bias)
    if case["groups"] == 1:
        return s, key, None
    of = torch.where(dead, x, s) if bias is None and case["group_top"] > 1 else key
    per = case["E"] // case["groups"]
    best = torch.sort(of.view(-1, case["groups"], per), dim=-1, descending=True, stable=True)[0]
    best = best[..., :case["group_top"]]
    value = torch.where(best == -math.inf, 0.0, best).sum(-1)
    value = torch.where(best[..., 0] == -math.inf, -math.inf, value)
    first = torch.sort(value, dim=-1, descending=True, stable=True)[1][:, :case["topk_groups"]]
    is_open = torch.zeros_like(value, dtype=torch.bool).scatter_(1, first, True)
    return s, torch.where(is_open.repeat_interleave(per, 1), key, -math.inf), value


def _logits(case, gen):
    """Router logits.  With a bias or summed group values the choice compares rounded sums,
    which no two implementations round alike: tokens whose choice hangs on two of those
    within 1e-6 of each other, and not equal, are drawn again, so that every choice is the
    formula's."""
    T, E = case["T"], case["E"]
    dev = "cuda"
    tilt = torch.randn(E, generator=gen, device=dev) * 0.5

    def tokens(n):
        x = (torch.randn(n, E, generator=gen, device=dev) * 1.5 + tilt).to(DT[case["dtype"]])
        if case["masked"]:
            # some experts closed, and padding tokens that no expert may take
            x = x.masked_fill(torch.rand(n, E, generator=gen, device=dev) < 0.05, -math.inf)
            x[torch.rand(n, generator=gen, device=dev) < 1 / 16] = -math.inf
        return x

    # steps of 0.001, as an update by a fixed step leaves them
    bias = torch.randint(-60, 61, (E,), generator=gen, device=dev) * 0.001 if case["bias"] else None
    x = tokens(T)
    if case["bias"] or case["group_top"] > 1:
        for _ in range(40):
            _, key, value = _choice(x.double(), None if bias is None else bias.double(), case)
            close = torch.zeros(T, dtype=torch.bool, device=dev)
            for v in (key, value):
                if v is not None:
                    v = torch.sort(v, dim=-1, descending=True)[0][:, :max(case["k"], case["groups"]) + 1]
                    gap = v[:, :-1] - v[:, 1:]
                    close |= ((gap > 0) & (gap < 1e-6)).any(-1)
            at = close.nonzero().flatten()
            if not len(at):
                break
            x[at] = tokens(len(at))
    return x, bias


def _chosen(case, gen, rows_E=None):
    """Expert ids [T, k]: distinct in a token, unevenly loaded, -1 for a padding token."""
    T, k, E = case["T"], case["k"], rows_E or case["E"]
    tilt = torch.randn(E, generator=gen, device="cuda")
    noise = torch.rand(T, E, generator=gen, device="cuda").clamp_min_(1e-9)
    ids = (tilt - torch.log(-torch.log(noise))).argsort(-1, descending=True)[:, :k].to(torch.int32)
    if k > E:
        ids = torch.cat([ids, ids.new_full((T, k - E), -1)], 1)
    if case["masked"]:
        ids[torch.rand(T, generator=gen, device="cuda") < 1 / 16] = -1
    return ids.contiguous()


def _order(ids, E):
    """m_sizes, src and pos of ids by a stable sort."""
    flat = ids.flatten().long()
    at = torch.where(flat < 0, E, flat)
    order = torch.sort(at, stable=True)[1]
    m_sizes = (at[:, None] == torch.arange(E, device=at.device)).sum(0) if at.numel() * E < 1 << 26 \
        else torch.zeros(E + 1, dtype=torch.int64, device=at.device).index_add_(
            0, at, torch.ones_like(at))[:E]
    rows = torch.arange(len(flat), device=at.device)
    used = rows < m_sizes.sum()
    src = torch.where(used, order, -1).to(torch.int32)
    pos = torch.empty_like(order)
    pos[order] = rows
    return m_sizes, src, torch.where(flat < 0, -1, pos).to(torch.int32).view(ids.shape)


def _codes(shape, gen):
    """INT8 codes of normal values whose largest of a row is about 4 sigma."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    return (x * 31).round().clamp(-127, 127).to(torch.int8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    op, st = case["op"], {"case": case}
    if op == "route":
        st["x"], st["bias"] = _logits(case, gen)
        if case["grad"]:
            st["dw"] = torch.randn(case["T"], case["k"], generator=gen, device="cuda")
    elif op == "plan":
        st["ids"] = _chosen(case, gen)
    elif op == "quantize":
        st["x"] = (torch.randn(case["T"], case["K"], generator=gen, device="cuda")
                   * torch.exp(torch.randn(case["T"], 1, generator=gen, device="cuda"))).to(DT[case["dtype"]])
        st["src"] = _order(_chosen(case, gen, 64), 64)[1] if case["gather"] else None
    elif op == "dense":
        st["a"], st["b"] = _codes((case["M"], case["K"]), gen), _codes((case["N"], case["K"]), gen)
        st["sa"] = torch.rand(case["M"], generator=gen, device="cuda") * 0.03 + 0.01
        st["sb"] = torch.rand(case["N"], generator=gen, device="cuda") * 0.0003 + 0.0001
        st["bias"] = torch.randn(case["N"], generator=gen, device="cuda").bfloat16() if case["bias"] else None
    elif op == "grouped":
        G, N, K = case["G"], case["N"], case["K"]
        st["sizes"] = _sizes(case, seed)
        st["m_sizes"] = torch.tensor(st["sizes"], dtype=torch.int64, device="cuda")
        st["a"] = _codes((case["total"], K), gen)
        st["b"] = torch.stack([_codes((N, K), gen) for _ in range(G)])
        st["sa"] = torch.rand(case["total"], generator=gen, device="cuda") * 0.03 + 0.01
        st["sb"] = torch.rand(G, N, generator=gen, device="cuda") * 0.0003 + 0.0001
    else:
        T, k, H = case["T"], case["k"], case["H"]
        _, st["src"], st["pos"] = _order(_chosen(case, gen, 64), 64)
        st["y"] = torch.randn(T * k, H, generator=gen, device="cuda").to(DT[case["dtype"]])
        w = torch.rand(T, k, generator=gen, device="cuda") + 0.05
        st["w"] = w / w.sum(-1, keepdim=True)
        if case["grad"]:
            st["dout"] = torch.randn(T, H, generator=gen, device="cuda").to(DT[case["dtype"]])
    if own:
        _bs()
    return st


# ------------------------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    import block_scaled_precision_mma_gb300 as bs
    c = st["case"]
    op = c["op"]
    if op == "route":
        ids, w = bs.moe_route(st["x"], c["k"], score=c["score"], bias=st["bias"],
                              groups=c["groups"], topk_groups=c["topk_groups"],
                              group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"])
        if not c["grad"]:
            return ids, w
        return ids, w, bs.moe_route_backward(st["x"], ids, st["dw"], score=c["score"],
                                             renormalize=c["renorm"], scale=c["scale"])
    if op == "plan":
        return bs.moe_plan(st["ids"], c["E"])
    if op == "quantize":
        return bs.int8_quantize(st["x"], src=st["src"], k=c["k"])
    if op == "dense":
        return bs.int8_gemm(st["a"], st["sa"], st["b"], st["sb"], bias=st["bias"], dtype=DT[c["dtype"]])
    if op == "grouped":
        return bs.grouped_int8_gemm(st["a"], st["sa"], st["b"], st["sb"], st["m_sizes"],
                                    dtype=DT[c["dtype"]])
    out = bs.moe_combine(st["y"], st["pos"], st["w"])
    if not c["grad"]:
        return out
    return (out,) + tuple(bs.moe_combine_backward(st["dout"], st["y"], st["src"], st["pos"], st["w"]))


def _run_plain(st):
    c = st["case"]
    op = c["op"]
    if op == "route":
        x = st["x"].float()
        s, key, _ = _choice(x, st["bias"], c)
        best, ids = torch.sort(key, dim=-1, descending=True, stable=True)
        best, ids = best[:, :c["k"]], ids[:, :c["k"]]
        used = best > -math.inf
        p = torch.where(used, s.gather(1, ids), 0.0)
        total = p.sum(-1, keepdim=True)
        share = torch.where(total > 0, p / total, 0.0)
        w = (share if c["renorm"] else p) * c["scale"]
        out = torch.where(used, ids, -1).to(torch.int32), w
        if not c["grad"]:
            return out
        g = torch.where(used, st["dw"], 0.0) * c["scale"]
        if c["renorm"]:
            # of the scores: ds = (g - <g, share>) / total
            ds = torch.where(total > 0, (g - (g * share).sum(-1, keepdim=True)) / total, 0.0)
        else:
            ds = g
        full = torch.zeros_like(s).scatter_add_(1, ids, torch.where(used, ds, 0.0))
        if c["score"] == "softmax":
            dx = s * (full - (full * s).sum(-1, keepdim=True))
        else:
            dx = full * s * (1 - s)
        return out + (dx.to(st["x"].dtype),)
    if op == "plan":
        return _order(st["ids"], c["E"])
    if op == "quantize":
        x = st["x"].float()
        if st["src"] is not None:
            at = st["src"].long()
            x = torch.where((at >= 0)[:, None], x[at.clamp_min(0) // c["k"]], 0.0)
        s = x.abs().amax(-1) / 127
        s = torch.where(s == 0, 1.0, s)
        return torch.round(x / s[:, None]).clamp(-127, 127).to(torch.int8), s
    if op == "dense":
        d = (st["a"].float() @ st["b"].float().T) * st["sa"][:, None] * st["sb"]
        return (d if st["bias"] is None else d + st["bias"].float()).to(DT[c["dtype"]])
    if op == "grouped":
        parts = torch.split(st["a"], st["sizes"])
        d = torch.cat([a.float() @ st["b"][g].float().T * st["sb"][g]
                       for g, a in enumerate(parts) if len(a)])
        return (d * st["sa"][:, None]).to(DT[c["dtype"]])
    used = st["pos"] >= 0
    at = st["pos"].clamp_min(0).long()
    w = torch.where(used, st["w"], 0.0)
    y = st["y"][at].float()
    out = (y * w[..., None]).sum(1).to(st["y"].dtype)
    if not c["grad"]:
        return out
    dout = st["dout"].float()
    dw = torch.where(used, (y * dout[:, None]).sum(-1), 0.0)
    slot = st["src"].clamp_min(0).long()
    dy = torch.where((st["src"] >= 0)[:, None], w.flatten()[slot][:, None] * dout[slot // c["k"]], 0.0)
    return out, dy.to(st["y"].dtype), dw


# ------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    st = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None   # whole numbers only
    if op == "route":
        return _exact_route(case, st)
    if op == "quantize":
        # the codes are whole numbers of FP32 steps; only the scale has a value of its own
        big = st["x"].double().abs().amax(1)
        if st["src"] is not None:
            big = torch.cat([big, big.new_zeros(1)])
            big = big[torch.where(st["src"] < 0, case["T"], st["src"].long() // case["k"])]
        big[big == 0] = 127
        return None, big / 127
    if op == "dense":
        d = torch.einsum("mk,nk->mn", st["a"].double(), st["b"].double())
        d = d * torch.outer(st["sa"].double(), st["sb"].double())
        return d + st["bias"].double() if case["bias"] else d
    if op == "grouped":
        d = torch.zeros(case["total"], case["N"], dtype=torch.float64, device="cuda")
        row = 0
        for g, m in enumerate(st["sizes"]):
            if m:
                d[row:row + m] = torch.einsum("mk,nk->mn", st["a"][row:row + m].double(),
                                              st["b"][g].double() * st["sb"][g].double()[:, None])
            row += m
        return d * st["sa"].double()[:, None]
    T, k, H = case["T"], case["k"], case["H"]
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    dy = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = (st["pos"][:, j] >= 0).nonzero().flatten()
        r = st["pos"][t, j].long()
        w = st["w"][t, j].double()[:, None]
        out[t] += w * st["y"][r].double()
        if case["grad"]:
            dw[t, j] = torch.einsum("th,th->t", st["y"][r].double(), st["dout"][t].double())
            dy[r] = w * st["dout"][t].double()
    return (out, dy, dw) if case["grad"] else out


def _exact_route(case, st):
    import numpy as np
    T, E, k = case["T"], case["E"], case["k"]
    x = st["x"].double().cpu().numpy()
    bias = None if st["bias"] is None else st["bias"].double().cpu().numpy()
    with np.errstate(all="ignore"):
        if case["score"] == "softmax":
            m = x.max(1)
            m[m == -np.inf] = 0
            s = np.exp(x - m[:, None])
            s /= np.maximum(s.sum(1), 1e-300)[:, None]
        else:
            s = 1 / (1 + np.exp(-x))
    key = x.copy() if bias is None else np.where(x == -np.inf, -np.inf, s + bias)
    if case["groups"] > 1:
        by = (np.where(x == -np.inf, -np.inf, s) if bias is None and case["group_top"] > 1 else key)
        by = np.sort(by.reshape(T, case["groups"], -1), axis=2)[:, :, ::-1][:, :, :case["group_top"]]
        lead = by[:, :, 0]
        value = np.where(lead == -np.inf, -np.inf, np.where(by == -np.inf, 0, by).sum(2))
        rank = np.argsort(np.argsort(-value, axis=1, kind="stable"), axis=1, kind="stable")
        key[np.repeat(rank >= case["topk_groups"], E // case["groups"], axis=1)] = -np.inf
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    used = np.take_along_axis(key, ids, 1) > -np.inf
    p = np.take_along_axis(s, ids, 1) * used
    total = p.sum(1, keepdims=True)
    norm = np.where(total > 0, total, 1) if case["renorm"] else np.ones_like(total)
    w = p / norm * case["scale"]
    ids_out = np.where(used, ids, -1).astype(np.int32)
    if not case["grad"]:
        return ids_out, w
    g = st["dw"].double().cpu().numpy() * used
    dp = case["scale"] * g / norm
    if case["renorm"]:
        dp = (dp - (g * w).sum(1, keepdims=True) / norm) * used
    ds = np.zeros_like(s)
    np.put_along_axis(ds, ids, dp, 1)
    dx = s * (1 - s) * ds if case["score"] == "sigmoid" else s * ds - s * (s * ds).sum(1, keepdims=True)
    return ids_out, w, dx
