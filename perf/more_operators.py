"""Cases of the residual branch's operators: the norm before a block, the step after it (norm,
gate, dropout, residual and the next block's norm), their gradients, dropout by itself, and the
expert layer of a decoding step.

``own`` false: plain elementary torch operations in FP32.  ``own`` true: the calls a user
makes of block_scaled_precision_mma_gb300.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
BITS = {"bf16": 16, "f32": 32, "e4m3": 8.25, "e5m2": 8.25, "int8": 8, "e2m1": 4.25}   # with their scales
FLOAT8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of eight sequences: the norm before a block
        {"name": "enter_step", "op": "enter", "T": 8, "H": 7168, "dtype": "bf16", "out": "bf16",
         "norm": "rms", "bias": False, "grad": False},
        # a prompt's rows, normed straight into an MXFP8 product's operand
        {"name": "enter_prompt", "op": "enter", "T": 16384, "H": 7168, "dtype": "bf16",
         "out": "e4m3", "norm": "rms", "bias": False, "grad": False},
        # a training step with an FP32 residual stream: forward, and the gradients with the
        # stream's own added
        {"name": "enter_train", "op": "enter", "T": 16383, "H": 4096, "dtype": "f32",
         "out": "bf16", "norm": "layer", "bias": True, "grad": True},
        # a decoding step of 32 sequences after a block: norm, gate by channel, residual, and the
        # next block's norm
        {"name": "leave_step", "op": "leave", "T": 32, "H": 7168, "dtype": "bf16", "ydtype": "bf16",
         "norm": "rms", "bias": False, "rows": 32, "x_scale": 1.0, "y_scale": 1.0, "p": 0.0,
         "next": "rms", "out": "bf16", "grad": False},
        # a prompt: residual and the next norm into an MXFP8 operand
        {"name": "leave_prompt", "op": "leave", "T": 16384, "H": 4096, "dtype": "bf16",
         "ydtype": "bf16", "norm": "none", "bias": False, "rows": 0, "x_scale": 1.0, "y_scale": 1.0,
         "p": 0.0, "next": "rms", "out": "e4m3", "grad": False},
        # a training step of ragged sequences: norm, a gate for each 2048 rows, dropout and the next
        # block's norm, and the gradients of what came before that one
        {"name": "leave_train", "op": "leave", "T": 15000, "H": 7168, "dtype": "bf16",
         "ydtype": "bf16", "norm": "rms", "bias": False, "rows": 2048, "x_scale": 1.0,
         "y_scale": 0.5, "p": 0.1, "next": "rms", "out": "bf16", "grad": True},
        # dropout of a small batch's activations, forward and backward
        {"name": "dropout_small", "op": "dropout", "T": 512, "H": 1024, "dtype": "bf16", "p": 0.1,
         "grad": True},
        # ... and of a long one's inner activations
        {"name": "dropout_train", "op": "dropout", "T": 16384, "H": 14336, "dtype": "bf16",
         "p": 0.1, "grad": True},
        # the expert layer of one token: the eight chosen experts' weights are read for one row
        {"name": "moe_token", "op": "moe", "T": 1, "E": 64, "k": 8, "H": 7168, "F": 2048,
         "fmt": "e4m3", "act": "silu", "masked": False},
        # a small layer, two sequences
        {"name": "moe_small", "op": "moe", "T": 2, "E": 32, "k": 4, "H": 1024, "F": 2048,
         "fmt": "bf16", "act": "silu", "masked": False},
        # a decoding step of 32 sequences: nearly every expert has a row or a few
        {"name": "moe_step", "op": "moe", "T": 32, "E": 64, "k": 8, "H": 7168, "F": 2048,
         "fmt": "int8", "act": "silu", "masked": False},
        # few wide experts in MXFP4, three sequences
        {"name": "moe_wide", "op": "moe", "T": 3, "E": 8, "k": 2, "H": 4096, "F": 14336,
         "fmt": "e2m1", "act": "gelu", "masked": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["enter", "leave", "leave", "dropout", "moe"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op == "moe":
        fmt = rng.choice(["bf16", "int8", "e4m3", "e5m2", "e2m1"])
        step = {"bf16": 8, "int8": 16}.get(fmt, 32)
        E = _log(rng, 2, 128)
        k = rng.randint(1, min(8, E))
        H = step * max(1, _log(rng, 256, 7168) // step)
        F = step * max(1, _log(rng, 128, min(14336, max(256, 64 * 2048 * 7168 // (E * H)))) // step)
        return {"op": op, "T": _log(rng, 1, 32), "E": E, "k": k, "H": H, "F": F, "fmt": fmt,
                "act": rng.choice(["silu", "gelu", "relu"]), "masked": flag()}
    dtype = rng.choice(["bf16", "f32"])
    if op == "dropout":
        H = 8 * _log(rng, 8, 1792)
        return {"op": op, "T": _log(rng, 1, 16384 * 14336 // H // 2), "H": H, "dtype": dtype,
                "p": rng.choice([0.05, 0.1, 0.5]), "grad": flag()}
    grad = flag()
    out = rng.choice(["bf16", "f32"] if dtype == "f32" else ["bf16"]) if grad or flag() \
        else rng.choice(["e4m3", "e5m2"])
    step = 32 if out in FLOAT8 else 8
    H = step * max(1, _log(rng, 64, 8192) // step)
    T = _log(rng, 1, 15000 * 7168 // H // (2 if dtype == "f32" else 1))
    case = {"op": op, "T": min(T, 65536), "H": H, "dtype": dtype, "out": out}
    if op == "enter":
        norm = rng.choice(["rms", "layer"])
        return {**case, "norm": norm, "bias": norm == "layer" and flag(), "grad": grad}
    norm = rng.choice(["none", "rms", "layer"])
    after = rng.choice(["none", "rms", "layer"]) if out not in FLOAT8 else rng.choice(["rms", "layer"])
    # one gate for all rows, for each sequence (the last one may be short), or for each row
    rows = rng.choice([0, case["T"], max(1, case["T"] // rng.randint(2, 9)), 1])
    return {**case, "ydtype": "bf16" if dtype == "bf16" or out == "bf16" else "f32", "norm": norm,
            "bias": norm == "layer" and flag(), "rows": rows, "x_scale": rng.choice([1.0, 1.0, 0.75]),
            "y_scale": rng.choice([1.0, 0.5]), "p": rng.choice([0.0, 0.1]) if grad else 0.0,
            "next": after, "grad": grad}


def work(case):
    op, T, H = case["op"], case["T"], case["H"]
    if op == "moe":
        E, k, F = case["E"], case["k"], case["F"]
        busy = E * (1 - (1 - k / E) ** T)   # experts that some token chose, on average
        b = busy * 3 * F * H * BITS[case["fmt"]] / 8 + 4 * T * H + 8 * T * k
        if case["fmt"] == "int8":
            b += busy * 4 * (2 * F + H)
        return {"bytes": b, "flops": 6 * T * k * F * H}
    n, s = T * H, SIZE[case["dtype"]]
    if op == "dropout":
        return {"bytes": 2 * n * s * (2 if case["grad"] else 1), "flops": n * (2 if case["grad"] else 1)}
    so = BITS[case["out"]] / 8
    if op == "enter":
        b, f = n * (s + so), 6 * n
        if case["grad"]:      # x is needed again, but need not be read again
            b, f = b + n * (so + s + s), f + 12 * n
        return {"bytes": b + 4 * H * (2 if case["grad"] else 1), "flops": f}
    sy = SIZE[case["ydtype"]]
    gates = -(-T // case["rows"]) * H if case["rows"] else 0
    b, f = n * (2 * s + sy) + gates * sy, 12 * n
    if case["next"] != "none":
        b += n * so
    if case["grad"]:          # y is needed again, but need not be read again
        b, f = b + n * (s + sy) + gates * 4, f + 20 * n
        if case["x_scale"] != 1:
            b += n * s
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------------------- the inputs

def _experts(shape, fmt, gen):
    """Weights [E, rows, K] of standard deviation about K^-1/2, and their scales."""
    E, rows, K = shape
    dev = "cuda"
    if fmt == "bf16":
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16) * K ** -0.5, None
    if fmt == "int8":
        codes = torch.empty(shape, dtype=torch.int8, device=dev)
        for e in range(E):
            x = torch.randn(rows, K, generator=gen, device=dev, dtype=torch.bfloat16)
            codes[e] = (x * 31).round().clamp(-127, 127).to(torch.int8)
        return codes, (torch.rand(E, rows, generator=gen, device=dev) + 0.5) / 31 / K ** 0.5
    size = {"e4m3": 6, "e5m2": 6, "e2m1": 1}[fmt]     # log2 of the codes' typical value
    low = 127 - size - round(math.log2(K) / 2)
    scales = torch.randint(low - 1, low + 2, (E, rows, K // 32), generator=gen, device=dev).to(torch.uint8)
    if fmt == "e2m1":
        return torch.randint(0, 256, (E, rows, K // 2), generator=gen, device=dev, dtype=torch.uint8), scales
    codes = torch.empty(shape, dtype=torch.uint8, device=dev)
    for e in range(E):
        x = torch.randn(rows, K, generator=gen, device=dev) * 2.0 ** size
        codes[e] = x.clamp(-448, 448).to(FLOAT8[fmt]).view(torch.uint8)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 29)
    dev, op, T, H, st = "cuda", case["op"], case["T"], case["H"], {"case": case}
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    if op == "moe":
        E, k, F = case["E"], case["k"], case["F"]
        st["x"] = rnd(T, H).bfloat16()
        ids = torch.rand(T, E, generator=gen, device=dev).argsort(-1)[:, :k].to(torch.int32)
        w = torch.rand(T, k, generator=gen, device=dev) + 0.05
        if case["masked"]:      # a padding token now and then, and choices that were dropped
            ids[torch.rand(T, generator=gen, device=dev) < 1 / 16] = -1
            ids[torch.rand(T, k, generator=gen, device=dev) < 1 / 16] = -1
        st["ids"], st["w"] = ids.contiguous(), w / w.sum(-1, keepdim=True)
        st["w_in"], st["s_in"] = _experts((E, 2 * F, H), case["fmt"], gen)
        st["w_out"], st["s_out"] = _experts((E, H, F), case["fmt"], gen)
    else:
        # channels of a residual stream differ in size and are not centred
        spread, shift = torch.exp(0.5 * rnd(H)), 0.3 * rnd(H)
        st["x"] = (rnd(T, H) * spread + shift).to(DT[case["dtype"]])
        st["rng"] = torch.stack([torch.randint(0, 1 << 62, (), generator=gen, device=dev),
                                 torch.randint(0, 1 << 40, (), generator=gen, device=dev)])
        if case["grad"]:
            st["dout"] = rnd(T, H).to(DT[case["dtype"]])
    if op in ("enter", "leave"):
        if op == "leave":
            ydt = DT[case["ydtype"]]
            st["y"] = (rnd(T, H) * spread - shift).to(ydt)
            st["gate"] = (0.5 * rnd(-(-T // case["rows"]), H)).to(ydt) if case["rows"] else None
            st["w2"] = 1 + 0.1 * rnd(H) if case["next"] != "none" else None
        st["w"] = 1 + 0.1 * rnd(H) if case["norm"] != "none" else None
        st["b"] = 0.1 * rnd(H) if case["bias"] else None
        if case["grad"] and op == "enter":
            st["dh"] = rnd(T, H).to(DT[case["out"]])
    if own:
        import block_scaled_precision_mma_gb300 as bs
        bs.build()
    return st


# ------------------------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _operand(got, fmt):
    """MX codes and scales as the values they stand for."""
    if fmt not in FLOAT8:
        return got
    return got[0].view(FLOAT8[fmt]), got[1].view(torch.float8_e8m0fnu)


def _run_own(st):
    import block_scaled_precision_mma_gb300 as bs
    c = st["case"]
    op = c["op"]
    if op == "moe":
        return bs.moe_step(st["x"], st["ids"], st["w"], st["w_in"], st["w_out"], s_in=st["s_in"],
                           s_out=st["s_out"], fmt=c["fmt"], act=c["act"])
    if op == "dropout":
        y = bs.dropout(st["x"], c["p"], st["rng"])
        return (y, bs.dropout(st["dout"], c["p"], st["rng"])) if c["grad"] else y
    if op == "enter":
        h = bs.branch_enter(st["x"], st["w"], st["b"], norm=c["norm"], fmt=c["out"])
        if not c["grad"]:
            return _operand(h, c["out"])
        return (h,) + bs.branch_enter_backward(st["dh"], st["x"], st["w"], norm=c["norm"],
                                               dres=st["dout"], bias=c["bias"])
    form = dict(norm=c["norm"], gate=st["gate"], gate_rows=c["rows"], x_scale=c["x_scale"],
                y_scale=c["y_scale"], p=c["p"], rng=st["rng"])
    if c["next"] == "none":
        done = (bs.branch_leave(st["x"], st["y"], st["w"], st["b"], **form),)
    else:
        done = bs.branch_leave(st["x"], st["y"], st["w"], st["b"], next_norm=c["next"],
                               next_weight=st["w2"], fmt=c["out"], **form)
        done = (done[0], _operand(done[1] if len(done) == 2 else done[1:], c["out"]))
    if not c["grad"]:
        return done
    return done + bs.branch_leave_backward(st["dout"], st["y"], st["w"], st["b"], **form)


EPS = 1e-6


def _normed(x, norm):
    """(n, r): x normed, and what it was multiplied by."""
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _norm_grad(dz, n, r, norm):
    d = dz - n * (dz * n).mean(-1, keepdim=True)
    return r * (d - dz.mean(-1, keepdim=True) if norm == "layer" else d)


def _stored(h, fmt):
    """FP32 rows in the output's type; MX: per 32 values a power of two, the codes rounded."""
    if fmt not in FLOAT8:
        return h.to(DT[fmt])
    top, emax = (448.0, 8) if fmt == "e4m3" else (57344.0, 15)
    blocks = h.view(h.shape[0], -1, 32)
    amax = blocks.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 1 - emax, 0).clamp(-127, 127)
    codes = (blocks * torch.exp2(-e.float())[..., None]).clamp(-top, top).to(FLOAT8[fmt])
    return codes.view(h.shape), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _kept(shape, p, rng):
    """The dropout mask: Philox4x32-10 of counter (block of eight values, offset), the seed as its
    key, 16 bits a value."""
    n = shape[0] * shape[1]
    low, high = (lambda v: v & 0xFFFFFFFF), (lambda v: (v >> 32) & 0xFFFFFFFF)  # noqa: E731
    at = torch.arange(n // 8, device=rng.device)
    k0, k1 = low(rng[0]), high(rng[0])
    a, b, c, d = low(at), high(at), low(rng[1]).expand_as(at), high(rng[1]).expand_as(at)
    for _ in range(10):      # the generator's rounds
        u, v = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = high(v) ^ b ^ k0, low(v), high(u) ^ d ^ k1, low(u)
        k0, k1 = low(k0 + 0x9E3779B9), low(k1 + 0xBB67AE85)
    words = torch.stack([a, b, c, d], -1)
    halves = torch.stack([words & 0xFFFF, words >> 16], -1).view(shape)
    return halves >= _threshold(p)


def _threshold(p):
    return min(round(p * 65536), 65535)


def _values(codes, scales, fmt):
    """The FP32 values of weights."""
    if fmt == "bf16":
        return codes.float()
    if fmt == "int8":
        return codes.float() * scales[..., None]
    if fmt == "e2m1":
        lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
        v = lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    else:
        v = codes.view(FLOAT8[fmt]).float()
    v = v.view(*v.shape[:-1], -1, 32) * torch.exp2(scales.float() - 127)[..., None]
    return v.flatten(-2)


def _act(x, act):
    if act == "relu":
        return torch.where(x > 0, x, 0.0)
    return x / (1 + torch.exp(-x)) if act == "silu" else x * (1 + torch.erf(x * 0.5 ** 0.5)) / 2


def _run_plain(st):
    c = st["case"]
    op, x = c["op"], st["x"].float()
    if op == "moe":
        T, k, E = c["T"], c["k"], c["E"]
        used = st["ids"] >= 0
        at = st["ids"].clamp_min(0).long().flatten()
        token = torch.arange(T, device=x.device).repeat_interleave(k)
        if T * k <= E:        # the slots' weights gathered, a row each
            u = (_values(st["w_in"][at], None if st["s_in"] is None else st["s_in"][at], c["fmt"])
                 @ x[token][..., None])[..., 0]
            gate, up = u[:, :c["F"]], u[:, c["F"]:]
            y = (_values(st["w_out"][at], None if st["s_out"] is None else st["s_out"][at], c["fmt"])
                 @ (_act(gate, c["act"]) * up)[..., None])[..., 0]
        else:                 # every expert on every token
            u = x @ _values(st["w_in"], st["s_in"], c["fmt"]).transpose(1, 2)
            gate, up = u[..., :c["F"]], u[..., c["F"]:]
            y = (_act(gate, c["act"]) * up) @ _values(st["w_out"], st["s_out"], c["fmt"]).transpose(1, 2)
            y = y[at, token]
        y = torch.where(used.flatten()[:, None], y * st["w"].flatten()[:, None], 0.0)
        return y.view(T, k, -1).sum(1).bfloat16()
    if op == "dropout":
        keep = _kept(x.shape, c["p"], st["rng"])
        scale = 65536 / (65536 - _threshold(c["p"]))
        y = torch.where(keep, x * scale, 0.0).to(st["x"].dtype)
        if not c["grad"]:
            return y
        return y, torch.where(keep, st["dout"].float() * scale, 0.0).to(st["x"].dtype)
    if op == "enter":
        n, r = _normed(x, c["norm"])
        h = n * st["w"]
        h = _stored(h if st["b"] is None else h + st["b"], c["out"])
        if not c["grad"]:
            return h
        dh = st["dh"].float()
        dx = (_norm_grad(dh * st["w"], n, r, c["norm"]) + st["dout"].float()).to(st["x"].dtype)
        return h, dx, (dh * n).sum(0), dh.sum(0) if c["bias"] else None
    y, n, r = st["y"].float(), None, None
    z = y
    if c["norm"] != "none":
        n, r = _normed(y, c["norm"])
        z = n * st["w"]
        z = z if st["b"] is None else z + st["b"]
    keep = _kept(x.shape, c["p"], st["rng"]) if c["p"] else None
    scale = 65536 / (65536 - _threshold(c["p"]))
    u = z if keep is None else torch.where(keep, z * scale, 0.0)
    rows = c["rows"] or c["T"]
    gate = None if st["gate"] is None else st["gate"].float().repeat_interleave(rows, 0)[:c["T"]]
    out = (c["x_scale"] * x + c["y_scale"] * (u if gate is None else gate * u)).to(st["x"].dtype)
    done = (out,)
    if c["next"] != "none":
        done = (out, _stored(_normed(out.float(), c["next"])[0] * st["w2"], c["out"]))
    if not c["grad"]:
        return done
    d = c["y_scale"] * st["dout"].float()
    dgate = None
    if gate is not None:
        of = d * u
        pad = -(-c["T"] // rows) * rows - c["T"]
        dgate = torch.cat([of, of.new_zeros(pad, c["H"])]).view(-1, rows, c["H"]).sum(1)
        d = d * gate
    dz = d if keep is None else torch.where(keep, d * scale, 0.0)
    dw = db = None
    dy = dz
    if c["norm"] != "none":
        dw, db = (dz * n).sum(0), dz.sum(0) if c["bias"] else None
        dy = _norm_grad(dz * st["w"], n, r, c["norm"])
    dx = st["dout"] if c["x_scale"] == 1 else (c["x_scale"] * st["dout"].float()).to(st["x"].dtype)
    return done + (dy.to(st["y"].dtype), dx, dw, db, dgate)


# ------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    st = prepare(case, seed)
    op, T, H = case["op"], case["T"], case["H"]
    wide = {k: v.double() for k, v in st.items()
            if isinstance(v, torch.Tensor) and v.is_floating_point() and op != "moe"}
    if op == "moe":
        return _exact_moe(case, st)
    if op == "dropout":
        m = _exact_mask(T * H, case["p"], st["rng"].tolist()).view(T, H)
        return (wide["x"] * m, wide["dout"] * m) if case["grad"] else wide["x"] * m
    weight, bias = wide.get("w"), wide.get("b")
    if op == "enter":
        h, pull = _exact_norm(wide["x"], case["norm"], weight, bias)
        if not case["grad"]:
            return _exact_operand(h, case["out"])
        dx, dw, db = pull(wide["dh"])
        return h, dx + wide["dout"], dw, db if case["bias"] else None
    z, pull = _exact_norm(wide["y"], case["norm"], weight, bias)
    m = _exact_mask(T * H, case["p"], st["rng"].tolist()).view(T, H) if case["p"] else 1.0
    of = torch.arange(T, device="cuda") // (case["rows"] or T)
    g = wide["gate"][of] if "gate" in wide else 1.0
    branch = g * m * case["y_scale"]
    out = torch.addcmul(wide["x"] * case["x_scale"], branch * torch.ones_like(z), z)
    done = (out,)
    if case["next"] != "none":
        # the next block's norm is of the row as it is stored
        h, _ = _exact_norm(out.to(st["x"].dtype).double(), case["next"], wide["w2"], None)
        done = out, _exact_operand(h, case["out"])
    if not case["grad"]:
        return done
    total, dg = wide["dout"], None
    if "gate" in wide:
        dg = torch.zeros_like(wide["gate"]).index_add_(0, of, total * z * m * case["y_scale"])
    dy, dw, db = pull(total * branch)
    return done + (dy, total * case["x_scale"], dw, db if case["bias"] else None, dg)


def _exact_norm(x, norm, weight, bias):
    """n(x) * weight + bias and its gradients' function."""
    if norm == "none":
        return x, lambda d: (d, None, None)
    H = x.shape[1]
    mean = torch.einsum("th->t", x) / H if norm == "layer" else torch.zeros_like(x[:, 0])
    var = torch.einsum("th,th->t", x, x) / H - mean ** 2
    sd = (var + EPS).sqrt()[:, None]
    n = (x - mean[:, None]) / sd

    def pull(d):
        dn = d * weight
        inner = torch.einsum("th,th->t", dn, n)[:, None] / H
        centre = torch.einsum("th->t", dn)[:, None] / H if norm == "layer" else 0.0
        return (dn - centre - inner * n) / sd, torch.einsum("th,th->h", d, n), torch.einsum("th->h", d)

    return (n * weight if bias is None else torch.addcmul(bias, n, weight)), pull


def _exact_operand(h, fmt):
    if fmt not in FLOAT8:
        return h
    at = h.unflatten(1, (-1, 32))
    big = at.abs().max(2).values
    scale = torch.pow(2.0, torch.floor(torch.log2(big)) - (8 if fmt == "e4m3" else 15))
    scale[big == 0] = 1
    most, lowest, bits = (448, -6, 3) if fmt == "e4m3" else (57344, -14, 2)
    v = (at / scale[..., None]).clamp(-most, most)
    step = torch.pow(2.0, torch.floor(torch.log2(v.abs().clamp_min(2.0 ** lowest))) - bits)
    return ((v / step).round() * step).clamp(-most, most).flatten(1), scale


def _exact_mask(n, p, numbers):
    """0 or 1 / (1 - p) for each value, the generator in unsigned 64-bit integers on the host."""
    import numpy as np
    seed, offset = (v & (2 ** 64 - 1) for v in numbers)
    drop = min(round(p * 65536), 65535)
    kept = np.empty(n, dtype=bool)
    half, mask = np.uint64(32), np.uint64(0xFFFFFFFF)
    for at in range(0, n // 8, 1 << 18):
        ctr = np.arange(at, min(at + (1 << 18), n // 8), dtype=np.uint64)
        x = [ctr & mask, ctr >> half, np.full_like(ctr, offset & 0xFFFFFFFF), np.full_like(ctr, offset >> 32)]
        key = [seed & 0xFFFFFFFF, seed >> 32]
        for _ in range(10):
            first, second = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
            x = [(second >> half) ^ x[1] ^ np.uint64(key[0]), second & mask,
                 (first >> half) ^ x[3] ^ np.uint64(key[1]), first & mask]
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        values = np.stack([w >> np.uint64(16 * h) & np.uint64(0xFFFF) for w in x for h in (0, 1)], 1)
        kept[8 * at:8 * (at + len(ctr))] = (values >= drop).ravel()
    return torch.from_numpy(kept).cuda().double() / (1 - drop / 65536)


def _exact_moe(case, st):
    T, F = case["T"], case["F"]
    out = torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")

    def weight(name, e):
        w, s = st["w_" + name][e], st["s_" + name]
        if case["fmt"] == "bf16":
            return w.double()
        if case["fmt"] == "int8":
            return w.double() * s[e].double()[:, None]
        if case["fmt"] == "e2m1":
            w = torch.stack((w % 16, w // 16), 2).reshape(w.shape[0], -1).long()
            size = w % 8
            v = torch.where(size < 2, size * 0.5, (1 + 0.5 * (size % 2)) * 2.0 ** (size // 2 - 1).double())
            v = torch.where(w > 7, -v, v).double()
        else:
            v = w.view(FLOAT8[case["fmt"]]).double()
        return v * (2.0 ** (s[e].double() - 127)).repeat_interleave(32, 1)

    for e in st["ids"].unique().tolist():
        if e < 0:
            continue
        t, j = (st["ids"] == e).nonzero(as_tuple=True)
        u = torch.einsum("th,fh->tf", st["x"][t].double(), weight("in", e))
        g, up = u[:, :F], u[:, F:]
        if case["act"] == "silu":
            g = g * torch.sigmoid(g)
        elif case["act"] == "gelu":
            g = g * 0.5 * torch.special.erfc(-g / math.sqrt(2))
        else:
            g = g.clamp_min(0)
        y = torch.einsum("tf,hf->th", g * up, weight("out", e))
        out.index_add_(0, t, y * st["w"][t, j].double()[:, None])
    return out
