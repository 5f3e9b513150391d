"""The residual branch's operators on the GPU against their definitions in 64 bits.

Tolerances.  An output rounded to type t is off by half a step, finfo(t).eps / 2 of its value.
Before that, FP32: a thread adds up to 32 values and the row's threads are joined in at most 10
steps, so a sum of positive terms is within 42 * 2^-24 of itself; half of that in a square root's
argument, the reciprocal root 2 ulp, each product half of one: a normed value is within 2^-18 of
the size of its terms, |v| / sd + mean|v| / sd (the mean that is taken off is off by that much).
A gradient goes through two such sums and their products: 2^-16 of its terms' sizes.  A sum over
the rows adds at most 64 rows in a run here and joins at most 304 runs: with each term's own
error below 2^-15 of the terms' sizes."""
import pytest
import torch

import block_scaled_precision_mma_gb300 as bs
from tests import branch_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GUARD = 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bs.build()
    bs.load()
    torch.cuda.init()


def guarded(shape, dtype):
    """An output inside a buffer whose ends must keep what they hold."""
    n = 1
    for s in shape:
        n *= s
    raw = torch.full((n + 2 * GUARD,), 77, dtype=dtype, device="cuda")
    return raw, raw[GUARD:GUARD + n].view(shape)


def intact(raw):
    return bool((raw[:GUARD] == 77).all() and (raw[-GUARD:] == 77).all())


def near(got, want, size, what):
    got, want = got.double().cpu(), want.double()
    tol = torch.finfo(what).eps / 2 * want.abs() + size
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][:3], want[bad][:3],
                           torch.broadcast_to(tol, bad.shape)[bad][:3])


def rows(g, T, H, dtype, mean=0.3):
    x = torch.randn(T, H, generator=g) * torch.exp(0.5 * torch.randn(H, generator=g))
    return (x + mean * torch.randn(H, generator=g)).to(DT[dtype])


def columns(g, H, want):
    return torch.randn(H, generator=g) if want else None


def wide(t):
    return None if t is None else t.double()


def dev(t):
    return None if t is None else t.cuda()


def normed_size(v, kind, weight, bias, eps=1e-6):
    """2^-18 of the sizes of n(v) * weight + bias's terms."""
    if kind == "none":
        return 2.0 ** -24 * v.abs()
    _, r = ref.stats(v, kind, eps)
    size = (v.abs() + v.abs().mean(1, keepdim=True)) * r
    size = size if weight is None else size * weight.abs()
    return 2.0 ** -18 * (size if bias is None else size + bias.abs())


SIZES = [(1, 8), (3, 264), (6, 1024), (5, 1032), (33, 4096), (2, 4104), (9, 7168), (4, 8200), (3, 16384),
         (700, 520), (2500, 192), (1300, 408)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
def test_enter(T, H, kind, dtype, out):
    g = torch.Generator().manual_seed(T * 100003 + H)
    x, w, b = rows(g, T, H, dtype), columns(g, H, T % 2), columns(g, H, kind == "layer")
    raw, h = guarded((T, H), DT[out])
    bs.branch_enter(dev(x), dev(w), dev(b), norm=kind, fmt=out, out=h)
    torch.cuda.synchronize()
    assert intact(raw)
    want = ref.norm(x.double(), kind, wide(w), wide(b))
    near(h, want, normed_size(x.double(), kind, wide(w), wide(b)), DT[out])


@pytest.mark.parametrize("T,H", [(1, 32), (3, 288), (5, 1024), (70, 2080), (9, 7168), (3, 16384)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3", "e5m2", "e2m1"])
def test_operands_are_the_quantisers(T, H, fmt):
    """Codes and scales are exactly what the library's quantisers make of the FP32 rows."""
    g = torch.Generator().manual_seed(T * 1009 + H)
    x, w = dev(rows(g, T, H, "f32")), dev(columns(g, H, True))
    x[T // 2, H // 2] = 1e4            # a row whose other blocks are small
    if T > 2:
        x[1] = 0                       # a row of zeros
    h = bs.branch_enter(x, w, fmt="f32")
    want = bs.int8_quantize(h) if fmt == "int8" else bs.mx_quantize(h, fmt)
    raw, out = guarded(tuple(want[0].shape), want[0].dtype)
    sraw, scales = guarded(tuple(want[1].shape), want[1].dtype)
    bs.branch_enter(x, w, fmt=fmt, out=out, scales=scales)
    torch.cuda.synchronize()
    assert intact(raw) and intact(sraw)
    assert torch.equal(out, want[0]) and torch.equal(scales, want[1])
    # and after a block, of the stored row
    y = dev(rows(g, T, H, "f32"))
    o, codes, scales = bs.branch_leave(x, y, next_norm="rms", next_weight=w, fmt=fmt)
    want = bs.branch_enter(o, w, fmt=fmt)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


def leave_case(g, T, H, dtype, ydtype, kind, gate_rows, p):
    c = {"x": rows(g, T, H, dtype), "y": rows(g, T, H, ydtype, -0.2)}
    c["w"] = columns(g, H, kind != "none" and H % 16 == 0)
    c["b"] = columns(g, H, kind == "layer")
    c["gate"] = torch.randn(-(-T // gate_rows), H, generator=g).to(DT[ydtype]) if gate_rows else None
    c["rng"] = torch.tensor([(T << 33) + H, 7 + (1 << 35)])
    c["keep"] = ref.mask(T * H, p, (T << 33) + H, 7 + (1 << 35)).view(T, H) if p else 1.0
    return c


LEAVES = [
    # T, H, norm, rows a gate, x_scale, y_scale, p
    (1, 8, "none", 0, 1.0, 1.0, 0.0),
    (3, 264, "rms", 3, 1.0, 0.5, 0.1),
    (7, 1024, "layer", 2, 0.75, 1.0, 0.5),
    (5, 1032, "none", 1, 1.0, -1.5, 0.0),
    (33, 4096, "rms", 10, 1.0, 1.0, 0.05),
    (9, 7168, "layer", 100, 1.0, 1.0, 0.0),
    (4, 8200, "rms", 1, 0.0, 1.0, 0.999),
    (3, 16384, "layer", 2, 1.0, 1.0, 0.3),
    (1300, 520, "rms", 97, 1.0, 0.5, 0.1),
    (1000, 2048, "layer", 300, 0.75, 0.5, 0.1),
    (5000, 264, "none", 2, 1.0, 1.0, 0.1),
    (700, 7168, "rms", 650, 1.0, 1.0, 0.1),
    (600, 104, "layer", 7, 1.0, 0.5, 0.1),
    (2600, 256, "layer", 1, 1.0, 0.5, 0.1),
    (900, 480, "layer", 350, 0.75, 1.0, 0.2),
    (3000, 72, "rms", 1000, 1.0, 1.0, 0.0),
    (800, 2992, "layer", 1, 1.0, 1.0, 0.1),
    (500, 6144, "layer", 170, 1.0, 0.5, 0.1),
]


@pytest.mark.parametrize("T,H,kind,gate_rows,xs,ys,p", LEAVES)
@pytest.mark.parametrize("dtype,ydtype", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
def test_leave(T, H, kind, gate_rows, xs, ys, p, dtype, ydtype):
    c = leave_case(torch.Generator().manual_seed(T * 17 + H), T, H, dtype, ydtype, kind, gate_rows, p)
    form = dict(norm=kind, gate=dev(c["gate"]), gate_rows=gate_rows or None, x_scale=xs, y_scale=ys, p=p,
                rng=dev(c["rng"]))
    raw, out = guarded((T, H), DT[dtype])
    bs.branch_leave(dev(c["x"]), dev(c["y"]), dev(c["w"]), dev(c["b"]), out=out, **form)
    x, y, w, b, gate = (wide(c[k]) for k in ("x", "y", "w", "b", "gate"))
    want = ref.leave(x, y, kind, w, b, gate, gate_rows or 1, xs, ys, c["keep"])
    g = ref.gate_of(gate, gate_rows or 1, T)
    g = g if gate is None else g.abs()
    size = abs(ys) * g * c["keep"] * (normed_size(y, kind, w, b) + 2.0 ** -21 * ref.norm(y, kind, w, b).abs())
    near(out, want, size + 2.0 ** -22 * (xs * x).abs(), DT[dtype])
    assert intact(raw)
    # in place, and with the next block's norm of what is stored
    x2 = dev(c["x"])
    for after in ("rms", "layer"):
        if after == "layer":
            x2.copy_(c["x"])
        raw, h = guarded((T, H), DT[ydtype])
        o, h2 = bs.branch_leave(x2, dev(c["y"]), dev(c["w"]), dev(c["b"]), out=x2, next_norm=after,
                                next_weight=dev(c["w"]), next_out=h, **form)
        assert o is x2 and h2 is h and torch.equal(x2, out) and intact(raw)
        near(h, ref.norm(out.double().cpu(), after, w), normed_size(out.double().cpu(), after, w, None),
             DT[ydtype])


@pytest.mark.parametrize("T,H,kind,gate_rows,xs,ys,p", LEAVES)
@pytest.mark.parametrize("dtype,ydtype", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
def test_leave_backward(T, H, kind, gate_rows, xs, ys, p, dtype, ydtype):
    gen = torch.Generator().manual_seed(T * 19 + H)
    c = leave_case(gen, T, H, dtype, ydtype, kind, gate_rows, p)
    dout = torch.randn(T, H, generator=gen).to(DT[dtype])
    raw, dy_out = guarded((T, H), DT[ydtype])
    call = lambda **k: bs.branch_leave_backward(  # noqa: E731
        dev(dout), dev(c["y"]), dev(c["w"]), dev(c["b"]), norm=kind, gate=dev(c["gate"]),
        gate_rows=gate_rows or None, x_scale=xs, y_scale=ys, p=p, rng=dev(c["rng"]), **k)
    dy, dx, dw, db, dgate = call(dy=dy_out)
    torch.cuda.synchronize()
    assert dy is dy_out and intact(raw)
    y, w, b, gate, d = (wide(t) for t in (c["y"], c["w"], c["b"], c["gate"], dout))
    of = ys * d * c["keep"]
    dz = of * ref.gate_of(gate, gate_rows or 1, T)
    want, wantw, wantb, size, sizew, sizeb = ref.norm_grad(dz, y, kind, w)
    near(dy, want, 2.0 ** -16 * size, DT[ydtype])
    near(dx, xs * d, 0.0, DT[dtype])
    assert (dw is None) == (c["w"] is None) and (db is None) == (c["b"] is None)
    if dw is not None:
        near(dw, wantw, 2.0 ** -15 * sizew, torch.float32)
    if db is not None:
        near(db, wantb, 2.0 ** -15 * sizeb, torch.float32)
    if gate is not None:
        at = torch.arange(T) // gate_rows
        z = ref.norm(y, kind, w, b)
        # a term of * z is off by of times what z is off by, normed_size(), where n * w and b cancel
        # too; its products and the sum add 2^-15 of it
        term = of.abs() * (2.0 ** -15 * z.abs() + normed_size(y, kind, w, b))
        near(dgate, torch.zeros_like(gate).index_add_(0, at, of * z),
             torch.zeros_like(gate).index_add_(0, at, term), torch.float32)
    # the same call, the same bits
    again = call()
    for a, e in zip(again, (dy, dx, dw, db, dgate)):
        assert (a is None and e is None) or torch.equal(a, e)


@pytest.mark.parametrize("T,H,gate_rows", [(40, 192, 7), (300, 1040, 1), (300, 4096, 130), (20, 8224, 3)])
def test_a_gates_gradient_alone(T, H, gate_rows):
    """A sum that is not wanted changes no other."""
    c = leave_case(torch.Generator().manual_seed(T + H), T, H, "bf16", "bf16", "layer", gate_rows, 0.1)
    dout, y, w, b, gate, rng = (dev(c[k]) for k in ("x", "y", "w", "b", "gate", "rng"))
    dy, dx, dw, db, dgate = bs.branch_leave_backward(dout, y, w, b, norm="layer", gate=gate, gate_rows=gate_rows,
                                                     x_scale=0.5, y_scale=0.5, p=0.1, rng=rng)
    for keep in ((), (2,), (3,), (4,), (2, 3), (2, 4), (3, 4)):
        raw = [guarded(t.shape, t.dtype) for t in (dy, dx, dw, db, dgate)]
        ptr = lambda t: t.data_ptr()  # noqa: E731
        got = [r[1] if i < 2 or i in keep else None for i, r in enumerate(raw)]
        status = bs.load().branch_leave_backward(
            ptr(dout), 0, ptr(y), 0, T, H, 2, 1e-6, ptr(w), ptr(b), ptr(gate), gate_rows, 0.5, 0.5, 0.1, ptr(rng),
            *(None if t is None else ptr(t) for t in got), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert status == 0
        for t, e, r in zip(got, (dy, dx, dw, db, dgate), raw):
            assert intact(r[0])
            if t is not None:   # (a kernel for fewer sums may round another way)
                near(t, e.double().cpu(), 2.0 ** -14 * e.double().cpu().abs().amax(), t.dtype)


@pytest.mark.parametrize("T,H", SIZES + [(1000, 1024), (900, 4096), (500, 7168), (400, 16384)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype,hdtype", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
def test_enter_backward(T, H, kind, dtype, hdtype):
    g = torch.Generator().manual_seed(T * 23 + H)
    x, w, dh = rows(g, T, H, dtype), columns(g, H, T != 3), torch.randn(T, H, generator=g).to(DT[hdtype])
    dres = rows(g, T, H, dtype) if T % 2 else None
    raw, dx = guarded((T, H), DT[dtype])
    _, dw, db = bs.branch_enter_backward(dev(dh), dev(x), dev(w), norm=kind, dres=dev(dres),
                                         bias=kind == "layer", dx=dx)
    torch.cuda.synchronize()
    assert intact(raw) and (dw is None) == (w is None) and (db is None) == (kind != "layer")
    want, wantw, wantb, size, sizew, sizeb = ref.norm_grad(dh.double(), x.double(), kind, wide(w))
    if dres is not None:
        want, size = want + dres.double(), size + dres.double().abs()
    near(dx, want, 2.0 ** -16 * size, DT[dtype])
    if dw is not None:
        near(dw, wantw, 2.0 ** -15 * sizew, torch.float32)
    if db is not None:
        near(db, wantb, 2.0 ** -15 * sizeb, torch.float32)


def test_gradients_are_differences():
    """The gradients against central differences of the operators themselves (FP32)."""
    g = torch.Generator().manual_seed(3)
    T, H = 6, 40
    c = {k: torch.randn(s, generator=g).cuda() for k, s in
         {"x": (T, H), "y": (T, H), "weight": (H,), "bias": (H,), "gate": (2, H)}.items()}
    rng = torch.tensor([9, 9]).cuda()
    form = dict(norm="layer", gate_rows=4, x_scale=0.75, y_scale=0.5, p=0.25, rng=rng)
    dout = torch.randn(T, H, generator=g).cuda()
    names = ("y", "x", "weight", "bias", "gate")
    grads = dict(zip(names, bs.branch_leave_backward(dout, c["y"], c["weight"], c["bias"], gate=c["gate"], **form)))
    for name in names:
        u = torch.randn(c[name].shape, generator=g).cuda()
        step = 1e-2
        loss = [(bs.branch_leave(**{**c, name: c[name] + s * u}, **form) * dout).double().sum()
                for s in (step, -step)]
        want = (grads[name].double() * u).sum()
        # 240 terms of size about 3 rounded at 2^-24 over the step: below 2e-3; the third
        # derivatives of a norm of 40 values along a direction of size 1 a value stay below 20 a
        # term, of random signs: 16 terms' worth of 20 * step^2 / 6
        assert abs(float((loss[0] - loss[1]) / (2 * step) - want)) < 8e-3


@pytest.mark.parametrize("n", [1, 7, 8, 9, 2047, 8192, 8195, 100003])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9999999])
def test_dropout(n, dtype, p):
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, generator=g).to(DT[dtype])
    seed, offset = -12345678901234, (1 << 33) + n
    rng = torch.tensor([seed, offset]).cuda()
    raw, out = guarded((n,), DT[dtype])
    bs.dropout(dev(x), p, rng, out=out)
    torch.cuda.synchronize()
    m = ref.mask(n, p, seed, offset) if p else torch.ones(n, dtype=torch.float64)
    near(out, x.double() * m, 2.0 ** -22 * (x.double() * m).abs(), DT[dtype])
    assert intact(raw) and torch.equal((out == 0).cpu() | (x == 0), (m == 0) | (x == 0))
    again = dev(x)
    assert torch.equal(bs.dropout(again, p, rng, out=again), out)      # in place


def test_dropout_is_the_branchs():
    """branch_leave drops what dropout drops for the same numbers, on a long tensor too."""
    T, H = 3000, 1024
    y = torch.ones(T, H, device="cuda")
    rng = torch.tensor([5, 6]).cuda()
    got = bs.branch_leave(torch.zeros_like(y), y, p=0.3, rng=rng)
    assert torch.equal(got, bs.dropout(y, 0.3, rng))
    dy = bs.branch_leave_backward(y, y, p=0.3, rng=rng)[0]
    assert torch.equal(dy, got)
    drop = ref.threshold(0.3) / 65536
    share = float((got == 0).double().mean())
    assert abs(share - drop) < 5 * (drop * (1 - drop) / (T * H)) ** 0.5


def test_rows_past_32_bits_of_values():
    """The last rows of more than 2^31 values give what they give by themselves."""
    T, H, n = 270000, 8192, 5
    g = torch.Generator(device="cuda").manual_seed(9)
    x, y = (torch.empty(T, H, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    x.normal_(generator=g), y.normal_(generator=g)
    w = torch.randn(H, generator=g, device="cuda")
    gate = torch.randn(2, H, generator=g, device="cuda").bfloat16()
    rows_ = T - 1000    # of the first gate
    form = dict(norm="layer", x_scale=0.75, y_scale=0.5)
    codes, scales = bs.branch_enter(x, w, fmt="e4m3")
    want = bs.branch_enter(x[-n:].contiguous(), w, fmt="e4m3")
    assert torch.equal(codes[-n:], want[0]) and torch.equal(scales[-n:], want[1])
    out, h = bs.branch_leave(x, y, w, w, gate=gate, gate_rows=rows_, next_norm="rms", next_weight=w, **form)
    want = bs.branch_leave(x[-n:].contiguous(), y[-n:].contiguous(), w, w, gate=gate[1:], gate_rows=n, next_norm="rms",
                           next_weight=w, **form)
    assert torch.equal(out[-n:], want[0]) and torch.equal(h[-n:], want[1])
    dy, dx, dw, db, dgate = bs.branch_leave_backward(x, y, w, w, gate=gate, gate_rows=rows_, **form)
    want = bs.branch_leave_backward(x[-n:].contiguous(), y[-n:].contiguous(), w, w, gate=gate[1:], gate_rows=n, **form)
    assert torch.equal(dy[-n:], want[0]) and torch.equal(dx[-n:], want[1])
    # the second gate's rows by themselves: other runs of rows, so only as near as the sums are
    part = bs.branch_leave_backward(x[rows_:].contiguous(), y[rows_:].contiguous(), w, w, gate=gate[1:], gate_rows=T,
                                    **form)[4]
    near(dgate[1:], part.cpu(), 2.0 ** -14 * 1000 ** 0.5 * part.cpu().abs().amax(), torch.float32)
    del codes, scales, h, dy, dx
    rng = torch.tensor([3, 5], device="cuda")
    kept = bs.branch_leave(x, y, p=0.25, rng=rng, x_scale=0.0)
    assert torch.equal(kept.view(-1)[-n * H:], bs.dropout(y, 0.25, rng).view(-1)[-n * H:])
    assert abs((kept[-n:] == 0).float().mean().item() - 0.25) < 0.02
    # another row has another mask
    assert not torch.equal(kept[-1] == 0, kept[T - 1 - (1 << 32) // H // 2] == 0)


def test_special_values_stay_in_their_rows():
    """Infinities and NaN: a dropped one is 0, a kept one is the row's own matter."""
    T, H = 6, 1024
    g = torch.Generator().manual_seed(8)
    x, y = torch.randn(T, H, generator=g).cuda(), torch.randn(T, H, generator=g).cuda()
    rng = torch.tensor([1, 1]).cuda()
    clean = bs.branch_leave(x, y, norm="rms", p=0.5, rng=rng, next_norm="layer")
    keep = (ref.mask(T * H, 0.5, 1, 1) > 0).view(T, H)
    bad = y.clone()
    bad[2, 3], bad[4, 5] = float("nan"), float("inf")
    out, h = bs.branch_leave(x, bad, norm="rms", p=0.5, rng=rng, next_norm="layer")
    for t in (0, 1, 3, 5):
        assert torch.equal(out[t], clean[0][t]) and torch.equal(h[t], clean[1][t])
    assert torch.equal(out[2].cpu().isnan(), keep[2])
    plain = bs.branch_leave(x, bad, p=0.5, rng=rng)
    assert torch.equal(plain.isfinite().cpu(), bad.isfinite().cpu() | ~keep)
    z = bs.branch_enter(torch.zeros(2, H, device="cuda"), norm="layer")
    assert torch.equal(z, torch.zeros_like(z))
    far = 1000 + torch.randn(3, H, generator=g, dtype=torch.float64)     # a mean far from zero
    near(bs.branch_enter(far.float().cuda(), norm="layer"), ref.norm(far.float().double(), "layer"),
         normed_size(far.float().double(), "layer", None, None), torch.float32)


def test_empty():
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.empty(0, 64, dtype=dtype, device="cuda")
        w = torch.ones(64, device="cuda")
        assert bs.branch_enter(x, w).shape == (0, 64)
        assert bs.branch_leave(x, x, w, norm="rms").shape == (0, 64)
        _, dw, db = bs.branch_enter_backward(x, x, w, bias=True)
        assert not dw.any() and not db.any()
        dy, dx, dw, db, dg = bs.branch_leave_backward(x, x, w, w, norm="rms", gate=x, gate_rows=4)
        assert not dw.any() and not db.any() and dg.shape == (0, 64)
        assert bs.dropout(x, 0.5, torch.zeros(2, dtype=torch.int64, device="cuda")).shape == (0, 64)


def test_captured_and_on_other_streams():
    """A captured training step replayed with new numbers and inputs, eager calls between the
    replays; the same calls on two other streams at once."""
    T, H = 300, 2048
    g = torch.Generator().manual_seed(4)
    x, y, dout = (torch.randn(T, H, generator=g).bfloat16().cuda() for _ in range(3))
    w, rng = torch.randn(H, generator=g).cuda(), torch.tensor([3, 0]).cuda()
    gate = torch.randn(4, H, generator=g).bfloat16().cuda()

    def step(x, y, dout):
        h = bs.branch_enter(x, w, norm="rms")
        out, h2 = bs.branch_leave(x, y, w, norm="layer", gate=gate, gate_rows=90, p=0.2, rng=rng, next_norm="rms")
        d, dw2, _ = bs.branch_enter_backward(dout, out, w, dres=dout)
        return (h, out, h2, dw2) + bs.branch_leave_backward(d, y, w, norm="layer", gate=gate, gate_rows=90,
                                                            p=0.2, rng=rng)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bs.reserve_workspace(bs.branch_backward_workspace_bytes(T, H))
        bs.device_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        rng[1] += 1
        got = step(x, y, dout)
    seen = []
    for i in range(3):
        x.copy_(torch.randn(T, H, generator=g).bfloat16())
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.default_stream())
            graph.replay()
        s.synchronize()
        replayed = [t.clone() for t in got if t is not None]
        assert int(rng[1]) == i + 1
        for a, b in zip(replayed, (t for t in step(x, y, dout) if t is not None)):
            assert torch.equal(a, b)
        seen.append(replayed[1])
    assert not torch.equal(seen[0], seen[1])

    want = [t for t in step(x, y, dout) if t is not None]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    results = []
    for _ in range(4):
        for q in streams:
            with torch.cuda.stream(q):
                results.append([t for t in step(x, y, dout) if t is not None])
    torch.cuda.synchronize()
    for r in results:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_capture_without_a_workspace_is_refused():
    T, H = 64, 16384
    x = torch.randn(T, H).bfloat16().cuda()
    w = torch.ones(H).cuda()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(bs.BsmmaError) as e:
        with torch.cuda.graph(graph, stream=s):
            bs.branch_enter_backward(x, x, w)
    assert e.value.code == bs.STATUS.index("BSMMA_ERR_WORKSPACE")
