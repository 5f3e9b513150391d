"""Gradients of branch_leave where the gate is another one for each row, or has no gradient, and of
many rows a worker, against their definitions in 64 bits; tolerances as in test_gpu_branch.py.
"""
import pytest
import torch

import block_scaled_precision_mma_gb300 as bs
from tests import branch_ref as ref
from tests.test_gpu_branch import DT, dev, guarded, intact, leave_case, near, normed_size, wide

pytestmark = pytest.mark.gpu
TYPES = [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bs.build()
    bs.load()
    torch.cuda.init()


def wanted(c, dout, kind, rows, ys, p_keep):
    """(value, size of its error) of dy, dweight, dbias and dgate."""
    y, w, b, gate, d = (wide(t) for t in (c["y"], c["w"], c["b"], c["gate"], dout))
    T = len(y)
    of = ys * d * p_keep
    dz = of * ref.gate_of(gate, rows, T)
    dy, dw, db, size, sizew, sizeb = ref.norm_grad(dz, y, kind, w)
    at = torch.arange(T, device=y.device) // rows
    z = ref.norm(y, kind, w, b)
    term = of.abs() * (2.0 ** -15 * z.abs() + normed_size(y, kind, w, b))
    sums = [torch.zeros_like(gate).index_add_(0, at, t) for t in (of * z, term)]
    return {"dy": (dy, 2.0 ** -16 * size), "dw": (dw, None if dw is None else 2.0 ** -15 * sizew),
            "db": (db, None if db is None else 2.0 ** -15 * sizeb), "dgate": tuple(sums)}


@pytest.mark.parametrize("T,H", [(300, 8), (300, 256), (70, 264), (300, 512), (70, 520), (300, 1024), (40, 1032),
                                 (170, 7168), (20, 8192), (9, 8200)])
@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
@pytest.mark.parametrize("dtype,ydtype", TYPES)
def test_a_gate_for_each_row_without_a_bias(T, H, kind, dtype, ydtype):
    g = torch.Generator().manual_seed(T * 29 + H)
    c = leave_case(g, T, H, dtype, ydtype, kind, 1, 0.1)
    c["b"] = None
    dout = torch.randn(T, H, generator=g).to(DT[dtype])
    raw, dy_out = guarded((T, H), DT[ydtype])
    dy, _, dw, db, dgate = bs.branch_leave_backward(
        dev(dout), dev(c["y"]), dev(c["w"]), norm=kind, gate=dev(c["gate"]), gate_rows=1, y_scale=0.5, p=0.1,
        rng=dev(c["rng"]), dy=dy_out)
    torch.cuda.synchronize()
    assert intact(raw) and db is None
    want = wanted(c, dout, kind, 1, 0.5, c["keep"])
    near(dy, *want["dy"], DT[ydtype])
    near(dgate, *want["dgate"], torch.float32)
    if dw is not None:
        near(dw, *want["dw"], torch.float32)


@pytest.mark.parametrize("T,H,rows", [(60, 248, 7), (60, 512, 1), (60, 1000, 60), (200, 2048, 9), (200, 7168, 1),
                                      (200, 4096, 130), (9, 8224, 4)])
@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
@pytest.mark.parametrize("dtype,ydtype", TYPES)
def test_each_gradient_left_out(T, H, rows, kind, dtype, ydtype):
    """A sum that is not wanted changes no other, whatever the types; a gate without a gradient."""
    g = torch.Generator().manual_seed(T * 31 + H + rows)
    c = leave_case(g, T, H, dtype, ydtype, kind, rows, 0.1)
    c["w"] = None if kind == "none" else torch.randn(H, generator=g)
    dout = torch.randn(T, H, generator=g).to(DT[dtype])
    want = wanted(c, dout, kind, rows, 0.5, c["keep"])
    d = {k: dev(c[k]) for k in ("y", "w", "b", "gate", "rng")}
    dout = dev(dout)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    normed = () if kind == "none" else ("dw", "db")
    shape = {"dw": (H,), "db": (H,), "dgate": tuple(c["gate"].shape)}
    for names in ((), ("dgate",), normed, normed[:1], normed[1:], normed[:1] + ("dgate",), normed[1:] + ("dgate",)):
        raw = {"dy": guarded((T, H), DT[ydtype])}
        for n in names:
            raw[n] = guarded(shape[n], torch.float32)
        at = lambda n: ptr(raw[n][1]) if n in raw else None  # noqa: E731
        status = bs.load().branch_leave_backward(
            ptr(dout), bs.DTYPES[dout.dtype], ptr(d["y"]), bs.DTYPES[d["y"].dtype], T, H, bs.NORMS[kind], 1e-6,
            ptr(d["w"]), ptr(d["b"]), ptr(d["gate"]), rows, 1.0, 0.5, 0.1, ptr(d["rng"]), at("dy"), None, at("dw"),
            at("db"), at("dgate"), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert status == 0
        for n, (buffer, got) in raw.items():
            assert intact(buffer)
            near(got, *want[n], got.dtype)


@pytest.mark.parametrize("T,H,rows", [(30400, 1536, 7), (30400, 1536, 64), (30400, 4096, 7), (30400, 7168, 64),
                                      (30400, 7168, 3000), (60000, 264, 3), (121600, 1000, 13), (6000, 8200, 7)])
@pytest.mark.parametrize("kind,bias", [("rms", False), ("layer", True)])
@pytest.mark.parametrize("dtype,ydtype", TYPES)
def test_many_rows_and_gates_a_worker(T, H, rows, kind, bias, dtype, ydtype):
    """A worker (at least 152 of them, at most 16 an SM) adds R <= T / 152 + 1 rows in a run, over several gates, and
    a thread of the second launch at most 304 runs, eight threads a column: a sum's own error is below
    (R + 312) 2^-24 of its terms' sizes, and a term's 2^-18, as a normed value's (3 products: 2^-22)."""
    g = torch.Generator(device="cuda").manual_seed(T + H + rows)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    y = (rnd(T, H) * torch.exp(0.5 * rnd(H)) + 0.3 * rnd(H)).to(DT[ydtype])
    w, b, gate = rnd(H), rnd(H) if bias else None, rnd(-(-T // rows), H).to(DT[ydtype])
    dout = rnd(T, H).to(DT[dtype])
    _, _, dw, db, dgate = bs.branch_leave_backward(dout, y, w, b, norm=kind, gate=gate, gate_rows=rows, y_scale=0.5)
    v, at = y.double(), torch.arange(T, device="cuda") // rows
    mean, r = ref.stats(v, kind, 1e-6)
    n, size = (v - mean) * r, (v.abs() + v.abs().mean(1, keepdim=True)) * r
    of = 0.5 * dout.double()
    dz = of * gate.double()[at]
    run = lambda rows: (rows + 312) * 2.0 ** -24 + 2.0 ** -18 + 2.0 ** -22  # noqa: E731

    def close(got, want, tol):
        bad = ~((got.double() - want).abs() <= tol + 2.0 ** -24 * want.abs())
        assert not bad.any(), (int(bad.sum()), got[bad][:3], want[bad][:3], tol[bad][:3])

    most = T // 152 + 1
    close(dw, (dz * n).sum(0), run(most) * (dz.abs() * size).sum(0))
    if bias:
        close(db, dz.sum(0), run(most) * dz.abs().sum(0))
    z, zsize = n * w, size * w.abs()
    if bias:
        z, zsize = z + b, zsize + b.abs()
    sums = [torch.zeros_like(gate, dtype=torch.float64).index_add_(0, at, t) for t in (of * z, of.abs() * zsize)]
    close(dgate, sums[0], run(rows) * sums[1])
