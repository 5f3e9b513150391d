"""NaN and infinities in the residual branch's rows: what is dropped adds nothing to a gradient, what is
kept stays with its row and its sums."""
import pytest
import torch

import block_scaled_precision_mma_gb300 as bs
from tests import branch_ref as ref
from tests.test_gpu_branch import DT, dev, leave_case

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bs.build()
    bs.load()
    torch.cuda.init()


@pytest.mark.parametrize("T,H,rows", [(40, 264, 7), (40, 264, 1), (30, 1000, 30), (33, 1032, 8), (33, 1032, 1),
                                      (9, 8200, 4), (9, 8200, 1)])
@pytest.mark.parametrize("kind,bias", [("none", False), ("rms", False), ("layer", True), ("layer", False)])
@pytest.mark.parametrize("dtype,ydtype", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
def test_dropped_values_add_nothing_to_a_gradient(T, H, rows, kind, bias, dtype, ydtype):
    g = torch.Generator().manual_seed(T * 37 + H + rows)
    c = leave_case(g, T, H, dtype, ydtype, kind, rows, 0.5)
    c["w"] = None if kind == "none" else torch.randn(H, generator=g)
    c["b"] = torch.randn(H, generator=g) if bias else None
    kept = c["keep"] > 0
    dout = (torch.randn(T, H, generator=g) + 3).to(DT[dtype])
    call = lambda y: bs.branch_leave_backward(  # noqa: E731
        dev(dout), dev(y), dev(c["w"]), dev(c["b"]), norm=kind, gate=dev(c["gate"]), gate_rows=rows, y_scale=0.5, p=0.5,
        rng=dev(c["rng"]))
    clean = call(c["y"])
    assert all(t is None or t.isfinite().all() for t in clean)
    bad, rows_of = c["y"].clone(), {}
    for t, value in ((2, NAN), (5, INF), (8, -INF)):   # at dropped places, and in row 5 at a kept one too
        at = (~kept[t]).nonzero()[:: H // 40 or 1, 0]
        bad[t, at] = value
        rows_of[t] = kept[t]
    one = kept[5].nonzero()[3, 0]
    bad[5, one] = INF
    if kind == "none":
        rows_of = {5: torch.arange(H) == one}
    dy, dx, dw, db, dgate = call(bad)
    # the columns that a bad row keeps are NaN in its gate's sums (or the infinity's), the others are as they were
    touched = torch.zeros(c["gate"].shape, dtype=torch.bool)
    for t, columns in rows_of.items():
        touched[t // rows] |= columns
    touched = touched.cuda()
    assert not dgate[touched].isfinite().any() if kind in ("none", "layer") else not dgate[touched].isfinite().all()
    assert torch.equal(dgate[~touched], clean[4][~touched])
    if kind == "none":
        assert torch.equal(dy, clean[0])
        return
    others = [t for t in range(T) if t not in rows_of]
    assert torch.equal(dy[others], clean[0][others]) and dy[list(rows_of)].isnan().all()
    columns = torch.zeros(H, dtype=torch.bool)
    for kept_ in rows_of.values():
        columns |= kept_
    columns = columns.cuda()
    assert torch.equal(dw[~columns], clean[2][~columns]) and not dw[columns].isfinite().all()
    if bias:
        assert torch.equal(db, clean[3])


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("p", [0.0, 0.5])
def test_a_kept_nan_without_a_gradient(rows, p):
    """dgate is the sum of dout * z: 0 * NaN is NaN for a kept z, with or without dropout and norm."""
    T, H = 6, 64
    g = torch.Generator().manual_seed(rows)
    c = leave_case(g, T, H, "f32", "f32", "none", rows, p)
    kept = c["keep"] > 0 if p else torch.ones(T, H, dtype=torch.bool)
    dout = torch.randn(T, H, generator=g)
    y, at = c["y"].clone(), kept[4].nonzero()[2, 0]
    y[4, at], dout[4, at] = NAN, 0
    for kind in ("none", "rms"):
        dgate = bs.branch_leave_backward(dev(dout), dev(y), norm=kind, gate=dev(c["gate"]), gate_rows=rows, p=p,
                                         rng=dev(c["rng"]))[4]
        assert dgate[4 // rows, at].isnan()


@pytest.mark.parametrize("T,H", [(7, 200), (7, 512), (7, 1024), (5, 4096), (5, 16384)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [INF, -INF, 1e30])
def test_an_infinite_sum_of_squares(T, H, dtype, value):
    """RMS: the factor is 0, a finite value becomes 0 (the bias), an infinity NaN; other rows keep theirs."""
    g = torch.Generator().manual_seed(H)
    x, w, b = (torch.randn(s, generator=g) for s in ((T, H), (H,), (H,)))
    x = dev(x.to(DT[dtype]))
    w, b = dev(w), dev(b)
    bad = x.clone()
    bad[3, H // 2] = value
    finite = bad[3].isfinite()
    out = bs.branch_enter(bad, w, b)
    clean = bs.branch_enter(x, w, b)
    rows = [t for t in range(T) if t != 3]
    assert torch.equal(out[rows], clean[rows])
    assert torch.equal(out[3, finite], b.to(DT[dtype])[finite]) and out[3, ~finite].isnan().all()
    left, h = bs.branch_leave(x, bad, w, b, norm="rms", next_norm="rms", next_weight=w)
    assert torch.equal(left[3, finite], (x[3].float() + b).to(DT[dtype])[finite]) and left[3, ~finite].isnan().all()
    assert h[rows].isfinite().all() and h[3].isfinite().all() == bool(finite.all())
    # with the row's n of 0 nothing is added to its gradient or to the weight's
    dh = torch.randn(T, H, generator=g).to(DT[dtype]).cuda()
    dx, dw, _ = bs.branch_enter_backward(dh, bad, w, dres=x)
    want = bs.branch_enter_backward(dh, x, w, dres=x)
    assert torch.equal(dx[rows], want[0][rows])
    if finite.all():
        assert torch.equal(dx[3], x[3]) and dw.isfinite().all()
    else:
        assert dx[3].isnan().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_an_empty_batch_with_the_gate_of_all_rows(dtype):
    x, gate, w = torch.empty(0, 64, dtype=DT[dtype]).cuda(), torch.ones(1, 64, dtype=DT[dtype]).cuda(), torch.ones(64).cuda()
    out, h = bs.branch_leave(x, x, w, norm="rms", gate=gate, next_norm="rms")
    assert out.shape == h.shape == (0, 64)
    _, _, dw, _, dgate = bs.branch_leave_backward(x, x, w, norm="rms", gate=gate)
    assert dgate.shape == (1, 64) and not dgate.any() and not dw.any()
