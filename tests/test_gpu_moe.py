"""Routing, the expert order and the weighted sum on the GPU against their definitions in
64 bits.  Choices and orders are whole numbers and must be equal; inputs whose choice would
hang on the rounding of a sum (keys closer than 1e-6) are drawn again."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import block_scaled_precision_mma_gb300 as bs
from tests import expert_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bs.build()
    bs.load()
    torch.cuda.init()


def logits(g, T, E, dtype, closed=0.0):
    x = torch.from_numpy(g.standard_normal((T, E)).astype(np.float32) * 2)
    x[torch.from_numpy(g.random((T, E)) < closed)] = -np.inf
    return x.to(DT[dtype])


def separated(g, T, E, dtype, closed, k, score, bias, groups, topk_groups, group_top):
    x = logits(g, T, E, dtype, closed)
    for _ in range(50):
        key, value = ref.keys(x.double().numpy(), score, bias, groups, topk_groups, group_top)
        close = np.zeros(T, dtype=bool)
        for v in (key, value):
            if v is not None:
                v = -np.sort(-v, axis=1)[:, :max(k, groups) + 1]
                with np.errstate(invalid="ignore"):
                    gap = v[:, :-1] - v[:, 1:]
                close |= ((gap > 0) & (gap < 1e-6)).any(1)
        if not close.any():
            return x
        x[torch.from_numpy(close)] = logits(g, int(close.sum()), E, dtype, closed)
    raise AssertionError("no separated logits found")


# FP32 scores: |x - max| <= 20 rounds to 20 * 2^-24 at most, the exponential and the sums add
# a few ulp, the quotient one: below 2^-18 of the weight.
W_TOL = 2.0 ** -18

ROUTES = [
    # T, E, k, score, bias, groups, topk_groups, group_top, renormalize, scale, dtype, closed
    (1, 1, 1, "softmax", False, 1, 1, 1, True, 1.0, "f32", 0.0),
    (3, 7, 7, "softmax", False, 1, 1, 1, False, 1.0, "bf16", 0.0),
    (33, 8, 2, "softmax", False, 1, 1, 1, True, 1.0, "bf16", 0.3),
    (1025, 64, 6, "softmax", False, 8, 3, 1, False, 16.0, "f32", 0.0),
    (70, 60, 8, "softmax", True, 5, 2, 2, True, 1.0, "f32", 0.2),
    (40, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, "f32", 0.0),
    (40, 256, 8, "sigmoid", False, 8, 4, 2, True, 2.5, "bf16", 0.1),
    (9, 1024, 32, "sigmoid", True, 1, 1, 1, False, 1.0, "f32", 0.0),
    (9, 1023, 5, "softmax", True, 1, 1, 1, True, 1.0, "bf16", 0.0),
    (17, 96, 3, "sigmoid", False, 32, 1, 1, True, 1.0, "f32", 0.5),
    (12, 32, 4, "softmax", False, 32, 31, 2, True, 1.0, "f32", 0.0),
    (5, 300, 16, "softmax", False, 3, 3, 2, True, 1.0, "f32", 0.95),
    (1100, 30, 16, "softmax", True, 1, 1, 1, False, 1.0, "f32", 0.6),
    (6, 32, 16, "sigmoid", True, 4, 2, 2, True, 2.0, "bf16", 0.5),
    (8217, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, "f32", 0.0),
    (8223, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, "bf16", 0.5),
    (8222, 64, 6, "softmax", True, 4, 2, 2, False, 1.0, "f32", 0.2),
    (8216, 128, 8, "softmax", False, 1, 1, 1, True, 1.0, "f32", 0.3),
    (8216, 384, 7, "softmax", False, 1, 1, 1, False, 1.0, "f32", 0.0),
    (8218, 48, 5, "sigmoid", False, 2, 1, 2, True, 1.0, "bf16", 0.9),
    (8219, 1024, 8, "softmax", True, 1, 1, 1, True, 1.0, "f32", 0.0),
    (8221, 24, 3, "softmax", False, 1, 1, 1, False, 3.0, "f32", 0.95),
    (8225, 320, 4, "softmax", False, 8, 3, 1, False, 1.0, "bf16", 0.2),
    (8216, 8, 8, "softmax", False, 1, 1, 1, True, 1.0, "f32", 0.5),
    (8192, 64, 1, "softmax", False, 8, 1, 2, True, 1.0, "f32", 0.9),
]


@pytest.mark.parametrize("T,E,k,score,bias,groups,topk_groups,group_top,renorm,scale,dtype,closed", ROUTES)
def test_route(T, E, k, score, bias, groups, topk_groups, group_top, renorm, scale, dtype, closed):
    g = np.random.default_rng([71, T, E, k, groups])
    b = (g.integers(-60, 61, E) * np.float32(0.001)).astype(np.float32) if bias else None
    x = separated(g, T, E, dtype, closed, k, score, b, groups, topk_groups, group_top)
    ids, w = bs.moe_route(x.cuda(), k, score=score, bias=None if b is None else torch.from_numpy(b).cuda(),
                          groups=groups, topk_groups=topk_groups, group_top=group_top,
                          renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    ids_ref, w_ref = ref.route(x.double().numpy(), k, score, b, groups, topk_groups, group_top, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    assert np.all(np.abs(w.cpu().numpy() - w_ref) <= W_TOL * np.abs(w_ref) + 1e-37)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_take_the_lower_index(score):
    x = torch.zeros(4, 70)
    x[1, 40:] = 1
    x[2, ::3] = -0.0
    x[3, 69] = x[3, 5] = 3
    ids, _ = bs.moe_route(x.cuda(), 4, score=score)
    assert ids.tolist() == [[0, 1, 2, 3], [40, 41, 42, 43], [0, 1, 2, 3], [5, 69, 0, 1]]
    # tied groups too: each of the 7 groups has the same value
    ids, _ = bs.moe_route(x[:1].contiguous().cuda(), 4, score=score, groups=7, topk_groups=2,
                          group_top=2, bias=torch.zeros(70, device="cuda"))
    assert ids.tolist() == [[0, 1, 2, 3]]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masks_and_specials(score, bias):
    """Rows without an open expert, NaN, infinities, the type's lowest value."""
    low = float(np.finfo(np.float32).min)
    x = np.full((7, 33), -np.inf, dtype=np.float32)
    x[1, 32] = 0.5                      # one open expert, k = 3
    x[2] = np.nan
    x[2, 4] = 1
    x[3] = low                          # masked by the lowest value: still experts
    x[4, [3, 9]] = np.inf
    x[4, 1] = 2
    x[5] = low
    x[5, 20] = 1.5
    x[6] = np.linspace(-300, 300, 33)
    b = np.zeros(33, dtype=np.float32)
    b[1] = np.nan if bias else 0
    ids, w = bs.moe_route(torch.from_numpy(x).cuda(), 3, score=score,
                          bias=torch.from_numpy(b).cuda() if bias else None)
    torch.cuda.synchronize()
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    assert ids[0].tolist() == [-1, -1, -1] and w[0].tolist() == [0, 0, 0]
    assert ids[1].tolist() == [32, -1, -1] and w[1].tolist() == [1, 0, 0]
    assert ids[2].tolist() == [4, -1, -1] and w[2].tolist() == [1, 0, 0]
    assert ids[3].tolist() == ([0, 2, 3] if bias else [0, 1, 2])
    assert ids[4].tolist() == ([3, 9, -1] if bias else [3, 9, 1])
    # with a bias the keys are FP32 scores: 1 / (1 + e^-18.75) and all above round to 1, a tie
    assert ids[6][0] == (17 if bias and score == "sigmoid" else 32) and np.all(np.isfinite(w))
    if score == "softmax":
        assert np.allclose(w[3], 1 / 3) and np.allclose(w[4], [0.5, 0.5, 0]) and w[5].tolist() == [1, 0, 0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("groups,topk_groups,group_top", [(1, 1, 1), (4, 2, 1), (8, 3, 2)])
@pytest.mark.parametrize("score,bias,E,k", [("softmax", False, 64, 8), ("sigmoid", False, 192, 5),
                                            ("sigmoid", True, 128, 8), ("sigmoid", True, 1024, 3)])
def test_route_many_tokens_ties(score, bias, E, k, groups, topk_groups, group_top, dtype):
    """Few distinct values, so ties in almost every token, of experts and of groups; zeros of
    both signs, NaN, infinities, closed rows and groups; a NaN in the bias closes its expert."""
    T = 8209
    g = np.random.default_rng([79, E, k, groups])
    x = np.round(g.standard_normal((T, E)) * 4) / 2
    pick = g.random((T, E))
    for i, v in enumerate((np.nan, -np.inf, np.inf, -0.0)):
        x[(pick >= i * 0.02) & (pick < i * 0.02 + 0.02)] = v
    x[5] = -np.inf
    x[6] = np.nan
    x[7] = -0.0
    x[8, 1:] = -np.inf
    x[9:60, E // 8:] = -np.inf
    xt = torch.from_numpy(x).to(DT[dtype])
    x64 = xt.double().numpy()
    b = None
    if bias:
        b = (g.integers(0, 3, E) * 0.25).astype(np.float32)
        b[3] = np.nan
        x64[:, 3] = -np.inf
    ids, w = bs.moe_route(xt.cuda(), k, score=score, bias=None if b is None else torch.from_numpy(b).cuda(),
                          groups=groups, topk_groups=topk_groups, group_top=group_top)
    torch.cuda.synchronize()
    ids_ref, w_ref = ref.route(x64, k, score, None if b is None else np.nan_to_num(b), groups, topk_groups,
                               group_top)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    assert np.all(np.abs(w.cpu().numpy() - w_ref) <= W_TOL * np.abs(w_ref) + 1e-37)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(32, 8), (128, 1), (160, 5), (1024, 8), (64, 12), (65, 8), (2, 2), (1023, 3)])
def test_route_bf16_many_tokens(E, k, score, renorm):
    """BF16 logits over enough tokens for every kernel: few distinct values (ties in almost
    every token), zeros of both signs, NaN, infinities, the lowest value, closed experts."""
    T = 1037
    g = np.random.default_rng([78, E, k])
    x = np.round(g.standard_normal((T, E)) * 4) / 2
    pick = g.random((T, E))
    for i, v in enumerate((np.nan, -np.inf, np.inf, -0.0, float(torch.finfo(torch.bfloat16).min))):
        x[(pick >= i * 0.02) & (pick < i * 0.02 + 0.02)] = v
    x[5] = -np.inf
    x[6] = np.nan
    x[7] = -0.0
    x[8, 1:] = -np.inf
    xt = torch.from_numpy(x).bfloat16()
    ids, w = bs.moe_route(xt.cuda(), k, score=score, renormalize=renorm, scale=0.5)
    torch.cuda.synchronize()
    x64 = xt.double().numpy()
    ids_ref, w_ref = ref.route(x64, k, score, renormalize=renorm, scale=0.5)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    assert np.all(np.abs(w.cpu().numpy() - w_ref) <= W_TOL * np.abs(w_ref) + 1e-37)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,dtype", [(1, 1, 1, "f32"), (1101, 33, 3, "f32"), (1029, 1024, 7, "bf16"), (6, 33, 4, "f32"), (1030, 64, 8, "bf16"),
                                         (3, 1024, 32, "f32"), (5, 20, 20, "bf16")])
def test_route_backward(T, E, k, dtype, score, renorm):
    g = np.random.default_rng([72, T, E, k])
    x = logits(g, T, E, dtype, 0.1)
    if T > 2:
        x[1] = -np.inf
    ids, _ = bs.moe_route(x.cuda(), k, score=score, renormalize=renorm, scale=2.5)
    dw = torch.from_numpy(g.standard_normal((T, k)).astype(np.float32))
    dx = bs.moe_route_backward(x.cuda(), ids, dw.cuda(), score=score, renormalize=renorm, scale=2.5)
    torch.cuda.synchronize()
    assert dx.dtype == x.dtype
    want = ref.route_backward(x.double().numpy(), ids.cpu().numpy(), dw.numpy(), score, renorm, 2.5)
    # each element is a difference of terms no larger than scale * sum |dw| and is rounded to
    # its type once: FP32 steps of those terms, and half a BF16 step
    terms = 2.5 * np.abs(dw.numpy()).sum(1, keepdims=True)
    tol = 2.0 ** -18 * terms + (2.0 ** -8 if dtype == "bf16" else 0) * np.abs(want)
    assert np.all(np.abs(dx.double().cpu().numpy() - want) <= tol)


def test_route_backward_ignores_foreign_ids():
    x = torch.randn(2, 16, generator=torch.Generator().manual_seed(1)).cuda()
    ids = torch.tensor([[3, 16, -1], [1 << 20, -7, 5]], dtype=torch.int32).cuda()
    dw = torch.ones(2, 3).cuda()
    dx = bs.moe_route_backward(x, ids, dw, score="sigmoid", renormalize=False).cpu().numpy()
    s = 1 / (1 + np.exp(-x.double().cpu().numpy()))
    want = np.zeros((2, 16))
    want[0, 3], want[1, 5] = (s * (1 - s))[0, 3], (s * (1 - s))[1, 5]
    assert np.allclose(dx, want, atol=1e-6)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (5, 3, 2), (31, 1, 1024), (256, 8, 256), (512, 8, 256), (2049, 1, 7),
                                   (2050, 2, 1024), (10001, 5, 60),
                                   (300001, 4, 3)])
@pytest.mark.parametrize("unused", [0.0, 0.3, 1.0])
def test_plan(T, k, E, unused):
    g = np.random.default_rng([73, T, k, E])
    ids = np.minimum(g.integers(0, E, (T, k)), g.integers(0, E, (T, k))).astype(np.int32)
    ids[g.random((T, k)) < unused] = -1
    if unused == 0.3:
        ids.reshape(-1)[::17] = E + 3   # past the last expert: not used either
    m, src, pos = bs.moe_plan(torch.from_numpy(ids).cuda(), E)
    torch.cuda.synchronize()
    m_ref, src_ref, pos_ref = ref.plan(ids, E)
    assert np.array_equal(m.cpu().numpy(), m_ref)
    assert np.array_equal(src.cpu().numpy(), src_ref)
    assert np.array_equal(pos.cpu().numpy(), pos_ref)


def test_plan_of_nothing():
    m, src, pos = bs.moe_plan(torch.empty((0, 4), dtype=torch.int32, device="cuda"), 9,
                              m_sizes=torch.full((9,), 5, dtype=torch.int64, device="cuda"))
    assert m.tolist() == [0] * 9 and src.numel() == 0 and pos.shape == (0, 4)


def test_plan_one_expert_takes_all():
    """Every slot to one expert: the order is the slots' own."""
    ids = torch.full((3000, 4), 41, dtype=torch.int32, device="cuda")
    m, src, pos = bs.moe_plan(ids, 64)
    assert m.tolist() == [12000 if e == 41 else 0 for e in range(64)]
    assert torch.equal(src, torch.arange(12000, dtype=torch.int32, device="cuda"))
    assert torch.equal(pos.flatten(), src)


def test_plan_in_a_graph():
    T, k, E = 3000, 4, 32
    stream = torch.cuda.Stream()
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    out = [torch.empty(E, dtype=torch.int64, device="cuda"),
           torch.empty(T * k, dtype=torch.int32, device="cuda"),
           torch.empty((T, k), dtype=torch.int32, device="cuda")]
    with torch.cuda.stream(stream):
        bs.reserve_workspace(bs.moe_plan_workspace_bytes(T, k, E), stream)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            bs.moe_plan(ids, E, *out)
    for seed in range(2):
        new = np.random.default_rng([74, seed]).integers(-1, E, (T, k)).astype(np.int32)
        ids.copy_(torch.from_numpy(new))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, ref.plan(new, E)):
            assert np.array_equal(got.cpu().numpy(), want)


def filled(g, shape, dtype):
    return torch.from_numpy(g.standard_normal(shape).astype(np.float32)).to(DT[dtype])


def order(g, T, k, unused):
    """src, pos of a random plan over 5 experts."""
    ids = g.integers(0, 5, (T, k)).astype(np.int32)
    ids[g.random((T, k)) < unused] = -1
    if T > 1:
        ids[T // 2] = -1 if unused else ids[T // 2]
    _, src, pos = ref.plan(ids, 5)
    return src, pos


COMBINES = [(1, 1, 8, "bf16", 0.0), (1, 1, 4, "f32", 0.0), (7, 3, 1000, "bf16", 0.2),
            (5, 9, 2056, "f32", 0.3), (33, 8, 4096, "bf16", 0.1), (3, 32, 1032, "bf16", 0.0),
            (64, 2, 72, "f32", 0.5), (4, 8, 264, "bf16", 1.0), (301, 3, 88, "bf16", 0.2),
            (37, 17, 520, "f32", 0.1), (9, 2, 1016, "bf16", 0.0), (13, 1, 2048, "bf16", 0.1),
            (6, 1, 1028, "f32", 0.2), (11, 4, 4104, "bf16", 0.1), (10, 2, 4096, "bf16", 0.3),
            (129, 1, 520, "f32", 0.1), (3, 4, 512, "f32", 0.0), (5, 5, 3232, "bf16", 0.1),
            (200, 2, 8, "bf16", 0.1), (21, 4, 1536, "f32", 0.2), (2, 2, 8200, "f32", 0.0)]


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,H,dtype,unused", COMBINES)
def test_combine(T, k, H, dtype, unused, weighted):
    g = np.random.default_rng([75, T, k, H])
    _, pos = order(g, T, k, unused)
    y = filled(g, (T * k, H), dtype)
    w = torch.from_numpy(g.random((T, k)).astype(np.float32)) if weighted else None
    buf = torch.full((T * H + 128,), float("nan"), dtype=DT[dtype], device="cuda")
    out = buf[64:64 + T * H].view(T, H)
    bs.moe_combine(y.cuda(), torch.from_numpy(pos).cuda(), None if w is None else w.cuda(), out=out)
    torch.cuda.synchronize()
    assert bool(torch.isnan(buf[:64]).all() and torch.isnan(buf[64 + T * H:]).all())
    y64 = y.double().numpy()
    want = ref.combine(y64, pos, None if w is None else w.numpy())
    # k FP32 additions of terms whose magnitudes sum to `terms`, then one rounding
    terms = ref.combine(np.abs(y64), pos, None if w is None else w.numpy())
    tol = (k + 1) * 2.0 ** -24 * terms + (2.0 ** -8 if dtype == "bf16" else 0) * np.abs(want)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)


def test_combine_leaves_unused_rows_alone():
    """Rows that no slot uses are never read (here NaN), and rows past R add nothing."""
    y = torch.full((6, 64), float("nan"), device="cuda")
    y[1] = 2.0
    pos = torch.tensor([[1, -1], [6, 1], [1 << 30, -5]], dtype=torch.int32, device="cuda")
    out = bs.moe_combine(y, pos, torch.ones(3, 2, device="cuda"))
    assert out[:, 0].tolist() == [2.0, 2.0, 0.0] and bool(torch.isfinite(out).all())


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,H,dtype,unused", COMBINES)
def test_combine_backward(T, k, H, dtype, unused, weighted):
    g = np.random.default_rng([76, T, k, H])
    src, pos = order(g, T, k, unused)
    y, dout = filled(g, (T * k, H), dtype), filled(g, (T, H), dtype)
    y[torch.from_numpy(src < 0)] = float("nan")   # rows that nobody wrote
    w = torch.from_numpy(g.random((T, k)).astype(np.float32)) if weighted else None
    dy, dw = bs.moe_combine_backward(dout.cuda(), y.cuda() if weighted else None,
                                     torch.from_numpy(src).cuda(), torch.from_numpy(pos).cuda(),
                                     None if w is None else w.cuda())
    torch.cuda.synchronize()
    y64, d64 = np.nan_to_num(y.double().numpy()), dout.double().numpy()
    dy_ref, dw_ref = ref.combine_backward(d64, y64, pos, None if w is None else w.numpy())
    # one FP32 product, rounded to the type
    tol = (2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0)) * np.abs(dy_ref)
    assert np.all(np.abs(dy.double().cpu().numpy() - dy_ref) <= tol)
    if weighted:
        _, terms = ref.combine_backward(np.abs(d64), np.abs(y64), pos, w.numpy())
        # a thread's chain of fused steps, up to 32 elements of a short row, and the tree above it
        assert np.all(np.abs(dw.cpu().numpy() - dw_ref) <= (max(32, H / 256) + 16) * 2.0 ** -24 * terms)
    else:
        assert dw is None


def test_gradient_of_the_weighted_sum_by_differences():
    """<dout, out> along a direction of Y and of the weights, FP32: linear in each, so the
    difference quotient is the gradient but for the rounding of the sums."""
    g = np.random.default_rng([77])
    T, k, H = 6, 3, 512
    src, pos = order(g, T, k, 0.2)
    P, S = torch.from_numpy(pos).cuda(), torch.from_numpy(src).cuda()
    y, dout, vy = (filled(g, s, "f32").cuda() for s in ((T * k, H), (T, H), (T * k, H)))
    w, vw = (torch.from_numpy(g.random((T, k)).astype(np.float32)).cuda() for _ in range(2))
    dy, dw = bs.moe_combine_backward(dout, y, S, P, w)
    f = lambda a, b: (bs.moe_combine(a, P, b).double() * dout.double()).sum()  # noqa: E731
    # values of order sqrt(T k H) = 96, sums of 10^4 terms of order one rounded at 2^-24
    assert abs(f(y + vy, w) - f(y, w) - (dy.double() * vy.double()).sum()) < 1e-3
    assert abs(f(y, w + vw) - f(y, w) - (dw.double() * vw.double()).sum()) < 1e-3


def test_another_stream():
    s = torch.cuda.Stream()
    x = torch.randn(2000, 64, generator=torch.Generator().manual_seed(3)).cuda()
    y = torch.randn(8000, 128, generator=torch.Generator().manual_seed(4)).cuda()
    want_ids, want_w = bs.moe_route(x, 4)
    want = bs.moe_combine(y, bs.moe_plan(want_ids, 64)[2], want_w)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        ids, w = bs.moe_route(x, 4)
        out = bs.moe_combine(y, bs.moe_plan(ids, 64)[2], w)
    s.synchronize()
    assert torch.equal(ids, want_ids) and torch.equal(w, want_w) and torch.equal(out, want)


# where each routing kernel runs: tokens, experts, the logits' type
ROUTE_KERNELS = [(6, 24, "f32"), (6, 40, "bf16"), (7, 96, "f32"), (1025, 64, "bf16"), (1030, 160, "f32"),
                 (8200, 64, "f32"), (8201, 128, "bf16"), (1031, 30, "f32")]


def spread(g, shape, top, dtype):
    """Logits between top - 20 and top."""
    return torch.from_numpy((top - 20 * g.random(shape)).astype(np.float32)).to(DT[dtype])


@pytest.mark.parametrize("T,E,dtype", ROUTE_KERNELS)
@pytest.mark.parametrize("groups", [1, 2])
def test_route_weights_of_experts_far_below_the_largest(T, E, dtype, groups):
    """A bias chooses experts whose scores are 2^-150 and less of the row's largest: their
    renormalised weights are those of the definition all the same, and sum to the scale."""
    g = np.random.default_rng([94, T, E])
    k = 5
    x = spread(g, (T, E), -120.0, dtype)
    x[:, 3] = 90.0
    x[T // 2:, 3] = -20.0
    b = np.zeros(E, dtype=np.float32)
    chosen = np.arange(E - 10, E)
    b[chosen] = 2 + 0.125 * np.arange(10)
    ids, w = bs.moe_route(x.cuda(), k, bias=torch.from_numpy(b).cuda(), groups=groups, topk_groups=1, scale=2.0)
    torch.cuda.synchronize()
    ids_ref, w_ref = ref.route(x.double().numpy(), k, "softmax", b, groups, 1, 1, True, 2.0)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    assert np.allclose(w_ref.sum(1), 2)
    assert np.all(np.abs(w.cpu().numpy() - w_ref) <= W_TOL * np.abs(w_ref) + 1e-37)


@pytest.mark.parametrize("T,E,dtype", ROUTE_KERNELS)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("top", [-60.0, -84.0, -95.0, -400.0])
def test_route_sigmoid_weights_of_small_scores(T, E, dtype, bias, top):
    """All scores far below 1, and below FP32's range: the weights are still their shares."""
    g = np.random.default_rng([95, T, E])
    k = 4
    x = spread(g, (T, E), top, dtype)
    if T > 6:
        x[T // 2:, 1::2] = 3.0      # rows with large scores among the small ones
        x[T // 2:, 0] = 0.25
    b = (0.125 * np.arange(E)).astype(np.float32) if bias else None
    ids, w = bs.moe_route(x.cuda(), k, score="sigmoid", bias=None if b is None else torch.from_numpy(b).cuda())
    torch.cuda.synchronize()
    # (with a bias the keys are FP32 sums: a score below 2^-23 of it leaves it as it is)
    ids_ref, w_ref = ref.route(x.double().numpy(), k, "sigmoid", b)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    assert np.allclose(w_ref.sum(1), 1)
    assert np.all(np.abs(w.cpu().numpy() - w_ref) <= W_TOL * np.abs(w_ref) + 1e-37)


@pytest.mark.parametrize("T", [4, 1100, 8200])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E", [16, 64])
def test_route_sigmoid_weights_of_vanished_scores(T, E, dtype):
    """Scores that vanish in 64 bits too (a mask of the type's lowest value) sum to 0: weights 0."""
    x = torch.full((T, E), float(torch.finfo(DT[dtype]).min), dtype=DT[dtype])
    x[T // 2:, 5] = -700.0
    ids, w = bs.moe_route(x.cuda(), 3, score="sigmoid")
    assert ids[0].tolist() == [0, 1, 2] and w[0].tolist() == [0, 0, 0]
    assert ids[-1].tolist() == [5, 0, 1] and w[-1].tolist() == [1, 0, 0]


def small_scores_gradient(x, ids, dw, scale):
    """Of renormalised sigmoid weights, from the shares' logarithms: p_j (1 - q_j) (d_j - sum p d)."""
    log_q = -np.logaddexp(0, -np.take_along_axis(x, np.maximum(ids, 0), 1))
    log_q[ids < 0] = -np.inf
    p = np.exp(log_q - np.logaddexp.reduce(log_q, axis=1, keepdims=True))
    d = scale * np.where(ids < 0, 0, dw)
    dx = np.zeros(x.shape)
    grad = p * -np.expm1(log_q) * (d - (p * d).sum(1, keepdims=True))
    for t, j in zip(*np.nonzero(ids >= 0)):
        dx[t, ids[t, j]] = grad[t, j]
    return dx


@pytest.mark.parametrize("T,k", [(6, 5), (6, 20), (1100, 8), (1100, 12)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("top", [-60.0, -84.0, -95.0, -400.0])
def test_route_backward_of_small_sigmoid_scores(T, k, dtype, top):
    """Renormalised shares of scores far below 1, and below FP32's range: sums of the scores
    and their reciprocals leave the range, the gradient does not."""
    g = np.random.default_rng([96, T, k])
    E = 40
    x = spread(g, (T, E), top, dtype)
    x[T // 2:, ::3] = 2.5           # rows with large scores among the chosen
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[1, 1:] = -1
    dw = torch.from_numpy(g.standard_normal((T, k)).astype(np.float32))
    dx = bs.moe_route_backward(x.cuda(), torch.from_numpy(ids).cuda(), dw.cuda(), score="sigmoid", scale=2.5)
    torch.cuda.synchronize()
    want = small_scores_gradient(x.double().numpy(), ids, dw.double().numpy(), 2.5)
    if top > -300:   # the Jacobians' squares of the sums are within the range of 64 bits
        assert np.allclose(want, ref.route_backward(x.double().numpy(), ids, dw.numpy(), "sigmoid", True, 2.5),
                           rtol=1e-9, atol=1e-12)
    # as in test_route_backward
    terms = 2.5 * np.abs(dw.numpy()).sum(1, keepdims=True)
    tol = 2.0 ** -18 * terms + (2.0 ** -8 if dtype == "bf16" else 0) * np.abs(want)
    assert np.all(np.abs(dx.double().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("T", [4, 1100])
def test_route_backward_of_vanished_sigmoid_scores(T):
    """Weights that are 0 because no score is left have no gradient."""
    x = torch.full((T, 16), float(np.finfo(np.float32).min))
    ids = torch.arange(3, dtype=torch.int32).repeat(T, 1)
    dx = bs.moe_route_backward(x.cuda(), ids.cuda(), torch.randn(T, 3).cuda(), score="sigmoid")
    assert not dx.any()


def test_the_training_example_with_padding_tokens():
    """Tokens that no expert takes leave rows that no expert owns; the BF16 product wants
    every row owned.  Against the layer in 64 bits."""
    spec = importlib.util.spec_from_file_location(
        "expert_layer", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py"))
    layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(layer)
    g = np.random.default_rng([98])
    T, E, k, H = 70, 6, 2, 128
    x, dout = (filled(g, (T, H), "bf16") for _ in range(2))
    w = (filled(g, (E, H, H), "f32") / 12).bfloat16()
    xl = logits(g, T, E, "bf16")
    pad = np.arange(0, T, 5)
    xl[pad] = -np.inf
    xl[3, 2:] = -np.inf                 # fewer experts than k: one slot unused
    xl[3, 1] = -np.inf
    out, dy, dx = layer.train_step(x.cuda(), xl.cuda(), k, w.cuda(), dout.cuda())
    torch.cuda.synchronize()
    assert bs.device_status() == 0
    ids, wt = ref.route(xl.double().numpy(), k, "softmax")
    rows = np.einsum("th,eoh->teo", x.double().numpy(), w.double().numpy())
    want, dw = np.zeros((T, H)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if ids[t, j] >= 0:
                want[t] += wt[t, j] * rows[t, ids[t, j]]
                dw[t, j] = rows[t, ids[t, j]] @ dout[t].double().numpy()
    # BF16 rows of y (2^-9 of each of two terms) and of the result
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -7 * np.abs(rows).max(1))
    assert not out[pad].any() and not dx[pad].any()
    want = ref.route_backward(xl.double().numpy(), ids, dw, "softmax", True, 1.0)
    # dw: a dot product of BF16 rows, 2^-9 of terms that sum to |rows| . |dout|; the gradient its differences
    terms = np.einsum("teo,to->te", np.abs(rows), np.abs(dout.double().numpy())).max(1, keepdims=True)
    assert np.all(np.abs(dx.double().cpu().numpy() - want) <= 2.0 ** -7 * terms)
