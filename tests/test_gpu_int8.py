"""INT8 quantisation and products on the GPU.  Codes and scales are FP32 decisions and must
match bit for bit; an integer product is exact in FP32 with unit scales, so every index,
tail and group boundary is checked by equality."""
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


def rows_of(g, rows, K, dtype):
    """Rows of different size, with an all-zero, a subnormal, a huge and a halfway row."""
    x = g.standard_normal((rows, K)).astype(np.float32) * np.float32(2) ** g.integers(-6, 7, (rows, 1))
    if rows > 4:
        x[0] = 0
        x[1] *= np.float32(2.0 ** -135)
        x[2] *= np.float32(2.0 ** 110)
        x[3] = (np.arange(K) % 254 - 127) + np.float32(0.5)      # halves once scaled by 1
        x[3, 0] = 127
        x[4] *= np.float32(2.0 ** -149 * 60)
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 16), (9, 48), (130, 512), (33, 1040), (7, 7168), (6, 16400),
                                    (6, 40000), (21, 256), (50, 128), (37, 144),
                                    (19, 1664)])
def test_quantize_bit_exact(rows, K, dtype):
    x = rows_of(np.random.default_rng([80, rows, K]), rows, K, dtype)
    codes, scales = bs.int8_quantize(x.cuda())
    torch.cuda.synchronize()
    c_ref, s_ref = ref.int8_quantize(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), s_ref)
    assert np.array_equal(codes.cpu().numpy(), c_ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [64, 2304])
def test_quantize_gathered(K, dtype):
    g = np.random.default_rng([81, K])
    x = rows_of(g, 20, K, dtype)
    src = np.concatenate([g.permutation(60), [-1, -5, 60, 1 << 30]]).astype(np.int32)
    codes, scales = bs.int8_quantize(x.cuda(), src=torch.from_numpy(src).cuda(), k=3)
    torch.cuda.synchronize()
    c_ref, s_ref = ref.int8_quantize(x.float().numpy(), src, 3)
    assert np.array_equal(scales.cpu().numpy(), s_ref)
    assert np.array_equal(codes.cpu().numpy(), c_ref)
    assert not codes[60:].any() and scales[60:].tolist() == [1, 1, 1, 1]


def test_quantize_near_halves_bit_exact():
    """Quotients within a few ulp of a half, for many scales: where a product with the
    reciprocal would round the other way."""
    g = np.random.default_rng([82])
    s = (g.random(512) + 0.5).astype(np.float32)
    amax = (s * np.float32(127)).astype(np.float32)
    x = ((g.integers(-126, 126, (512, 256)) + 0.5) * s[:, None]).astype(np.float32)
    x = x.view(np.int32) + g.integers(-2, 3, x.shape).astype(np.int32)
    x = x.view(np.float32).copy()
    x[:, 0] = amax
    codes, scales = bs.int8_quantize(torch.from_numpy(x).cuda())
    c_ref, s_ref = ref.int8_quantize(x)
    assert np.array_equal(scales.cpu().numpy(), s_ref)
    assert np.array_equal(codes.cpu().numpy(), c_ref)


@pytest.fixture(params=[(0, 0), (1, 0), (32, 0), (64, 0), (128, 0), (256, 0), (192, 1), (256, 1)],
                ids=["auto", "few", "t32", "t64", "t128", "t256", "f192", "f256"])
def variant(request):
    """Runs the test with each of the kernels."""
    bs.set_int8_variant(*request.param)
    yield request.param
    bs.set_int8_variant(0)


def codes(g, *shape):
    return g.integers(-128, 128, shape).astype(np.int8)


def product(a, b):
    return a.astype(np.float64) @ b.astype(np.float64).T


def dense(a, sa, b, sb, bias=None, dtype="f32"):
    """int8_gemm into a buffer with guard bands."""
    M, N = len(a), len(b)
    buf = torch.full((M * N + 128,), float("nan"), dtype=DT[dtype], device="cuda")
    out = buf[64:64 + M * N].view(M, N)
    up = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    bs.int8_gemm(up(a), up(sa), up(b), up(sb), bias=None if bias is None else bias.cuda(), out=out)
    torch.cuda.synchronize()
    assert bs.device_status() == 0
    assert bool(torch.isnan(buf[:64]).all() and torch.isnan(buf[64 + M * N:]).all())
    return out.double().cpu().numpy()


SHAPES = [(1, 1, 16), (1, 257, 48), (3, 130, 4096), (8, 100, 144), (9, 64, 1040), (17, 513, 64),
          (31, 1000, 272), (33, 255, 128), (64, 256, 512), (65, 300, 2304), (127, 129, 96),
          (129, 513, 160), (200, 1024, 528), (256, 256, 16), (257, 511, 1024), (700, 777, 1600),
          (1500, 2049, 320)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_dense_product_is_exact(M, N, K, variant):
    g = np.random.default_rng([83, M, N, K])
    a, b = codes(g, M, K), codes(g, N, K)
    one = lambda n: np.ones(n, dtype=np.float32)  # noqa: E731
    assert np.array_equal(dense(a, one(M), b, one(N)), product(a, b))


@pytest.mark.parametrize("M", [2, 40, 300])
def test_dense_largest_values_are_exact(M, variant):
    """Every product +-2^14: partial sums of 2^24 at K = 1024, the longest that must be exact."""
    K, N = 1024, 160
    a = np.full((M, K), -128, dtype=np.int8)
    b = np.full((N, K), -128, dtype=np.int8)
    b[1::2] = 127
    one = lambda n: np.ones(n, dtype=np.float32)  # noqa: E731
    assert np.array_equal(dense(a, one(M), b, one(N)), product(a, b))


@pytest.mark.parametrize("M", [5, 200])
def test_dense_one_sided_sums_round_as_fp32(M, variant):
    """Partial sums past 2^24: each of at most K / 16 accumulator steps may round (or cut) at
    2^-23 of the sum."""
    K, N = 14336, 96
    a = np.full((M, K), 127, dtype=np.int8)
    b = np.full((N, K), 127, dtype=np.int8)
    b[::3, ::7] = 90
    one = lambda n: np.ones(n, dtype=np.float32)  # noqa: E731
    want = product(a, b)
    assert np.all(np.abs(dense(a, one(M), b, one(N)) - want) <= K / 16 * 2.0 ** -23 * want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("M,N,K", [(1, 130, 256), (12, 77, 512), (70, 513, 4096), (300, 600, 2064)])
def test_dense_scales_and_bias(M, N, K, bias, dtype, variant):
    g = np.random.default_rng([84, M, N, K])
    a, b = codes(g, M, K), codes(g, N, K)
    sa, sb = (g.random(n).astype(np.float32) * 0.02 + 0.001 for n in (M, N))
    bb = torch.from_numpy(g.standard_normal(N).astype(np.float32)).bfloat16() if bias else None
    want = ref.int8_gemm(a, sa, b, sb, None if bb is None else bb.float().numpy())
    plain = np.abs(ref.int8_gemm(a, sa, b, sb))
    # the exact integer sum times two FP32 scales, one addition, one rounding to the type
    tol = 4 * 2.0 ** -24 * (plain + np.abs(want)) + (2.0 ** -8 if dtype == "bf16" else 0) * np.abs(want)
    assert np.all(np.abs(dense(a, sa, b, sb, bb, dtype) - want) <= tol)


@pytest.mark.parametrize("M", [4, 150])
def test_dense_of_no_k(M):
    z = np.zeros((M, 0), dtype=np.int8), np.zeros((24, 0), dtype=np.int8)
    one = lambda n: np.ones(n, dtype=np.float32)  # noqa: E731
    bias = torch.arange(24).bfloat16()
    assert np.array_equal(dense(z[0], one(M), z[1], one(24), bias), np.tile(np.arange(24.0), (M, 1)))
    assert not dense(z[0], one(M), z[1], one(24)).any()


@pytest.mark.parametrize("M,N,K", [(7, 4096, 8192), (100, 2304, 8208), (260, 1300, 4112), (600, 3000, 2064)])
def test_dense_split_units_are_exact(M, N, K, variant):
    """Few units of a long K: the last wave is split over the idle SM pairs."""
    g = np.random.default_rng([90, M, N, K])
    a, b = codes(g, M, K), codes(g, N, K)
    one = lambda n: np.ones(n, dtype=np.float32)  # noqa: E731
    assert np.array_equal(dense(a, one(M), b, one(N)), product(a, b))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_dense_long_sums_repeat(dtype, variant):
    """Hundreds of stages in a row, many launches: the loads of a ring may come in any order."""
    g = np.random.default_rng([88])
    a, b = (torch.from_numpy(g.integers(-15, 16, (n, 13776)).astype(np.int8)).cuda() for n in (1100, 520))
    ones = [torch.ones(n, device="cuda") for n in (1100, 520)]
    want = (a.double() @ b.double().T).to(DT[dtype])   # below 2^24: exact before the rounding
    for _ in range(40):
        out = bs.int8_gemm(a, ones[0], b, ones[1], dtype=DT[dtype])
        assert torch.equal(out, want)


@pytest.mark.slow
def test_dense_many_units(variant):
    """More units than SM pairs, with a split remainder, both accumulators in turn."""
    M, N, K = 1543, 9000, 1072
    g = np.random.default_rng([91])
    a, b = codes(g, M, K), codes(g, N, K)
    one = lambda n: np.ones(n, dtype=np.float32)  # noqa: E731
    got = dense(a, one(M), b, one(N))
    want = (torch.from_numpy(a).cuda().double() @ torch.from_numpy(b).cuda().double().T).cpu().numpy()
    assert np.array_equal(got, want)


def grouped(a, sa, b, sb, sizes, dtype="f32"):
    T, N = len(a), b.shape[1]
    buf = torch.full((T * N + 128,), float("nan"), dtype=DT[dtype], device="cuda")
    out = buf[64:64 + T * N].view(T, N)
    up = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    bs.grouped_int8_gemm(up(a), up(sa), up(b), up(sb), torch.tensor(sizes, device="cuda"), out=out)
    torch.cuda.synchronize()
    assert bool(torch.isnan(buf[:64]).all() and torch.isnan(buf[64 + T * N:]).all())
    return out.double().cpu().numpy()


SPLITS = [[5], [0, 0, 3, 0], [1, 0, 7, 9, 0, 2, 64, 11], [3, 0, 300, 1, 0, 129, 2, 5],
          [128, 128, 0, 256], [0] * 100 + [1, 2] + [0] * 50 + [33], [1] * 260, [600, 1, 255, 257],
          [2] * 1024]


@pytest.mark.parametrize("extra", [0, 5], ids=["full", "rows_left"])
@pytest.mark.parametrize("sizes", SPLITS, ids=lambda s: f"G{len(s)}_T{sum(s)}")
def test_grouped_product_is_exact(sizes, extra, variant):
    g = np.random.default_rng([85, len(sizes), sum(sizes)])
    G, T, N, K = len(sizes), sum(sizes), 200, 144
    a, b = codes(g, T + extra, K), codes(g, G, N, K)
    sa = np.float32(2) ** g.integers(-3, 4, T + extra).astype(np.float32)   # exact scales
    sb = np.float32(2) ** g.integers(-3, 4, (G, N)).astype(np.float32)
    got = grouped(a, sa, b, sb, sizes)
    assert bs.device_status() == 0
    row = 0
    for i, m in enumerate(sizes):
        assert np.array_equal(got[row:row + m], ref.int8_gemm(a[row:row + m], sa[row:row + m], b[i], sb[i]))
        row += m
    assert np.isnan(got[T:]).all()      # rows past the sum are left as they are


@pytest.mark.parametrize("T,N,K,G", [(20, 1000, 1552, 6), (900, 769, 1552, 6), (2200, 384, 80, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grouped_types_and_tails(T, N, K, G, dtype, variant):
    g = np.random.default_rng([86, T, N, K])
    sizes = g.multinomial(T, np.arange(G) / (G * (G - 1) / 2)).tolist()
    a, b = codes(g, T, K), codes(g, G, N, K)
    sa = g.random(T).astype(np.float32)
    sb = g.random((G, N)).astype(np.float32)
    got = grouped(a, sa, b, sb, sizes, dtype)
    row = 0
    for i, m in enumerate(sizes):
        want = ref.int8_gemm(a[row:row + m], sa[row:row + m], b[i], sb[i])
        tol = (4 * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0)) * np.abs(want)
        assert np.all(np.abs(got[row:row + m] - want) <= tol)
        row += m


@pytest.mark.parametrize("T", [24, 900])
@pytest.mark.parametrize("bad", [[10, -1, 5, 0], [10, 900, 0, 0], [1 << 40, 0, 0, 0], [0, 0, 0, -(1 << 62)]])
def test_grouped_bad_sizes_write_nothing(bad, T, variant):
    D = torch.full((T, 256), 5.0, device="cuda")
    X = torch.ones((T, 128), dtype=torch.int8, device="cuda")
    W = torch.ones((4, 256, 128), dtype=torch.int8, device="cuda")
    bs.grouped_int8_gemm(X, torch.ones(T, device="cuda"), W, torch.ones((4, 256), device="cuda"),
                         torch.tensor(bad, device="cuda"), out=D)
    assert bs.device_status() == 7
    assert bool((D == 5).all())


def test_grouped_without_rows(variant):
    W = torch.ones((4, 256, 128), dtype=torch.int8, device="cuda")
    D = bs.grouped_int8_gemm(torch.empty((0, 128), dtype=torch.int8, device="cuda"),
                             torch.empty(0, device="cuda"), W, torch.ones((4, 256), device="cuda"),
                             torch.zeros(4, dtype=torch.int64, device="cuda"))
    assert bs.device_status() == 0 and D.shape == (0, 256)


@pytest.mark.parametrize("M,N,K", [(3, 512, 8192), (100, 1000, 4096), (1000, 1000, 1040)])
def test_same_call_same_bits(M, N, K, variant):
    g = np.random.default_rng([87, M])
    a, b = codes(g, M, K), codes(g, N, K)
    sa, sb = g.random(M).astype(np.float32), g.random(N).astype(np.float32)
    assert np.array_equal(dense(a, sa, b, sb), dense(a, sa, b, sb))


def test_products_in_a_graph_on_a_stream(variant):
    """Captured without a reservation and replayed on new inputs and a new split."""
    G, N, K, T = 5, 300, 272, 90
    stream = torch.cuda.Stream()
    g = np.random.default_rng([88])
    X = torch.zeros((T, K), dtype=torch.int8, device="cuda")
    W = torch.from_numpy(codes(g, G, N, K)).cuda()
    sX, sW = torch.ones(T, device="cuda"), torch.ones((G, N), device="cuda")
    m = torch.zeros(G, dtype=torch.int64, device="cuda")
    D, D2 = torch.empty((T, N), device="cuda"), torch.empty((T, N), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        bs.grouped_int8_gemm(X, sX, W, sW, m, out=D, stream=stream)
        bs.int8_gemm(X, sX, W[1], sW[1], out=D2, stream=stream)
    for sizes in ([90, 0, 0, 0, 0], [1, 40, 0, 9, 40]):
        a = codes(g, T, K)
        X.copy_(torch.from_numpy(a))
        m.copy_(torch.tensor(sizes))
        graph.replay()
        torch.cuda.synchronize()
        which = np.repeat(np.arange(G), sizes)
        w = W.cpu().numpy()
        want = np.stack([product(a[i:i + 1], w[which[i]])[0] for i in range(T)])
        assert np.array_equal(D.double().cpu().numpy(), want)
        assert np.array_equal(D2.double().cpu().numpy(), product(a, w[1]))
    assert bs.device_status() == 0


def test_the_expert_layer_end_to_end():
    """Route, order, quantise in that order, multiply, sum: against the same layer in 64 bits
    on the quantised values."""
    g = np.random.default_rng([89])
    T, E, k, H, F = 50, 12, 3, 256, 320
    x = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).bfloat16()
    logits = torch.from_numpy(g.standard_normal((T, E)).astype(np.float32))
    logits[7] = -float("inf")           # a padding token
    w, sw = codes(g, E, F, H), g.random((E, F)).astype(np.float32) * 0.01
    ids, wt = bs.moe_route(logits.cuda(), k)
    m, src, pos = bs.moe_plan(ids, E)
    cx, sx = bs.int8_quantize(x.cuda(), src=src, k=k)
    y = bs.grouped_int8_gemm(cx, sx, torch.from_numpy(w).cuda(), torch.from_numpy(sw).cuda(), m,
                             dtype=torch.float32)
    out = bs.moe_combine(y, pos, wt)
    torch.cuda.synchronize()
    assert bs.device_status() == 0
    c_ref, s_ref = ref.int8_quantize(x.float().numpy())
    ids_ref, w_ref = ref.route(logits.double().numpy(), k, "softmax")
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    want = np.zeros((T, F))
    for t in range(T):
        for j in range(k):
            if ids_ref[t, j] >= 0:
                e = ids_ref[t, j]
                want[t] += w_ref[t, j] * ref.int8_gemm(c_ref[t:t + 1], s_ref[t:t + 1], w[e], sw[e])[0]
    assert not out[7].any()
    # weights within 2^-18, sums of three FP32 terms
    assert np.all(np.abs(out.cpu().numpy() - want) <= 2.0 ** -16 * np.abs(want).max())


# Scales whose product leaves FP32's range, alone or with another's: subnormal and zero products,
# overflowing ones, a huge scale beside a tiny or a subnormal one.
TOKEN_SCALES = [1.3 * 2.0 ** -80, 1.3 * 2.0 ** 100, 1.1 * 2.0 ** 120, 1.1 * 2.0 ** -130, 0.0, 0.02, -2.0 ** 90]
CHANNEL_SCALES = [1.7 * 2.0 ** -65, 1.7 * 2.0 ** 60, 1.2 * 2.0 ** -130, 1.2 * 2.0 ** 120, 0.003, 0.0, -0.5,
                  1.9 * 2.0 ** -90, 1.4 * 2.0 ** -55]


def check_wide(got, sums, sa, sb, bias, dtype):
    """(sum * sA) * sB + bias in 64 bits, where no step leaves the range; what rounds past the
    type's largest number is infinite.  Three FP32 roundings and the type's, each half a step of
    a subnormal at least."""
    with np.errstate(over="ignore"):
        plain = sums * np.outer(sa.astype(np.float64), sb.astype(np.float64))
        want = plain if bias is None else plain + bias
        wide = np.abs(want) >= 2.0 ** 128 - 2.0 ** (119 if dtype == "bf16" else 103)
    assert np.array_equal(got[wide], np.sign(want[wide]) * np.inf)
    tol = 4 * 2.0 ** -24 * (np.abs(plain) + np.abs(want)) + 2.0 ** -147
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * np.abs(want) + 2.0 ** -133
    assert np.all(np.abs(got[~wide] - want[~wide]) <= tol[~wide])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M,N,K", [(5, 70, 144), (60, 300, 272), (7, 600, 4096), (900, 1030, 2064)])
def test_dense_scales_of_any_size(M, N, K, bias, dtype, variant):
    """Also units split along K; a row of zeros, whose sums are 0 whatever the scales."""
    g = np.random.default_rng([92, M, N, K])
    a, b = codes(g, M, K), codes(g, N, K)
    a[0] = a[M // 2] = 0
    sa = np.resize(np.float32(TOKEN_SCALES), M)
    sb = np.resize(np.float32(CHANNEL_SCALES), N)
    sa[0], sa[M // 2] = 1.1 * 2.0 ** 120, 1.3 * 2.0 ** 100
    bb = torch.from_numpy(g.standard_normal(N).astype(np.float32)).bfloat16() if bias else None
    check_wide(dense(a, sa, b, sb, bb, dtype), product(a, b), sa, sb, None if bb is None else bb.double().numpy(), dtype)


@pytest.mark.parametrize("sizes", [[3, 0, 20, 1], [130, 0, 300, 5]], ids=lambda s: f"T{sum(s)}")
def test_grouped_scales_of_any_size(sizes, variant):
    g = np.random.default_rng([93, sum(sizes)])
    G, T, N, K = len(sizes), sum(sizes), 200, 144
    a, b = codes(g, T, K), codes(g, G, N, K)
    a[2] = a[T // 2] = 0
    sa = np.resize(np.float32(TOKEN_SCALES), T)
    sb = np.resize(np.float32(CHANNEL_SCALES), G * N).reshape(G, N)
    got = grouped(a, sa, b, sb, sizes)
    assert bs.device_status() == 0
    row = 0
    for i, m in enumerate(sizes):
        check_wide(got[row:row + m], product(a[row:row + m], b[i]), sa[row:row + m], sb[i], None, "f32")
        row += m


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [16, 64, 512, 2048, 7168, 40000])
def test_quantize_shows_what_is_not_finite(K, dtype):
    """A NaN in a row makes its scale NaN and an infinity makes it infinite, wherever in the row
    they are; the rows beside it are as they would be alone."""
    g = np.random.default_rng([97, K])
    x = g.standard_normal((9, K)).astype(np.float32)
    for r, (at, v) in enumerate([(0, np.nan), (K - 1, np.nan), (K // 2 + 1, -np.nan), (K // 2, np.inf), (1, -np.inf)]):
        x[r, at] = v
    x[5, [0, K - 1]] = np.inf, np.nan
    xt = torch.from_numpy(x).to(DT[dtype])
    c, s = bs.int8_quantize(xt.cuda())
    torch.cuda.synchronize()
    s = s.cpu().numpy()
    assert np.isnan(s[[0, 1, 2, 5]]).all() and np.isposinf(s[[3, 4]]).all()
    c_ref, s_ref = ref.int8_quantize(xt[6:].float().numpy())
    assert np.array_equal(s[6:], s_ref) and np.array_equal(c[6:].cpu().numpy(), c_ref)


@pytest.mark.parametrize("M,N,K", [(100, 2304, 8208), (700, 1000, 4112)])
def test_products_in_a_graph_with_reserved_workspaces(M, N, K, variant):
    """With the workspaces reserved a captured call widens its rows by a pass of its own (two
    launches, the second started early) and splits its units along K, as outside a graph."""
    G = 3
    stream = torch.cuda.Stream()
    bs.reserve_workspace(2 * M * K, stream)
    g = np.random.default_rng([100, M])
    X = torch.zeros((M, K), dtype=torch.int8, device="cuda")
    W = torch.from_numpy(codes(g, G, N, K)).cuda()
    sX, sW = torch.ones(M, device="cuda"), torch.ones((G, N), device="cuda")
    m = torch.zeros(G, dtype=torch.int64, device="cuda")
    D, D2 = torch.empty((M, N), device="cuda"), torch.empty((M, N), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    before = bs.launch_count()
    with torch.cuda.graph(graph, stream=stream):
        bs.int8_gemm(X, sX, W[1], sW[1], out=D2, stream=stream)
        bs.grouped_int8_gemm(X, sX, W, sW, m, out=D, stream=stream)
    if variant != (0, 0):
        assert bs.launch_count() - before == (4 if variant[1] else 2)
    w = W.double()
    for sizes in ([M, 0, 0], [M - 33, 1, 32], [10, M - 90, 80]):
        a = torch.from_numpy(codes(g, M, K)).cuda()
        which = torch.repeat_interleave(torch.arange(G), torch.tensor(sizes)).cuda()
        per_group = torch.stack([a.double() @ w[i].T for i in range(G)])
        want = per_group[which, torch.arange(M, device="cuda")].float()
        X.copy_(a)
        m.copy_(torch.tensor(sizes))
        for _ in range(3):   # one after another, the workspaces as the last left them
            D.fill_(float("nan"))
            D2.fill_(float("nan"))
            graph.replay()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(D, want)
            assert torch.equal(D2, per_group[1].float())
    assert bs.device_status() == 0
