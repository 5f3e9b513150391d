"""The decoding step's expert layer on the GPU against its definition in 64 bits.

Tolerance: the inner row is rounded to BF16 once (2^-9 of each value, counted as 2^-8 of the
values' sizes with the activation's own error), a sum of K products in FP32 is within 2^-16 of
the products' sizes (chains of at most K / 64 steps of four, 16 partial sums, K <= 14336), and the
output is rounded to BF16."""
import numpy as np
import pytest
import torch

import block_scaled_precision_mma_gb300 as bs
from tests import branch_ref as ref

pytestmark = pytest.mark.gpu
FORMS = ["bf16", "int8", "e4m3", "e5m2", "e2m1"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bs.build()
    bs.load()
    torch.cuda.init()


def experts(g, E, rows, K, fmt):
    """Weights of size about K^-1/2 in a form, and their scales."""
    w = torch.randn(E, rows, K, generator=g) / K ** 0.5
    if fmt == "bf16":
        return w.bfloat16(), None
    if fmt == "int8":
        s = w.abs().amax(2) / 127
        return torch.round(w / s[..., None]).to(torch.int8), s
    pack = 2 if fmt == "e2m1" else 1
    s = torch.randint(118, 124, (E, rows, K // 32), generator=g, dtype=torch.uint8)
    codes = torch.randint(0, 256, (E, rows, K // pack), generator=g, dtype=torch.uint8)
    if fmt == "e4m3":
        codes[(codes & 0x7F) == 0x7F] = 0x01          # no NaN; subnormals stay
    if fmt == "e5m2":
        codes[(codes & 0x7C) == 0x7C] = 0x02
        s -= 16                                       # its codes go up to 57344
    return codes, s


def case(seed, T, E, k, H, F, fmt, masked=False):
    g = torch.Generator().manual_seed(seed)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :k].to(torch.int32)
    if masked:
        ids[torch.rand(T, generator=g) < 0.3] = -1
        ids[torch.rand(T, k, generator=g) < 0.2] = -1
        ids[torch.rand(T, k, generator=g) < 0.1] = E + 5
    c = {"x": torch.randn(T, H, generator=g).bfloat16(), "ids": ids.contiguous(),
         "weights": torch.rand(T, k, generator=g) - 0.1}
    c["w_in"], c["s_in"] = experts(g, E, 2 * F, H, fmt)
    c["w_out"], c["s_out"] = experts(g, E, H, F, fmt)
    return c


def run(c, fmt, act="silu", guard=64):
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    T, H = c["x"].shape
    raw = torch.full((T * H + 2 * guard,), 77, dtype=torch.bfloat16, device="cuda")
    out = raw[guard:guard + T * H].view(T, H)
    bs.moe_step(**d, fmt=fmt, act=act, out=out)
    torch.cuda.synchronize()
    assert bs.device_status() == 0
    assert (raw[:guard] == 77).all() and (raw[guard + T * H:] == 77).all()
    return out.clone()


def check(got, c, fmt, act="silu"):
    want, size = ref.moe_step(c["x"].double(), c["ids"], c["weights"].double(),
                              ref.weights(c["w_in"], c["s_in"], fmt), ref.weights(c["w_out"], c["s_out"], fmt), act)
    tol = size + 2.0 ** -8 * want.abs()
    bad = ~((got.double().cpu() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), got.cpu()[bad][:3], want[bad][:3], tol[bad][:3])


CASES = [
    # T, E, k, H, F, act, masked
    (1, 1, 1, 32, 32, "silu", False),
    (1, 8, 2, 64, 96, "gelu", False),
    (2, 5, 3, 1056, 160, "silu", True),
    (3, 4, 4, 224, 544, "relu", False),
    (8, 3, 2, 512, 256, "none", True),
    (9, 2, 1, 288, 64, "silu", False),
    (16, 4, 3, 160, 288, "gelu", True),
    (17, 3, 3, 96, 1024, "silu", False),
    (32, 16, 4, 256, 128, "silu", True),
    (31, 2, 2, 128, 96, "silu", False),
    (32, 40, 16, 64, 32, "silu", True),
    (5, 1024, 32, 32, 32, "silu", False),
    (3, 5, 2, 544, 1120, "silu", False),       # 17 and 35 blocks a row: scales in two words
    (29, 6, 2, 224, 2080, "relu", True),
]


@pytest.mark.parametrize("T,E,k,H,F,act,masked", CASES)
@pytest.mark.parametrize("fmt", FORMS)
def test_against_64_bits(T, E, k, H, F, act, masked, fmt):
    c = case(T * 1000 + E, T, E, k, H, F, fmt, masked)
    got = run(c, fmt, act)
    check(got, c, fmt, act)
    assert torch.equal(run(c, fmt, act), got)      # the same call, the same bits


@pytest.mark.parametrize("fmt,H,F", [("bf16", 72, 40), ("bf16", 8, 8), ("int8", 48, 16), ("int8", 16, 80)])
def test_odd_sizes(fmt, H, F):
    """Sizes that are whole 16-byte pieces and no more."""
    c = case(H + F, 4, 6, 2, H, F, fmt)
    check(run(c, fmt), c, fmt)


@pytest.mark.parametrize("fmt,H", [("bf16", 168), ("int8", 208), ("e4m3", 288), ("e5m2", 32), ("e2m1", 352)])
@pytest.mark.parametrize("T,k,F", [(5, 8, 4640), (13, 3, 4672)])
def test_many_short_rows(T, k, F, fmt, H):
    """Enough units of short rows to take them in wider units."""
    c = case(T + H, T, 40, k, H, F, fmt, True)
    got = run(c, fmt)
    check(got, c, fmt)
    assert torch.equal(run(c, fmt), got)


def test_long_rows():
    for fmt in ("bf16", "e2m1"):
        c = case(5, 2, 2, 1, 4096, 2080, fmt)
        check(run(c, fmt), c, fmt)


@pytest.mark.parametrize("fmt,H,F", [("bf16", 65536, 8), ("bf16", 8, 65536), ("int8", 65536, 16), ("int8", 16, 65536),
                                     ("e4m3", 65536, 32), ("e5m2", 32, 65536), ("e2m1", 65536, 32)])
def test_longest_rows(fmt, H, F):
    c = case(H % 1000 + F, 2, 2, 1, H, F, fmt)
    check(run(c, fmt), c, fmt)


@pytest.mark.parametrize("T,E,k", [(32, 64, 32), (1, 1024, 1024), (32, 1024, 32)])
def test_most_choices(T, E, k):
    c = case(T + E, T, E, k, 32, 32, "int8")
    check(run(c, "int8"), c, "int8")


def test_weights_past_32_bits_of_bytes():
    """The last expert of more than 2^32 bytes gives what it gives as one of two."""
    E, H, F = 700, 8192, 512
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randint(-127, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    w_in, w_out = rnd(2, 2 * F, H), rnd(2, H, F)
    s_in, s_out = (torch.rand(s, generator=g, device="cuda") / 1024 for s in ((2, 2 * F), (2, H)))
    x = torch.randn(3, H, generator=g, device="cuda").bfloat16()
    ids = torch.tensor([[0, 1], [1, -1], [1, 0]], device="cuda", dtype=torch.int32)
    weights = torch.rand(3, 2, generator=g, device="cuda")
    want = bs.moe_step(x, ids, weights, w_in, w_out, s_in, s_out, fmt="int8")
    many = []
    for t in (w_in, w_out, s_in, s_out):
        all_ = torch.zeros((E,) + t.shape[1:], dtype=t.dtype, device="cuda")
        all_[3], all_[E - 1] = t[0], t[1]
        many.append(all_)
    assert many[0].numel() > 1 << 32
    ids = torch.where(ids == 0, 3, torch.where(ids == 1, E - 1, ids))
    assert torch.equal(bs.moe_step(x, ids, weights, *many, fmt="int8"), want) and want.isfinite().all() and want.any()


def test_same_expert_twice_and_no_expert():
    """A token that names an expert twice, one whose choices are all dropped, and every token on one
    expert (more columns than a tile)."""
    for fmt in ("bf16", "int8", "e4m3"):
        c = case(7, 30, 4, 4, 96, 64, fmt)
        c["ids"][:] = 2
        c["ids"][3] = -1
        c["ids"][5] = torch.tensor([1, 2, 1, 0])
        got = run(c, fmt)
        check(got, c, fmt)
        assert not got[3].any()
        assert torch.equal(run(c, fmt), got)
        c["ids"][:] = -1
        assert not run(c, fmt).any()


def test_unread_values():
    """A NaN weight of a dropped slot, NaN tokens and experts that nobody chose do not show
    elsewhere; what a token has is its own."""
    c = case(11, 6, 8, 2, 96, 64, "bf16")
    c["ids"][:, 0], c["ids"][:, 1] = 1, torch.tensor([2, 3, -1, 2, 3, 2])
    clean = run(c, "bf16")
    c["weights"][2, 1] = float("nan")
    c["w_in"][5], c["w_out"][6] = float("nan"), float("inf")
    c["x"][4] = float("nan")
    got = run(c, "bf16")
    assert got[4].isnan().all()
    for t in (0, 1, 2, 3, 5):
        assert torch.equal(got[t], clean[t])


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m1"])
@pytest.mark.parametrize("H,F", [(96, 224), (32, 160)])
def test_unread_scales(fmt, H, F):
    """Rows whose blocks end inside a stage: the scales behind a row's last are another row's, or
    another expert's, and a NaN there is not the row's."""
    c = case(H + F, 6, 4, 1, H, F, fmt)
    c["ids"][:, 0] = torch.tensor([0, 2, 0, 2, 0, -1])
    clean = run(c, fmt)
    for e in (1, 3):
        c["s_in"][e] = c["s_out"][e] = 255
    assert torch.equal(run(c, fmt), clean)
    c["s_out"][0, 5] = 255
    got = run(c, fmt)
    assert got[[0, 2, 4], 5].isnan().all()
    clean[[0, 2, 4], 5] = got[[0, 2, 4], 5] = 0
    assert torch.equal(got, clean)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "e2m1"])
def test_every_code_and_scale(fmt):
    """Every finite code under every block scale that leaves FP32 finite sums: one weight a row and
    a token of ones reads it back."""
    codes = torch.arange(256, dtype=torch.uint8) if fmt != "e2m1" else torch.arange(16, dtype=torch.uint8)
    if fmt == "e4m3":
        codes = codes[(codes & 0x7F) != 0x7F]
    if fmt == "e5m2":
        codes = codes[(codes & 0x7C) != 0x7C]
    n = len(codes)
    H, F = 32, 32
    pack = 2 if fmt == "e2m1" else 1
    # the inner row is (1, 0, ..), the output's row r is W2[r][0] = one code times its scale
    for low in range(0, 254, 32):
        scales = torch.arange(low, min(low + 32, 254))
        rows = n * len(scales)
        rows = (rows + 31) // 32 * 32
        H = rows
        one = {"e4m3": 0x38, "e5m2": 0x3C, "e2m1": 0x02}[fmt]
        w_in = torch.zeros(1, 2 * F, H // pack, dtype=torch.uint8)
        w_in[0, 0, 0] = w_in[0, F, 0] = one
        w_out = torch.zeros(1, H, F // pack, dtype=torch.uint8)
        s_out = torch.full((1, H, 1), 127, dtype=torch.uint8)
        for i, s in enumerate(scales):
            w_out[0, i * n:(i + 1) * n, 0] = codes
            s_out[0, i * n:(i + 1) * n, 0] = int(s)
        x = torch.zeros(1, H).bfloat16()
        x[0, 0] = 1
        got = bs.moe_step(x.cuda(), torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.ones(1, 1).cuda(),
                          w_in.cuda(), w_out.cuda(), s_in=torch.full((1, 2 * F, H // 32), 127, dtype=torch.uint8).cuda(),
                          s_out=s_out.cuda(), fmt=fmt, act="none")
        want = ref.weights(w_out, s_out, fmt)[0, :, 0]
        # exact but for what BF16 cannot hold: below 2^-126 steps of 2^-133, above its largest infinity
        want = want.float().bfloat16().double()
        sure = (want == 0) | (want.abs() >= 2.0 ** -118)
        assert torch.equal(got[0].double().cpu()[sure], want[sure])


def test_capture_and_streams():
    """Captured and replayed with other choices; two streams at once; after the router."""
    c = case(21, 8, 16, 4, 512, 256, "int8")
    d = {k: None if v is None else v.cuda() for k, v in c.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bs.reserve_workspace(bs.moe_step_workspace_bytes(8, 4, 512, 256))
        bs.device_status()
    logits = torch.randn(8, 16, generator=torch.Generator().manual_seed(1)).cuda()
    graph = torch.cuda.CUDAGraph()
    args = [d[k] for k in ("w_in", "w_out", "s_in", "s_out")]
    with torch.cuda.graph(graph, stream=s):
        ids, w = bs.moe_route(logits, 4)
        got = bs.moe_step(d["x"], ids, w, *args, fmt="int8")
    for i in range(3):
        logits.copy_(torch.randn(8, 16, generator=torch.Generator().manual_seed(50 + i)))
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.default_stream())
            graph.replay()
        s.synchronize()
        ids2, w2 = bs.moe_route(logits, 4)
        want = bs.moe_step(d["x"], ids2, w2, *args, fmt="int8")
        assert torch.equal(ids, ids2) and torch.equal(got, want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for q in streams:
            with torch.cuda.stream(q):
                outs.append(bs.moe_step(d["x"], ids2, w2, *args, fmt="int8"))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    with pytest.raises(bs.BsmmaError) as e:
        big = case(3, 32, 2, 2, 32, 4096, "bf16")
        big = {k: None if v is None else v.cuda() for k, v in big.items()}
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=torch.cuda.Stream()):
            bs.moe_step(**big)
    assert e.value.code == bs.STATUS.index("BSMMA_ERR_WORKSPACE")
