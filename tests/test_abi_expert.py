"""Argument checks of the expert layer's entry points: on the host, before any launch."""
import pytest
import torch

import block_scaled_precision_mma_gb300 as bs

FAKE = 0x10000          # never dereferenced: every case fails validation first
ODD = 0x10008
INVALID, MISALIGNED = 1, 3


@pytest.fixture(scope="module")
def lib():
    bs.build()
    return bs.load()


def route(lib, logits=FAKE, dtype=1, T=4, E=64, k=4, score=0, bias=FAKE, groups=8, top=4, gtop=2,
          renorm=1, scale=1.0, ids=FAKE, w=FAKE):
    return lib.moe_route(logits, dtype, T, E, k, score, bias, groups, top, gtop, renorm, scale, ids, w,
                         None)


@pytest.mark.parametrize("change,expect", [
    (dict(dtype=2), INVALID), (dict(T=-1), INVALID), (dict(E=0, groups=1, top=1), INVALID),
    (dict(E=1032), INVALID), (dict(k=0), INVALID), (dict(k=33), INVALID), (dict(k=30, top=3), INVALID),
    (dict(score=2), INVALID), (dict(groups=0), INVALID), (dict(groups=7), INVALID),
    (dict(groups=64, top=40), INVALID), (dict(top=0), INVALID), (dict(top=9), INVALID),
    (dict(gtop=0), INVALID), (dict(gtop=3), INVALID), (dict(renorm=2), INVALID),
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(w=None), INVALID),
    (dict(logits=ODD), MISALIGNED), (dict(ids=FAKE + 2), MISALIGNED), (dict(bias=FAKE + 1), MISALIGNED),
    (dict(T=0, logits=None, ids=None, w=None), 0),
])
def test_route_refusals(lib, change, expect):
    assert route(lib, **change) == expect


@pytest.mark.parametrize("args,expect", [
    # (logits, dtype, T, E, k, score, renormalize, scale, ids, dweights, dlogits)
    ((FAKE, 1, 4, 64, 65, 0, 1, 1.0, FAKE, FAKE, FAKE), INVALID),
    ((FAKE, 1, 4, 2000, 4, 0, 1, 1.0, FAKE, FAKE, FAKE), INVALID),
    ((FAKE, 1, 4, 64, 4, 0, 1, 1.0, None, FAKE, FAKE), INVALID),
    ((FAKE, 1, 4, 64, 4, 0, 1, 1.0, FAKE, None, FAKE), INVALID),
    ((FAKE, 1, 4, 64, 4, 0, 1, 1.0, FAKE, FAKE, ODD), MISALIGNED),
    ((None, 0, 0, 64, 4, 1, 0, 1.0, None, None, None), 0),
])
def test_route_backward_refusals(lib, args, expect):
    assert lib.moe_route_backward(*args, None) == expect


@pytest.mark.parametrize("args,expect", [
    # (ids, T, k, E, m_sizes, src, pos)
    ((FAKE, -1, 4, 8, FAKE, FAKE, FAKE), INVALID), ((FAKE, 4, 0, 8, FAKE, FAKE, FAKE), INVALID),
    ((FAKE, 4, 4, 0, FAKE, FAKE, FAKE), INVALID), ((FAKE, 4, 4, 1025, FAKE, FAKE, FAKE), INVALID),
    ((FAKE, 1 << 30, 2, 8, FAKE, FAKE, FAKE), INVALID), ((FAKE, 4, 4, 8, None, FAKE, FAKE), INVALID),
    ((None, 4, 4, 8, FAKE, FAKE, FAKE), INVALID), ((FAKE, 4, 4, 8, FAKE, None, FAKE), INVALID),
    ((FAKE, 4, 4, 8, FAKE + 4, FAKE, FAKE), MISALIGNED), ((FAKE, 4, 4, 8, FAKE, FAKE + 2, FAKE), MISALIGNED),
])
def test_plan_refusals(lib, args, expect):
    assert lib.moe_plan(*args, None) == expect


def test_plan_workspace(lib):
    assert lib.moe_plan_workspace_bytes(0, 8, 64) == 0
    assert lib.moe_plan_workspace_bytes(256, 8, 64) == 0
    assert lib.moe_plan_workspace_bytes(257, 8, 64) > 0


@pytest.mark.parametrize("args,expect", [
    # (x, dtype, x_rows, K, src, k, rows, codes, scales)
    ((FAKE, 2, 4, 64, None, 1, 4, FAKE, FAKE), INVALID), ((FAKE, 0, 4, 40, None, 1, 4, FAKE, FAKE), INVALID),
    ((FAKE, 0, 4, 0, None, 1, 4, FAKE, FAKE), INVALID), ((FAKE, 0, 4, 64, None, 1, 5, FAKE, FAKE), INVALID),
    ((FAKE, 0, 4, 64, FAKE, 0, 4, FAKE, FAKE), INVALID), ((None, 0, 4, 64, None, 1, 4, FAKE, FAKE), INVALID),
    ((FAKE, 0, 4, 64, None, 1, 4, None, FAKE), INVALID), ((ODD, 0, 4, 64, None, 1, 4, FAKE, FAKE), MISALIGNED),
    ((FAKE, 0, 4, 64, None, 1, 4, ODD, FAKE), MISALIGNED), ((FAKE, 0, 4, 64, None, 1, 4, FAKE, FAKE + 2), MISALIGNED),
    ((None, 0, 0, 64, None, 1, 0, None, None), 0),
])
def test_int8_quantize_refusals(lib, args, expect):
    assert lib.int8_quantize(*args, None) == expect


@pytest.mark.parametrize("args,expect", [
    # (A, sA, B, sB, bias, D, d_dtype, M, N, K)
    ((FAKE, FAKE, FAKE, FAKE, None, FAKE, 0, 4, 4, 24), INVALID),
    ((FAKE, FAKE, FAKE, FAKE, None, FAKE, 2, 4, 4, 32), INVALID),
    ((FAKE, FAKE, FAKE, FAKE, None, FAKE, 0, -4, 4, 32), INVALID),
    ((FAKE, FAKE, FAKE, FAKE, None, FAKE, 0, 1 << 31, 4, 32), INVALID),
    ((None, FAKE, FAKE, FAKE, None, FAKE, 0, 4, 4, 32), INVALID),
    ((FAKE, None, FAKE, FAKE, None, FAKE, 0, 4, 4, 32), INVALID),
    ((FAKE, FAKE, FAKE, FAKE, None, None, 0, 4, 4, 32), INVALID),
    ((ODD, FAKE, FAKE, FAKE, None, FAKE, 0, 4, 4, 32), MISALIGNED),
    ((FAKE, FAKE, FAKE, FAKE, None, ODD, 1, 4, 4, 32), MISALIGNED),
    ((FAKE, FAKE, FAKE, FAKE + 2, None, FAKE, 1, 4, 4, 32), MISALIGNED),
    ((FAKE, FAKE, FAKE, FAKE, FAKE + 1, FAKE, 1, 4, 4, 32), MISALIGNED),
    ((None, None, None, None, None, None, 0, 0, 4, 32), 0), ((None, None, None, None, None, None, 0, 4, 0, 32), 0),
])
def test_int8_gemm_refusals(lib, args, expect):
    assert lib.int8_gemm(*args, None) == expect


@pytest.mark.parametrize("args,expect", [
    # (X, sX, W, sW, D, d_dtype, m_sizes, total_M, G, N, K)
    ((FAKE, FAKE, FAKE, FAKE, FAKE, 0, FAKE, 8, 4, 64, 40), INVALID),
    ((FAKE, FAKE, FAKE, FAKE, FAKE, 0, FAKE, 8, 0, 64, 64), INVALID),
    ((FAKE, FAKE, FAKE, FAKE, FAKE, 0, FAKE, 8, 1025, 64, 64), INVALID),
    ((FAKE, FAKE, FAKE, FAKE, FAKE, 0, FAKE, -1, 4, 64, 64), INVALID),
    ((FAKE, FAKE, FAKE, FAKE, FAKE, 0, FAKE, 8, 4, 0, 64), INVALID),
    ((FAKE, FAKE, FAKE, FAKE, FAKE, 0, None, 8, 4, 64, 64), INVALID),
    ((FAKE, FAKE, FAKE, FAKE, FAKE, 0, FAKE, 8, 1024, 1 << 21, 64), INVALID),
    ((None, FAKE, FAKE, FAKE, FAKE, 0, FAKE, 8, 4, 64, 64), INVALID),
    ((FAKE, FAKE, ODD, FAKE, FAKE, 0, FAKE, 8, 4, 64, 64), MISALIGNED),
    ((FAKE, FAKE, FAKE, FAKE, FAKE, 0, FAKE + 4, 8, 4, 64, 64), MISALIGNED),
])
def test_grouped_int8_gemm_refusals(lib, args, expect):
    assert lib.grouped_int8_gemm(*args, None) == expect


@pytest.mark.parametrize("args,expect", [
    # (Y, dtype, R, H, pos, weights, T, k, out)
    ((FAKE, 0, 8, 12, FAKE, FAKE, 4, 2, FAKE), MISALIGNED), ((FAKE, 1, 8, 6, FAKE, FAKE, 4, 2, FAKE), MISALIGNED),
    ((FAKE, 0, 8, 0, FAKE, FAKE, 4, 2, FAKE), INVALID), ((FAKE, 0, 8, (1 << 24) + 8, FAKE, FAKE, 4, 2, FAKE), INVALID), ((FAKE, 0, 8, 16, FAKE, FAKE, 4, 33, FAKE), INVALID),
    ((FAKE, 3, 8, 16, FAKE, FAKE, 4, 2, FAKE), INVALID), ((None, 0, 8, 16, FAKE, FAKE, 4, 2, FAKE), INVALID),
    ((FAKE, 0, 8, 16, None, FAKE, 4, 2, FAKE), INVALID), ((ODD, 0, 8, 16, FAKE, FAKE, 4, 2, FAKE), MISALIGNED),
    ((None, 0, 0, 16, None, None, 0, 2, None), 0),
])
def test_combine_refusals(lib, args, expect):
    assert lib.moe_combine(*args, None) == expect


@pytest.mark.parametrize("args,expect", [
    # (dout, dtype, H, Y, src, pos, weights, T, k, dY, dweights)
    ((FAKE, 0, 16, None, FAKE, FAKE, FAKE, 4, 2, FAKE, FAKE), INVALID),
    ((FAKE, 0, 16, FAKE, None, FAKE, FAKE, 4, 2, FAKE, FAKE), INVALID),
    ((FAKE, 0, 16, FAKE, FAKE, FAKE, FAKE, 4, 2, None, FAKE), INVALID),
    ((FAKE, 0, 20, FAKE, FAKE, FAKE, FAKE, 4, 2, FAKE, FAKE), MISALIGNED),
    ((FAKE, 0, 16, FAKE, FAKE, FAKE, FAKE, 4, 2, ODD, FAKE), MISALIGNED),
    ((None, 0, 16, None, None, None, None, 0, 2, None, None), 0),
])
def test_combine_backward_refusals(lib, args, expect):
    assert lib.moe_combine_backward(*args, None) == expect


@pytest.mark.parametrize("tile,fp16,expect", [(0, 0, 0), (1, 0, 0), (64, 0, 0), (256, 1, 0), (192, 1, 0), (0, 0, 0),
                                              (192, 0, INVALID), (64, 1, INVALID), (0, 1, INVALID),
                                              (-1, 0, INVALID), (2, 0, INVALID), (32, 2, INVALID)])
def test_int8_variant_refusals(lib, tile, fp16, expect):
    assert lib.bsmma_set_int8_variant(tile, fp16) == expect
    assert lib.bsmma_set_int8_variant(0, 0) == 0


def test_python_side_refusals():
    """Types and shapes are checked before pointers are taken (CPU tensors suffice)."""
    i8, f = torch.zeros((4, 32), dtype=torch.int8), torch.zeros(4)
    for call in (lambda: bs.moe_route(torch.zeros((4, 8), dtype=torch.float64), 2),
                 lambda: bs.moe_route(torch.zeros(4, 8), 2, bias=torch.zeros(7)),
                 lambda: bs.moe_route_backward(torch.zeros(4, 8), torch.zeros((4, 2), dtype=torch.int64), f),
                 lambda: bs.moe_plan(torch.zeros((4, 2), dtype=torch.int64), 8),
                 lambda: bs.moe_combine(torch.zeros(8, 8), torch.zeros((4, 2), dtype=torch.int32), torch.zeros(4, 3)),
                 lambda: bs.moe_combine_backward(torch.zeros(4, 8), None, torch.zeros(8, dtype=torch.int32),
                                                 torch.zeros((4, 2), dtype=torch.int32), torch.zeros(4, 2)),
                 lambda: bs.int8_quantize(torch.zeros((4, 32), dtype=torch.float16)),
                 lambda: bs.int8_gemm(i8, f, i8.float(), f),
                 lambda: bs.int8_gemm(i8, f, i8, torch.zeros(5)),
                 lambda: bs.grouped_int8_gemm(i8, f, i8[None], f[None], torch.zeros(2, dtype=torch.int64)),
                 lambda: bs.int8_gemm(i8, f, i8, f)):          # right types, not on a GPU
        with pytest.raises(ValueError):
            call()
