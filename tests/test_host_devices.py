"""One process on two devices: what a kernel's set-up leaves (its shared-memory attribute, how
many of its clusters or blocks fit) belongs to the device it was made on.  On the recorder: a
launch of more than 48 KB of shared memory fails on a device where the attribute was not set."""
import pytest

from tests import host_calls as hc
from tests.host_calls import P, LAUNCH

S = 0x5000   # a stream


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return hc.load(tmp_path_factory.mktemp("devices"))


def int8(dtype, tile, fp16):
    def call(lib):
        assert lib.bsmma_set_int8_variant(tile, fp16) == 0
        # few rows take the few-row kernel's other width
        return [lib.int8_gemm(P, P, P, P, None, P, dtype, m, 4096, 512, S) for m in (4, 16, 2000)] + \
            [lib.grouped_int8_gemm(P, P, P, P, P, dtype, P, 2000, 8, 4096, 512, S)]
    return call


def dense(variant):
    def call(lib):
        lib.bsmma_set_dense_variant(variant)
        formats = [(layout, f, f) for layout in range(3) for f in (0, 1)] + [(0, 2, 2)]
        return [lib.mx_gemm(P, P, P, P, P, 4096, 4096, 512, *f, S) for f in formats] + \
            [lib.mx_gemm_bias_act(P, P, P, P, P, act, P, 4096, 4096, 512, 0, 0, 0, S) for act in range(4)]
    return call


def grouped_fp8(width):
    def call(lib):
        lib.bsmma_set_grouped_tile_width(width)
        return [lib.grouped_fp8_gemm(P, P, P, P, P, P, 4096, 8, 4096, 512, S)]
    return call


def grouped_bf16(variant, width):
    def call(lib):
        lib.bsmma_set_grouped_variant(variant)
        lib.bsmma_set_grouped_tile_width(width)
        return [lib.grouped_bf16_gemm(P, P, P, P, 4096, 8, 4096, 512, S)]
    return call


def quantisers(lib):
    return [lib.mx_quantize(P, d, 4096, 4096, f, c, P, P, S) for d in (0, 1) for f, c in ((0, 0), (2, 0), (1, 1))] + \
        [lib.fp8_group_quantize(P, d, 4096, 4096, P, 8, P, P, S) for d in (0, 1)] + \
        [lib.fp8_block_quantize(P, d, 8, 4096, 4096, P, P, S) for d in (0, 1)]


CALLS = {f"int8_{'f32' if d else 'bf16'}_{t}_{f}": int8(d, t, f) for d in (0, 1)
         for t, f in ((1, 0), (32, 0), (64, 0), (128, 0), (256, 0), (192, 1), (256, 1))}
CALLS.update({f"dense_{v}": dense(v) for v in (1, 3)})
CALLS.update({f"grouped_fp8_{w}": grouped_fp8(w) for w in (128, 256)})
CALLS.update({f"grouped_bf16_{v}_{w}": grouped_bf16(v, w) for v, w in ((1, 128), (1, 256), (3, 0))})
CALLS["quantisers"] = quantisers


@pytest.mark.parametrize("name", CALLS)
def test_second_device_is_set_up_by_itself(lib, name):
    blocks = {}
    for device in (0, 1, 0):
        lib.fake_set_device(device)
        lib.fake_clear()
        status = CALLS[name](lib)
        lib.fake_set_device(0)
        lib.bsmma_set_int8_variant(0, 0)
        lib.bsmma_set_dense_variant(0)
        lib.bsmma_set_grouped_variant(0)
        lib.bsmma_set_grouped_tile_width(0)
        assert not any(status), (device, status)
        got = [(e.name, e.value) for e in hc.events(lib) if e.kind == LAUNCH]
        assert got and blocks.setdefault(device, got) == got
    # persistent kernels on SM pairs: two blocks for each cluster that fits, 76 and 10 here
    pairs = [[v for n, v in blocks[d] if "pair_kernel" in n or "2sm_kernel" in n] for d in (0, 1)]
    assert all(v <= 152 for v in pairs[0]) and all(v <= 20 for v in pairs[1])
