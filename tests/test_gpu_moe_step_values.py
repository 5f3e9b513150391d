"""What moe_step holds of tokens and inner rows with weights in codes, where the values say it exactly:
the inner row keeps FP16's eleven bits over a power of two for each 32 values, a token what is at
least 2^-29 of its largest value, and neither depends on where in BF16's range the values lie.
The sums here are of powers of two and a few bits, exact in FP32, so the output is the definition's
value, rounded once."""
import pytest
import torch

import block_scaled_precision_mma_gb300 as bs
from tests import branch_ref as ref

pytestmark = pytest.mark.gpu
CODES = ["int8", "e4m3", "e5m2", "e2m1"]
ONE = {"int8": 1, "e4m3": 0x38, "e5m2": 0x3C, "e2m1": 0x02}
MINUS = {"int8": -1, "e4m3": 0xB8, "e5m2": 0xBC, "e2m1": 0x0A}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bs.build()
    bs.load()
    torch.cuda.init()


class Weights:
    """[2, rows, K] of zeros, of which expert 1 gets ones or minus ones times powers of two."""

    def __init__(self, rows, K, fmt):
        self.fmt, self.value = fmt, torch.zeros(2, rows, K, dtype=torch.int8 if fmt == "int8" else torch.uint8)
        self.scale = (torch.ones(2, rows) if fmt == "int8" else
                      torch.full((2, rows, K // 32), 127, dtype=torch.uint8))

    def set(self, row, col, sign=1, power=0):
        """One weight; all of a row's (INT8) or of a block's (MX) have one power."""
        self.value[1, row, col] = (ONE if sign > 0 else MINUS)[self.fmt]
        if self.fmt == "int8":
            self.scale[1, row] = 2.0 ** power
        else:
            self.scale[1, row, col // 32] = 127 + power

    def codes(self):
        if self.fmt != "e2m1":
            return self.value
        return self.value[..., ::2] | self.value[..., 1::2] << 4


def run(x, w_in, w_out, weight=1.0):
    """moe_step of expert 1, and the definition in 64 bits rounded to BF16."""
    T, fmt = len(x), w_in.fmt
    x = x.bfloat16()
    ids = torch.ones(T, 1, dtype=torch.int32)
    wt = torch.full((T, 1), weight)
    got = bs.moe_step(x.cuda(), ids.cuda(), wt.cuda(), w_in.codes().cuda(), w_out.codes().cuda(), w_in.scale.cuda(),
                      w_out.scale.cuda(), fmt=fmt, act="none").cpu()
    assert bs.device_status() == 0
    want, _ = ref.moe_step(x.double(), ids, wt.double(), ref.weights(w_in.codes(), w_in.scale, fmt),
                           ref.weights(w_out.codes(), w_out.scale, fmt), "none")
    return got, want.float().bfloat16()


@pytest.mark.parametrize("fmt", CODES)
@pytest.mark.parametrize("T", [1, 9, 17])
@pytest.mark.parametrize("bits", [8, 9, 10])
def test_an_inner_value_keeps_eleven_bits(fmt, T, bits):
    """(1 + 2^-bits) - 1, of two inner values, of one block of 32 and of two."""
    H, F = 64, 160
    pairs = [(0, 1), (31, 2), (33, 64), (159, 5), (100, 99), (128, 127)]
    w_in, w_out = Weights(2 * F, H, fmt), Weights(H, F, fmt)
    for a, b in pairs:
        for f in (a, b):
            w_in.set(f, 0)
            w_in.set(F + f, 40)
        w_in.set(a, 1)
    for r in range(H):
        a, b = pairs[r % len(pairs)]
        w_out.set(r, a)
        w_out.set(r, b, -1)
    x = torch.zeros(T, H)
    x[:, 0], x[:, 1], x[:, 40] = 1, 2.0 ** -bits, 1
    got, want = run(x, w_in, w_out)
    assert torch.equal(got, want) and bool((want.abs() == 2.0 ** -bits).any())


@pytest.mark.parametrize("fmt", CODES)
@pytest.mark.parametrize("shift", [0, 100, -100])
@pytest.mark.parametrize("T", [1, 10])
def test_a_token_keeps_small_values(fmt, shift, T):
    """Values with all of BF16's bits down to 2^-29 of the token's largest, the token anywhere in BF16's
    range: each inner value is one of the token's, and each output one of the inner values."""
    H = F = 64
    w_in, w_out = Weights(2 * F, H, fmt), Weights(H, F, fmt)
    for f in range(F):
        w_in.set(f, f, power=-shift)
        w_in.set(F + f, 1, power=-shift)
        w_out.set(f, f)
    x = torch.zeros(T, H)
    x[:, 0], x[:, 1] = 255 / 128, 1
    for f in range(2, F):
        x[:, f] = (1 + f / 128) * 2.0 ** -(f % 29) * (-1) ** f
    x[:, 2] = (1 + 1 / 128) * 2.0 ** -28
    got, want = run(x * 2.0 ** shift, w_in, w_out)
    assert torch.equal(got, want)
    # (2^-100 times the smallest is subnormal: it has what bits BF16 leaves it)
    assert torch.equal(want[:, 2:].float(), (x * 2.0 ** shift).bfloat16().float()[:, 2:] * 2.0 ** -shift)


@pytest.mark.parametrize("fmt", CODES)
def test_subnormal_and_largest_tokens(fmt):
    H = F = 64
    for value, power in ((2.0 ** -133, 112), (127 * 2.0 ** -133, 110), (255 * 2.0 ** 120, -110), (2.0 ** 127, -105)):
        w_in, w_out = Weights(2 * F, H, fmt), Weights(H, F, fmt)
        for f in range(F):
            w_in.set(f, f, power=power)
            w_in.set(F + f, 1, power=power)
            w_out.set(f, (f + 7) % F, -1, power=20 if power > 0 else -20)
        x = torch.zeros(3, H)
        x[0, :] = value
        x[1, 1], x[1, 5] = value, -value
        x[2, 3] = value
        got, want = run(x, w_in, w_out)
        assert torch.equal(got, want) and want[:2].any() and want.isfinite().all() and not got[2].any()


@pytest.mark.parametrize("fmt", CODES)
@pytest.mark.parametrize("T", [1, 12])
@pytest.mark.parametrize("order", [(60, -60, 0, 30, -30), (-60, 60, 0, -50, 50)])
def test_inner_blocks_of_unequal_size(fmt, T, order):
    """Blocks of 32 inner values that are 2^120 apart, each with all of its bits, and brought back to one
    size by the second weights."""
    H, F = 96, 160
    w_in, w_out = Weights(2 * F, H, fmt), Weights(H, F, fmt)
    for f in range(F):
        w_in.set(f, f % 32, power=order[f // 32])
        w_in.set(F + f, 32)
    for r in range(H):
        for b in range(F // 32) if fmt != "int8" and r % 2 else [r % 5]:
            w_out.set(r, 32 * b + (r + 3 * b) % 32, power=-order[b])
    x = torch.zeros(T, H)
    x[:, :32] = 1 + torch.arange(32) / 128
    x[:, 32] = 1
    got, want = run(x, w_in, w_out, 0.5)
    assert torch.equal(got, want) and bool((want.float() >= 0.5).all())
