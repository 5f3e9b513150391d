"""The 64-bit references of the residual branch: the generator against its published answers, the
gradients against central differences (no GPU)."""
import numpy as np
import pytest
import torch

from tests import branch_ref as ref


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_philox_known_answers(counter, key, want):
    """The known-answer vectors published with the generator."""
    assert tuple(int(v) for v in ref.philox(np.array([counter], dtype=np.uint64), key)[0]) == want


def test_mask_keeps_its_share():
    """n values kept with probability q: the count is within 5 standard deviations, the mean of
    the mask 1; other seeds and offsets give other masks, and a later start the same values."""
    n, p = 1 << 16, 0.1
    m = ref.mask(n, p, 3, 5)
    q = 1 - ref.threshold(p) / 65536
    assert abs(float((m > 0).sum()) - n * q) < 5 * (n * q * (1 - q)) ** 0.5
    assert torch.equal(m[800:], ref.mask(n - 800, p, 3, 5, first=800))
    for other in ((3, 6), (4, 5), (3 + (1 << 32), 5), (3, 5 + (1 << 32))):
        assert not torch.equal(m, ref.mask(n, p, *other))


@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
def test_gradients_are_difference_quotients(kind):
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    T, H = 5, 8
    p = {"x": rnd(T, H), "y": rnd(T, H) + 0.3, "gate": rnd(3, H)}
    if kind != "none":
        p |= {"weight": rnd(H), "bias": rnd(H)}
    keep = ref.mask(T * H, 0.25, 1, 2).view(T, H)
    dout = rnd(T, H)

    def loss(**q):
        return float((ref.leave(kind=kind, rows=2, xs=0.75, ys=0.5, keep=keep, **q) * dout).sum())

    of = 0.5 * dout * keep
    dz = of * ref.gate_of(p["gate"], 2, T)
    dy, dw, db = ref.norm_grad(dz, p["y"], kind, p.get("weight"))[:3]
    z = ref.norm(p["y"], kind, p.get("weight"), p.get("bias"))
    dgate = torch.zeros(3, H, dtype=torch.float64).index_add_(0, torch.arange(T) // 2, of * z)
    want = {"x": 0.75 * dout, "y": dy, "gate": dgate, "weight": dw, "bias": db}
    h = 1e-5
    for name, v in p.items():
        for i in range(v.numel()):
            up, down = v.clone(), v.clone()
            up.view(-1)[i] += h
            down.view(-1)[i] -= h
            diff = (loss(**{**p, name: up}) - loss(**{**p, name: down})) / (2 * h)
            # third derivatives of a row's norm stay below 100 at these values: h^2 / 6 of them,
            # and 1e-15 of a loss of at most about 20 over h
            assert abs(diff - float(want[name].reshape(-1)[i])) < 1e-8, (name, i)
