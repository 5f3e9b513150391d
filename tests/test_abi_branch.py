"""Refusals of the residual branch's operators: argument errors are found on the host, before
anything is launched (the addresses here are never read)."""
import pytest
import torch

import block_scaled_precision_mma_gb300 as bs

A = 0x10000
S = {n: i for i, n in enumerate(bs.STATUS)}
OK, ARG, UNSUP, ALIGN = (S["BSMMA_" + n] for n in ("OK", "ERR_INVALID_ARG", "ERR_UNSUPPORTED", "ERR_MISALIGNED"))
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    bs.build()
    return bs.load()


ENTER = dict(x=A, x_dtype=0, T=4, H=64, norm=1, eps=1e-6, weight=A, bias=None, form=0, out=A, scales=None,
             stream=None)
LEAVE = dict(x=A, x_dtype=0, y=A, y_dtype=0, T=4, H=64, norm=1, eps=1e-6, weight=A, bias=A, gate=A,
             gate_rows=2, x_scale=1.0, y_scale=1.0, p=0.1, rng=A, out=A, next=1, next_eps=1e-6,
             next_weight=A, next_bias=None, next_form=0, next_out=A, next_scales=None, stream=None)
ENTER_B = dict(dh=A, h_dtype=0, x=A, x_dtype=0, T=4, H=64, norm=1, eps=1e-6, weight=A, dres=A, dx=A,
               dweight=A, dbias=A, stream=None)
LEAVE_B = dict(dout=A, x_dtype=0, y=A, y_dtype=0, T=4, H=64, norm=1, eps=1e-6, weight=A, bias=A, gate=A,
               gate_rows=2, x_scale=1.0, y_scale=1.0, p=0.1, rng=A, dy=A, dx=A, dweight=A, dbias=A,
               dgate=A, stream=None)
DROP = dict(x=A, dtype=0, n=100, p=0.5, rng=A, y=A, stream=None)

COMMON = [(dict(T=-1), ARG), (dict(T=1 << 31), ARG), (dict(H=0), ARG), (dict(H=7), ARG), (dict(H=12), ALIGN),
          (dict(H=16392), ARG), (dict(x_dtype=2), ARG), (dict(norm=3), ARG), (dict(eps=0.0), ARG),
          (dict(eps=-1.0), ARG), (dict(eps=NAN), ARG), (dict(eps=INF), ARG), (dict(weight=A + 4), ALIGN)]
FORMS = [(dict(form=6), ARG), (dict(form=-1), ARG), (dict(form=1), UNSUP), (dict(form=2), ARG),
         (dict(form=0, scales=A), ARG), (dict(form=3, scales=A, H=72), ARG), (dict(form=4), ARG),
         (dict(form=2, scales=A + 2), ALIGN), (dict(form=5, scales=A, out=A + 8), ALIGN), (dict(out=None), ARG)]
DROPS = [(dict(p=1.0), ARG), (dict(p=-0.1), ARG), (dict(p=NAN), ARG), (dict(rng=None), ARG), (dict(rng=A + 4), ALIGN)]


def refused(lib, name, base, cases):
    for change, want in cases:
        assert set(change) <= set(base), change
        assert getattr(lib, name)(*{**base, **change}.values()) == want, (name, change)


def test_enter(lib):
    refused(lib, "branch_enter", ENTER, COMMON + FORMS + [
        (dict(norm=0), ARG), (dict(bias=A + 8), ALIGN), (dict(x=None), ARG), (dict(x=A + 8), ALIGN),
        (dict(T=0, x=None, out=None), OK)])


def test_leave(lib):
    pre = lambda c: {{"form": "next_form", "out": "next_out", "scales": "next_scales"}.get(k, k): v  # noqa: E731
                     for k, v in c.items()}
    refused(lib, "branch_leave", LEAVE, COMMON + [(pre(c), w) for c, w in FORMS] + DROPS + [
        (dict(y_dtype=1), UNSUP), (dict(norm=0), ARG), (dict(norm=0, bias=None), ARG),
        (dict(gate_rows=0), ARG), (dict(gate=A + 8), ALIGN), (dict(x=None), ARG), (dict(y=None), ARG),
        (dict(out=None), ARG), (dict(y=A + 2), ALIGN), (dict(out=A + 2), ALIGN), (dict(next=3), ARG),
        (dict(next=0), ARG), (dict(next=0, next_weight=None), ARG), (dict(next_eps=0.0), ARG),
        (dict(next_weight=A + 4), ALIGN),
        (dict(T=0, x=None, y=None, out=None, next_out=None), OK)])


def test_enter_backward(lib):
    refused(lib, "branch_enter_backward", ENTER_B, COMMON + [
        (dict(norm=0), ARG), (dict(h_dtype=1), UNSUP), (dict(dh=None), ARG), (dict(x=None), ARG),
        (dict(dx=None), ARG), (dict(dres=A + 8), ALIGN), (dict(dweight=A + 4), ALIGN), (dict(dbias=A + 4), ALIGN)])


def test_leave_backward(lib):
    refused(lib, "branch_leave_backward", LEAVE_B, COMMON + DROPS + [
        (dict(y_dtype=1), UNSUP), (dict(norm=0), ARG), (dict(norm=0, weight=None, bias=None), ARG),
        (dict(gate=None), ARG), (dict(gate_rows=-1), ARG), (dict(dy=None), ARG), (dict(dout=None), ARG),
        (dict(dx=A + 8), ALIGN), (dict(dgate=A + 4), ALIGN)])


def test_dropout(lib):
    refused(lib, "dropout", DROP, DROPS + [
        (dict(n=-1), ARG), (dict(n=1 << 40), ARG), (dict(dtype=2), ARG), (dict(x=None), ARG), (dict(y=None), ARG),
        (dict(x=A + 8), ALIGN), (dict(n=0, x=None, y=None), OK)])


def test_workspace_bytes():
    assert bs.branch_backward_workspace_bytes(0, 64) == 0
    assert bs.branch_backward_workspace_bytes(1, 64) == 4 * 64 * 4
    assert bs.branch_backward_workspace_bytes(1 << 20, 16384) <= 64 << 20


def test_binding_refuses():
    """Types and shapes are checked before pointers are taken (CPU tensors suffice)."""
    x, w, h = torch.zeros(4, 64), torch.zeros(64), torch.zeros((4, 64), dtype=torch.bfloat16)
    rng = torch.zeros(2, dtype=torch.int64)
    calls = [lambda: bs.branch_enter(x.double(), w),
                 lambda: bs.branch_enter(x, w.bfloat16()),
                 lambda: bs.branch_enter(x, torch.zeros(32)),
                 lambda: bs.branch_enter(x, w, out=h),
                 lambda: bs.branch_enter(x, w, fmt="bf16", scales=w),
                 lambda: bs.branch_leave(x, h[:3]),
                 lambda: bs.branch_leave(x, h, gate=x),
                 lambda: bs.branch_leave(x, h, gate=h, gate_rows=2),
                 lambda: bs.branch_leave(x, h, gate=h, gate_rows=0),
                 lambda: bs.branch_leave(x, h, p=0.5),
                 lambda: bs.branch_leave(x, h, p=0.5, rng=rng.int()),
                 lambda: bs.branch_enter_backward(h[:2], x, w),
                 lambda: bs.branch_enter_backward(h, x, w, dres=h),
                 lambda: bs.branch_leave_backward(x, h, w, dy=x),
                 lambda: bs.dropout(x, 0.5, None),
                 lambda: bs.dropout(x, 0.5, torch.zeros(3, dtype=torch.int64)),
                 lambda: bs.dropout(x.half(), 0.5, rng),
                 lambda: bs.branch_enter(x, w)]          # the last: right types, not on a GPU
    for call in calls:
        with pytest.raises(ValueError) as e:
            call()
        assert ("current device" in str(e.value)) == (call is calls[-1])
