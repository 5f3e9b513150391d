"""Refusals of moe_step: argument errors are found on the host, before anything is launched (the
addresses here are never read)."""
import pytest
import torch

import block_scaled_precision_mma_gb300 as bs

A = 0x10000
S = {n: i for i, n in enumerate(bs.STATUS)}
OK, ARG, UNSUP, ALIGN = (S["BSMMA_" + n] for n in ("OK", "ERR_INVALID_ARG", "ERR_UNSUPPORTED", "ERR_MISALIGNED"))
BASE = dict(x=A, T=4, H=64, ids=A, weights=A, k=2, E=8, F=64, form=0, w_in=A, s_in=None, w_out=A, s_out=None,
            act=3, out=A, stream=None)


def test_refusals():
    bs.build()
    lib = bs.load()
    for change, want in [
            (dict(T=-1), ARG), (dict(T=33), ARG), (dict(k=0), ARG), (dict(k=300), ARG), (dict(k=2000), ARG),
            (dict(E=0), ARG), (dict(E=1025), ARG), (dict(H=0), ARG), (dict(H=65544), ARG), (dict(F=0), ARG),
            (dict(F=65544), ARG), (dict(H=60), ARG), (dict(F=4), ARG), (dict(form=1), UNSUP), (dict(form=6), ARG),
            (dict(form=-1), ARG), (dict(form=2), ARG), (dict(s_in=A), ARG), (dict(s_out=A), ARG),
            (dict(form=2, s_in=A, s_out=A, H=72), ARG), (dict(form=3, s_in=A, s_out=A, F=48), ARG),
            (dict(form=5, s_in=A), ARG), (dict(act=4), ARG), (dict(act=-1), ARG), (dict(x=None), ARG),
            (dict(ids=None), ARG), (dict(weights=None), ARG), (dict(w_in=None), ARG), (dict(w_out=None), ARG),
            (dict(out=None), ARG), (dict(x=A + 8), ALIGN), (dict(w_in=A + 8), ALIGN), (dict(w_out=A + 2), ALIGN),
            (dict(out=A + 8), ALIGN), (dict(ids=A + 2), ALIGN), (dict(weights=A + 1), ALIGN),
            (dict(form=2, s_in=A + 2, s_out=A), ALIGN), (dict(form=3, s_in=A, s_out=A + 1), ALIGN), (dict(T=0, x=None, out=None), OK)]:
        assert lib.moe_step(*{**BASE, **change}.values()) == want, change


def test_workspace_bytes():
    assert bs.moe_step_workspace_bytes(0, 2, 64, 64) == 0
    # at least the inner rows, and no more than those, the tokens, their powers of two and the table
    assert 4 * 2 * 64 * 2 <= bs.moe_step_workspace_bytes(4, 2, 64, 64) <= 1 << 15
    assert bs.moe_step_workspace_bytes(33, 2, 64, 64) == 0


def test_binding_refuses():
    x, ids, w = torch.zeros(4, 64).bfloat16(), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    w_in, w_out = torch.zeros(3, 64, 64).bfloat16(), torch.zeros(3, 64, 32).bfloat16()
    s_in, s_out = torch.zeros(3, 64), torch.zeros(3, 64)
    calls = [lambda: bs.moe_step(x.float(), ids, w, w_in, w_out),
                 lambda: bs.moe_step(x, ids.long(), w, w_in, w_out),
                 lambda: bs.moe_step(x, ids, w[:3], w_in, w_out),
                 lambda: bs.moe_step(x, ids, w, w_in[:2], w_out),
                 lambda: bs.moe_step(x, ids, w, w_in, w_out[:, :, :16]),
                 lambda: bs.moe_step(x, ids, w, w_in, w_out, s_in=s_in, s_out=s_out),
                 lambda: bs.moe_step(x, ids, w, w_in.to(torch.int8), w_out.to(torch.int8), fmt="int8"),
                 lambda: bs.moe_step(x, ids, w, w_in.to(torch.int8), w_out.to(torch.int8), s_in=s_in[:2],
                                     s_out=s_out, fmt="int8"),
                 lambda: bs.moe_step(x, ids, w, w_in.to(torch.uint8), w_out.to(torch.uint8), s_in=s_in,
                                     s_out=s_out, fmt="e4m3"),
                 lambda: bs.moe_step(x, ids, w, w_in, w_out)]          # the last: right types, not on a GPU
    for call in calls:
        with pytest.raises(ValueError) as e:
            call()
        assert ("current device" in str(e.value)) == (call is calls[-1])
