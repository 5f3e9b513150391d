"""What the binding refuses of the residual branch's, dropout's and moe_step's tensors before a
kernel could read them, on stand-ins: any tensor of a call that is on another device than the
current one, on the host, or not contiguous."""
import pytest
import torch

import block_scaled_precision_mma_gb300 as bs


class Here(torch.Tensor):
    """A host tensor that says it is on device 0."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


class Away(Here):
    def get_device(self):
        return 1


class Host(torch.Tensor):
    pass


@pytest.fixture
def calls(monkeypatch):
    """The C calls that were made, in place of the library."""
    made = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: made.append((name, a)) or 0

    monkeypatch.setattr(bs, "load", lambda path=None: Lib())
    monkeypatch.setattr(bs, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return made


T, H, E, k, F = 4, 64, 8, 2, 32
f32, bf16, u8, i32, i64 = torch.float32, torch.bfloat16, torch.uint8, torch.int32, torch.int64
ROWS, COLUMNS = ((T, H), bf16), ((H,), f32)
FORMS = {
    "branch_enter": (dict(x=ROWS, weight=COLUMNS, bias=COLUMNS, out=((T, H), u8), scales=((T, H // 32), u8)),
                     dict(fmt="e4m3")),
    "branch_enter_backward": (dict(dh=ROWS, x=ROWS, weight=COLUMNS, dres=ROWS, dx=ROWS), dict(bias=True)),
    "branch_leave": (dict(x=ROWS, y=ROWS, weight=COLUMNS, bias=COLUMNS, gate=((2, H), bf16), rng=((2,), i64), out=ROWS,
                          next_weight=COLUMNS, next_bias=COLUMNS, next_out=((T, H), torch.int8),
                          next_scales=((T,), f32)),
                     dict(norm="rms", gate_rows=2, p=0.1, next_norm="layer", fmt="int8")),
    "branch_leave_backward": (dict(dout=ROWS, y=ROWS, weight=COLUMNS, bias=COLUMNS, gate=((2, H), bf16),
                                   rng=((2,), i64), dy=ROWS, dx=ROWS), dict(norm="rms", gate_rows=2, p=0.1)),
    "dropout": (dict(x=ROWS, rng=((2,), i64), out=ROWS), dict(p=0.1)),
    "moe_step": (dict(x=ROWS, ids=((T, k), i32), weights=((T, k), f32), w_in=((E, 2 * F, H), u8),
                      w_out=((E, H, F), u8), s_in=((E, 2 * F, H // 32), u8), s_out=((E, H, F // 32), u8), out=ROWS),
                 dict(fmt="e4m3")),
}


def tensors(form, of=Here, bad=None):
    make = lambda n: of if n == bad else Here  # noqa: E731
    return {n: torch.zeros(s, dtype=d).as_subclass(make(n)) for n, (s, d) in form.items()}


@pytest.mark.parametrize("name", FORMS)
def test_a_call_with_everything_here_is_made(calls, name):
    form, more = FORMS[name]
    t = tensors(form)
    getattr(bs, name)(**t, **more)
    assert [c[0] for c in calls] == [name]
    for v in t.values():          # each one's address is passed
        assert v.data_ptr() in calls[0][1]


@pytest.mark.parametrize("name,bad", [(n, b) for n in FORMS for b in FORMS[n][0]])
@pytest.mark.parametrize("of", [Away, Host])
def test_a_tensor_elsewhere_is_refused(calls, name, bad, of):
    form, more = FORMS[name]
    with pytest.raises(ValueError, match="on the current device"):
        getattr(bs, name)(**tensors(form, of, bad), **more)
    assert not calls


@pytest.mark.parametrize("name,bad", [(n, b) for n in FORMS for b in FORMS[n][0]])
def test_a_strided_tensor_is_refused(calls, name, bad):
    form, more = FORMS[name]
    t = tensors(form)
    shape, dtype = form[bad]
    t[bad] = torch.zeros(shape[:-1] + (2 * shape[-1],), dtype=dtype)[..., ::2].as_subclass(Here)
    with pytest.raises(ValueError, match="contiguous"):
        getattr(bs, name)(**t, **more)
    assert not calls


@pytest.mark.parametrize("rows", [None, 1, 100])
def test_an_empty_batch_takes_the_gate_of_all_rows(calls, rows):
    here = lambda *s, dtype=bf16: torch.ones(*s, dtype=dtype).as_subclass(Here)  # noqa: E731
    x = here(0, H)
    for gates in (0, 1):
        gate = here(gates, H)
        assert bs.branch_leave(x, x, gate=gate, gate_rows=rows).shape == (0, H)
        dgate = bs.branch_leave_backward(x, x, gate=gate, gate_rows=rows)[4]
        assert dgate.shape == (gates, H) and dgate.dtype == f32 and not dgate.any()
    for bad in (here(2, H), here(1, H + 8), here(1, H, dtype=f32)):
        with pytest.raises(ValueError, match="gate must be"):
            bs.branch_leave(x, x, gate=bad, gate_rows=rows)
    y = here(5, H)
    with pytest.raises(ValueError, match="gate must be"):
        bs.branch_leave(y, y, gate=here(1, H), gate_rows=4)
