"""moe_step and the residual branch's gradients on the recorder in place of the CUDA runtime: a
call's launches pass data through the stream's workspace, so two host threads' calls on one
stream must not mix, and kernels are set up on every device that they run on."""
import ctypes
import threading
import time

import pytest

from tests import host_calls as hc
from tests.host_calls import LAUNCH, P, i32, i64, p

f32 = ctypes.c_float


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    lib = hc.load(tmp_path_factory.mktemp("step"))
    lib.moe_step.argtypes = [p, i64, i64, p, p, i32, i32, i64, i32, p, p, p, p, i32, p, p]
    lib.branch_enter.argtypes = [p, i32, i64, i64, i32, f32, p, p, i32, p, p, p]
    lib.branch_enter_backward.argtypes = [p, i32, p, i32, i64, i64, i32, f32, p, p, p, p, p, p]
    lib.branch_leave_backward.argtypes = [p, i32, p, i32, i64, i64, i32, f32, p, p, p, i64, f32, f32, f32, p, p, p,
                                          p, p, p, p]
    lib.dropout.argtypes = [p, i32, i64, f32, p, p, p]
    return lib


def step(lib, stream, i, form=0, T=8):
    scales = P if form else None
    return lib.moe_step(P, T, 512 + 512 * i, P, P, 4, 16, 256, form, P, scales, P, scales, 3, P, stream)


def enter_grad(lib, stream, i, H=4096, types=(0, 0)):
    return lib.branch_enter_backward(P, types[1], P, types[0], 300 + i, H, 1, 1e-6, P, None, P, P, P, stream)


def leave_grad(lib, stream, i, H=4096, types=(0, 0)):
    return lib.branch_leave_backward(P, types[0], P, types[1], 300 + i, H, 2, 1e-6, P, P, P, 70, 1.0, 0.5, 0.1, P, P,
                                     P, P, P, P, stream)


def plan(lib, stream, i):
    return lib.moe_plan(P, 3000 + 500 * i, 4, 64, P, P, P, stream)


# the call, and the kernel that a call of it launches last
CALLS = {"step": (step, "step_out_kernel"), "enter": (enter_grad, "sum_kernel"), "leave": (leave_grad, "sum_kernel"),
         "plan": (plan, "plan_place_kernel")}
PAIRS = [("step", "step"), ("step", "plan"), ("enter", "leave"), ("leave", "step")]


@pytest.mark.parametrize("a,b", PAIRS)
def test_calls_on_one_stream_do_not_interleave(lib, a, b):
    stream = 0x9000 + 16 * PAIRS.index((a, b))
    lib.fake_clear()
    lib.fake_set_delay_us(300)
    last, failed = {}, []
    start = threading.Barrier(2)

    def work(name):
        last[lib.fake_thread()] = CALLS[name][1]
        start.wait()
        for i in range(8):
            if CALLS[name][0](lib, stream, i) != 0:
                failed.append(name)
            time.sleep(0.0007)

    threads = [threading.Thread(target=work, args=(n,)) for n in (a, b)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    lib.fake_set_delay_us(0)
    assert not failed
    inside = None   # the thread whose call is under way
    for e in hc.events(lib):
        assert inside in (None, e.thread), (inside, e)
        inside = None if e.kind == LAUNCH and last[e.thread] in e.name else e.thread


def test_second_device_is_set_up_by_itself(lib):
    S = 0x9800

    def calls():
        types = ((0, 0), (1, 1), (1, 0))
        return [step(lib, S, i, form, T) for form in (0, 2, 3, 4, 5) for T in (1, 8, 9, 32) for i in (0, 1, 7)] + \
            [grad(lib, S, 0, H, t) for grad in (enter_grad, leave_grad) for t in types for H in (512, 4096, 7168, 16384)] + \
            [lib.branch_enter(P, x, T, H, 1, 1e-6, P, P, 0, P, None, S) for x in (0, 1) for T in (3, 5000)
             for H in (512, 4096, 16384)] + \
            [lib.dropout(P, 0, n, 0.5, P, P, S) for n in (1, 1 << 20)]

    blocks = {}
    for device in (0, 1, 0):
        lib.fake_set_device(device)
        lib.fake_clear()
        status = calls()
        lib.fake_set_device(0)
        assert not any(status), (device, status)
        got = [(e.name, e.value) for e in hc.events(lib) if e.kind == LAUNCH]
        assert got and blocks.setdefault(device, got) == got
    # persistent products: at most a block an SM (152 and 20 here), and no more of the clusters that
    # share an output unit than run at one time (76 and 10 here, of up to eight blocks)
    for device, sms, clusters in ((0, 152, 76), (1, 20, 10)):
        assert all(v <= sms for n, v in blocks[device] if "step_in" in n)
        assert all(v <= 8 * clusters for n, v in blocks[device] if "step_out" in n)
