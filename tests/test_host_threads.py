"""Entry points that use a stream's workspace, called from several host threads on one stream.
A call looks its workspace up and then enqueues several launches that pass data through it:
another thread's call in between would overwrite that data, and growing the workspace would
free it.  On the recorder no GPU is involved; the GPU test compares results."""
import threading
import time

import pytest
import torch

import block_scaled_precision_mma_gb300 as bs
from tests import host_calls as hc
from tests.host_calls import P, LAUNCH


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return hc.load(tmp_path_factory.mktemp("threads"))


def plan(lib, stream, i):
    return lib.moe_plan(P, 3000 + 500 * i, 4, 64, P, P, P, stream)


def product(lib, stream, i):
    lib.bsmma_set_int8_variant(192, 1)
    return lib.int8_gemm(P, P, P, P, None, P, 0, 512 + 256 * i, 512, 512, stream)


def dense(lib, stream, i):
    return lib.mx_gemm(P, P, P, P, P, 512 + 256 * i, 512, 512, 0, 0, 0, stream)


def dense_bias(lib, stream, i):
    return lib.mx_gemm_bias_act(P, P, P, P, P, 2, P, 512 + 256 * i, 512, 512, 0, 0, 0, stream)


def dense_noalloc(lib, stream, i):
    return lib.mx_gemm_noalloc(P, P, P, P, P, 512, 512, 512, 0, 0, 0, stream)


def reserve(lib, stream, i):
    return lib.bsmma_reserve_workspace((i + 1) << 24, stream)


# the call, and the kernel that a call of it launches last
CALLS = {"plan": (plan, "plan_place_kernel"), "product": (product, "int8_pair_kernel"), "dense": (dense, "mx_gemm_2sm_kernel"),
         "dense_bias": (dense_bias, "mx_gemm_2sm_kernel"), "dense_noalloc": (dense_noalloc, "mx_gemm_2sm_kernel"),
         "reserve": (reserve, None)}


PAIRS = [("plan", "plan"), ("product", "product"), ("plan", "product"), ("dense", "plan"), ("dense", "dense_bias"),
         ("dense_noalloc", "dense_noalloc"), ("plan", "reserve"), ("product", "reserve"), ("dense", "reserve")]


@pytest.mark.parametrize("a,b", PAIRS)
def test_calls_on_one_stream_do_not_interleave(lib, a, b):
    stream = 0x7000 + 16 * PAIRS.index((a, b))
    lib.fake_clear()
    lib.fake_set_delay_us(300)
    last, failed = {}, []
    start = threading.Barrier(2)

    def work(name):
        last[lib.fake_thread()] = CALLS[name][1]
        start.wait()
        for i in range(12):
            if CALLS[name][0](lib, stream, i) != 0:
                failed.append(name)
            time.sleep(0.0007)   # lets the other thread in: the delays keep the library's mutex taken

    threads = [threading.Thread(target=work, args=(n,)) for n in (a, b)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    lib.fake_set_delay_us(0)
    lib.bsmma_set_int8_variant(0, 0)
    assert not failed
    inside = None   # the thread whose call is under way
    for e in hc.events(lib):
        assert inside in (None, e.thread), (inside, e)
        if last[e.thread] is not None:
            inside = None if e.kind == LAUNCH and last[e.thread] in e.name else e.thread


@pytest.mark.gpu
def test_two_threads_on_one_stream_get_their_own_results():
    bs.build()
    bs.load()
    torch.cuda.init()
    K, N, T, E = 512, 384, 3000, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    b = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    ones = torch.ones(2048, device="cuda")
    inputs, want = [], []
    for i in range(2):
        a = torch.randint(-128, 128, (1024 + 512 * i, K), generator=g, device="cuda", dtype=torch.int8)
        ids = torch.randint(-1, E, (T + 999 * i, 4), generator=g, device="cuda", dtype=torch.int32)
        inputs.append((a, ids))
        d = (a.double() @ b.double().T).float()   # below 2^24: exact
        flat = torch.where(ids.flatten() < 0, E, ids.flatten())
        used = int((flat < E).sum())
        src = torch.sort(flat, stable=True)[1].int()
        src[used:] = -1
        want.append((d, src))
    torch.cuda.synchronize()
    bs.set_int8_variant(192, True)
    wrong = []
    start = threading.Barrier(2)

    def work(i):
        a, ids = inputs[i]
        got = []
        start.wait()
        for _ in range(200):
            got.append((bs.int8_gemm(a, ones[:len(a)], b, ones[:N], dtype=torch.float32),
                        bs.moe_plan(ids, E)[1]))
        torch.cuda.synchronize()
        wrong.extend((i, j) for j, v in enumerate(got)
                     if not all(torch.equal(x, y) for x, y in zip(v, want[i])))

    try:
        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        bs.set_int8_variant(0)
    assert not wrong and bs.device_status() == 0
