"""moe_step's sums are cut by sizes and ids alone: a device with fewer SMs, or with room for fewer
clusters of a size, gets the same kernels and the same blocks to a unit (on the recorder)."""
import ctypes

import pytest

from tests import host_calls as hc
from tests.host_calls import LAUNCH, P, i32, i64, p

ROOM = {0: {2: 76, 4: 36, 8: 15}, 1: {2: 10, 4: 5, 8: 2}}
SIZES = [(1, 8, 8, 32), (1, 8, 2048, 256), (3, 2, 4096, 14336), (9, 4, 448, 8192), (32, 8, 7168, 2048),
         (18, 8, 4720, 432), (29, 16, 544, 8640), (4, 2, 65536, 64), (30, 30, 320, 4096), (2, 4, 1024, 2048)]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    lib = hc.load(tmp_path_factory.mktemp("split"))
    lib.moe_step.argtypes = [p, i64, i64, p, p, i32, i32, i64, i32, p, p, p, p, i32, p, p]
    for device, room in ROOM.items():
        for blocks, n in room.items():
            lib.fake_set_clusters(device, blocks, n)
    return lib


@pytest.mark.parametrize("form", [0, 2, 3, 5])
def test_every_device_cuts_alike(lib, form):
    cut = {}
    for device, sms in ((0, 152), (1, 20)):
        lib.fake_set_device(device)
        lib.fake_clear()
        for T, k, H, F in SIZES:
            if form != 0:
                H, F = (H + 31) // 32 * 32, (F + 31) // 32 * 32
            scales = P if form else None
            assert lib.moe_step(P, T, H, P, P, k, 64, F, form, P, scales, P, scales, 3, P, 0x9000) == 0
        cluster = [lib.fake_event_cluster(i) for i in range(lib.fake_events())]
        launches = [(e, c) for e, c in zip(hc.events(lib), cluster) if e.kind == LAUNCH]
        lib.fake_set_device(0)
        cut[device] = [(e.name, c) for e, c in launches]
        for e, c in launches:
            if "step_in" in e.name:
                assert c == 1 and e.value <= sms
            if "step_out" in e.name:     # whole clusters, no more than run at one time
                assert e.value % c == 0 and e.value // c <= ROOM[device].get(c, sms)
    assert cut[0] == cut[1]
    assert len({c for n, c in cut[0] if "step_out" in n}) >= 3 and len({n for n, c in cut[0] if "step_in" in n}) >= 3
