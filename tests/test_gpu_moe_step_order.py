"""moe_step reads what the launches just ahead of it wrote: choices from the router, tokens, and expert
weights that were quantised or copied for the call, without a wait on the host in between."""
import pytest
import torch

import block_scaled_precision_mma_gb300 as bs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bs.build()
    bs.load()
    torch.cuda.init()


def operand(w, fmt):
    """Expert weights [E, rows, K] in a form, made by the library's quantisers."""
    E, rows, K = w.shape
    if fmt == "bf16":
        return w.bfloat16(), None
    flat = w.reshape(E * rows, K).contiguous()
    codes, scales = bs.int8_quantize(flat) if fmt == "int8" else bs.mx_quantize(flat, fmt)
    return codes.view(E, rows, -1), scales.view((E, rows) if fmt == "int8" else (E, rows, -1))


@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3", "e5m2", "e2m1"])
@pytest.mark.parametrize("T,E,k,H,F", [(1, 8, 2, 1024, 512), (6, 12, 3, 288, 2080), (20, 16, 4, 512, 256)])
@pytest.mark.parametrize("captured", [False, True])
def test_written_by_the_launches_ahead(T, E, k, H, F, fmt, captured):
    g = torch.Generator(device="cuda").manual_seed(T + H)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    sets = [(rnd(T, E), rnd(T, H).bfloat16(), rnd(E, 2 * F, H) / H ** 0.5, rnd(E, H, F) / F ** 0.5) for _ in range(4)]
    want = []
    for logits, x, w_in, w_out in sets:
        (c_in, s_in), (c_out, s_out) = operand(w_in, fmt), operand(w_out, fmt)
        ids, weights = bs.moe_route(logits, k)
        torch.cuda.synchronize()
        want.append(bs.moe_step(x, ids, weights, c_in, c_out, s_in, s_out, fmt=fmt))
        torch.cuda.synchronize()
    now = [t.clone() for t in sets[0]]

    def chain():
        logits, x, w_in, w_out = now
        ids, weights = bs.moe_route(logits, k)
        (c_in, s_in), (c_out, s_out) = operand(w_in, fmt), operand(w_out, fmt)
        ids2, weights2 = bs.moe_route(logits, k)
        a = bs.moe_step(x, ids2, weights2, c_in, c_out, s_in, s_out, fmt=fmt)     # after the router
        (c_out, s_out), (c_in, s_in) = operand(w_out, fmt), operand(w_in, fmt)
        b = bs.moe_step(x, ids, weights, c_in, c_out, s_in, s_out, fmt=fmt)       # after the weights
        return a, b

    if captured:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            bs.reserve_workspace(bs.moe_step_workspace_bytes(T, k, H, F))
            chain()                                  # every kernel is set up
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = chain()
    outs = []
    for i in (1, 2, 3, 0, 2, 1) * 3:
        for to, t in zip(now, sets[i]):
            to.copy_(t)
        if captured:
            graph.replay()
        outs += [(i, t.clone()) for t in (got if captured else chain())]
    torch.cuda.synchronize()
    assert bs.device_status() == 0
    for i, t in outs:
        assert torch.equal(t, want[i])
