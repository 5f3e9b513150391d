"""The residual branch's operators, the router, moe_step and the products together, as a block's
decoding and training steps use them (examples/residual_block.py)."""
import importlib.util
import os

import pytest
import torch

import block_scaled_precision_mma_gb300 as bs

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def block():
    bs.build()
    bs.load()
    spec = importlib.util.spec_from_file_location("residual_block", os.path.join(ROOT, "examples", "residual_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("argv", [
    [], ["--tokens", "1", "--rows", "77", "--experts", "8", "--k", "2", "--hidden", "512", "--inner", "288"]])
def test_example_runs(block, argv, capsys):
    block.main(argv)
    assert "decoding" in capsys.readouterr().out


def train_case(T, H):
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    p = {"norm": 1 + 0.1 * rnd(H), "post": 1 + 0.1 * rnd(H), "rows": 100,
         "m_sizes": torch.tensor([T], device="cuda"), "w": (rnd(H, H) / H ** 0.5).bfloat16(),
         "gate": rnd(-(-T // 100), H).bfloat16()}
    return p, rnd(T, H).bfloat16(), rnd(T, H).bfloat16(), torch.tensor([3, 8], device="cuda")


def test_training_gradients(block):
    """Every gradient of the block against autograd in FP32.  What differs is BF16 rows: h, y, dy, dh
    and the outputs, half a step of 2^-8 of a value each (2^-9 / sqrt(3) in the norm), at most five in
    a row, and those a product sums are independent: under 2^-7 in the norm."""
    p, x, dout, rng = train_case(730, 1032)
    out, grads = block.train_step(x, p, dout, rng, 0.2)
    keep = bs.dropout(torch.ones(x.shape, device="cuda"), 0.2, rng)
    want_out, want = block.plain_train(x, p, dout, keep)
    assert block.off(out, want_out) < 2.0 ** -8
    for name, v in grads.items():
        assert v.shape == want[name].shape and block.off(v, want[name]) < 2.0 ** -7, name


def test_captured_training_step_beside_an_eager_one(block):
    """The step captured while an eager step's tensors live, replayed with other inputs and numbers."""
    p, x, dout, rng = train_case(256, 512)
    eager = block.train_step(x, p, dout, rng, 0.2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bs.reserve_workspace(bs.branch_backward_workspace_bytes(256, 512))
        block.train_step(x, p, dout, rng, 0.2)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        rng[1] += 1
        out, grads = block.train_step(x, p, dout, rng, 0.2)
    for i in range(2):
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        want_out, want = block.train_step(x, p, dout, rng, 0.2)
        assert torch.equal(out, want_out)
        for k in want:
            # (the weight's own gradient is the library's product, whose algorithm may differ)
            assert k == "w" or torch.equal(grads[k], want[k]), k
        assert not torch.equal(out, eager[0])
