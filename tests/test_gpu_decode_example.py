"""The example's decoder: the cache's operators and the sparse FFN run together.

Nothing here needs a tolerance: a step gives the same bits from a graph, on other pages, and to a fork.
"""

import importlib.util
import os
import subprocess
import sys

import pytest

from gpu_util import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PATH = os.path.join(ROOT, "examples", "decode.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("decode_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _started(example, window, sinks, code, mode, seqs=4):
    model = example.Decoder(2, seqs, 200, window, sinks, code, page_tokens=32, mode=mode)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn(seqs, 70, model.d, device="cuda", generator=g).half()
    return model, example.norm(model.prompts(x))


def _step(example, model, x):
    n = model.seqs
    return example.norm(model.run(x, example.ints(range(n)), example.ints([1] * n), example.ints(range(n + 1)), 1))


@pytest.mark.parametrize("mode", ["predicted", "dense"])
@pytest.mark.parametrize("window, sinks, code", [(0, 0, "e4m3"), (40, 3, "int8")])
def test_graph_fork_and_compaction_keep_the_bits(example, window, sinks, code, mode):
    announce(f"decode example, window {window}, {mode}")
    eager, x = _started(example, window, sinks, code, mode)
    want, y = [], x
    for _ in range(40):
        y = _step(example, eager, y)
        want.append(y)
    model, x2 = _started(example, window, sinks, code, mode)
    assert torch.equal(x, x2)
    state = x2.clone()
    torch.cuda.synchronize()
    graph = model.capture(state)
    for i in range(20):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(state, want[i]), f"step {i}"
    # sequences 2 and 3 become forks of 0 and 1: from here on they repeat them, on pages of their own
    model.cache.free(example.ints([2, 3]))
    model.cache.fork(example.ints([0, 1]), example.ints([2, 3]))
    state[2:] = state[:2]
    for i in range(20, 40):
        if i == 30:
            model.cache.compact()
            live = int((model.cache.refs > 0).sum())
            assert bool((model.cache.refs[:live] > 0).all())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(state[2:], state[:2]), f"step {i}"
        # a predicted batch computes the union of its tokens' masks, so there every row depends on the others
        assert mode == "predicted" or torch.equal(state[:2], want[i][:2]), f"step {i}"
    model.cache.check_failed()
    assert model.cache.lens.tolist() == [110] * 4


def test_command(example):
    announce("decode example, command")
    out = subprocess.run([sys.executable, PATH, "--layers", "2", "--seqs", "4", "--prompt", "50", "--tokens", "8"],
                         capture_output=True, text=True, timeout=100)
    assert out.returncode == 0, out.stderr[-2000:]
    assert "tokens/s" in out.stdout and "after the fork" in out.stdout
