"""The example's decoder with 4-bit projections, rotated and normalised queries and keys, and beams on one prompt: the
operators run together, with the cache's own and the sparse FFN.

Nothing here needs a tolerance: a step gives the same bits from a graph, and beams fed alike stay alike.
"""

import subprocess
import sys

import pytest

from gpu_util import announce
from test_gpu_decode_example import PATH, example  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _started(example, prompts, beams, code, tokens):
    model = example.Decoder(2, prompts * beams, tokens + 60, 0, 0, code, page_tokens=32, mode="dense", q4=True, rope=True,
                            beams=beams)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn(prompts, tokens, model.d, device="cuda", generator=g).half()
    return model, example.norm(model.prompts(x))


@pytest.mark.parametrize("prompts, beams, code, tokens", [(2, 3, "e4m3", 100), (1, 8, "int8", 333), (3, 1, "e4m3", 33)])
def test_graph_keeps_the_bits(example, prompts, beams, code, tokens):
    announce(f"decode options, {prompts} prompts of {tokens}, {beams} beams")
    eager, x = _started(example, prompts, beams, code, tokens)
    assert x.shape[0] == prompts * beams and bool(torch.isfinite(x).all())
    other = x.clone()
    other[beams - 1] = other[beams - 1].neg()       # one beam goes its own way
    want, y = [], other
    for _ in range(20):
        y = example.norm(eager.run(y, *eager.step()))
        want.append(y)
    model, x2 = _started(example, prompts, beams, code, tokens)
    assert torch.equal(x, x2)
    state = other.clone()
    torch.cuda.synchronize()
    graph = model.capture(state)
    for i in range(20):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(state, want[i]), f"step {i}"
        for p in range(prompts):
            rows = state[p * beams:(p + 1) * beams]
            if p == 0:
                rows = rows[:-1]
            assert all(torch.equal(row, rows[0]) for row in rows), f"step {i}"
    model.cache.check_failed()
    assert model.cache.lens.tolist() == [tokens + 20] * (prompts * beams)
    if beams > 1:   # the prompt's whole pages are held once
        assert int((model.cache.refs == beams).sum()) == prompts * (tokens // 32)


@pytest.mark.parametrize("options", [["--q4"], ["--rope"], ["--beams", "4"], ["--q4", "--rope", "--beams", "2", "--code", "int8"]])
def test_command(example, options):
    announce(f"decode example, {options}")
    out = subprocess.run([sys.executable, PATH, "--layers", "2", "--seqs", "4", "--prompt", "80", "--tokens", "8", *options],
                         capture_output=True, text=True, timeout=100)
    assert out.returncode == 0, out.stderr[-2000:]
    assert "tokens/s" in out.stdout and "after the fork" in out.stdout


@pytest.mark.parametrize("options", [["--beams", "3"], ["--beams", "0"], ["--beams", "2", "--window", "64"]])
def test_command_refuses(example, options):
    out = subprocess.run([sys.executable, PATH, "--seqs", "8", *options], capture_output=True, text=True, timeout=100)
    assert out.returncode == 2 and "--beams" in out.stderr
