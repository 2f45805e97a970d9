"""Reserve where it cannot, or need not, take a free page for every page of tokens.  Integers against the oracle, bytes
against what was stored; no tolerances."""

import numpy as np
import pytest

import oracle

from gpu_util import announce
from test_gpu_kv import _ids, _state

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _cache(pages, page=32, seqs=6, width=9, layers=1):
    import activation_sparse_decode_relu_amd as pi
    return pi.KVCache(2, 1, 64, pages, page, seqs, width, layers=layers)


def _reserve(c, model, seqs, counts, page):
    """One call on the cache and on the oracle's (table, lens, refs); returns what the oracle says failed."""
    _, failed = oracle.kv_reserve(*model, seqs, counts, page)
    c.reserve(_ids(seqs), _ids(counts))
    assert _state(c) == model
    assert int(c.failed.item()) == failed
    c.failed.zero_()
    return failed


# ---- more than the pool has ------------------------------------------------------------------------------


@pytest.mark.parametrize("pages", [1, 4, 7])
def test_a_request_larger_than_the_whole_pool(pages):
    announce(f"kv reserve, more than {pages} pages")
    for seqs, counts in (([0], [32 * pages + 1]), ([0], [32 * 9]), ([0, 1, 2], [32 * 9, 1, 0]), ([1, 0], [32 * pages, 32 * 9])):
        c = _cache(pages)
        model = _state(c)
        assert _reserve(c, model, seqs, counts, 32) > 0
    c = _cache(pages)
    model = _state(c)
    assert _reserve(c, model, [3], [32 * pages], 32) == 0          # exactly the pool
    assert _reserve(c, model, [3, 4], [1, 0], 32) > 0


# ---- a sequence that reserve refused ---------------------------------------------------------------------


def _read_all(c, layer, s, count):
    got = [torch.full((count, c.desc.kv_heads, c.desc.head_dim), 7.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    c.read(layer, got[0], got[1], _ids([s]), _ids([0, count]))
    return got


@pytest.mark.parametrize("spare", [0, 1])
def test_append_leaves_a_refused_sequence_alone(spare):
    """Two forks on a pool with no page (or one) for the copies a step needs: nothing that is stored changes for the
    sequence that was refused, in any layer, and it goes on once there is room."""
    announce(f"kv append after a refused reserve, {spare} spare pages")
    page, held = 64, 40
    c = _cache(1 + spare, page, layers=2)
    g = torch.Generator(device="cuda")
    g.manual_seed(30)
    kv = [torch.randn(held, 1, 64, device="cuda", generator=g).half() for _ in range(4)]
    c.reserve(_ids([0]), _ids([held]))
    for layer in range(2):
        c.append(layer, kv[2 * layer], kv[2 * layer + 1], _ids([0]), _ids([0, held]))
    c.fork(_ids([0]), _ids([1]))
    before = [[_read_all(c, layer, s, held) for s in range(2)] for layer in range(2)]
    big = 100 * torch.randn(2, 1, 64, device="cuda", generator=g).half()
    for _ in range(2):                                             # as a captured step would, twice
        c.reserve(_ids([0, 1]), _ids([1, 1]))
        for layer in range(2):
            c.append(layer, big, -big, _ids([0, 1]), _ids([0, 1, 2]))
    lens = c.lens.tolist()
    # with one spare page sequence 0 gets it at the first step and sequence 1, then alone on the old page, grows at the second
    assert lens[:2] == ([held, held] if spare == 0 else [held + 2, held + 1])
    for layer in range(2):
        for s in range(2):
            if lens[s] == held:
                for a, b in zip(_read_all(c, layer, s, held), before[layer][s]):
                    assert torch.equal(a, b), f"layer {layer}, sequence {s}: stored tokens changed"
    for layer in range(2):                                         # what was stored, from the definition
        models = [oracle.KvModel(1, 64, "e4m3", "f16") for _ in range(4)]
        for s in range(2):
            for m, x, sign in ((models[2 * s], kv[2 * layer], 1), (models[2 * s + 1], kv[2 * layer + 1], -1)):
                m.append(x.double().cpu().numpy())
                for _ in range(lens[s] - held):
                    m.append(sign * big[s:s + 1].double().cpu().numpy())
            for got, m in zip(_read_all(c, layer, s, lens[s]), models[2 * s:2 * s + 2]):
                assert np.array_equal(got.double().cpu().numpy(), m.values)
    if spare == 0:
        assert int(c.failed.item()) == 4
        c.free(_ids([1]))
        c.reserve(_ids([0]), _ids([1]))
        c.append(0, big[:1], -big[:1], _ids([0]), _ids([0, 1]))
        m = oracle.KvModel(1, 64, "e4m3", "f16")
        m.append(kv[0].double().cpu().numpy())
        m.append(big[:1].double().cpu().numpy())
        assert c.lens.tolist()[0] == held + 1
        assert np.array_equal(_read_all(c, 0, 0, held + 1)[0].double().cpu().numpy(), m.values)


def test_a_refused_sequence_whose_length_the_caller_sets():
    """A caller that keeps table and lengths itself is not held back by an earlier refusal."""
    announce("kv append after a refused reserve, lengths set by the caller")
    c = _cache(2)
    x = torch.randn(40, 1, 64, device="cuda").half()
    c.reserve(_ids([0]), _ids([40]))
    c.append(0, x, x, _ids([0]), _ids([0, 40]))
    c.reserve(_ids([0]), _ids([100]))
    c.lens[0] = 41
    c.append(0, 2 * x[:1], 2 * x[:1], _ids([0]), _ids([0, 1]))
    m = oracle.KvModel(1, 64, "e4m3", "f16")
    m.append(x.double().cpu().numpy())
    m.append(2 * x[:1].double().cpu().numpy())
    assert np.array_equal(_read_all(c, 0, 0, 41)[0].double().cpu().numpy(), m.values)


def test_freed_and_forked_rows_take_tokens_again():
    announce("kv append after a refused reserve, free and fork")
    c = _cache(3, seqs=3)
    x = torch.randn(32, 1, 64, device="cuda").half()
    c.reserve(_ids([0, 1]), _ids([32, 64]))
    c.reserve(_ids([0]), _ids([1]))                                # no page left
    c.free(_ids([0]))
    c.reserve(_ids([0]), _ids([32]))                               # the length at which it was refused
    c.append(0, x, x, _ids([0]), _ids([0, 32]))
    m = oracle.KvModel(1, 64, "e4m3", "f16")
    m.append(x.double().cpu().numpy())
    assert np.array_equal(_read_all(c, 0, 0, 32)[0].double().cpu().numpy(), m.values)
    assert int(c.failed.item()) == 1


def test_a_request_for_no_tokens_is_no_refusal():
    """It can fail behind another that does; what is waiting to be stored is stored, and what was refused stays refused."""
    announce("kv append after a reserve of nothing")
    c = _cache(4)
    x = torch.randn(41, 1, 64, device="cuda").half()
    c.reserve(_ids([0]), _ids([40]))
    c.reserve(_ids([1, 0]), _ids([200, 0]))                        # both counted, the second only for its place
    assert int(c.failed.item()) == 2
    c.append(0, x[:40], x[:40], _ids([0]), _ids([0, 40]))
    m = oracle.KvModel(1, 64, "e4m3", "f16")
    m.append(x[:40].double().cpu().numpy())
    assert np.array_equal(_read_all(c, 0, 0, 40)[0].double().cpu().numpy(), m.values)
    c.reserve(_ids([0]), _ids([200]))
    c.reserve(_ids([0]), _ids([0]))
    c.append(0, x[40:], x[40:], _ids([0]), _ids([0, 1]))
    assert np.array_equal(_read_all(c, 0, 0, 40)[0].double().cpu().numpy(), m.values)
