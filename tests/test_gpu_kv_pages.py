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


# ---- lengths that the caller lowers ----------------------------------------------------------------------


def _counts_hold(model):
    table, _, refs = model
    named = [0] * len(refs)
    for row in table:
        for p in row:
            if p >= 0:
                named[p] += 1
    return named == refs


def test_pages_past_a_lowered_length_are_used_again():
    """Guessed tokens that were not taken: their pages stay with the sequence and none is lost."""
    announce("kv reserve after a rollback")
    c = _cache(8)
    model = _state(c)
    _reserve(c, model, [0, 1], [34, 70], 32)
    for new_len in (31, 0, 34, 1):
        c.lens[0] = new_len
        model[1][0] = new_len
        _reserve(c, model, [0], [36 - new_len], 32)
        assert _counts_hold(model) and sum(r > 0 for r in model[2]) == 5
    c.lens[1] = 64
    model[1][1] = 64
    _reserve(c, model, [1, 0], [1, 60], 32)                        # 65 tokens on the page it has; 96 take one more
    assert sum(r > 0 for r in model[2]) == 6
    oracle.kv_free(*model, [0, 1])
    c.free(_ids([0, 1]))
    assert _state(c) == model and not any(model[2])


def test_a_shared_page_past_a_lowered_length_is_let_go():
    announce("kv reserve after a rollback of forks")
    c = _cache(9)
    model = _state(c)
    _reserve(c, model, [0], [70], 32)
    oracle.kv_fork(*model, [0, 0], [1, 2])
    c.fork(_ids([0, 0]), _ids([1, 2]))
    for s, n in ((0, 32), (1, 40), (2, 20)):
        c.lens[s] = n
        model[1][s] = n
    _reserve(c, model, [0, 1, 2], [40, 1, 0], 32)                  # 0: two pages anew; 1: a copy; 2: nothing
    assert _counts_hold(model)
    _reserve(c, model, [1, 2], [30, 80], 32)
    assert _counts_hold(model)
    oracle.kv_free(*model, [0, 1, 2])
    c.free(_ids([0, 1, 2]))
    assert _state(c) == model and not any(model[2])


def test_a_page_that_is_named_but_free_is_anyones():
    """A caller that has given a page back by its count alone: the entry is replaced, whoever gets the page."""
    announce("kv reserve, an entry past the length that names a free page")
    c = _cache(6)
    model = _state(c)
    _reserve(c, model, [0, 1], [70, 32], 32)                       # 0, 1, 2 and 3
    for t, part in ((c.lens, model[1]), (c.refs, model[2])):
        at, value = (0, 32) if t is c.lens else (1, 0)             # page 1 is in column 1 of sequence 0
        t[at] = value
        part[at] = value
    _reserve(c, model, [1, 0], [1, 40], 32)                        # 1 takes page 1; 0 takes 4 and keeps 2
    assert model[0][0][:3] == [0, 4, 2] and model[0][1][:2] == [3, 1] and _counts_hold(model)


def test_rollbacks_over_a_long_use():
    """Random reserves, rollbacks, forks, frees and compactions: table, lengths and counts as the oracle's, and every count
    the number of entries that name the page."""
    announce("kv pages, random use with rollbacks")
    rng = np.random.default_rng(31)
    for page, pages in ((32, 30), (96, 18)):
        c = _cache(pages, page, seqs=8, width=6)
        model = _state(c)
        table, lens, refs = model
        for step in range(120):
            kind, some = rng.integers(0, 7), rng.permutation(8)[:rng.integers(1, 6)].tolist()
            if kind <= 2:
                _reserve(c, model, some, [int(x) for x in rng.choice([0, 1, 1, 5, page, 70, 200], len(some))], page)
            elif kind == 3:
                for s in some:
                    lens[s] = int(rng.integers(0, lens[s] + 1))
                c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
            elif kind == 4:
                oracle.kv_free(*model, some[:2])
                c.free(_ids(some[:2]))
            elif kind == 5:
                dst = [s for s in range(8) if all(p < 0 for p in table[s])][:3]
                live = [s for s in range(8) if lens[s] > 0]
                if not dst or not live:
                    continue
                src = [live[int(rng.integers(len(live)))] for _ in dst]
                oracle.kv_fork(*model, src, dst)
                c.fork(_ids(src), _ids(dst))
            else:
                oracle.kv_compact(table, refs)
                c.compact()
            assert _state(c) == model and _counts_hold(model), f"step {step}"


def test_tokens_after_a_rollback():
    """What is stored after a rollback: the kept tokens, and new ones on the pages that were kept."""
    announce("kv append after a rollback")
    c = _cache(4)
    x = torch.randn(90, 1, 64, device="cuda").half().clamp(-2, 2)
    c.reserve(_ids([0]), _ids([70]))
    c.append(0, x[:70], -x[:70], _ids([0]), _ids([0, 70]))
    c.lens[0] = 30                                                 # inside a block of 32
    c.reserve(_ids([0]), _ids([40]))
    c.append(0, x[50:], -x[50:], _ids([0]), _ids([0, 40]))
    got = torch.empty(2, 70, 1, 64, dtype=torch.float16, device="cuda")
    c.read(0, got[0], got[1], _ids([0]), _ids([0, 70]))
    want = torch.cat([x[:30], x[50:]])
    # a block keeps the exponent that dropped tokens brought, -7 at most for amax <= 2: a value is off by half a step of e4m3,
    # 2^-4 of it, or by 2^-10 2^-7 below the normal range, where a larger exponent may round it a second time
    for t, sign in ((got[0], 1), (got[1], -1)):
        err = (t.double() - sign * want.double()).abs()
        assert bool((err <= 2.0 ** -4 * want.double().abs() + 2.0 ** -16).all())
    assert int((c.refs > 0).sum()) == 3


def test_rollbacks_of_more_sequences_than_threads():
    """1500 sequences, some of them forks, every third set back; then one that grows by more columns than a wave has lanes."""
    announce("kv reserve, 1500 sequences with rollbacks")
    rng = np.random.default_rng(32)
    n, pages, width = 1500, 7000, 100
    c = _cache(pages, seqs=n, width=width)
    model = _state(c)
    table, lens, refs = model
    order = rng.permutation(n).tolist()
    _reserve(c, model, order[:1200], [int(x) for x in rng.integers(1, 150, 1200)], 32)
    oracle.kv_fork(*model, order[:300], order[1200:])
    c.fork(_ids(order[:300]), _ids(order[1200:]))
    for s in range(0, n, 3):
        lens[s] = int(rng.integers(0, lens[s] + 1))
    c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    _reserve(c, model, rng.permutation(n).tolist(), [int(x) for x in rng.integers(0, 70, n)], 32)
    assert _counts_hold(model)
    long = order[-1]
    for value in (32 * width, 40):
        _reserve(c, model, [long, order[0]], [value - lens[long], 1], 32)
        assert lens[long] == value and _counts_hold(model)
        lens[long] = 7
        c.lens[long] = 7
    _reserve(c, model, [long], [32 * width - 7], 32)
    assert lens[long] == 32 * width and _counts_hold(model)
    oracle.kv_free(*model, list(range(n)))
    c.free(_ids(range(n)))
    assert _state(c) == model and not any(refs)
