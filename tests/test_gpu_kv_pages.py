"""Reserve where it cannot, or need not, take a free page for every page of tokens.  Integers against the oracle, bytes
against what was stored; no tolerances."""

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
