"""Attention over the cache where a call is cut up: parts of an item that are joined, more pieces than a launch has
workgroups, splits of a tile's tokens, and pages past 2^31 bytes.  Oracle and bounds are those of test_gpu_kv."""

import pytest

from gpu_util import announce
from test_gpu_kv import Rig

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("heads, new", [((16, 1, 64), 4), ((16, 1, 128), 4), ((17, 1, 64), 3), ((12, 2, 128), 5), ((4, 4, 64), 1)])
def test_parts_joined_in_two_levels(heads, new):
    """From 9 parts on the joined parts are joined again; 16 to 64 rows."""
    announce(f"kv attend, parts {heads} {new}")
    lens = [4100, 33, 2500]
    r = Rig(lens, *heads, 64, "bf16" if new % 2 else "f16", "e4m3", seed=40)
    r.append(lens)
    r.attend([new, 1, new])
    r.attend([1, new, 0])
    r.attend([new, 1, new], window=1500, sinks=40)


@pytest.mark.parametrize("n", [63, 64, 65, 130])
def test_uneven_lengths_around_a_wave_of_sequences(n):
    announce(f"kv attend, {n} uneven sequences")
    lens = [1 + (97 * i * i) % 61 for i in range(n)]
    lens[n // 2], lens[n - 1] = 3000, 900
    r = Rig(lens, 2, 1, 64, 32, "f16", "int8", seed=41)
    r.append(lens)
    r.attend([1] * n)
    r.attend([min(lens[i], 70) if i % 9 == 4 or i == n - 1 else 0 for i in range(n)])


def test_more_pieces_than_workgroups():
    """600 sequences of 8 cached heads: a workgroup takes several pieces, and some of them are parts."""
    announce("kv attend, 600 sequences")
    lens = [1 + i % 37 for i in range(600)]
    lens[3], lens[299], lens[599] = 2000, 700, 1500
    r = Rig(lens, 8, 8, 64, 32, "f16", "e4m3", seed=42)
    r.append(lens)
    r.attend([1] * 600)


@pytest.mark.parametrize("heads", [(8, 1, 64), (2, 2, 128)])
def test_many_splits_of_a_tile(heads):
    """Few tiles of rows over many tokens: more splits than the joining kernel loads at once, the last one short."""
    announce(f"kv attend, splits {heads}")
    group = heads[0] // heads[1]
    rows = 72 // group if group > 1 else 70
    lens = [rows + 2801, 40]
    r = Rig(lens, *heads, 64, "bf16", "e4m3", seed=43)
    r.append(lens)
    r.attend([rows, 40])
    r.attend([rows, 3], window=700, sinks=5)


def test_pages_past_two_gib():
    announce("kv, pages past 2 GiB")
    r = Rig([300, 70, 90], 8, 8, 128, 64, "f16", "e4m3", seed=44, spare=40000)
    assert r.cache.k.numel() > 1 << 31 and int(r.cache.table.max()) * 8 * 64 * 128 > 1 << 31
    r.append([300, 70, 90])
    r.check_stored()
    r.attend([1, 1, 1])
    r.attend([80, 70, 3])
    r.cache.compact()
    assert int(r.cache.table.max()) == int((r.cache.refs > 0).sum()) - 1
    r.check_stored()
    r.attend([1, 2, 1])


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), -float("inf")])
@pytest.mark.parametrize("rows", [2, 90])
def test_a_query_that_is_not_finite_stays_alone(rows, bad):
    """One element of one query spoils its own output and no other's."""
    announce(f"kv attend, query {bad}, {rows} rows")
    r = Rig([400], 4, 2, 64, 32, "f16", "e4m3", seed=45)
    r.append([400])
    q = torch.from_numpy(1.5 * r.rng.standard_normal((rows, 4, 64))).half()
    spoiled = q.clone()
    spoiled[rows // 2, 1, 5] = bad
    out = torch.full((rows, 4, 64), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.empty(rows, 4, device="cuda")
    ids = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0], [0, rows])]
    r.cache.attend(0, spoiled.cuda(), out, *ids, rows, lse=lse)
    clean, clean_lse = torch.empty_like(out), torch.empty_like(lse)
    r.cache.attend(0, q.cuda(), clean, *ids, rows, lse=clean_lse)
    assert not bool(torch.isfinite(out[rows // 2, 1]).all())
    out[rows // 2, 1], lse[rows // 2, 1] = clean[rows // 2, 1], clean_lse[rows // 2, 1]
    r.compare(q, out, lse, [0, rows], [0], 0, 0, None)
