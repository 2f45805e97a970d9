"""The cache's calls at the edges of what they take: states only the device knows, and values at the ends of their types.
Oracle and bounds are those of test_gpu_kv unless a test says otherwise."""

import numpy as np
import pytest

import oracle

from gpu_util import announce
from test_gpu_kv import DT, EPS, Rig, _f64, _ids

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# ---- values at the ends of their types -------------------------------------------------------------------


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("heads", [(2, 2, 64), (8, 1, 128)])
def test_the_largest_values_give_finite_outputs(act, code, heads):
    """The type's largest value is stored as the next power of two, past the type: outputs are held to its finite
    range, as read's are.  A mean of one value is that value, up to 2^-10 of it, and rounds or is held to the same number."""
    announce(f"kv attend, largest values {act} {code} {heads}")
    top = torch.finfo(DT[act]).max
    n = 700
    r = Rig([n, 40], *heads, 64, act, code, seed=50)
    v = [r.tokens(c, heads[1], 0.5) for c in (n, 40)]
    v = torch.cat(v)
    v[:, :, 3], v[:, :, 17] = top, -top
    v[:, :, 40] = float("inf")
    r.append([n, 40], v=v)
    r.check_stored()
    for counts in ([1, 1], [6, 3], [130, 40]):
        total = sum(counts)
        q = r.tokens(total, heads[0]).cuda()
        out = torch.full((total, heads[0], heads[2]), float("nan"), dtype=DT[act], device="cuda")
        starts = _ids([0, counts[0], total])
        r.cache.attend(0, q, out, _ids([0, 1]), starts, max(counts))
        assert bool(torch.isfinite(out).all())
        assert bool((out[:, :, 3] == top).all()) and bool((out[:, :, 17] == -top).all()) and bool((out[:, :, 40] == top).all())


# ---- states that only the device knows -------------------------------------------------------------------


@pytest.mark.parametrize("first", [-1, -31, -32, -33, -70, -(1 << 31), (1 << 31) - 1])
def test_read_from_before_the_first_token(first):
    """Tokens before the first are not there: they read as 0, and no row is left out."""
    announce(f"kv read from {first}")
    r = Rig([100, 70], 2, 2, 64, 32, seed=51)
    r.append([100, 70])
    got = [torch.full((140, 2, 64), 7.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    r.cache.read(0, got[0], got[1], _ids([1, 0]), _ids([0, 75, 140]), first=_ids([first, 95]))
    for t, models in ((got[0], r.k), (got[1], r.v)):
        want = np.zeros((140, 2, 64))
        for row in range(75):
            if 0 <= first + row < 70:
                want[row] = models[1].values[first + row]
        want[75:80] = models[0].values[95:100]
        assert np.array_equal(_f64(t), want)


@pytest.mark.parametrize("length", [-1, -(1 << 31), 129, 1 << 20, (1 << 31) - 1])
def test_a_length_out_of_range_is_no_length(length):
    """Lengths below 0 or past the table's columns (4 pages of 32 here) read as nothing and write nothing."""
    announce(f"kv, a length of {length}")
    r = Rig([70, 90], 8, 2, 64, 32, seed=52)
    r.append([70, 90])
    assert r.cache.table.shape[1] * 32 == 128
    r.cache.table[0] = torch.tensor([0, 1, 2, 3], dtype=torch.int32)   # pages in every column, whosever they are
    r.cache.lens[0] = length
    bytes_before = [getattr(r.cache, n).clone() for n in ("k", "v", "k_exp", "v_exp")]
    t = r.tokens(3, 2).cuda()
    r.cache.append(0, t, t, _ids([0]), _ids([0, 3]))
    for n, old in zip(("k", "v", "k_exp", "v_exp"), bytes_before):
        assert torch.equal(getattr(r.cache, n), old), n
    got = [torch.full((128, 2, 64), 7.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    r.cache.read(0, got[0], got[1], _ids([0]), _ids([0, 128]))
    assert not bool(got[0].any()) and not bool(got[1].any())
    for rows in (2, 40):
        q = r.tokens(rows, 8).cuda()
        out = torch.full((rows, 8, 64), float("nan"), dtype=torch.float16, device="cuda")
        lse = torch.zeros(rows, 8, device="cuda")
        r.cache.attend(0, q, out, _ids([0]), _ids([0, rows]), rows, lse=lse)
        assert bool((out == 0).all()) and bool((lse == -float("inf")).all())


# ---- blocks of V far smaller than others -----------------------------------------------------------------


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("nats", [16, 24, 32, 40, 48])
@pytest.mark.parametrize("heads, rows", [((4, 1, 64), 1), ((8, 1, 64), 7), ((8, 1, 64), 9), ((2, 2, 128), 70)])
def test_a_tiny_block_with_a_large_score(code, nats, heads, rows):
    """One token's V is 1 and its score 0; a later block's V is 2^-100 and one of its scores `nats`.  The output is the
    first token's share, e^-nats, far above what the tiny block adds.  Bound: that of test_gpu_kv, its floor 2^-30 a token of
    the row's own largest term (never more than mass)."""
    announce(f"kv attend, tiny block {code} {nats} {heads} {rows}")
    n = 160 + rows
    r = Rig([n], *heads, 64, "bf16", code, seed=53)
    k, v = torch.zeros(n, heads[1], heads[2]), torch.zeros(n, heads[1], heads[2])
    v[0] = 1.0
    v[128:160] = 2.0 ** -100
    k[130, :, 0] = nats                                # exact in both codes
    r.append([n], k=k.bfloat16(), v=v.bfloat16())
    r.check_stored()
    q = torch.zeros(rows, heads[0], heads[2])
    q[..., 0] = 1.0
    q = q.bfloat16()
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(rows, heads[0], device="cuda")
    r.cache.attend(0, q.cuda(), out, _ids([0]), _ids([0, rows]), rows, scale=1.0, lse=lse)
    ref, ref_lse, mass, reach = oracle.kv_attend(_f64(q), r.k[0].values, r.v[0].values, scale=1.0)
    dx = reach * ((heads[2] + 4) * 2.0 ** -24 + 2.0 ** -23)
    rel = np.expm1(2 * dx) + (n + 16) * 2.0 ** -24 + 2.0 ** -11 + n * 2.0 ** -30
    assert np.all(np.abs(_f64(out) - ref) <= rel[..., None] * mass + EPS["bf16"] * np.abs(ref))
    assert np.all(np.abs(_f64(lse) - ref_lse) <= dx + (n + 16) * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(ref_lse)))


# ---- what a table may hold, and what it holds ------------------------------------------------------------


@pytest.mark.parametrize("window, sinks", [(0, 0), (50, 2), ((1 << 31) - 1, (1 << 31) - 1)])
def test_a_table_far_larger_than_its_sequences(window, sinks):
    """9 sequences on 8 cached heads with room for 2^30 tokens each: what they hold decides, not what the table could."""
    import activation_sparse_decode_relu_amd as pi
    announce(f"kv attend, a table of 2^30 tokens, window {window}")
    lens = [1, 5000, 33, 64, 100, 7, 300, 31, 4097]
    r = Rig(lens, 8, 8, 64, 4096, seed=54)
    own = {name: getattr(r.cache, name) for name in ("k", "v", "k_exp", "v_exp", "lens", "refs")}
    narrow = r.cache.table
    r.cache = pi.KVCache(8, 8, 64, r.cache.desc.pages, 4096, len(lens), 1 << 18, buffers=own)
    r.cache.table[:, :narrow.shape[1]] = narrow
    r.append(lens)
    r.attend([1] * 9, window, sinks)
    r.attend([1, 5, 0, 2, 1, 1, 70, 3, 1], window, sinks)


# ---- streams ---------------------------------------------------------------------------------------------


@pytest.mark.parametrize("named", [True, False])
def test_a_cache_dropped_while_another_stream_works(named):
    """The pages stay reserved until that stream is past its calls, whether it is named or is the current one."""
    import activation_sparse_decode_relu_amd as pi
    announce("kv, a cache dropped early")
    side = torch.cuda.Stream()
    c = pi.KVCache(4, 4, 64, 400, 32, 4, 100)
    ids, counts = _ids(range(4)), _ids([3000] * 4)
    c.reserve(ids, counts)
    size = c.k.numel()
    x = torch.randn(12000, 4, 64, device="cuda").half()
    starts = _ids(range(0, 12001, 3000))
    c.append(0, x, x, ids, starts)
    q, one = torch.randn(4, 4, 64, device="cuda").half(), _ids(range(5))
    want, got = torch.empty_like(q), torch.empty_like(q)
    c.attend(0, q, want, ids, one, 1)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)                   # cycles: some 25 ms before the call's turn
        if not named:
            c.attend(0, q, got, ids, one, 1)
    if named:
        c.attend(0, q, got, ids, one, 1, stream=side)
    del c
    torch.full((size,), 255, dtype=torch.uint8, device="cuda")   # takes any memory of that size that is free
    side.synchronize()
    assert torch.equal(got, want)


def test_a_cache_made_on_a_stream_is_empty_there():
    """The buffers a cache makes for itself are set before the given stream's first call, however late the current one is."""
    import activation_sparse_decode_relu_amd as pi
    announce("kv create on another stream")
    side = torch.cuda.Stream()
    ids, counts = _ids([0, 2]), _ids([40, 33])
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                      # cycles: some 50 ms before the current stream gets to the fills
    c = pi.KVCache(2, 1, 64, 6, 32, 3, 4, stream=side)
    c.reserve(ids, counts, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert c.lens.tolist() == [40, 0, 33] and c.refs.tolist() == [1, 1, 1, 1, 0, 0]
    assert c.table.tolist() == [[0, 1, -1, -1], [-1] * 4, [2, 3, -1, -1]] and int(c.failed.item()) == 0


# ---- more blocks than a wave has lanes -------------------------------------------------------------------
# A wave looks up the pages of 64 blocks at a time, a lane each.


def test_a_whole_prompt_past_a_waves_blocks():
    """Tile attention with no split: workgroups that pass over up to 136 blocks look pages up three times, and the last
    time for part of a wave."""
    announce("kv attend, prompt of 4330")
    n, heads = 4330, 8
    r = Rig([n], heads, heads, 64, 32, "bf16", "e4m3", seed=55)
    r.append([n])
    # 34 tiles of rows on 8 heads: with n = 1 that is 272 items, past the 256 from which tokens are not split
    q = torch.from_numpy(1.5 * r.rng.standard_normal((n, heads, 64))).bfloat16()
    out = torch.full((n, heads, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(n, heads, device="cuda")
    r.cache.attend(0, q.cuda(), out, _ids([0]), _ids([0, n]), n, lse=lse)
    torch.cuda.synchronize()
    for a, b in ((0, 40), (2040, 2060), (2170, 2180), (4090, 4110), (4290, 4330)):   # the oracle's loops are slow: some rows
        ref, ref_lse, mass, reach = oracle.kv_attend(_f64(q[a:b]), r.k[0].values[:b], r.v[0].values[:b])
        dx = reach * (68 * 2.0 ** -24 + 2.0 ** -23)
        rel = np.expm1(2 * dx) + (n + 16) * 2.0 ** -24 + 2.0 ** -11
        tol = rel[..., None] * mass + EPS["bf16"] * np.abs(ref) + 2.0 ** -30 * n * np.abs(r.v[0].values).max()
        assert np.all(np.abs(_f64(out[a:b]) - ref) <= tol), f"rows {a} to {b}"
        assert np.all(np.abs(_f64(lse[a:b]) - ref_lse) <= dx + (n + 16) * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(ref_lse)))


@pytest.mark.parametrize("heads, new, n, length", [((33, 1, 128), 1, 64, 35000), ((1, 1, 64), 1, 96, 80000)])
def test_steps_past_a_waves_blocks(heads, new, n, length):
    """Step attention in pieces of more than 256 blocks, four waves each: every wave looks pages up more than once, and the
    last time for part of a wave.  The sequences share the pages of the first (forks), so the cache stays small; three of
    them are compared."""
    announce(f"kv attend, pieces past a wave's blocks {heads} {n} x {length}")
    import activation_sparse_decode_relu_amd as pi
    page = 128
    lens = [length - 7 * i for i in range(n)]
    r = Rig([length], *heads, page, "f16", "e4m3", seed=56)
    r.append([length])
    own = {name: getattr(r.cache, name) for name in ("k", "v", "k_exp", "v_exp")}
    wide = pi.KVCache(*heads, r.cache.desc.pages, page, n, r.cache.table.shape[1], buffers=own)
    wide.table.copy_(r.cache.table.expand(n, -1))
    wide.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    q = torch.from_numpy(1.5 * r.rng.standard_normal((n * new, heads[0], heads[2]))).half()
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    lse = torch.empty(n * new, heads[0], device="cuda")
    wide.attend(0, q.cuda(), out, _ids(range(n)), _ids(range(0, n * new + 1, new)), new, lse=lse)
    torch.cuda.synchronize()
    k, v = list(r.k), list(r.v)
    for i in (0, n // 2, n - 1):
        for models, full in ((r.k, k), (r.v, v)):
            m = oracle.KvModel(heads[1], heads[2], "e4m3", "f16")
            m.values = full[0].values[:lens[i]]
            models[0] = m
        a, b = i * new, (i + 1) * new
        r.compare(q[a:b], out[a:b], lse[a:b], [0, b - a], [0], 0, 0, None)
