"""Attention of groups that share the beginning of their caches, on the GPU against the float64 oracle.

The bounds are those of test_gpu_kv.py: joining the shared tokens with the others adds two products and a sum to each of the
two sums, which (T + 16) 2^-24 there covers.  What is shared is compared with a look through the table on the host.
"""

import copy

import numpy as np
import pytest

from gpu_util import announce
from test_gpu_kv import DT, Rig, _ids

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Family(Rig):
    """Groups of sequences: the first of each stores the prefix, the others are forked from it, then each stores its own
    tokens.  prefixes[g] tokens, own[g] a list: tokens of each member of group g behind the prefix."""

    def __init__(self, prefixes, own, heads, kv_heads, dim, page, act="f16", code="e4m3", seed=0, layers=1, layer=0):
        self.members = [len(o) for o in own]
        n = sum(self.members)
        flat = [t for o in own for t in o]
        whole = [p for p, o in zip(prefixes, own) for _ in o]
        width = max(-(-(a + b) // page) for a, b in zip(whole, flat)) + 2
        super().__init__([0] * n, heads, kv_heads, dim, page, act, code, seed, layers, layer, spare=n * width)
        import activation_sparse_decode_relu_amd as pi
        self.page = page
        pool = sum(-(-p // page) for p in prefixes) + sum(-(-t // page) + 3 for t in flat)
        self.cache = pi.KVCache(heads, kv_heads, dim, pool, page, n, width, act_dtype=act, code=code, layers=layers)
        for name in ("k", "v", "k_exp", "v_exp"):
            getattr(self.cache, name).fill_(255)
        first = np.concatenate([[0], np.cumsum(self.members)]).tolist()
        self.groups = first
        leaders = [first[g] for g in range(len(own))]
        self.grow(prefixes, leaders)
        for g, lead in enumerate(leaders):
            rest = list(range(lead + 1, first[g + 1]))
            if rest:
                self.cache.fork(_ids([lead] * len(rest)), _ids(rest))
            for s in rest:
                self.k[s], self.v[s] = copy.deepcopy(self.k[lead]), copy.deepcopy(self.v[lead])
        self.grow(flat, list(range(n)))

    def grow(self, counts, seqs):
        """The next counts[i] tokens of seqs[i], stored on the rig's layer."""
        self.cache.reserve(_ids(seqs), _ids(counts))
        self.cache.check_failed()
        k, v = self.tokens(sum(counts), self.kvh), self.tokens(sum(counts), self.kvh, 0.5)
        starts = np.concatenate([[0], np.cumsum(counts)])
        for i, s in enumerate(seqs):
            self.k[s].append(k[starts[i]:starts[i + 1]].double().numpy())
            self.v[s].append(v[starts[i]:starts[i + 1]].double().numpy())
        if sum(counts):
            self.cache.append(self.layer, k.cuda(), v.cuda(), _ids(seqs), _ids(starts))

    def shared(self, seqs, counts, groups):
        """What each group shares, from the table."""
        table, lens = self.cache.table.tolist(), self.cache.lens.tolist()
        got = []
        for g in range(len(groups) - 1):
            mine = list(range(groups[g], groups[g + 1]))
            limit = max(min([lens[seqs[i]] - counts[i] for i in mine]), 0) if len(mine) > 1 else 0
            cols = 0
            while cols * self.page < limit and len({table[seqs[i]][cols] for i in mine}) == 1:
                cols += 1
            got.append(min(limit, cols * self.page) // 32 * 32)
        return got

    def step(self, counts, groups=None, seqs=None, state=None, scale=None, q=None, max_rows=None):
        """attend_shared of the last counts[i] tokens of seqs[i]; returns what the plan says."""
        seqs = list(range(self.n)) if seqs is None else seqs
        groups = self.groups if groups is None else groups
        total, starts = sum(counts), np.concatenate([[0], np.cumsum(counts)])
        if q is None:
            q = torch.from_numpy(1.5 * self.rng.standard_normal((total, self.heads, self.dim))).to(DT[self.act])
        out = torch.full((total, self.heads, self.dim), float("nan"), dtype=DT[self.act], device="cuda")
        lse = torch.full((total, self.heads), float("nan"), device="cuda")
        plan = torch.full((len(groups) - 1 + len(seqs),), -9, dtype=torch.int32, device="cuda")
        ids = _ids(seqs), _ids(starts), _ids(groups)
        self.cache.share(*ids, plan)
        most = max(starts[groups[g + 1]] - starts[groups[g]] for g in range(len(groups) - 1))
        self.cache.attend_shared(self.layer, q.cuda(), out, *ids, plan, max(counts), int(max_rows or most), scale, lse, state)
        torch.cuda.synchronize()
        want = self.shared(seqs, counts, groups)
        plan = plan.tolist()
        assert plan[:len(want)] == want
        assert plan[len(want):] == [w for g, w in enumerate(want) for _ in range(groups[g + 1] - groups[g])]
        self.compare(q, out, lse, starts, seqs, 0, 0, scale)
        return want


@pytest.mark.parametrize("heads", [(8, 2, 128), (16, 2, 64), (4, 4, 128), (3, 3, 64), (32, 1, 64)])
@pytest.mark.parametrize("act, code", [("f16", "e4m3"), ("bf16", "int8"), ("f16", "int8"), ("bf16", "e4m3")])
def test_groups_of_several_sizes(act, code, heads):
    announce(f"shared groups {act} {code} {heads}")
    f = Family([300, 64, 33, 700], [[5, 1, 40, 0], [70], [2, 2], [1, 100, 33]], *heads, 32, act, code, seed=1)
    n = f.n
    f.grow([1] * n, list(range(n)))
    assert f.step([1] * n)[3] == 672
    f.grow([3, 0, 2, 1, 4, 1, 0, 0, 2, 3][:n], list(range(n)))
    f.step([3, 0, 2, 1, 4, 1, 0, 0, 2, 3][:n])


@pytest.mark.parametrize("members", [2, 3, 4, 5, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("heads", [(8, 1, 128), (8, 1, 64), (6, 2, 128), (2, 2, 64)])
def test_rows_of_a_group(members, heads):
    """From few rows of a cached head to many: both kernels, and each number of row tiles."""
    announce(f"shared members {members} {heads}")
    f = Family([500], [[(7 * i) % 50 + 1 for i in range(members)]], *heads, 64, "f16", "e4m3", seed=members)
    f.step([1] * members)


@pytest.mark.parametrize("new", [2, 5, 9, 20, 70])
@pytest.mark.parametrize("heads", [(8, 1, 128), (16, 2, 64), (4, 4, 64)])
def test_several_new_tokens(new, heads):
    """Guessed tokens, and pieces of prompts behind a shared one: own tokens through both kernels."""
    announce(f"shared new {new} {heads}")
    f = Family([200, 96], [[new, new + 30, 100], [new + 1, new]], *heads, 32, "bf16", "int8", seed=new)
    f.step([new] * 5)
    f.step([1, new, max(new // 2, 1), 0, new])


@pytest.mark.parametrize("members, heads", [(2, (4, 1, 64)), (3, (16, 1, 128)), (20, (8, 1, 128)), (6, (4, 2, 64))])
def test_long_prefixes(members, heads):
    """Cut into pieces whose parts are joined."""
    announce(f"shared long {members} {heads}")
    f = Family([9000], [[(31 * i) % 700 + 1 for i in range(members)]], *heads, 128, "f16", "e4m3", seed=3)
    f.step([1] * members)


def test_long_own_tokens():
    announce("shared, long own tokens")
    f = Family([100], [[6000, 1, 3000]], 4, 1, 64, 64, "f16", "e4m3", seed=4)
    f.step([1] * 3)
    f = Family([100], [[3000, 90]], 16, 2, 64, 64, "f16", "int8", seed=4)
    f.step([80, 80])


def test_many_groups_and_sequences():
    """More groups, and more sequences, than a wave has lanes."""
    announce("shared, many groups")
    rng = np.random.default_rng(5)
    own = [rng.integers(1, 40, rng.integers(1, 4)).tolist() for _ in range(90)]
    f = Family(rng.integers(0, 150, 90).tolist(), own, 2, 1, 64, 32, "f16", "e4m3", seed=5)
    f.step([1] * f.n)
    f.step([min(i % 3, own_tokens) for i, own_tokens in enumerate(t for o in own for t in o)])


def test_many_rows_of_many_groups():
    """The kernel of many rows with more than 64 items of both kinds."""
    announce("shared, many rows of many groups")
    f = Family([64] * 70, [[20, 20]] * 70, 16, 1, 64, 32, "bf16", "e4m3", seed=6)
    f.step([9] * f.n)


@pytest.mark.parametrize("page", [32, 64, 256])
def test_prefixes_that_end_anywhere(page):
    announce(f"shared ends, pages of {page}")
    for prefix in (0, 1, 31, 32, 33, page - 1, page, page + 1, 3 * page, 3 * page + 17):
        f = Family([prefix], [[3, 1, 2]], 4, 2, 64, page, "f16", "e4m3", seed=prefix)
        assert f.step([1, 1, 1])[0] == prefix // page * page


def test_nothing_of_their_own():
    """Forks that have not grown: the last shared page is shared as a whole, and the new tokens end the sharing."""
    announce("shared, forks as they are")
    f = Family([100], [[0, 0, 0]], 4, 2, 64, 64, "f16", "e4m3", seed=7)
    assert f.step([1, 1, 1])[0] == 96
    assert f.step([40, 1, 0])[0] == 32       # the first one's rows begin at token 60


def test_tables_that_differ():
    """Sharing ends at the first page that differs or is none, whatever comes after it."""
    announce("shared, tables that differ")
    f = Family([640, 640], [[5, 5], [5, 5, 5]], 4, 2, 64, 64, "f16", "e4m3", seed=8)
    assert f.step([1] * 5) == [640, 640]
    table = f.cache.table.clone()
    spare = int((f.cache.refs == 0).nonzero()[0])
    page = int(table[1, 4])
    for name in ("k", "v", "k_exp", "v_exp"):    # sequence 1's fifth page is a copy
        t = getattr(f.cache, name)
        t[:, spare] = t[:, page]
    f.cache.table[1, 4] = spare
    assert f.step([1] * 5) == [256, 640]
    f.cache.table.copy_(table)
    # groups across the families: pages differ from the first on; and a group in another order
    assert f.step([1] * 5, groups=[0, 1, 3, 5]) == [0, 0, 640]
    assert f.step([1] * 5, seqs=[4, 0, 2, 3, 1], groups=[0, 1, 2, 4, 5]) == [0, 0, 640, 0]


def test_sequences_that_hold_little():
    """A member shorter than what the others share, one that holds nothing, one of fewer tokens than rows."""
    announce("shared, short members")
    f = Family([320], [[5, 5, 5, 5]], 4, 2, 64, 32, "f16", "e4m3", seed=9)
    for cut in (200, 33, 1):
        f.cache.lens[2] = cut
        for m in (f.k[2], f.v[2]):
            m.values = m.values[:cut]
        assert f.step([1] * 4)[0] == (cut - 1) // 32 * 32
    f.step([1, 1, 3, 1])                          # two rows before the first token: zeros
    f.cache.lens[2] = 0
    for m in (f.k[2], f.v[2]):
        m.values = m.values[:0]
    assert f.step([1, 1, 2, 1])[0] == 0


def test_bad_numbers_and_plans():
    """Sequences and groups out of range, and a plan of nonsense, leave the other groups' rows right and touch nothing else."""
    announce("shared, bad numbers")
    f = Family([128, 128], [[9, 9], [9, 9, 9]], 4, 2, 64, 32, "f16", "e4m3", seed=10)
    q = torch.randn(6, 4, 64).half().cuda()
    lse = torch.empty(6, 4, device="cuda")
    for plan, seqs, groups in (([128, 1 << 30, 128, 128, -5, 33, 1 << 20], [0, 1, 2, 3, 4], [0, 2, 5]),
                               ([128, 0, 128, 128, 0, 0, 0], [0, 1, -3, 77, 4], [0, 2, 5]),
                               ([128, 64, 128, 128, 64, 64, 64], [0, 1, 2, 3, 4], [0, 2, 99])):
        out = torch.full((6, 4, 64), 7.0, dtype=torch.float16, device="cuda")
        before = {name: getattr(f.cache, name).clone() for name in ("k", "v", "table", "lens", "refs")}
        f.cache.attend_shared(0, q, out, _ids(seqs), _ids([0, 1, 2, 3, 4, 5]), _ids(groups), _ids(plan), 1, 3, lse=lse)
        torch.cuda.synchronize()
        f.compare(q[:2].cpu(), out[:2], lse[:2], [0, 1, 2], [0, 1], 0, 0, None)
        assert bool((out[5] == 7).all())          # a row of no sequence
        for name, t in before.items():
            assert torch.equal(t, getattr(f.cache, name))
    plan = torch.zeros(7, dtype=torch.int32, device="cuda")
    f.cache.share(_ids([0, 1, -3, 77, 4]), _ids([0, 1, 2, 3, 4, 5]), _ids([0, 2, 5]), plan)
    assert plan.tolist() == [128, 0, 128, 128, 0, 0, 0]
    f.cache.share(_ids([0, 1, 2, 3, 4]), _ids([0, 1, 2, 3, 4, 5]), _ids([1, 2, 4]), plan)     # 0 and 4 in no group
    assert plan.tolist() == [0, 128, 0, 0, 128, 128, 0]


@pytest.mark.parametrize("scale", [None, 2.0, 1e-4])
@pytest.mark.parametrize("loud", ["prefix", "own"])
def test_scores_far_apart(scale, loud):
    """One part's scores are far above the other's: its weight vanishes beside it."""
    announce(f"shared scores {scale} {loud}")
    f = Family([96], [[40, 40, 40]], 4, 2, 64, 32, "bf16", "e4m3", seed=11)
    f.step([1, 1, 1], scale=scale)
    big = Family([96], [[0, 0]], 2, 1, 64, 32, "bf16", "e4m3", seed=12)
    tokens = big.tokens

    def louder(count, heads, spread=1.0):
        return tokens(count, heads, spread) * (30.0 if loud == "own" and spread == 1.0 else 1.0 if spread == 1.0 else 2.0 ** -20)
    big.tokens = louder
    big.grow([10, 50], [0, 1])
    big.step([2, 1], scale=scale)


def test_strides_state_and_no_lse():
    announce("shared strides")
    f = Family([200], [[9, 30, 9]], 8, 2, 64, 64, "f16", "e4m3", seed=13)
    qkv = torch.randn(3, 12, 64).half().cuda()
    ids = _ids([0, 1, 2]), _ids([0, 1, 2, 3]), _ids([0, 3])
    plan = torch.empty(4, dtype=torch.int32, device="cuda")
    f.cache.share(*ids, plan)
    want, lse = torch.empty(3, 8, 64, dtype=torch.float16, device="cuda"), torch.empty(3, 8, device="cuda")
    f.cache.attend_shared(0, qkv[:, :8].contiguous(), want, *ids, plan, 1, 3, lse=lse)
    need = f.cache.state_floats(3)
    state = torch.full((need + 4,), float("nan"), device="cuda")
    out = torch.full((8, 4, 64), 7.0, dtype=torch.float16, device="cuda").transpose(0, 1)
    f.cache.attend_shared(0, qkv[:, :8], out[:3], *ids, plan, 1, 3, state=state)
    assert torch.equal(out[:3], want) and bool((out[3] == 7).all()) and bool(state[-4:].isnan().all())
    f.compare(qkv[:, :8].cpu(), want, lse, [0, 1, 2, 3], [0, 1, 2], 0, 0, None)
    import activation_sparse_decode_relu_amd as pi
    with pytest.raises(pi.PiError) as e:
        f.cache.attend_shared(0, qkv[:, :8], out[:3], *ids, plan, 1, 3, state=state[:100])
    assert e.value.status == 2
    with pytest.raises(pi.PiError):
        f.cache.attend_shared(0, qkv[:, :8], out[:3], *ids, plan, 1, 3, state=state.half())


def test_layers():
    """A plan holds for every layer; each layer's pages are its own."""
    announce("shared layers")
    f = Family([100], [[3, 40]], 4, 2, 64, 32, "f16", "e4m3", seed=14, layers=3, layer=2)
    f.step([1, 2])


def test_same_bits_whoever_is_last():
    announce("shared bits")
    f = Family([5000], [[(37 * i) % 300 + 1 for i in range(12)]], 8, 1, 64, 64, "f16", "e4m3", seed=15)
    q = torch.randn(12, 8, 64).half().cuda()
    ids = _ids(range(12)), _ids(range(13)), _ids([0, 12])
    plan = torch.empty(13, dtype=torch.int32, device="cuda")
    f.cache.share(*ids, plan)
    outs = []
    for _ in range(6):
        out = torch.empty(12, 8, 64, dtype=torch.float16, device="cuda")
        f.cache.attend_shared(0, q, out, *ids, plan, 1, 12)
        outs.append(out)
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("members, heads", [(4, (4, 2, 64)), (30, (8, 2, 64))])
def test_steps_in_a_graph(members, heads):
    """reserve, rotate, append, share and attend_shared as one graph: every replay gives the eager step's bits."""
    announce(f"shared graph {members}")
    import activation_sparse_decode_relu_amd as pi
    rope = pi.Rope(64)
    runs = []
    for captured in (False, True):
        f = Family([150], [[1 + i % 5 for i in range(members)]], *heads, 32, "f16", "e4m3", seed=16)
        h, kvh, dim = heads
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        data = torch.randn(8, members, h + 2 * kvh, dim, device="cuda", generator=g).half()
        t = torch.zeros(members, h + 2 * kvh, dim, dtype=torch.float16, device="cuda")
        out = torch.zeros(members, h, dim, dtype=torch.float16, device="cuda")
        seqs, starts, groups, one = _ids(range(members)), _ids(range(members + 1)), _ids([0, members]), _ids([1] * members)
        plan = torch.zeros(1 + members, dtype=torch.int32, device="cuda")

        def step():
            q, k, v = t[:, :h], t[:, h:h + kvh], t[:, h + kvh:]
            f.cache.reserve(seqs, one)
            f.cache.share(seqs, starts, groups, plan)
            f.cache.rotate(rope, q, q, k, k, seqs, starts)
            f.cache.append(0, k, v, seqs, starts)
            f.cache.attend_shared(0, q, out, seqs, starts, groups, plan, 1, members)

        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph() if captured else None
        if captured:
            with torch.cuda.graph(graph):
                step()
        got = []
        for i in range(8):
            t.copy_(data[i])
            graph.replay() if captured else step()
            torch.cuda.synchronize()
            got.append((out.clone(), plan.clone()))
        f.cache.check_failed()
        runs.append(got)
    for i, (a, b) in enumerate(zip(*runs)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), f"step {i}"
    assert runs[0][-1][1].tolist() == [128] * (members + 1)


def test_another_stream():
    announce("shared stream")
    f = Family([300], [[7, 9, 20]], 4, 2, 64, 32, "f16", "e4m3", seed=17)
    q = torch.randn(3, 4, 64).half().cuda()
    ids = _ids([0, 1, 2]), _ids([0, 1, 2, 3]), _ids([0, 3])
    outs = []
    torch.cuda.synchronize()
    for stream in (None, torch.cuda.Stream()):
        plan, out = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty_like(q)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        f.cache.share(*ids, plan, stream=stream)
        f.cache.attend_shared(0, q, out, *ids, plan, 1, 3, stream=stream)
        torch.cuda.synchronize()
        outs.append(out)
    assert torch.equal(*outs)


@pytest.mark.parametrize("times", [1, 10])
@pytest.mark.parametrize("order", [1, -1])
def test_rows_that_fill_tiles(times, order):
    """Groups whose rows end at, before and behind 128 of them, or that have none: up to 64 groups and more."""
    announce(f"shared, rows that fill tiles, {times} times, {order}")
    counts = [(64, 63), (64, 64), (65, 64), (0, 0), (128, 127), (128, 128), (128, 129), (0, 0), (0, 0), (66, 0), (0, 1)][::order] * times
    f = Family([64] * len(counts), [[max(c, 1) for c in pair] for pair in counts], 1, 1, 64, 32, "f16", "e4m3", seed=7)
    f.step([c for pair in counts for c in pair])


def test_no_rows():
    announce("shared, no rows")
    f = Family([64], [[1, 1]], 4, 2, 64, 32)
    assert f.cache.state_floats(0) == 0
    f.cache.share(_ids([0, 1]), _ids([0, 0, 0]), _ids([0, 2]), plan := torch.zeros(3, dtype=torch.int32, device="cuda"))
    q = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    f.cache.attend_shared(0, q, q.clone(), _ids([0, 1]), _ids([0, 0, 0]), _ids([0, 2]), plan, 0, 0)
    torch.cuda.synchronize()
    assert plan.tolist() == [64, 64, 64]


@pytest.mark.parametrize("new", [1, 70])
def test_plan_past_a_full_sequence(new):
    """A plan that says more than a sequence which fills its row of the table holds: the other group's rows are right."""
    announce(f"shared, plan past a full sequence, {new} new")
    f = Family([96, 96], [[new, new], [new, new]], 4, 2, 64, 32, "f16", "e4m3", seed=18)
    f.cache.lens[2:] = f.cache.table.shape[1] * 32
    before = {name: getattr(f.cache, name).clone() for name in ("k", "v", "table", "lens", "refs")}
    q = torch.randn(4 * new, 4, 64).half()
    out, lse = torch.empty(4 * new, 4, 64, dtype=torch.float16, device="cuda"), torch.empty(4 * new, 4, device="cuda")
    for much in (1 << 20, 0x7fffffff):
        f.cache.attend_shared(0, q.cuda(), out, _ids(range(4)), _ids(range(0, 4 * new + 1, new)), _ids([0, 2, 4]),
                              _ids([96, much, 96, 96, much, much]), new, 2 * new, lse=lse)
        torch.cuda.synchronize()
        f.compare(q[:2 * new], out[:2 * new], lse[:2 * new], [0, new, 2 * new], [0, 1], 0, 0, None)
        for name, t in before.items():
            assert torch.equal(t, getattr(f.cache, name))


@pytest.mark.parametrize("act, code", [("f16", "e4m3"), ("bf16", "int8"), ("bf16", "e4m3"), ("f16", "int8")])
@pytest.mark.parametrize("groups, members, new, heads", [
    (1, 3, 5, (8, 1, 128)),     # shared tokens in parts, joined by a launch: 120 rows of a head, 40 own
    (2, 4, 9, (16, 2, 128)),    # the same with several heads, 72 own rows: the kernel of many rows behind it
    (1, 5, 3, (8, 1, 128)),     # 24 own rows, which join the parts themselves
    (2, 2, 4, (8, 2, 128)),     # 32 and 16 rows
    (1, 2, 2, (16, 2, 128)),    # 32 rows, and 16 own
    (4, 2, 6, (64, 8, 128)),    # 48 own rows of 64 items
    (8, 2, 3, (64, 8, 128)),    # 48 rows of 64 groups' heads, and 24 own
    (8, 4, 2, (64, 8, 128)),    # 64 rows, and 16 own
    (8, 1, 8, (64, 8, 128))])   # lone sequences: 64 rows, nothing shared
def test_wide_heads(groups, members, new, heads, act, code):
    """128 dims, each number of row tiles on both sides, over prefixes that are cut."""
    announce(f"shared wide {groups} x {members}, {new} new, {heads} {act} {code}")
    f = Family([2500 - 300 * g for g in range(groups)], [[new + (13 * i + 5 * g) % 90 for i in range(members)] for g in range(groups)],
               *heads, 64, act, code, seed=new)
    f.step([new] * f.n)
    if new > 2:
        f.step([1 + (i % new) for i in range(f.n - 1)] + [new])
