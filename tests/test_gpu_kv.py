"""The attention cache on the GPU against the float64 oracle: what is stored, attention, and the pages.

Bounds.  Stored values are exact, so read() has to match bit for bit.  Attention: a score is a sum of
head_dim products in fp32, off by at most (head_dim + 4) 2^-24 of scale * sum |q k| (plus its own
rounding, 2^-23 of it), which enters exp and the logarithm as it is; exp2 and the sums of T tokens
add (T + 16) 2^-24; the products with V take exp() rounded to fp16, 2^-11 of each term, with a floor of
2^-30 of the row's largest term; the output is rounded once (half a step of its type).
"""

import numpy as np
import pytest

import oracle

from gpu_util import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}      # half a step, relative
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}   # half the smallest step


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _ids(values):
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


def _f64(t):
    return t.double().cpu().numpy()


class Rig:
    """A cache with its oracle: sequences of given lengths on pages in a shuffled order."""

    def __init__(self, lens, heads, kv_heads, dim, page, act="f16", code="e4m3", seed=0, layers=1, layer=0, spare=3):
        import activation_sparse_decode_relu_amd as pi
        self.rng = np.random.default_rng(seed)
        self.n, self.heads, self.kvh, self.dim, self.act, self.code, self.layer = len(lens), heads, kv_heads, dim, act, code, layer
        width = max(max(-(-t // page) for t in lens), 1) + 1
        pool = sum(-(-t // page) for t in lens) + spare
        self.cache = pi.KVCache(heads, kv_heads, dim, pool, page, self.n, width, act_dtype=act, code=code, layers=layers)
        for name in ("k", "v", "k_exp", "v_exp"):   # memory as it comes: every code a NaN, every exponent the largest
            getattr(self.cache, name).fill_(255)
        order = self.rng.permutation(pool)[:pool - spare].tolist()
        table = np.full((self.n, width), -1, dtype=np.int32)
        for i, t in enumerate(lens):
            for j in range(-(-t // page)):
                table[i, j] = order.pop()
                self.cache.refs[int(table[i, j])] = 1
        self.cache.table.copy_(torch.from_numpy(table))
        self.k = [oracle.KvModel(kv_heads, dim, code, act) for _ in lens]
        self.v = [oracle.KvModel(kv_heads, dim, code, act) for _ in lens]

    def tokens(self, count, heads, spread=1.0):
        x = self.rng.standard_normal((count, heads, self.dim)) * np.exp(spread * self.rng.standard_normal((count, heads, 1)))
        return torch.from_numpy(x).to(DT[self.act])

    def append(self, counts, seqs=None, k=None, v=None):
        """The next counts[i] tokens of seqs[i]."""
        seqs = list(range(self.n)) if seqs is None else seqs
        total = sum(counts)
        k = self.tokens(total, self.kvh) if k is None else k
        v = self.tokens(total, self.kvh, 0.5) if v is None else v
        starts = np.concatenate([[0], np.cumsum(counts)])
        for i, s in enumerate(seqs):
            self.k[s].append(_f64(k[starts[i]:starts[i + 1]]))
            self.v[s].append(_f64(v[starts[i]:starts[i + 1]]))
        lens = [m.values.shape[0] for m in self.k]
        self.cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        self.cache.append(self.layer, k.cuda(), v.cuda(), _ids(seqs), _ids(starts))

    def check_stored(self):
        lens = [m.values.shape[0] for m in self.k]
        starts = np.concatenate([[0], np.cumsum(lens)])
        got = [torch.full((int(starts[-1]), self.kvh, self.dim), 7.0, dtype=DT[self.act], device="cuda") for _ in range(2)]
        self.cache.read(self.layer, got[0], got[1], _ids(range(self.n)), _ids(starts))
        for name, models, t in (("k", self.k, got[0]), ("v", self.v, got[1])):
            want = np.concatenate([m.values for m in models])
            want = torch.from_numpy(np.clip(want, -oracle.KV_MAX[self.act], oracle.KV_MAX[self.act])).to(DT[self.act])
            assert torch.equal(t.cpu(), want), f"{name}: {int((t.cpu() != want).sum())} stored values differ"

    def attend(self, counts, window=0, sinks=0, scale=None, seqs=None, q=None, max_new=None, q_std=1.5):
        seqs = list(range(self.n)) if seqs is None else seqs
        total = sum(counts)
        if q is None:
            q = torch.from_numpy(q_std * self.rng.standard_normal((total, self.heads, self.dim))).to(DT[self.act])
        starts = np.concatenate([[0], np.cumsum(counts)])
        out = torch.full((total, self.heads, self.dim), float("nan"), dtype=DT[self.act], device="cuda")
        lse = torch.full((total, self.heads), float("nan"), device="cuda")
        self.cache.attend(self.layer, q.cuda(), out, _ids(seqs), _ids(starts), max_new or max(counts), window, sinks, scale,
                          lse)
        torch.cuda.synchronize()
        return self.compare(q, out, lse, starts, seqs, window, sinks, scale)

    def compare(self, q, out, lse, starts, seqs, window, sinks, scale):
        worst = 0.0
        got, got_lse = _f64(out), _f64(lse)
        for i, s in enumerate(seqs):
            a, b = starts[i], starts[i + 1]
            if a == b:
                continue
            k, v = self.k[s].values, self.v[s].values
            ref, ref_lse, mass, reach = oracle.kv_attend(_f64(q[a:b]), k, v, window, sinks, scale)
            t = k.shape[0]
            dx = reach * ((self.dim + 4) * 2.0 ** -24 + 2.0 ** -23)
            rel = np.expm1(2 * dx) + (t + 16) * 2.0 ** -24
            floor = 2.0 ** -30 * t * (np.abs(v).max() if t else 0.0)
            tol = (rel + 2.0 ** -11)[..., None] * mass + EPS[self.act] * np.abs(ref) + floor + TINY[self.act]
            err = np.abs(got[a:b] - ref)
            assert np.all(err <= tol), f"sequence {s}: out off by {np.max(err / tol):.2f} times its bound"
            none = np.isneginf(ref_lse)
            assert np.array_equal(np.isneginf(got_lse[a:b]), none), f"sequence {s}: rows that see nothing"
            lerr = np.abs(np.where(none, 0, got_lse[a:b]) - np.where(none, 0, ref_lse))
            ltol = dx + (t + 16) * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(np.where(none, 0, ref_lse)))
            assert np.all(lerr <= ltol), f"sequence {s}: lse off by {np.max(lerr / ltol):.2f} times its bound"
            assert np.all(got[a:b][none] == 0)
            worst = max(worst, float(np.max(err / tol)))
        return worst


# ---- what is stored --------------------------------------------------------------------------------


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("act", ["f16", "bf16"])
def test_stored_values(act, code, dim):
    announce(f"kv store {act} {code} {dim}")
    r = Rig([70, 1, 129, 33, 32], 4, 2, dim, 64, act, code, seed=1)
    r.append([37, 0, 64, 31, 32])
    r.check_stored()
    r.append([1, 1, 1, 1], seqs=[0, 1, 2, 3])          # single tokens, out of the first's blocks' range
    r.append([32, 64, 1], seqs=[0, 2, 3])
    r.check_stored()


def test_a_growing_block_is_requantized_step_by_step():
    announce("kv store, growing block")
    for code in ("e4m3", "int8"):
        r = Rig([40], 2, 2, 64, 32, "bf16", code, seed=2)
        for step in range(40):                         # each token up to twice the last
            r.append([1], k=r.tokens(1, 2) * 1.7 ** (step % 23), v=r.tokens(1, 2) * 2.0 ** (step - 20))
        r.check_stored()


def test_extreme_values():
    announce("kv store, zeros, infinities, NaN, subnormals")
    for act in ("f16", "bf16"):
        for code in ("e4m3", "int8"):
            r = Rig([64], 2, 2, 64, 32, act, code, seed=3)
            k, v = r.tokens(64, 2), r.tokens(64, 2)
            k[3] = 0
            k[:32, 1] = 0                              # a block of zeros
            v[5, 0, 7], v[6, 0, 9], v[40, 1, 3] = float("inf"), float("nan"), -float("inf")
            k[32:, 0] = torch.finfo(DT[act]).tiny
            k[33, 0, :8] = torch.finfo(DT[act]).smallest_normal / 4
            r.append([64], k=k, v=v)
            r.check_stored()


def test_read_windows_and_missing_pages():
    announce("kv read, offsets")
    import activation_sparse_decode_relu_amd  # noqa: F401
    r = Rig([100, 70], 2, 2, 64, 32, seed=4)
    r.append([100, 70])
    r.cache.table[1, 1] = -1                           # a hole: tokens 32..63 of sequence 1
    got = [torch.full((90, 2, 64), 7.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    r.cache.read(0, got[0], got[1], _ids([1, 0]), _ids([0, 60, 90]), first=_ids([20, 85]))
    k1 = np.concatenate([r.k[1].values, np.zeros((40, 2, 64))])
    k1[32:64] = 0
    want = np.concatenate([k1[20:80], np.concatenate([r.k[0].values, np.zeros((40, 2, 64))])[85:115]])
    assert torch.equal(got[0].cpu(), torch.from_numpy(want).half())
    v1 = np.concatenate([r.v[1].values, np.zeros((40, 2, 64))])
    v1[32:64] = 0
    want = np.concatenate([v1[20:80], np.concatenate([r.v[0].values, np.zeros((40, 2, 64))])[85:115]])
    assert torch.equal(got[1].cpu(), torch.from_numpy(want).half())


# ---- attention -------------------------------------------------------------------------------------

HEADS = [(4, 4, 64), (8, 1, 64), (16, 1, 128), (6, 2, 128), (32, 2, 64), (17, 1, 64)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("act, code", [("f16", "e4m3"), ("bf16", "int8"), ("bf16", "e4m3"), ("f16", "int8")])
def test_single_tokens(heads, act, code):
    announce(f"kv attend step {heads} {act} {code}")
    lens = [1, 2, 31, 32, 33, 64, 100, 257, 700]
    r = Rig(lens, *heads, 64, act, code, seed=5)
    r.append(lens)
    r.attend([1] * len(lens))
    r.attend([1, 1, 1], seqs=[8, 0, 6])


@pytest.mark.parametrize("page", [32, 96, 128])
@pytest.mark.parametrize("heads", [(8, 2, 64), (2, 2, 128)])
def test_long_sequence_is_split(heads, page):
    announce(f"kv attend long {heads} page {page}")
    r = Rig([9001, 40, 5000], *heads, page, seed=6)
    r.append([9001, 40, 5000])
    r.attend([1, 1, 1])
    r.attend([3, 1, 2])


@pytest.mark.parametrize("new", [2, 4, 5, 7])
@pytest.mark.parametrize("heads", HEADS)
def test_few_tokens(heads, new):
    announce(f"kv attend few {heads} {new}")
    lens = [new, new + 1, 33, 64, 130]
    r = Rig(lens, *heads, 64, "bf16" if new % 2 else "f16", "e4m3", seed=7)
    r.append(lens)
    r.attend([new, 1, new, 0, 2])
    r.attend([1, new, 0, new, new], max_new=new + 3)


@pytest.mark.parametrize("act, code", [("f16", "e4m3"), ("bf16", "int8")])
@pytest.mark.parametrize("heads", [(4, 4, 128), (8, 1, 64), (6, 2, 128), (32, 2, 64)])
def test_prompts_and_pieces(heads, act, code):
    announce(f"kv attend prompts {heads} {act} {code}")
    lens = [1, 65, 128, 300, 517]
    r = Rig(lens, *heads, 32, act, code, seed=8)
    r.append(lens)
    r.attend(lens)
    r.attend([1, 30, 128, 150, 66])


@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (16, 4), (33, 33), (100, 4), (64, 0), (5000, 3)])
@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 1, 128)])
def test_windows_and_sinks(heads, window, sinks):
    announce(f"kv attend window {window} sinks {sinks} {heads}")
    lens = [1, 20, 33, 97, 400, 701]
    r = Rig(lens, *heads, 64, seed=9)
    r.append(lens)
    r.attend([1] * 6, window, sinks)
    r.attend([1, 3, 5, 7, 2, 4], window, sinks)
    r.attend(lens, window, sinks)
    r.attend([0, 7, 33, 50, 130, 90], window, sinks)


def test_rows_that_see_nothing():
    """Lengths of zero, fewer tokens than rows, sequences that are not there, and no pages."""
    announce("kv attend, empty rows")
    r = Rig([40, 3, 64, 50], 8, 2, 64, 32, seed=10)
    r.append([40, 3, 64, 50])
    for rows in (5, 40):                               # a few, and more than one tile of rows
        q = r.tokens(4 * rows, 8)
        out = torch.full((4 * rows, 8, 64), float("nan"), dtype=torch.float16, device="cuda")
        lse = torch.full((4 * rows, 8), float("nan"), device="cuda")
        r.cache.lens.copy_(torch.tensor([40, 3, 0, 50], dtype=torch.int32))
        r.cache.attend(0, q.cuda(), out, _ids([99, 1, 2, -1]), _ids([0, rows, 2 * rows, 3 * rows, 4 * rows]), rows, lse=lse)
        torch.cuda.synchronize()
        gone = torch.ones(4 * rows, dtype=torch.bool)
        gone[2 * rows - 3:2 * rows] = False            # the last three rows of sequence 1 stand in the cache
        assert torch.all(out.cpu()[gone] == 0) and torch.all(lse.cpu()[gone] == -float("inf"))
        r.compare(q[rows:2 * rows], out[rows:2 * rows], lse[rows:2 * rows], [0, rows], [1], 0, 0, None)
        # a hole in the table: those tokens are not there
        r.cache.lens.copy_(torch.tensor([40, 3, 64, 50], dtype=torch.int32))
        saved = r.cache.table.clone()
        r.cache.table[2, 0] = 1 << 28
        q = r.tokens(rows, 8)
        r.cache.attend(0, q.cuda(), out[:rows], _ids([2]), _ids([0, rows]), rows, lse=lse[:rows])
        torch.cuda.synchronize()
        full_k, full_v = r.k[2].values, r.v[2].values
        for j in range(rows):
            p = 64 - rows + j
            if p < 32:
                assert torch.all(out[j] == 0) and torch.all(lse[j] == -float("inf"))
                continue
            ref, ref_lse, mass, _ = oracle.kv_attend(_f64(q[j:j + 1]), full_k[32:p + 1], full_v[32:p + 1])
            assert np.all(np.abs(_f64(out[j]) - ref[0]) <= 2.0 ** -10 * (mass[0] + np.abs(ref[0])) + 2.0 ** -24)
            assert np.all(np.abs(_f64(lse[j]) - ref_lse[0]) <= 1e-4)
        r.cache.table.copy_(saved)


def test_large_and_uneven_scores():
    """Scores of thousands, one token that takes all, values of very different size from block to block,
    and blocks of zeros."""
    announce("kv attend, uneven blocks")
    for act in ("f16", "bf16"):
        r = Rig([300], 4, 2, 64, 32, act, "e4m3", seed=11)
        k, v = r.tokens(300, 2, 0.5), r.tokens(300, 2, 0.0)
        size = torch.ones(300)
        size[32:64], size[64:96], size[96:128], size[200:] = 2.0 ** -12, 2.0 ** 9, 0.0, 2.0 ** -3
        v = (v.float() * size[:, None, None]).to(DT[act])
        k[150] *= 20
        r.append([300], k=k, v=v)
        r.attend([1], q_std=0.3)
        r.attend([1], q_std=60.0)
        r.attend([200], q_std=4.0)
        r.attend([3], scale=1e-4)
    r = Rig([200], 2, 2, 128, 64, "bf16", "int8", seed=12)
    v = r.tokens(200, 2)
    v[:64] *= 2.0 ** 60
    v[64:128] *= 2.0 ** -60
    v[128:] = 0
    r.append([200], v=v)
    r.attend([1])
    r.attend([199])
    r.attend([2], window=40)


def test_tiny_values_and_queries():
    announce("kv attend, subnormal values")
    for act, unit in (("f16", 2.0 ** -22), ("bf16", 2.0 ** -120)):
        r = Rig([70], 4, 2, 64, 32, act, "int8", seed=13)
        r.append([70], k=(r.tokens(70, 2).float() * unit).to(DT[act]), v=(r.tokens(70, 2).float() * unit).to(DT[act]))
        r.attend([1])
        r.attend([33], q=(r.tokens(33, 4).float() * unit).to(DT[act]))


def test_strides():
    """q, k and v as slices of one projection, out in the order [heads][rows]."""
    announce("kv attend, strides")
    r = Rig([90, 33], 8, 2, 128, 64, "bf16", "e4m3", seed=14)
    wide = r.tokens(123, 12).cuda()
    q, k, v = wide[:, :8], wide[:, 8:10], wide[:, 10:]
    starts = [0, 90, 123]
    for i in range(2):
        r.k[i].append(_f64(k[starts[i]:starts[i + 1]]))
        r.v[i].append(_f64(v[starts[i]:starts[i + 1]]))
    r.cache.lens.copy_(torch.tensor([90, 33], dtype=torch.int32))
    r.cache.append(0, k, v, _ids([0, 1]), _ids(starts))
    r.check_stored()
    out = torch.full((8, 123, 128), float("nan"), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    lse = torch.empty(123, 8, device="cuda")
    r.cache.attend(0, q, out, _ids([0, 1]), _ids(starts), 90, lse=lse)
    r.compare(q, out, lse, starts, [0, 1], 0, 0, None)
    back = torch.empty(123, 4, 128, dtype=torch.bfloat16, device="cuda")
    r.cache.read(0, back[:, :2], back[:, 2:], _ids([0, 1]), _ids(starts))
    assert np.array_equal(_f64(back[:, :2]), np.concatenate([m.values for m in r.k]))
    assert np.array_equal(_f64(back[:, 2:]), np.concatenate([m.values for m in r.v]))


def test_many_sequences():
    """More sequences than a wave has lanes, with gaps among those that have rows."""
    announce("kv attend, 150 sequences")
    lens = [1 + (37 * i) % 90 for i in range(150)]
    r = Rig(lens, 4, 2, 64, 32, seed=15)
    r.append(lens)
    r.check_stored()
    r.attend([1] * 150)
    r.attend([min(i % 4, lens[i]) for i in range(150)])
    r.attend([min(70, lens[i]) if i % 3 else 0 for i in range(150)])


def test_layers_do_not_touch_each_other():
    announce("kv layers")
    r = Rig([50], 4, 2, 64, 32, seed=16, layers=3, layer=1)
    r.append([50])
    r.check_stored()
    r.attend([2])
    for i in (0, 2):
        assert torch.all(r.cache.k[i] == 255) and torch.all(r.cache.v_exp[i] == 255)


def test_same_bits_every_time_and_on_another_stream():
    announce("kv attend, repeatable")
    r = Rig([3000, 17, 800], 8, 2, 64, 64, seed=17)
    r.append([3000, 17, 800])
    for counts in ([1, 1, 1], [7, 2, 5], [200, 17, 64]):
        total = sum(counts)
        q = r.tokens(total, 8).cuda()
        seqs, starts = _ids(range(3)), _ids(np.concatenate([[0], np.cumsum(counts)]))
        outs = []
        side = torch.cuda.Stream()
        for rep in range(4):
            out = torch.full((total, 8, 64), float("nan"), dtype=torch.float16, device="cuda")
            if rep == 3:
                side.wait_stream(torch.cuda.current_stream())
                r.cache.attend(0, q, out, seqs, starts, max(counts), stream=side)
                torch.cuda.current_stream().wait_stream(side)
            else:
                r.cache.attend(0, q, out, seqs, starts, max(counts))
            outs.append(out)
        torch.cuda.synchronize()
        for o in outs[1:]:
            assert torch.equal(o, outs[0])


def test_refusals_of_the_library():
    import activation_sparse_decode_relu_amd as pi
    announce("kv refusals")
    r = Rig([10], 4, 2, 64, 32, seed=18)
    r.append([10])
    q = r.tokens(2, 4).cuda()
    out = torch.empty_like(q)
    seqs, starts = _ids([0]), _ids([0, 2])
    c = r.cache
    for kw in (dict(max_new=0), dict(max_new=3), dict(max_new=2, window=-1), dict(max_new=2, sinks=-1),
               dict(max_new=2, scale=0.0), dict(max_new=2, scale=float("inf")), dict(max_new=2, scale=float("nan"))):
        with pytest.raises(pi.PiError) as e:
            c.attend(0, q, out, seqs, starts, **kw)
        assert e.value.status == 1
    for layer in (-1, 1):
        with pytest.raises(pi.PiError):
            c.attend(layer, q, out, seqs, starts, 2)
    odd = torch.empty(2 * 4 * 64 + 8, dtype=torch.float16, device="cuda")[1:513].view(2, 4, 64)
    with pytest.raises(pi.PiError):
        c.attend(0, odd, out, seqs, starts, 2)          # not 16-byte aligned
    with pytest.raises(pi.PiError):
        c.attend(0, q, torch.empty(2, 4, 68, dtype=torch.float16, device="cuda")[..., :64], seqs, starts, 2)
    with pytest.raises(pi.PiError):
        c.free(_ids([0, 0]))                            # more sequences than the table has rows
    empty = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    c.attend(0, empty, empty, seqs, _ids([0, 0]), 1)    # no rows: nothing to do
    c.close()
    with pytest.raises(pi.PiError):
        c.free(seqs)


# ---- pages -----------------------------------------------------------------------------------------


def _state(c):
    return c.table.cpu().tolist(), c.lens.cpu().tolist(), c.refs.cpu().tolist()


def _pool(pages=40, seqs=8, width=6, layers=2, page=32, seed=20):
    import activation_sparse_decode_relu_amd as pi
    c = pi.KVCache(4, 2, 64, pages, page, seqs, width, layers=layers)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    for name in ("k", "v", "k_exp", "v_exp"):
        t = getattr(c, name)
        t.copy_(torch.randint(0, 256, t.shape, dtype=torch.uint8, device="cuda", generator=g))
    return c


def _check(c, before, state, copies):
    """The cache against integers worked out by the oracle, and the bytes the copies moved."""
    assert _state(c) == state
    for name, old in before.items():
        want = old.clone()
        for a, b in copies:
            want[:, b] = old[:, a]
        assert torch.equal(getattr(c, name), want), name


def _bytes(c):
    return {name: getattr(c, name).clone() for name in ("k", "v", "k_exp", "v_exp")}


def test_pages_over_a_long_use():
    """Random reserves, forks, frees and compactions, every one against the oracle."""
    announce("kv pages, random use")
    rng = np.random.default_rng(21)
    for page, pages in ((32, 40), (96, 25)):
        c = _pool(pages=pages, page=page)
        table, lens, refs = _state(c)
        failed = 0
        for step in range(60):
            before, kind = _bytes(c), rng.integers(0, 5)
            some = rng.permutation(8)[:rng.integers(1, 6)].tolist()
            copies = []
            if kind <= 1:
                counts = [int(x) for x in rng.choice([0, 1, 1, 5, page, 70], len(some))]
                copies, bad = oracle.kv_reserve(table, lens, refs, some, counts, page)
                failed += bad
                c.reserve(_ids(some), _ids(counts))
            elif kind == 2:
                oracle.kv_free(table, lens, refs, some)
                c.free(_ids(some))
            elif kind == 3:
                dst = [s for s in range(8) if lens[s] == 0][:3]
                live = [s for s in range(8) if lens[s] > 0]
                if not dst or not live:
                    continue
                src = [live[int(rng.integers(len(live)))] for _ in dst]
                oracle.kv_fork(table, lens, refs, src, dst)
                c.fork(_ids(src), _ids(dst))
            else:
                copies = oracle.kv_compact(table, refs)
                c.compact()
            _check(c, before, (table, lens, refs), copies)
        assert int(c.failed.item()) == failed


def test_reserve_of_a_large_pool():
    """More sequences than the deciding workgroup has threads, a pool of several of its passes, and one page too few."""
    announce("kv reserve, large pool")
    import activation_sparse_decode_relu_amd as pi
    rng = np.random.default_rng(22)
    n, pages = 1500, 9000
    c = pi.KVCache(2, 1, 64, pages, 32, n, 8)
    refs = (rng.random(pages) < 0.75).astype(np.int32)
    c.refs.copy_(torch.from_numpy(refs))
    counts = rng.integers(0, 100, n)
    free = int((refs == 0).sum())
    state = ([[-1] * 8 for _ in range(n)], [0] * n, refs.tolist())
    for part in (counts, counts):
        _, failed = oracle.kv_reserve(*state, list(range(n)), part.tolist(), 32)
        c.reserve(_ids(range(n)), _ids(part))
        got = _state(c)
        assert got == state
        assert int(c.failed.item()) == failed
        c.failed.zero_()
    assert free > 0
    refs = np.array(state[2])
    drop = rng.random(n) < 0.5
    gone = [i for i in range(n) if drop[i]]
    oracle.kv_free(*state, gone)
    c.free(_ids(gone))
    # pages in use by no sequence stay in use: they move like the others
    oracle.kv_compact(state[0], state[2])
    c.compact()
    assert _state(c) == state


def test_check_failed_raises_once():
    import activation_sparse_decode_relu_amd as pi
    announce("kv check_failed")
    c = _pool(pages=2)
    c.reserve(_ids([0, 1, 2]), _ids([32, 32, 1]))
    with pytest.raises(pi.PiError):
        c.check_failed()
    c.check_failed()
    assert _state(c)[1][:3] == [32, 32, 0]


def test_page_calls_ignore_what_is_out_of_range():
    announce("kv pages, out of range")
    c = _pool(pages=6)
    c.reserve(_ids([0]), _ids([40]))
    state = _state(c)
    c.reserve(_ids([-1, 99, 1]), _ids([1, 1, -5]))
    c.free(_ids([-3, 1000]))
    c.fork(_ids([0, 77]), _ids([88, 1]))
    assert _state(c) == state and int(c.failed.item()) == 3


# ---- graphs ----------------------------------------------------------------------------------------


def test_a_decode_step_in_a_graph():
    """Reserve, append and attend captured once and replayed: each replay equals the eager result."""
    import activation_sparse_decode_relu_amd as pi
    announce("kv graph")
    heads, kvh, dim, n = 8, 2, 64, 3

    def fresh():
        c = pi.KVCache(heads, kvh, dim, 30, 32, n, 6)
        c.reserve(_ids(range(n)), _ids([30, 1, 65]))
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        kv = torch.randn(96, kvh, dim, device="cuda", generator=g).half()
        c.append(0, kv, -kv, _ids(range(n)), _ids([0, 30, 31, 96]))
        return c, g

    seqs, starts, ones = _ids(range(n)), _ids([0, 1, 2, 3]), _ids([1] * n)
    eager, gen = fresh()
    steps, want = [], []
    for _ in range(6):
        q, k, v = (torch.randn(n, h, dim, device="cuda", generator=gen).half() for h in (heads, kvh, kvh))
        steps.append((q, k, v))
        out = torch.empty_like(q)
        eager.reserve(seqs, ones)
        eager.append(0, k, v, seqs, starts)
        eager.attend(0, q, out, seqs, starts, 1)
        want.append(out)
    c, _ = fresh()
    q, k, v = (t.clone() for t in steps[0])
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.reserve(seqs, ones)
        c.append(0, k, v, seqs, starts)
        c.attend(0, q, out, seqs, starts, 1)
    for (sq, sk, sv), w in zip(steps, want):
        q.copy_(sq)
        k.copy_(sk)
        v.copy_(sv)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
        torch.randn(1000, device="cuda").sum().item()   # eager work between the replays
    assert _state(c) == _state(eager)
