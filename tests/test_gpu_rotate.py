"""Norms and rotation of queries and keys on the GPU against float64 (angles in 80 bits).

Bounds, in units of 2^-24 of gain (|a| + |b|) of a pair as normalised: the norm 14 (a sum of squares in 12 additions,
halved by the root; the root's reciprocal 4, three products, the mean), a sine or cosine 16 (2^-20), the angle 4
(2^-32 of a turn and its rounding), the gain 1, the two products 2: 37, taken as 40.  The output is rounded once.
"""

import numpy as np
import pytest

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


def _ref(x, pos, freqs, layout, gain, norm, eps):
    """(result, bound without the last rounding) in float64; x [rows][heads][D]."""
    x = x.double().cpu().numpy()
    unit = 0.0
    if norm is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * norm.double().cpu().numpy()
        unit = 14.0
    rot = 2 * len(freqs)
    turns = np.asarray(pos, np.longdouble)[:, None] * np.asarray(freqs, np.longdouble) / (2 * np.longdouble(np.pi) + 2 * np.longdouble("1.2246467991473531772e-16"))
    t = 2 * np.pi * np.asarray(turns - np.rint(turns), np.float64)
    c, s = gain * np.cos(t)[:, None], gain * np.sin(t)[:, None]
    y, tol = x.copy(), unit * 2.0 ** -24 * np.abs(x)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if layout == "interleaved" else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    both = 40 * 2.0 ** -24 * gain * (np.abs(x[..., a]) + np.abs(x[..., b]))
    tol[..., a], tol[..., b] = both, both
    return y, tol


class Rig:
    def __init__(self, lens, heads=8, kv_heads=2, dim=128, act="f16", seed=0, pages=300, **rope):
        import activation_sparse_decode_relu_amd as pi
        self.rng = np.random.default_rng(seed)
        self.heads, self.kvh, self.dim, self.act, self.lens = heads, kv_heads, dim, act, lens
        self.cache = pi.KVCache(heads, kv_heads, dim, 1, 4096, len(lens), pages, act_dtype=act)
        self.cache.lens.copy_(_ids(lens))
        self.rope = pi.Rope(dim, **rope)
        self.layout, self.gain = rope.get("layout", "half"), rope.get("gain", 1.0)

    def tokens(self, rows, heads):
        x = self.rng.standard_normal((rows, heads, self.dim)) * np.exp(self.rng.standard_normal((rows, heads, 1)))
        return torch.from_numpy(x).to(DT[self.act]).cuda()

    def norms(self):
        return [torch.from_numpy(1 + 0.3 * self.rng.standard_normal(self.dim)).to(DT[self.act]).cuda() for _ in range(2)]

    def compare(self, got, x, pos, norm, eps=1e-6):
        ref, tol = _ref(x, pos, self.rope.freqs(), self.layout, self.gain, norm, eps)
        tol = tol * (1 + EPS[self.act]) + EPS[self.act] * np.abs(ref) + TINY[self.act]
        err = np.abs(got.double().cpu().numpy() - ref)
        assert np.all(err <= tol), f"off by {np.max(err / tol):.2f} times its bound"

    def run(self, counts, seqs=None, norm=True, eps=1e-6, positions=None):
        seqs = list(range(len(self.lens))) if seqs is None else seqs
        rows = sum(counts)
        starts = np.concatenate([[0], np.cumsum(counts)])
        q, k = self.tokens(rows, self.heads), self.tokens(rows, self.kvh)
        qn, kn = self.norms() if norm else (None, None)
        qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
        given = None if positions is None else _ids(positions)
        self.cache.rotate(self.rope, q, qo, k, ko, _ids(seqs), _ids(starts), positions=given, q_norm=qn, k_norm=kn, eps=eps)
        torch.cuda.synchronize()
        pos = positions
        if pos is None:
            pos = [self.lens[s] - c + j for s, c in zip(seqs, counts) for j in range(c)]
        self.compare(qo, q, pos, qn, eps)
        self.compare(ko, k, pos, kn, eps)
        return q, k, qo, ko


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("norm", [True, False])
def test_layouts(act, dim, layout, norm):
    announce(f"rotate {act} {dim} {layout} norm {norm}")
    Rig([70, 1, 5000, 33], 8, 2, dim, act, layout=layout, seed=dim).run([7, 1, 40, 0], norm=norm)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim, rot", [(64, r) for r in range(0, 65, 16)] + [(128, r) for r in range(0, 129, 16)])
def test_part_of_the_head(dim, rot, layout):
    announce(f"rotate part {rot} of {dim} {layout}")
    q, k, qo, ko = Rig([90, 20], 4, 4, dim, "f16", layout=layout, rot_dims=rot, seed=rot).run([30, 20], norm=False)
    assert torch.equal(qo[..., rot:], q[..., rot:]) and torch.equal(ko[..., rot:], k[..., rot:])
    Rig([90, 20], 4, 4, dim, "f16", layout=layout, rot_dims=rot, seed=rot).run([30, 20])


@pytest.mark.parametrize("heads, kvh, dim", [(1, 1, 64), (1, 1, 128), (3, 1, 64), (5, 5, 128), (7, 1, 128), (71, 1, 64),
                                             (32, 32, 128), (128, 8, 64), (1024, 1, 64), (56, 56, 128)])
@pytest.mark.parametrize("counts", [[1, 1], [3, 130]])
def test_heads(heads, kvh, dim, counts):
    announce(f"rotate heads {heads} {kvh} {dim}")
    Rig([700, 900], heads, kvh, dim, "bf16", seed=heads).run(counts)


@pytest.mark.parametrize("scaling", [dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                     dict(scaling="bands", factor=32.0, original=8192, base=500000.0, gain=1.25),
                                     dict(freqs=[0.0, 1e-12, 3.14159, 1.0] * 16)])
def test_scaling_and_far_positions(scaling):
    """Up to the longest sequence a cache can have, where an angle in fp32 would be off by whole turns."""
    announce(f"rotate scaling {scaling}")
    lens = [(1 << 30) - 3, (1 << 20) + 7, 12345677, 1000, 1 << 24]
    r = Rig(lens, 4, 1, 128, "f16", pages=1 << 18, seed=1, **scaling)
    r.run([5, 1, 70, 64, 2])


@pytest.mark.parametrize("norm", [True, False])
def test_given_positions(norm):
    announce("rotate positions")
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 77, 77, 3]
    Rig([5, 5], 4, 2, 64, "bf16", seed=5).run([3, 5], norm=norm, positions=pos)


def test_many_sequences_and_empty_ones():
    announce("rotate many sequences")
    rng = np.random.default_rng(3)
    counts = rng.integers(0, 3, 300).tolist()
    lens = [int(c + x) for c, x in zip(counts, rng.integers(0, 9000, 300))]
    order = rng.permutation(300).tolist()
    Rig(lens, 4, 1, 64, "f16", seed=3).run([counts[s] for s in order], seqs=order)


def test_rows_of_no_sequence_and_bad_numbers():
    """Rows past the last sequence's end stay; sequences and lengths out of range do no harm, their neighbours are right."""
    announce("rotate stray rows")
    for given in (None, [4] * 12):
        r = Rig([100, 50, 60, 5], 4, 2, 64, "f16", seed=6)
        q, k = r.tokens(12, 4), r.tokens(12, 2)
        qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
        r.cache.lens[2] = 1 << 30                    # past the table
        r.cache.rotate(r.rope, q, qo, k, ko, _ids([0, 99, 2, 1]), _ids([0, 3, 5, 6, 9]), positions=None if given is None else _ids(given))
        torch.cuda.synchronize()
        assert bool((qo[9:] == 7).all()) and bool((ko[9:] == 7).all())
        rows = [0, 1, 2, 6, 7, 8]
        pos = [97, 98, 99, 47, 48, 49] if given is None else [4] * 6
        r.compare(qo[rows], q[rows], pos, None)
        r.compare(ko[rows], k[rows], pos, None)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place_in_a_fused_projection(layout):
    announce("rotate in place")
    r = Rig([40, 41, 3], 8, 2, 128, "f16", layout=layout, rot_dims=96, seed=8)
    rows = 60
    qkv = torch.randn(rows, 12, 128, device="cuda").half()
    was = qkv.clone()
    qn, kn = r.norms()
    q, k = qkv[:, :8], qkv[:, 8:10]
    seqs, starts = _ids([0, 1, 2]), _ids([0, 30, 58, 60])
    qo, ko = torch.empty(8, rows, 128, device="cuda").half().transpose(0, 1), torch.empty_like(k)
    r.cache.rotate(r.rope, q, qo, k, ko, seqs, starts, q_norm=qn, k_norm=kn)
    r.cache.rotate(r.rope, q, q, k, k, seqs, starts, q_norm=qn, k_norm=kn)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, 10:], was[:, 10:])
    pos = list(range(10, 40)) + list(range(13, 41)) + [1, 2]
    r.compare(qo, was[:, :8], pos, qn)
    r.compare(ko, was[:, 8:10], pos, kn)


def test_norm_extremes():
    """Zero heads give zeros, one large or tiny element its own weight; one norm may be given without the other."""
    announce("rotate extremes")
    for act in ("f16", "bf16"):
        r = Rig([9], 2, 1, 64, act, seed=2)
        q, k = torch.zeros(3, 2, 64, dtype=DT[act], device="cuda"), r.tokens(3, 1)
        q[1, 0, 5], q[2, 1, 40] = 60000.0, 2.0 ** -24
        qn, kn = r.norms()
        for norms in ((qn, None), (None, kn), (qn, kn)):
            qo, ko = torch.empty_like(q), torch.empty_like(k)
            r.cache.rotate(r.rope, q, qo, k, ko, _ids([0]), _ids([0, 3]), q_norm=norms[0], k_norm=norms[1], eps=1e-12)
            assert bool((qo[0] == 0).all())
            r.compare(qo, q, [6, 7, 8], norms[0], 1e-12)
            r.compare(ko, k, [6, 7, 8], norms[1], 1e-12)


def test_a_head_does_not_touch_another():
    announce("rotate heads apart")
    r = Rig([50], 8, 4, 64, "f16", rot_dims=32, seed=4)
    q, k = r.tokens(20, 8), r.tokens(20, 4)
    qn, kn = r.norms()
    outs = []
    for bad in (False, True):
        if bad:
            q[3, 5, 50], k[4, 0, 1] = float("nan"), float("inf")
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        r.cache.rotate(r.rope, q, qo, k, ko, _ids([0]), _ids([0, 20]), q_norm=qn, k_norm=kn)
        outs.append((qo, ko))
    (a, b), (c, d) = outs
    assert bool(c[3, 5].isnan().all())
    c[3, 5], d[4, 0] = a[3, 5], b[4, 0]
    assert torch.equal(a, c) and torch.equal(b, d)
    # without norms a dim that is not turned is passed on beside others' NaN
    q[3, 5, 1] = float("inf")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    r.cache.rotate(r.rope, q, qo, k, ko, _ids([0]), _ids([0, 20]))
    assert torch.equal(qo[3, 5, 32:50], q[3, 5, 32:50]) and torch.equal(qo[3, 5, 51:], q[3, 5, 51:])


def test_streams_and_graphs():
    """A graph takes the positions from the lengths as they are at each replay."""
    announce("rotate graph")
    r = Rig([50, 60], 8, 2, 128, "f16", seed=7)
    q, k = r.tokens(2, 8), r.tokens(2, 2)
    qn, kn = r.norms()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    seqs, starts = _ids([0, 1]), _ids([0, 1, 2])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r.cache.rotate(r.rope, q, qo, k, ko, seqs, starts, q_norm=qn, k_norm=kn, stream=s)
    torch.cuda.synchronize()
    r.compare(qo, q, [49, 59], qn)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.cache.rotate(r.rope, q, qo, k, ko, seqs, starts, q_norm=qn, k_norm=kn)
    for step in range(1, 5):
        r.cache.lens += 1
        qo.zero_()
        graph.replay()
        torch.cuda.synchronize()
        r.compare(qo, q, [49 + step, 59 + step], qn)
        r.compare(ko, k, [49 + step, 59 + step], kn)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("heads, kvh, dim", [(30, 5, 128), (33, 11, 64), (13, 13, 128)])
@pytest.mark.parametrize("counts", [[250, 1, 0, 40], [900, 3, 1, 500]])
def test_several_heads_a_wave(counts, heads, kvh, dim, layout):
    """Calls in which a wave takes two and four times its heads, with heads left over; with norms, without, and a part turned."""
    announce(f"rotate {counts} {heads} {kvh} {dim} {layout}")
    r = Rig([5000, 70, 9, 501], heads, kvh, dim, "f16", layout=layout, rot_dims=dim // 2, seed=heads)
    r.run(counts)
    r.run(counts, norm=False)
