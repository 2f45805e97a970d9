"""Products with 4-bit weights on the GPU against float64.

Bounds.  A group's sum is a product of whole numbers 24 + q with x, begun with -24 sum x, itself summed in fp32: 32 terms
of at most 24 |x| and 33 of at most 55 of the group's sum |x| (the beginning among them), each addition off by 2^-24:
(32 * 24 + 33 * 55) 2^-24 < 2600 * 2^-24 of it, times the scale.  The G groups, the waves, bias and add join in fp32:
(G + 12) 2^-24 of the terms' magnitudes.  y is rounded once: half a step of its type.  With more than 64 rows a
weight is rounded to fp16, relative to the row's largest scale in [8, 16): half a step, 2^-11 of it, or 2^-25 / 8 of that
scale where that is more; scales of less than 2^-17 of the largest lose as little, times 8; and bf16 rows of x are fp16
relative to their largest in [2^14, 2^15): exact, or off by 2^-25 / 2^14 of it.
"""

import numpy as np
import pytest

import oracle
from synth.layers import pack_nibbles, quantize_q4g32

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


class Rig:
    def __init__(self, d_in, d_out, act="f16", bias=False, seed=0):
        import activation_sparse_decode_relu_amd as pi
        self.rng = rng = np.random.default_rng(seed)
        self.d_in, self.d_out, self.act = d_in, d_out, act
        w = rng.standard_normal((d_out, d_in)) * np.exp(rng.standard_normal((d_out, 1)))
        codes, scales = quantize_q4g32(w)
        codes[0, :2] = (0x88, 0x7F)                  # -8, -8, -1, 7
        self.w = oracle.dequant_q4g32(codes, scales)
        self.s = np.repeat(scales.astype(np.float64), 32, axis=1)
        self.bias = rng.standard_normal(d_out).astype(np.float32) if bias else None
        up = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
        self.m = pi.Linear(up(codes), up(scales), act_dtype=act, bias=up(self.bias))

    def x(self, rows):
        v = self.rng.standard_normal((rows, self.d_in)) * np.exp(self.rng.standard_normal((1, self.d_in)))
        return torch.from_numpy(v).to(DT[self.act])

    def check(self, x, y, add=None):
        x = x.double().cpu().numpy()
        more = np.zeros((x.shape[0], self.d_out)) if add is None else add.double().cpu().numpy()
        bias = np.zeros(self.d_out) if self.bias is None else self.bias.astype(np.float64)
        ref = x @ self.w.T + bias + more
        mass = np.abs(x) @ np.abs(self.w).T + np.abs(bias) + np.abs(more)
        tol = (2600 * 2.0 ** -24 * (np.abs(x) @ self.s.T) + (self.d_in // 32 + 12) * 2.0 ** -24 * mass +
               EPS[self.act] * np.abs(ref) + TINY[self.act])
        tol += 2.0 ** -25 * (np.abs(x).sum(1, keepdims=True) * self.s.max(1))          # scales kept relative to the row's largest
        if x.shape[0] > 64:
            tol += 2.0 ** -11 * (np.abs(x) @ np.abs(self.w).T) * (1 + EPS[self.act])
            tol += 2.0 ** -39 * np.abs(x).max(1, keepdims=True) * np.abs(self.w).sum(1)
        err = np.abs(y.double().cpu().numpy() - ref)
        assert np.all(err <= tol), f"off by {np.max(err / tol):.2f} times its bound"

    def run(self, rows, add=False):
        x = self.x(rows)
        more = torch.from_numpy(self.rng.standard_normal((rows, self.d_out))).to(DT[self.act]) if add else None
        y = torch.full((rows, self.d_out), float("nan"), dtype=DT[self.act], device="cuda")
        self.m.forward(x.cuda(), y, None if more is None else more.cuda())
        torch.cuda.synchronize()
        self.check(x, y, more)


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 32, 33, 63, 64, 65, 100, 128, 129, 300])
def test_rows(rows, act):
    announce(f"linear rows {rows} {act}")
    Rig(1024, 80, act, bias=True, seed=rows).run(rows, add=rows % 2 == 0)


@pytest.mark.parametrize("d_in", [32, 64, 96, 224, 256, 288, 512, 736, 2048, 2080, 8192, 11008])
@pytest.mark.parametrize("rows", [1, 7, 40, 130])
def test_widths(d_in, rows):
    announce(f"linear d_in {d_in}, rows {rows}")
    Rig(d_in, 100, "f16", seed=d_in).run(rows)


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("d_in, d_out", [(512, 200), (768, 100), (1312, 333), (4096, 129), (11008, 1000)])
@pytest.mark.parametrize("rows", [65, 127, 128, 129, 400])
def test_split_columns(rows, d_in, d_out, act):
    """Few workgroups: the columns in ranges whose sums are joined."""
    announce(f"linear split {rows} {d_in} {d_out} {act}")
    Rig(d_in, d_out, act, bias=True, seed=rows).run(rows, add=True)


@pytest.mark.parametrize("d_out", [1, 2, 15, 16, 17, 31, 33, 63, 65, 127, 129, 1000, 5001])
@pytest.mark.parametrize("rows", [1, 16, 64, 200])
def test_outputs(d_out, rows):
    announce(f"linear d_out {d_out}, rows {rows}")
    Rig(320, d_out, "bf16", bias=True, seed=d_out).run(rows, add=True)


@pytest.mark.parametrize("rows", [1, 3, 6, 16, 48, 150])
@pytest.mark.parametrize("act", ["f16", "bf16"])
def test_whole_numbers_are_exact(rows, act):
    """x, the codes and the scales are such that every sum is exact: y has to be equal, and every code is met."""
    import activation_sparse_decode_relu_amd as pi
    announce(f"linear lattice {rows} {act}")
    rng = np.random.default_rng(rows)
    d_in, d_out = 608, 75
    q = rng.integers(-8, 8, (d_out, d_in))
    scales = np.exp2(rng.integers(-3, 3, (d_out, d_in // 32))).astype(np.float16)
    codes = pack_nibbles(q)
    x = rng.integers(-2, 3, (rows, d_in)).astype(np.float64)
    ref = x @ oracle.dequant_q4g32(codes, scales).T
    m = pi.Linear(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), act_dtype=act)
    y = torch.empty(rows, d_out, dtype=DT[act], device="cuda")
    m.forward(torch.from_numpy(x).to(DT[act]).cuda(), y)
    assert torch.equal(y.cpu(), torch.from_numpy(ref).to(DT[act]))


@pytest.mark.parametrize("rows", [1, 5, 40, 140])
def test_strides_and_what_lies_beside(rows):
    announce(f"linear strides {rows}")
    r = Rig(288, 77, "f16", bias=True, seed=3)
    wide = torch.full((rows, 288 + 40), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, 16:304] = r.x(rows).cuda()
    x = wide[:, 16:304]
    big = torch.full((rows + 1, 100), 7.0, dtype=torch.float16, device="cuda")
    add = torch.randn(1, 77, device="cuda").half().expand(rows, 77)
    r.m.forward(x, big[:rows, 3:80], add)
    r.check(x, big[:rows, 3:80], add)
    assert bool((big[:rows, :3] == 7).all()) and bool((big[:rows, 80:] == 7).all()) and bool((big[rows] == 7).all())
    same = add.contiguous()
    r.m.forward(x, same, same)                       # into what is added
    assert torch.equal(same, big[:rows, 3:80])


@pytest.mark.parametrize("act", ["f16", "bf16"])
def test_a_row_does_not_touch_another(act):
    """Rows with infinities and NaN are not finite, the others keep their bits; the order of rows does not matter."""
    announce(f"linear rows apart {act}")
    for rows in (2, 4, 13, 40, 70):
        r = Rig(512, 48, act, seed=rows)
        x = r.x(rows).cuda()
        y, z = (torch.empty(rows, 48, dtype=DT[act], device="cuda") for _ in range(2))
        r.m.forward(x, y)
        bad = x.clone()
        bad[1, 3], bad[0, 100] = float("inf"), float("nan")
        r.m.forward(bad, z)
        assert not bool(z[:2].isfinite().any()) and torch.equal(z[2:], y[2:])
        r.m.forward(x.flip(0).contiguous(), z)
        assert torch.equal(z.flip(0), y)


@pytest.mark.parametrize("act, value", [("f16", 65504.0), ("f16", 2.0 ** -24), ("f16", 3 * 2.0 ** -16), ("bf16", 2.0 ** 117),
                                        ("bf16", 2.0 ** -100)])
def test_extreme_inputs(act, value):
    announce(f"linear extremes {act} {value}")
    import activation_sparse_decode_relu_amd as pi
    q = np.zeros((16, 64), dtype=np.int64)
    q[:, 0], q[:, 40] = np.arange(16) - 8, 1
    scales = np.full((16, 2), 2.0 ** -8 if value > 1 else 1.0, dtype=np.float16)
    m = pi.Linear(torch.from_numpy(pack_nibbles(q)).cuda(), torch.from_numpy(scales).cuda(), act_dtype=act)
    x = torch.zeros(3, 64, dtype=DT[act])
    x[:, 0] = value
    x[1, 40] = value
    ref = x.double() @ torch.from_numpy(oracle.dequant_q4g32(pack_nibbles(q), scales)).T
    y = torch.empty(3, 16, dtype=DT[act], device="cuda")
    m.forward(x.cuda(), y)
    assert torch.equal(y.cpu(), ref.to(DT[act]))


def test_scratch_of_the_callers():
    announce("linear scratch")
    import activation_sparse_decode_relu_amd as pi
    r = Rig(320, 40, "bf16", seed=12)
    x = r.x(70).cuda()
    y, z = (torch.empty(70, 40, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    r.m.forward(x, y)
    need = r.m.scratch_bytes(70)
    scratch = torch.full((need + 16,), 77, dtype=torch.uint8, device="cuda")
    r.m.forward(x, z, scratch=scratch)
    assert torch.equal(y, z) and bool((scratch[need:] == 77).all())
    with pytest.raises(pi.PiError) as e:
        r.m.forward(x, z, scratch=scratch[:need - 1])
    assert e.value.status == 2


@pytest.mark.parametrize("rows", [20, 50, 100, 260])
def test_rows_of_very_different_size(rows):
    """bf16 rows from 2^-100 to 2^100, zero rows among them: each is as accurate as alone."""
    announce(f"linear row sizes {rows}")
    r = Rig(512, 33, "bf16", seed=rows)
    x = r.x(rows)
    x *= torch.exp2(torch.from_numpy(r.rng.integers(-100, 100, (rows, 1)).astype(np.float32))).bfloat16()
    x[3] = 0
    y = torch.empty(rows, 33, dtype=torch.bfloat16, device="cuda")
    r.m.forward(x.cuda(), y)
    r.check(x, y)


def test_scales_of_very_different_size():
    """Rows of W from fp16's smallest scales to its largest."""
    announce("linear scale sizes")
    import activation_sparse_decode_relu_amd as pi
    rng = np.random.default_rng(8)
    q = rng.integers(-8, 8, (48, 256))
    scales = np.exp2(rng.integers(-24, 16, (48, 1)) + np.zeros((1, 8))).astype(np.float16)
    scales[5], scales[6, 3] = 0, 65504
    codes = pack_nibbles(q)
    m = pi.Linear(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), act_dtype="bf16")
    w = oracle.dequant_q4g32(codes, scales)
    for rows in (1, 10, 30, 60, 100):
        x = torch.from_numpy(rng.integers(-3, 4, (rows, 256)).astype(np.float64)).bfloat16()
        y = torch.empty(rows, 48, dtype=torch.bfloat16, device="cuda")
        m.forward(x.cuda(), y)
        ref = x.double().numpy() @ w.T
        keep = [i for i in range(48) if i != 6]     # exact sums; row 6 mixes 65504 with smaller ones
        assert torch.equal(y.cpu()[:, keep], torch.from_numpy(ref).bfloat16()[:, keep]), f"{rows} rows"
        mass = np.abs(x.double().numpy()) @ np.abs(w).T
        assert np.all(np.abs(y.cpu().double().numpy() - ref)[:, 6] <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -14) * mass[:, 6])


def test_no_rows():
    r = Rig(64, 8)
    r.m.forward(torch.empty(0, 64, dtype=torch.float16, device="cuda"), torch.empty(0, 8, dtype=torch.float16, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows", [1, 24, 130])
def test_streams_and_graphs(rows):
    """Calls at the same time on two streams, and a graph whose replays follow other work."""
    announce(f"linear streams {rows}")
    r = Rig(2048, 500, "f16", bias=True, seed=9)
    x = r.x(rows).cuda()
    want, one, two = (torch.empty(rows, 500, dtype=torch.float16, device="cuda") for _ in range(3))
    r.m.forward(x, want)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        r.m.forward(x, one, stream=a)
        r.m.forward(x, two, stream=b)
    torch.cuda.synchronize()
    assert torch.equal(one, want) and torch.equal(two, want)
    inp = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.m.forward(inp, one)
    for i in range(4):
        inp.copy_(x * (i + 1) if i < 2 else x)
        r.m.forward(inp, two)
        one.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(one, two)
    assert torch.equal(one, want)


def test_weights_made_on_another_stream():
    announce("linear, packed on a stream")
    import activation_sparse_decode_relu_amd as pi
    r = Rig(4096, 2000, seed=4)
    codes, scales = quantize_q4g32(np.random.default_rng(1).standard_normal((2000, 4096)))
    s = torch.cuda.Stream()
    m = pi.Linear(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), stream=s)
    x = r.x(2).cuda()
    y, z = (torch.empty(2, 2000, dtype=torch.float16, device="cuda") for _ in range(2))
    s.wait_stream(torch.cuda.current_stream())
    m.forward(x, y, stream=s)
    torch.cuda.synchronize()
    pi.Linear(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()).forward(x, z)
    assert torch.equal(y, z)


@pytest.mark.parametrize("rows", [1, 33])
def test_weights_past_4_gib(rows):
    """Packed weights of more than 2^32 bytes: the last rows of the matrix are where they belong."""
    announce(f"linear 4 GiB, rows {rows}")
    import activation_sparse_decode_relu_amd as pi
    d_in, d_out, tail = 8192, 1 << 20, 64
    codes = torch.zeros(d_out, d_in // 2, dtype=torch.uint8, device="cuda")
    scales = torch.ones(d_out, d_in // 32, dtype=torch.float16, device="cuda")
    rng = np.random.default_rng(2)
    q = rng.integers(-8, 8, (tail, d_in))
    codes[-tail:] = torch.from_numpy(pack_nibbles(q)).cuda()
    m = pi.Linear(codes, scales)
    assert m.packed.numel() > 1 << 32
    x = torch.from_numpy(rng.integers(-1, 2, (rows, d_in)).astype(np.float64)).half()
    y = torch.full((rows, d_out), float("nan"), dtype=torch.float16, device="cuda")
    m.forward(x.cuda(), y)
    want = x.double() @ torch.from_numpy(q.astype(np.float64)).T
    assert bool((y[:, :-tail] == 0).all()) and torch.equal(y[:, -tail:].cpu(), want.half())


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 3, 16, 24, 64, 100])
def test_small_scales_beside_large_ones(rows, act):
    """x is zero where a row's largest scale is: what the small ones bring is all there is.  Codes and x are powers of two, so
    each output is one exact product, with scales of all of fp16's bits, unless the row's largest is 2^13 or more: its scales
    are divided by up to 8 and may lose half a step of 2^-24 of that."""
    announce(f"linear small scales {rows} {act}")
    import activation_sparse_decode_relu_amd as pi
    rng = np.random.default_rng(rows)
    groups, tops = 12, np.arange(-24, 16)
    d_out = 2 * len(tops)
    q = np.zeros((d_out, 32 * groups), dtype=np.int64)
    scales = np.exp2(rng.integers(-24, np.repeat(tops, 2)[:, None] + 1, (d_out, groups))) * (1 + rng.integers(0, 1024, (d_out, groups)) / 1024)
    scales[:, 0] = np.exp2(np.repeat(tops, 2))
    scales = np.minimum(scales, 1.999 * scales[:, :1]).astype(np.float16)
    q[:, ::32] = rng.choice([-8, -4, -2, -1, 1, 2, 4], (d_out, groups))
    m = pi.Linear(torch.from_numpy(pack_nibbles(q)).cuda(), torch.from_numpy(scales).cuda(), act_dtype=act)
    x = np.zeros((rows, 32 * groups))
    at = rng.integers(1, groups, rows)
    x[np.arange(rows), 32 * at] = np.exp2(rng.integers(-2, 3, rows))
    y = torch.empty(rows, d_out, dtype=DT[act], device="cuda")
    m.forward(torch.from_numpy(x).to(DT[act]).cuda(), y)
    want = torch.from_numpy(x @ (q * np.repeat(scales.astype(np.float64), 32, axis=1)).T)
    exact = torch.from_numpy(scales.max(1) < 8192)
    assert torch.equal(y.cpu()[:, exact], want.to(DT[act])[:, exact])
    want = want.clamp(-float(torch.finfo(DT[act]).max), float(torch.finfo(DT[act]).max))
    err = (y.cpu().double().clamp(-float(torch.finfo(DT[act]).max), float(torch.finfo(DT[act]).max)) - want).abs()
    assert bool((err <= EPS[act] * want.abs() + TINY[act] + 2.0 ** -22 * 8 * x.max()).all())


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [65, 130, 300])
def test_scratch_of_other_calls(rows, act):
    """Columns are split into as many ranges as the scratch holds: that of more rows, which may take less, is enough."""
    announce(f"linear scratch of other calls {rows} {act}")
    r = Rig(4096, 200, act, bias=True, seed=rows)
    x, add = r.x(rows), torch.from_numpy(r.rng.standard_normal((rows, 200))).to(DT[act])
    need, whole = r.m.scratch_bytes(rows), r.m.scratch_bytes(60000, upto=True)
    least = 0 if act == "f16" else -(-rows * 8192 // 256) * 256 + -(-rows * 4 // 256) * 256
    assert r.m.scratch_bytes(60000) < need if act == "f16" else least < need < whole
    sums = rows * 200 * 4
    for size in sorted({least, least + sums, least + 2 * sums, least + 2 * sums + 300, least + 5 * sums, need - 1, need, need + 999}):
        scratch = torch.full((size + 4096,), 77, dtype=torch.uint8, device="cuda")
        y = torch.full((rows, 200), float("nan"), dtype=DT[act], device="cuda")
        r.m.forward(x.cuda(), y, add.cuda(), scratch=scratch[:size])
        torch.cuda.synchronize()
        r.check(x, y, add)
        assert bool((scratch[size:] == 77).all())
    if act == "f16":
        big = torch.empty(r.m.scratch_bytes(60000), dtype=torch.uint8, device="cuda")
        r.m.forward(x.cuda(), y, add.cuda(), scratch=big)
        r.check(x, y, add)
