"""Products with 4-bit weights without a GPU: the C ABI's symbols and refusals, and the binding's checks."""

import ctypes
import os
import re
import subprocess

import pytest

torch = pytest.importorskip("torch")
pi = pytest.importorskip("activation_sparse_decode_relu_amd")
from activation_sparse_decode_relu_amd import linear as lin  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "pi_linear.h")
FAKE = 0x10000


def _declared():
    return sorted(set(re.findall(r"^\s*(?:pi_status|int32_t)\s+(pi_linear_\w+)\s*\(", open(HEADER).read(), re.M)))


def test_symbols():
    assert set(_declared()) == set(pi.LINEAR_EXPORTED)
    for name in _declared():
        assert hasattr(pi.LIB, name), f"{name} is declared in pi_linear.h but not exported"
    assert pi.LIB.pi_linear_abi_version() == lin.LINEAR_ABI_VERSION


def test_header_is_plain_c(tmp_path):
    for cc, flags in (("gcc", ["-std=c99", "-xc"]), ("g++", ["-std=c++17", "-xc++"])):
        src = tmp_path / "use.c"
        src.write_text('#include "pi_linear.h"\nint main(void) { pi_linear_desc d; (void)d; return PI_LINEAR_ABI_VERSION - 1; }\n')
        subprocess.run([cc, *flags, "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only", "-I",
                        os.path.join(ROOT, "include"), str(src)], check=True)


def test_struct_layouts():
    assert ctypes.sizeof(lin.LinearDesc) == 12
    assert ctypes.sizeof(lin.LinearArgs) == 72


@pytest.mark.parametrize("d_in, d_out, tiles, slabs", [(32, 1, 1, 1), (256, 16, 1, 1), (288, 17, 2, 2), (8192, 10240, 640, 32)])
def test_packed_bytes(d_in, d_out, tiles, slabs):
    assert pi.linear_packed_bytes(pi.linear_desc(d_in, d_out)) == tiles * slabs * 2304 + 64 * tiles


@pytest.mark.parametrize("bad", [dict(d_in=0), dict(d_in=48), dict(d_in=-32), dict(d_in=(1 << 20) + 32), dict(d_out=0),
                                 dict(d_out=(1 << 24) + 1), dict(act_dtype=2), dict(act_dtype=-1)])
def test_bad_descriptors(bad):
    with pytest.raises(pi.PiError) as e:
        pi.linear_packed_bytes(pi.linear_desc(**{**dict(d_in=64, d_out=8), **bad}))
    assert e.value.status == 1 and pi.last_error()


def test_numbers_past_32_bits():
    with pytest.raises(pi.PiError):
        pi.linear_desc(1 << 32, 8)
    with pytest.raises(KeyError):
        pi.linear_desc(64, 8, "f32")


@pytest.mark.parametrize("change, status", [
    (dict(w=None), 1), (dict(w=FAKE + 2), 1), (dict(scales=None), 1), (dict(scales=FAKE + 1), 1), (dict(bias=FAKE + 2), 1),
    (dict(packed=None), 2), (dict(packed=FAKE + 16), 2), (dict(size=2304 + 63), 2)])
def test_create_refusals(change, status):
    a = {**dict(w=FAKE, scales=FAKE, bias=None, packed=FAKE, size=2304 + 64), **change}
    d, h = pi.linear_desc(64, 8), ctypes.c_void_p()
    st = pi.LIB.pi_linear_create(ctypes.byref(d), a["w"], a["scales"], a["bias"], a["packed"], a["size"], None, ctypes.byref(h))
    assert st == status and not h.value


def test_null_handles():
    a, h = lin.LinearArgs(), ctypes.c_void_p()
    assert pi.LIB.pi_linear_forward(None, ctypes.byref(a), None) == 1
    assert pi.LIB.pi_linear_destroy(None) == 1
    assert pi.LIB.pi_linear_create(None, None, None, None, None, 0, None, ctypes.byref(h)) == 1
    assert pi.LIB.pi_linear_packed_bytes(None, None) == 1


class _Handle:
    """A handle as the library lays it out, for refusals that come before anything is enqueued: desc, packed, bias."""

    def __init__(self, d_in, d_out, act="f16"):
        class Raw(ctypes.Structure):
            _fields_ = [("desc", lin.LinearDesc), ("packed", ctypes.c_void_p), ("bias", ctypes.c_void_p)]
        self.raw = Raw(pi.linear_desc(d_in, d_out, act), FAKE, None)

    def forward(self, **change):
        a = {**dict(x=FAKE, add=None, y=FAKE, x_stride=64, add_stride=0, y_stride=8, scratch=None, scratch_bytes=0, rows=2), **change}
        return pi.LIB.pi_linear_forward(ctypes.byref(self.raw), ctypes.byref(lin.LinearArgs(**a)), None)


@pytest.mark.parametrize("change", [dict(rows=-1), dict(rows=(1 << 24) + 1), dict(x=None), dict(x=FAKE + 8), dict(y=None),
                                    dict(y=FAKE + 1), dict(add=FAKE + 1), dict(x_stride=68), dict(x_stride=-64), dict(x_stride=(1 << 23) + 8),
                                    dict(add=FAKE, add_stride=-8), dict(y_stride=7)])
def test_forward_refusals(change):
    assert _Handle(64, 8).forward(**change) == 1 and pi.last_error()


def test_scratch():
    """fp16 rows and factors (bf16), and a sum for each range of columns where few workgroups would be busy."""
    def need(d_in, d_out, rows, act):
        out = ctypes.c_size_t(9)
        assert pi.LIB.pi_linear_scratch_bytes(ctypes.byref(_Handle(d_in, d_out, act).raw), rows, ctypes.byref(out)) == 0
        return out.value
    assert [need(8192, 8192, rows, "bf16") for rows in (0, 1, 64)] == [0, 0, 0]
    assert need(64, 8, 65, "f16") == 0 and need(64, 8, 65, "bf16") == 8448 + 512    # one slab: one range
    assert need(4096, 12288, 2000, "f16") == 0                                   # workgroups enough
    assert need(8192, 8192, 128, "f16") == 8 * 128 * 8192 * 4                    # 64 of them, 32 slabs in 8 ranges
    assert need(7168, 21504, 100, "bf16") == 100 * 7168 * 2 + 512 + 3 * 100 * 21504 * 4
    h, out, size = _Handle(64, 8, "bf16"), ctypes.c_size_t(9), 8448 + 512
    for bad in (dict(scratch=None), dict(scratch=FAKE + 8), dict(scratch_bytes=size - 1)):
        assert h.forward(rows=65, **{**dict(scratch=FAKE, scratch_bytes=size), **bad}) == 2
    assert pi.LIB.pi_linear_scratch_bytes(None, 1, ctypes.byref(out)) == 1
    assert pi.LIB.pi_linear_scratch_bytes(ctypes.byref(h.raw), -1, ctypes.byref(out)) == 1
    assert pi.LIB.pi_linear_scratch_bytes(ctypes.byref(h.raw), 1, None) == 1


def test_no_rows_enqueue_nothing():
    assert _Handle(64, 8).forward(rows=0, x=None, y=None) == 0


# ---- the binding -----------------------------------------------------------------------------------


def _closed(act="f16"):
    m = object.__new__(pi.Linear)
    m.desc, m.handle, m.device = pi.linear_desc(64, 8, act), ctypes.c_void_p(), torch.device("cpu")
    m._act = lin._ACT_TORCH[m.desc.act_dtype]
    return m


def _rejects(fn, needle):
    with pytest.raises(pi.PiError) as e:
        fn()
    assert e.value.status == 1 and needle in str(e.value), str(e.value)


@pytest.mark.parametrize("x, y, add, needle", [
    (None, (5, 8), None, "x must be a torch tensor"), ((5, 32), (5, 8), None, "x must be [rows][64]"),
    ((5, 64), (4, 8), None, "y must be [5][8]"), ((5, 64), (5, 8), (5, 64), "add must be [5][8]")])
def test_shapes(x, y, add, needle):
    make = lambda s: None if s is None else torch.zeros(s, dtype=torch.float16)  # noqa: E731
    _rejects(lambda: _closed().forward(make(x), make(y), make(add)), needle)


def test_tensor_refusals():
    m, h = _closed(), torch.float16
    x, y = torch.zeros(5, 64, dtype=h), torch.zeros(5, 8, dtype=h)
    _rejects(lambda: m.forward(x.bfloat16(), y), "x is torch.bfloat16")
    _rejects(lambda: m.forward(x, y.float()), "y is torch.float32")
    _rejects(lambda: m.forward(torch.zeros(5, 128, dtype=h)[:, ::2], y), "innermost")
    _rejects(lambda: m.forward(x, y[:1].expand(5, 8)), "overlap")
    _rejects(lambda: m.forward(x.to("meta"), y), "x is on meta")
    m.handle = None
    _rejects(lambda: m.forward(x, y), "closed")


def test_weights_are_checked():
    w, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.float16)
    _rejects(lambda: pi.Linear(w, s), "CUDA")
    _rejects(lambda: pi.Linear(w.float(), s), "w is torch.float32")
    _rejects(lambda: pi.Linear(w, s.T), "scales must be")
    _rejects(lambda: pi.Linear(w, s, bias=torch.zeros(9)), "bias must be [8]")
    _rejects(lambda: pi.Linear(w, None), "scales must be a torch tensor")
    _rejects(lambda: pi.Linear(w[0], s), "w must be")
    _rejects(lambda: pi.Linear(w[:, :8], s), "d_in=16 must be")


@pytest.mark.parametrize("act", ["f16", "bf16"])
@pytest.mark.parametrize("d_in, d_out", [(4096, 12288), (8192, 8192), (512, 100), (11008, 4096), (64, 8), (2048, 40000)])
def test_a_scratch_for_all_numbers_of_rows(d_in, d_out, act):
    """upto is the most of all smaller calls, and no call of fewer rows needs more than a larger one's, to be answered at all."""
    h, out, most, least = _Handle(d_in, d_out, act), ctypes.c_size_t(0), 0, 0
    for rows in list(range(60, 700)) + list(range(700, 9000, 37)):
        assert pi.LIB.pi_linear_scratch_bytes(ctypes.byref(h.raw), rows, ctypes.byref(out)) == 0
        most = max(most, out.value)
        if rows > 64 and act == "bf16":     # fp16 rows and their factors, as one range of columns needs them
            need = -(-rows * d_in * 2 // 256) * 256 + -(-rows * 4 // 256) * 256
            assert least <= need <= out.value
            least = need
            assert h.forward(rows=rows, x_stride=d_in, y_stride=d_out, scratch=FAKE, scratch_bytes=need - 1) == 2
            assert str(need) in pi.last_error()
        before = out.value
        assert pi.LIB.pi_linear_scratch_bytes_upto(ctypes.byref(h.raw), rows, ctypes.byref(out)) == 0
        assert before <= out.value
        if rows < 700:
            assert out.value == most
    m = _closed()
    m.handle = ctypes.pointer(h.raw)
    assert m.scratch_bytes(rows, upto=True) == out.value
    m.handle = None
    for bad in ((None, 1, out), (ctypes.byref(h.raw), -1, out), (ctypes.byref(h.raw), (1 << 24) + 1, out)):
        assert pi.LIB.pi_linear_scratch_bytes_upto(bad[0], bad[1], ctypes.byref(out)) == 1
    assert pi.LIB.pi_linear_scratch_bytes_upto(ctypes.byref(h.raw), 1, None) == 1
