"""The attention cache without a GPU: the oracle against values fixed by hand, the C ABI's symbols and
refusals, and the binding's checks of its arguments."""

import ctypes
import os
import re
import subprocess
from types import SimpleNamespace

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pi = pytest.importorskip("activation_sparse_decode_relu_amd")
from activation_sparse_decode_relu_amd import kvcache as kvc  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "pi_kv.h")


# ---- the oracle ------------------------------------------------------------------------------------


@pytest.mark.parametrize("amax, code, e", [(448.0, "e4m3", 0), (448.1, "e4m3", 1), (224.0, "e4m3", -1),
                                           (127.0, "int8", 0), (127.01, "int8", 1), (63.5, "int8", -1), (0.0, "int8", -126),
                                           (1.0, "e4m3", -8), (1.0, "int8", -6), (2.0 ** -140, "e4m3", -126),
                                           (3.38e38, "e4m3", 120)])
def test_exponent(amax, code, e):
    assert oracle.kv_exponent(amax, code) == e


@pytest.mark.parametrize("x, e, code, want", [
    (1.06, 0, "e4m3", 1.0), (1.0625, 0, "e4m3", 1.0), (1.1875, 0, "e4m3", 1.25),      # ties go to even
    (0.0146, 0, "e4m3", 2 ** -6 * 0.875), (2 ** -10, 0, "e4m3", 0.0), (3 * 2 ** -10, 0, "e4m3", 2 ** -8),
    (447.0, 0, "e4m3", 448.0), (0.5, 0, "int8", 0.0), (1.5, 0, "int8", 2.0), (-2.5, 0, "int8", -2.0), (5.0, 1, "int8", 4.0),
    (-7.0, 1, "int8", -8.0)])
def test_round(x, e, code, want):
    assert float(oracle.kv_round(np.array(x), e, code)) == want


def test_round_matches_torch_e4m3():
    x = np.linspace(-448, 448, 20011).astype(np.float32)
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.kv_round(x, 0, "e4m3"), t)


def test_model_requantizes_and_keeps_other_blocks():
    m = oracle.KvModel(1, 1, "int8", "f16")
    m.append(np.full((3, 1, 1), 100.0))              # e = 0
    assert m.exps == [[0]] and np.all(m.values == 100.0)
    m.append(np.full((30, 1, 1), 333.0))             # 29 join block 0 (e = 2), one opens block 1
    assert m.exps == [[2], [2]]
    assert np.all(m.values[:3] == 100.0) and np.all(m.values[3:] == 332.0)     # 83 * 4
    m.append(np.array([[[np.nan]], [[np.inf]]]))
    assert m.exps[1] == [oracle.kv_exponent(65504.0, "int8")] and m.values[33, 0, 0] == 0.0


def test_visible():
    assert list(np.flatnonzero(oracle.kv_visible(9, 12, 3, 2))) == [0, 1, 7, 8, 9]
    assert list(np.flatnonzero(oracle.kv_visible(1, 12, 3, 2))) == [0, 1]
    assert list(np.flatnonzero(oracle.kv_visible(2, 4, 0, 7))) == [0, 1, 2]
    assert not oracle.kv_visible(-1, 4, 0, 4).any()


def test_attend_of_two_tokens():
    k = np.array([[[0.0]], [[np.log(3.0)]]])
    v = np.array([[[4.0]], [[8.0]]])
    out, lse, mass, _ = oracle.kv_attend(np.ones((1, 1, 1)), k, v, scale=1.0)
    assert out[0, 0, 0] == pytest.approx(7.0) and lse[0, 0] == pytest.approx(np.log(4.0)) and mass[0, 0, 0] == pytest.approx(7.0)
    out, lse, _, _ = oracle.kv_attend(np.ones((3, 1, 1)), k, v, scale=1.0)      # the first row stands before the cache
    assert np.all(out[0] == 0) and lse[0, 0] == -np.inf and out[1, 0, 0] == 4.0


def test_pages_fork_grow_compact():
    table, lens, refs = [[1, 3, -1], [-1, -1, -1], [5, -1, -1]], [40, 0, 32], [0, 1, 0, 1, 0, 1]
    oracle.kv_fork(table, lens, refs, [0], [1])
    assert table[1] == [1, 3, -1] and refs == [0, 2, 0, 2, 0, 1]
    copies, failed = oracle.kv_reserve(table, lens, refs, [1, 2], [1, 1], 32)
    assert copies == [(3, 0)] and failed == 0 and table == [[1, 3, -1], [1, 0, -1], [5, 2, -1]]
    assert lens == [40, 41, 33] and refs == [1, 2, 1, 1, 0, 1]
    oracle.kv_free(table, lens, refs, [0])
    assert refs == [1, 1, 1, 0, 0, 1] and oracle.kv_compact(table, refs) == [(5, 3)]
    assert table == [[-1, -1, -1], [1, 0, -1], [3, 2, -1]] and refs == [1, 1, 1, 1, 0, 0]
    assert oracle.kv_reserve(table, lens, refs, [1, 2], [24, 33], 32) == ([], 0)    # 65 and 66 tokens: 3 pages each
    assert lens == [0, 65, 66] and table[1:] == [[1, 0, 4], [3, 2, 5]]
    assert oracle.kv_reserve(table, lens, refs, [1, 2], [31, 31], 32) == ([], 1)    # 97 tokens need a fourth column


# ---- the C ABI -------------------------------------------------------------------------------------


def _declared():
    return sorted(set(re.findall(r"^\s*(?:pi_status|int32_t)\s+(pi_kv_\w+)\s*\(", open(HEADER).read(), re.M)))


def test_symbols():
    assert set(_declared()) == set(pi.KV_EXPORTED)
    for name in _declared():
        assert hasattr(pi.LIB, name), f"{name} is declared in pi_kv.h but not exported"
    assert pi.LIB.pi_kv_abi_version() == kvc.KV_ABI_VERSION


def test_header_is_plain_c(tmp_path):
    for cc, flags in (("gcc", ["-std=c99", "-xc"]), ("g++", ["-std=c++17", "-xc++"])):
        src = tmp_path / "use.c"
        src.write_text('#include "pi_kv.h"\nint main(void) { pi_kv_desc d; (void)d; return PI_KV_ABI_VERSION - 1; }\n')
        subprocess.run([cc, *flags, "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only", "-I",
                        os.path.join(ROOT, "include"), str(src)], check=True)


GOOD = dict(heads=8, kv_heads=2, head_dim=64, pages=9, page_tokens=64, max_seqs=3, max_seq_pages=4, layers=2)


@pytest.mark.parametrize("bad, status", [
    (dict(heads=7), 1), (dict(heads=0), 1), (dict(kv_heads=0), 1), (dict(heads=2048), 1), (dict(head_dim=0), 1),
    (dict(head_dim=80), 4), (dict(head_dim=256), 4), (dict(page_tokens=16), 1), (dict(page_tokens=48), 1),
    (dict(page_tokens=8192), 1), (dict(pages=0), 1), (dict(pages=(1 << 20) + 1), 1), (dict(layers=0), 1), (dict(max_seqs=0), 1),
    (dict(max_seq_pages=0), 1), (dict(max_seq_pages=1 << 25), 1), (dict(act_dtype=2), 1), (dict(code=-1), 1)])
def test_bad_descriptors(bad, status):
    with pytest.raises(pi.PiError) as e:
        pi.kv_workspace_bytes(pi.kv_desc(**{**GOOD, **bad}))
    assert e.value.status == status and pi.last_error()


def test_unknown_names():
    with pytest.raises(KeyError):
        pi.kv_desc(**GOOD, act_dtype="f32")
    with pytest.raises(KeyError):
        pi.kv_desc(**GOOD, code="int4")


FAKE = 0x10000


def _create(ws=FAKE, ws_bytes=None, **buf):
    d = pi.kv_desc(**GOOD)
    need = pi.kv_workspace_bytes(d)
    base = {name: FAKE for name, _ in kvc.KvBuffers._fields_}
    b = kvc.KvBuffers(**{**base, **buf})
    h = ctypes.c_void_p()
    st = pi.LIB.pi_kv_create(ctypes.byref(d), ctypes.byref(b), ws, need if ws_bytes is None else ws_bytes, None, ctypes.byref(h))
    return st, h


@pytest.mark.parametrize("buf", [dict(k=None), dict(v=FAKE + 8), dict(k_exp=None), dict(v_exp=None), dict(table=FAKE + 2),
                                 dict(lens=None), dict(refs=None), dict(failed=None)])
def test_create_refuses_bad_buffers(buf):
    st, h = _create(**buf)
    assert st == 1 and not h.value


def test_create_refuses_a_bad_workspace():
    need = pi.kv_workspace_bytes(pi.kv_desc(**GOOD))
    for ws, size in ((None, need), (FAKE + 16, need), (FAKE, need - 1)):
        assert _create(ws, size)[0] == 2


def test_null_handles():
    rows, batch, args = kvc.KvRows(FAKE, 64, 64), kvc.KvBatch(FAKE, FAKE, 1, 1), kvc.KvAttendArgs()
    r, b, a, lib = ctypes.byref(rows), ctypes.byref(batch), ctypes.byref(args), pi.LIB
    assert lib.pi_kv_append(None, 0, r, r, b, None) == 1
    assert lib.pi_kv_read(None, 0, r, r, b, None, None) == 1
    assert lib.pi_kv_attend(None, 0, a, b, None) == 1
    assert lib.pi_kv_reserve(None, FAKE, FAKE, 1, None) == 1
    assert lib.pi_kv_free(None, FAKE, 1, None) == 1
    assert lib.pi_kv_fork(None, FAKE, FAKE, 1, None) == 1
    assert lib.pi_kv_compact(None, None) == 1
    assert lib.pi_kv_destroy(None) == 1
    assert lib.pi_kv_create(None, None, None, 0, None, None) == 1


# ---- the binding -----------------------------------------------------------------------------------
# A cache whose handle is closed: an argument that got past the checks shows as "the cache is closed".

NULL_STREAM = SimpleNamespace(cuda_stream=0)


def _cache(act="f16"):
    c = object.__new__(pi.KVCache)
    c.desc = pi.kv_desc(**GOOD, act_dtype=act)
    c.handle, c.device, c._act = None, torch.device("cpu"), kvc._ACT_TORCH[c.desc.act_dtype]
    return c


def _rejects(fn, needle):
    with pytest.raises(pi.PiError) as e:
        fn()
    assert e.value.status == 1 and needle in str(e.value), str(e.value)


def _args(dtype=torch.float16):
    t = dict(q=torch.zeros(5, 8, 64, dtype=dtype), out=torch.zeros(5, 8, 64, dtype=dtype),
             k=torch.zeros(5, 2, 64, dtype=dtype), v=torch.zeros(5, 2, 64, dtype=dtype),
             seqs=torch.zeros(2, dtype=torch.int32), starts=torch.zeros(3, dtype=torch.int32))
    return SimpleNamespace(**t)


def test_good_arguments_reach_the_handle():
    for act, dtype in (("f16", torch.float16), ("bf16", torch.bfloat16)):
        c, a = _cache(act), _args(dtype)
        wide = torch.zeros(5, 12 * 64, dtype=dtype)
        strided = [t.unflatten(1, (-1, 64)) for t in wide.split([512, 128, 128], 1)]
        _rejects(lambda: c.attend(0, a.q, a.out, a.seqs, a.starts, 1, lse=torch.zeros(5, 8)), "closed")
        _rejects(lambda: c.attend(0, strided[0], a.out.transpose(0, 1).contiguous().transpose(0, 1), a.seqs, a.starts, 1), "closed")
        _rejects(lambda: c.append(0, strided[1], strided[2], a.seqs, a.starts), "closed")
        _rejects(lambda: c.append(0, a.k[:, :1].expand(5, 2, 64), a.v, a.seqs, a.starts), "closed")    # inputs may be expanded
        _rejects(lambda: c.read(0, a.k, a.v, a.seqs, a.starts, a.seqs), "closed")
        for fn in (lambda: c.reserve(a.seqs, a.seqs), lambda: c.free(a.seqs), lambda: c.fork(a.seqs, a.seqs)):
            _rejects(lambda: fn(), "closed")


@pytest.mark.parametrize("change, needle", [
    (dict(q=None), "q must be a torch tensor"), (dict(q=torch.zeros(5, 8, 64)), "q is torch.float32"),
    (dict(q=torch.zeros(5, 2, 64, dtype=torch.float16)), "q must be [rows][8][64]"),
    (dict(q=torch.zeros(5, 8, 128, dtype=torch.float16)[..., ::2]), "innermost"),
    (dict(q=torch.zeros(5, 8, 64, dtype=torch.float16, device="meta")), "q is on meta"),
    (dict(out=torch.zeros(4, 8, 64, dtype=torch.float16)), "out must be [5][8][64]"),
    (dict(out=torch.zeros(1, 8, 64, dtype=torch.float16).expand(5, 8, 64)), "overlap"),
    (dict(seqs=torch.zeros(2, dtype=torch.int64)), "seqs must be a contiguous int32"),
    (dict(seqs=[0, 1]), "seqs must be a torch tensor"),
    (dict(starts=torch.zeros(2, dtype=torch.int32)), "starts must have 3 entries"),
    (dict(starts=torch.zeros(6, dtype=torch.int32)[::2]), "starts must be a contiguous"),
    (dict(lse=torch.zeros(5, 8, dtype=torch.float16)), "lse is"), (dict(lse=torch.zeros(8, 5)), "lse must be")])
def test_attend_refusals(change, needle):
    c, a = _cache(), _args()
    kw = {**dict(q=a.q, out=a.out, seqs=a.seqs, starts=a.starts, max_new=1), **change}
    _rejects(lambda: c.attend(0, **kw), needle)


def test_store_and_page_refusals():
    c, a = _cache(), _args()
    _rejects(lambda: c.append(0, a.q, a.v, a.seqs, a.starts), "k must be")
    _rejects(lambda: c.append(0, a.k, a.v[:4], a.seqs, a.starts), "v must be [5]")
    _rejects(lambda: c.read(0, a.k, a.v.bfloat16(), a.seqs, a.starts), "v_out is")
    _rejects(lambda: c.read(0, a.k, a.v, a.seqs, a.starts, a.starts), "first must have 2")
    _rejects(lambda: c.read(0, a.k[:, :1].expand(5, 2, 64), a.v, a.seqs, a.starts), "overlap")
    _rejects(lambda: c.reserve(a.seqs, a.starts), "counts must have 2")
    _rejects(lambda: c.fork(a.seqs, a.starts), "dst must have 2")
    _rejects(lambda: c.free(a.seqs.float()), "seqs must be")


def test_a_cache_needs_a_gpu_and_sound_buffers():
    _rejects(lambda: pi.KVCache(**GOOD, device="cpu"), "CUDA")
    _rejects(lambda: pi.KVCache(**GOOD, device="cpu", buffers=dict(lens=torch.zeros(3))), "lens is torch.float32")
    _rejects(lambda: pi.KVCache(**GOOD, device="cpu", buffers=dict(refs=torch.zeros(8, dtype=torch.int32))), "refs must be [9]")
    _rejects(lambda: pi.KVCache(**GOOD, device="cpu", buffers=dict(foo=1)), "unknown buffer")
