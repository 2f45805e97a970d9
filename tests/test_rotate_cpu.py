"""Rotation by position without a GPU: the frequencies, the C ABI's symbols and refusals, and the binding's checks."""

import ctypes
import math
import os
import re
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")
pi = pytest.importorskip("activation_sparse_decode_relu_amd")
from activation_sparse_decode_relu_amd import kvcache as kvc  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000


def test_symbols():
    text = open(os.path.join(ROOT, "include", "pi_kv.h")).read()
    names = set(re.findall(r"^\s*pi_status\s+(pi_rope_\w+)\s*\(", text, re.M))
    assert names == set(pi.ROPE_EXPORTED) and all(hasattr(pi.LIB, n) for n in names)


def test_plain_frequencies():
    f = pi.Rope(128).freqs()
    assert len(f) == 64 and f[0] == 1.0 and f[32] == pytest.approx(0.01, rel=1e-14)
    assert f == pytest.approx([10000.0 ** (-i / 64) for i in range(64)], rel=1e-14)
    assert pi.Rope(64, rot_dims=16, base=500000.0).freqs() == pytest.approx([500000.0 ** (-i / 8) for i in range(8)], rel=1e-14)
    assert pi.Rope(64, rot_dims=0).freqs() == []


def test_scaled_frequencies():
    f = pi.Rope(128, rot_dims=64).freqs()
    assert pi.Rope(128, rot_dims=64, scaling="linear", factor=4.0).freqs() == pytest.approx([x / 4 for x in f], rel=1e-14)
    ntk = pi.Rope(128, rot_dims=64, scaling="ntk", factor=8.0).freqs()
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(f[-1] / 8, rel=1e-13)     # the slowest is stretched by the factor
    bands = pi.Rope(128, rot_dims=64, scaling="bands", factor=8.0, original=4096, low=1.0, high=4.0).freqs()
    for x, y in zip(f, bands):
        turns = 4096 * x / (2 * math.pi)
        assert turns < 4 or y == x
        assert turns > 1 or y == pytest.approx(x / 8, rel=1e-14)
        assert x / 8 <= y * (1 + 1e-14) and y <= x
    # half way between the bands
    mid = pi.Rope(64, 16, scaling="bands", base=1.0, factor=3.0, original=2 * math.pi * 2.5, low=1.0, high=4.0).freqs()
    assert mid == pytest.approx([0.5 + 0.5 / 3] * 8, rel=1e-14)


def test_given_frequencies():
    given = [0.0, 1e-9, 0.1, 0.2, 0.3, 1.0, 2.0, math.pi]
    assert pi.Rope(64, 16, freqs=given).freqs() == given


@pytest.mark.parametrize("bad, status", [
    (dict(head_dim=80), 4), (dict(rot_dims=24), 4), (dict(rot_dims=15), 1), (dict(rot_dims=80), 1), (dict(rot_dims=-16), 1),
    (dict(layout=2), 1), (dict(scaling=4), 1), (dict(base=0.5), 1), (dict(base=math.nan), 1), (dict(base=math.inf), 1),
    (dict(gain=0.0), 1), (dict(gain=math.inf), 1), (dict(gain=1e39), 1), (dict(scaling="linear", factor=0.5), 1),
    (dict(scaling="ntk", factor=math.nan), 1), (dict(scaling="bands", factor=2.0), 1),
    (dict(scaling="bands", factor=2.0, original=64, low=3.0, high=3.0), 1),
    (dict(scaling="bands", factor=2.0, original=64, low=-1.0), 1), (dict(rot_dims=16, freqs=[0.1] * 7 + [3.2]), 1),
    (dict(rot_dims=16, freqs=[-0.1] * 8), 1), (dict(rot_dims=16, freqs=[math.nan] * 8), 1), (dict(rot_dims=16, freqs=[1.0] * 7), 1),
    (dict(rot_dims=16, freqs=[1.0] * 8, scaling="linear"), 1), (dict(rot_dims=1 << 32), 1)])
def test_bad_ropes(bad, status):
    with pytest.raises(pi.PiError) as e:
        pi.Rope(**{**dict(head_dim=64), **bad})
    assert e.value.status == status


def test_unknown_names():
    with pytest.raises(KeyError):
        pi.Rope(64, layout="neox")
    with pytest.raises(KeyError):
        pi.Rope(64, scaling="dynamic")


def test_null_handles():
    out, h = (ctypes.c_double * 64)(), ctypes.c_void_p()
    assert pi.LIB.pi_rope_create(None, ctypes.byref(h)) == 1 and pi.LIB.pi_rope_create(None, None) == 1
    assert pi.LIB.pi_rope_destroy(None) == 1 and pi.LIB.pi_rope_freqs(None, out) == 1
    args, batch = kvc.KvRotateArgs(), kvc.KvBatch(FAKE, FAKE, 1, 1)
    assert pi.LIB.pi_kv_rotate(None, None, ctypes.byref(args), ctypes.byref(batch), None) == 1


# ---- a handle over addresses that nobody reads: every refusal comes before anything is enqueued ---------


class _Raw(ctypes.Structure):
    _fields_ = [("desc", kvc.KvDesc), ("buf", kvc.KvBuffers), ("ws", ctypes.c_void_p), ("layout", ctypes.c_size_t * 8)]


def _rotate(rope_dim=64, n=1, rows=2, **change):
    raw = _Raw(pi.kv_desc(8, 2, 64, 9, 64, 3, 4), kvc.KvBuffers(*[FAKE] * 9), FAKE)
    r = kvc.KvRows(FAKE, 640, 64)
    a = {**dict(q=r, q_out=r, k=r, k_out=r, q_norm=FAKE, k_norm=FAKE, positions=None, eps=1e-6), **change}
    rope = pi.Rope(rope_dim)
    batch = kvc.KvBatch(FAKE, FAKE, n, rows)
    st = pi.LIB.pi_kv_rotate(ctypes.byref(raw), rope.handle, ctypes.byref(kvc.KvRotateArgs(**a)), ctypes.byref(batch), None)
    return st, pi.last_error()


@pytest.mark.parametrize("change", [
    dict(rope_dim=128), dict(n=0), dict(n=4), dict(rows=-1), dict(eps=0.0), dict(eps=float("nan")), dict(q_norm=FAKE + 8),
    dict(k_norm=FAKE + 2), dict(positions=FAKE + 2), dict(q=kvc.KvRows(None, 640, 64)), dict(q_out=kvc.KvRows(FAKE + 8, 640, 64)),
    dict(k=kvc.KvRows(FAKE, 644, 64)), dict(k_out=kvc.KvRows(FAKE, -640, 64))])
def test_refusals(change):
    st, why = _rotate(**change)
    assert st == 1 and why


def test_no_rows_enqueue_nothing():
    none = kvc.KvRows(None, 0, 0)
    assert _rotate(rows=0, q=none, q_out=none, k=none, k_out=none)[0] == 0


# ---- the binding -----------------------------------------------------------------------------------


def _cache(act="f16"):
    c = object.__new__(pi.KVCache)
    c.desc = pi.kv_desc(heads=8, kv_heads=2, head_dim=64, pages=9, page_tokens=64, max_seqs=3, max_seq_pages=4, act_dtype=act)
    c.handle, c.device, c._act = None, torch.device("cpu"), kvc._ACT_TORCH[c.desc.act_dtype]
    return c


def _args(**change):
    h = torch.float16
    q, k = torch.zeros(5, 8, 64, dtype=h), torch.zeros(5, 2, 64, dtype=h)
    base = dict(rope=pi.Rope(64), q=q, q_out=q, k=k, k_out=k, seqs=torch.zeros(2, dtype=torch.int32),
                starts=torch.zeros(3, dtype=torch.int32))
    return SimpleNamespace(**{**base, **change}).__dict__


@pytest.mark.parametrize("change, needle", [
    ({}, "closed"), (dict(positions=torch.zeros(5, dtype=torch.int32)), "closed"),
    (dict(q_norm=torch.zeros(64, dtype=torch.float16)), "closed"), (dict(rope=None), "rope must be a Rope"),
    (dict(q=torch.zeros(5, 8, 64)), "q is torch.float32"), (dict(k=torch.zeros(4, 2, 64, dtype=torch.float16)), "k must be [5]"),
    (dict(q_out=torch.zeros(5, 2, 64, dtype=torch.float16)), "q_out must be [5][8][64]"),
    (dict(k_out=torch.zeros(1, 2, 64, dtype=torch.float16).expand(5, 2, 64)), "k_out: its rows overlap"),
    (dict(q_norm=torch.zeros(64)), "q_norm is"), (dict(k_norm=torch.zeros(8, 64, dtype=torch.float16)), "k_norm must be [64]"),
    (dict(positions=torch.zeros(4, dtype=torch.int32)), "positions must have 5"),
    (dict(positions=torch.zeros(5, dtype=torch.int64)), "positions must be a contiguous int32"),
    (dict(starts=torch.zeros(2, dtype=torch.int32)), "starts must have 3")])
def test_binding(change, needle):
    with pytest.raises(pi.PiError) as e:
        _cache().rotate(**_args(**change))
    assert e.value.status == 1 and needle in str(e.value), str(e.value)


@pytest.mark.parametrize("gain", [1e-50, -1e-50, -1.0, 1e39, math.nan])
def test_gains_outside_fp32(gain):
    """A gain that fp32 holds as 0 would clear every turned dim."""
    with pytest.raises(pi.PiError) as e:
        pi.Rope(64, gain=gain)
    assert e.value.status == 1 and "gain" in str(e.value)
    assert pi.Rope(64, gain=1e-38).desc.gain == 1e-38
