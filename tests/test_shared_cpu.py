"""Attention of groups that share their beginning, without a GPU: refusals of the C ABI and of the binding."""

import ctypes
import subprocess

import pytest

torch = pytest.importorskip("torch")
pi = pytest.importorskip("activation_sparse_decode_relu_amd")
from activation_sparse_decode_relu_amd import kvcache as kvc  # noqa: E402

FAKE = 0x10000


class _Raw(ctypes.Structure):   # a handle over addresses that nobody reads: every refusal comes before anything is enqueued
    _fields_ = [("desc", kvc.KvDesc), ("buf", kvc.KvBuffers), ("ws", ctypes.c_void_p), ("layout", ctypes.c_size_t * 8)]


def _raw():
    return _Raw(pi.kv_desc(8, 2, 64, 9, 64, 3, 4), kvc.KvBuffers(*[FAKE] * 9), FAKE)


NEED = 256 * 4 * 8 * 68 * 4      # 4 rows of 4 query heads: few workgroups, so the shared tokens are split over up to 512 / 2


def test_state_bytes():
    out, raw = ctypes.c_size_t(0), _raw()
    assert pi.LIB.pi_kv_state_bytes(ctypes.byref(raw), 4, ctypes.byref(out)) == 0 and out.value == NEED
    assert pi.LIB.pi_kv_state_bytes(ctypes.byref(raw), 0, ctypes.byref(out)) == 0 and out.value == 0
    assert pi.LIB.pi_kv_state_bytes(ctypes.byref(raw), -1, ctypes.byref(out)) == 1
    assert pi.LIB.pi_kv_state_bytes(ctypes.byref(raw), 4, None) == 1
    assert pi.LIB.pi_kv_state_bytes(None, 4, ctypes.byref(out)) == 1


def _attend(layer=0, n=3, rows=4, handle=True, **change):
    raw, r = _raw(), kvc.KvRows(FAKE, 512, 64)
    a = dict(q=r, out=r, lse=None, max_new=2, window=0, sinks=0, scale=0.125)
    s = dict(groups=FAKE, plan=FAKE, state=FAKE, state_bytes=NEED, n_groups=2, max_rows=3)
    a.update({k: v for k, v in change.items() if k in a})
    s.update({k: v for k, v in change.items() if k in s})
    return pi.LIB.pi_kv_attend_shared(ctypes.byref(raw) if handle else None, layer, ctypes.byref(kvc.KvAttendArgs(**a)),
                                      ctypes.byref(kvc.KvSharedArgs(**s)), ctypes.byref(kvc.KvBatch(FAKE, FAKE, n, rows)), None)


@pytest.mark.parametrize("change, status", [
    (dict(handle=False), 1), (dict(layer=1), 1), (dict(n=0), 1), (dict(n=4), 1), (dict(rows=-1), 1), (dict(max_new=0), 1),
    (dict(max_new=5), 1), (dict(window=8), 4), (dict(sinks=1), 4), (dict(window=-1), 1), (dict(scale=0.0), 1), (dict(groups=None), 1),
    (dict(groups=FAKE + 2), 1), (dict(plan=None), 1), (dict(n_groups=0), 1), (dict(n_groups=4), 1), (dict(max_rows=0), 1),
    (dict(max_rows=5), 1), (dict(state=None), 2), (dict(state=FAKE + 8), 2), (dict(state_bytes=NEED - 1), 2),
    (dict(q=kvc.KvRows(None, 512, 64)), 1), (dict(out=kvc.KvRows(FAKE + 2, 512, 64)), 1), (dict(lse=FAKE + 1), 1)])
def test_refusals(change, status):
    assert _attend(**change) == status and pi.last_error()


def test_no_rows_enqueue_nothing():
    none = kvc.KvRows(None, 0, 0)
    assert _attend(rows=0, q=none, out=none, max_new=0, max_rows=0, state=None, state_bytes=0) == 0


def test_share_refusals():
    raw, b = _raw(), kvc.KvBatch(FAKE, FAKE, 3, 4)

    def share(h=raw, batch=b, groups=FAKE, n=2, plan=FAKE):
        return pi.LIB.pi_kv_share(None if h is None else ctypes.byref(h), None if batch is None else ctypes.byref(batch),
                                  groups, n, plan, None)

    assert [share(h=None), share(batch=None), share(groups=None), share(groups=FAKE + 1), share(n=0), share(n=4), share(plan=None),
            share(plan=FAKE + 2), share(batch=kvc.KvBatch(FAKE, FAKE, 4, 4)), share(batch=kvc.KvBatch(None, FAKE, 3, 4))] == [1] * 10


# ---- the binding -----------------------------------------------------------------------------------


def _cache():
    c = object.__new__(pi.KVCache)
    c.desc = pi.kv_desc(heads=8, kv_heads=2, head_dim=64, pages=9, page_tokens=64, max_seqs=3, max_seq_pages=4)
    c.handle, c.device, c._act = None, torch.device("cpu"), torch.float16
    return c


def _ints(n):
    return torch.zeros(n, dtype=torch.int32)


@pytest.mark.parametrize("change, needle", [
    ({}, "closed"), (dict(groups=_ints(1)), "groups must have 2 to 4"), (dict(groups=_ints(5)), "groups must have 2 to 4"),
    (dict(plan=_ints(4)), "plan must have 5"), (dict(groups=torch.zeros(3)), "groups must be a contiguous int32"),
    (dict(starts=_ints(3)), "starts must have 4"), (dict(q=torch.zeros(5, 8, 64)), "q is torch.float32"),
    (dict(out=torch.zeros(4, 8, 64, dtype=torch.float16)), "out must be [5]"), (dict(lse=torch.zeros(5, 2)), "lse must be"),
    (dict(max_rows=1 << 32), "does not fit")])
def test_binding(change, needle):
    q = torch.zeros(5, 8, 64, dtype=torch.float16)
    a = {**dict(layer=0, q=q, out=q.clone(), seqs=_ints(3), starts=_ints(4), groups=_ints(3), plan=_ints(5), max_new=2,
                max_rows=3), **change}
    with pytest.raises(pi.PiError) as e:
        _cache().attend_shared(**a)
    assert e.value.status == 1 and needle in str(e.value), str(e.value)


def test_share_binding():
    for groups, plan, needle in ((_ints(3), _ints(5), "closed"), (_ints(3), _ints(6), "plan must have 5"),
                                 (_ints(6), _ints(5), "groups must have")):
        with pytest.raises(pi.PiError) as e:
            _cache().share(_ints(3), _ints(4), groups, plan)
        assert needle in str(e.value)


# ---- which blocks the kernel of few rows looks up --------------------------------------------------------

SPANS = r"""
#include "kv_items.h"

// Lanes look up blocks 0 .. 63 of a sequence's span, the last again where there are fewer: none may lie past the table's
// columns, whatever the plan says, and with a plan that fits, the span is what the sequence holds behind it.
int main() {
  pik::KvSharedArgs A{};
  const int cap = 4;   // blocks that the table has room for
  for (int len = 0; len <= 32 * cap; ++len)
    for (int rows = 1; rows <= len + 3; ++rows)
      for (int shared = 0; shared <= 32 * cap; shared += 32) {
        const pik::Span s = pik::item_span<pik::ATTEND_OWN>(A, len, shared, len - rows, len - 1);
        for (int lane = 0; lane < 64; ++lane) {
          const int last = s.count() > 0 ? s.count() - 1 : 0, block = s.block(lane < last ? lane : last);
          if (block < 0 || block >= cap) return 1;
        }
        if (shared <= len - rows && (s.block(0) != shared / 32 || s.end != (len + 31) / 32)) return 2;
      }
  return 0;
}
"""


def test_no_block_past_the_table(tmp_path):
    from activation_sparse_decode_relu_amd._build import CSRC, hipcc
    (tmp_path / "spans.hip").write_text(SPANS)
    subprocess.run([hipcc(), "--cuda-host-only", "-std=c++17", "-O1", "-I", CSRC, str(tmp_path / "spans.hip"), "-o",
                    str(tmp_path / "spans")], check=True, timeout=100)
    assert subprocess.run([str(tmp_path / "spans")], timeout=20).returncode == 0


@pytest.mark.parametrize("heads, kv_heads, dim", [(8, 2, 64), (64, 8, 128), (128, 8, 64), (32, 32, 128), (1024, 1, 64), (300, 300, 64)])
def test_a_state_for_all_numbers_of_rows(heads, kv_heads, dim):
    """What a number of rows is said to take serves fewer rows too, whose shared tokens may be taken in more parts."""
    raw = _Raw(pi.kv_desc(heads, kv_heads, dim, 9, 64, 3, 4), kvc.KvBuffers(*[FAKE] * 9), FAKE)
    out, least = ctypes.c_size_t(0), 0
    group = heads // kv_heads
    for rows in range(0, 3000):
        items = (rows * group + 127) // 128 * kv_heads
        parts = 512 // items if 0 < items <= 256 else 1
        assert pi.LIB.pi_kv_state_bytes(ctypes.byref(raw), rows, ctypes.byref(out)) == 0
        least = max(least, parts * rows * heads * (dim + 4) * 4)     # of one group's sequences
        assert out.value == least, rows
