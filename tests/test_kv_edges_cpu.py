"""The attention cache's binding without a GPU: arguments at the edges of their types, and whose memory a stream holds."""

import contextlib
import ctypes
from types import SimpleNamespace

import pytest

from test_kv_cpu import GOOD, _args, _cache, _rejects

torch = pytest.importorskip("torch")
pi = pytest.importorskip("activation_sparse_decode_relu_amd")
from activation_sparse_decode_relu_amd import kvcache as kvc  # noqa: E402


@pytest.mark.parametrize("value", [1 << 31, 1 << 32, (1 << 32) + 1, -(1 << 31) - 1, -(1 << 32)])
def test_numbers_past_32_bits_are_refused(value):
    """They do not come round to a layer, a window or a size that is valid."""
    c, a = _cache(), _args()
    _rejects(lambda: c.append(value, a.k, a.v, a.seqs, a.starts), "layer")
    _rejects(lambda: c.read(value, a.k, a.v, a.seqs, a.starts), "layer")
    _rejects(lambda: c.attend(value, a.q, a.out, a.seqs, a.starts, 1), "layer")
    if value > 0:
        many = a.k[:1].expand(value, 2, 64)
        _rejects(lambda: c.append(0, many, many, a.seqs, a.starts), "rows")
    for name in ("max_new", "window", "sinks"):
        _rejects(lambda: c.attend(0, a.q, a.out, a.seqs, a.starts, **{**dict(max_new=1), name: value}), name)
    for name in GOOD:
        _rejects(lambda: pi.kv_desc(**{**GOOD, name: value}), name)
    for name in ("act_dtype", "code"):
        _rejects(lambda: pi.kv_desc(**GOOD, **{name: value}), name)


OWNED = ("k", "v", "k_exp", "v_exp", "table", "lens", "refs", "failed", "refused", "workspace")


class _Memory:
    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream)


def test_a_stream_holds_the_caches_own_memory():
    """A cache that is dropped while a stream still works on it keeps its memory until that stream is past its calls."""
    c, side, other = _cache(), SimpleNamespace(cuda_stream=5), SimpleNamespace(cuda_stream=9)
    c._met, mine = set(), {name: _Memory() for name in OWNED}
    for name, m in mine.items():
        setattr(c, name, m)
    arg = _Memory()
    assert c._stream(side, (arg, None)) == 5
    assert arg.streams == [side]
    for name, m in mine.items():
        assert m.streams == [side], name
    c._stream(other, ())
    c._stream(side, (arg,))
    assert arg.streams == [side, side]                  # another call's tensor, as far as the cache knows
    for name, m in mine.items():
        assert m.streams[:2] == [side, other], name


# ---- devices -----------------------------------------------------------------------------------------------


class _Second:
    """The second of two devices; tensors of any count as its own."""
    index = 1

    def __eq__(self, other):
        return True

    def __ne__(self, other):
        return False


@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_the_caches_device(monkeypatch, current):
    """Whatever device is the current one, the library is called with the cache's, and the current one is left as it was."""
    now, calls = [current], []

    @contextlib.contextmanager
    def device(index):
        before, now[0] = now[0], index
        yield
        now[0] = before

    def recorder(name):
        def fn(*args):
            calls.append((name, now[0]))
            return 0
        return fn

    names = ("append", "read", "attend", "reserve", "free", "fork", "compact")
    monkeypatch.setattr(kvc, "LIB", SimpleNamespace(**{f"pi_kv_{n}": recorder(n) for n in names}))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index=None: SimpleNamespace(cuda_stream=0))
    c, a = _cache(), _args()
    c.device, c.handle, c._met, c._lone = _Second(), ctypes.c_void_p(), set(), False
    for name in OWNED:
        setattr(c, name, _Memory())
    c.append(0, a.k, a.v, a.seqs, a.starts)
    c.read(0, a.k, a.v, a.seqs, a.starts)
    c.attend(0, a.q, a.out, a.seqs, a.starts, 1)
    c.reserve(a.seqs, a.seqs)
    c.free(a.seqs)
    c.fork(a.seqs, a.seqs)
    c.compact()
    assert calls == [(n, 1) for n in names] and now == [current]
