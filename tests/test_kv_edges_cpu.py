"""The attention cache's binding without a GPU: arguments at the edges of their types, and whose memory a stream holds."""

from types import SimpleNamespace

import pytest

from test_kv_cpu import GOOD, _args, _cache, _rejects

torch = pytest.importorskip("torch")
pi = pytest.importorskip("activation_sparse_decode_relu_amd")


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
