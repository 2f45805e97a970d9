"""The attention cache's binding without a GPU: arguments at the edges of their types, and whose memory a stream holds."""

from types import SimpleNamespace

import pytest

from test_kv_cpu import GOOD, _args, _cache, _rejects

torch = pytest.importorskip("torch")
pi = pytest.importorskip("activation_sparse_decode_relu_amd")
