"""Activation-sparse ReLU FFN decode, attention over an 8-bit paged cache, and products with 4-bit weights, on MI355X
(gfx950).

The compute lives in libpi_ffn.so (hand-written HIP kernels behind the C ABIs in
include/pi_ffn.h, include/pi_kv.h and include/pi_linear.h); this package is its thin Python binding.
"""

from .binding import (  # noqa: F401
    DTYPES,
    EXPORTED,
    FFNLayer,
    LIB,
    LIB_PATH,
    MODES,
    PHASES,
    PiDesc,
    PiError,
    PiWeights,
    check,
    last_error,
    make_desc,
    probe_read,
    upload_layer,
    workspace_bytes,
)
from .kvcache import KV_EXPORTED, ROPE_EXPORTED, KVCache, Rope, kv_desc, kv_workspace_bytes  # noqa: F401
from .linear import LINEAR_EXPORTED, Linear, linear_desc, linear_packed_bytes  # noqa: F401
