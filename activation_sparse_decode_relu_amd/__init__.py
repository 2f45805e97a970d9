"""Activation-sparse ReLU FFN decode, and attention over an 8-bit paged cache, on MI355X (gfx950).

The compute lives in libpi_ffn.so (hand-written HIP kernels behind the C ABIs in
include/pi_ffn.h and include/pi_kv.h); this package is its thin Python binding.
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
from .kvcache import KV_EXPORTED, KVCache, kv_desc, kv_workspace_bytes  # noqa: F401
