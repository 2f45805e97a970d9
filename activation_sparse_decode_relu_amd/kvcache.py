"""ctypes binding of the 8-bit paged attention cache (the C ABI declared in include/pi_kv.h).

Argument marshalling only, as in binding.py: every tensor is checked on the host before its address
is passed, a failed check raises PiError(PI_ERR_INVALID) and nothing is enqueued.  Calls only enqueue
work on the current stream (or the given one); nothing here waits for the GPU except check_failed.
"""

from __future__ import annotations

import ctypes

import torch

from .binding import LIB, PI_ERR_INVALID, PiError, _invalid, check

PI_KV_F16, PI_KV_BF16 = range(2)
PI_KV_E4M3, PI_KV_INT8 = range(2)
KV_BLOCK = 32
KV_ABI_VERSION = 3   # PI_KV_ABI_VERSION of the header this binding follows

ACTS = {"f16": PI_KV_F16, "bf16": PI_KV_BF16}
CODES = {"e4m3": PI_KV_E4M3, "int8": PI_KV_INT8}
_ACT_TORCH = {PI_KV_F16: torch.float16, PI_KV_BF16: torch.bfloat16}

KV_EXPORTED = ("pi_kv_abi_version", "pi_kv_workspace_bytes", "pi_kv_create", "pi_kv_destroy", "pi_kv_append",
               "pi_kv_read", "pi_kv_attend", "pi_kv_reserve", "pi_kv_free", "pi_kv_fork", "pi_kv_compact", "pi_kv_rotate",
               "pi_kv_share", "pi_kv_state_bytes", "pi_kv_attend_shared")
ROPE_EXPORTED = ("pi_rope_create", "pi_rope_destroy", "pi_rope_freqs")
LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3}

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class KvDesc(ctypes.Structure):
    _fields_ = [(name, _i32) for name in ("heads", "kv_heads", "head_dim", "page_tokens", "pages", "layers",
                                          "max_seqs", "max_seq_pages", "act_dtype", "code")]


class KvBuffers(ctypes.Structure):
    _fields_ = [(name, _vp) for name in ("k", "v", "k_exp", "v_exp", "table", "lens", "refs", "failed", "refused")]


_OWNED = tuple(name for name, _ in KvBuffers._fields_) + ("workspace",)   # a cache's tensors


class KvBatch(ctypes.Structure):
    _fields_ = [("seqs", _vp), ("starts", _vp), ("n", _i32), ("rows", _i32)]


class KvRows(ctypes.Structure):
    _fields_ = [("data", _vp), ("token_stride", _i64), ("head_stride", _i64)]


class KvAttendArgs(ctypes.Structure):
    _fields_ = [("q", KvRows), ("out", KvRows), ("lse", _vp), ("max_new", _i32), ("window", _i32), ("sinks", _i32),
                ("scale", ctypes.c_float)]


class RopeDesc(ctypes.Structure):
    _fields_ = ([(name, _i32) for name in ("head_dim", "rot_dims", "layout", "scaling")] +
                [(name, ctypes.c_double) for name in ("base", "factor", "original", "low", "high", "gain")] +
                [("freqs", ctypes.POINTER(ctypes.c_double))])


class KvRotateArgs(ctypes.Structure):
    _fields_ = [("q", KvRows), ("q_out", KvRows), ("k", KvRows), ("k_out", KvRows), ("q_norm", _vp), ("k_norm", _vp),
                ("positions", _vp), ("eps", ctypes.c_float)]


class KvSharedArgs(ctypes.Structure):
    _fields_ = [("groups", _vp), ("plan", _vp), ("state", _vp), ("state_bytes", ctypes.c_size_t), ("n_groups", _i32),
                ("max_rows", _i32)]


def _declare() -> None:
    p = ctypes.POINTER
    sigs = dict(pi_kv_workspace_bytes=[p(KvDesc), p(ctypes.c_size_t)],
                pi_kv_create=[p(KvDesc), p(KvBuffers), _vp, ctypes.c_size_t, _vp, p(_vp)],
                pi_kv_destroy=[_vp],
                pi_kv_append=[_vp, _i32, p(KvRows), p(KvRows), p(KvBatch), _vp],
                pi_kv_read=[_vp, _i32, p(KvRows), p(KvRows), p(KvBatch), _vp, _vp],
                pi_kv_attend=[_vp, _i32, p(KvAttendArgs), p(KvBatch), _vp],
                pi_kv_reserve=[_vp, _vp, _vp, _i32, _vp],
                pi_kv_free=[_vp, _vp, _i32, _vp],
                pi_kv_fork=[_vp, _vp, _vp, _i32, _vp],
                pi_kv_compact=[_vp, _vp],
                pi_kv_rotate=[_vp, _vp, p(KvRotateArgs), p(KvBatch), _vp],
                pi_kv_share=[_vp, p(KvBatch), _vp, _i32, _vp, _vp],
                pi_kv_state_bytes=[_vp, _i32, p(ctypes.c_size_t)],
                pi_kv_attend_shared=[_vp, _i32, p(KvAttendArgs), p(KvSharedArgs), p(KvBatch), _vp],
                pi_rope_create=[p(RopeDesc), p(_vp)],
                pi_rope_destroy=[_vp],
                pi_rope_freqs=[_vp, p(ctypes.c_double)])
    for name, args in sigs.items():
        fn = getattr(LIB, name)
        fn.restype, fn.argtypes = ctypes.c_int, args
    LIB.pi_kv_abi_version.restype, LIB.pi_kv_abi_version.argtypes = _i32, []
    got = LIB.pi_kv_abi_version()
    if got != KV_ABI_VERSION:
        raise ImportError(f"the library's attention cache has ABI version {got}, this binding expects {KV_ABI_VERSION}; "
                          "rebuild it")


_declare()
_byref = ctypes.byref


def _in32(**numbers) -> None:
    """Refuse numbers that the C ABI takes in 32 bits and that do not fit: ctypes would cut them."""
    for name, value in numbers.items():
        if not -0x80000000 <= value <= 0x7fffffff:
            raise _invalid(f"{name}={value} does not fit in 32 bits")


def kv_desc(heads, kv_heads, head_dim, pages, page_tokens, max_seqs, max_seq_pages, layers=1, act_dtype="f16",
            code="e4m3") -> KvDesc:
    act = ACTS[act_dtype] if isinstance(act_dtype, str) else int(act_dtype)
    c = CODES[code] if isinstance(code, str) else int(code)
    sizes = dict(heads=heads, kv_heads=kv_heads, head_dim=head_dim, page_tokens=page_tokens, pages=pages, layers=layers,
                 max_seqs=max_seqs, max_seq_pages=max_seq_pages, act_dtype=act, code=c)
    sizes = {name: int(value) for name, value in sizes.items()}
    _in32(**sizes)
    return KvDesc(*sizes.values())


def kv_workspace_bytes(desc: KvDesc) -> int:
    out = ctypes.c_size_t(0)
    check(LIB.pi_kv_workspace_bytes(_byref(desc), _byref(out)))
    return int(out.value)


class Rope:
    """The rotation of a head's first rot_dims dims (all of them unless given) by position, for KVCache.rotate.

    Pair i turns by base^(-2 i / rot_dims) a position; layout "half" pairs dims i and i + rot_dims / 2, "interleaved"
    2 i and 2 i + 1.  For contexts longer than the trained ones the frequencies are scaled by `factor`: "linear" (all of
    them), "ntk" (a larger base), "bands" (by the turns a pair makes within the `original` length: none of it from
    `high` turns on, all of it up to `low`; pi_kv.h has the formulas).  `gain` multiplies cosines and sines.  `freqs`
    (rot_dims / 2 numbers, radians a position) takes the place of base and scaling.  Host memory only.
    """

    def __init__(self, head_dim, rot_dims=None, layout="half", base=10000.0, scaling="none", factor=1.0, original=0.0,
                 low=1.0, high=32.0, gain=1.0, freqs=None):
        self.handle = None
        whole = dict(head_dim=head_dim, rot_dims=head_dim if rot_dims is None else rot_dims,
                     layout=LAYOUTS[layout] if isinstance(layout, str) else layout,
                     scaling=SCALINGS[scaling] if isinstance(scaling, str) else scaling)
        whole = {name: int(value) for name, value in whole.items()}
        _in32(**whole)
        self.desc = d = RopeDesc(*whole.values(), base, factor, original, low, high, gain, None)
        if freqs is not None:
            freqs = [float(f) for f in freqs]
            if len(freqs) != d.rot_dims // 2:
                raise _invalid(f"freqs must have rot_dims / 2 = {d.rot_dims // 2} entries, got {len(freqs)}")
            d.freqs = (ctypes.c_double * len(freqs))(*freqs)
        handle = _vp()
        check(LIB.pi_rope_create(_byref(d), _byref(handle)))
        self.handle = handle

    def freqs(self) -> list:
        """The frequencies as scaled, in radians a position."""
        out = (ctypes.c_double * max(self.desc.rot_dims // 2, 1))()
        check(LIB.pi_rope_freqs(self.handle, out))
        return list(out)[:self.desc.rot_dims // 2]

    def __del__(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            LIB.pi_rope_destroy(self.handle)
            self.handle = None


class KVCache:
    """A paged cache of keys and values in 8-bit codes, the attention that reads it, and what brings queries and keys there.

    One object holds every layer's pages; the table, the lengths and the reference counts are shared by
    the layers.  All of them are device tensors that the caller may read or set between calls:

        k, v           uint8 [layers][pages][kv_heads * page_tokens * head_dim]   codes (layout: pi_kv.h)
        k_exp, v_exp   uint8 [layers][pages][kv_heads * page_tokens / 32]         exponents + 127
        table          int32 [max_seqs][max_seq_pages]    pages of each sequence, -1 where there is none
        lens           int32 [max_seqs]                   tokens of each sequence
        refs           int32 [pages]                      table entries that name a page; 0 = free
        failed         int32 [1]                          sequences that reserve could not grow
        refused        int32 [max_seqs]                   lens + 1 of each of them until it grows, else 0

    `buffers` may bring any of them; the others are made here, empty.  A step of a decode loop is

        cache.reserve(seqs, ones)                     # a token each: pages, and lens += 1
        for layer in range(layers):
            cache.append(layer, k, v, seqs, starts)
            cache.attend(layer, q, out, seqs, starts, max_new=1)

    seqs (int32 [n]) names rows of the table, and starts (int32 [n + 1]) says which rows of q, k and v are
    whose: those of seqs[i] are [starts[i], starts[i + 1]).  Tensors of tokens are [rows][heads][head_dim],
    with any strides that are multiples of 8 elements (a slice of a fused projection, say), the innermost
    contiguous.  Calls share one workspace: serialise them on one stream, or order the streams.
    """

    def __init__(self, heads, kv_heads, head_dim, pages, page_tokens, max_seqs, max_seq_pages, act_dtype="f16",
                 code="e4m3", layers=1, buffers=None, workspace=None, device="cuda", stream=None):
        self.handle = None
        self.desc = d = kv_desc(heads, kv_heads, head_dim, pages, page_tokens, max_seqs, max_seq_pages, layers, act_dtype,
                                code)
        need = kv_workspace_bytes(d)
        given = dict(buffers or {})
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device = device
        per_page = d.kv_heads * d.page_tokens * d.head_dim
        exps = d.kv_heads * (d.page_tokens // KV_BLOCK)
        shapes = dict(k=(d.layers, d.pages, per_page), v=(d.layers, d.pages, per_page),
                      k_exp=(d.layers, d.pages, exps), v_exp=(d.layers, d.pages, exps),
                      table=(d.max_seqs, d.max_seq_pages), lens=(d.max_seqs,), refs=(d.pages,), failed=(1,),
                      refused=(d.max_seqs,))
        for name, shape in shapes.items():
            dtype = torch.int32 if name in ("table", "lens", "refs", "failed", "refused") else torch.uint8
            t = given.pop(name, None)
            if t is None:
                if dtype is torch.uint8:
                    t = torch.empty(shape, dtype=dtype, device=device)
                else:
                    t = torch.full(shape, -1 if name == "table" else 0, dtype=dtype, device=device)
            self._dense(t, name, dtype, shape)
            setattr(self, name, t)
        if given:
            raise _invalid(f"unknown buffer {sorted(given)[0]!r}")
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        if not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
            raise _invalid(f"workspace must be a contiguous tensor on {device}")
        self.workspace = workspace
        self._met, self._lone = set(), torch.cuda.device_count() == 1
        if device.type != "cuda":
            raise _invalid(f"the cache must be on a CUDA device, not {device}")
        self._act = _ACT_TORCH[d.act_dtype]
        if stream is not None:   # it is the buffers' first user, and they were filled on the current one
            stream.wait_stream(torch.cuda.current_stream(device.index))
        handle = _vp()
        buf = KvBuffers(*[getattr(self, name).data_ptr() for name, _ in KvBuffers._fields_])
        self._run(LIB.pi_kv_create, _byref(d), _byref(buf), workspace.data_ptr(),
                  workspace.numel() * workspace.element_size(), self._stream(stream, ()), _byref(handle))
        self.handle = handle

    def close(self) -> None:
        if getattr(self, "handle", None) is not None and self.handle.value:
            check(LIB.pi_kv_destroy(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---- checks -----------------------------------------------------------------------------------

    def _dense(self, t, name, dtype, shape) -> None:
        if not isinstance(t, torch.Tensor):
            raise _invalid(f"{name} must be a torch tensor, not {type(t).__name__}")
        if t.device != self.device:
            raise _invalid(f"{name} is on {t.device}, the cache is on {self.device}")
        if t.dtype is not dtype:
            raise _invalid(f"{name} is {t.dtype}, expected {dtype}")
        if t.shape != shape:
            raise _invalid(f"{name} must be {list(shape)}, got {list(t.shape)}")
        if not t.is_contiguous():
            raise _invalid(f"{name} is not contiguous")

    def _ids(self, t, name, n=None) -> int:
        """An int32 vector (of n entries, if given); returns its length."""
        if not isinstance(t, torch.Tensor):
            raise _invalid(f"{name} must be a torch tensor, not {type(t).__name__}")
        if t.device != self.device:
            raise _invalid(f"{name} is on {t.device}, the cache is on {self.device}")
        if t.dtype is not torch.int32 or t.dim() != 1 or not t.is_contiguous():
            raise _invalid(f"{name} must be a contiguous int32 vector, got {t.dtype} {list(t.shape)}")
        if n is not None and t.shape[0] != n:
            raise _invalid(f"{name} must have {n} entries, got {t.shape[0]}")
        return t.shape[0]

    def _rows(self, t, name, heads, rows=None) -> KvRows:
        """A token tensor [rows][heads][head_dim] of the activations' type, innermost contiguous."""
        if not isinstance(t, torch.Tensor):
            raise _invalid(f"{name} must be a torch tensor, not {type(t).__name__}")
        if t.device != self.device:
            raise _invalid(f"{name} is on {t.device}, the cache is on {self.device}")
        if t.dtype is not self._act:
            raise _invalid(f"{name} is {t.dtype}, expected {self._act}")
        shape, dim = t.shape, self.desc.head_dim
        if len(shape) != 3 or shape[1] != heads or shape[2] != dim or (rows is not None and shape[0] != rows):
            raise _invalid(f"{name} must be [{'rows' if rows is None else rows}][{heads}][{dim}], got {list(shape)}")
        token, head, inner = t.stride()
        if inner != 1:
            raise _invalid(f"{name}: the innermost dimension is not contiguous")
        return KvRows(t.data_ptr(), token, head)

    def _writable(self, t, name) -> None:
        """A tensor that a call writes may not be an expanded view: rows must not overlap."""
        if t.is_contiguous():
            return
        token, head, _ = t.stride()
        rows, heads, dim = t.shape
        a, b = ((token, rows), (head, heads)) if token <= head else ((head, heads), (token, rows))
        if (a[1] > 1 and a[0] < dim) or (b[1] > 1 and b[0] < a[0] * (a[1] - 1) + dim):
            raise _invalid(f"{name}: its rows overlap")

    def _stream(self, stream, tensors) -> int:
        """The stream's handle.  Memory that is let go of stays reserved until the stream is past the call: the given
        tensors where the caller names a stream (the current one is theirs to mind, as everywhere in torch), and, once for
        each stream that the cache meets, the cache's own."""
        if stream is None:
            stream = torch.cuda.current_stream(self.device.index)
        else:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        handle = stream.cuda_stream
        if handle not in self._met:
            self._met.add(handle)
            for name in _OWNED:
                getattr(self, name).record_stream(stream)
        return handle or None

    def _run(self, fn, *args) -> None:
        """Call the library on the cache's device: kernels start on the current one."""
        if self._lone or torch.cuda.current_device() == self.device.index:
            check(fn(*args))
        else:
            with torch.cuda.device(self.device.index):
                check(fn(*args))

    def _live(self):
        if self.handle is None:
            raise _invalid("the cache is closed")
        return self.handle

    # ---- tokens -----------------------------------------------------------------------------------

    def append(self, layer, k, v, seqs, starts, stream=None) -> None:
        """Store the last tokens of each sequence: rows [starts[i], starts[i + 1]) of k and v
        [rows][kv_heads][head_dim] are the last of the lens[seqs[i]] tokens of seqs[i] (reserve has
        counted them).  A sequence that reserve refused stores nothing.  Blocks of 32 tokens and a head
        share an exponent: see pi_kv.h."""
        n, heads = self._ids(seqs, "seqs"), self.desc.kv_heads
        self._ids(starts, "starts", n + 1)
        kr = self._rows(k, "k", heads)
        rows = k.shape[0]
        vr = self._rows(v, "v", heads, rows)
        if (layer | rows) >> 31:   # below 0, or too large for some
            _in32(layer=layer, rows=rows)
        batch = KvBatch(seqs.data_ptr(), starts.data_ptr(), n, rows)
        self._run(LIB.pi_kv_append, self._live(), layer, _byref(kr), _byref(vr), _byref(batch),
                  self._stream(stream, (k, v, seqs, starts)))

    def read(self, layer, k_out, v_out, seqs, starts, first=None, stream=None) -> None:
        """Read tokens back: rows [starts[i], starts[i + 1]) of k_out and v_out get the tokens of seqs[i]
        from first[i] on (from 0 where first is None); tokens past the end or before the first read as 0."""
        n, heads = self._ids(seqs, "seqs"), self.desc.kv_heads
        self._ids(starts, "starts", n + 1)
        kr = self._rows(k_out, "k_out", heads)
        rows = k_out.shape[0]
        vr = self._rows(v_out, "v_out", heads, rows)
        if (layer | rows) >> 31:
            _in32(layer=layer, rows=rows)
        self._writable(k_out, "k_out")
        self._writable(v_out, "v_out")
        if first is not None:
            self._ids(first, "first", n)
        batch = KvBatch(seqs.data_ptr(), starts.data_ptr(), n, rows)
        self._run(LIB.pi_kv_read, self._live(), layer, _byref(kr), _byref(vr), _byref(batch),
                  None if first is None else first.data_ptr(),
                  self._stream(stream, (k_out, v_out, seqs, starts, first)))

    def attend(self, layer, q, out, seqs, starts, max_new, window=0, sinks=0, scale=None, lse=None, stream=None) -> None:
        """Attention of the last tokens of each sequence over the cache, which holds them already: row
        starts[i] + j of q [rows][heads][head_dim] is token p = lens[seqs[i]] - count + j and sees the tokens
        u <= p (with a window: those with u > p - window or u < sinks).  out gets softmax(scale q K^T) V, zeros
        for a row that sees nothing; lse (fp32 [rows][heads]), if given, the logarithm of the softmax's
        denominator.  max_new: at least the largest count of rows of a sequence (rows past it are not
        computed).  scale: head_dim ** -0.5 unless given."""
        d = self.desc
        n = self._ids(seqs, "seqs")
        self._ids(starts, "starts", n + 1)
        qr = self._rows(q, "q", d.heads)
        rows = q.shape[0]
        orow = self._rows(out, "out", d.heads, rows)
        self._writable(out, "out")
        if lse is not None:
            self._dense(lse, "lse", torch.float32, (rows, d.heads))
        if (layer | rows | max_new | window | sinks) >> 31:
            _in32(layer=layer, rows=rows, max_new=max_new, window=window, sinks=sinks)
        args = KvAttendArgs(qr, orow, None if lse is None else lse.data_ptr(), max_new, window, sinks,
                            d.head_dim ** -0.5 if scale is None else scale)
        batch = KvBatch(seqs.data_ptr(), starts.data_ptr(), n, rows)
        self._run(LIB.pi_kv_attend, self._live(), layer, _byref(args), _byref(batch),
                  self._stream(stream, (q, out, seqs, starts, lse)))

    def _groups(self, groups, plan, n) -> int:
        """Check groups and plan for n sequences; returns the number of groups."""
        count = self._ids(groups, "groups") - 1
        if not 1 <= count <= n:
            raise _invalid(f"groups must have 2 to {n + 1} entries, got {count + 1}")
        self._ids(plan, "plan", count + n)
        return count

    def share(self, seqs, starts, groups, plan, stream=None) -> None:
        """How much the sequences of each group share: group g is seqs[groups[g]:groups[g + 1]] (groups int32, ascending
        from 0 to len(seqs)), and plan (int32 [groups + sequences]) gets, for each group and then for each sequence, the
        number of leading tokens whose pages the whole group names alike, among those held before this call's rows.
        Once a step is enough for all layers: a plan holds until lengths or pages change."""
        n = self._ids(seqs, "seqs")
        self._ids(starts, "starts", n + 1)
        count = self._groups(groups, plan, n)
        batch = KvBatch(seqs.data_ptr(), starts.data_ptr(), n, (1 << 24))   # starts alone say which rows there are
        self._run(LIB.pi_kv_share, self._live(), _byref(batch), groups.data_ptr(), count, plan.data_ptr(),
                  self._stream(stream, (seqs, starts, groups, plan)))

    def state_floats(self, rows) -> int:
        """Elements of the fp32 scratch that attend_shared takes for any number of rows up to `rows`."""
        if rows >> 31:
            _in32(rows=rows)
        out = ctypes.c_size_t(0)
        check(LIB.pi_kv_state_bytes(self._live(), rows, _byref(out)))
        return int(out.value) // 4

    def attend_shared(self, layer, q, out, seqs, starts, groups, plan, max_new, max_rows, scale=None, lse=None, state=None,
                      stream=None) -> None:
        """attend (whole sequences, no window) for groups of sequences that begin with the same pages: what `plan` (share)
        says a group shares is read and multiplied once for all of its rows.  max_rows: at least the largest count of
        rows of a group.  state: fp32 scratch of state_floats(rows) elements, made here unless given.  For long prompts and many
        sequences: where little is shared attend is faster (pi_kv.h says from where on this one is)."""
        d = self.desc
        n = self._ids(seqs, "seqs")
        self._ids(starts, "starts", n + 1)
        count = self._groups(groups, plan, n)
        qr = self._rows(q, "q", d.heads)
        rows = q.shape[0]
        orow = self._rows(out, "out", d.heads, rows)
        self._writable(out, "out")
        if lse is not None:
            self._dense(lse, "lse", torch.float32, (rows, d.heads))
        if (layer | rows | max_new | max_rows) >> 31:
            _in32(layer=layer, rows=rows, max_new=max_new, max_rows=max_rows)
        handle = self._live()
        if state is None:
            size = self.state_floats(rows)
            if stream is None:
                state = torch.empty(size, dtype=torch.float32, device=self.device)
            else:   # of the stream that uses it
                with torch.cuda.stream(stream):
                    state = torch.empty(size, dtype=torch.float32, device=self.device)
        if not isinstance(state, torch.Tensor) or state.device != self.device or state.dtype is not torch.float32 or \
                not state.is_contiguous():
            raise _invalid(f"state must be a contiguous torch.float32 tensor on {self.device}")
        args = KvAttendArgs(qr, orow, None if lse is None else lse.data_ptr(), max_new, 0, 0,
                            d.head_dim ** -0.5 if scale is None else scale)
        more = KvSharedArgs(groups.data_ptr(), plan.data_ptr(), state.data_ptr(), state.numel() * 4, count, max_rows)
        batch = KvBatch(seqs.data_ptr(), starts.data_ptr(), n, rows)
        self._run(LIB.pi_kv_attend_shared, handle, layer, _byref(args), _byref(more), _byref(batch),
                  self._stream(stream, (q, out, seqs, starts, groups, plan, lse, state)))

    def rotate(self, rope, q, q_out, k, k_out, seqs, starts, positions=None, q_norm=None, k_norm=None, eps=1e-6,
               stream=None) -> None:
        """Queries [rows][heads][head_dim] and keys [rows][kv_heads][head_dim] as append and attend take them: each head
        divided by its root mean square and times q_norm or k_norm ([head_dim] of the activations' type), where that is
        given; then turned by its token's position as `rope` says: row starts[i] + j of seqs[i] is token
        lens[seqs[i]] - count + j (reserve has counted it), or positions[row] (int32).  Outputs may be the inputs
        themselves."""
        if not isinstance(rope, Rope):
            raise _invalid(f"rope must be a Rope, not {type(rope).__name__}")
        d = self.desc
        n = self._ids(seqs, "seqs")
        self._ids(starts, "starts", n + 1)
        qr = self._rows(q, "q", d.heads)
        rows = q.shape[0]
        kr = self._rows(k, "k", d.kv_heads, rows)
        qo = qr if q_out is q else self._rows(q_out, "q_out", d.heads, rows)
        ko = kr if k_out is k else self._rows(k_out, "k_out", d.kv_heads, rows)
        self._writable(q_out, "q_out")
        self._writable(k_out, "k_out")
        for t, name in ((q_norm, "q_norm"), (k_norm, "k_norm")):
            if t is not None:
                self._dense(t, name, self._act, (d.head_dim,))
        if positions is not None:
            self._ids(positions, "positions", rows)
        if rows >> 31:
            _in32(rows=rows)
        args = KvRotateArgs(qr, qo, kr, ko, None if q_norm is None else q_norm.data_ptr(),
                            None if k_norm is None else k_norm.data_ptr(),
                            None if positions is None else positions.data_ptr(), eps)
        batch = KvBatch(seqs.data_ptr(), starts.data_ptr(), n, rows)
        self._run(LIB.pi_kv_rotate, self._live(), rope.handle, _byref(args), _byref(batch),
                  self._stream(stream, (q, q_out, k, k_out, seqs, starts, positions, q_norm, k_norm)))

    # ---- pages ------------------------------------------------------------------------------------

    def reserve(self, seqs, counts, stream=None) -> None:
        """Room for counts[i] more tokens of seqs[i], counted in lens: free pages from the lowest number
        up, and a page of its own for a sequence whose partly filled last page is shared.  A sequence
        whose length the caller has lowered (guessed tokens that were not taken) uses its pages again.  What does
        not fit stays as it is, takes no tokens from append, and is counted in `failed` (check_failed)."""
        n = self._ids(seqs, "seqs")
        self._ids(counts, "counts", n)
        self._run(LIB.pi_kv_reserve, self._live(), seqs.data_ptr(), counts.data_ptr(), n, self._stream(stream, (seqs, counts)))

    def free(self, seqs, stream=None) -> None:
        """Drop the sequences' pages: their table rows become -1, their lengths 0."""
        n = self._ids(seqs, "seqs")
        self._run(LIB.pi_kv_free, self._live(), seqs.data_ptr(), n, self._stream(stream, (seqs,)))

    def fork(self, src, dst, stream=None) -> None:
        """Let dst[i] (which holds nothing) continue src[i] on the same pages, shared until one of them
        grows."""
        n = self._ids(src, "src")
        self._ids(dst, "dst", n)
        self._run(LIB.pi_kv_fork, self._live(), src.data_ptr(), dst.data_ptr(), n, self._stream(stream, (src, dst)))

    def compact(self, stream=None) -> None:
        """Move the pages in use to the front of the pool, in every layer; table and refs follow."""
        self._run(LIB.pi_kv_compact, self._live(), self._stream(stream, ()))

    def check_failed(self) -> None:
        """Wait for the current stream and raise PiError if any reserve since the last check could not grow a sequence."""
        count = int(self.failed.item())
        if count:
            self.failed.zero_()
            raise PiError(PI_ERR_INVALID, f"{count} sequences could not grow: too few free pages or table columns")
