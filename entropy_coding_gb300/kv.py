"""A key/value cache in 8 or 4 bits: writing tokens, reading them back, and
attention; and what queries and keys go through first, their heads' norms and
the rotation by their positions.

The cache is a pool of blocks of tokens. In the 8-bit one (``KVCache``) each
block and key/value head has E4M3 codes and one float32 scale, for K and for V;
in the 4-bit one (``KV4Cache``) each token and head has E2M1 codes and a scale
byte for every 16 columns. The calls take either. A batch names sequences of
uneven length by a block table and their lengths, all on the device. The
operators run in the CUDA kernels of ``libzc.so`` (include/zc.h, zc_kv_*),
launch on the current stream (or ``stream``, a torch stream or a handle) and
do not synchronise; errors that only the device can see are OR-ed into the
cache's status, which ``KVCache.check`` reads. Tensors that the caller gives,
a cache's and a batch's among them, are ready on the stream of a call and
outlive it there (``Tensor.record_stream``), and so does a stream that is
given by its handle outlive the cache; what a call makes for itself is seen to.

The cache serves: nothing here is differentiable, and outputs never require
gradients, whatever the inputs do. Queries are 16-bit, as the tensor cores take
them; heads go up to 128 columns, which is what a tile's queries, operands and
sums fill of shared and of tensor memory. The rotation takes a cache's heads, in
float32 too, and positions from the batch.
"""
from __future__ import annotations

import ctypes
import decimal
import warnings

import torch

__all__ = ["KVCache", "KV4Cache", "KVBatch", "KVRotation", "kv_write", "kv_read", "kv_read_into", "kv_attend", "kv_attend_into",
           "kv_rotate", "kv_rotate_into"]

_BF16, _FP16, _FP32 = 4, 5, 6
_CODE = {torch.bfloat16: _BF16, torch.float16: _FP16, torch.float32: _FP32}
_CAUSAL, _INTERLEAVED = 1, 2
HOOK_COPY_STALL = 1  # test hook (zc_kv_set_test_hooks)


class _Cache(ctypes.Structure):
    _fields_ = [("d_k", ctypes.c_void_p), ("d_v", ctypes.c_void_p), ("d_k_scale", ctypes.c_void_p),
                ("d_v_scale", ctypes.c_void_p), ("block_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64),
                ("n_blocks", ctypes.c_uint32), ("kv_heads", ctypes.c_uint32), ("block_tokens", ctypes.c_uint32),
                ("head_dim", ctypes.c_uint32)]


class _Rotation(ctypes.Structure):
    _fields_ = [("d_turns", ctypes.c_void_p), ("rot_dim", ctypes.c_uint32), ("flags", ctypes.c_uint32),
                ("d_q_weight", ctypes.c_void_p), ("d_k_weight", ctypes.c_void_p), ("weight_dtype", ctypes.c_int),
                ("eps", ctypes.c_float)]


class _Batch(ctypes.Structure):
    _fields_ = [("d_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("d_cu", ctypes.c_void_p),
                ("d_lens", ctypes.c_void_p), ("n_seqs", ctypes.c_uint32), ("total_tokens", ctypes.c_uint32),
                ("max_tokens", ctypes.c_uint32), ("table_width", ctypes.c_uint32)]


class _Rows(ctypes.Structure):
    _fields_ = [("d_data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


# Calls that a check found to have reported an error: CTAs that gave up never came to their counters, so that a workspace
# that was in use before then is zeroed before it is used again.
_failures = 0
# zc_kv_write, zc_kv_read, zc_kv_attend and its two sizes, the same of the 4-bit cache, and zc_kv_rotate, once the library is
# loaded; a cache's are those from its _calls on
_entry = None
# the module of the calls on torch tensors (csrc/binding), once a cache is made; False where there is none (no compiler, a
# folder that cannot be written): every call goes through ctypes then
_torch = None
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _fail(what: str):
    from . import EINVAL, ZcError
    raise ZcError(EINVAL, what)


def declare(L: ctypes.CDLL) -> None:
    """Argument types of the zc_kv_* entry points."""
    vp, u32, u64, i32 = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int
    for f in (L.zc_kv_write, L.zc_kv_read, L.zc_kv4_write, L.zc_kv4_read):
        f.restype = i32
        f.argtypes = [vp, vp, i32, vp, vp, vp, vp]
    for f in (L.zc_kv_attend, L.zc_kv4_attend):
        f.restype = i32
        f.argtypes = [vp, vp, i32, u32, vp, vp, vp, ctypes.c_double, u32, u32, vp, u64, vp, vp]
    L.zc_kv_rotate.restype = i32
    L.zc_kv_rotate.argtypes = [vp, vp, i32, u32, u32, u32, vp, vp, vp, vp, vp, vp]
    L.zc_kv_set_test_hooks.restype = None
    L.zc_kv_set_test_hooks.argtypes = [u32]
    for f in (L.zc_kv_attend_workspace_size, L.zc_kv_attend_counter_bytes, L.zc_kv4_attend_workspace_size,
              L.zc_kv4_attend_counter_bytes):
        f.restype = u64
        f.argtypes = [vp, vp, u32]


def _entries():
    """The entry points, kept: a decoding step calls them for every layer."""
    global _entry
    if _entry is None:
        from . import lib
        L = lib()
        _entry = (L.zc_kv_write, L.zc_kv_read, L.zc_kv_attend, L.zc_kv_attend_workspace_size, L.zc_kv_attend_counter_bytes,
                  L.zc_kv4_write, L.zc_kv4_read, L.zc_kv4_attend, L.zc_kv4_attend_workspace_size, L.zc_kv4_attend_counter_bytes,
                  L.zc_kv_rotate)
    return _entry


_addresses: dict = {}


def _quick(first: int):
    """Addresses of a kind of cache's entry points and of zc_kv_rotate, for the calls that the module makes in one step, or
    None without the module."""
    global _torch
    if _torch is None:
        from . import _build
        try:
            _torch = _build.load_module()
        except (OSError, RuntimeError, ImportError) as e:
            _torch = False
            warnings.warn(f"the key/value cache's calls go through ctypes, which takes longer on the host: {e}", RuntimeWarning, stacklevel=4)
    if not _torch:
        return None
    if first not in _addresses:
        e = _entries()
        _addresses[first] = tuple(ctypes.cast(f, ctypes.c_void_p).value for f in (*e[first:first + 3], e[10]))
    return _addresses[first]


def _outer(t: torch.Tensor, least: int, what: str) -> int:
    """Distance between a tensor's outermost slices, each of ``least`` elements. A single slice has none of its own;
    slices that overlap (an expanded tensor) are refused, since the kernels step from one to the next."""
    if t.shape[0] <= 1:
        return least
    if t.stride(0) < least:
        _fail(f"{what} overlap: stride {t.stride(0)} for {least} elements")
    return t.stride(0)


class KVCache:
    """A pool of cache blocks, over tensors that the caller owns.

    ``k``, ``v``: float8_e4m3fn (or uint8) CUDA tensors [n_blocks, kv_heads,
    block_tokens, head_dim], contiguous within a block; ``k_scale``,
    ``v_scale``: float32 [n_blocks, kv_heads]. Slices of a larger pool along
    the block dimension (one layer of several) are fine as long as K and V
    have the same strides. ``KVCache.empty`` allocates one."""

    _calls = 0     # of _entries()
    _quick = None  # write, read, attend and rotate's addresses, for the calls that the module makes

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride():
            _fail("KVCache: k and v are [n_blocks, kv_heads, block_tokens, head_dim] with the same strides")
        n, h, b, d = k.shape
        if any(t.dtype not in (torch.float8_e4m3fn, torch.uint8) for t in (k, v)):
            _fail("KVCache: codes are float8_e4m3fn or uint8")
        if k.stride()[1:] != (b * d, d, 1):
            _fail("KVCache: a block's codes are contiguous")
        for t in (k_scale, v_scale):
            if t.shape != (n, h) or t.dtype != torch.float32 or t.stride(1) != 1:
                _fail("KVCache: scales are float32 [n_blocks, kv_heads]")
        if k_scale.stride() != v_scale.stride():
            _fail("KVCache: k_scale and v_scale have the same strides")
        block_stride, scale_stride = _outer(k, h * b * d, "KVCache: blocks"), _outer(k_scale, h, "KVCache: scales of blocks")
        if not all(t.is_cuda and t.device == k.device for t in (k, v, k_scale, v_scale)):
            _fail("KVCache expects CUDA tensors of one device")
        self._set(k, v, k_scale, v_scale, block_stride, scale_stride, h, b, d)

    def _set(self, k, v, k_scale, v_scale, block_stride, scale_stride, h, b, d) -> None:
        n = k.shape[0]
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_blocks, self.kv_heads, self.block_tokens, self.head_dim = n, h, b, d
        self.device, self._index = k.device, k.device.index
        self._many = torch.cuda.device_count() > 1
        with torch.cuda.device(self.device):
            self.status = torch.zeros(1, dtype=torch.int32, device=k.device)
            self._ready = torch.cuda.Event()
            self._ready.record()
        self._streams = {_raw_stream(self._index)}  # that know of the status
        self._c = _Cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                         block_stride, scale_stride, n, h, b, d)
        self._ref = ctypes.addressof(self._c)
        self._status = self.status.data_ptr()
        self._quick = _quick(self._calls)

    def _meet(self, handle: int) -> None:
        """A stream's first call: it comes after the status was made, and the status outlives its calls. (A graph is
        captured with the device at rest, and its owner keeps the cache.)"""
        stream = torch.cuda.ExternalStream(handle, device=self.device)
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return
            stream.wait_event(self._ready)
            self.status.record_stream(stream)
        self._streams.add(handle)

    @classmethod
    def empty(cls, n_blocks: int, kv_heads: int, head_dim: int, block_tokens: int = 64, device="cuda") -> "KVCache":
        """A cache of zeros."""
        shape = (n_blocks, kv_heads, block_tokens, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (torch.ones(shape[:2], dtype=torch.float32, device=device) for _ in range(2))
        return cls(k, v, ks, vs)

    def check(self) -> None:
        """Raise ZcError if a call on this cache reported an error (and forget
        it). Waits for the device: for calls on every stream. Batches are as
        good as new after it; one that is used by a captured graph wants
        ``KVBatch.reset`` before the next replay."""
        global _failures
        from . import ZcError
        torch.cuda.synchronize(self.device)
        st = int(self.status.item())
        if st:
            self.status.zero_()
            torch.cuda.synchronize(self.device)  # forgotten before any later call reports
            _failures += 1
            raise ZcError(st, "zc_kv (device)")


class KV4Cache(KVCache):
    """A pool of cache blocks in 4 bits, over tensors that the caller owns.

    ``k``, ``v``: uint8 CUDA tensors [n_blocks, kv_heads, block_tokens, row] of
    E2M1 codes, two columns to a byte (the even one in the low half) and row =
    (head_dim + 31) // 32 * 16 bytes; ``k_scale``, ``v_scale``: uint8 [n_blocks,
    kv_heads, block_tokens, head_dim / 16], the bits 14 to 7 of a float16: a
    number is code * scale. All are contiguous within a block; slices of a
    larger pool along the block dimension are fine as long as K and V have the
    same strides and blocks begin on 16 bytes. ``KV4Cache.empty`` allocates
    one. Every call that takes a ``KVCache`` takes it."""

    _calls = 5

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        if any(t.dim() != 4 or t.dtype != torch.uint8 for t in (k, v, k_scale, v_scale)):
            _fail("KV4Cache: codes and scales are uint8 [n_blocks, kv_heads, block_tokens, ...]")
        n, h, b, row = k.shape
        groups = k_scale.shape[3]
        if k.shape != v.shape or k.stride() != v.stride() or k_scale.shape != v_scale.shape or k_scale.stride() != v_scale.stride():
            _fail("KV4Cache: K and V have the same sizes and strides")
        if k_scale.shape[:3] != k.shape[:3] or row != (groups + 1) // 2 * 16:
            _fail("KV4Cache: scales are [n_blocks, kv_heads, block_tokens, head_dim / 16], rows of codes (head_dim + 31) // 32 * 16 bytes")
        if k.stride()[1:] != (b * row, row, 1) or k_scale.stride()[1:] != (b * groups, groups, 1):
            _fail("KV4Cache: a block's codes, and its scales, are contiguous")
        strides = _outer(k, h * b * row, "KV4Cache: blocks"), _outer(k_scale, h * b * groups, "KV4Cache: scales of blocks")
        if not all(t.is_cuda and t.device == k.device for t in (k, v, k_scale, v_scale)):
            _fail("KV4Cache expects CUDA tensors of one device")
        self._set(k, v, k_scale, v_scale, *strides, h, b, 16 * groups)

    @classmethod
    def empty(cls, n_blocks: int, kv_heads: int, head_dim: int, block_tokens: int = 64, device="cuda") -> "KV4Cache":
        """A cache of zeros."""
        if head_dim % 16 or not 16 <= head_dim <= 128:
            _fail("KV4Cache: head_dim is a multiple of 16 up to 128")
        shape = (n_blocks, kv_heads, block_tokens)
        k, v, ks, vs = (torch.zeros(*shape, m, dtype=torch.uint8, device=device)
                        for m in ((head_dim + 31) // 32 * 16,) * 2 + (head_dim // 16,) * 2)
        return cls(k, v, ks, vs)


class KVBatch:
    """The sequences of a call: their block table, their new tokens and their
    lengths with them, made once for all layers of a step.

    ``block_table`` int32 [n_seqs, width]; ``cu_tokens`` int32 [n_seqs + 1]:
    sequence s has the rows cu[s] .. cu[s + 1] of a call's tensors; ``lens``
    int32 [n_seqs]: tokens of each sequence, those rows being its last.
    ``total_tokens`` and ``max_tokens`` (of one sequence) are the host's
    numbers. The tensors may change between calls (a captured graph is
    replayed with new lengths) as long as the totals hold. The batch keeps
    attention's workspaces, one for each stream: a captured graph that may
    overlap with other calls uses a batch of its own, and the batch is kept as
    long as its graphs."""

    def __init__(self, block_table: torch.Tensor, cu_tokens: torch.Tensor, lens: torch.Tensor, total_tokens: int,
                 max_tokens: int):
        n = lens.numel()
        if any(t.dtype != torch.int32 or not t.is_cuda or t.device != lens.device for t in (block_table, cu_tokens, lens)):
            _fail("KVBatch expects int32 CUDA tensors of one device")
        if block_table.dim() != 2 or block_table.shape[0] != n or cu_tokens.shape != (n + 1,) or lens.dim() != 1:
            _fail("KVBatch: block_table is [n_seqs, width], cu_tokens [n_seqs + 1], lens [n_seqs]")
        if (n and block_table.stride(1) != 1) or not cu_tokens.is_contiguous() or not lens.is_contiguous():
            _fail("KVBatch: rows of the table, cu_tokens and lens are contiguous")
        if not (0 <= max_tokens <= total_tokens <= max_tokens * n) or total_tokens > 0x7FFFFFFF:
            _fail("KVBatch: max_tokens <= total_tokens <= max_tokens * n_seqs")
        self.block_table, self.cu_tokens, self.lens = block_table, cu_tokens, lens
        self.n_seqs, self.total_tokens, self.max_tokens = n, total_tokens, max_tokens
        self.device, self._index = lens.device, lens.device.index
        self._c = _Batch(block_table.data_ptr(), _outer(block_table, block_table.shape[1], "KVBatch: rows of the table"),
                         cu_tokens.data_ptr(), lens.data_ptr(), n, total_tokens, max_tokens, block_table.shape[1])
        self._ref = ctypes.addressof(self._c)
        self._ws: dict = {}

    def workspace(self, cache: KVCache, heads: int, stream=None) -> tuple:
        """(address, bytes, tensor) of the workspace for attention of this batch
        over such a cache, made on a stream's first call and kept for its calls:
        its counters are zeroed before them, and it is not handed on before they
        have run. A captured call takes one that another stream's calls use, or
        memory of its graph, zeroed by each replay."""
        with torch.cuda.device(cache.device):
            return tuple(self._workspace(cache, heads, stream, _handle(stream, cache))[:3])

    def _workspace(self, cache: KVCache, heads: int, stream, handle: int) -> list:
        """The workspace as [address, bytes, tensor, errors found before it was zeroed, its counters]."""
        if stream is not None:
            with _on(stream, cache.device):
                return self._workspace(cache, heads, None, handle)
        key = (cache.kv_heads, cache.head_dim, heads, handle, cache._calls)
        ws = self._ws.get(key)
        if ws is not None and ws[3] == _failures:
            return ws
        capturing = torch.cuda.is_current_stream_capturing()
        if ws is None:
            if capturing:
                for k, other in self._ws.items():
                    if k[:3] == key[:3] and k[4] == key[4] and other[3] == _failures:
                        return other
            size, counters = (int(f(cache._ref, self._ref, heads)) for f in _entries()[cache._calls + 3:cache._calls + 5])
            t = torch.empty(max(size, 16), dtype=torch.uint8, device=cache.device)
            ws = [t.data_ptr(), size, t, -1, t[:counters]]
        ws[4].zero_()
        if not capturing:  # (else it is the graph that zeroes)
            ws[3] = _failures
            self._ws[key] = ws
        return ws

    def reset(self) -> None:
        """Zero the workspaces' counters again, for the replays of a graph that was
        captured with this batch, after a call that reported an error. Waits for
        the device."""
        torch.cuda.synchronize(self.device)
        for ws in self._ws.values():
            ws[4].zero_()
        torch.cuda.synchronize(self.device)


def _rows(t: torch.Tensor, shape, device, what: str) -> _Rows:
    if t.shape != shape or t.device != device:
        _fail(f"{what} is a tensor {tuple(shape)} on the cache's device")
    token, head, one = t.stride()
    if one != 1:
        _fail(f"{what} is contiguous in its last dimension")
    return _Rows(t.data_ptr(), token, head)


def _handle(stream, cache: KVCache) -> int:
    if stream is None:
        handle = _raw_stream(cache._index)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if handle not in cache._streams:
        cache._meet(handle)
    return handle


def _on(stream, device):
    """Memory made for a call belongs to the stream that it runs on."""
    if stream is None:
        return torch.cuda.device(device)
    s = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(s)


def _elsewhere(cache: KVCache, batch: KVBatch, what: str) -> bool:
    """Whether the cache's device is not the current one, on which an entry point launches."""
    if batch._index != cache._index:
        _fail(f"{what}: the batch is on another device than the cache")
    return _current_device() != cache._index


def _at_once(cache: KVCache, batch: KVBatch, stream):
    """The addresses for a call that the module makes in one step, or None: on the current stream, with the cache's device
    the current one and the batch on it."""
    if stream is None and (not cache._many or batch._index == cache._index == _current_device()):
        return cache._quick
    return None


def _check(st: int, what: str) -> None:
    if st:
        from . import ZcError
        raise ZcError(st, what)


def _move(fn, what, cache, batch, k, v, stream):
    if cache._many and _elsewhere(cache, batch, what):
        with torch.cuda.device(cache._index):
            return _move(fn, what, cache, batch, k, v, stream)
    code = _CODE.get(k.dtype)
    if code is None or v.dtype != k.dtype:
        _fail(f"{what}: k and v are bfloat16, float16 or float32")
    shape = (batch.total_tokens, cache.kv_heads, cache.head_dim)
    rk, rv = _rows(k, shape, cache.device, "k"), _rows(v, shape, cache.device, "v")
    _check(fn(cache._ref, batch._ref, code, ctypes.addressof(rk), ctypes.addressof(rv), cache._status,
              _handle(stream, cache)), what)


def kv_write(cache: KVCache, batch: KVBatch, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    """Quantise the batch's tokens into the cache (zc_kv_write, zc_kv4_write). ``k``, ``v``:
    [total_tokens, kv_heads, head_dim] in bfloat16, float16 or float32, any
    strides that are multiples of 16 bytes (views of a fused projection)."""
    quick = _at_once(cache, batch, stream)
    if quick is not None:
        st = _torch.move(quick[0], cache._ref, batch._ref, cache._status, _handle(None, cache), cache._index, batch.total_tokens,
                         cache.kv_heads, cache.head_dim, k, v)
        if st is not None:
            return _check(st, "zc_kv_write")
    _move(_entries()[cache._calls], "zc_kv_write", cache, batch, k, v, stream)


def kv_read_into(cache: KVCache, batch: KVBatch, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    """Read the batch's tokens back into ``k`` and ``v`` (zc_kv_read)."""
    _move(_entries()[cache._calls + 1], "zc_kv_read", cache, batch, k, v, stream)


def kv_read(cache: KVCache, batch: KVBatch, dtype: torch.dtype = torch.bfloat16, stream=None):
    """The batch's tokens as (k, v), [total_tokens, kv_heads, head_dim]."""
    if cache._many and _elsewhere(cache, batch, "zc_kv_read"):
        with torch.cuda.device(cache._index):
            return kv_read(cache, batch, dtype, stream)
    code = _CODE.get(dtype)
    if code is None:
        _fail("zc_kv_read: bfloat16, float16 or float32")
    quick = _at_once(cache, batch, stream)
    if quick is not None:
        r = _torch.read(quick[1], cache._ref, batch._ref, cache._status, _handle(None, cache), cache._index, batch.total_tokens,
                        cache.kv_heads, cache.head_dim, code)
        if type(r) is not tuple:
            _check(r, "zc_kv_read")
        return r
    heads, dim, device = cache.kv_heads, cache.head_dim, cache.device
    shape = (batch.total_tokens, heads, dim)
    if stream is None:
        k = torch.empty(shape, dtype=dtype, device=device)
        v = torch.empty(shape, dtype=dtype, device=device)
    else:
        with _on(stream, device):
            k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
    rk, rv = _Rows(k.data_ptr(), heads * dim, dim), _Rows(v.data_ptr(), heads * dim, dim)
    _check(_entries()[cache._calls + 1](cache._ref, batch._ref, code, ctypes.addressof(rk), ctypes.addressof(rv), cache._status,
                         _handle(stream, cache)), "zc_kv_read")
    return k, v


def _attend(cache, batch, code, heads, q, out, lse, scale, causal, window, stream):
    if cache._many and _elsewhere(cache, batch, "zc_kv_attend"):
        with torch.cuda.device(cache._index):
            return _attend(cache, batch, code, heads, q, out, lse, scale, causal, window, stream)
    if not 0 <= window <= 0x7FFFFFFF:
        _fail("zc_kv_attend: window >= 0")
    handle = _handle(stream, cache)
    ws = batch._ws.get((cache.kv_heads, cache.head_dim, heads, handle, cache._calls))
    if ws is None or ws[3] != _failures:
        ws = batch._workspace(cache, heads, stream, handle)
    _check(_entries()[cache._calls + 2](cache._ref, batch._ref, code, heads, ctypes.addressof(q), ctypes.addressof(out), lse,
                         cache.head_dim ** -0.5 if scale is None else scale, _CAUSAL if causal else 0, window, ws[0],
                         ws[1], cache._status, handle), "zc_kv_attend")


def _query(cache, batch, q):
    """Type code, heads and rows of a query tensor."""
    code = _CODE.get(q.dtype)
    if code is None or code == _FP32:
        _fail("zc_kv_attend: q is bfloat16 or float16")
    heads = q.shape[1] if q.dim() == 3 else 0
    return code, heads, _rows(q, (batch.total_tokens, heads, cache.head_dim), cache.device, "q")


def kv_attend_into(cache: KVCache, batch: KVBatch, q: torch.Tensor, out: torch.Tensor, lse: torch.Tensor | None = None,
                   scale: float | None = None, causal: bool = True, window: int = 0, stream=None) -> None:
    """Attention of the batch's tokens over the cache (zc_kv_attend) into
    ``out`` and, if given, ``lse`` (float32 [total_tokens, heads])."""
    code, heads, rq = _query(cache, batch, q)
    if out.dtype != q.dtype:
        _fail("zc_kv_attend: out has q's type")
    ro = _rows(out, q.shape, cache.device, "out")
    if lse is not None and (lse.shape != q.shape[:2] or lse.dtype != torch.float32 or not lse.is_contiguous() or
                            lse.device != cache.device):
        _fail("zc_kv_attend: lse is float32 [total_tokens, heads]")
    _attend(cache, batch, code, heads, rq, ro, None if lse is None else lse.data_ptr(), scale, causal, window, stream)


def kv_attend(cache: KVCache, batch: KVBatch, q: torch.Tensor, scale: float | None = None, causal: bool = True,
              window: int = 0, stream=None):
    """Attention of the batch's tokens over the cache: (out, lse).

    ``q`` [total_tokens, heads, head_dim], bfloat16 or float16; heads is a
    multiple of the cache's. A query at position p sees the positions j < lens
    with j <= p (``causal``) and j > p - window (``window`` > 0). ``scale``
    defaults to head_dim ** -0.5. The tokens' own keys and values are in the
    cache already (kv_write first)."""
    quick = _at_once(cache, batch, stream)
    if quick is not None and q.dim() == 3 and 0 <= window <= 0x7FFFFFFF:
        handle, dim = _handle(None, cache), cache.head_dim
        ws = batch._ws.get((cache.kv_heads, dim, q.shape[1], handle, cache._calls))
        if ws is not None and ws[3] == _failures:
            r = _torch.attend(quick[2], cache._ref, batch._ref, cache._status, handle, cache._index, batch.total_tokens,
                              cache.kv_heads, dim, q, dim ** -0.5 if scale is None else scale, _CAUSAL if causal else 0, window,
                              ws[0], ws[1])
            if r is not None:
                if type(r) is not tuple:
                    _check(r, "zc_kv_attend")
                return r
    code, heads, rq = _query(cache, batch, q)
    shape, device = q.shape, cache.device
    if stream is None:
        out = torch.empty(shape, dtype=q.dtype, device=device)
        lse = torch.empty(shape[:2], dtype=torch.float32, device=device)
    else:
        with _on(stream, device):
            out = torch.empty(shape, dtype=q.dtype, device=device)
            lse = torch.empty(shape[:2], dtype=torch.float32, device=device)
    dim = cache.head_dim
    _attend(cache, batch, code, heads, rq, _Rows(out.data_ptr(), heads * dim, dim), lse.data_ptr(), scale, causal, window,
            stream)
    return out, lse


class KVRotation:
    """The angles of a position rotation, made once for a model.

    ``frequencies``: radians that each pair of columns turns by for one
    position, numbers or a float tensor, a multiple of 8 of them (usually
    base ** (-2 i / rot_dim), or scaled as a model's long-context recipe wants);
    they are kept as 64-bit fractions of a turn, so that an angle is as good at
    position 10^9 as at 1. Pair i is the columns i and i + rot_dim / 2, or 2 i and
    2 i + 1 (``interleaved``); columns from rot_dim = 2 * len(frequencies) on
    are not turned. A rotation is kept as long as the graphs that it is used
    by."""

    def __init__(self, frequencies, interleaved: bool = False, device="cuda"):
        numbers = frequencies.double().flatten().tolist() if isinstance(frequencies, torch.Tensor) else [float(f) for f in frequencies]
        if len(numbers) % 8 or len(numbers) > 64 or not all(abs(f) < 2.0 ** 20 for f in numbers):
            _fail("KVRotation: a multiple of 8 frequencies, up to 64, finite and below 2^20")
        turns = [fraction_of_turn(f) for f in numbers]
        self.rot_dim, self.interleaved = 2 * len(turns), bool(interleaved)
        self.turns = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device)
        self.device, self._index = self.turns.device, self.turns.device.index
        self._address = self.turns.data_ptr() if turns else 0
        self._flags = _INTERLEAVED if self.interleaved else 0
        self._ready = None
        if self.turns.is_cuda:
            with torch.cuda.device(self.device):
                self._ready = torch.cuda.Event()
                self._ready.record()
                self._streams = {_raw_stream(self._index)}  # that come after the table was made

    def _meet(self, handle: int) -> None:
        """As KVCache._meet, for the table."""
        stream = torch.cuda.ExternalStream(handle, device=self.device)
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return
            stream.wait_event(self._ready)
            self.turns.record_stream(stream)
        self._streams.add(handle)


# 2^256 / (2 pi), which holds any frequency's fraction of a turn to more than 64 bits
with decimal.localcontext(decimal.Context(prec=100)):
    _TURN = int(decimal.Decimal(2) ** 256 / decimal.Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281"))


def fraction_of_turn(frequency: float) -> int:
    """A frequency in radians as a fraction of a turn in units of 2^-64, modulo a turn, rounded to nearest."""
    above, below = frequency.as_integer_ratio()
    below <<= 192
    return (2 * above * _TURN + below) // (2 * below) % (1 << 64)


def _rotate(cache, batch, rotation, code, rows, heads, q_weight, k_weight, eps, stream):
    if cache._many and _elsewhere(cache, batch, "zc_kv_rotate"):
        with torch.cuda.device(cache._index):
            return _rotate(cache, batch, rotation, code, rows, heads, q_weight, k_weight, eps, stream)
    if rotation._index != cache._index:
        _fail("zc_kv_rotate: the rotation is on another device than the cache")
    kind = 0
    for w in (q_weight, k_weight):
        if w is None:
            continue
        if w.shape != (cache.head_dim,) or w.device != cache.device or w.dtype not in _CODE or not w.is_contiguous():
            _fail("zc_kv_rotate: weights are [head_dim], contiguous, on the cache's device")
        if kind not in (0, _CODE[w.dtype]) or _CODE[w.dtype] not in (code, _FP32):
            _fail("zc_kv_rotate: both weights are float32, or of q's type")
        kind = _CODE[w.dtype]
    handle = _handle(stream, cache)
    if handle not in rotation._streams:
        rotation._meet(handle)
    r = _Rotation(rotation._address, rotation.rot_dim, rotation._flags, None if q_weight is None else q_weight.data_ptr(),
                  None if k_weight is None else k_weight.data_ptr(), kind, eps)
    _check(_entries()[10](batch._ref, ctypes.addressof(r), code, cache.head_dim, heads, cache.kv_heads,
                          *map(ctypes.addressof, rows), cache._status, handle), "zc_kv_rotate")


def _pair(cache, batch, q, k, what=""):
    """Type code, query heads and rows of queries and keys."""
    code = _CODE.get(q.dtype)
    if code is None or k.dtype != q.dtype:
        _fail("zc_kv_rotate: q and k are bfloat16, float16 or float32")
    heads = q.shape[1] if q.dim() == 3 else 0
    return code, heads, [_rows(q, (batch.total_tokens, heads, cache.head_dim), cache.device, "q" + what),
                         _rows(k, (batch.total_tokens, cache.kv_heads, cache.head_dim), cache.device, "k" + what)]


def kv_rotate_into(cache: KVCache, batch: KVBatch, rotation: KVRotation, q: torch.Tensor, k: torch.Tensor, q_out: torch.Tensor,
                   k_out: torch.Tensor, q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                   eps: float = 1e-6, stream=None) -> None:
    """``kv_rotate`` into ``q_out`` and ``k_out``, which may be ``q`` and ``k``
    themselves but may not overlap with them otherwise."""
    code, heads, rows = _pair(cache, batch, q, k)
    out, heads_out, rows_out = _pair(cache, batch, q_out, k_out, "_out")
    if out != code or heads_out != heads:
        _fail("zc_kv_rotate: the outputs have q's type and heads")
    for x, y in ((q, q_out), (k, k_out)):
        if x.data_ptr() == y.data_ptr() and x.stride() != y.stride():
            _fail("zc_kv_rotate: outputs in place have the inputs' strides")
    _rotate(cache, batch, rotation, code, rows + rows_out, heads, q_weight, k_weight, eps, stream)


def kv_rotate(cache: KVCache, batch: KVBatch, rotation: KVRotation, q: torch.Tensor, k: torch.Tensor,
              q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6, stream=None):
    """Queries and keys as they are attended with and written: (q, k), each
    head's columns divided by their root mean square (with ``eps``) and
    multiplied by the weights, where these are given (float32 or q's type,
    [head_dim]), and turned by the token's position in its sequence
    (zc_kv_rotate). ``q`` [total_tokens, heads, head_dim], ``k``
    [total_tokens, kv_heads, head_dim] in bfloat16, float16 or float32, any
    strides that are multiples of 16 bytes (views of a fused projection).
    Sums are float32, and a number is rounded once."""
    quick = _at_once(cache, batch, stream)
    if quick is not None and rotation._index == cache._index:
        handle = _handle(None, cache)
        if handle not in rotation._streams:
            rotation._meet(handle)
        r = _torch.rotate(quick[3], batch._ref, cache._status, handle, cache._index, batch.total_tokens, cache.kv_heads,
                          cache.head_dim, rotation._address, rotation.rot_dim, rotation._flags, q, k, q_weight, k_weight, eps)
        if r is not None:
            if type(r) is not tuple:
                _check(r, "zc_kv_rotate")
            return r
    code, heads, rows = _pair(cache, batch, q, k)
    if stream is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=cache.device)
        k_out = torch.empty(k.shape, dtype=q.dtype, device=cache.device)
    else:
        with _on(stream, cache.device):
            q_out, k_out = (torch.empty(x.shape, dtype=q.dtype, device=cache.device) for x in (q, k))
    dim = cache.head_dim
    rows += [_Rows(q_out.data_ptr(), heads * dim, dim), _Rows(k_out.data_ptr(), cache.kv_heads * dim, dim)]
    _rotate(cache, batch, rotation, code, rows, heads, q_weight, k_weight, eps, stream)
    return q_out, k_out
