"""Serving operators over a paged key/value cache held in 8 bits (C ABI: ``include/fa_cache.h``).

``KVCache`` holds the pools and their scales; ``cache_append`` writes new tokens, ``cache_attention`` attends to the
cached ones (a tree of drafted tokens among them), ``cache_evict`` keeps the heaviest and latest; ``verify_drafts``
decides which drafts stay, and ``cache_accept`` brings those together.  Like the dense operators in ``fa``, these functions
check device, dtype, shape and strides, allocate what they return (and the scratch) if it is not given, and call the
C ABI on the current torch stream, or on ``stream`` (a raw cudaStream_t); every step of the computation runs in the
CUDA library.  Lengths and page tables stay on the device: no call synchronises, and each can be captured into a CUDA
graph that follows lengths which change between replays.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

from . import fa as _fa

torch = None  # imported with the first cache: not for those who only build, and not once a call

FA_CACHE_E4M3, FA_CACHE_INT8 = 0, 1

CACHE_EXPORTED = ("fa_cache_accept", "fa_cache_append", "fa_cache_attn", "fa_cache_attn_tree",
                  "fa_cache_attn_tree_workspace_bytes", "fa_cache_attn_workspace_bytes", "fa_cache_evict",
                  "fa_cache_evict_workspace_bytes", "fa_verify_drafts")

_P, _LL, _I, _F = ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int, ctypes.c_float


class FaCache(ctypes.Structure):
    """Layout of ``fa_cache`` in include/fa_cache.h."""
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("k_strides", _LL * 3),
                ("v_strides", _LL * 3), ("P", _I), ("H_kv", _I), ("page", _I), ("D", _I), ("kind", _I)]


class FaCacheAppendArgs(ctypes.Structure):
    """Layout of ``fa_cache_append_args`` in include/fa_cache.h."""
    _fields_ = [("cache", FaCache), ("k", _P), ("v", _P), ("k_strides", _LL * 3), ("v_strides", _LL * 3),
                ("table", _P), ("table_stride", _LL), ("lens", _P), ("n_new", _P), ("weights", _P),
                ("positions", _P), ("seen", _P), ("B", _I), ("n", _I), ("M", _I), ("W", _I), ("dtype", _I),
                ("stream", _P)]


class FaCacheAttnArgs(ctypes.Structure):
    """Layout of ``fa_cache_attn_args`` in include/fa_cache.h."""
    _fields_ = [("cache", FaCache), ("q", _P), ("o", _P), ("lse", _P), ("weights", _P), ("q_strides", _LL * 3),
                ("o_strides", _LL * 3), ("table", _P), ("table_stride", _LL), ("lens", _P), ("n_q", _P), ("B", _I),
                ("H_q", _I), ("n", _I), ("M", _I), ("W", _I), ("scale", _F), ("causal", _I), ("window", _I),
                ("softcap", _F), ("dtype", _I), ("workspace", _P), ("workspace_bytes", _LL), ("stream", _P)]


class FaCacheAttnTreeArgs(ctypes.Structure):
    """Layout of ``fa_cache_attn_tree_args`` in include/fa_cache.h."""
    _fields_ = [("attn", FaCacheAttnArgs), ("tree", _P), ("tree_stride", _LL)]


class FaVerifyDraftsArgs(ctypes.Structure):
    """Layout of ``fa_verify_drafts_args`` in include/fa_cache.h."""
    _fields_ = [("p", _P), ("q", _P), ("p_strides", _LL * 2), ("q_strides", _LL * 2), ("tokens", _P),
                ("tokens_stride", _LL), ("tree", _P), ("tree_stride", _LL), ("u", _P), ("u_stride", _LL),
                ("u_next", _P), ("n_q", _P), ("path", _P), ("count", _P), ("token", _P), ("B", _I), ("n", _I),
                ("V", _I), ("dtype", _I), ("stream", _P)]


class FaCacheAcceptArgs(ctypes.Structure):
    """Layout of ``fa_cache_accept_args`` in include/fa_cache.h."""
    _fields_ = [("cache", FaCache), ("table", _P), ("table_stride", _LL), ("lens", _P), ("n_q", _P), ("path", _P),
                ("path_stride", _LL), ("count", _P), ("weights", _P), ("lens_out", _P), ("B", _I), ("n", _I),
                ("M", _I), ("W", _I), ("stream", _P)]


class FaCacheEvictArgs(ctypes.Structure):
    """Layout of ``fa_cache_evict_args`` in include/fa_cache.h."""
    _fields_ = [("cache", FaCache), ("table", _P), ("table_stride", _LL), ("lens", _P), ("weights", _P),
                ("positions", _P), ("into", _P), ("into_stride", _LL), ("weights_out", _P), ("positions_out", _P),
                ("lens_out", _P), ("B", _I), ("M", _I), ("W", _I), ("M_into", _I), ("W_out", _I), ("keep", _I),
                ("recent", _I), ("workspace", _P), ("workspace_bytes", _LL), ("stream", _P)]


_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = _fa.load_library()
        for name, args in (("fa_cache_append", FaCacheAppendArgs), ("fa_cache_attn", FaCacheAttnArgs),
                           ("fa_cache_attn_tree", FaCacheAttnTreeArgs), ("fa_verify_drafts", FaVerifyDraftsArgs),
                           ("fa_cache_accept", FaCacheAcceptArgs), ("fa_cache_evict", FaCacheEvictArgs)):
            getattr(lib, name).argtypes = [ctypes.POINTER(args)]
            getattr(lib, name).restype = ctypes.c_int
            if name + "_workspace_bytes" in CACHE_EXPORTED:
                size = getattr(lib, name + "_workspace_bytes")
                size.argtypes, size.restype = [ctypes.POINTER(args)], ctypes.c_longlong
        _lib = lib
    return _lib


# ----------------------------------------------------------------- raw C entry points

def fa_cache_append(args: FaCacheAppendArgs) -> int:
    return _library().fa_cache_append(ctypes.byref(args))


def fa_cache_attn(args: FaCacheAttnArgs) -> int:
    return _library().fa_cache_attn(ctypes.byref(args))


def fa_cache_attn_workspace_bytes(args: FaCacheAttnArgs) -> int:
    """``fa_cache_attn_workspace_bytes`` of include/fa_cache.h (-1: invalid arguments)."""
    return _library().fa_cache_attn_workspace_bytes(ctypes.byref(args))


def fa_cache_attn_tree(args: FaCacheAttnTreeArgs) -> int:
    return _library().fa_cache_attn_tree(ctypes.byref(args))


def fa_cache_attn_tree_workspace_bytes(args: FaCacheAttnTreeArgs) -> int:
    """``fa_cache_attn_tree_workspace_bytes`` of include/fa_cache.h (-1: invalid arguments)."""
    return _library().fa_cache_attn_tree_workspace_bytes(ctypes.byref(args))


def fa_verify_drafts(args: FaVerifyDraftsArgs) -> int:
    return _library().fa_verify_drafts(ctypes.byref(args))


def fa_cache_accept(args: FaCacheAcceptArgs) -> int:
    return _library().fa_cache_accept(ctypes.byref(args))


def fa_cache_evict(args: FaCacheEvictArgs) -> int:
    return _library().fa_cache_evict(ctypes.byref(args))


def fa_cache_evict_workspace_bytes(args: FaCacheEvictArgs) -> int:
    """``fa_cache_evict_workspace_bytes`` of include/fa_cache.h (-1: invalid arguments)."""
    return _library().fa_cache_evict_workspace_bytes(ctypes.byref(args))


# ----------------------------------------------------------------- torch convenience layer

def _import_torch():
    global torch
    import torch


class KVCache:
    """The pools of a paged cache: k, v [P, H_kv, page, D] in ``torch.float8_e4m3fn`` or ``torch.int8`` (unit inner
    stride, the other strides multiples of 16), and one fp32 scale for each block and head, [P, H_kv].  A key is its
    stored value times its block's scale.  The tensors are the caller's; this object only keeps them together, with
    their addresses: it cannot be given others later."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "c", "device")

    def __init__(self, k, v, k_scale, v_scale):
        _import_torch()
        if k.dim() != 4:
            raise ValueError(f"k must be [P, H_kv, page, D] (got {tuple(k.shape)})")
        if k.dtype not in (torch.float8_e4m3fn, torch.int8):
            raise ValueError(f"k dtype {k.dtype} is not float8_e4m3fn or int8")
        if v.dtype != k.dtype or v.shape != k.shape:
            raise ValueError(f"v must be {k.dtype} {tuple(k.shape)} (got {v.dtype} {tuple(v.shape)})")
        for name, t in (("k", k), ("v", v)):
            if t.stride(3) != 1:
                raise ValueError(f"{name} must have unit stride along its last dimension")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if tuple(t.shape) != tuple(k.shape[:2]) or t.dtype != torch.float32 or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous fp32 [P, H_kv] = {tuple(k.shape[:2])} tensor")
        for name, t in (("k", k), ("v", v), ("k_scale", k_scale), ("v_scale", v_scale)):
            if not t.is_cuda or t.device != k.device:
                raise ValueError(f"{name} must be a CUDA tensor on {k.device}")
        c = FaCache()
        c.k, c.v, c.k_scale, c.v_scale = k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr()
        c.k_strides[:], c.v_strides[:] = k.stride()[:3], v.stride()[:3]
        c.P, c.H_kv, c.page, c.D = k.shape
        c.kind = FA_CACHE_INT8 if k.dtype == torch.int8 else FA_CACHE_E4M3
        for name, x in zip(self.__slots__, (k, v, k_scale, v_scale, c, k.device)):
            object.__setattr__(self, name, x)

    def __setattr__(self, name, value):
        raise AttributeError(f"KVCache.{name} cannot be set: calls use the tensors that the cache was made of")

    def __copy__(self):
        return self


def kv_cache(pages, H_kv, D, *, page=64, dtype=None, device="cuda") -> KVCache:
    """A new, empty cache of ``pages`` blocks (``dtype``: torch.float8_e4m3fn, the default, or torch.int8)."""
    _import_torch()
    dtype = torch.float8_e4m3fn if dtype is None else dtype
    k, v = (torch.zeros((pages, H_kv, page, D), dtype=torch.uint8, device=device).view(dtype) for _ in range(2))
    ks, vs = (torch.zeros((pages, H_kv), dtype=torch.float32, device=device) for _ in range(2))
    return KVCache(k, v, ks, vs)


# The checks below run on every call of a decoding loop: each reads an attribute once.

def _on(device, name, t, dtype, shape=None):
    """An argument tensor: dtype, shape, contiguous, on the cache's device."""
    if t.dtype is not dtype or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be {dtype}" + (f" {tuple(shape)}" if shape is not None else "") +
                         f" (got {t.dtype} {tuple(t.shape)})")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor on {device}")
    return t.data_ptr()


def _int32(name, x):
    """A count for the C ABI, which would take a longer one's low 32 bits."""
    if not -0x80000000 <= x <= 0x7fffffff:
        raise ValueError(f"{name} ({x}) must fit 32 bits")


def _table(device, name, table, B, width):
    """An int32 [B, M] table, unit inner stride: (pointer, row stride, M)."""
    shape = table.shape
    if len(shape) != 2 or shape[0] != B or table.dtype is not torch.int32 or table.device != device:
        raise ValueError(f"{name} must be an int32 [B = {B}, {width}] tensor on {device} "
                         f"(got {table.dtype} {tuple(shape)})")
    strides = table.stride()
    if strides[1] != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return table.data_ptr(), strides[0], shape[1]


def _tree(device, tree, B, n):
    """An int32 [B, n] tree, or [n] for all sequences: (pointer, stride between sequences)."""
    shape = tree.shape
    if shape != (n,) and shape != (B, n) or tree.dtype is not torch.int32 or tree.device != device:
        raise ValueError(f"tree must be an int32 [B, n] = [{B}, {n}] or [{n}] tensor on {device} "
                         f"(got {tree.dtype} {tuple(shape)})")
    strides = tree.stride()
    if strides[-1] != 1 and n > 1:
        raise ValueError("tree must have unit stride along its last dimension")
    return tree.data_ptr(), strides[0] if len(shape) == 2 else 0


def _rows(name, t):
    """Strides {batch, head, row} of a 4-D tensor with unit inner stride."""
    strides = t.stride()
    if strides[3] != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return strides[:3]


def _trackers(device, H, weights, positions, B):
    """(weights pointer, positions pointer, W) of fp32 and int32 [B, H_kv, W] trackers, each of which may be None."""
    w = p = None
    W = 0
    if weights is not None:
        if weights.dim() != 3:
            raise ValueError(f"weights must be [B, H_kv, W] (got {tuple(weights.shape)})")
        W = weights.shape[2]
        w = _on(device, "weights", weights, torch.float32, (B, H, W))
    if positions is not None:
        if positions.dim() != 3 or (weights is not None and positions.shape[2] != W):
            raise ValueError(f"positions must be [B, H_kv, W], W common to weights and positions "
                             f"(got {tuple(positions.shape)})")
        W = positions.shape[2]
        p = _on(device, "positions", positions, torch.int32, (B, H, W))
    return w, p, W


_DTYPES = {}


def _dtype(t, name):
    if not _DTYPES:
        _DTYPES.update({torch.float32: _fa.FA_DTYPE_F32, torch.bfloat16: _fa.FA_DTYPE_BF16,
                        torch.float16: _fa.FA_DTYPE_F16})
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} dtype {t.dtype} is not bfloat16, float16 or float32")
    return code


@contextlib.contextmanager
def _foreign(device, stream):
    """The cache's device, and ``stream`` as torch's current one: what is allocated meanwhile belongs to the stream
    that uses it."""
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
                yield


def _call(device, stream, work):
    """Run ``work(raw stream)`` on the cache's device and on the given or the current stream."""
    if stream is None and torch._C._cuda_getDevice() == device.index:
        return work(torch._C._cuda_getCurrentRawStream(device.index))
    with _foreign(device, stream):
        return work(torch.cuda.current_stream(device).cuda_stream)


def _with_scratch(a, need, workspace, device, call):
    """Run ``call(a)`` with ``need`` bytes of scratch: ``workspace`` if given, else memory of the stream, taken straight
    from torch's caching allocator (a tensor around it would cost a decoding loop more than the memory does) and given
    back behind the call: the allocator hands it out again only to work queued later on the same stream."""
    if need < 0:
        _fa._check(_fa.FA_ERR_INVALID_ARGUMENT)
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous CUDA tensor on {device}")
        base = workspace.data_ptr()
        start = (base + 255) // 256 * 256
        if workspace.numel() * workspace.element_size() - (start - base) < need:
            raise ValueError(f"workspace holds fewer than the {need} bytes (256-byte aligned) required")
        a.workspace, a.workspace_bytes = start, need
        _fa._check(call(a))
        return
    base = torch._C._cuda_cudaCachingAllocator_raw_alloc(need + 256, a.stream or 0)
    try:
        a.workspace, a.workspace_bytes = (base + 255) // 256 * 256, need
        _fa._check(call(a))
    finally:
        torch._C._cuda_cudaCachingAllocator_raw_delete(base)


def cache_append(cache, k, v, table, lens, *, n_new=None, weights=None, positions=None, seen=None, stream=None):
    """Write new tokens k, v [B, H_kv, n, D] (bf16, fp16 or fp32, unit inner stride) behind the ``lens`` (int32 [B])
    tokens that each sequence holds, in the blocks that ``table`` (int32 [B, M]) names.

    n_new: int32 [B], the new tokens of each sequence (all n if None).
    weights, positions: fp32 and int32 [B, H_kv, W] (see ``cache_evict``): new slots get weight 0 and the positions
    seen[b], seen[b] + 1, ... (``seen``: int32 [B], tokens seen so far; ``lens`` if None).

    A block's scale is the least power of two that its new values fit under, or the one that it had if that is
    larger; where it grows, the block's older tokens are rounded to it.  ``lens`` is not changed.
    """
    shape, device, c = k.shape, cache.device, cache.c
    if len(shape) != 4 or shape != v.shape or k.dtype is not v.dtype:
        raise ValueError(f"k and v must be 4-D [B, H_kv, n, D] and alike (got {tuple(k.shape)} {k.dtype}, "
                         f"{tuple(v.shape)} {v.dtype})")
    B, H, n, D = shape
    if H != c.H_kv or D != c.D:
        raise ValueError(f"k has {H} heads of {D}, the cache {c.H_kv} of {c.D}")
    if k.device != device or v.device != device:
        raise ValueError(f"k and v must be CUDA tensors on {device}")
    t_ptr, t_stride, M = _table(device, "table", table, B, "M")
    l_ptr = _on(device, "lens", lens, torch.int32, (B,))
    n_ptr = None if n_new is None else _on(device, "n_new", n_new, torch.int32, (B,))
    s_ptr = None if seen is None else _on(device, "seen", seen, torch.int32, (B,))
    w_ptr, p_ptr, W = _trackers(device, H, weights, positions, B)
    dtype, ks, vs = _dtype(k, "k"), _rows("k", k), _rows("v", v)
    if B == 0 or n == 0:
        return

    def work(raw):
        _fa._check(fa_cache_append(FaCacheAppendArgs(
            c, k.data_ptr(), v.data_ptr(), ks, vs, t_ptr, t_stride, l_ptr, n_ptr, w_ptr, p_ptr, s_ptr, B, n, M, W, dtype,
            raw)))

    _call(device, stream, work)


def cache_attention(q, cache, table, lens, *, n_q=None, scale=None, causal=True, window=0, softcap=0.0, weights=None,
                    out=None, lse=None, workspace=None, stream=None, tree=None):
    """O and L of the query rows q [B, H_q, n, D] (bf16 or fp16, unit inner stride) over the cached tokens; returns
    (o, lse).

    lens: int32 [B], the tokens that each sequence holds, the query rows' own (appended before) among them; the last
    of the n rows stands at the last token.  n_q: int32 [B], the rows of each sequence (all n if None); rows behind
    them, and rows that see no key, get O = 0 and L = -inf.
    scale (1 / sqrt(D)), causal, window, softcap: as in ``attention``, the causal diagonal at the rows' positions.
    weights: fp32 [B, H_kv, W], W >= every length: the attention weight that each cached token got, summed over rows
    and the heads of its group, is added.
    tree: int32 [B, n] (or [n], one tree for all sequences): the rows are drafts, row i behind row tree[b, i] < i, or
    behind the last token before the drafts if that is -1.  A draft sees the tokens before the drafts, itself and the
    drafts above it; its position, for the window, is that of a sequence that ends with it.  At most 1024 rows.
    workspace: optional device tensor of at least ``fa_cache_attn_workspace_bytes`` (with a tree,
    ``fa_cache_attn_tree_workspace_bytes``) bytes, 256-byte aligned (allocated here if None).
    """
    shape, device, c = q.shape, cache.device, cache.c
    if len(shape) != 4 or shape[3] != c.D:
        raise ValueError(f"q must be 4-D [B, H_q, n, D = {c.D}] (got {tuple(shape)})")
    B, Hq, n, D = shape
    dtype = _dtype(q, "q")
    if dtype == _fa.FA_DTYPE_F32:
        raise ValueError(f"q dtype {q.dtype} is not bfloat16 or float16")
    if q.device != device:
        raise ValueError(f"q must be a CUDA tensor on {device}")
    t_ptr, t_stride, M = _table(device, "table", table, B, "M")
    l_ptr = _on(device, "lens", lens, torch.int32, (B,))
    n_ptr = None if n_q is None else _on(device, "n_q", n_q, torch.int32, (B,))
    w_ptr, _, W = (None, None, 0) if weights is None else _trackers(device, c.H_kv, weights, None, B)
    qs = _rows("q", q)
    if window:
        _int32("window", window)
    if out is not None and (out.shape != shape or out.dtype is not q.dtype or out.device != device):
        raise ValueError(f"out must be {q.dtype} {tuple(shape)} on {device}")
    if lse is not None:
        _on(device, "lse", lse, torch.float32, (B, Hq, n))
    if tree is not None:
        if not causal:
            raise ValueError("a tree's rows see no row behind them: causal must be True")
        nodes = _tree(device, tree, B, n)  # (beside `tree`, which has to live until the call is queued)

    def work(raw):
        o, os = out, None
        if o is None:
            if q.is_contiguous():
                o, os = torch.empty_like(q), qs
            else:
                o = torch.empty(shape, dtype=q.dtype, device=device)
        l = torch.empty((B, Hq, n), dtype=torch.float32, device=device) if lse is None else lse
        if B and Hq and n:
            a = FaCacheAttnArgs(c, q.data_ptr(), o.data_ptr(), l.data_ptr(), w_ptr, qs, os or _rows("out", o), t_ptr, t_stride,
                                l_ptr, n_ptr, B, Hq, n, M, W, 1.0 / math.sqrt(D) if scale is None else scale,
                                bool(causal), window, softcap, dtype, None, 0, raw)
            if tree is None:
                _with_scratch(a, fa_cache_attn_workspace_bytes(a), workspace, device, fa_cache_attn)
            else:
                t = FaCacheAttnTreeArgs(a, *nodes)
                _with_scratch(t.attn, fa_cache_attn_tree_workspace_bytes(t), workspace, device,
                              lambda _: fa_cache_attn_tree(t))
        return o, l

    return _call(device, stream, work)


def cache_evict(cache, table, lens, weights, positions=None, *, keep, recent=0, into=None, weights_out=None,
                positions_out=None, lens_out=None, workspace=None, stream=None):
    """Keep at most ``keep`` tokens of every sequence, chosen per K/V head: the ``recent`` latest, then those with the
    largest accumulated weight (ties: the lowest slot).  Returns the new lengths, int32 [B].

    weights, positions: fp32 and int32 [B, H_kv, W], what ``cache_attention`` and ``cache_append`` keep up.
    In place (``into`` None): kept tokens behind ``keep`` move into the slots that became free below it, with their
    weights and positions.  With ``into`` (int32 [B, M_into], blocks of the same cache that ``table`` does not use) the
    kept tokens are copied there in ascending order, their weights and positions to ``weights_out`` and
    ``positions_out`` ([B, H_kv, W_out], W_out >= keep) where these are given, and the sources stay; positions may
    then be None (a token's position is its slot).
    lens_out: where the new lengths go (may be ``lens``); allocated here if None.
    """
    device, c, B = cache.device, cache.c, table.shape[0]
    t_ptr, t_stride, M = _table(device, "table", table, B, "M")
    l_ptr = _on(device, "lens", lens, torch.int32, (B,))
    w_ptr, p_ptr, W = _trackers(device, c.H_kv, weights, positions, B)
    i_ptr, i_stride, M_into, wo_ptr, po_ptr, W_out = None, 0, 0, None, None, 0
    if into is not None:
        i_ptr, i_stride, M_into = _table(device, "into", into, B, "M_into")
        wo_ptr, po_ptr, W_out = _trackers(device, c.H_kv, weights_out, positions_out, B)
    elif weights_out is not None or positions_out is not None:
        raise ValueError("weights_out and positions_out go with into; in place, weights and positions are changed")
    _int32("keep", keep)
    _int32("recent", recent)
    if lens_out is not None:
        _on(device, "lens_out", lens_out, torch.int32, (B,))

    def work(raw):
        n = torch.empty(B, dtype=torch.int32, device=device) if lens_out is None else lens_out
        if B:
            a = FaCacheEvictArgs(c, t_ptr, t_stride, l_ptr, w_ptr, p_ptr, i_ptr, i_stride, wo_ptr, po_ptr, n.data_ptr(),
                                 B, M, W, M_into, W_out, keep, recent, None, 0, raw)
            _with_scratch(a, fa_cache_evict_workspace_bytes(a), workspace, device, fa_cache_evict)
        return n

    return _call(device, stream, work)


def _nodes(device, name, t, dtype, B, n):
    """A [B, n] argument, unit inner stride: (pointer, row stride)."""
    if t.dtype is not dtype or t.shape != (B, n) or t.device != device:
        raise ValueError(f"{name} must be {dtype} [B, n] = [{B}, {n}] on {device} (got {t.dtype} {tuple(t.shape)})")
    strides = t.stride()
    if strides[1] != 1 and n > 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return t.data_ptr(), strides[0]


def verify_drafts(p, tokens, tree, u, u_next, *, p_draft=None, n_q=None, stream=None):
    """Which drafts of a tree stay, and the token behind them: so that both are distributed as the target's
    probabilities p [B, n, V] (bf16, fp16 or fp32, unit inner stride) say.  Returns (path, count, token), int32 [B, n],
    [B] and [B].

    Node 0 of each sequence is its last token, which stays; node i is a draft of ``tokens[b, i]`` behind node
    ``tree[b, i]`` (int32 [B, n] each; a tree [n] serves all), and p[b, i] are the target's probabilities behind it.
    p_draft: [B, n, V] like p: row i the probabilities that node i's children were drawn from, independently; None if
    the children of a node are distinct candidates that were not drawn (the most likely tokens, say).
    u, u_next: fp32 [B, n] and [B], uniform random numbers in [0, 1).
    n_q: int32 [B], the nodes of each sequence (all n if None).

    From node 0 the path goes on to the first child that is accepted, one with probability p / p_draft (at most 1), the
    next ones against what the rejected ones left of p, until no child is; ``token`` is drawn from what is left there.
    path[b]: the path's nodes, ascending from 0, then -1; count[b]: how many.  A one-hot p keeps the drafts that are
    its tokens.
    """
    if torch is None:
        _import_torch()
    shape, device = p.shape, p.device
    if len(shape) != 3 or not p.is_cuda:
        raise ValueError(f"p must be a 3-D CUDA tensor [B, n, V] (got {tuple(shape)} on {device})")
    B, n, V = shape
    dtype = _dtype(p, "p")
    for name, t in (("p", p), ("p_draft", p_draft)):
        if t is not None and V > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must have unit stride along its last dimension")
    if p_draft is not None and (p_draft.shape != shape or p_draft.dtype is not p.dtype or p_draft.device != device):
        raise ValueError(f"p_draft must be {p.dtype} {tuple(shape)} on {device}")
    k_ptr, k_stride = _nodes(device, "tokens", tokens, torch.int32, B, n)
    t_ptr, t_stride = _tree(device, tree, B, n)
    u_ptr, u_stride = _nodes(device, "u", u, torch.float32, B, n)
    x_ptr = _on(device, "u_next", u_next, torch.float32, (B,))
    n_ptr = None if n_q is None else _on(device, "n_q", n_q, torch.int32, (B,))
    if n == 0 or V == 0:
        raise ValueError("n and V must be > 0")

    def work(raw):
        path, count, token = (torch.empty(s, dtype=torch.int32, device=device) for s in ((B, n), (B,), (B,)))
        if B:
            _fa._check(fa_verify_drafts(FaVerifyDraftsArgs(
                p.data_ptr(), None if p_draft is None else p_draft.data_ptr(), p.stride()[:2],
                (0, 0) if p_draft is None else p_draft.stride()[:2], k_ptr, k_stride, t_ptr, t_stride, u_ptr, u_stride,
                x_ptr, n_ptr, path.data_ptr(), count.data_ptr(), token.data_ptr(), B, n, V, dtype, raw)))
        return path, count, token

    return _call(device, stream, work)


def cache_accept(cache, table, lens, path, count, *, n_q=None, weights=None, lens_out=None, stream=None):
    """Of the drafts that end each sequence's ``lens`` (int32 [B]) tokens, those of a path become its next tokens, the
    others are dropped.  Returns the new lengths, int32 [B].

    path, count: int32 [B, n] and [B] as ``verify_drafts`` gives them: the rows that stay, ascending, and how many.
    n_q: int32 [B], the drafts of each sequence (all n if None).
    weights: fp32 [B, H_kv, W], moved along; positions need no change.
    lens_out: where the new lengths go (may be ``lens``, but no other argument's memory); allocated here if None.  With
    caches of several layers, each call is given the lengths that the drafts are counted in.
    """
    device, c, B = cache.device, cache.c, table.shape[0]
    t_ptr, t_stride, M = _table(device, "table", table, B, "M")
    l_ptr = _on(device, "lens", lens, torch.int32, (B,))
    if path.dim() != 2:
        raise ValueError(f"path must be [B, n] (got {tuple(path.shape)})")
    n = path.shape[1]
    p_ptr, p_stride = _nodes(device, "path", path, torch.int32, B, n)
    k_ptr = _on(device, "count", count, torch.int32, (B,))
    n_ptr = None if n_q is None else _on(device, "n_q", n_q, torch.int32, (B,))
    w_ptr, _, W = (None, None, 0) if weights is None else _trackers(device, c.H_kv, weights, None, B)
    if n == 0:
        raise ValueError("path must hold at least one row")
    if lens_out is not None:
        _on(device, "lens_out", lens_out, torch.int32, (B,))

    def work(raw):
        out = torch.empty(B, dtype=torch.int32, device=device) if lens_out is None else lens_out
        if B:
            _fa._check(fa_cache_accept(FaCacheAcceptArgs(c, t_ptr, t_stride, l_ptr, n_ptr, p_ptr, p_stride, k_ptr,
                                                         w_ptr, out.data_ptr(), B, n, M, W, raw)))
        return out

    return _call(device, stream, work)
