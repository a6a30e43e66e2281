"""Python binding of the cache calls around a verify round: the plan of the draft
trees, the norm and rotation of queries and keys, the attention of the draft
nodes over a paged 8-bit cache, and the append of the accepted rows.  The C ABI
and its conventions are in ``include/spec_verify.h``.

One round of a layer, ``parents`` [B, N] and a ``KvCache`` in hand::

    positions, ancestors = spec_tree_plan(parents, cache.lengths, max_depth)       # once per round
    q, k = spec_qk_norm_rope(q, k, positions, inv_freq, q_weight=qw, k_weight=kw)
    out = spec_tree_attention(q, k, v, cache, ancestors)
    ...                                                                            # logits, spec_verify_tree_*
    spec_kv_append(k, v, num_accepted, cache, accept_index=accept_index)

The last call writes the new lengths over ``cache.lengths``.  Layers whose caches share
that tensor append with ``out_lengths=after`` instead and copy ``after`` to it once
all of them are through.

Argument checks happen before anything is enqueued.  Calls run on
``torch.cuda.current_stream`` of the tensors' device unless a stream is given;
outputs are allocated on that stream, and tensors may be dropped as soon as a call
returns, whichever stream it runs on.  Without a ``workspace`` each (device,
stream) has one of its own, whose status word ``spec_cache_status`` reads, and a
call that is being captured into a CUDA graph gets one that belongs to the
graph (give it a ``workspace`` to read the status of its replays).
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from .spec_verify import SPEC_BF16, SPEC_F32, _check, _dtype, lib, spec_read_device_status, spec_workspace_init

_I32, _F32 = torch.int32, torch.float32


class _CCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("k_pages", "v_pages", "k_scale", "v_scale", "k_open", "v_open", "page_table", "slots", "lengths")] + [
        ("num_pages", ctypes.c_int64), ("page_table_stride", ctypes.c_int64), ("num_slots", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32)]


def _need(t, name, dtype, shape, device):
    """A contiguous tensor of this type, shape and device, or an error that says what it is."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, expected {device}")


_strides = {}


def _rows4(t, name, shape, dtype, device):
    """A [B, N, H, D] tensor with unit stride in D; its pointer and strides for the library."""
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError(f"{name} must be a [B, N, heads, D] tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    s = t.stride()
    if s[3] != 1 and shape[3] > 1:
        raise ValueError(f"{name} must have unit stride in its last dim")
    return t.data_ptr(), _strides.get(s) or _new_strides(s)


def _new_strides(s):
    if len(_strides) > 4096:
        _strides.clear()
    c = _strides[s] = (ctypes.c_int64 * 3)(s[0], s[1], s[2])
    return c


def _packed(N, H, D):
    """The strides of a contiguous [B, N, H, D] tensor for the library."""
    s = (N * H * D, H * D, D, 1)
    return _strides.get(s) or _new_strides(s)


class KvCache:
    """The paged 8-bit cache of one layer for a batch of B sequences.

    ``k_pages`` / ``v_pages`` [num_pages, kv_heads, page_size, head_dim] float8_e4m3fn,
    ``k_scale`` / ``v_scale`` [num_pages, kv_heads] f32, ``k_open`` / ``v_open``
    [num_slots, kv_heads, 2 * page_size, head_dim] bf16, ``page_table`` [B, max_pages]
    int32 (rows may be strided), ``lengths`` [B] int32 (negative: no sequence in the row),
    ``slots`` [B] int32 or None (sequence b uses ring b).  Holds the tensors; what they hold
    may change between calls, the tensors may not (``batch`` makes a cache with others).
    """

    def __init__(self, k_pages, v_pages, k_scale, v_scale, k_open, v_open, page_table, lengths, slots=None):
        if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
            raise ValueError("k_pages must be a [num_pages, kv_heads, page_size, head_dim] tensor")
        dev = k_pages.device
        P, H, page, D = k_pages.shape
        if D not in (64, 128):
            raise ValueError(f"head_dim {D} is not 64 or 128")
        if page not in (16, 32, 64, 128):
            raise ValueError(f"page_size {page} is not 16, 32, 64 or 128")
        f8 = torch.float8_e4m3fn
        _need(k_pages, "k_pages", f8, (P, H, page, D), dev)
        _need(v_pages, "v_pages", f8, (P, H, page, D), dev)
        _need(k_scale, "k_scale", _F32, (P, H), dev)
        _need(v_scale, "v_scale", _F32, (P, H), dev)
        if not isinstance(k_open, torch.Tensor) or k_open.dim() != 4:
            raise ValueError("k_open must be a [num_slots, kv_heads, 2 * page_size, head_dim] tensor")
        S = k_open.shape[0]
        _need(k_open, "k_open", torch.bfloat16, (S, H, 2 * page, D), dev)
        _need(v_open, "v_open", torch.bfloat16, (S, H, 2 * page, D), dev)
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table must be a [B, max_pages] tensor")
        B, M = page_table.shape
        if page_table.dtype != _I32 or page_table.device != dev:
            raise TypeError(f"page_table must be int32 on {dev}")
        if M > 1 and page_table.stride(1) != 1:
            raise ValueError("page_table must have unit stride in its last dim")
        _need(lengths, "lengths", _I32, (B,), dev)
        if slots is not None:
            _need(slots, "slots", _I32, (B,), dev)
        elif S < B:
            raise ValueError(f"{S} rings for {B} sequences and no slots")
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.k_open, self.v_open, self.page_table, self.lengths, self.slots = k_open, v_open, page_table, lengths, slots
        self.B, self.kv_heads, self.page_size, self.head_dim, self.device = B, H, page, D, dev
        stride = page_table.stride(0) if B > 1 else max(M, 1)
        self._c = _CCache(k_pages.data_ptr() or None, v_pages.data_ptr() or None, k_scale.data_ptr() or None,
                          v_scale.data_ptr() or None, k_open.data_ptr() or None, v_open.data_ptr() or None,
                          page_table.data_ptr() or None, None if slots is None else slots.data_ptr() or None,
                          lengths.data_ptr() or None, P, stride, S, M, H, D, page)
        self._ref = ctypes.byref(self._c)

    def __setattr__(self, name, value):
        if "_ref" in self.__dict__:                # the library would go on with the old tensor's address
            raise AttributeError(f"{name}: a KvCache keeps its tensors; use batch() or make another")
        object.__setattr__(self, name, value)

    @classmethod
    def allocate(cls, num_pages, kv_heads, page_size, head_dim, page_table, lengths, slots=None, num_slots=None):
        """An empty cache for these page ids; ``num_slots`` rings (default: one per sequence)."""
        dev = page_table.device
        n = page_table.shape[0] if num_slots is None else int(num_slots)
        pool = [torch.zeros((num_pages, kv_heads, page_size, head_dim), dtype=torch.uint8, device=dev)
                .view(torch.float8_e4m3fn) for _ in range(2)]
        scale = [torch.ones((num_pages, kv_heads), dtype=_F32, device=dev) for _ in range(2)]
        ring = [torch.zeros((n, kv_heads, 2 * page_size, head_dim), dtype=torch.bfloat16, device=dev) for _ in range(2)]
        return cls(*pool, *scale, *ring, page_table, lengths, slots)

    def tensors(self):
        """What the cache holds."""
        return (self.k_pages, self.v_pages, self.k_scale, self.v_scale, self.k_open, self.v_open, self.page_table,
                self.lengths, self.slots)

    def batch(self, page_table, lengths, slots=None):
        """The same pages and rings for another batch of sequences."""
        return KvCache(self.k_pages, self.v_pages, self.k_scale, self.v_scale, self.k_open, self.v_open, page_table,
                       lengths, slots)


def spec_cache_workspace_bytes(B: int, N: int, q_heads: int, head_dim: int) -> int:
    """Workspace of the cache calls for B sequences of N nodes (0: out of range)."""
    return int(lib().spec_cache_workspace_bytes(B, N, q_heads, head_dim))


_cache_ws = {}
_ws_bytes = {}
_STATE_BYTES = 65792                               # SPEC_CACHE_STATE_BYTES


_same = contextlib.nullcontext()


def _on(device, stream):
    """The handle of a call's stream and the context that makes it and its device current."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, got {device}")
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        return stream.cuda_stream, torch.cuda.stream(stream)
    handle = torch._C._cuda_getCurrentRawStream(device.index)
    return handle, _same if torch._C._cuda_getDevice() == device.index else torch.cuda.device(device)


def _share(device, stream, used, made):
    """Of a call on a stream that is not the current one: the memory of the tensors that it uses is not handed out again
    before it is through, nor that of the outputs that it allocated while the current stream reads them."""
    if stream is None:
        return
    current = torch.cuda.current_stream(device)
    if current.cuda_stream != stream.cuda_stream:
        for t in used:
            if t is not None:
                t.record_stream(stream)
        for t in made:
            t.record_stream(current)


def _workspace(workspace, device, handle, B, N, q_heads, head_dim):
    """The caller's workspace, or the stream's own; the stream and its device are current."""
    if workspace is not None:
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != device:
            raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
        return workspace
    key = (B, N, q_heads, head_dim)
    need = _ws_bytes.get(key)
    if need is None:
        if len(_ws_bytes) > 4096:
            _ws_bytes.clear()
        need = _ws_bytes[key] = max(spec_cache_workspace_bytes(*key), 256)
    at = (device.index, handle)
    buf = _cache_ws.get(at)
    if torch._C._cuda_isCurrentStreamCapturing():  # replays of several graphs may overlap: one each
        buf = torch.empty(need, dtype=torch.uint8, device=device)
        spec_workspace_init(buf[:_STATE_BYTES])    # part of every replay: no more than has to be zero
    elif buf is None or buf.numel() < need:
        old, buf = buf, torch.empty(need, dtype=torch.uint8, device=device)
        spec_workspace_init(buf[:_STATE_BYTES])
        if old is not None:
            buf[:4].copy_(old[:4])                 # what earlier calls reported stays readable
        _cache_ws[at] = buf
    return buf


def spec_cache_status(device=None, stream=None) -> int:
    """The status bits (``1 << code``) that cache calls without a ``workspace`` have set on this stream (default: the
    device's current one) since the last read; clears them and synchronises the stream.  0 if there was no such call."""
    device = torch.device("cuda" if device is None else device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    handle, current = _on(device, stream)
    buf = _cache_ws.get((device.index, handle))
    if buf is None:
        return 0
    with current:
        return spec_read_device_status(buf)


def spec_tree_plan(parents, lengths, max_depth: int = 64, *, N: int | None = None, out_positions=None,
                   out_ancestors=None, workspace=None, stream=None):
    """Positions [B, N] int32 and ancestor masks [B, N, ceil(N/32)] int32 of draft trees.

    ``parents`` [B, N] int32 as in ``spec_verify_tree_*``, or None for chains of ``N`` nodes;
    ``lengths`` [B] int32, the cached tokens of each sequence.
    """
    if not isinstance(lengths, torch.Tensor) or lengths.dim() != 1:
        raise ValueError("lengths must be a [B] tensor")
    dev, B = lengths.device, lengths.shape[0]
    _need(lengths, "lengths", _I32, (B,), dev)
    if parents is not None:
        if N is None:
            N = parents.shape[-1]
        _need(parents, "parents", _I32, (B, N), dev)
    elif N is None:
        raise ValueError("give parents, or N for chains")
    s, current = _on(dev, stream)
    given, made = [out_positions, out_ancestors], []
    with current:
        if out_positions is None:
            made.append(out_positions := lengths.new_empty((B, N)))
        else:
            _need(out_positions, "out_positions", _I32, (B, N), dev)
        if out_ancestors is None:
            made.append(out_ancestors := lengths.new_empty((B, N, (N + 31) // 32)))
        else:
            _need(out_ancestors, "out_ancestors", _I32, (B, N, (N + 31) // 32), dev)
        ws = _workspace(workspace, dev, s, 1, 1, 1, 64)
        _check(lib().spec_tree_plan(B, N, int(max_depth), None if parents is None else parents.data_ptr(),
                                    lengths.data_ptr(), out_positions.data_ptr(), out_ancestors.data_ptr(),
                                    ws.data_ptr(), ws.numel(), s), "spec_tree_plan")
    if stream is not None:
        _share(dev, stream, (parents, lengths, workspace, *given), made)
    return out_positions, out_ancestors


def _weights(pairs, D, device):
    """(dtype code, pointers) of the given norm weights, which share a type."""
    dt, ptrs = None, []
    for name, w in pairs:
        if w is None:
            ptrs.append(None)
            continue
        if not isinstance(w, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if dt is not None and w.dtype != dt:
            raise TypeError("q_weight and k_weight must have the same dtype")
        dt = w.dtype
        if dt not in (torch.bfloat16, _F32):
            raise TypeError(f"{name} must be bf16 or f32, got {dt}")
        _need(w, name, dt, (D,), device)
        ptrs.append(w.data_ptr())
    return (SPEC_F32 if dt == _F32 else SPEC_BF16), ptrs


def _frequencies(inv_freq, device):
    if inv_freq is None:
        return None, 0
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a [rot_dim / 2] tensor")
    n = inv_freq.shape[0]
    _need(inv_freq, "inv_freq", _F32, (n,), device)
    return inv_freq.data_ptr(), 2 * n


def spec_qk_norm_rope(q, k, positions, inv_freq, *, q_weight=None, k_weight=None, eps: float = 1e-6,
                      interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """Per-head RMS norm (where a weight is given) and rotary positions of ``q``
    [B, N, q_heads, D] and ``k`` [B, N, kv_heads, D] (bf16 or f32, any strides with unit
    stride in D), in one pass.  ``positions`` [B, N] int32 (negative: zeros are written),
    ``inv_freq`` f32 [rot_dim / 2] or None.  Returns ``(q_out, k_out)``, which may be the inputs."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a [B, N, heads, D] tensor")
    B, N, Hq, D = q.shape
    dev, dt = q.device, _dtype(q)
    Hk = k.shape[2] if isinstance(k, torch.Tensor) and k.dim() == 4 else -1
    qp, qs = _rows4(q, "q", (B, N, Hq, D), q.dtype, dev)
    kp, ks = _rows4(k, "k", (B, N, Hk, D), q.dtype, dev)
    _need(positions, "positions", _I32, (B, N), dev)
    wdt, (qw, kw) = _weights((("q_weight", q_weight), ("k_weight", k_weight)), D, dev)
    freq, rot = _frequencies(inv_freq, dev)
    s, current = _on(dev, stream)
    given, made = (q_out, k_out), []
    with current:
        if q_out is None:
            made.append(q_out := q.new_empty((B, N, Hq, D)))
            qop, qos = q_out.data_ptr(), _packed(N, Hq, D)
        else:
            qop, qos = _rows4(q_out, "q_out", (B, N, Hq, D), q.dtype, dev)
        if k_out is None:
            made.append(k_out := q.new_empty((B, N, Hk, D)))
            kop, kos = k_out.data_ptr(), _packed(N, Hk, D)
        else:
            kop, kos = _rows4(k_out, "k_out", (B, N, Hk, D), q.dtype, dev)
        _check(lib().spec_qk_norm_rope(B, N, Hq, Hk, D, qp, qs, kp, ks, dt, positions.data_ptr(), freq, rot,
                                       int(bool(interleaved)), qw, kw, wdt, eps, qop, qos, kop, kos, s),
               "spec_qk_norm_rope")
    if stream is not None:
        _share(dev, stream, (q, k, positions, inv_freq, q_weight, k_weight, *given), made)
    return q_out, k_out


def spec_tree_attention(q, k, v, cache: KvCache, ancestors=None, *, scale: float | None = None, out=None, lse=None,
                        return_lse: bool = False, workspace=None, stream=None):
    """Attention of the nodes over the cache and, by ``ancestors`` [B, N, ceil(N/32)]
    int32 (None: chains), each other.  ``q`` [B, N, q_heads, D], ``k`` / ``v``
    [B, N, kv_heads, D] bf16; ``scale`` defaults to D^(-1/2).  Returns ``out``
    [B, N, q_heads, D] bf16, or ``(out, lse)`` with ``return_lse`` (lse f32 [B, N, q_heads])."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a [B, N, heads, D] tensor")
    B, N, Hq, D = q.shape
    dev, bf = cache.device, torch.bfloat16
    if B != cache.B or D != cache.head_dim:
        raise ValueError(f"q is {tuple(q.shape)}, the cache holds {cache.B} sequences with head_dim {cache.head_dim}")
    qp, qs = _rows4(q, "q", (B, N, Hq, D), bf, dev)
    kp, ks = _rows4(k, "k", (B, N, cache.kv_heads, D), bf, dev)
    vp, vs = _rows4(v, "v", (B, N, cache.kv_heads, D), bf, dev)
    if ancestors is not None:
        _need(ancestors, "ancestors", _I32, (B, N, (N + 31) // 32), dev)
    s, current = _on(dev, stream)
    given, made = (out, lse), []
    with current:
        if out is None:
            made.append(out := q.new_empty((B, N, Hq, D)))
        else:
            _need(out, "out", bf, (B, N, Hq, D), dev)
        if lse is not None:
            _need(lse, "lse", _F32, (B, N, Hq), dev)
        elif return_lse:
            made.append(lse := q.new_empty((B, N, Hq), dtype=_F32))
        ws = _workspace(workspace, dev, s, B, N, Hq, D)
        _check(lib().spec_tree_attention(B, N, Hq, cache._ref, qp, qs, kp, ks, vp, vs,
                                         None if ancestors is None else ancestors.data_ptr(),
                                         1.0 / math.sqrt(D) if scale is None else scale, out.data_ptr(),
                                         None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel(),
                                         s), "spec_tree_attention")
    if stream is not None:
        _share(dev, stream, (q, k, v, ancestors, workspace, *given, *cache.tensors()), made)
    return (out, lse) if return_lse else out


def spec_kv_append(k, v, num_accepted, cache: KvCache, *, accept_index=None, inv_freq=None, k_weight=None,
                   eps: float = 1e-6, interleaved: bool = False, out_lengths=None, workspace=None, stream=None):
    """Add the first ``num_accepted[b] + 1`` rows of each sequence's path to its cache.

    ``k`` / ``v`` [B, T, kv_heads, D] bf16 or f32; ``num_accepted`` [B] int32 (None: every
    row); ``accept_index`` [B, width] int32 picks the rows (None: rows 0, 1, ...).  With
    ``inv_freq`` / ``k_weight`` keys are rotated / normed on the way.  The new lengths are
    written to ``out_lengths`` (default: the cache's own ``lengths``) and returned.  Where several layers'
    caches share their ``lengths``, the default is for none of them but the last: the others would append
    behind rows that they do not have."""
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be a [B, T, heads, D] tensor")
    B, T = k.shape[:2]
    dev, H, D = cache.device, cache.kv_heads, cache.head_dim
    if B != cache.B:
        raise ValueError(f"k holds {B} sequences, the cache {cache.B}")
    dt = _dtype(k)
    kp, ks = _rows4(k, "k", (B, T, H, D), k.dtype, dev)
    vp, vs = _rows4(v, "v", (B, T, H, D), k.dtype, dev)
    width = T
    if num_accepted is not None:
        _need(num_accepted, "num_accepted", _I32, (B,), dev)
    if accept_index is not None:
        width = accept_index.shape[-1]
        _need(accept_index, "accept_index", _I32, (B, width), dev)
    wdt, (kw,) = _weights((("k_weight", k_weight),), D, dev)
    freq, rot = _frequencies(inv_freq, dev)
    if out_lengths is None:
        out_lengths = cache.lengths
    _need(out_lengths, "out_lengths", _I32, (B,), dev)
    s, current = _on(dev, stream)
    with current:
        ws = _workspace(workspace, dev, s, 1, 1, 1, 64)
        _check(lib().spec_kv_append(B, T, width, cache._ref, kp, ks, vp, vs, dt,
                                    None if num_accepted is None else num_accepted.data_ptr(),
                                    None if accept_index is None else accept_index.data_ptr(), freq, rot,
                                    int(bool(interleaved)), kw, wdt, eps, out_lengths.data_ptr(), ws.data_ptr(),
                                    ws.numel(), s), "spec_kv_append")
    if stream is not None:
        _share(dev, stream, (k, v, num_accepted, accept_index, inv_freq, k_weight, out_lengths, workspace, *cache.tensors()), ())
    return out_lengths
