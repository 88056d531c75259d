"""GB300 (sm_103a) fused attention forward: thin Python binding of the C ABI.

Every function here only marshals torch tensors (device pointers, sizes,
strides, the current CUDA stream) into the C library ``libattn_fwd.so``; all
arithmetic runs in the library's CUDA kernels.  There is no fallback: if the
library is missing and cannot be built, or a call fails, an exception is
raised.  Output tensors are allocated with torch when not given.  Work goes to
the current stream; ``stream=s`` makes a call what it is under
``torch.cuda.stream(s)``, allocations included.

    o, lse = attn_fwd(q, k, v, causal=True)                 # [B,H,L,d]
    o, lse = attn_fwd_varlen(q, k, v, cu_q, cu_k, max_q)    # [total,H,d]
    o, lse = attn_fwd_paged(q, k_pool, v_pool, block_table, seqlens_k)
    o, lse = attn_splitkv_combine(o_part, lse_part)
    mask, depth = attn_tree_mask(parents)                   # drafted tokens' tree
    o, lse = attn_fwd_paged_tree(q, k_pool, v_pool, block_table, seqlens_k, mask)
    table, lens, refs = attn_cache_reorder(block_table, seqlens, page_refs, index, page)
    table, lens, refs, free = attn_cache_reserve(k_pool, v_pool, table, lens, refs, add)
    lens, refs = attn_cache_accept(k_pool, v_pool, table, lens, refs, path, path_lens, tree_lens)
    table, refs, page_map = attn_cache_compact(k_pool, v_pool, table, lens, refs)
    slots, positions, cu, seq = attn_cache_slots(table, lens, add, tokens, page, num_pages)
    inv_freq = attn_rope_freqs(rotary_dim)                  # fp64, once per model
    q, k = attn_rope(q, k, inv_freq, positions)
    q = attn_cache_append(k, v, k_pool, v_pool, slots, q=q, inv_freq=inv_freq, positions=positions)
    o, state = attn_linear_fwd(q, k, v, log_decay)          # [B,H,L,d], a decay per head
    o, state = attn_linear_fwd_varlen(q, k, v, cu, max_seqlen, log_decay, state=state)
    o = attn_linear_step(q, k, v, log_decay, state)         # one token each, state in place
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import math

import torch

from . import _lib

__all__ = ["attn_fwd", "attn_fwd_varlen", "attn_fwd_paged", "attn_splitkv_combine",
           "attn_paged_workspace_bytes", "attn_paged_auto_splits", "attn_device_error",
           "attn_selftest_timeout", "attn_last_kernel_name", "attn_paged_window_pages", "attn_paged_keep_splits",
           "attn_fwd_paged_noalloc", "attn_dense_schedule", "attn_tree_mask",
           "attn_tree_workspace_bytes", "attn_fwd_paged_tree", "attn_cache_reorder",
           "attn_cache_reserve", "attn_cache_accept", "attn_cache_compact",
           "attn_cache_slots", "attn_rope_freqs", "attn_rope", "attn_cache_append",
           "attn_linear_workspace_bytes", "attn_linear_fwd", "attn_linear_fwd_varlen", "attn_linear_step",
           "gqa_pack", "AttnError", "library"]


class AttnError(RuntimeError):
    def __init__(self, status: int, fn: str):
        self.status = status
        super().__init__(f"{fn}: {_lib.STATUS.get(status, status)}")


def library() -> ctypes.CDLL:
    return _lib._lib or _lib.load()


def _check(status: int, fn: str):
    if status != 0:
        raise AttnError(status, fn)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return _lib.ATTN_BF16
    if t.dtype == torch.float16:
        return _lib.ATTN_F16
    if t.dtype == torch.float8_e4m3fn:
        return _lib.ATTN_E4M3
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    """The address of a tensor for the C library (None: NULL)."""
    return None if t is None else t.data_ptr()


# The current stream's handle without building a Stream object (3 us a call on a
# Grace host, the query itself 0.1 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream):
    if stream is None and _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _call(fn, device, *args):
    """Calls a library function whose last argument is the stream: ``device``'s current one."""
    index = device.index
    if index is None or device.type != "cuda":
        raise ValueError("the tensors must be on a CUDA device")
    if index != _current_device():
        with torch.cuda.device(device):
            return fn(*args, _stream(None))
    return fn(*args, _raw_stream(index) if _raw_stream is not None else _stream(None))


def _opts(scale, causal, softcap, sink, window=None, top_left=False, alibi=None, bias=None,
          scale_p=None, scale_o=None, sink_tokens=0):
    o = _lib.attn_opts()
    o.scale = float(scale) if scale is not None else 0.0
    o.causal = 1 if causal else 0
    o.softcap = float(softcap) if softcap else 0.0
    o.sink = sink.data_ptr() if sink is not None else None
    if window is not None:
        o.use_window = 1
        o.window_left, o.window_right = int(window[0]), int(window[1])
    o.top_left = 1 if top_left else 0
    if alibi is not None:
        o.alibi_slopes = alibi.data_ptr()
        o.alibi_stride = 0 if alibi.dim() == 1 else int(alibi.stride(0))
    if bias is not None:
        o.bias = bias.data_ptr()
        o.bias_strides = _lib.attn_strides(*_bias_strides(bias))
    o.scale_p = float(scale_p) if scale_p else 0.0
    o.scale_o = float(scale_o) if scale_o else 0.0
    o.sink_tokens = int(sink_tokens)
    return o


def _check_alibi(alibi, B, Hq, device):
    """ALiBi slopes: fp32 [Hq] (shared by every batch) or [B, Hq] (row-contiguous)."""
    if alibi is None:
        return None
    if alibi.dtype != torch.float32 or alibi.device != device or alibi.stride(-1) != 1 or \
            alibi.shape[-1] != Hq or alibi.dim() not in (1, 2) or \
            (alibi.dim() == 2 and alibi.shape[0] != B):
        raise ValueError("alibi_slopes must be fp32 [Hq] or [B, Hq] on the same device")
    return alibi


def _bias_strides(bias):
    """(batch, head, row) element strides of a bias viewed as [B, Hq, Lq, Lk]
    (size-1 broadcast dimensions get stride 0)."""
    if bias.dim() != 4 or bias.stride(3) != 1:
        raise ValueError("bias must be 4-D [B|1, Hq|1, Lq, Lk] with a unit key stride")
    return tuple(0 if bias.shape[i] == 1 else bias.stride(i) for i in range(3))


def _strides_bhld(t):
    s = t.stride()
    if s[3] != 1:
        raise ValueError("innermost (head-dim) stride must be 1")
    return _lib.attn_strides(s[0], s[1], s[2])


def _strides_thd(t):
    s = t.stride()
    if s[2] != 1:
        raise ValueError("innermost (head-dim) stride must be 1")
    return _lib.attn_strides(0, s[1], s[0])


def _check_sink(sink, Hq, device):
    if sink is None:
        return None
    if sink.dtype != torch.float32 or sink.numel() != Hq or sink.device != device:
        raise ValueError("sink must be fp32 [Hq] on the same device")
    return sink.contiguous()


def _on_stream(fn):
    """With ``stream`` given, the call runs as under ``torch.cuda.stream(stream)``: what it
    allocates and copies on the way belongs to the stream that uses it.  A function that
    names ``stream`` among its parameters takes it by position too."""
    names = list(inspect.signature(fn).parameters)
    at = names.index("stream") if "stream" in names else len(names)

    @functools.wraps(fn)
    def call(*args, **kwargs):
        if "stream" not in kwargs and len(args) <= at:
            return fn(*args, **kwargs)
        stream = kwargs.pop("stream", None)
        if len(args) > at:
            stream, args = args[at], args[:at] + (None,) + args[at + 1:]
        if stream is None:
            return fn(*args, **kwargs)
        with torch.cuda.stream(stream):
            return fn(*args, **kwargs)
    return call


def _outputs(q, o, lse, lse_shape):
    """(o, lse or None): new tensors, or the given ones checked (o like q, any strides)."""
    if o is None:
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    elif o.dtype is not q.dtype or o.device != q.device or o.shape != q.shape:
        raise ValueError("o must be like q")
    if lse is True:
        return o, torch.empty(lse_shape, dtype=torch.float32, device=q.device)
    if not isinstance(lse, torch.Tensor):
        return o, None
    if lse.dtype is not torch.float32 or lse.numel() != math.prod(lse_shape) or not lse.is_contiguous() or \
            lse.device != q.device:
        raise ValueError(f"lse must be contiguous fp32 {list(lse_shape)}")
    return o, lse


def _check_alike(q, k, v, dims):
    """Types, devices and shapes of a dense or packed call (strides are checked by the library)."""
    dt, dev, shape = q.dtype, q.get_device(), k.shape
    if k.dtype is not dt or v.dtype is not dt or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("q, k and v must be of one type and on one device")
    if len(shape) != dims or v.shape != shape or shape[-1] != q.shape[-1]:
        raise ValueError("k and v must be alike, with q's head dimension")


@_on_stream
def attn_fwd(q, k, v, o=None, lse=True, causal=False, scale=None, softcap=0.0, sink=None,
             stream=None, window=None, top_left=False, alibi_slopes=None, bias=None,
             scale_p=None, scale_o=None, sink_tokens=0):
    """Dense attention.  q [B,Hq,Lq,d], k/v [B,Hkv,Lk,d] (any strides with d-stride 1).
    ``window`` = (left, right) keeps keys i+Lk-Lq-left <= j <= i+Lk-Lq+right (a
    negative side is unbounded); ``top_left`` drops the Lk-Lq shift; the first ``sink_tokens``
    keys stay visible left of the window.
    ``alibi_slopes``: fp32 [Hq] or [B,Hq]; ``bias``: [B|1,Hq|1,Lq,Lk] in the input
    dtype, added to the scaled score.  float8_e4m3fn inputs (d = 128) run the FP8 path: O is
    e4m3, scale_o * scale_p * softmax(S) V saturated.  Returns (o [B,Hq,Lq,d], lse fp32
    [B,Hq,Lq] or None)."""
    B, Hq, Lq, d = q.shape
    _check_alike(q, k, v, 4)
    Bk, Hkv, Lk, _ = k.shape
    if Bk != B:
        raise ValueError("k and v must be [B,Hkv,Lk,d]")
    o, lse_t = _outputs(q, o, lse, (B, Hq, Lq))
    sink = _check_sink(sink, Hq, q.device)
    alibi_slopes = _check_alibi(alibi_slopes, B, Hq, q.device)
    if bias is not None:
        if bias.dtype != q.dtype or bias.device != q.device:
            raise ValueError("bias must have the input dtype and device")
        if bias.dim() != 4 or bias.shape[3] < Lk or any(x not in (1, y) for x, y in zip(bias.shape, (B, Hq, Lq))):
            raise ValueError("bias must be [B|1, Hq|1, Lq|1, Lk]")
    opts = _opts(scale, causal, softcap, sink, window, top_left, alibi_slopes, bias, scale_p,
                 scale_o, sink_tokens)
    st = library().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse_t), B, Hq, Hkv, Lq, Lk,
                            d, _dtype_code(q), _strides_bhld(q), _strides_bhld(k),
                            _strides_bhld(v), _strides_bhld(o), ctypes.byref(opts),
                            _stream(stream))
    _check(st, "attn_fwd")
    return o, lse_t


@_on_stream
def attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, o=None, lse=True,
                    causal=False, scale=None, softcap=0.0, sink=None, stream=None, window=None,
                    top_left=False, alibi_slopes=None, scale_p=None, scale_o=None, sink_tokens=0):
    """Group mode.  q [total_q,Hq,d], k/v [total_k,Hkv,d], cu_seqlens int32 [B+1] on the
    device.  Returns (o [total_q,Hq,d], lse fp32 [Hq,total_q] or None)."""
    total_q, Hq, d = q.shape
    _check_alike(q, k, v, 3)
    total_k, Hkv, _ = k.shape
    B = cu_seqlens_q.numel() - 1
    for cu in (cu_seqlens_q, cu_seqlens_k):
        if cu.dtype != torch.int32 or cu.device != q.device or not cu.is_contiguous():
            raise ValueError("cu_seqlens must be contiguous int32 on the device")
    if cu_seqlens_k.numel() != B + 1:
        raise ValueError("both cu_seqlens must be [B+1]")
    o, lse_t = _outputs(q, o, lse, (Hq, total_q))
    sink = _check_sink(sink, Hq, q.device)
    alibi_slopes = _check_alibi(alibi_slopes, B, Hq, q.device)
    opts = _opts(scale, causal, softcap, sink, window, top_left, alibi_slopes, None, scale_p,
                 scale_o, sink_tokens)
    st = library().attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse_t),
                                   _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), B, total_q, total_k,
                                   int(max_seqlen_q), Hq, Hkv, d, _dtype_code(q),
                                   _strides_thd(q), _strides_thd(k), _strides_thd(v),
                                   _strides_thd(o), ctypes.byref(opts), _stream(stream))
    _check(st, "attn_fwd_varlen")
    return o, lse_t


def attn_paged_workspace_bytes(B, Lq, Hq, d, num_splits) -> int:
    return int(library().attn_paged_workspace_bytes(B, Lq, Hq, d, num_splits))


def attn_paged_auto_splits(B, Hkv, max_pages_per_seq) -> int:
    return int(library().attn_paged_auto_splits(B, Hkv, max_pages_per_seq))


def attn_paged_keep_splits(B, Hkv, page_size, window_pages) -> int:
    """The split count of calls with ``sink_tokens`` over windows of this many pages."""
    return int(library().attn_paged_keep_splits(B, Hkv, page_size, window_pages))


def attn_paged_window_pages(Lq, page_size, max_pages_per_seq, window=None, causal=False,
                            top_left=False, sink_tokens=0) -> int:
    """Pages of one sequence the paged split layout tiles (W of attn_fwd_paged)."""
    opts = _opts(None, causal, 0.0, None, window, top_left, sink_tokens=sink_tokens)
    return int(library().attn_paged_window_pages(Lq, page_size, max_pages_per_seq,
                                                 ctypes.byref(opts)))


def gqa_pack(Hq, Hkv) -> int:
    """Query heads per tile the library packs for Hq / Hkv (PackGQA): g when
    g = Hq / Hkv is 2, 4, 8 or 16, else 1."""
    g = Hq // Hkv if Hkv > 0 and Hq % Hkv == 0 else 1
    return g if g in (2, 4, 8, 16) else 1


def attn_dense_schedule(B, Hq, Lq, Lk, grid, causal=False, window=None, top_left=False, Hkv=None,
                        sink_tokens=0):
    """The static schedule attn_fwd runs on `grid` CTAs for a dense masked
    problem: a list of `grid` lists of work items (CTA by CTA, in run order),
    or None where the problem keeps the plain snake order.  Hkv defaults to
    Hq (no head packing)."""
    Hkv = Hq if Hkv is None else Hkv
    opts = _opts(None, causal, 0.0, None, window, top_left, sink_tokens=sink_tokens)
    pack = gqa_pack(Hq, Hkv)
    per = 256 // pack
    n = B * (Hq // pack) * ((Lq + per - 1) // per) if Lq > 0 else 0
    off = (ctypes.c_int32 * (max(grid, 0) + 1))()
    item = (ctypes.c_int32 * max(n, 1))()
    st = library().attn_dense_schedule(B, Hq, Hkv, Lq, Lk, ctypes.byref(opts), grid, off, item)
    if st == 2:
        return None
    _check(st, "attn_dense_schedule")
    return [list(item[off[c]:off[c + 1]]) for c in range(grid)]


def _check_paged(q, k_pool, v_pool, block_table, seqlens_k, o):
    """What the paged kernels take for granted of their tensors; returns max_pages."""
    dev, dt = q.get_device(), q.dtype
    for t in (q, k_pool, v_pool, block_table, seqlens_k):
        if not t.is_contiguous() or t.get_device() != dev:
            raise ValueError("paged inputs must be contiguous and on one device")
    if o is not None and not o.is_contiguous():
        raise ValueError("o must be contiguous")
    if block_table.dtype is not torch.int32 or seqlens_k.dtype is not torch.int32:
        raise ValueError("block_table and seqlens_k must be int32")
    shape = k_pool.shape
    if k_pool.dtype is not dt or v_pool.dtype is not dt or v_pool.shape != shape or shape[3] != q.shape[3]:
        raise ValueError("the pools [num_pages,page,Hkv,d] must be alike, of q's type and head dimension")
    B, max_pages = block_table.shape
    if B != q.shape[0] or seqlens_k.numel() != B:
        raise ValueError("block_table must be [B,max_pages], seqlens_k [B]")
    return max_pages


@_on_stream
def attn_fwd_paged(q, k_pool, v_pool, block_table, seqlens_k, num_splits=0, o=None, lse=True,
                   causal=False, scale=None, softcap=0.0, sink=None, workspace=None,
                   stream=None, window=None, top_left=False, alibi_slopes=None, sink_tokens=0):
    """Paged KV.  q [B,Lq,Hq,d], pools [num_pages,page,Hkv,d], block_table int32
    [B,max_pages], seqlens_k int32 [B] (all on the device, contiguous).
    Returns (o [B,Lq,Hq,d], lse fp32 [B,Hq,Lq] or None)."""
    B, Lq, Hq, d = q.shape
    num_pages, page, Hkv, _ = k_pool.shape
    max_pages = _check_paged(q, k_pool, v_pool, block_table, seqlens_k, o)
    o, lse_t = _outputs(q, o, lse, (B, Hq, Lq))
    if Lq * (Hq // Hkv) > 16:
        num_splits = 1  # chunked prefill: the prefill kernel, no split-KV scratch
    elif num_splits == 0:
        pages = attn_paged_window_pages(Lq, page, max_pages, window, causal, top_left, sink_tokens)
        if sink_tokens > 0 and window is not None and 0 <= window[0] < 1 << 30:
            num_splits = attn_paged_keep_splits(B, Hkv, page, pages)
        else:
            num_splits = attn_paged_auto_splits(B, Hkv, pages)
    o_part = lse_part = None
    if num_splits > 1:
        rows = B * Hq * Lq
        need = num_splits * rows * (d + 1)
        if workspace is not None and (workspace.dtype is not torch.float32 or workspace.device != q.device or
                                      workspace.dim() != 1 or not workspace.is_contiguous()):
            raise ValueError("workspace must be contiguous fp32 [n] on the same device")
        if workspace is None or workspace.numel() < need:
            workspace = torch.empty(need, dtype=torch.float32, device=q.device)
        o_part = workspace[: num_splits * rows * d]
        lse_part = workspace[num_splits * rows * d: need]
    sink = _check_sink(sink, Hq, q.device)
    alibi_slopes = _check_alibi(alibi_slopes, B, Hq, q.device)
    opts = _opts(scale, causal, softcap, sink, window, top_left, alibi_slopes,
                 sink_tokens=sink_tokens)
    st = library().attn_fwd_paged(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
                                  _ptr(seqlens_k), _ptr(o), _ptr(lse_t), B, Lq, Hq, Hkv, d,
                                  _dtype_code(q), page, num_pages, max_pages, num_splits,
                                  _ptr(o_part), _ptr(lse_part), ctypes.byref(opts),
                                  _stream(stream))
    _check(st, "attn_fwd_paged")
    return o, lse_t


@_on_stream
def attn_fwd_paged_noalloc(q, k_pool, v_pool, block_table, seqlens_k, num_splits=0, o=None,
                           lse=True, causal=False, scale=None, softcap=0.0, sink=None,
                           stream=None, window=None, top_left=False, alibi_slopes=None,
                           sink_tokens=0):
    """attn_fwd_paged for callers that cannot allocate device scratch: the split
    partials live in a fixed 16 MiB array inside the library (shared by all
    calls on a GPU; calls overlapping on the GPU race).  Outputs are allocated
    here only when not given."""
    B, Lq, Hq, d = q.shape
    num_pages, page, Hkv, _ = k_pool.shape
    max_pages = _check_paged(q, k_pool, v_pool, block_table, seqlens_k, o)
    o, lse_t = _outputs(q, o, lse, (B, Hq, Lq))
    sink = _check_sink(sink, Hq, q.device)
    alibi_slopes = _check_alibi(alibi_slopes, B, Hq, q.device)
    opts = _opts(scale, causal, softcap, sink, window, top_left, alibi_slopes,
                 sink_tokens=sink_tokens)
    st = library().attn_fwd_paged_noalloc(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
                                          _ptr(seqlens_k), _ptr(o), _ptr(lse_t), B, Lq, Hq, Hkv,
                                          d, _dtype_code(q), page, num_pages,
                                          max_pages, num_splits, ctypes.byref(opts),
                                          _stream(stream))
    _check(st, "attn_fwd_paged_noalloc")
    return o, lse_t


@functools.lru_cache(maxsize=256)
def attn_tree_workspace_bytes(T, Hq, Hkv, d) -> int:
    """Bytes of device memory attn_fwd_paged_tree works in."""
    return int(library().attn_tree_workspace_bytes(T, Hq, Hkv, d))


def _ints(device, names, *tensors):
    """Each given tensor is contiguous int32 on ``device``."""
    for t in tensors:
        if t is not None and not (t.dtype is torch.int32 and t.device == device and t.is_contiguous()):
            raise ValueError(f"{names} must be contiguous int32 on {device}")


@_on_stream
def attn_tree_mask(parents, tree_lens=None, mask=None, depth=None):
    """Visibility masks and depths of draft trees.  parents int32 [B,T] (-1: follows the
    sequence's last token), tree_lens int32 [B] or None.  Returns (mask int32
    [B,T,ceil(T/32)], its 32 bits per word the nodes a node sees, depth int32 [B,T])."""
    B, T = parents.shape
    W, dev = (T + 31) // 32, parents.device
    if mask is None:
        mask = torch.empty((B, T, W), dtype=torch.int32, device=dev)
    if depth is None:
        depth = torch.empty((B, T), dtype=torch.int32, device=dev)
    _ints(dev, "parents, tree_lens, mask and depth", parents, tree_lens, mask, depth)
    if mask.shape != (B, T, W) or depth.shape != (B, T) or \
            (tree_lens is not None and tree_lens.shape != (B,)):
        raise ValueError("tree_lens is [B], mask [B,T,ceil(T/32)], depth [B,T]")
    _check(_call(library().attn_tree_mask, dev, parents.data_ptr(), _ptr(tree_lens),
                 mask.data_ptr(), depth.data_ptr(), B, T), "attn_tree_mask")
    return mask, depth


@_on_stream
def attn_fwd_paged_tree(q, k_pool, v_pool, block_table, seqlens_k, tree_mask, tree_lens=None,
                        tree_depth=None, o=None, lse=True, scale=None, softcap=0.0, sink=None,
                        workspace=None, window=None, sink_tokens=0):
    """Attention of drafted nodes over a paged cache.  q [B,T,Hq,d]; the nodes' K/V are the
    last T (or tree_lens[b]) of the seqlens_k[b] positions; node i sees every earlier
    position and the nodes of its tree_mask row (attn_tree_mask).  ``window`` = (left, -1)
    with tree_depth limits the earlier positions, the first ``sink_tokens`` staying visible; it
    cuts no nodes (where a path is longer than the window, clear those ancestors' bits).
    Returns (o [B,T,Hq,d], lse fp32 [B,Hq,T] or None)."""
    B, T, Hq, d = q.shape
    num_pages, page, Hkv, dk = k_pool.shape
    dev = q.device
    if o is None:
        o = torch.empty_like(q)
    lse_t = lse if isinstance(lse, torch.Tensor) else None
    if lse is True:
        lse_t = torch.empty((B, Hq, T), dtype=torch.float32, device=dev)
    for t in (q, k_pool, v_pool, o):
        if t.dtype != q.dtype or t.device != dev or not t.is_contiguous():
            raise ValueError("q, the pools and o must be contiguous, of one type and on one device")
    _ints(dev, "block_table, seqlens_k and the tree tensors", block_table, seqlens_k, tree_mask, tree_lens,
          tree_depth)
    if dk != d or v_pool.shape != k_pool.shape or block_table.dim() != 2 or \
            block_table.shape[0] != B or seqlens_k.shape != (B,) or \
            tree_mask.shape != (B, T, (T + 31) // 32) or o.shape != q.shape or \
            (tree_lens is not None and tree_lens.shape != (B,)) or \
            (tree_depth is not None and tree_depth.shape != (B, T)) or \
            (lse_t is not None and (lse_t.shape != (B, Hq, T) or lse_t.dtype != torch.float32 or
                                    lse_t.device != dev or not lse_t.is_contiguous())):
        raise ValueError("shapes: q, o [B,T,Hq,d], pools [pages,page,Hkv,d], block_table [B,max_pages], "
                         "seqlens_k, tree_lens [B], tree_mask [B,T,ceil(T/32)], tree_depth [B,T], "
                         "lse fp32 [B,Hq,T]")
    if workspace is None:
        workspace = torch.empty(attn_tree_workspace_bytes(T, Hq, Hkv, d), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the same device")
    if sink is not None:
        sink = _check_sink(sink, Hq, dev)
    opts = _opts(scale, False, softcap, sink, window, sink_tokens=sink_tokens)
    st = _call(library().attn_fwd_paged_tree, dev, q.data_ptr(), k_pool.data_ptr(),
               v_pool.data_ptr(), block_table.data_ptr(), seqlens_k.data_ptr(), tree_mask.data_ptr(),
               _ptr(tree_lens), _ptr(tree_depth), o.data_ptr(), _ptr(lse_t), B, T, Hq, Hkv, d,
               _dtype_code(q), page, num_pages, block_table.shape[1], workspace.data_ptr(),
               workspace.numel() * workspace.element_size(), ctypes.byref(opts))
    _check(st, "attn_fwd_paged_tree")
    return o, lse_t


def _pools(k_pool, v_pool, page_refs):
    """(layers, num_pages, page, row bytes) of pools [num_pages,page,Hkv,d] or
    [layers,num_pages,page,Hkv,d]."""
    shape = k_pool.shape
    if shape != v_pool.shape or k_pool.dtype is not v_pool.dtype or len(shape) not in (4, 5) or \
            not k_pool.is_contiguous() or not v_pool.is_contiguous() or \
            not k_pool.device == v_pool.device == page_refs.device:
        raise ValueError("the pools must be contiguous [num_pages,page,Hkv,d] or "
                         "[layers,num_pages,page,Hkv,d], alike, on the tables' device")
    num_pages, page, Hkv, d = shape[-4:]
    if page_refs.shape[0] != num_pages:
        raise ValueError("page_refs must be [num_pages]")
    return shape[0] if len(shape) == 5 else 1, num_pages, page, Hkv * d * k_pool.element_size()


def _cache_state(block_table, seqlens, page_refs, *per_sequence):
    """(device, B, max_pages) of a cache's tables, checked with further int32 tensors that
    have one entry per sequence."""
    dev = block_table.device
    _ints(dev, "the cache's tables and what goes with them", block_table, seqlens, page_refs, *per_sequence)
    B, max_pages = block_table.shape
    for t in (seqlens, *per_sequence):
        if t.shape[0] != B:
            raise ValueError("one entry per sequence (row of block_table) is needed")
    return dev, B, max_pages


@_on_stream
def attn_cache_reorder(block_table, seqlens, page_refs, index, page_size):
    """New sequence b is old sequence index[b] (int32 [B_out]; -1: an empty one): forks where
    an index repeats, permutes, frees what nobody takes.  Returns (block_table [B_out,
    max_pages], seqlens [B_out], page_refs)."""
    dev, B, max_pages = _cache_state(block_table, seqlens, page_refs)
    _ints(dev, "index", index)
    n = index.shape[0]
    table_out = torch.empty((n, max_pages), dtype=torch.int32, device=dev)
    lens_out, refs_out = torch.empty_like(index), torch.empty_like(page_refs)
    _check(_call(library().attn_cache_reorder, dev, block_table.data_ptr(), seqlens.data_ptr(),
                 page_refs.data_ptr(), index.data_ptr(), table_out.data_ptr(), lens_out.data_ptr(),
                 refs_out.data_ptr(), B, n, max_pages, page_refs.shape[0], int(page_size)),
           "attn_cache_reorder")
    return table_out, lens_out, refs_out


@_on_stream
def attn_cache_reserve(k_pool, v_pool, block_table, seqlens, page_refs, add):
    """Room for add[b] (int32 [B]) more tokens per sequence; shared partly filled last pages
    are copied first.  Returns (block_table, seqlens + add, page_refs, free int32 [1]: the
    free pages left, or minus the pages missing, and then nothing has changed)."""
    dev, B, max_pages = _cache_state(block_table, seqlens, page_refs, add)
    layers, num_pages, page, row = _pools(k_pool, v_pool, page_refs)
    table_out, lens_out = torch.empty_like(block_table), torch.empty_like(seqlens)
    refs_out, free = torch.empty_like(page_refs), torch.empty(1, dtype=torch.int32, device=dev)
    _check(_call(library().attn_cache_reserve, dev, k_pool.data_ptr(), v_pool.data_ptr(),
                 block_table.data_ptr(), seqlens.data_ptr(), page_refs.data_ptr(), add.data_ptr(),
                 table_out.data_ptr(), lens_out.data_ptr(), refs_out.data_ptr(), free.data_ptr(), B,
                 max_pages, num_pages, page, layers, row), "attn_cache_reserve")
    return table_out, lens_out, refs_out, free


@_on_stream
def attn_cache_accept(k_pool, v_pool, block_table, seqlens, page_refs, path, path_lens, tree_lens=None, T=None):
    """Keeps of each sequence's drafted nodes (the last tree_lens[b] positions, at most T; the
    last T without tree_lens) the nodes path[b, :path_lens[b]] (int32 [B,A], rising), moved
    together behind the tokens before them, and gives the pages past them back.  Returns
    (seqlens, page_refs); the pools are updated in place, the table stays."""
    dev, B, max_pages = _cache_state(block_table, seqlens, page_refs, path, path_lens,
                                     *(() if tree_lens is None else (tree_lens,)))
    layers, num_pages, page, row = _pools(k_pool, v_pool, page_refs)
    if T is None:
        if tree_lens is None:
            raise ValueError("T, the nodes of every sequence, is needed without tree_lens")
        T = max_pages * page
    elif T < 0:
        raise ValueError("T must not be negative")
    if path.dim() != 2:
        raise ValueError("path must be [B,A]")
    lens_out, refs_out = torch.empty_like(seqlens), torch.empty_like(page_refs)
    _check(_call(library().attn_cache_accept, dev, k_pool.data_ptr(), v_pool.data_ptr(),
                 block_table.data_ptr(), seqlens.data_ptr(), page_refs.data_ptr(), path.data_ptr(),
                 path_lens.data_ptr(), _ptr(tree_lens), lens_out.data_ptr(), refs_out.data_ptr(), B,
                 path.shape[1], int(T), max_pages, num_pages, page, layers, row),
           "attn_cache_accept")
    return lens_out, refs_out


@_on_stream
def attn_cache_compact(k_pool, v_pool, block_table, seqlens, page_refs):
    """Moves the live pages to the pool's front (in place).  Returns (block_table, page_refs,
    page_map int32 [num_pages]: where each live page is now, -1 for a free one)."""
    dev, B, max_pages = _cache_state(block_table, seqlens, page_refs)
    layers, num_pages, page, row = _pools(k_pool, v_pool, page_refs)
    table_out, refs_out = torch.empty_like(block_table), torch.empty_like(page_refs)
    page_map = torch.empty_like(page_refs)
    work = torch.empty(num_pages + 1, dtype=torch.int32, device=dev)
    _check(_call(library().attn_cache_compact, dev, k_pool.data_ptr(), v_pool.data_ptr(),
                 block_table.data_ptr(), seqlens.data_ptr(), page_refs.data_ptr(), table_out.data_ptr(),
                 refs_out.data_ptr(), page_map.data_ptr(), work.data_ptr(), B, max_pages, num_pages, page,
                 layers, row), "attn_cache_compact")
    return table_out, refs_out, page_map


@_on_stream
def attn_cache_slots(block_table, seqlens, add, num_tokens, page_size, num_pages):
    """The slot map of the last add[b] (int32 [B]) of each sequence's seqlens[b] tokens, packed
    in order of the sequences, room for ``num_tokens`` of them (rows past the last: sequence
    -1, position 0, slot -1).  Returns (slots [num_tokens], positions [num_tokens], cu_seqlens
    [B+1], sequence [num_tokens]), int32."""
    dev, B, max_pages = _cache_state(block_table, seqlens, add)
    n = int(num_tokens)
    if not 0 <= n < 1 << 30:
        raise ValueError("num_tokens must not be negative, and below 2^30")
    slots = torch.empty(n, dtype=torch.int32, device=dev)
    positions, sequence = torch.empty_like(slots), torch.empty_like(slots)
    cu = torch.empty(B + 1, dtype=torch.int32, device=dev)
    _check(_call(library().attn_cache_slots, dev, block_table.data_ptr(), seqlens.data_ptr(), add.data_ptr(),
                 slots.data_ptr(), positions.data_ptr(), cu.data_ptr(), sequence.data_ptr(), B, n, max_pages,
                 int(num_pages), int(page_size)), "attn_cache_slots")
    return slots, positions, cu, sequence


_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "parts": 3, "ramp": 4}


def attn_rope_freqs(rotary_dim, base=10000.0, scaling="plain", factor=1.0, original_len=0.0, slow_turns=1.0,
                    fast_turns=32.0, device="cuda"):
    """Rotary frequencies base^(-2i / rotary_dim), fp64 [rotary_dim / 2] on ``device``, scaled for
    long contexts: "linear" (all divided by factor), "base" (a larger base), "parts" and
    "ramp" (pairs of at most slow_turns turns in original_len positions divided by
    factor, those of fast_turns or more kept, between them weighted by turns or by index)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(_SCALINGS)}")
    f = (ctypes.c_double * max(1, int(rotary_dim) // 2))()
    _check(library().attn_rope_freqs(int(rotary_dim), float(base), _SCALINGS[scaling], float(factor),
                                     float(original_len), float(slow_turns), float(fast_turns), f),
           "attn_rope_freqs")
    return torch.tensor(list(f), dtype=torch.float64, device=device)


def _rope_opts(inv_freq, d, device, interleaved, inverse, scale):
    if inv_freq.dtype is not torch.float64 or inv_freq.dim() != 1 or inv_freq.device != device or \
            not inv_freq.is_contiguous() or 2 * inv_freq.shape[0] > d:
        raise ValueError("inv_freq must be contiguous fp64 [rotary_dim / 2] on the same device, rotary_dim <= d")
    opts = _lib.attn_rope_opts(inv_freq.data_ptr(), 2 * inv_freq.shape[0], 1 if interleaved else 0,
                               1 if inverse else 0, float(scale))
    if opts.scale == 0:  # (in 32 bits: the library's name for 1)
        raise ValueError("scale must be above 0")
    return opts


def _like(t, out, name):
    """A new contiguous tensor like t, or ``out`` checked to be one (any strides)."""
    if out is None:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    if out.dtype is not t.dtype or out.device != t.device or out.shape != t.shape:
        raise ValueError(f"{name} must be like its input")
    return out


@functools.lru_cache(maxsize=512)
def _stride_struct(batch, head, row):
    return _lib.attn_strides(batch, head, row)


def _rows(t):
    """Strides of dense [B,H,L,d] or packed [N,H,d] rows (None: no tensor)."""
    if t is None:
        return _stride_struct(0, 0, 0)
    s = t.stride()
    if s[-1] != 1:
        raise ValueError("innermost (head-dim) stride must be 1")
    return _stride_struct(s[0], s[1], s[2]) if len(s) == 4 else _stride_struct(0, s[1], s[0])


@_on_stream
def attn_rope(q, k, inv_freq, positions=None, interleaved=False, inverse=False, scale=1.0, q_out=None, k_out=None):
    """Rotary positions.  q [B,Hq,L,d] and k [B,Hkv,L,d], or packed [N,H,d] (k may be None); the
    first 2 * len(inv_freq) elements of a head turn by position * inv_freq (attn_rope_freqs),
    in halves or interleaved pairs, times ``scale``.  positions int32 [L] or [B,L], packed [N];
    None: the row.  ``inverse`` turns back: with the same ``scale`` the transpose, which takes a gradient
    back; with 1 / scale it undoes the rotation.  q_out and k_out may be q and k.  Returns (q_out, k_out)."""
    shape, dev = q.shape, q.device
    if len(shape) == 4:
        B, Hq, L, d = shape
    elif len(shape) == 3:
        B, (L, Hq, d) = 1, shape
    else:
        raise ValueError("q must be [B,Hq,L,d] or [N,Hq,d]")
    Hkv = 0
    if k is not None:
        other = k.shape
        if len(other) == len(shape):
            Hkv = other[1]
        if k.dtype is not q.dtype or k.device != dev or \
                other != ((B, Hkv, L, d) if len(shape) == 4 else (L, Hkv, d)):
            raise ValueError("k must be like q but for its heads")
    stride = 0
    if positions is not None:
        _ints(dev, "positions", positions)
        if positions.shape == (L,):
            pass
        elif len(shape) == 4 and positions.shape == (B, L):
            stride = L
        else:
            raise ValueError("positions must be [L] or [B,L], of packed rows [N]")
    opts = _rope_opts(inv_freq, d, dev, interleaved, inverse, scale)
    q_out = _like(q, q_out, "q_out")
    if k is not None:
        k_out = _like(k, k_out, "k_out")
    elif k_out is not None:
        raise ValueError("k_out without k")
    _check(_call(library().attn_rope, dev, q.data_ptr(), q_out.data_ptr(), _ptr(k), _ptr(k_out), _ptr(positions),
                 stride, B, L, Hq, Hkv, d, _dtype_code(q), _rows(q), _rows(q_out), _rows(k), _rows(k_out),
                 ctypes.byref(opts)), "attn_rope")
    return q_out, k_out


@_on_stream
def attn_cache_append(k, v, k_pool, v_pool, slots, q=None, inv_freq=None, positions=None, interleaved=False,
                      scale=1.0, q_out=None):
    """Writes packed new tokens' k and v [N,Hkv,d] into the pools [num_pages,page,Hkv,d] by slot
    (int32 [N], attn_cache_slots; -1: not written; no slot twice).  With ``inv_freq`` and
    ``positions`` (int32 [N]) k is rotated on the way, and so is q [N,Hq,d], every row, into
    q_out (q itself, or a new tensor).  Returns q_out (None without q)."""
    dev, dt = k.device, k.dtype
    if k.dim() != 3 or v.shape != k.shape or v.dtype is not dt or v.device != dev:
        raise ValueError("k and v must be [N,Hkv,d], alike")
    N, Hkv, d = k.shape
    if k_pool.dim() != 4 or v_pool.shape != k_pool.shape or k_pool.shape[2:] != (Hkv, d) or \
            not k_pool.dtype is v_pool.dtype is dt or not k_pool.device == v_pool.device == dev or \
            not k_pool.is_contiguous() or not v_pool.is_contiguous():
        raise ValueError("the pools must be contiguous [num_pages,page,Hkv,d], of k's type, on its device")
    _ints(dev, "slots and positions", slots, positions)
    if slots.shape != (N,) or (positions is not None and positions.shape != (N,)):
        raise ValueError("slots and positions must be [N]")
    Hq = 0
    if q is not None:
        if q.dim() != 3 or q.dtype is not dt or q.device != dev or q.shape[0] != N or q.shape[2] != d:
            raise ValueError("q must be [N,Hq,d], of k's type, on its device")
        Hq = q.shape[1]
        q_out = _like(q, q_out, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    opts = None
    if inv_freq is not None:
        if positions is None:
            raise ValueError("positions are needed to rotate")
        opts = ctypes.byref(_rope_opts(inv_freq, d, dev, interleaved, False, scale))
    _check(_call(library().attn_cache_append, dev, _ptr(q), _ptr(q_out), k.data_ptr(), v.data_ptr(),
                 k_pool.data_ptr(), v_pool.data_ptr(), slots.data_ptr(), _ptr(positions), N, Hq, Hkv, d,
                 _dtype_code(k), k_pool.shape[1], k_pool.shape[0], _rows(q), _rows(q_out), _rows(k), _rows(v), opts),
           "attn_cache_append")
    return q_out


@functools.lru_cache(maxsize=256)
def attn_linear_workspace_bytes(B, Hq, max_seqlen, tokens, d) -> int:
    """Bytes of device memory attn_linear_fwd (tokens = B * L) and attn_linear_fwd_varlen (tokens = total)
    work in (may be 0)."""
    return int(library().attn_linear_workspace_bytes(B, Hq, max_seqlen, tokens, d))


def _linear_states(log_decay, state, state_out, state_index, B, Hq, d, device):
    """(state, state_out, num_states) of a linear-attention call, checked."""
    if log_decay.dtype is not torch.float32 or log_decay.shape != (Hq,) or log_decay.device != device or \
            not log_decay.is_contiguous():
        raise ValueError("log_decay must be contiguous fp32 [Hq] on the same device")
    if state_index is not None:
        _ints(device, "state_index", state_index)
        if state_index.shape != (B,):
            raise ValueError("state_index must be [B]")
    if state_out is True:
        if state_index is None:
            state_out = torch.empty((B, Hq, d, d), dtype=torch.float32, device=device)
        elif state is None:
            raise ValueError("with state_index and no state, state_out must be a tensor, None or False")
        else:
            state_out = state
    elif state_out is False:
        state_out = None
    n = None
    for s in (state, state_out):
        if s is None:
            continue
        if s.dtype is not torch.float32 or s.device != device or s.dim() != 4 or s.shape[1:] != (Hq, d, d) or \
                not s.is_contiguous() or (state_index is None and s.shape[0] != B) or n not in (None, s.shape[0]):
            raise ValueError("states must be contiguous fp32 [B,Hq,d,d] ([n,Hq,d,d] with state_index), alike")
        n = s.shape[0]
    return state, state_out, n or 0


def _linear_workspace(workspace, B, Hq, max_seqlen, tokens, d, device):
    need = attn_linear_workspace_bytes(B, Hq, max_seqlen, tokens, d)
    if workspace is None:
        return (torch.empty(need, dtype=torch.uint8, device=device) if need else None), need
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the same device")
    return workspace, workspace.numel() * workspace.element_size()


@_on_stream
def attn_linear_fwd(q, k, v, log_decay, state=None, state_out=True, state_index=None, scale=None, o=None,
                    workspace=None):
    """Linear attention with a decay per head: S_t = e^log_decay S_(t-1) + k_t v_t^T, o_t = scale *
    q_t^T S_t.  q [B,Hq,L,d], k/v [B,Hkv,L,d], log_decay fp32 [Hq] (<= 0).  ``state``: fp32
    [B,Hq,d,d] before the first token (None: 0); ``state_out``: where the last one goes (True: a
    new tensor; ``state`` itself: in place; False: not kept).  With ``state_index`` (int32 [B], -1:
    none) both are a pool's rows, and True means in place.  Returns (o, state_out)."""
    B, Hq, L, d = q.shape
    _check_alike(q, k, v, 4)
    Hkv = k.shape[1]
    if k.shape != (B, Hkv, L, d):
        raise ValueError("k and v must be [B,Hkv,L,d]")
    dev = q.device
    o = _like(q, o, "o")
    state, state_out, n = _linear_states(log_decay, state, state_out, state_index, B, Hq, d, dev)
    work, size = _linear_workspace(workspace, B, Hq, L, B * L, d, dev)
    st = _call(library().attn_linear_fwd, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
               log_decay.data_ptr(), _ptr(state), _ptr(state_out), _ptr(state_index), n, B, Hq, Hkv, L, d,
               _dtype_code(q), _rows(q), _rows(k), _rows(v), _rows(o), float(scale or 0.0), _ptr(work), size)
    _check(st, "attn_linear_fwd")
    return o, state_out


@_on_stream
def attn_linear_fwd_varlen(q, k, v, cu_seqlens, max_seqlen, log_decay, state=None, state_out=True, state_index=None,
                           scale=None, o=None, workspace=None):
    """attn_linear_fwd of packed sequences: q [total,Hq,d], k/v [total,Hkv,d], cu_seqlens int32
    [B+1] on the device, max_seqlen >= every length.  Rows behind the last sequence are not written."""
    total, Hq, d = q.shape
    _check_alike(q, k, v, 3)
    Hkv = k.shape[1]
    if k.shape[0] != total:
        raise ValueError("k and v must be [total,Hkv,d]")
    dev = q.device
    _ints(dev, "cu_seqlens", cu_seqlens)
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [B+1]")
    B = cu_seqlens.shape[0] - 1
    o = _like(q, o, "o")
    state, state_out, n = _linear_states(log_decay, state, state_out, state_index, B, Hq, d, dev)
    work, size = _linear_workspace(workspace, B, Hq, int(max_seqlen), total, d, dev)
    st = _call(library().attn_linear_fwd_varlen, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
               cu_seqlens.data_ptr(), log_decay.data_ptr(), _ptr(state), _ptr(state_out), _ptr(state_index), n, B,
               total, int(max_seqlen), Hq, Hkv, d, _dtype_code(q), _rows(q), _rows(k), _rows(v), _rows(o),
               float(scale or 0.0), _ptr(work), size)
    _check(st, "attn_linear_fwd_varlen")
    return o, state_out


@_on_stream
def attn_linear_step(q, k, v, log_decay, state, state_index=None, scale=None, o=None):
    """One token per sequence: q [B,Hq,d], k/v [B,Hkv,d]; ``state`` (fp32 [B,Hq,d,d], or a pool's rows
    by state_index) is read and updated in place.  Returns o [B,Hq,d]."""
    B, Hq, d = q.shape
    _check_alike(q, k, v, 3)
    Hkv = k.shape[1]
    if k.shape[0] != B:
        raise ValueError("k and v must be [B,Hkv,d]")
    dev = q.device
    o = _like(q, o, "o")
    _, _, n = _linear_states(log_decay, state, state, state_index, B, Hq, d, dev)
    st = _call(library().attn_linear_step, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
               log_decay.data_ptr(), state.data_ptr(), _ptr(state_index), n, B, Hq, Hkv, d, _dtype_code(q),
               _step_strides(q), _step_strides(k), _step_strides(v), _step_strides(o), float(scale or 0.0))
    _check(st, "attn_linear_step")
    return o


def _step_strides(t):
    s = t.stride()
    if s[2] != 1:
        raise ValueError("innermost (head-dim) stride must be 1")
    return _stride_struct(s[0], s[1], 0)


@_on_stream
def attn_splitkv_combine(o_partial, lse_partial, sink=None, dtype=torch.bfloat16, o=None,
                         lse=True, stream=None):
    """Merge split partials.  o_partial fp32 [S,B,Hq,Lq,d], lse_partial fp32 [S,B,Hq,Lq].
    Returns (o [B,Lq,Hq,d] in ``dtype``, lse fp32 [B,Hq,Lq] or None)."""
    S, B, Hq, Lq, d = o_partial.shape
    dev = o_partial.device
    if o_partial.dtype is not torch.float32 or lse_partial.dtype is not torch.float32 or \
            lse_partial.shape != o_partial.shape[:4] or lse_partial.device != dev:
        raise ValueError("o_partial must be fp32 [S,B,Hq,Lq,d], lse_partial fp32 [S,B,Hq,Lq]")
    if o is None:
        o = torch.empty((B, Lq, Hq, d), dtype=dtype, device=dev)
    elif o.shape != (B, Lq, Hq, d) or not o.is_contiguous() or o.device != dev:
        raise ValueError("o must be contiguous [B,Lq,Hq,d]")
    _, lse_t = _outputs(o, o, lse, (B, Hq, Lq))
    sink = _check_sink(sink, Hq, dev)
    # (Held by name until the call: a copy's memory may not go to the next copy.)
    o_partial, lse_partial = o_partial.contiguous(), lse_partial.contiguous()
    st = library().attn_splitkv_combine(_ptr(o_partial), _ptr(lse_partial), S, B, Hq, Lq, d,
                                        _ptr(sink), _ptr(o), _dtype_code(o), _ptr(lse_t),
                                        _stream(stream))
    _check(st, "attn_splitkv_combine")
    return o, lse_t


def attn_device_error() -> int:
    """Synchronises, reads and clears the device error word; returns its bits."""
    bits = ctypes.c_uint(0)
    st = library().attn_device_error(ctypes.byref(bits))
    if st not in (0, 4):
        raise AttnError(st, "attn_device_error")
    return int(bits.value)


def attn_selftest_timeout(timeout_ns: int, stream=None) -> None:
    _check(library().attn_selftest_timeout(int(timeout_ns), _stream(stream)),
           "attn_selftest_timeout")


def attn_last_kernel_name() -> str:
    return library().attn_last_kernel_name().decode()
