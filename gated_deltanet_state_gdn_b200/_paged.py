"""Binding of the paged key-value cache's entry points (argument marshalling only).

As in _binding: torch CUDA tensors in, checks of dtypes and shapes, outputs and workspaces from
torch's allocator, one call of the C entry point of the same name.  A call runs on ``stream``, or
on the current stream of the tensors' device; what it allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes
import functools
import math
import struct

import torch

from . import _binding as b

_DTYPES = {torch.bfloat16: b.GDN_BF16, torch.float16: b.GDN_F16}
_CACHE_DTYPES = {**_DTYPES, torch.float8_e4m3fn: b.GDN_E4M3}
_I32 = torch.int32
_NO_WINDOW = 1 << 30          # positions a row can hold at most: as far as a window can reach


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("rows", ctypes.c_int32), ("width", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class _Table(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("ref_count", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("rows", ctypes.c_int32), ("width", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32)]


# the bytes of the two, packed at once: filling a ctypes structure field by field would be a tenth
# of a small call's host time
_CACHE_BYTES = struct.Struct("@PPqqqPPPPqiiiiiii4x")
_TABLE_BYTES = struct.Struct("@PPPqiiii")


class _Pool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64),
                ("row_bytes", ctypes.c_int64)]


def _on_stream(first):
    """The call's device and stream: those of argument `first` unless they are current already."""
    def wrap(f):
        @functools.wraps(f)
        def call(*args, stream=None, **kw):
            t = args[0] if args else kw.get(first)
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise TypeError(f"{first} must be a CUDA tensor")
            if stream is not None:
                if stream.device != t.device:
                    raise ValueError(f"stream is on {stream.device}, {first} on {t.device}")
                with torch.cuda.stream(stream):
                    return f(*args, **kw)
            if t.get_device() != torch._C._cuda_getDevice():
                with torch.cuda.device(t.device):
                    return f(*args, **kw)
            return f(*args, **kw)
        return call
    return wrap


def _stream(device):
    """The current stream of `device`, as an address (torch.cuda.current_stream would make an
    object of it first, at a third of a small call's host time)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _at(t):
    return None if t is None else t.data_ptr()


def _here(t):
    return 0 if t is None else t.data_ptr()


def _status(t, device):
    """The status word, which the kernels write to: its address."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != _I32 or t.numel() < 1:
        raise TypeError(f"dev_status must be an int32 tensor on {device}")
    return t.data_ptr()


@functools.lru_cache(maxsize=256)
def _attn_workspace(lib, device, *sizes):
    """gdn_paged_attn_workspace_size: it depends on the device and these sizes alone."""
    return lib.gdn_paged_attn_workspace_size(*sizes)


def _tensor(name, t, dtype, shape, device, dense=True):
    """A tensor of the call as it is (written in place, or read where it lies)."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise TypeError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ints(name, t, n, device):
    """An int32 list that the call only reads."""
    if t is None:
        return None
    t = _tensor(name, t, _I32, (n,), device, dense=False)
    return t if t.is_contiguous() else t.contiguous()


def _rows_of(block_table, device):
    if not isinstance(block_table, torch.Tensor) or block_table.device != device \
            or block_table.dtype != _I32 or block_table.dim() != 2:
        raise TypeError(f"block_table must be a 2-d int32 tensor on {device}")
    rows, width = block_table.shape
    if width > 1 and block_table.stride(1) != 1:
        raise ValueError("the rows of block_table must be dense")
    return rows, width, block_table.stride(0)


def _cache(k_cache, v_cache, block_table, seq_lens, k_scale, v_scale):
    """The bytes of the call's gdn_paged_cache; its heads, head_dim, dtype code and rows."""
    dtype, device = k_cache.dtype, k_cache.device
    code = _CACHE_DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"k_cache must be bf16, fp16 or float8_e4m3fn, got {dtype}")
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, page_size, heads, head_dim]")
    _tensor("v_cache", v_cache, dtype, k_cache.shape, device, dense=False)
    P, S, H, D = k_cache.shape
    st, sv = k_cache.stride(), v_cache.stride()
    if D > 1 and (st[3] != 1 or sv[3] != 1):
        raise ValueError("the last dimension of k_cache and v_cache must be dense")
    if st != sv and any(x != y and n > 1 for x, y, n in zip(st, sv, k_cache.shape)):
        raise ValueError("k_cache and v_cache must have the same strides")
    rows, width, stride = _rows_of(block_table, device)
    _tensor("seq_lens", seq_lens, _I32, (rows,), device)
    if k_scale is not None:
        _tensor("k_scale", k_scale, torch.float32, (H,), device)
    if v_scale is not None:
        _tensor("v_scale", v_scale, torch.float32, (H,), device)
    return _CACHE_BYTES.pack(k_cache.data_ptr(), v_cache.data_ptr(), st[0], st[1], st[2],
                             _here(k_scale), _here(v_scale), block_table.data_ptr(),
                             seq_lens.data_ptr(), stride, rows, width, P, S, H, D, code), H, D, code, rows


def _row_strides(name, t, heads, D, unit):
    """[..., heads, D] as tokens by heads: the tensor and its strides; copied where its tokens are
    not evenly spaced or do not start on multiples of `unit` elements."""
    if t.dim() < 3 or t.shape[-1] != D or (heads and t.shape[-2] != heads):
        raise ValueError(f"{name} must be [..., {heads or 'heads'}, {D}]")
    st, sh = t.stride(), t.shape
    ok = (D == 1 or st[-1] == 1) and t.data_ptr() % (unit * 2) == 0
    ok = ok and (sh[-2] == 1 or st[-2] % unit == 0)
    n, ts = 1, 0                    # tokens so far, from the innermost axis, and their stride
    for i in range(t.dim() - 3, -1, -1):
        if sh[i] == 1:
            continue
        if n == 1:
            ts = st[i]
        elif st[i] != n * ts:
            ok = False
        n *= sh[i]
    if not ok or (n > 1 and ts % unit):
        t = t.clone(memory_format=torch.contiguous_format)
        return t, t.stride(-3) if t.dim() > 2 else 0, t.stride(-2)
    return t, ts, st[-2]


def _raise(status, where):
    if status != b.GDN_OK:
        raise b.GdnError(status, where)


@_on_stream("k")
def gdn_kv_append(k, v, k_cache, v_cache, block_table, seq_lens, slots=None, row_offsets=None, *,
                  k_scale=None, v_scale=None, dev_status=None):
    """Write new tokens' keys and values to the pages of their positions.

    k, v: [N, heads, D] ([1, N, heads, D] likewise) or [B, T, heads, D], bf16 or fp16 (views of a
    packed projection are read where they lie); k_cache, v_cache: [num_pages, page_size, heads, D]
    of the same type or float8_e4m3fn (any strides with D dense, the same for both), written in
    place; block_table: [rows, width] int32; seq_lens: [rows] int32, counting the new tokens already; slots: [B]
    int32 rows of the table (negative: padding) or None (request b is row b); row_offsets: [B+1]
    int32, or None for equally many tokens a request; k_scale, v_scale: [heads] fp32 or None,
    for an 8-bit cache.  Returns (k_cache, v_cache).
    """
    dt = _DTYPES.get(k.dtype)
    if dt is None:
        raise TypeError(f"k must be bf16 or fp16, got {k.dtype}")
    cache, heads, D, _, rows = _cache(k_cache, v_cache, block_table, seq_lens, k_scale, v_scale)
    device = k.device
    if k_cache.device != device:
        raise TypeError(f"k_cache must be on {device}")
    _tensor("v", v, k.dtype, k.shape, device, dense=False)
    k, kt, kh = _row_strides("k", k, heads, D, 8)
    v, vt, vh = _row_strides("v", v, heads, D, 8)
    N = math.prod(k.shape[:-2])
    if slots is not None:
        B = slots.shape[0]
    elif row_offsets is not None:
        B = row_offsets.shape[0] - 1
    else:
        B = k.shape[0] if k.dim() == 4 else rows
    if k.dim() == 4 and row_offsets is None and k.shape[0] not in (1, B):
        raise ValueError(f"k has {k.shape[0]} requests, slots {B}")
    slots = _ints("slots", slots, B, device)
    row_offsets = _ints("row_offsets", row_offsets, B + 1, device)
    _raise(b.lib().gdn_kv_append(_at(k), _at(v), kt, kh, vt, vh, cache,
                                 _at(slots), _at(row_offsets), B, N, dt,
                                 _status(dev_status, device), _stream(device)), "gdn_kv_append")
    return k_cache, v_cache


@_on_stream("q")
def gdn_paged_attn(q, k_cache, v_cache, block_table, seq_lens, slots=None, *, scale=None,
                   window: int = 0, k_scale=None, v_scale=None, out=None, lse=None,
                   return_lse: bool = False, dev_status=None):
    """Softmax attention of each request's last T tokens over its pages.

    q: [B, T, Hq, D] bf16 or fp16 (a view of a packed projection is read where it lies); the
    cache and its tables as for gdn_kv_append, which has written the T tokens; slots: [B] int32
    rows of the table (negative: padding, whose rows of a given ``out`` and ``lse`` keep their
    values and are zeros and -inf otherwise) or None (request b is row b); ``scale`` None
    selects 1/sqrt(D); ``window`` > 0 limits a token to the last that many positions.
    Returns out [B, T, Hq, D], with ``return_lse`` or ``lse`` also lse [B, T, Hq] fp32.
    """
    dt = _DTYPES.get(q.dtype)
    if dt is None:
        raise TypeError(f"q must be bf16 or fp16, got {q.dtype}")
    if q.dim() != 4:
        raise ValueError("q must be [B, T, Hq, D]")
    B, T, Hq, D = q.shape
    device = q.device
    if k_cache.device != device:
        raise TypeError(f"k_cache must be on {device}")
    cache, heads, cache_dim, code, _ = _cache(k_cache, v_cache, block_table, seq_lens, k_scale, v_scale)
    q, qt, qh = _row_strides("q", q, 0, cache_dim, 2)
    slots = _ints("slots", slots, B, device)
    # Padding rows of a given tensor are kept.  Where both are made here the call clears theirs; one
    # made beside a given one is cleared first.
    flags = b.GDN_ZERO_PADDING if out is None and lse is None else 0
    if lse is not None:
        _tensor("lse", lse, torch.float32, (B, T, Hq), device)
    elif return_lse:
        lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float32, device=device) \
            if out is not None else q.new_empty((B, T, Hq), dtype=torch.float32)
    if out is not None:
        _tensor("out", out, q.dtype, (B, T, Hq, D), device)
    elif flags:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        out = torch.zeros((B, T, Hq, D), dtype=q.dtype, device=device)
    L = b.lib()
    nbytes = _attn_workspace(L, device, B, T, Hq, heads, D, code)
    ws = q.new_empty((max(nbytes, 16),), dtype=torch.uint8)
    _raise(L.gdn_paged_attn(_at(q), qt, qh, cache, _at(slots), B, T, Hq, dt,
                            1.0 / math.sqrt(D) if scale is None else float(scale), min(int(window), _NO_WINDOW),
                            _at(out), _at(lse), flags, _at(ws), nbytes,
                            _status(dev_status, device), _stream(device)), "gdn_paged_attn")
    return out if lse is None else (out, lse)


def _table(block_table, ref_count, seq_lens, page_size):
    """The bytes of the call's gdn_page_table; its rows and pages."""
    device = block_table.device
    rows, width, stride = _rows_of(block_table, device)
    _tensor("seq_lens", seq_lens, _I32, (rows,), device)
    if not isinstance(ref_count, torch.Tensor) or ref_count.dim() != 1:
        raise TypeError(f"ref_count must be a 1-d int32 tensor on {device}")
    pages = ref_count.shape[0]
    _tensor("ref_count", ref_count, _I32, (pages,), device)
    return _TABLE_BYTES.pack(block_table.data_ptr(), ref_count.data_ptr(), seq_lens.data_ptr(), stride,
                             rows, width, pages, int(page_size)), rows, pages


def _pools(pools, rows, device):
    """The arrays of a call: dimension 0 counts pages (or slots), the others are one dense block.
    Arrays without elements (windows of a conv of one tap) have nothing to copy."""
    if isinstance(pools, torch.Tensor):
        raise TypeError("pools must be a list of tensors")
    if not pools:
        return None, 0
    out = (_Pool * len(pools))()
    count = 0
    for i, t in enumerate(pools):
        if not isinstance(t, torch.Tensor) or t.device != device or t.dim() < 1:
            raise TypeError(f"pools[{i}] must be a tensor on {device}")
        if t.shape[0] != rows:
            raise ValueError(f"pools[{i}] must have {rows} rows, got {t.shape[0]}")
        n = t.numel() // rows
        if n == 0:
            continue
        if not t.is_contiguous():
            dense = 1           # the axes of a row, from the innermost, without holes
            for st, sz in sorted((s, z) for s, z in zip(t.stride()[1:], t.shape[1:]) if z > 1):
                if st != dense:
                    raise ValueError(f"the rows of pools[{i}] must be dense")
                dense *= sz
        stride = t.stride(0) if rows > 1 else n
        out[count] = _Pool(t.data_ptr(), stride * t.element_size(), n * t.element_size())
        count += 1
    return out, count


@_on_stream("block_table")
def gdn_page_resize(block_table, ref_count, seq_lens, row_list, new_lens, page_size: int,
                    pools=(), *, dev_status=None):
    """Give the listed rows of the page table new lengths: rows that get shorter give their pages
    back (0 frees a row), rows that get longer take the lowest-numbered free ones and a copy of a
    partly filled last page that they share.

    block_table: [rows, width] int32; ref_count: [num_pages] int32; seq_lens: [rows] int32, all
    updated in place; row_list, new_lens: [n] int32 (negative row: padding); pools: the tensors
    whose dimension 0 counts pages (keys and values of every layer), copied in place.
    Returns (block_table, ref_count, seq_lens).
    """
    device = block_table.device
    t, rows, num_pages = _table(block_table, ref_count, seq_lens, page_size)
    n = row_list.shape[0]
    row_list = _ints("row_list", row_list, n, device)
    new_lens = _ints("new_lens", new_lens, n, device)
    arr, count = _pools(pools, num_pages, device)
    L = b.lib()
    nbytes = L.gdn_page_workspace_size(num_pages, max(n, 1))
    ws = block_table.new_empty((nbytes,), dtype=torch.uint8)
    _raise(L.gdn_page_resize(t, _at(row_list), _at(new_lens), n, arr, count,
                             _at(ws), nbytes, _status(dev_status, device), _stream(device)),
           "gdn_page_resize")
    return block_table, ref_count, seq_lens


@_on_stream("block_table")
def gdn_page_fork(block_table, ref_count, seq_lens, parents, children, page_size: int, pools=(),
                  *, dev_status=None):
    """Make rows `children` of the page table copies of rows `parents`, sharing their pages.

    Tables as for gdn_page_resize, updated in place; parents, children: [n] int32 (negative:
    padding); pools: the tensors whose dimension 0 counts slots (the state pools of gdn_decode,
    the windows of gdn_conv1d), the rest of each one dense block (of a state pool with padded
    heads pass the heads, ``pool.unbind(1)``): row child becomes a copy of row parent.  What a
    child held is given back.  Returns (block_table, ref_count, seq_lens).
    """
    device = block_table.device
    t, rows, num_pages = _table(block_table, ref_count, seq_lens, page_size)
    n = parents.shape[0]
    parents = _ints("parents", parents, n, device)
    children = _ints("children", children, n, device)
    arr, count = _pools(pools, rows, device)
    _raise(b.lib().gdn_page_fork(t, _at(parents), _at(children), n, arr,
                                 count, _status(dev_status, device), _stream(device)), "gdn_page_fork")
    return block_table, ref_count, seq_lens


@_on_stream("block_table")
def gdn_page_compact(block_table, ref_count, seq_lens, page_size: int, pools=(), *,
                     page_map=None, dev_status=None):
    """Move the used pages to the lowest numbers, in every pool; tables follow.

    Tables and pools as for gdn_page_resize, updated in place.  Returns page_map [num_pages]
    int32: the new number of each used page, -1 for free ones.
    """
    device = block_table.device
    t, rows, num_pages = _table(block_table, ref_count, seq_lens, page_size)
    arr, count = _pools(pools, num_pages, device)
    if page_map is None:
        page_map = block_table.new_empty((num_pages,))
    else:
        _tensor("page_map", page_map, _I32, (num_pages,), device)
    L = b.lib()
    nbytes = L.gdn_page_workspace_size(num_pages, 0)
    ws = block_table.new_empty((nbytes,), dtype=torch.uint8)
    _raise(L.gdn_page_compact(t, _at(page_map), arr, count, _at(ws), nbytes,
                              _status(dev_status, device), _stream(device)), "gdn_page_compact")
    return page_map
