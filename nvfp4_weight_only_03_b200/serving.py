"""Binding of the operators between the projections of a decode step: block tables and slot maps
(paged_plan), new rows into the paged cache (kv_append), attention over it (paged_attention), and
adapters beside a projection (lora_add).

    plan = paged_plan(lens, new, table, free, head, block_size, tokens=T)
    kv_append(k, v, k_cache, v_cache, plan.slots)
    o = paged_attention(q, k_cache, v_cache, table, plan.starts, plan.lens)
    y = lora_add(y, x, a, b, index, scales)  # y += scales[i] * B_i (A_i x), i = index[row]

Lengths, tables and indexes stay on the device: no call copies anything to the host or waits, and
a captured call serves later lengths.  Every tensor of a call lies on one device, which need not
be the current one; the call runs on that device's current stream unless `stream` names another,
on which the inputs must then be ready.  Outputs that a call makes are allocated for the stream
it runs on.  Threads may call at the same time, on one stream or several; a workspace that a caller
passes serves one call at a time, while it is enqueued and while it runs.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import threading
from typing import NamedTuple, Optional

import torch

KV_BF16, KV_E4M3 = 0, 1
MAX_REQUESTS = 8192
MAX_RANK = 128

_lib = None  # the loaded library, set by declare

_p, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class KvCacheStruct(ctypes.Structure):
    """nvfp4_kv_cache_t."""
    _fields_ = [("k", _p), ("v", _p), ("type", _i32), ("heads", _i32), ("dim", _i32),
                ("block_size", _i32), ("blocks", _i64), ("block_stride", _i64),
                ("slot_stride", _i64), ("head_stride", _i64), ("k_scale", _f32),
                ("v_scale", _f32)]


class PlanStruct(ctypes.Structure):
    """nvfp4_paged_plan_t."""
    _fields_ = [("lens", _p), ("new_tokens", _p), ("requests", _i32), ("block_size", _i32),
                ("table", _p), ("ld_table", _i64), ("table_columns", _i64), ("free_pages", _p),
                ("free_count", _i64), ("head", _p), ("tokens", _i64), ("starts", _p),
                ("lens_out", _p), ("slots", _p), ("request", _p), ("positions", _p),
                ("head_out", _p), ("missing", _p)]


class AttnStruct(ctypes.Structure):
    """nvfp4_paged_attn_t."""
    _fields_ = [("q", _p), ("ldq", _i64), ("q_head_stride", _i64), ("o", _p), ("ldo", _i64),
                ("o_head_stride", _i64), ("tokens", _i64), ("heads", _i32), ("requests", _i32),
                ("table", _p), ("ld_table", _i64), ("table_columns", _i64), ("starts", _p),
                ("lens", _p), ("scale", _f32)]


class LoraStruct(ctypes.Structure):
    """nvfp4_lora_t."""
    _fields_ = [("a", _p), ("a_stride", _i64), ("a_ld", _i64), ("b", _p), ("b_stride", _i64),
                ("b_ld", _i64), ("scales", _p), ("ranks", _p), ("index", _p), ("adapters", _i32),
                ("rank", _i32)]


def declare(L) -> None:
    """Argument types of the entry points bound here."""
    sz = ctypes.c_size_t
    kv = ctypes.POINTER(KvCacheStruct)
    L.nvfp4_paged_plan.argtypes = [ctypes.POINTER(PlanStruct), _p]
    L.nvfp4_kv_append.argtypes = [_p, _i64, _i64, _p, _i64, _i64, _i64, _p, kv, _p]
    L.nvfp4_paged_attn_workspace_bytes.argtypes = [ctypes.c_int, ctypes.POINTER(sz)]
    L.nvfp4_paged_attn.argtypes = [ctypes.POINTER(AttnStruct), kv, _p, sz, _p]
    L.nvfp4_lora_workspace_bytes.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, _i64,
                                             ctypes.POINTER(sz)]
    L.nvfp4_lora_add.argtypes = [ctypes.POINTER(LoraStruct), _p, _i64, _p, _i64, _p, _i64,
                                 ctypes.c_int, _i64, _i64, _p, sz, _p]
    L.nvfp4_lora_check.argtypes = L.nvfp4_lora_add.argtypes[:-3]
    for f in (L.nvfp4_paged_plan, L.nvfp4_kv_append, L.nvfp4_paged_attn_workspace_bytes,
              L.nvfp4_paged_attn, L.nvfp4_lora_workspace_bytes, L.nvfp4_lora_add,
              L.nvfp4_lora_check):
        f.restype = ctypes.c_int
    global _lib
    _lib = L


def _load():
    return _nv().lib()


def _nv():
    import nvfp4_weight_only_03_b200 as nv
    return nv


# A call takes tens of microseconds on the device at most, so what it does on the host counts:
# the usual case (the tensors' device is current, no stream given) asks torch for plain numbers
# only; any other enters the device and the stream and starts again.  (A torch without these, as one
# built for CPUs, has the public functions, which are slower or raise when they are called.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing",
                     torch.cuda.is_current_stream_capturing)
_I32, _BF16, _F8, _F32 = torch.int32, torch.bfloat16, torch.float8_e4m3fn, torch.float32


def _elsewhere(first: torch.Tensor, stream) -> bool:
    """Whether the call has to enter another device or stream first."""
    index = first.get_device()
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    return stream is not None or index != _current_device()


@contextlib.contextmanager
def _entered(first: torch.Tensor, stream):
    dev = first.device
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(_nv()._stream_obj(stream, dev)):
                yield


def _same_device(index: int, name: str, t: torch.Tensor) -> None:
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _ints(t: torch.Tensor, name: str, n: int, index: int) -> int:
    """Address of n contiguous int32 on the call's device."""
    if t.dtype is not _I32:
        raise TypeError(f"{name} must be int32")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous [{n}], got {list(t.shape)}")
    if t.get_device() != index:
        _same_device(index, name, t)
    return t.data_ptr()


def _table_args(table: torch.Tensor, rows: int, index: int):
    if table.dtype is not _I32:
        raise TypeError("table must be int32")
    shape, stride = table.shape, table.stride()
    if len(shape) != 2 or shape[0] != rows or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"table must be [{rows}][columns] with unit inner stride")
    if table.get_device() != index:
        _same_device(index, "table", table)
    cols = shape[1]
    return cols, stride[0] if rows > 1 else cols


def _heads(t: torch.Tensor, name: str, index: int):
    """(token stride, head stride) of a bf16 [tokens][heads][dim] view."""
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be bfloat16")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or stride[2] != 1:
        raise ValueError(f"{name} must be [tokens][heads][dim] with unit inner stride")
    if t.get_device() != index:
        _same_device(index, name, t)
    n, h, d = shape
    head = stride[1] if h > 1 else d
    return stride[0] if n > 1 else max(h * head, d), head


def _cache_args(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: float, v_scale: float,
                index: int) -> KvCacheStruct:
    dtype = k_cache.dtype
    if (dtype is not _BF16 and dtype is not _F8) or v_cache.dtype is not dtype:
        raise TypeError("k_cache and v_cache must both be bfloat16 or both float8_e4m3fn")
    shape = k_cache.shape
    if len(shape) != 4 or shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must be [blocks][block_size][heads][dim]")
    blocks, block, heads, dim = shape
    stride, other = k_cache.stride(), v_cache.stride()
    page, slot, head, one = stride
    same = stride == other
    if heads == 1 or blocks <= 1 or not same:  # the stride of a single head or page says nothing
        def used(st):
            return (st[0] if blocks > 1 else block * st[1], st[1], st[2] if heads > 1 else dim,
                    st[3])
        page, slot, head, one = used(stride)
        same = used(other) == (page, slot, head, one)
    if one != 1 or not same:
        raise ValueError("k_cache and v_cache must have the same strides, the inner one 1")
    if k_cache.get_device() != index or v_cache.get_device() != index:
        _same_device(index, "k_cache", k_cache)
        _same_device(index, "v_cache", v_cache)
    return KvCacheStruct(k_cache.data_ptr(), v_cache.data_ptr(),
                         KV_BF16 if dtype is _BF16 else KV_E4M3, heads, dim, block, blocks, page,
                         slot, head, k_scale, v_scale)


def _workspace(kind: str, dim: int, index: int, st: int):
    """(workspace, its address, bytes, lock) for paged_attention of this head dim, or for any
    lora_add: the cached one of (device, current stream), or, while a graph is captured, one of the
    graph's own: two graphs never share one.  A call holds the lock while it enqueues: it may be two
    launches that hand data over in the workspace, and another thread's, on the same stream, may not
    come between them (the library is called without the interpreter's lock)."""
    capturing = _capturing()
    found = None if capturing else _workspaces.get((kind, dim, index, st))
    if found is None:
        dev = torch.device("cuda", index)
        if kind == "attn":
            need = paged_attention_workspace_bytes(dim)
        else:
            need = lora_workspace_bytes(_nv().MAX_ROWS, 1, MAX_RANK, 8)  # 64 KB, the most there is
        if capturing:
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
            if kind == "attn":
                ws[:2048].zero_()  # its words that have to be zero (one per SM, and the error word)
        else:
            # this cache holds the stream, so that its handle stays its own
            ws = _nv()._cached_workspace((kind, dim), need, dev, torch.cuda.current_stream(dev))
        found = ws, ws.data_ptr(), ws.numel(), threading.Lock()
        if not capturing:  # (the first thread's, for all)
            found = _workspaces.setdefault((kind, dim, index, st), found)
    return found


_workspaces: dict = {}


def _own_workspace(ws: torch.Tensor, index: int):
    """(address, bytes, lock) of a caller's workspace, which is the caller's to keep to one call at a
    time."""
    _same_device(index, "ws", ws)
    if not ws.is_contiguous():  # (its elements would count for more bytes than lie there in a row)
        raise ValueError("ws must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size(), threading.Lock()


def _fail(status: int, where: str):
    raise _nv().Nvfp4Error(status, where)


class PagedPlan(NamedTuple):
    """What paged_plan computes, all int32 on the device."""
    starts: torch.Tensor     # [requests + 1]: first token of each request, and the total
    lens: torch.Tensor       # [requests]: tokens in the cache once the new ones are there
    slots: torch.Tensor      # [tokens]: cache slot of each token, -1 for none
    request: torch.Tensor    # [tokens]: its request, -1 behind the last token
    positions: torch.Tensor  # [tokens]: its position in the request, 0 behind the last token
    head: torch.Tensor       # [1]: how many of the free list are taken now
    missing: torch.Tensor    # [1]: pages that were wanted and not there


def paged_plan(lens: torch.Tensor, new: torch.Tensor, table: torch.Tensor, free: torch.Tensor,
               head: torch.Tensor, block_size: int, tokens: int,
               out: Optional[PagedPlan] = None, stream=None) -> PagedPlan:
    """Block tables and slot maps of a batch from its requests' lengths (nvfp4_paged_plan).

    lens, new: int32 [requests], tokens in the cache and tokens to come.  table: int32
    [requests][columns], page of each block_size tokens of a request; the pages that the new
    tokens need are taken from free[head:] in request order and written into it (-1 where the
    list is spent).  tokens: length of the per-token outputs; those behind the last token are
    inert (slot -1, request -1, position 0).  out: the outputs to fill, as an earlier call
    returned them (none of them may be one of the inputs); by default new ones."""
    if _elsewhere(lens, stream):
        with _entered(lens, stream):
            return paged_plan(lens, new, table, free, head, block_size, tokens, out)
    index = lens.get_device()
    n = lens.numel()
    if not 0 <= block_size < 1 << 31:  # (a C int would take it for another number)
        raise ValueError("block_size must be in 0..2^31-1")
    cols, ld = _table_args(table, n, index)
    sizes = (n + 1, n, tokens, tokens, tokens, 1, 1)
    if out is None:
        if tokens < 0:
            raise ValueError("tokens must not be negative")
        whole = lens.new_empty(2 * n + 3 + 3 * tokens)
        # (views that do not share a version counter: half the time)
        out = PagedPlan._make(whole.unsafe_split_with_sizes(sizes))
        o0 = whole.data_ptr()
        o1 = o0 + 4 * n + 4
        o2 = o1 + 4 * n
        o3 = o2 + 4 * tokens
        o4 = o3 + 4 * tokens
        o5 = o4 + 4 * tokens
        o6 = o5 + 4
    else:
        o0, o1, o2, o3, o4, o5, o6 = (_ints(t, "out." + name, size, index)
                                      for name, t, size in zip(PagedPlan._fields, out, sizes))
    a = PlanStruct(_ints(lens, "lens", n, index), _ints(new, "new", n, index), n, block_size,
                   table.data_ptr(), ld, cols, _ints(free, "free", free.numel(), index),
                   free.numel(), _ints(head, "head", 1, index), tokens, o0, o1, o2, o3, o4, o5,
                   o6)
    status = (_lib or _load()).nvfp4_paged_plan(a, _raw_stream(index))
    if status:
        _fail(status, "nvfp4_paged_plan")
    return out


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              slots: torch.Tensor, k_scale: float = 1.0, v_scale: float = 1.0,
              stream=None) -> None:
    """Writes the rows of k and v into their slots of the paged cache (nvfp4_kv_append).

    k, v: bfloat16 [tokens][heads][dim], views into a fused projection's rows included.
    k_cache, v_cache: bfloat16 or float8_e4m3fn [blocks][block_size][heads][dim] (any strides
    with an inner one of 1, the same for both); a float8 cache holds e4m3(x / scale).  slots:
    int32 [tokens], page * block_size + place; rows with a negative slot, or one past the last
    page, are skipped.  No two rows should have one slot: it would hold values of either."""
    if _elsewhere(k, stream):
        with _entered(k, stream):
            return kv_append(k, v, k_cache, v_cache, slots, k_scale, v_scale)
    index = k.get_device()
    c = _cache_args(k_cache, v_cache, k_scale, v_scale, index)
    ldk, hk = _heads(k, "k", index)
    ldv, hv = _heads(v, "v", index)
    shape = k.shape
    n = shape[0]
    if shape != v.shape or shape[1] != c.heads or shape[2] != c.dim:
        raise ValueError(f"k and v must be [tokens][{c.heads}][{c.dim}]")
    status = (_lib or _load()).nvfp4_kv_append(
        k.data_ptr(), ldk, hk, v.data_ptr(), ldv, hv, n, _ints(slots, "slots", n, index), c,
        _raw_stream(index))
    if status:
        _fail(status, "nvfp4_kv_append")


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    table: torch.Tensor, starts: torch.Tensor, lens: torch.Tensor,
                    scale: Optional[float] = None, k_scale: float = 1.0, v_scale: float = 1.0,
                    out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                    stream=None, check: bool = False) -> torch.Tensor:
    """Causal attention of each request's newest tokens over its paged cache (nvfp4_paged_attn).

    q: bfloat16 [tokens][heads][dim]; tokens starts[r] .. starts[r+1]-1 are the last ones of
    request r's lens[r], already in the cache.  Query head h reads kv head h // (heads //
    kv_heads).  scale: of the scores, dim ** -0.5 by default.  out: bfloat16 like q (by default a
    new one); its rows behind the last token are not written.  A batch of more tokens than q has
    rows gets those rows, each at its own position.  ws: a workspace of
    paged_attention_workspace_bytes(dim) bytes, zero-filled before its first use; by default
    the cached one of (device, stream), or the graph's own during a capture, which nobody can look
    into: pass one to ask workspace_error(ws) after the replays.  check: synchronise and raise if a
    bounded wait in the kernel gave up (not during a capture)."""
    if _elsewhere(q, stream):
        with _entered(q, stream):
            return paged_attention(q, k_cache, v_cache, table, starts, lens, scale, k_scale,
                                   v_scale, out, ws, None, check)
    if check and _capturing():
        raise ValueError("check=True synchronises, which a capture cannot: ask workspace_error(ws) "
                         "after a replay")
    index = q.get_device()
    c = _cache_args(k_cache, v_cache, k_scale, v_scale, index)
    ldq, hq = _heads(q, "q", index)
    shape = q.shape
    tokens, heads, dim = shape
    if dim != c.dim or heads % max(c.heads, 1):
        raise ValueError(f"q must be [tokens][heads][{c.dim}], heads a multiple of {c.heads}")
    n = lens.numel()
    cols, ld = _table_args(table, n, index)
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else q.new_empty(shape)
        ldo, ho = heads * dim, dim
    else:
        if out.shape != shape:
            raise ValueError(f"out must be {list(shape)}")
        ldo, ho = _heads(out, "out", index)
    st = _raw_stream(index)
    if ws is None:
        ws, ws_at, ws_bytes, lock = _workspace("attn", dim, index, st)
    else:
        ws_at, ws_bytes, lock = _own_workspace(ws, index)
    a = AttnStruct(q.data_ptr(), ldq, hq, out.data_ptr(), ldo, ho, tokens, heads, n,
                   table.data_ptr(), ld, cols, _ints(starts, "starts", n + 1, index),
                   _ints(lens, "lens", n, index), dim ** -0.5 if scale is None else scale)
    lock.acquire()
    try:
        status = (_lib or _load()).nvfp4_paged_attn(a, c, ws_at, ws_bytes, st)
    finally:
        lock.release()
    if status:
        _fail(status, "nvfp4_paged_attn")
    if check:
        _nv()._check_error(ws, st, "nvfp4_paged_attn")
    return out


_attn_bytes: dict = {}
def paged_attention_workspace_bytes(dim: int) -> int:
    """Bytes of a paged_attention workspace for this head dim on the current device."""
    key = (_current_device(), dim)
    need = _attn_bytes.get(key)
    if need is None:
        b = ctypes.c_size_t()
        nv = _nv()
        nv._check(nv.lib().nvfp4_paged_attn_workspace_bytes(dim, ctypes.byref(b)),
                  "nvfp4_paged_attn_workspace_bytes")
        need = _attn_bytes[key] = int(b.value)
    return need


def _rows(t: torch.Tensor, name: str, m: Optional[int], n: int, index: int):
    """(M, row stride) of a bf16 [M][n] view; M is any if m is None."""
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be bfloat16")
    stride = t.stride()
    if len(stride) != 2:
        raise ValueError(f"{name} must be [M][{n}], got {list(t.shape)}")
    ld, one = stride
    rows, columns = t.shape
    if columns != n or (one != 1 and n > 1):
        raise ValueError(f"{name} must be [M][{n}] with unit inner stride, got {list(t.shape)}")
    if rows != m and m is not None:
        raise ValueError(f"{name} must have {m} rows, got {rows}")
    if t.get_device() != index:
        _same_device(index, name, t)
    return rows, ld if rows > 1 else n


def lora_workspace_bytes(m: int, adapters: int, rank: int, k: int) -> int:
    """Bytes of a lora_add workspace on the current device."""
    b = ctypes.c_size_t()
    nv = _nv()
    nv._check(nv.lib().nvfp4_lora_workspace_bytes(m, adapters, rank, k, ctypes.byref(b)),
              "nvfp4_lora_workspace_bytes")
    return int(b.value)


def lora_add(y: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
             index: torch.Tensor, scales: torch.Tensor, ranks: Optional[torch.Tensor] = None,
             out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    """out[m] = bf16(y[m] + scales[i] * B_i (A_i x[m])), i = index[m] (nvfp4_lora_add).

    y: bfloat16 [M][N], a projection of x: bfloat16 [M][K] (M up to 128).  a: bfloat16
    [adapters][rank][K]; b: bfloat16 [adapters][N][rank]; scales: float32 [adapters]; ranks:
    int32 [adapters], how many of `rank` each adapter uses (all by default).  index: int32 [M];
    a row whose index names no adapter (-1) keeps y.  out: y itself for an update in place, or
    a tensor apart from y and x; by default a new one.  ws: lora_workspace_bytes(M, adapters,
    rank, K) bytes of any content, by default the cached workspace of (device, stream)."""
    if _elsewhere(y, stream):
        with _entered(y, stream):
            return lora_add(y, x, a, b, index, scales, ranks, out, ws)
    return _lora(y, x, a, b, index, scales, ranks, out, ws, False)


def lora_behind(y: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                index: torch.Tensor, scales: torch.Tensor, ranks: Optional[torch.Tensor]):
    """Checks lora_add(y, ..., out=y) before the work that writes y is enqueued, and returns what
    enqueues it behind that work, given the stream."""
    if y.get_device() < 0:
        raise ValueError("tensors must be on a CUDA device")
    return _lora(y, x, a, b, index, scales, ranks, y, None, True)


def _lora(y, x, a, b, index, scales, ranks, out, ws, later: bool):
    """lora_add on the current device and stream; or, later, its checks and what then makes the call."""
    if x.dim() == 1:
        x = x.unsqueeze(0)
    dev = y.get_device()
    if a.dtype is not _BF16 or b.dtype is not _BF16:
        raise TypeError("a and b must be bfloat16")
    sa, sb, shape = a.stride(), b.stride(), b.shape
    if len(sa) != 3 or len(sb) != 3:
        raise ValueError("a must be [adapters][rank][K] and b [adapters][N][rank]")
    s, rank, k = a.shape
    adapters, n, columns = shape
    if adapters != s or columns != rank:
        raise ValueError(f"b must be [{s}][N][{rank}], got {list(shape)}")
    if (k > 1 and sa[2] != 1) or (rank > 1 and sb[2] != 1):
        raise ValueError("a and b must have unit inner strides")
    if a.get_device() != dev or b.get_device() != dev or scales.get_device() != dev:
        for name, t in (("a", a), ("b", b), ("scales", scales)):
            _same_device(dev, name, t)
    m, ldy = _rows(y, "y", None, n, dev)
    _, ldx = _rows(x, "x", m, k, dev)
    if scales.dtype is not _F32:
        raise TypeError("scales must be float32")
    if scales.shape != (s,) or not scales.is_contiguous():
        raise ValueError(f"scales must be contiguous [{s}]")
    if out is None:
        out = torch.empty_like(y) if ldy == n else y.new_empty((m, n))
        ldo = n
    else:
        ldo = ldy if out is y else _rows(out, "out", m, n, dev)[1]
    l = LoraStruct(a.data_ptr(), sa[0] if s > 1 else rank * k, sa[1] if rank > 1 else k,
                   b.data_ptr(), sb[0] if s > 1 else n * rank, sb[1] if n > 1 else rank,
                   scales.data_ptr(), None if ranks is None else _ints(ranks, "ranks", s, dev),
                   _ints(index, "index", m, dev), s, rank)
    lib = _lib or _load()
    if later:
        args = (l, x.data_ptr(), ldx, y.data_ptr(), ldy, out.data_ptr(), ldo, m, n, k)
        status = lib.nvfp4_lora_check(*args)
        if status:
            _fail(status, "nvfp4_lora_add")
        return functools.partial(_lora_later, y, dev, args)
    st = _raw_stream(dev)
    if ws is None:
        ws, ws_at, ws_bytes, lock = _workspace("lora", 0, dev, st)
    else:
        ws_at, ws_bytes, lock = _own_workspace(ws, dev)
    lock.acquire()  # (half the time of a with statement)
    try:
        status = lib.nvfp4_lora_add(l, x.data_ptr(), ldx, y.data_ptr(), ldy, out.data_ptr(), ldo, m, n,
                                    k, ws_at, ws_bytes, st)
    finally:
        lock.release()
    if status:
        _fail(status, "nvfp4_lora_add")
    return out


def _lora_later(y: torch.Tensor, dev: int, args, stream) -> None:
    if _elsewhere(y, stream):
        with _entered(y, stream):
            return _lora_later(y, dev, args, None)
    st = _raw_stream(dev)
    _, ws_at, ws_bytes, lock = _workspace("lora", 0, dev, st)
    with lock:
        status = _lib.nvfp4_lora_add(*args, ws_at, ws_bytes, st)
    if status:
        _fail(status, "nvfp4_lora_add")
