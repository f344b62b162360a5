"""KV-outer block-sparse attention over a paged KV cache, for GB300 (sm_103a).

Thin Python binding over the C ABI of ``libsa.so`` (``include/sa.h``).  The
functions carry the same names as the C entry points and do argument
marshalling only: every step of the method runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.

The three steps (crate alice-llm 2.0.0, module sparse_attention):

* :func:`sa_build_index` - CSR index keyed by (kv head, sparse block)
  (``types.rs``, KvOuterIndex);
* :func:`sa_forward` - per-edge partials o, m, l (``forward.rs``,
  kvouter_forward);
* :func:`sa_combine` - log-sum-exp merge per (query, q-head);
* :func:`sa_forward_combine` - steps 2 and 3 on a built index (one fused
  kernel for batches of one query per sequence);
* :func:`sa_attention` - the three on one stream without a host sync.

Around them, for serving:

* :func:`sa_store_kv` - new tokens' K/V into the paged cache (f32, bf16, or 8
  bits with a scale per page and kv head);
* :func:`sa_block_bounds` - the smallest and largest key per channel of the
  blocks that got new tokens;
* :func:`sa_select_blocks` - each query's topk blocks by those bounds: the
  ``selected`` of the steps above;
* :func:`sa_norm_rope` - before the store: head norms and position rotation of
  the new queries and keys;
* :func:`sa_decode_attention` - one new token per sequence over its whole cache
  or a window of it, without a selection;
* :func:`sa_load_kv` - rows of the cache read back.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass

import numpy as np
import torch

from . import _native
from ._native import (DTYPE_BF16, DTYPE_E4M3, DTYPE_F32, DTYPE_INT8, PATH_AUTO, PATH_CUDA_CORE, PATH_CUDA_CORE_GENERAL,
                      PATH_FUSED_DECODE, PATH_TENSOR_CORE, PATH_TENSOR_CORE_TF32, STATUS_NAMES)

__all__ = ["SAError", "Index", "sa_index_query_sizes", "sa_build_index",
           "sa_build_index_no_alloc", "sa_forward", "sa_forward_combine", "sa_forward_kernel_name",
           "sa_attention_kernel_name", "PATH_FUSED_DECODE",
           "sa_combine", "sa_attention", "sa_store_kv", "sa_block_bounds", "sa_select_blocks",
           "allocate_select_workspace", "sa_norm_rope", "sa_load_kv", "sa_decode_attention",
           "allocate_decode_workspace", "sa_get_status", "sa_clear_status", "sa_status_string",
           "sa_version", "allocate_index", "PATH_AUTO", "PATH_CUDA_CORE", "PATH_TENSOR_CORE",
           "PATH_TENSOR_CORE_TF32",
           "PATH_CUDA_CORE_GENERAL", "AttentionGraph", "sa_debug_stall", "sa_debug_cta_stats", "STALL_NONE",
           "STALL_INDEX_BARRIER", "STALL_FUSED_COPIES", "STALL_SELECT_COPIES"]

#: sa_debug_stall sites (a test hook: see include/sa.h)
STALL_NONE, STALL_INDEX_BARRIER, STALL_FUSED_COPIES, STALL_SELECT_COPIES = 0, 1, 2, 3


class SAError(RuntimeError):
    """A non-OK sa_status returned by the library."""

    def __init__(self, code: int, where: str):
        self.code = int(code)
        self.kind = STATUS_NAMES.get(self.code, f"UNKNOWN({code})")
        text = _native.load().sa_status_string(self.code).decode()
        super().__init__(f"{where}: {self.kind} ({text})")


def _causal(causal) -> int:
    """The C ABI's causal mode: 0 none, 1 right-aligned (the pages' rule), 2
    left-aligned (opt-in); booleans map to 0 / 1."""
    if isinstance(causal, (bool, np.bool_)):
        return int(causal)
    c = int(causal)
    if c not in (0, 1, 2):
        raise ValueError(f"causal must be 0, 1 or 2, got {causal!r}")
    return c


def _check(code: int, where: str) -> None:
    if code != _native.SA_OK:
        raise SAError(code, where)


def _ptr(t):
    """An address argument (ctypes takes the integer as it is)."""
    return None if t is None else t.data_ptr()


def _stream(stream, device):
    if stream is None:
        return _raw_stream(device)
    return stream.cuda_stream


def _allocating(stream):
    """Where a call makes its buffers: on the stream that is going to use them, so
    that memory freed elsewhere and still in use there is not handed out (the
    current stream where the call names none)."""
    return torch.cuda.stream(stream) if isinstance(stream, torch.cuda.Stream) else _NOTHING


_NOTHING = contextlib.nullcontext()


def _raw_stream(device):
    """The current stream's handle, without a Stream object where torch offers it."""
    index = device.index
    if _current_raw_stream is None or index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _current_raw_stream(index)


_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_HostWords = ctypes.c_int64 * 1


def _host_ptr(a: np.ndarray):
    """The address of a host array's data, as a pointer argument (a view of its
    buffer where it gives one, which is the quicker way)."""
    try:
        return _HostWords.from_buffer(a)
    except (TypeError, ValueError):      # read-only, or shorter than a word
        return a.__array_interface__["data"][0]


def _host_i64(a) -> np.ndarray:
    if type(a) is np.ndarray and a.dtype == np.int64 and a.flags.c_contiguous:
        return a
    if isinstance(a, torch.Tensor):
        a = a.detach().cpu().numpy()
    return np.ascontiguousarray(a, dtype=np.int64)


def _require(t, dtype, name, device=None):
    # the usual case in three calls; what is wrong is found out below
    try:
        if (t.dtype is dtype and t.is_contiguous() and
                (t.is_cuda if device is None else t.device == device)):
            return t
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _alike(index, dtype, *tensors) -> bool:
    """Whether all are contiguous CUDA tensors of device ``index`` and ``dtype``:
    the usual case of the checks below, in few calls (a decode step's call is
    shorter on the GPU than its checks on the host).  Where not, the checks
    one by one say what is wrong."""
    for t in tensors:
        if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
            return False
    return True


def sa_status_string(code: int) -> str:
    return _native.load().sa_status_string(int(code)).decode()


def sa_version() -> str:
    return _native.load().sa_version().decode()


def sa_index_query_sizes(tq, hkv, topk, batch, max_pages, block_size, page_size) -> dict:
    s = _native.SaIndexSizes()
    _check(_native.load().sa_index_query_sizes(tq, hkv, topk, batch, max_pages, block_size,
                                               page_size, ctypes.byref(s)),
           "sa_index_query_sizes")
    return {name: getattr(s, name) for name, _ in s._fields_}


@dataclass
class Index:
    """Device arrays of one KV-outer index plus the C struct that points at them."""

    sel_slots: torch.Tensor
    sel_offsets: torch.Tensor
    num_sel: torch.Tensor
    edge_head_base: torch.Tensor
    edges: torch.Tensor
    inv: torch.Tensor
    splits: torch.Tensor
    totals: torch.Tensor
    workspace: torch.Tensor
    sizes: dict
    c: _native.SaIndex

    @property
    def device(self):
        return self.totals.device

    def to_host(self) -> dict:
        """Copies of the index arrays, shaped and trimmed like the oracle's."""
        c = self.c
        tot = self.totals.cpu().numpy()
        E, S, U = int(tot[0]), int(tot[1]), int(tot[2])
        hkv, nbs, tq, topk = c.hkv, c.nbs, c.tq, c.topk
        return {
            "sel_slots": self.sel_slots[: hkv * nbs].cpu().numpy().reshape(hkv, nbs),
            "sel_offsets": self.sel_offsets.cpu().numpy().reshape(hkv, nbs + 1),
            "num_sel": self.num_sel.cpu().numpy(),
            "edge_head_base": self.edge_head_base.cpu().numpy(),
            "edges": self.edges.view(-1, 2)[:E].cpu().numpy(),
            "inv": self.inv.cpu().numpy().reshape(hkv, tq, topk),
            "splits": self.splits.view(-1, 4)[:S].cpu().numpy(),
            "n_units": U, "status": int(tot[3]),
        }


def allocate_index(tq, hkv, topk, batch, max_pages, block_size, page_size, device) -> Index:
    """Allocate (with torch) every array an index over these sizes needs."""
    s = sa_index_query_sizes(tq, hkv, topk, batch, max_pages, block_size, page_size)
    dev = torch.device(device)
    i32 = dict(dtype=torch.int32, device=dev)
    i64 = dict(dtype=torch.int64, device=dev)
    ws_words = (s["workspace_bytes"] + 255) // 8 + 32
    idx = Index(
        sel_slots=torch.empty(max(s["sel_slots"], 1), **i32),
        sel_offsets=torch.empty(max(s["sel_offsets"], 1), **i32),
        num_sel=torch.empty(max(s["num_sel"], 1), **i32),
        edge_head_base=torch.empty(max(s["edge_head_base"], 1), **i64),
        edges=torch.empty(max(s["edges"], 4), **i32),
        inv=torch.empty(max(s["inv"], 1), **i32),
        splits=torch.empty(max(s["splits"], 4), **i32),
        totals=torch.zeros(max(s["totals"], 4), **i64),
        workspace=torch.empty(ws_words, **i64),
        sizes=s,
        c=_native.SaIndex(),
    )
    c = idx.c
    c.sel_slots = idx.sel_slots.data_ptr()
    c.sel_offsets = idx.sel_offsets.data_ptr()
    c.num_sel = idx.num_sel.data_ptr()
    c.edge_head_base = idx.edge_head_base.data_ptr()
    c.edges = idx.edges.data_ptr()
    c.inv = idx.inv.data_ptr()
    c.splits = idx.splits.data_ptr()
    c.totals = idx.totals.data_ptr()
    base = idx.workspace.data_ptr()
    aligned = (base + 255) & ~255
    c.workspace = aligned
    c.workspace_bytes = idx.workspace.numel() * 8 - (aligned - base)
    return idx


def sa_build_index(selected, cu_seqlens_q_host, cu_seqlens_q, used_kv_lens, max_pages,
                   block_size, page_size, split_edges=0, index: Index | None = None,
                   stream=None) -> Index:
    """Step 1.  ``selected`` [tq, hkv, topk] int32 (device), ``cu_seqlens_q_host``
    the host copy (numpy / CPU tensor) of ``cu_seqlens_q`` [B+1] int64 (device),
    ``used_kv_lens`` [B] int32 (device) or None."""
    _require(selected, torch.int32, "selected")
    dev = selected.device
    tq, hkv, topk = (int(x) for x in selected.shape)
    cu_h = _host_i64(cu_seqlens_q_host)
    _require(cu_seqlens_q, torch.int64, "cu_seqlens_q", dev)
    batch = cu_h.size - 1
    if used_kv_lens is not None:
        _require(used_kv_lens, torch.int32, "used_kv_lens", dev)
    if index is None:
        with _allocating(stream):
            index = allocate_index(tq, hkv, topk, max(batch, 1), max_pages, block_size, page_size,
                                   dev)
    else:
        _check_index(index, tq, hkv, topk, batch, max_pages, block_size, page_size)
    _check(_on(
        dev, _native.load().sa_build_index, _ptr(selected), tq, hkv, topk, _host_ptr(cu_h),
        _ptr(cu_seqlens_q),
        batch, _ptr(used_kv_lens), max_pages, block_size, page_size, split_edges,
        ctypes.byref(index.c), _stream(stream, dev)), "sa_build_index")
    return index


def sa_build_index_no_alloc(selected, cu_seqlens_q_host, cu_seqlens_q, used_kv_lens, index: Index,
                            max_pages, block_size, page_size, split_edges=0, stream=None) -> Index:
    """Step 1 with the build's scratch taken from a fixed array inside the
    library instead of ``index.workspace``: for callers that cannot allocate
    device memory at call time.  ``index`` must already hold the output arrays
    (see :func:`allocate_index`).  Calls that overlap on the GPU share that
    array and race; the first call on a device must come before any stream
    capture on it."""
    _require(selected, torch.int32, "selected")
    dev = selected.device
    tq, hkv, topk = (int(x) for x in selected.shape)
    cu_h = _host_i64(cu_seqlens_q_host)
    _require(cu_seqlens_q, torch.int64, "cu_seqlens_q", dev)
    if used_kv_lens is not None:
        _require(used_kv_lens, torch.int32, "used_kv_lens", dev)
    _check_index(index, tq, hkv, topk, cu_h.size - 1, max_pages, block_size, page_size)
    _check(_on(
        dev, _native.load().sa_build_index_no_alloc, _ptr(selected), tq, hkv, topk, _host_ptr(cu_h),
        _ptr(cu_seqlens_q),
        cu_h.size - 1, _ptr(used_kv_lens), max_pages, block_size, page_size, split_edges,
        ctypes.byref(index.c), _stream(stream, dev)), "sa_build_index_no_alloc")
    return index


def _kv_dtype(k):
    if k.dtype == torch.float32:
        return DTYPE_F32
    if k.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"k_pages/v_pages must be float32 or bfloat16, got {k.dtype}")


_DTYPE_NAMES = {"f32": DTYPE_F32, "bf16": DTYPE_BF16, "e4m3": DTYPE_E4M3, "int8": DTYPE_INT8}


def _check_pool(k_pages, hkv, page_size, head_dim):
    """The scales are looked up by page id, so an 8-bit pool has to be what the
    call's sizes say: with other sizes an id inside the pool could lie past the
    scales."""
    if tuple(k_pages.shape[1:]) != (hkv, page_size, head_dim):
        raise ValueError(f"k_pages must be [num_pages, {hkv}, {page_size}, {head_dim}], got "
                         f"{tuple(k_pages.shape)}")


def _scaled(q, k_pages, v_pages, k_scales, v_scales, hkv, page_size, head_dim):
    """Checks of a call over an 8-bit cache: (q's type, the cache's, the scales'
    addresses); None for the other cache types, which take no scales."""
    dtype = k_pages.dtype
    if dtype is not torch.float8_e4m3fn and dtype is not torch.int8:
        if k_scales is not None or v_scales is not None:
            raise ValueError(f"a {k_pages.dtype} cache has no scales")
        return None
    code, act, index = _CACHE_DTYPES[dtype], _ACT_DTYPES.get(q.dtype), q.get_device()
    try:
        shape = k_pages.shape
        pool = shape[:2]
        if (act is not None and index >= 0 and q.is_contiguous() and
                shape[1:] == (hkv, page_size, head_dim) and v_pages.shape == shape and
                k_scales.shape == pool and v_scales.shape == pool and
                _alike(index, dtype, k_pages, v_pages) and
                _alike(index, torch.float32, k_scales, v_scales)):
            return act, code, k_scales.data_ptr(), v_scales.data_ptr()
    except AttributeError:
        pass
    _cache_dtype(k_pages, "k_pages")
    _check_pool(k_pages, hkv, page_size, head_dim)
    if act is None:
        raise TypeError(f"q must be float32 or bfloat16, got {q.dtype}")
    _require(q, q.dtype, "q")
    _require(k_pages, dtype, "k_pages", q.device)
    _require(v_pages, dtype, "v_pages", q.device)
    if v_pages.shape != k_pages.shape:
        raise ValueError("k_pages and v_pages must have one shape")
    ks, vs = _scales(k_scales, k_pages, "k_scales"), _scales(v_scales, v_pages, "v_scales")
    return act, code, _ptr(ks), _ptr(vs)


def _scaled_head(x, q, k_pages, v_pages, num_pages):
    """The first arguments of the entry points with scales."""
    act, code, ks, vs = x
    return (q.data_ptr(), act, k_pages.data_ptr(), v_pages.data_ptr(), ks, vs, num_pages, code)


def _check_call(dev, q, q_elems, tables, batch, max_pages, cu_seqlens_q, used_kv_lens,
                selected=None, shape=None):
    """That the tensors of a call are of its device, dense, and as large as its
    sizes say: the kernels take addresses and would read on past their ends."""
    i32 = [tables] if selected is None else [tables, selected]
    if used_kv_lens is not None:
        i32.append(used_kv_lens)
    try:
        if (_alike(dev.index, torch.int32, *i32) and _alike(dev.index, torch.int64, cu_seqlens_q) and
                q.numel() >= q_elems and tables.numel() >= batch * max_pages and
                cu_seqlens_q.numel() > batch and
                (used_kv_lens is None or used_kv_lens.numel() >= batch) and
                (selected is None or selected.shape == shape)):
            return
    except AttributeError:
        pass
    _require(tables, torch.int32, "block_tables", dev)
    _require(cu_seqlens_q, torch.int64, "cu_seqlens_q", dev)
    if used_kv_lens is not None:
        _require(used_kv_lens, torch.int32, "used_kv_lens", dev)
        if used_kv_lens.numel() < batch:
            raise ValueError(f"used_kv_lens needs {batch} values, has {used_kv_lens.numel()}")
    if selected is not None:
        _require(selected, torch.int32, "selected", dev)
        if tuple(selected.shape) != shape:
            raise ValueError(f"selected must be {shape}, got {tuple(selected.shape)}")
    for t, n, name in ((q, q_elems, "q"), (tables, batch * max_pages, "block_tables"),
                       (cu_seqlens_q, batch + 1, "cu_seqlens_q")):
        if t.numel() < n:
            raise ValueError(f"{name} needs {n} values, has {t.numel()}")


def _check_room(dev, *buffers):
    """That buffers handed in (tensor, dtype, elements, name) hold what the call
    writes to them."""
    index = dev.index
    for t, dtype, n, name in buffers:
        if t is not None and not (t.dtype is dtype and t.get_device() == index and
                                  t.is_contiguous() and t.numel() >= n):
            _require(t, dtype, name, dev)
            raise ValueError(f"{name} needs {n} values, has {t.numel()}")


def _check_partials(dev, partials, odt, rows, head_dim):
    if partials is not None:
        o, m, l = partials
        _check_room(dev, (o, odt, rows * head_dim, "o_partial"),
                    (m, torch.float32, rows, "m_partial"), (l, torch.float32, rows, "l_partial"))


def _check_index(index, tq, hkv, topk, batch, max_pages, block_size, page_size):
    """That an index handed in has room for one over these sizes (what the library
    refuses is left to it)."""
    if min(tq, hkv, topk, batch, block_size, page_size) <= 0 or block_size % page_size:
        return
    z, n = index.sizes, tq * hkv * topk
    nbs = batch * (max_pages // (block_size // page_size))
    if (z["edges"] < 2 * n or z["inv"] < n or z["splits"] < 4 * n or z["sel_slots"] < hkv * nbs or
            z["sel_offsets"] < hkv * (nbs + 1) or z["num_sel"] < hkv):
        raise ValueError("index was allocated for a smaller problem")


def sa_forward_kernel_name(tq, batch, hkv, hq, head_dim, block_size, page_size, kv_dtype="f32",
                           path=PATH_AUTO):
    """Name of the kernel sa_forward launches for this problem shape, or None
    where sa_forward would refuse it.  Host only."""
    dt = _DTYPE_NAMES[kv_dtype]
    name = _native.load().sa_forward_kernel_name(int(tq), int(batch), hq, hkv, head_dim,
                                                 block_size, page_size, dt, int(path))
    return None if name is None else name.decode()


def sa_attention_kernel_name(cu_seqlens_q_host, num_pages, hkv, hq, head_dim, block_size,
                             page_size, kv_dtype="f32", path=PATH_AUTO, causal=0):
    """The kernel sa_attention runs for steps 2 and 3 ("fused_dec_kernel" on
    the fused decode path), or None where it would refuse the call."""
    cu = _host_i64(cu_seqlens_q_host)
    dt = _DTYPE_NAMES[kv_dtype]
    name = _native.load().sa_attention_kernel_name(
        int(cu[-1]), len(cu) - 1, cu.ctypes.data, int(num_pages), hq, hkv, head_dim, block_size,
        page_size, dt, _causal(causal), int(path))
    return None if name is None else name.decode()


_PARTIAL_DTYPES = {"f32": (torch.float32, 0), "bf16": (torch.bfloat16, 1)}


def _partial_dtype(partial_dtype, o_partial):
    """(torch dtype, sa_dtype code) of the o partials: from ``o_partial`` when
    given (float32 or bfloat16), else ``partial_dtype`` ("f32" default, or
    "bf16": 16-bit o partials, an opt-in the pages do not have)."""
    if o_partial is not None:
        if partial_dtype is None and o_partial.dtype in _ACT_DTYPES:
            return o_partial.dtype, _ACT_DTYPES[o_partial.dtype]
        for name, (dt, code) in _PARTIAL_DTYPES.items():
            if o_partial.dtype == dt:
                if partial_dtype not in (None, name):
                    raise ValueError(f"o_partial is {o_partial.dtype}, partial_dtype {partial_dtype}")
                return dt, code
        raise TypeError(f"o_partial must be float32 or bfloat16, got {o_partial.dtype}")
    if partial_dtype is None:
        partial_dtype = "f32"
    if partial_dtype not in _PARTIAL_DTYPES:
        raise ValueError(f"partial_dtype must be 'f32' or 'bf16', got {partial_dtype!r}")
    return _PARTIAL_DTYPES[partial_dtype]


def partial_rows(index: Index, hq: int) -> int:
    """Row capacity of the partial buffers: tq * hkv * topk * qhead."""
    c = index.c
    return max(c.tq * c.hkv * c.topk * (hq // c.hkv), 1)


def sa_forward(q, k_pages, v_pages, index: Index, block_tables, cu_seqlens_q, used_kv_lens, hq,
               hkv, head_dim, block_size, page_size, softmax_scale, causal, o_partial=None,
               m_partial=None, l_partial=None, path=PATH_AUTO, stream=None, partial_dtype=None,
               q_scratch=None, k_scales=None, v_scales=None):
    """Step 2.  Returns (o_partial, m_partial, l_partial); the first
    totals[0] * qhead rows are valid.  ``partial_dtype="bf16"`` (or a
    bfloat16 ``o_partial``) stores o in bf16; ``q_scratch`` (a tensor of at
    least tq * hq * head_dim * 2 bytes, e.g. the combine's ``out``) lets the
    tensor-core kernel gather Q from a bf16 copy (both: sa_forward_ex).  An
    8-bit cache needs ``k_scales`` and ``v_scales`` [num_pages, hkv]; ``q`` may
    then be bfloat16 (sa_forward_scaled)."""
    x = _scaled(q, k_pages, v_pages, k_scales, v_scales, hkv, page_size, head_dim)
    if x is None:
        _require(q, torch.float32, "q")
        kvd = _kv_dtype(k_pages)
    dev = q.device
    _require(k_pages, k_pages.dtype, "k_pages", dev)
    _require(v_pages, k_pages.dtype, "v_pages", dev)
    c = index.c
    _check_call(dev, q, c.tq * hq * head_dim, block_tables, c.batch, c.max_pages, cu_seqlens_q,
                used_kv_lens)
    page_elems = hkv * page_size * head_dim
    num_pages = k_pages.numel() // page_elems if page_elems > 0 else 0
    rows = partial_rows(index, hq) if hkv > 0 and hq % max(hkv, 1) == 0 else 1
    odt, ocode = _partial_dtype(partial_dtype, o_partial)
    _check_partials(dev, (o_partial, m_partial, l_partial), odt, rows, head_dim)
    with _allocating(stream):
        if o_partial is None:
            o_partial = torch.empty((rows, head_dim), dtype=odt, device=dev)
        if m_partial is None:
            m_partial = torch.empty(rows, dtype=torch.float32, device=dev)
        if l_partial is None:
            l_partial = torch.empty(rows, dtype=torch.float32, device=dev)
    L = _native.load()
    mid = (ctypes.byref(index.c), _ptr(block_tables), _ptr(cu_seqlens_q), _ptr(used_kv_lens), hq,
           hkv, head_dim, block_size, page_size, softmax_scale, _causal(causal))
    tail = (_ptr(o_partial), _ptr(m_partial), _ptr(l_partial), path, _stream(stream, dev))
    if x is not None:
        if q_scratch is not None:
            raise ValueError("q_scratch does not apply to an 8-bit cache")
        _check(_on(dev, L.sa_forward_scaled, *_scaled_head(x, q, k_pages, v_pages, num_pages),
                   *mid, ocode, *tail), "sa_forward_scaled")
        return o_partial, m_partial, l_partial
    head = (_ptr(q), _ptr(k_pages), _ptr(v_pages), num_pages, kvd, *mid)
    if q_scratch is not None:
        need = index.c.tq * hq * head_dim * 2
        if q_scratch.device != dev or q_scratch.numel() * q_scratch.element_size() < need:
            raise ValueError(f"q_scratch needs {need} bytes on {dev}")
    if ocode or q_scratch is not None:
        _check(_on(dev, L.sa_forward_ex, *head, ocode, *tail, _ptr(q_scratch)), "sa_forward_ex")
    else:
        _check(_on(dev, L.sa_forward, *head, *tail), "sa_forward")
    return o_partial, m_partial, l_partial


def sa_combine(index: Index, o_partial, m_partial, l_partial, hq, head_dim, out=None, lse=None,
               with_lse=True, stream=None):
    """Step 3.  Returns (out [tq, hq, d], lse [tq, hq] or None).  A bfloat16
    ``o_partial`` is read as 16-bit o partials (sa_combine_ex)."""
    dev = o_partial.device
    tq = index.c.tq
    _, ocode = _partial_dtype(None, o_partial)
    _check_room(dev, (out, torch.float32, tq * hq * head_dim, "out"),
                (lse, torch.float32, tq * hq, "lse"))
    with _allocating(stream):
        if out is None:
            out = torch.empty((tq, hq, head_dim), dtype=torch.float32, device=dev)
        if lse is None and with_lse:
            lse = torch.empty((tq, hq), dtype=torch.float32, device=dev)
    L = _native.load()
    tail = (_ptr(o_partial), _ptr(m_partial), _ptr(l_partial), hq, head_dim, _ptr(out), _ptr(lse),
            _stream(stream, dev))
    if ocode:
        _check(_on(dev, L.sa_combine_ex, ctypes.byref(index.c), ocode, *tail), "sa_combine_ex")
    else:
        _check(_on(dev, L.sa_combine, ctypes.byref(index.c), *tail), "sa_combine")
    return out, lse


def sa_forward_combine(q, k_pages, v_pages, index: Index, selected, cu_seqlens_q_host,
                       cu_seqlens_q, used_kv_lens, block_tables, hq, head_dim, block_size,
                       page_size, softmax_scale, causal, split_edges=0, partials=None, out=None,
                       lse=None, with_lse=True, path=PATH_AUTO, stream=None, partial_dtype=None,
                       k_scales=None, v_scales=None):
    """Steps 2 and 3 on a built index (the fused decode kernel where it
    applies).  Returns (out, lse, (o, m, l)).  ``partial_dtype="bf16"`` (or a
    bfloat16 o in ``partials``): 16-bit o partials.  ``k_scales``, ``v_scales``:
    see :func:`sa_attention`."""
    x = _scaled(q, k_pages, v_pages, k_scales, v_scales, index.c.hkv, page_size, head_dim)
    if x is None:
        _require(q, torch.float32, "q")
        kvd = _kv_dtype(k_pages)
    dev = q.device
    c = index.c
    hkv = c.hkv
    if x is None:
        _require(k_pages, k_pages.dtype, "k_pages", dev)
        _require(v_pages, k_pages.dtype, "v_pages", dev)
    cu_h = _host_i64(cu_seqlens_q_host)
    _check_call(dev, q, c.tq * hq * head_dim, block_tables, c.batch, c.max_pages, cu_seqlens_q,
                used_kv_lens, selected, (c.tq, c.hkv, c.topk))
    rows = partial_rows(index, hq) if hkv > 0 and hq % max(hkv, 1) == 0 else 1
    odt, ocode = _partial_dtype(partial_dtype, None if partials is None else partials[0])
    _check_partials(dev, partials, odt, rows, head_dim)
    _check_room(dev, (out, q.dtype, c.tq * hq * head_dim, "out"),
                (lse, torch.float32, c.tq * hq, "lse"))
    with _allocating(stream):
        if partials is None:
            partials = (torch.empty((rows, head_dim), dtype=odt, device=dev),
                        torch.empty(rows, dtype=torch.float32, device=dev),
                        torch.empty(rows, dtype=torch.float32, device=dev))
        if out is None:
            out = torch.empty((c.tq, hq, head_dim), dtype=q.dtype, device=dev)
        if lse is None and with_lse:
            lse = torch.empty((c.tq, hq), dtype=torch.float32, device=dev)
    page_elems = hkv * page_size * head_dim
    num_pages = k_pages.numel() // page_elems if page_elems > 0 else 0
    o, m, l = partials
    L = _native.load()
    mid = (ctypes.byref(c), _ptr(selected), _host_ptr(cu_h),
           _ptr(cu_seqlens_q), _ptr(used_kv_lens), _ptr(block_tables), hq, head_dim, block_size,
           page_size, softmax_scale, _causal(causal), split_edges)
    tail = (_ptr(o), _ptr(m), _ptr(l), _ptr(out), _ptr(lse), path, _stream(stream, dev))
    if x is not None:
        _check(_on(dev, L.sa_forward_combine_scaled, *_scaled_head(x, q, k_pages, v_pages, num_pages),
                   *mid, ocode, *tail), "sa_forward_combine_scaled")
        return out, lse, partials
    head = (_ptr(q), _ptr(k_pages), _ptr(v_pages), num_pages, kvd, *mid)
    if ocode:
        _check(_on(dev, L.sa_forward_combine_ex, *head, ocode, *tail), "sa_forward_combine_ex")
    else:
        _check(_on(dev, L.sa_forward_combine, *head, *tail), "sa_forward_combine")
    return out, lse, partials


def sa_attention(q, k_pages, v_pages, selected, cu_seqlens_q_host, cu_seqlens_q, used_kv_lens,
                 block_tables, hq, hkv, head_dim, block_size, page_size, softmax_scale, causal,
                 split_edges=0, index: Index | None = None, partials=None, out=None, lse=None,
                 with_lse=True, path=PATH_AUTO, stream=None, partial_dtype=None, k_scales=None,
                 v_scales=None):
    """Steps 1-3 in one call.  Returns (out, lse, index, (o, m, l)).  Pass
    ``index`` / ``partials`` / ``out`` back in to reuse their memory.
    ``partial_dtype="bf16"`` (or a bfloat16 o in ``partials``): 16-bit o
    partials (sa_attention_ex).  A float8_e4m3fn or int8 cache needs
    ``k_scales`` and ``v_scales`` [num_pages, hkv] (see :func:`sa_store_kv`);
    ``q`` may then be bfloat16, and ``out`` has its type (sa_attention_scaled)."""
    x = _scaled(q, k_pages, v_pages, k_scales, v_scales, hkv, page_size, head_dim)
    if x is None:
        _require(q, torch.float32, "q")
        kvd = _kv_dtype(k_pages)
    dev = q.device
    if x is None:
        _require(k_pages, k_pages.dtype, "k_pages", dev)
        _require(v_pages, k_pages.dtype, "v_pages", dev)
    tq, hkv_s, topk = selected.shape
    cu_h = _host_i64(cu_seqlens_q_host)
    batch = cu_h.size - 1
    max_pages = block_tables.shape[1]
    _check_call(dev, q, tq * hq * head_dim, block_tables, batch, max_pages, cu_seqlens_q,
                used_kv_lens, selected, (tq, hkv_s if hkv <= 0 else hkv, topk))
    rows = max(tq * hkv_s * topk * (hq // max(hkv_s, 1)), 1)
    odt, ocode = _partial_dtype(partial_dtype, None if partials is None else partials[0])
    _check_partials(dev, partials, odt, rows, head_dim)
    _check_room(dev, (out, q.dtype, tq * hq * head_dim, "out"), (lse, torch.float32, tq * hq, "lse"))
    if index is not None:
        _check_index(index, tq, hkv, topk, batch, max_pages, block_size, page_size)
    with _allocating(stream):
        if index is None:
            index = allocate_index(tq, hkv_s, topk, max(batch, 1), max_pages, block_size,
                                   page_size, dev)
        if partials is None:
            partials = (torch.empty((rows, head_dim), dtype=odt, device=dev),
                        torch.empty(rows, dtype=torch.float32, device=dev),
                        torch.empty(rows, dtype=torch.float32, device=dev))
        if out is None:
            out = torch.empty((tq, hq, head_dim), dtype=q.dtype, device=dev)
        if lse is None and with_lse:
            lse = torch.empty((tq, hq), dtype=torch.float32, device=dev)
    page_elems = hkv * page_size * head_dim
    num_pages = k_pages.numel() // page_elems if page_elems > 0 else 0
    o, m, l = partials
    L = _native.load()
    mid = (_ptr(selected), tq, topk, _host_ptr(cu_h), _ptr(cu_seqlens_q),
           batch, _ptr(used_kv_lens), _ptr(block_tables), max_pages, hq, hkv, head_dim, block_size,
           page_size, softmax_scale, _causal(causal), split_edges, ctypes.byref(index.c))
    tail = (_ptr(o), _ptr(m), _ptr(l), _ptr(out), _ptr(lse), path, _stream(stream, dev))
    if x is not None:
        _check(_on(dev, L.sa_attention_scaled, *_scaled_head(x, q, k_pages, v_pages, num_pages),
                   *mid, ocode, *tail), "sa_attention_scaled")
        return out, lse, index, partials
    head = (_ptr(q), _ptr(k_pages), _ptr(v_pages), num_pages, kvd, *mid)
    if ocode:
        _check(_on(dev, L.sa_attention_ex, *head, ocode, *tail), "sa_attention_ex")
    else:
        _check(_on(dev, L.sa_attention, *head, *tail), "sa_attention")
    return out, lse, index, partials


class AttentionGraph:
    """Steps 1-3 (sa_attention) captured once into a CUDA graph on fixed
    buffers and replayed: for small decode batches, where the launches of
    the index, forward and combine kernels cost as much as their work.

    Every argument is bound at capture: the device tensors by address (their
    contents may change between replays: new queries, selections, block
    tables, lengths) and the host-side facts the library decides on at call
    time (cu_seqlens_q_host, head counts, sizes, path), which must then stay
    what they were.  ``replay()`` enqueues the graph on the current stream
    and returns (out, lse); status checks go through ``sa_get_status(self.index)``.
    """

    def __init__(self, q, k_pages, v_pages, selected, cu_seqlens_q_host, cu_seqlens_q,
                 used_kv_lens, block_tables, hq, hkv, head_dim, block_size, page_size,
                 softmax_scale, causal, split_edges=0, path=PATH_AUTO, partial_dtype=None,
                 k_scales=None, v_scales=None):
        args = (q, k_pages, v_pages, selected, cu_seqlens_q_host, cu_seqlens_q, used_kv_lens,
                block_tables, hq, hkv, head_dim, block_size, page_size, softmax_scale, causal)
        kw = dict(split_edges=split_edges, path=path, k_scales=k_scales, v_scales=v_scales)
        # one eager call first: buffers, library load and kernel attributes
        self.out, self.lse, self.index, self.partials = sa_attention(
            *args, partial_dtype=partial_dtype, **kw)
        torch.cuda.synchronize(q.device)
        status = sa_get_status(self.index)
        if status != 0:
            raise SAError(status, "AttentionGraph (eager call)")
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.device(q.device), torch.cuda.graph(self.graph):
            sa_attention(*args, index=self.index, partials=self.partials, out=self.out,
                         lse=self.lse, **kw)

    def replay(self):
        self.graph.replay()
        return self.out, self.lse


def _on(dev, fn, *args) -> int:
    """fn(*args) with the device of the call's tensors as the current one."""
    index = dev.index
    if index is None or index == _current_device():
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


# (the tensors at hand are CUDA tensors, so CUDA is initialised)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


_CACHE_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16,
                 torch.float8_e4m3fn: DTYPE_E4M3, torch.int8: DTYPE_INT8}
_ACT_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}


def _cache_dtype(pages, name):
    if not isinstance(pages, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if pages.dtype not in _CACHE_DTYPES:
        raise TypeError(f"{name} must be float32, bfloat16, float8_e4m3fn or int8, got {pages.dtype}")
    if pages.dim() != 4:
        raise ValueError(f"{name} must be [num_pages, hkv, page_size, head_dim]")
    return _CACHE_DTYPES[pages.dtype]


def _scales(scales, pages, name):
    """The scales [num_pages, hkv] of an 8-bit cache (None for the others)."""
    if pages.dtype is not torch.float8_e4m3fn and pages.dtype is not torch.int8:
        if scales is not None:
            raise ValueError(f"{name}: a {pages.dtype} cache has no scales")
        return None
    if scales is None:
        raise ValueError(f"{name} [num_pages, hkv] are needed with a {pages.dtype} cache")
    try:
        if (scales.shape == tuple(pages.shape)[:2] and
                _alike(pages.get_device(), torch.float32, scales)):
            return scales
    except AttributeError:
        pass
    _require(scales, torch.float32, name, pages.device)
    if scales.shape != pages.shape[:2]:
        raise ValueError(f"{name} must be {tuple(pages.shape[:2])}, got {tuple(scales.shape)}")
    return scales


def _batch_args(cu_seqlens_q_host, cu_seqlens_q, used_kv_lens, tables, dev, name):
    """Host prefix lengths after the checks that sequences and tables agree."""
    cu_h = _host_i64(cu_seqlens_q_host)
    batch = cu_h.size - 1
    try:
        if (_alike(dev.index, torch.int32, used_kv_lens, *tables) and
                _alike(dev.index, torch.int64, cu_seqlens_q) and
                cu_seqlens_q.numel() == batch + 1 and used_kv_lens.numel() == batch and
                all([t.dim() == 2 and t.shape[0] == batch for t in tables])):
            return cu_h, batch
    except AttributeError:
        pass
    _require(cu_seqlens_q, torch.int64, "cu_seqlens_q", dev)
    _require(used_kv_lens, torch.int32, "used_kv_lens", dev)
    if cu_seqlens_q.numel() != cu_h.size or used_kv_lens.numel() != batch:
        raise ValueError("cu_seqlens_q [batch + 1] and used_kv_lens [batch] disagree with "
                         "cu_seqlens_q_host")
    for t, n in zip(tables, name):
        _require(t, torch.int32, n, dev)
        if len(t.shape) != 2 or t.shape[0] != batch:
            raise ValueError(f"{n} must have a row for each of the {batch} sequences")
    return cu_h, batch


def _status_word(status, dev):
    if status is not None:
        _require(status, torch.int64, "status", dev)
    return _ptr(status)


def sa_store_kv(k, v, k_pages, v_pages, block_tables, cu_seqlens_q_host, cu_seqlens_q,
                used_kv_lens, k_scales=None, v_scales=None, status=None, stream=None) -> None:
    """Store new tokens' K/V rows in the paged cache.  ``k``, ``v`` [tq, hkv,
    d] float32 or bfloat16, channels contiguous (slices of a fused projection
    will do); ``used_kv_lens`` the lengths with the new tokens, which take each
    sequence's last positions.  A float8_e4m3fn or int8 cache has ``k_scales``
    and ``v_scales`` [num_pages, hkv], renewed with the pages (powers of two;
    see sa.h).  ``status``: a zeroed int64 CUDA tensor that keeps the first
    device-detected error."""
    if not _store_args_usual(k, v, k_pages, v_pages, k_scales, v_scales):
        _check_store_args(k, v, k_pages, v_pages, k_scales, v_scales)
    dev = k_pages.device
    num_pages, hkv, page_size, d = k_pages.shape
    cu_h, batch = _batch_args(cu_seqlens_q_host, cu_seqlens_q, used_kv_lens, (block_tables,), dev,
                              ("block_tables",))
    ks0, ks1, _ = k.stride()
    vs0, vs1, _ = v.stride()
    _check(_on(dev, _native.load().sa_store_kv, k.data_ptr(), v.data_ptr(), _ACT_DTYPES[k.dtype],
               ks0, ks1, vs0, vs1, k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_scales),
               _ptr(v_scales), num_pages, _CACHE_DTYPES[k_pages.dtype], block_tables.data_ptr(),
               block_tables.shape[1], _host_ptr(cu_h), cu_seqlens_q.data_ptr(), batch, k.shape[0],
               used_kv_lens.data_ptr(), hkv, d, page_size, _status_word(status, dev),
               _stream(stream, dev)), "sa_store_kv")


def _store_args_usual(k, v, k_pages, v_pages, k_scales, v_scales) -> bool:
    try:
        dtype, act, shape, new = k_pages.dtype, k.dtype, k_pages.shape, k.shape
        index = k_pages.get_device()
        num_pages, hkv, _, d = shape
        tq, heads, channels = new
        if not (index >= 0 and act in _ACT_DTYPES and v.dtype is act and v.shape == new and
                heads == hkv and channels == d and k.get_device() == index and
                v.get_device() == index and k.stride(2) == 1 and v.stride(2) == 1 and
                v_pages.shape == shape and _alike(index, dtype, k_pages, v_pages)):
            return False
        if dtype is torch.float8_e4m3fn or dtype is torch.int8:
            return (k_scales.shape == (num_pages, hkv) and v_scales.shape == (num_pages, hkv) and
                    _alike(index, torch.float32, k_scales, v_scales))
        return dtype in _CACHE_DTYPES and k_scales is None and v_scales is None
    except (AttributeError, TypeError, ValueError):
        return False


def _check_store_args(k, v, k_pages, v_pages, k_scales, v_scales) -> None:
    _cache_dtype(k_pages, "k_pages")
    dev = k_pages.device
    _require(k_pages, k_pages.dtype, "k_pages", dev)
    _require(v_pages, k_pages.dtype, "v_pages", dev)
    if v_pages.shape != k_pages.shape:
        raise ValueError("k_pages and v_pages must have one shape")
    _, hkv, _, d = k_pages.shape
    for t, name in ((k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype not in _ACT_DTYPES or t.dtype != k.dtype:
            raise TypeError(f"{name} must be float32 or bfloat16 (both alike), got {t.dtype}")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
        if t.shape != (k.shape[0], hkv, d):
            raise ValueError(f"{name} must be [tq, {hkv}, {d}], got {tuple(t.shape)}")
        if t.stride(2) != 1 and t.numel():
            raise ValueError(f"{name}: channels must be contiguous")
    _scales(k_scales, k_pages, "k_scales")
    _scales(v_scales, v_pages, "v_scales")


def _check_bounds(bounds, hkv, d, dev):
    _require(bounds, torch.bfloat16, "bounds", dev)
    if len(bounds.shape) != 4 or bounds.shape[1:] != (hkv, 2, d):
        raise ValueError(f"bounds must be [rows, {hkv}, 2, {d}], got {tuple(bounds.shape)}")


def sa_block_bounds(k_pages, block_tables, cu_seqlens_q_host, cu_seqlens_q, used_kv_lens, bounds,
                    bound_tables, block_size, k_scales=None, status=None, stream=None):
    """Renew the bounds of every block that holds a new token: ``bounds``
    [rows, hkv, 2, d] bfloat16 (smallest, largest key per channel), row
    ``bound_tables[b, j]`` (int32 [batch, msb], -1 = skip) for block j of
    sequence b.  Returns ``bounds``."""
    code = _cache_dtype(k_pages, "k_pages")
    dev = k_pages.device
    _require(k_pages, k_pages.dtype, "k_pages")
    num_pages, hkv, page_size, d = k_pages.shape
    ks = _scales(k_scales, k_pages, "k_scales")
    _check_bounds(bounds, hkv, d, dev)
    cu_h, batch = _batch_args(cu_seqlens_q_host, cu_seqlens_q, used_kv_lens,
                              (block_tables, bound_tables), dev, ("block_tables", "bound_tables"))
    _check(_on(dev, _native.load().sa_block_bounds, k_pages.data_ptr(), _ptr(ks), num_pages, code,
               block_tables.data_ptr(), block_tables.shape[1], _host_ptr(cu_h),
               cu_seqlens_q.data_ptr(), batch, int(cu_h[-1]), used_kv_lens.data_ptr(), hkv, d,
               block_size, page_size, bound_tables.data_ptr(), bound_tables.shape[1],
               bounds.shape[0], bounds.data_ptr(), _status_word(status, dev),
               _stream(stream, dev)), "sa_block_bounds")
    return bounds


def allocate_select_workspace(tq, batch, hkv, head_dim, msb, device) -> torch.Tensor:
    """Scratch for :func:`sa_select_blocks` over these sizes (msb: columns of
    the bound tables), to be kept from call to call."""
    n = ctypes.c_size_t(0)
    _check(_native.load().sa_select_workspace_size(tq, batch, hkv, head_dim, msb, ctypes.byref(n)),
           "sa_select_workspace_size")
    return torch.empty(n.value + 256, dtype=torch.uint8, device=device)


def sa_select_blocks(q, bounds, bound_tables, cu_seqlens_q_host, cu_seqlens_q, used_kv_lens,
                     block_size, topk, causal, sink_blocks=0, local_blocks=0, selected=None,
                     workspace=None, status=None, stream=None):
    """Each (query, kv head)'s ``topk`` blocks with the highest upper bound of
    q.k summed over the GQA lanes: ``selected`` [tq, hkv, topk] int32,
    ascending, -1 behind the last.  ``q`` [tq, hq, d] float32 or bfloat16;
    ``bounds`` and ``bound_tables`` as in :func:`sa_block_bounds`;
    ``sink_blocks`` first and ``local_blocks`` last blocks always come in."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if q.dtype not in _ACT_DTYPES:
        raise TypeError(f"q must be float32 or bfloat16, got {q.dtype}")
    _require(q, q.dtype, "q")
    dev = q.device
    if q.dim() != 3 or not isinstance(bounds, torch.Tensor) or bounds.dim() != 4:
        raise ValueError("q must be [tq, hq, d], bounds [rows, hkv, 2, d]")
    tq, hq, d = q.shape
    hkv = bounds.shape[1]
    _check_bounds(bounds, hkv, d, dev)
    cu_h, batch = _batch_args(cu_seqlens_q_host, cu_seqlens_q, used_kv_lens, (bound_tables,), dev,
                              ("bound_tables",))
    msb = bound_tables.shape[1]
    if selected is None:
        with _allocating(stream):
            selected = torch.empty((tq, hkv, int(topk)), dtype=torch.int32, device=dev)
    else:
        _require(selected, torch.int32, "selected", dev)
        if selected.shape != (tq, hkv, topk):
            raise ValueError(f"selected must be {(tq, hkv, int(topk))}, got {tuple(selected.shape)}")
    if workspace is None:
        with _allocating(stream):
            workspace = allocate_select_workspace(tq, batch, hkv, d, msb, dev)
    else:
        _require(workspace, torch.uint8, "workspace", dev)
    base = workspace.data_ptr()
    aligned = (base + 255) & ~255
    _check(_on(dev, _native.load().sa_select_blocks, q.data_ptr(), _ACT_DTYPES[q.dtype], tq, hq,
               hkv, d, bounds.data_ptr(), bounds.shape[0], bound_tables.data_ptr(), msb,
               _host_ptr(cu_h), cu_seqlens_q.data_ptr(), batch, used_kv_lens.data_ptr(), block_size,
               topk, _causal(causal), sink_blocks, local_blocks, selected.data_ptr(), aligned,
               max(workspace.numel() - (aligned - base), 0), _status_word(status, dev),
               _stream(stream, dev)), "sa_select_blocks")
    return selected


def sa_norm_rope(q, k, q_weight, k_weight, inv_freq, positions=None, cu_seqlens_q_host=None,
                 cu_seqlens_q=None, used_kv_lens=None, eps=1e-6, freq_axes=None, interleaved=False,
                 q_out=None, k_out=None, out_dtype=None, status=None, stream=None):
    """RMS norm of each head of new tokens' ``q`` [tq, hq, d] and ``k`` [tq, hkv, d]
    (float32 or bfloat16, channels contiguous; either may be None) with the
    weights ``q_weight`` / ``k_weight`` [d] (None: no norm), then rotation of the
    first ``2 * inv_freq.numel()`` channels (``inv_freq`` float32, None: none) by
    the token's position: pairs (i, i + half), or (2 i, 2 i + 1) where
    ``interleaved``.  ``positions`` int32 [tq] or [axes, tq], with ``freq_axes``
    int32 (per pair, its axis) in the latter case; without positions each
    sequence's last positions, as :func:`sa_store_kv` takes them from the same
    ``cu_seqlens_q_host``, ``cu_seqlens_q`` and ``used_kv_lens``.  Returns
    (q_out, k_out), of ``out_dtype`` (default: the input's type); an output handed
    in may be its input."""
    x = _rope_usual(q, k, q_weight, k_weight, inv_freq, q_out, k_out, out_dtype)
    if x is None:
        q_out, k_out, x = _check_rope(q, k, q_weight, k_weight, inv_freq, q_out, k_out, out_dtype,
                                      stream)
    dev, tq, hq, hkv, d, src, wt, out, strides = x
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    cu_h = used = None
    axes = batch = 0
    if positions is not None:
        _require(positions, torch.int32, "positions", dev)
        if positions.dim() not in (1, 2) or positions.shape[-1] != tq:
            raise ValueError(f"positions must be [{tq}] or [axes, {tq}]")
        axes = 1 if positions.dim() == 1 else positions.shape[0]
        if axes > 1 and rot and freq_axes is None:
            raise ValueError(f"freq_axes must say which of the {axes} axes turns each pair")
        positions = positions.data_ptr()
    elif rot:
        if cu_seqlens_q_host is None or cu_seqlens_q is None or used_kv_lens is None:
            raise ValueError("positions, or cu_seqlens_q_host, cu_seqlens_q and used_kv_lens, are needed")
        cu, batch = _batch_args(cu_seqlens_q_host, cu_seqlens_q, used_kv_lens, (), dev, ())
        cu_h, cu_d, used = _host_ptr(cu), cu_seqlens_q.data_ptr(), used_kv_lens.data_ptr()
    if cu_h is None:
        cu_d = None
    if freq_axes is not None:
        _require(freq_axes, torch.int32, "freq_axes", dev)
        if freq_axes.numel() * 2 != rot:
            raise ValueError(f"freq_axes must have {rot // 2} values")
    q_st, k_st, qo_st, ko_st = strides
    _check(_on(dev, _native.load().sa_norm_rope, _ptr(q), _ptr(k), _ACT_DTYPES[src], q_st[0],
               q_st[1], k_st[0], k_st[1], None if q is None else _ptr(q_weight),
               None if k is None else _ptr(k_weight), _ACT_DTYPES[wt], eps, _ptr(inv_freq), rot,
               _ptr(freq_axes), 1 if interleaved else 0, positions, axes, tq, cu_h, cu_d, batch,
               used, tq, hq, hkv, d, _ptr(q_out), _ptr(k_out), _ACT_DTYPES[out], qo_st[0], qo_st[1],
               ko_st[0], ko_st[1], _status_word(status, dev), _stream(stream, dev)), "sa_norm_rope")
    return q_out, k_out


def _rope_usual(q, k, q_weight, k_weight, inv_freq, q_out, k_out, out_dtype):
    """What a call needs to know of its tensors where all are given and as they should
    be; None where not (:func:`_check_rope` then says what is wrong, or makes outputs)."""
    try:
        src, out, shape, kshape = q.dtype, q_out.dtype, q.shape, k.shape
        index, wt = q.get_device(), q_weight.dtype
        tq, hq, d = shape
        tk, hkv, dk = kshape
        strides = q.stride(), k.stride(), q_out.stride(), k_out.stride()
        if (index >= 0 and src in _ACT_DTYPES and out in _ACT_DTYPES and wt in _ACT_DTYPES and
                k.dtype is src and k_out.dtype is out and (out_dtype is None or out_dtype is out) and
                tk == tq and dk == d and q_out.shape == shape and k_out.shape == kshape and
                strides[0][2] == 1 and strides[1][2] == 1 and strides[2][2] == 1 and
                strides[3][2] == 1 and k.get_device() == index and q_out.get_device() == index and
                k_out.get_device() == index and
                (q.data_ptr() != q_out.data_ptr() or (src is out and strides[0] == strides[2])) and
                (k.data_ptr() != k_out.data_ptr() or (src is out and strides[1] == strides[3])) and
                _alike(index, wt, q_weight, k_weight) and q_weight.numel() == d and
                k_weight.numel() == d and _alike(index, torch.float32, inv_freq)):
            return q.device, tq, hq, hkv, d, src, wt, out, strides
    except (AttributeError, ValueError):
        pass
    return None


def _check_rope(q, k, q_weight, k_weight, inv_freq, q_out, k_out, out_dtype, stream):
    given = q if q is not None else k
    src = _heads(given, "k" if q is None else "q")
    dev, (tq, _, d) = given.device, given.shape
    for t, name in ((q, "q"), (k, "k")):
        if t is not None and (_heads(t, name) != src or t.device != dev or t.shape[0] != tq or
                              t.shape[2] != d):
            raise ValueError("q and k must have one type, device, number of tokens and of channels")
    made = []
    for t, out, name in ((q, q_out, "q_out"), (k, k_out, "k_out")):
        if t is None:
            if out is not None:
                raise ValueError(f"{name} without its input")
        elif out is None:
            if (out_dtype or t.dtype) not in _ACT_DTYPES:
                raise TypeError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
            with _allocating(stream):
                out = torch.empty(t.shape, dtype=out_dtype or t.dtype, device=dev)
        else:
            _heads(out, name)
            if out.shape != t.shape or out.device != dev:
                raise ValueError(f"{name} must be {tuple(t.shape)} on {dev}")
            if out_dtype is not None and out.dtype != out_dtype:
                raise TypeError(f"{name} must be {out_dtype}, got {out.dtype}")
            if (t.numel() and out.data_ptr() == t.data_ptr() and
                    (out.dtype != t.dtype or out.stride() != t.stride())):
                raise ValueError(f"{name} in its input's place must have its type and strides")
        made.append(out)
    q_out, k_out = made
    if q_out is not None and k_out is not None and q_out.dtype != k_out.dtype:
        raise TypeError("q_out and k_out must have one type")
    wt = None
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            if not isinstance(w, torch.Tensor) or w.dtype not in _ACT_DTYPES:
                raise TypeError(f"{name} must be a float32 or bfloat16 tensor")
            wt = wt or w.dtype
            _require(w, wt, name, dev)
            if w.numel() != d:
                raise ValueError(f"{name} must have {d} values")
    if inv_freq is not None:
        _require(inv_freq, torch.float32, "inv_freq", dev)
    strides = [(0, 0, 1) if t is None else t.stride() for t in (q, k, q_out, k_out)]
    out = q_out if q_out is not None else k_out
    return q_out, k_out, (dev, tq, 0 if q is None else q.shape[1], 0 if k is None else k.shape[1], d,
                          src, wt or torch.float32, out.dtype, strides)


def _heads(t, name):
    """The type of a [tokens, heads, channels] activation, after its checks."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _ACT_DTYPES:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, channels]")
    if t.numel() and t.stride(2) != 1 and t.shape[2] != 1:
        raise ValueError(f"{name}: channels must be contiguous")
    return t.dtype


def _pool(k_pages, v_pages, k_scales, v_scales):
    """Checks of a cache of any type: its type's code."""
    code = _CACHE_DTYPES.get(getattr(k_pages, "dtype", None))
    try:
        shape, index = k_pages.shape, k_pages.get_device()
        if code is not None and index >= 0 and len(shape) == 4 and v_pages.shape == shape and (
                _alike(index, k_pages.dtype, k_pages, v_pages)):
            if code != DTYPE_E4M3 and code != DTYPE_INT8:
                if k_scales is None and v_scales is None:
                    return code
            elif (k_scales.shape == shape[:2] and v_scales.shape == shape[:2] and
                  _alike(index, torch.float32, k_scales, v_scales)):
                return code
    except AttributeError:
        pass
    code = _cache_dtype(k_pages, "k_pages")
    _require(k_pages, k_pages.dtype, "k_pages")
    _require(v_pages, k_pages.dtype, "v_pages", k_pages.device)
    if v_pages.shape != k_pages.shape:
        raise ValueError("k_pages and v_pages must have one shape")
    _scales(k_scales, k_pages, "k_scales")
    _scales(v_scales, v_pages, "v_scales")
    return code


def sa_load_kv(k_pages, v_pages, block_tables, cu_seqlens_host, cu_seqlens, used_kv_lens, k=None,
               v=None, dtype=None, k_scales=None, v_scales=None, status=None, stream=None):
    """Read rows of the cache back: with the lengths of a :func:`sa_store_kv` call the
    rows that it stored, each sequence's last ``cu_seqlens`` positions below
    ``used_kv_lens`` (the whole sequence where both agree).  Returns (k, v) [rows,
    hkv, d] of ``dtype`` (float32 or bfloat16; default: that of ``k``, else the
    cache's, bfloat16 for 8 bits); ``k`` / ``v`` handed in may be strided.  Rows that the
    cache does not hold become 0."""
    code = _pool(k_pages, v_pages, k_scales, v_scales)
    dev = k_pages.device
    num_pages, hkv, page_size, d = k_pages.shape
    cu_h, batch = _batch_args(cu_seqlens_host, cu_seqlens, used_kv_lens, (block_tables,), dev,
                              ("block_tables",))
    rows = int(cu_h[-1]) if cu_h.size else 0
    shape = (rows, hkv, d)
    try:
        ks0, ks1, ks2 = k.stride()
        vs0, vs1, vs2 = v.stride()
        out, index = k.dtype, dev.index
        usual = (out in _ACT_DTYPES and v.dtype is out and (dtype is None or dtype is out) and
                 k.shape == shape and v.shape == shape and ks2 == 1 and vs2 == 1 and
                 k.get_device() == index and v.get_device() == index)
    except (AttributeError, ValueError):
        usual = False
    if not usual:
        k, v, out = _check_rows(k, v, dtype, (max(rows, 0), hkv, d), k_pages, stream)
        ks0, ks1, _ = k.stride()
        vs0, vs1, _ = v.stride()
    _check(_on(dev, _native.load().sa_load_kv, k_pages.data_ptr(), v_pages.data_ptr(),
               _ptr(k_scales), _ptr(v_scales), num_pages, code, block_tables.data_ptr(),
               block_tables.shape[1], _host_ptr(cu_h), cu_seqlens.data_ptr(), batch, rows,
               used_kv_lens.data_ptr(), hkv, d, page_size, k.data_ptr(), v.data_ptr(),
               _ACT_DTYPES[out], ks0, ks1, vs0, vs1, _status_word(status, dev),
               _stream(stream, dev)), "sa_load_kv")
    return k, v


def _check_rows(k, v, dtype, shape, k_pages, stream):
    """The outputs of a :func:`sa_load_kv` call, made where not given, and their type."""
    dev = k_pages.device
    if dtype is None:
        some = k if k is not None else v
        dtype = some.dtype if some is not None else (
            torch.float32 if k_pages.dtype is torch.float32 else torch.bfloat16)
    if dtype not in _ACT_DTYPES:
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    made = []
    for t, name in ((k, "k"), (v, "v")):
        if t is None:
            with _allocating(stream):
                t = torch.empty(shape, dtype=dtype, device=dev)
        elif _heads(t, name) != dtype or t.shape != shape or t.device != dev:
            raise ValueError(f"{name} must be {shape} of {dtype} on {dev}")
        made.append(t)
    return made[0], made[1], dtype


def allocate_decode_workspace(batch, hq, hkv, head_dim, device) -> torch.Tensor:
    """Scratch for :func:`sa_decode_attention` over these sizes, to be kept from call
    to call."""
    n = ctypes.c_size_t(0)
    _check(_native.load().sa_decode_workspace_size(batch, hq, hkv, head_dim, ctypes.byref(n)),
           "sa_decode_workspace_size")
    return torch.empty(n.value + 256, dtype=torch.uint8, device=device)


def sa_decode_attention(q, k_pages, v_pages, block_tables, used_kv_lens, softmax_scale, window=0,
                        k_scales=None, v_scales=None, out=None, lse=None, with_lse=True,
                        workspace=None, status=None, stream=None):
    """One new token per sequence over its whole cache: query b of ``q`` [batch, hq, d]
    (float32 or bfloat16) attends over the positions below ``used_kv_lens[b]``, the
    last ``window`` of them where that is not 0.  Any cache type (with ``k_scales`` and
    ``v_scales`` for 8 bits) and any hq / hkv.  ``workspace``: see
    :func:`allocate_decode_workspace`; calls that overlap need one each.  Returns (out, lse): out of q's type, lse
    [batch, hq] float32; a sequence of length 0 gets 0 and -inf."""
    code = _pool(k_pages, v_pages, k_scales, v_scales)
    dev = k_pages.device
    num_pages, hkv, page_size, d = k_pages.shape
    try:
        index, dtype = dev.index, q.dtype
        batch, hq, channels = q.shape
        usual = (dtype in _ACT_DTYPES and channels == d and _alike(index, dtype, q, out) and
                 out.shape == q.shape and _alike(index, torch.float32, lse) and
                 lse.shape == (batch, hq) and _alike(index, torch.int32, block_tables, used_kv_lens) and
                 used_kv_lens.shape == (batch,) and block_tables.dim() == 2 and
                 block_tables.shape[0] == batch and _alike(index, torch.uint8, workspace))
    except (AttributeError, TypeError, ValueError):
        usual = False
    if not usual:
        batch, hq = _check_decode(q, d, dev, block_tables, used_kv_lens, out, lse, workspace)
        with _allocating(stream):
            if out is None:
                out = torch.empty((batch, hq, d), dtype=q.dtype, device=dev)
            if lse is None and with_lse:
                lse = torch.empty((batch, hq), dtype=torch.float32, device=dev)
            if workspace is None:
                workspace = allocate_decode_workspace(batch, hq, hkv, d, dev)
    base, at, to = workspace.data_ptr(), q.data_ptr(), out.data_ptr()
    aligned = (base + 255) & ~255
    if at == to and batch:
        raise ValueError("out must not be q")
    _check(_on(dev, _native.load().sa_decode_attention, at, _ACT_DTYPES[q.dtype],
               k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_scales), _ptr(v_scales), num_pages, code,
               block_tables.data_ptr(), block_tables.shape[1], used_kv_lens.data_ptr(), batch, hq,
               hkv, d, page_size, softmax_scale, window, to, _ptr(lse), aligned,
               max(workspace.numel() - (aligned - base), 0), _status_word(status, dev),
               _stream(stream, dev)), "sa_decode_attention")
    return out, lse


def _check_decode(q, d, dev, block_tables, used_kv_lens, out, lse, workspace):
    """What is wrong with a :func:`sa_decode_attention` call's tensors, if anything is:
    else (batch, hq)."""
    if getattr(q, "dtype", None) not in _ACT_DTYPES:
        raise TypeError("q must be a float32 or bfloat16 tensor")
    _require(q, q.dtype, "q", dev)
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError(f"q must be [batch, hq, {d}], got {tuple(q.shape)}")
    batch, hq, _ = q.shape
    _require(block_tables, torch.int32, "block_tables", dev)
    _require(used_kv_lens, torch.int32, "used_kv_lens", dev)
    if block_tables.dim() != 2 or block_tables.shape[0] != batch or used_kv_lens.numel() != batch:
        raise ValueError(f"block_tables and used_kv_lens must have a row for each of the {batch} sequences")
    _check_room(dev, (out, q.dtype, batch * hq * d, "out"), (lse, torch.float32, batch * hq, "lse"))
    if workspace is not None:
        _require(workspace, torch.uint8, "workspace", dev)
    return batch, hq


def sa_get_status(index: Index, stream=None) -> int:
    """Synchronise and return the device status code (0 = OK)."""
    return int(_on(index.device, _native.load().sa_get_status, ctypes.byref(index.c),
                   _stream(stream, index.device)))


def sa_clear_status(index: Index, stream=None) -> None:
    _check(_on(index.device, _native.load().sa_clear_status, ctypes.byref(index.c),
               _stream(stream, index.device)), "sa_clear_status")


def sa_debug_stall(site: int, spin_limit: int = 0) -> None:
    """Test hook: make the bounded wait at ``site`` run out on every launch
    from now on (STALL_INDEX_BARRIER, STALL_FUSED_COPIES, STALL_SELECT_COPIES), with ``spin_limit``
    tries per wait (0 = the library default); STALL_NONE restores normal
    operation."""
    _check(_native.load().sa_debug_stall(int(site), int(spin_limit)), "sa_debug_stall")


def sa_debug_cta_stats(stats=None) -> None:
    """Test hook: with ``stats`` (a zeroed int64 CUDA tensor of 3 * n_ctas
    elements) every later tensor-core forward adds each CTA's claimed rows
    and units and writes its busy cycles there; None turns it off."""
    if stats is None:
        _check(_native.load().sa_debug_cta_stats(None, 0), "sa_debug_cta_stats")
        return
    _require(stats, torch.int64, "stats")
    _check(_native.load().sa_debug_cta_stats(_ptr(stats), stats.numel() // 3),
           "sa_debug_cta_stats")
