"""Python binding of libli, the B200 LightningIndexer (C ABI in include/li.h).

The binding only marshals arguments: every step of the indexer and of the
sparse attention that consumes its output runs in the CUDA kernels of
``libli.so``.  Functions keep the C names (``li_indexer``,
``li_quant_indexer``, ``li_topk``, ``li_sparse_attention``,
``li_output_shape``, ``li_workspace_size``, ``li_read_device_status``, ...)
and take torch CUDA tensors, passing their device pointers and the current
CUDA stream.  ``indexer(...)`` and ``sparse_attention(...)`` are convenience
wrappers that allocate the outputs (and the indexer's workspace) with torch.

There is no fallback: if ``libli.so`` is missing or fails to load, importing
the functions raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libli.so")

LI_OK = 0
STATUS_NAMES = {0: "LI_OK", 1: "LI_ERR_NULL", 2: "LI_ERR_SHAPE", 3: "LI_ERR_DTYPE",
                4: "LI_ERR_LAYOUT", 5: "LI_ERR_UNSUPPORTED", 6: "LI_ERR_WORKSPACE",
                7: "LI_ERR_CUDA", 8: "LI_ERR_DEVICE"}
DTYPE = {"bf16": 0, "fp16": 1, "fp32": 2, "e4m3": 3, "int8": 4}
LAYOUT = {"BSND": 0, "TND": 1, "PA_BSND": 2}
DEV_BAD_QLEN, DEV_BAD_KLEN, DEV_BAD_BLOCK, DEV_NEG_SCALE, DEV_TIMEOUT = 1, 2, 4, 8, 16
DEV_BAD_INDEX = 32
DEV_NO_PAGES, DEV_BAD_ROW = 64, 128
ROPE_PAIRING = {"half": 0, "interleaved": 1}
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
INT64_MAX = (1 << 63) - 1
# LI_NOALLOC_SCRATCH_BYTES of include/li.h: the scratch li_indexer_noalloc holds
NOALLOC_SCRATCH_BYTES = 32 << 20

EXPORTS = ("li_output_shape", "li_workspace_size", "li_indexer", "li_quant_indexer", "li_topk",
           "li_last_error", "li_read_device_status", "li_selftest_bounded_wait",
           "li_last_launch_count", "li_set_profile_events", "li_indexer_noalloc",
           "li_sparse_attention", "li_rope", "li_rope_frequencies", "li_pages_workspace_size",
           "li_pages_copy", "li_pages_reserve", "li_pages_fork", "li_pages_free", "li_pages_compact",
           "li_segment_pool", "li_segment_select", "li_segment_attention")


class LiError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("%s: %s" % (STATUS_NAMES.get(status, str(status)), msg))
        self.status = status


class Params(ctypes.Structure):
    """Mirror of li_params."""
    _fields_ = [
        ("layout_q", ctypes.c_int32), ("layout_k", ctypes.c_int32),
        ("dtype_qk", ctypes.c_int32), ("dtype_w", ctypes.c_int32),
        ("dtype_scale", ctypes.c_int32),
        ("B", ctypes.c_int32), ("S1", ctypes.c_int32), ("S2", ctypes.c_int32),
        ("T1", ctypes.c_int32), ("T2", ctypes.c_int32), ("N1", ctypes.c_int32),
        ("N2", ctypes.c_int32), ("D", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("key_block_stride", ctypes.c_int64),
        ("sparse_count", ctypes.c_int32), ("sparse_mode", ctypes.c_int32),
        ("pre_tokens", ctypes.c_int64), ("next_tokens", ctypes.c_int64),
        ("return_value", ctypes.c_int32), ("max_seqlen_k", ctypes.c_int32),
        ("init_num", ctypes.c_int32), ("local_num", ctypes.c_int32),
        ("cmp_ratio", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("cmp_residual_k", ctypes.c_void_p),
    ]


class SfaParams(ctypes.Structure):
    """Mirror of li_sfa_params (sparse attention over the selected keys)."""
    _fields_ = [
        ("layout_q", ctypes.c_int32), ("layout_kv", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("B", ctypes.c_int32), ("S1", ctypes.c_int32), ("S2", ctypes.c_int32),
        ("T1", ctypes.c_int32), ("T2", ctypes.c_int32),
        ("N1", ctypes.c_int32), ("D", ctypes.c_int32), ("Dv", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32), ("sparse_count", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float), ("reserved", ctypes.c_int32),
    ]


class RopeParams(ctypes.Structure):
    """Mirror of li_rope_params (rotary positions)."""
    _fields_ = [
        ("dtype", ctypes.c_int32), ("rows", ctypes.c_int32), ("N1", ctypes.c_int32), ("N2", ctypes.c_int32),
        ("D", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("rot_offset", ctypes.c_int32),
        ("pairing", ctypes.c_int32), ("inverse", ctypes.c_int32), ("mscale", ctypes.c_float),
        ("q_row_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
        ("k_row_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
        ("q_out_row_stride", ctypes.c_int64), ("q_out_head_stride", ctypes.c_int64),
        ("k_out_row_stride", ctypes.c_int64), ("k_out_head_stride", ctypes.c_int64),
        ("reserved", ctypes.c_int32),
    ]


class PagesParams(ctypes.Structure):
    """Mirror of li_pages_params (the pages of a cache)."""
    _fields_ = [("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("B", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class PagePool(ctypes.Structure):
    """Mirror of li_page_pool (one pool of a cache)."""
    _fields_ = [("base", ctypes.c_void_p), ("page_bytes", ctypes.c_int64), ("page_stride", ctypes.c_int64)]


class SegmentParams(ctypes.Structure):
    """Mirror of li_segment_params (segment-sparse attention)."""
    _fields_ = [
        ("layout_q", ctypes.c_int32), ("layout_kv", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("B", ctypes.c_int32), ("S1", ctypes.c_int32), ("S2", ctypes.c_int32),
        ("T1", ctypes.c_int32), ("T2", ctypes.c_int32),
        ("N1", ctypes.c_int32), ("N2", ctypes.c_int32), ("D", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
        ("kv_block_stride", ctypes.c_int64),
        ("seg_size", ctypes.c_int32), ("seg_count", ctypes.c_int32), ("init_segs", ctypes.c_int32),
        ("local_segs", ctypes.c_int32), ("max_segs", ctypes.c_int32), ("sparse_mode", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float), ("reserved", ctypes.c_int32),
    ]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libli.so (loudly failing when it is absent)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libli.so is not built (run python -m sparse_attention_top_n1_b200.build)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        P = ctypes.POINTER(Params)
        G, L_, S_ = (ctypes.POINTER(t) for t in (PagesParams, PagePool, SegmentParams))
        sig = {
            "li_output_shape": (ctypes.c_int, [P, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(i32)]),
            "li_workspace_size": (ctypes.c_int, [P, ctypes.POINTER(sz)]),
            "li_indexer": (ctypes.c_int, [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "li_quant_indexer": (ctypes.c_int, [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "li_topk": (ctypes.c_int, [vp, i64, vp, i32, i32, vp, vp, vp]),
            "li_last_error": (ctypes.c_char_p, []),
            "li_read_device_status": (ctypes.c_int, [vp, vp, ctypes.POINTER(i32)]),
            "li_selftest_bounded_wait": (ctypes.c_int, [vp, i64, vp]),
            "li_last_launch_count": (i32, []),
            "li_set_profile_events": (None, [ctypes.POINTER(ctypes.c_void_p), i32]),
            "li_indexer_noalloc": (ctypes.c_int, [P, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
            "li_sparse_attention": (ctypes.c_int, [ctypes.POINTER(SfaParams), vp, vp, vp, vp, vp,
                                                   vp, vp, vp, vp, vp, vp]),
            "li_rope": (ctypes.c_int, [ctypes.POINTER(RopeParams)] + [vp] * 7),
            "li_rope_frequencies": (ctypes.c_int, [i32, i32, ctypes.c_double, ctypes.c_double, i32, ctypes.c_double,
                                                   ctypes.c_double, vp, ctypes.POINTER(ctypes.c_float)]),
            "li_pages_workspace_size": (ctypes.c_int, [G, ctypes.POINTER(sz)]),
            "li_pages_copy": (ctypes.c_int, [G, L_, i32, vp, vp, i32, vp, vp]),
            "li_pages_reserve": (ctypes.c_int, [G] + [vp] * 9 + [sz, vp]),
            "li_pages_fork": (ctypes.c_int, [G, L_, i32, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]),
            "li_pages_free": (ctypes.c_int, [G, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]),
            "li_pages_compact": (ctypes.c_int, [G, L_, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
            "li_segment_pool": (ctypes.c_int, [S_] + [vp] * 7),
            "li_segment_select": (ctypes.c_int, [S_] + [vp] * 7),
            "li_segment_attention": (ctypes.c_int, [S_] + [vp] * 11),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(status: int):
    if status != LI_OK:
        raise LiError(status, lib().li_last_error().decode())


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


_torch = None


def _load_torch():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


class _Alloc:
    """Allocations of one call on `device` that launches on `stream` (None: the
    device's current one).  They come from the launch stream's memory, so that no
    work of another stream is still under way in them; outputs are also marked as
    used by the current stream, where the caller reads and frees them.  A
    workspace has to be kept until after the launch."""

    def __init__(self, stream, device):
        torch = self.torch = _load_torch()
        self.device, self.on = device, None
        if stream is None or device.type != "cuda":
            return
        on = stream
        if not hasattr(stream, "cuda_stream"):             # a raw handle; 0 and 1 name the default stream
            h = int(getattr(stream, "value", stream) or 0)
            on = torch.cuda.ExternalStream(h, device=device) if h > 1 else torch.cuda.default_stream(device)
        reader = torch.cuda.current_stream(device)
        if on.cuda_stream != reader.cuda_stream:
            self.on, self.reader = on, reader

    def workspace(self, *shape, dtype):
        if self.on is None:
            return self.torch.empty(shape, dtype=dtype, device=self.device)
        with self.torch.cuda.stream(self.on):
            return self.torch.empty(shape, dtype=dtype, device=self.device)

    def output(self, *shape, dtype):
        t = self.workspace(*shape, dtype=dtype)
        if self.on is not None:
            t.record_stream(self.reader)
        return t


def make_params(problem=None, **kw) -> Params:
    """Build li_params from an object with the attribute names of li_params
    (layouts and dtypes given as strings) and/or keyword overrides."""
    f = {}
    if problem is not None:
        for name, _ in Params._fields_:
            if hasattr(problem, name):
                f[name] = getattr(problem, name)
    f.update(kw)
    f.setdefault("N2", 1)
    f.setdefault("pre_tokens", INT64_MAX)
    f.setdefault("next_tokens", INT64_MAX)
    f.setdefault("dtype_scale", "fp32")
    for name in ("layout_q", "layout_k"):
        if isinstance(f.get(name), str):
            f[name] = LAYOUT[f[name]]
    for name in ("dtype_qk", "dtype_w", "dtype_scale"):
        if isinstance(f.get(name), str):
            f[name] = DTYPE[f[name]]
    return Params(**{k: v for k, v in f.items() if k in dict(Params._fields_)})


# ---------------------------------------------------------------- C-ABI calls

def li_output_shape(params: Params):
    dims = (ctypes.c_int64 * 4)()
    nd = ctypes.c_int32()
    _check(lib().li_output_shape(ctypes.byref(params), dims, ctypes.byref(nd)))
    return tuple(dims[i] for i in range(nd.value))


def li_workspace_size(params: Params) -> int:
    n = ctypes.c_size_t()
    _check(lib().li_workspace_size(ctypes.byref(params), ctypes.byref(n)))
    return n.value


def li_indexer(params, query, key, weights, act_seq_q, act_seq_k, block_table, sparse_indices,
               sparse_values, workspace, workspace_bytes=None, stream=None):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib().li_indexer(ctypes.byref(params), _ptr(query), _ptr(key), _ptr(weights),
                            _ptr(act_seq_q), _ptr(act_seq_k), _ptr(block_table),
                            _ptr(sparse_indices), _ptr(sparse_values), _ptr(workspace),
                            workspace_bytes, _stream(stream)))


def li_quant_indexer(params, query, key, weights, q_scale, k_scale, act_seq_q, act_seq_k,
                     block_table, sparse_indices, sparse_values, workspace,
                     workspace_bytes=None, stream=None):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib().li_quant_indexer(ctypes.byref(params), _ptr(query), _ptr(key), _ptr(weights),
                                  _ptr(q_scale), _ptr(k_scale), _ptr(act_seq_q),
                                  _ptr(act_seq_k), _ptr(block_table), _ptr(sparse_indices),
                                  _ptr(sparse_values), _ptr(workspace), workspace_bytes,
                                  _stream(stream)))


def li_topk(scores, ld, row_len, rows, k, sparse_indices, sparse_values=None, stream=None):
    _check(lib().li_topk(_ptr(scores), ld, _ptr(row_len), rows, k, _ptr(sparse_indices),
                         _ptr(sparse_values), _stream(stream)))


def li_indexer_noalloc(params, query, key, weights, act_seq_q, act_seq_k, block_table,
                       sparse_indices, sparse_values, stream=None):
    """li_indexer with the library's built-in scratch instead of a workspace
    (see include/li.h: for callers that cannot allocate device memory)."""
    _check(lib().li_indexer_noalloc(ctypes.byref(params), _ptr(query), _ptr(key), _ptr(weights),
                                    _ptr(act_seq_q), _ptr(act_seq_k), _ptr(block_table),
                                    _ptr(sparse_indices), _ptr(sparse_values), _stream(stream)))


def make_sfa_params(problem=None, **kw) -> SfaParams:
    """li_sfa_params from an object with its field names (layouts and dtype as
    strings; softmax_scale 0 or absent = 1/sqrt(D)) and/or keyword overrides."""
    f = {}
    if problem is not None:
        for name, _ in SfaParams._fields_:
            if hasattr(problem, name):
                f[name] = getattr(problem, name)
    f.update(kw)
    for name in ("layout_q", "layout_kv"):
        if isinstance(f.get(name), str):
            f[name] = LAYOUT[f[name]]
    if isinstance(f.get("dtype"), str):
        f["dtype"] = DTYPE[f["dtype"]]
    if not f.get("softmax_scale"):
        f["softmax_scale"] = f.get("D", 128) ** -0.5
    return SfaParams(**{k: v for k, v in f.items() if k in dict(SfaParams._fields_)})


def li_sparse_attention(params: SfaParams, query, key, value, sparse_indices, act_seq_q, act_seq_k,
                        block_table, out, lse=None, status=None, stream=None):
    _check(lib().li_sparse_attention(ctypes.byref(params), _ptr(query), _ptr(key), _ptr(value),
                                     _ptr(sparse_indices), _ptr(act_seq_q), _ptr(act_seq_k),
                                     _ptr(block_table), _ptr(out), _ptr(lse), _ptr(status),
                                     _stream(stream)))


def sparse_attention(params: SfaParams, query, key, value, sparse_indices, *, act_seq_q=None,
                     act_seq_k=None, block_table=None, want_lse=True, status=None, stream=None):
    """Run li_sparse_attention, allocating out [rows, N1, Dv] (the query's dtype)
    and, when asked, lse [rows, N1] fp32.  Returns (out, lse or None)."""
    rows = params.B * params.S1 if params.layout_q == LAYOUT["BSND"] else params.T1
    new = _Alloc(stream, query.device).output
    out = new(rows, params.N1, params.Dv, dtype=query.dtype)
    lse = new(rows, params.N1, dtype=_torch.float32) if want_lse else None
    li_sparse_attention(params, query, key, value, sparse_indices, act_seq_q, act_seq_k, block_table,
                        out, lse, status, stream)
    return out, lse


def li_read_device_status(workspace, stream=None) -> int:
    """SYNCHRONISING: the LI_DEV_* bits left by the last call on `workspace`."""
    flags = ctypes.c_int32()
    st = lib().li_read_device_status(_ptr(workspace), _stream(stream), ctypes.byref(flags))
    if st not in (LI_OK, 8):
        _check(st)
    return flags.value


def li_selftest_bounded_wait(status_word, timeout_ns: int, stream=None):
    _check(lib().li_selftest_bounded_wait(_ptr(status_word), timeout_ns, _stream(stream)))


def li_last_launch_count() -> int:
    return lib().li_last_launch_count()


def li_set_profile_events(events):
    """Record per-stage CUDA events in later calls (list of 4 torch.cuda.Event
    created with enable_timing=True), or turn it off with None."""
    if not events:
        lib().li_set_profile_events(None, 0)
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    lib().li_set_profile_events(arr, len(events))


def li_last_error() -> str:
    return lib().li_last_error().decode()


# ---------------------------------------------------------------- convenience

def alloc_workspace(params: Params, device="cuda"):
    import torch
    n = li_workspace_size(params)
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def indexer(params: Params, query, key, weights, *, act_seq_q=None, act_seq_k=None,
            block_table=None, q_scale=None, k_scale=None, cmp_residual_k=None, workspace=None,
            out=None, stream=None):
    """Run li_indexer / li_quant_indexer, allocating outputs (and workspace).

    cmp_residual_k (int32 [B] on the device) is stored into params before the
    call.  Returns (sparse_indices, sparse_values); sparse_values is an empty
    (0,) tensor when return_value is 0, as the CANN guide's output rule says.
    """
    if cmp_residual_k is not None:
        params.cmp_residual_k = _ptr(cmp_residual_k)
    shape = li_output_shape(params)
    alloc = _Alloc(stream, query.device)
    if out is None:
        idx = alloc.output(*shape, dtype=_torch.int32)
        val = alloc.output(*(shape if params.return_value else (0,)), dtype=_torch.float32)
    else:
        idx, val = out
    if workspace is None:
        workspace = alloc.workspace(max(li_workspace_size(params), 256), dtype=_torch.uint8)
    vptr = val if params.return_value else None
    if params.dtype_qk == DTYPE["e4m3"] or params.dtype_qk == DTYPE["int8"]:
        li_quant_indexer(params, query, key, weights, q_scale, k_scale, act_seq_q, act_seq_k,
                         block_table, idx, vptr, workspace, stream=stream)
    else:
        li_indexer(params, query, key, weights, act_seq_q, act_seq_k, block_table, idx, vptr,
                   workspace, stream=stream)
    return idx, val


# ---------------------------------------------------------------- rotary positions

def _arg(name, t, index, dtype, numel):
    """Pointer of a tensor argument, after its checks: on device `index`, of
    `dtype`, contiguous with `numel` elements (None: strides and size are the
    caller's)."""
    if t.get_device() != index:
        raise ValueError("%s is on %s, the call's first tensor on %s"
                         % (name, t.device, "cuda:%d" % index if index >= 0 else "the host"))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, not %s" % (name, dtype, t.dtype))
    if numel is not None and (t.numel() != numel or not t.is_contiguous()):
        raise ValueError("%s must be contiguous with %d elements, not %s" % (name, numel, tuple(t.shape)))
    return t.data_ptr()


def _strided(name, t, index, dtype, extent):
    """The same for a tensor whose strides the parameters say: `extent` elements
    from its first one on have to lie in its memory."""
    p = _arg(name, t, index, dtype, None)
    room = t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
    if room < extent:
        raise ValueError("%s has %d elements of memory, the call's strides reach over %d" % (name, room, extent))
    return p


def _opt(name, t, index, dtype, numel):
    return None if t is None else _arg(name, t, index, dtype, numel)


def _torch_dtype(code):
    torch = _load_torch()
    return torch.bfloat16 if code == 0 else torch.float16 if code == 1 else torch.float32


def _launch(index, f, *args, stream=None, held=None):
    """Call a library function for tensors on CUDA device `index`: the current
    device and stream are that device's.  `held`: memory that only this call
    refers to, kept until its kernels are in the stream."""
    torch = _torch
    if index < 0:
        raise ValueError("the call's tensors must be on a CUDA device")
    if index == torch._C._cuda_getDevice():
        st = f(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(index):
            st = f(*args, _stream(stream))
    if st:
        _check(st)


def make_rope_params(problem=None, **kw) -> RopeParams:
    """li_rope_params from an object with its field names (dtype and pairing as
    strings) and/or keyword overrides; mscale defaults to 1, N2 to 0 (no key)."""
    f = {}
    if problem is not None:
        f.update((n, getattr(problem, n)) for n, _ in RopeParams._fields_ if hasattr(problem, n))
    f.update(kw)
    f.setdefault("mscale", 1.0)
    if isinstance(f.get("dtype"), str):
        f["dtype"] = DTYPE[f["dtype"]]
    if isinstance(f.get("pairing"), str):
        f["pairing"] = ROPE_PAIRING[f["pairing"]]
    return RopeParams(**f)


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_positions: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(inv_freq, mscale): radians per position of each pair (fp64 tensor on the
    host, to be moved to the device once) and the factor for make_rope_params."""
    import torch
    out = torch.empty(max(1, rot_dim // 2), dtype=torch.float64)
    m = ctypes.c_float()
    _check(lib().li_rope_frequencies(ROPE_SCALING[scaling], rot_dim, base, factor, original_positions, beta_fast,
                                     beta_slow, out.data_ptr(), ctypes.byref(m)))
    return out, m.value


def li_rope(params: RopeParams, positions, inv_freq, query, key, query_out, key_out, stream=None):
    _check(lib().li_rope(ctypes.byref(params), _ptr(positions), _ptr(inv_freq), _ptr(query), _ptr(key),
                         _ptr(query_out), _ptr(key_out), _stream(stream)))


def _heads(name, t, index, dtype, p, N, row, head):
    """Pointer of N heads per row at the given strides (0: dense)."""
    last = (p.rows - 1) * (row or N * p.D) + (N - 1) * (head or p.D)
    return _strided(name, t, index, dtype, last + p.D if p.rows > 0 else 0)


def rope(params: RopeParams, positions, inv_freq, query, key=None, *, out=None, key_out=None, stream=None):
    """Rotate query [.., N1, D] and key [.., N2, D] by their rows' positions,
    allocating dense outputs unless they are given (query and key themselves for
    in place).  Returns (out, key_out or None)."""
    torch = _load_torch()
    p, d, dt = params, query.get_device(), _torch_dtype(params.dtype)
    rows, D = p.rows, p.D
    nq = rows * p.N1 * D
    q = (_heads("query", query, d, dt, p, p.N1, p.q_row_stride, p.q_head_stride) if p.q_row_stride or p.q_head_stride
         else _arg("query", query, d, dt, nq))
    if out is None:
        out = _Alloc(stream, query.device).output(rows, p.N1, D, dtype=dt)
    o = (_heads("out", out, d, dt, p, p.N1, p.q_out_row_stride, p.q_out_head_stride)
         if p.q_out_row_stride or p.q_out_head_stride else _arg("out", out, d, dt, nq))
    k = ko = None
    if key is not None:
        if key_out is None:
            key_out = _Alloc(stream, query.device).output(rows, p.N2, D, dtype=dt)
        nk = rows * p.N2 * D
        k = (_heads("key", key, d, dt, p, p.N2, p.k_row_stride, p.k_head_stride) if p.k_row_stride or p.k_head_stride
             else _arg("key", key, d, dt, nk))
        ko = (_heads("key_out", key_out, d, dt, p, p.N2, p.k_out_row_stride, p.k_out_head_stride)
              if p.k_out_row_stride or p.k_out_head_stride else _arg("key_out", key_out, d, dt, nk))
    _launch(d, lib().li_rope, ctypes.byref(p), _arg("positions", positions, d, torch.int32, rows),
            _arg("inv_freq", inv_freq, d, torch.float64, p.rot_dim // 2), q, k, o, ko, stream=stream)
    return out, key_out


# ---------------------------------------------------------------- pages of a cache

def make_pages_params(**kw) -> PagesParams:
    return PagesParams(**kw)


def page_pools(pools):
    """Descriptors of pool tensors [num_pages, ...] (axis 0 may be strided, a
    page itself is contiguous and overlaps no other), for the pages calls; they
    take a list too."""
    if isinstance(pools, ctypes.Array):
        return pools
    arr = (PagePool * len(pools))()
    for d, t in zip(arr, pools):
        if t.dim() < 1:
            raise ValueError("a pool needs the page as its axis 0")
        es, n = t.element_size(), t.shape[0]
        each = t.numel() // n if n else 0
        if n and not t.is_contiguous() and not t[0].is_contiguous():
            raise ValueError("a pool's pages must be contiguous")
        if n > 1 and t.stride(0) < each:
            raise ValueError("a pool's pages overlap: %d elements apart, %d in each" % (t.stride(0), each))
        d.base = t.data_ptr()
        d.page_bytes = each * es
        d.page_stride = (t.stride(0) if n > 1 else each) * es
    arr.tensors = list(pools)
    return arr


def li_pages_workspace_size(params: PagesParams) -> int:
    n = ctypes.c_size_t()
    _check(lib().li_pages_workspace_size(ctypes.byref(params), ctypes.byref(n)))
    return n.value


def alloc_pages_workspace(params: PagesParams, device="cuda"):
    import torch
    return torch.empty(li_pages_workspace_size(params), dtype=torch.uint8, device=device)


def _pools_on(pools, params, index):
    arr = page_pools(pools)
    for t in getattr(arr, "tensors", ()):
        if t.get_device() != index:
            raise ValueError("a pool is on %s, the call's other tensors on cuda:%d" % (t.device, index))
        if t.shape[0] != params.num_pages:
            raise ValueError("a pool has %d pages, not %d" % (t.shape[0], params.num_pages))
    return arr


def _pages_state(params, table, lens, refs, out, workspace, status, stream):
    """Checks the state, allocates what is not given; returns (device index, out,
    pointers of the state, of the outputs, of status and the workspace, and the
    workspace itself: to be held until the launch)."""
    torch = _load_torch()
    p, i32, d = params, torch.int32, table.get_device()
    B, pages = p.B, p.num_pages
    n = B * p.max_pages_per_seq
    if out is None:
        new = _Alloc(stream, table.device).output
        out = tuple(new(*t.shape, dtype=i32) for t in (table, lens, refs))
    if workspace is None:
        workspace = _Alloc(stream, table.device).workspace(li_pages_workspace_size(p), dtype=torch.uint8)
    state = _arg("table", table, d, i32, n), _arg("lens", lens, d, i32, B), _arg("refs", refs, d, i32, pages)
    to = out
    if to[0] is table and to[1] is lens and to[2] is refs:               # in place: checked already
        after = state
    else:
        after = (_arg("table_out", to[0], d, i32, n), _arg("lens_out", to[1], d, i32, B),
                 _arg("refs_out", to[2], d, i32, pages))
    return d, out, state, after, (_opt("status", status, d, i32, 1), _arg("workspace", workspace, d, torch.uint8, workspace.numel()),
                                  workspace.numel()), workspace


def pages_copy(params: PagesParams, pools, src, dst, *, status=None, stream=None):
    """li_pages_copy: page src[i] -> page dst[i] of every pool (int32 tensors)."""
    i32 = _load_torch().int32
    d, n = src.get_device(), src.numel()
    s, t = _arg("src", src, d, i32, n), _arg("dst", dst, d, i32, n)
    arr = _pools_on(pools, params, d)
    _launch(d, lib().li_pages_copy, ctypes.byref(params), arr, len(arr), s, t, n, _opt("status", status, d, i32, 1),
            stream=stream)


def pages_reserve(params: PagesParams, table, lens, refs, new_lens, *, out=None, workspace=None, status=None, stream=None):
    """li_pages_reserve.  Returns (table, lens, refs) after the call: new
    tensors, or `out` (which may be the inputs, for in place)."""
    d, out, state, after, rest, held = _pages_state(params, table, lens, refs, out, workspace, status, stream)
    _launch(d, lib().li_pages_reserve, ctypes.byref(params), *state, _arg("new_lens", new_lens, d, _torch.int32, params.B),
            *after, *rest, stream=stream, held=held)
    return out


def pages_fork(params: PagesParams, pools, table, lens, refs, src_rows, dst_rows, *, out=None, workspace=None,
               status=None, stream=None):
    """li_pages_fork: row dst_rows[i] becomes a child of row src_rows[i]."""
    d, out, state, after, rest, held = _pages_state(params, table, lens, refs, out, workspace, status, stream)
    n, i32 = src_rows.numel(), _torch.int32
    s, t = _arg("src_rows", src_rows, d, i32, n), _arg("dst_rows", dst_rows, d, i32, n)
    arr = _pools_on(pools, params, d)
    _launch(d, lib().li_pages_fork, ctypes.byref(params), arr, len(arr), *state, s, t, n, *after, *rest, stream=stream,
            held=held)
    return out


def pages_free(params: PagesParams, table, lens, refs, rows, *, out=None, workspace=None, status=None, stream=None):
    """li_pages_free: empties the rows `rows` (int32)."""
    d, out, state, after, rest, held = _pages_state(params, table, lens, refs, out, workspace, status, stream)
    n = rows.numel()
    _launch(d, lib().li_pages_free, ctypes.byref(params), *state, _arg("rows", rows, d, _torch.int32, n), n, *after, *rest,
            stream=stream, held=held)
    return out


def pages_compact(params: PagesParams, pools, table, lens, refs, *, out=None, workspace=None, status=None, stream=None):
    """li_pages_compact: the live pages become the first ones of the pool."""
    d, out, state, after, rest, held = _pages_state(params, table, lens, refs, out, workspace, status, stream)
    arr = _pools_on(pools, params, d)
    _launch(d, lib().li_pages_compact, ctypes.byref(params), arr, len(arr), *state, *after, *rest, stream=stream, held=held)
    return out


# ---------------------------------------------------------------- segment-sparse attention

def make_segment_params(problem=None, **kw) -> SegmentParams:
    """li_segment_params from an object with its field names (layouts and dtype
    as strings; softmax_scale 0 or absent = 1/sqrt(D)) and/or keyword overrides."""
    f = {}
    if problem is not None:
        f.update((n, getattr(problem, n)) for n, _ in SegmentParams._fields_ if hasattr(problem, n))
    f.update(kw)
    for name in ("layout_q", "layout_kv"):
        if isinstance(f.get(name), str):
            f[name] = LAYOUT[f[name]]
    if isinstance(f.get("dtype"), str):
        f["dtype"] = DTYPE[f["dtype"]]
    if not f.get("softmax_scale"):
        f["softmax_scale"] = f.get("D", 128) ** -0.5
    return SegmentParams(**f)


def _segment_rows(p):
    return p.B * p.S1 if p.layout_q == 0 else p.T1


def _segment_keys(name, t, p, index):
    """Pointer of the key (or value) tensor, after its checks."""
    dt, row = _torch_dtype(p.dtype), p.N2 * p.D
    if p.layout_kv != 2:
        return _arg(name, t, index, dt, (p.B * p.S2 if p.layout_kv == 0 else p.T2) * row)
    if not p.kv_block_stride:
        return _arg(name, t, index, dt, p.num_blocks * p.block_size * row)
    return _strided(name, t, index, dt, (p.num_blocks - 1) * p.kv_block_stride + p.block_size * row)


def _segment_lens(p, index, act_seq_q, act_seq_k, block_table, status):
    """Pointers of the lengths, the block table and status, after their checks."""
    i32, B = _torch.int32, p.B
    table = None
    if block_table is not None:
        table = (_arg("block_table", block_table, index, i32, B * p.max_blocks_per_seq) if p.layout_kv == 2
                 else block_table.data_ptr())
    return (_opt("act_seq_q", act_seq_q, index, i32, B), _opt("act_seq_k", act_seq_k, index, i32, B), table,
            _opt("status", status, index, i32, 1))


def segment_pool(params: SegmentParams, key, *, act_seq_k=None, block_table=None, first=None, pooled=None, status=None,
                 stream=None):
    """li_segment_pool: the segments' mean keys, fp32 [B, max_segs, N2, D].  With
    `first` (int32 [B]) and `pooled` only the segments of the tokens from there
    on are refreshed; segments behind a sequence keep what `pooled` holds
    (undefined in a newly allocated one)."""
    torch = _load_torch()
    p, d = params, key.get_device()
    k = _segment_keys("key", key, p, d)
    if pooled is None:
        if first is not None:
            raise ValueError("first refreshes an existing pooled tensor: pass pooled")
        pooled = _Alloc(stream, key.device).output(p.B, p.max_segs, p.N2, p.D, dtype=torch.float32)
    _, lens, table, st = _segment_lens(p, d, None, act_seq_k, block_table, status)
    _launch(d, lib().li_segment_pool, ctypes.byref(p), k, lens, table, _opt("first", first, d, torch.int32, p.B),
            _arg("pooled", pooled, d, torch.float32, p.B * p.max_segs * p.N2 * p.D), st, stream=stream)
    return pooled


def segment_select(params: SegmentParams, query, pooled, *, act_seq_q=None, act_seq_k=None, out=None, status=None,
                   stream=None):
    """li_segment_select: the chosen segments of each row and key head, int32
    [rows, N2, seg_count], ascending, -1 behind them."""
    torch = _load_torch()
    p, d = params, query.get_device()
    rows, N2, D, count = _segment_rows(p), p.N2, p.D, p.seg_count
    q = _arg("query", query, d, _torch_dtype(p.dtype), rows * p.N1 * D)
    if out is None:
        out = _Alloc(stream, query.device).output(rows, N2, count, dtype=torch.int32)
    q_lens, k_lens, _, st = _segment_lens(p, d, act_seq_q, act_seq_k, None, status)
    _launch(d, lib().li_segment_select, ctypes.byref(p), q, _arg("pooled", pooled, d, torch.float32, p.B * p.max_segs * N2 * D),
            q_lens, k_lens, _arg("out", out, d, torch.int32, rows * N2 * count), st, stream=stream)
    return out


def segment_attention(params: SegmentParams, query, key, value, seg_idx, *, act_seq_q=None, act_seq_k=None,
                      block_table=None, out=None, lse=None, want_lse=True, status=None, stream=None):
    """li_segment_attention, allocating out [rows, N1, D] (the query's dtype) and,
    when asked, lse [rows, N1] fp32.  Returns (out, lse or None)."""
    torch = _load_torch()
    p, d, dt = params, query.get_device(), _torch_dtype(params.dtype)
    rows, N1, D = _segment_rows(p), p.N1, p.D
    n = rows * N1 * D
    q, k, v = _arg("query", query, d, dt, n), _segment_keys("key", key, p, d), _segment_keys("value", value, p, d)
    if out is None:
        out = _Alloc(stream, query.device).output(rows, N1, D, dtype=dt)
    if lse is None and want_lse:
        lse = _Alloc(stream, query.device).output(rows, N1, dtype=torch.float32)
    q_lens, k_lens, table, st = _segment_lens(p, d, act_seq_q, act_seq_k, block_table, status)
    _launch(d, lib().li_segment_attention, ctypes.byref(p), q, k, v,
            _arg("seg_idx", seg_idx, d, torch.int32, rows * p.N2 * p.seg_count), q_lens, k_lens, table,
            _arg("out", out, d, dt, n), _opt("lse", lse, d, torch.float32, rows * N1), st, stream=stream)
    return out, lse
