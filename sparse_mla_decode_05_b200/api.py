"""Thin Python binding over the C ABI in include/sparse_mla.h.

Argument marshalling only: every step of the decode runs in the CUDA
library.  Torch tensors supply device pointers and the current stream.
There is no fallback: if the shared library is missing this module raises
on import.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsparse_mla.so")

H, D_QK, D_V, TILE = 64, 576, 512, 64
NSPLIT_STREAMK = -1          # smla_shape.nsplit asking for the stream-K plan
KV_BF16, KV_FP8_E4M3_ROWSCALE, KV_DSV4_PAGED = 0, 1, 2
DSV4_PAGE_BYTES, DSV4_D_QK = 37376, 512   # DeepSeek-V4 page: 64 x 576 slot bytes + 64 x 8 scale bytes

STATUS = {0: "SMLA_OK", 1: "SMLA_ERR_INVALID_ARG", 2: "SMLA_ERR_UNSUPPORTED", 3: "SMLA_ERR_WORKSPACE",
          4: "SMLA_ERR_CUDA", 5: "SMLA_ERR_DEVICE_TIMEOUT", 6: "SMLA_ERR_DEVICE_INDEX",
          7: "SMLA_ERR_DEVICE_LAYOUT"}


class SmlaError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {STATUS.get(code, code)}")
        self.code = code


class SmlaShape(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("d_qk", ctypes.c_int32),
        ("d_v", ctypes.c_int32), ("topk", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
        ("num_kv_rows", ctypes.c_int64), ("page_size", ctypes.c_int32),
        ("pages_per_seq", ctypes.c_int32), ("nsplit", ctypes.c_int32), ("tokens_per_seq", ctypes.c_int32),
    ]


class IndexerShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("max_ctx", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("pages_per_seq", ctypes.c_int32), ("reserved", ctypes.c_int32), ("num_key_rows", ctypes.c_int64)]


IX_HEADS, IX_DIM = 64, 128
ROPE_MAX_DIM = 256
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}          # smla_dtype


class RopeConfig(ctypes.Structure):
    _fields_ = [("rope_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("original_ctx", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double), ("mscale", ctypes.c_double)]


class RopeTableData(ctypes.Structure):
    _fields_ = [("rope_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("mscale", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("step", ctypes.c_uint64 * (ROPE_MAX_DIM // 2))]


class RopeShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("offset", ctypes.c_int32), ("dtype", ctypes.c_int32), ("transpose", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("x_token_stride", ctypes.c_int64), ("x_head_stride", ctypes.c_int64),
                ("y_token_stride", ctypes.c_int64), ("y_head_stride", ctypes.c_int64)]


class AppendShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("x_stride", ctypes.c_int64), ("num_kv_rows", ctypes.c_int64),
                ("x_dtype", ctypes.c_int32), ("kv_dtype", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("pages_per_seq", ctypes.c_int32), ("batch", ctypes.c_int32), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class EvictShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_ctx", ctypes.c_int32), ("budget", ctypes.c_int32),
                ("sinks", ctypes.c_int32), ("recent", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("pages_per_seq", ctypes.c_int32), ("new_pages_per_seq", ctypes.c_int32),
                ("num_kv_rows", ctypes.c_int64), ("num_key_rows", ctypes.c_int64)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m sparse_mla_decode_05_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, SZ, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    SP = ctypes.POINTER(SmlaShape)
    lib.sparse_mla_abi_version.restype = I32
    lib.sparse_mla_status_string.restype = ctypes.c_char_p
    lib.sparse_mla_status_string.argtypes = [I32]
    lib.sparse_mla_plan_nsplit.restype = I32
    lib.sparse_mla_plan_nsplit.argtypes = [SP]
    lib.sparse_mla_plan_merge.restype = I32
    lib.sparse_mla_plan_merge.argtypes = [SP]
    lib.sparse_mla_workspace_size.restype = SZ
    lib.sparse_mla_workspace_size.argtypes = [SP]
    lib.sparse_mla_decode.restype = I32
    lib.sparse_mla_decode.argtypes = [SP, P, P, P, P, P, F32, P, P, P, SZ, P]
    lib.sparse_mla_decode_split.restype = I32
    lib.sparse_mla_decode_split.argtypes = [SP, P, P, P, P, P, F32, P, P, P, SZ,
                                            ctypes.POINTER(I32), P]
    lib.sparse_mla_combine.restype = I32
    lib.sparse_mla_combine.argtypes = [I32, I32, I32, I32, P, P, P, P, P]
    lib.sparse_mla_get_device_error.restype = I32
    lib.sparse_mla_get_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    lib.sparse_mla_decode_static_scratch.restype = I32
    lib.sparse_mla_decode_static_scratch.argtypes = [SP, P, P, P, P, P, F32, P, P, P]
    lib.sparse_mla_decode_stalled.restype = I32
    lib.sparse_mla_decode_stalled.argtypes = [SP, P, P, P, F32, P, P, ctypes.c_int64, P]
    IP = ctypes.POINTER(IndexerShape)
    lib.sparse_mla_indexer_scores.restype = I32
    lib.sparse_mla_indexer_scores.argtypes = [IP, P, P, P, P, P, P, P]
    lib.sparse_mla_indexer_topk.restype = I32
    lib.sparse_mla_indexer_topk.argtypes = [IP, P, P, P, P]
    lib.sparse_mla_indexer.restype = I32
    lib.sparse_mla_indexer.argtypes = [IP, P, P, P, P, P, P, P, P]
    lib.sparse_mla_host_staging_size.restype = SZ
    lib.sparse_mla_host_staging_size.argtypes = [SP]
    lib.sparse_mla_decode_host.restype = I32
    lib.sparse_mla_decode_host.argtypes = [SP, P, P, P, P, P, F32, P, P, P, SZ, P]
    lib.sparse_mla_rope_init.restype = I32
    lib.sparse_mla_rope_init.argtypes = [ctypes.POINTER(RopeConfig), ctypes.POINTER(RopeTableData)]
    TP = ctypes.POINTER(RopeTableData)
    lib.sparse_mla_rope.restype = I32
    lib.sparse_mla_rope.argtypes = [ctypes.POINTER(RopeShape), TP, P, P, P, P]
    lib.sparse_mla_cache_append.restype = I32
    lib.sparse_mla_cache_append.argtypes = [ctypes.POINTER(AppendShape), P, P, TP, P, P, P, P, P, P, P]
    lib.sparse_mla_attn_weights.restype = I32
    lib.sparse_mla_attn_weights.argtypes = [SP, P, P, P, P, P, P, F32, P, P]
    lib.sparse_mla_accumulate_weights.restype = I32
    lib.sparse_mla_accumulate_weights.argtypes = [I32, ctypes.c_int64, I32, P, P, F32, P, P]
    EP = ctypes.POINTER(EvictShape)
    lib.sparse_mla_evict_select.restype = I32
    lib.sparse_mla_evict_select.argtypes = [EP, P, P, P, P, P, P]
    lib.sparse_mla_evict_compact.restype = I32
    lib.sparse_mla_evict_compact.argtypes = [EP, P, P, P, P, P, P, P, P]
    lib.sparse_mla_evict.restype = I32
    lib.sparse_mla_evict.argtypes = [EP, P, P, P, P, P, P, P, P, P, P, P]
    return lib


lib = _load()


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def make_shape(batch: int, topk: int, num_kv_rows: int, *, fp8: bool = False, dsv4: bool = False,
               page_size: int = 0, pages_per_seq: int = 0, nsplit: int = 0, tokens_per_seq: int = 0) -> SmlaShape:
    kind = KV_DSV4_PAGED if dsv4 else (KV_FP8_E4M3_ROWSCALE if fp8 else KV_BF16)
    return SmlaShape(batch, H, DSV4_D_QK if dsv4 else D_QK, D_V, topk, kind,
                     num_kv_rows, page_size, pages_per_seq, nsplit, tokens_per_seq)


def _tokens(q) -> int:
    """Query tokens per sequence: q is [B, 64, d] (one) or [B, T, 64, d]."""
    return q.shape[1] if q.dim() == 4 else 1


def _result_shapes(q):
    """(out, lse) shapes for q [B, (T,) 64, d]."""
    lead = tuple(q.shape[:-2])
    return lead + (H, D_V), lead + (H,)


def is_dsv4(kv) -> bool:
    """A DeepSeek-V4 paged cache: uint8 [pages, 37376]."""
    return kv.dtype == torch.uint8 and kv.dim() == 2 and kv.shape[1] == DSV4_PAGE_BYTES


def shape_for(q, kv, indices, *, page_table=None, page_size: int = 0, nsplit: int = 0) -> SmlaShape:
    """The shape of one call: q [B, 64, d] with indices [B, topk], or q
    [B, T, 64, d] with indices [B, T, topk] (T query tokens per sequence)."""
    dsv4 = is_dsv4(kv)
    T = _tokens(q)
    return make_shape(q.shape[0], indices.shape[-1], kv.shape[0] * (64 if dsv4 else 1),
                      fp8=(kv.dtype == torch.uint8 and not dsv4), dsv4=dsv4, page_size=page_size,
                      pages_per_seq=0 if page_table is None else page_table.shape[1], nsplit=nsplit,
                      tokens_per_seq=T if T > 1 else 0)


def plan_nsplit(shape: SmlaShape) -> int:
    return lib.sparse_mla_plan_nsplit(ctypes.byref(shape))


def plan_merge(shape: SmlaShape) -> int:
    """0: one split; 1: splits merged inside the split kernel (cluster);
    2: partials merged by the combine kernel; 3: stream-K (one CTA per SM
    over the rows' tiles, a shared row merged by its last CTA)."""
    return lib.sparse_mla_plan_merge(ctypes.byref(shape))


def workspace_size(shape: SmlaShape) -> int:
    return lib.sparse_mla_workspace_size(ctypes.byref(shape))


def _check_inputs(q, kv, indices, kv_row_scale, page_table, page_size):
    dsv4 = is_dsv4(kv)
    d_qk = DSV4_D_QK if dsv4 else D_QK
    if q.dtype != torch.bfloat16 or q.dim() not in (3, 4) or q.shape[-2:] != (H, d_qk):
        raise ValueError(f"q must be bf16 [B, 64, {d_qk}] or [B, T, 64, {d_qk}]")
    if not dsv4 and (kv.dim() != 2 or kv.shape[1] != D_QK or kv.dtype not in (torch.bfloat16, torch.uint8)):
        raise ValueError("kv must be [N, 576] bf16 or uint8 (fp8 e4m3fn codes), or uint8 [pages, 37376] "
                         "DeepSeek-V4 pages")
    if indices.dtype != torch.int32 or indices.dim() != q.dim() - 1 or indices.shape[:-1] != q.shape[:-2]:
        raise ValueError("indices must be int32 [B, topk] ([B, T, topk] for q [B, T, 64, d])")
    if dsv4:
        if kv_row_scale is not None:
            raise ValueError("DeepSeek-V4 pages carry their own scales: kv_row_scale must be None")
        if page_size != 64:
            raise ValueError("DeepSeek-V4 pages are paged: page_size must be 64")
    elif kv.dtype == torch.uint8 and (kv_row_scale is None or kv_row_scale.dtype != torch.float32):
        raise ValueError("fp8 cache needs float32 kv_row_scale [N]")
    if page_size and (page_table is None or page_table.dtype != torch.int32):
        raise ValueError("paged cache needs int32 page_table [B, pages_per_seq]")
    for t in (q, kv, indices, kv_row_scale, page_table):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous CUDA tensors")


def decode(q, kv, indices, scale: float, *, kv_row_scale=None, page_table=None, page_size: int = 0,
           nsplit: int = 0, out=None, lse=None, workspace=None):
    """out [B,64,512] bf16, lse [B,64] fp32 = sparse-MLA decode (one call to
    sparse_mla_decode).  Allocates out / lse / workspace with torch when not
    given."""
    _check_inputs(q, kv, indices, kv_row_scale, page_table, page_size)
    shape = shape_for(q, kv, indices, page_table=page_table, page_size=page_size, nsplit=nsplit)
    dev = q.device
    o_shape, l_shape = _result_shapes(q)
    if out is None:
        out = torch.empty(o_shape, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(l_shape, dtype=torch.float32, device=dev)
    ws_bytes = workspace_size(shape)
    if workspace is None and ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    st = lib.sparse_mla_decode(ctypes.byref(shape), _ptr(q), _ptr(kv), _ptr(kv_row_scale),
                               _ptr(page_table), _ptr(indices), float(scale), _ptr(out), _ptr(lse),
                               _ptr(workspace), 0 if workspace is None else workspace.numel(),
                               _stream(dev))
    if st != 0:
        raise SmlaError(st, "sparse_mla_decode")
    return out, lse


# Scratch size of decode_static_scratch (SMLA_STATIC_SCRATCH_BYTES).
STATIC_SCRATCH_BYTES = 24 << 20


def decode_static_scratch(q, kv, indices, scale: float, out, lse, *, kv_row_scale=None, page_table=None,
                          page_size: int = 0, nsplit: int = 0):
    """sparse_mla_decode_static_scratch: the decode step into caller-given
    ``out`` [B,64,512] bf16 and ``lse`` [B,64] fp32, with the split partials
    in the library's own static device scratch (STATIC_SCRATCH_BYTES), for
    callers that cannot allocate.  Calls that overlap in time on one device
    share that scratch and race; issue them on one stream."""
    _check_inputs(q, kv, indices, kv_row_scale, page_table, page_size)
    shape = shape_for(q, kv, indices, page_table=page_table, page_size=page_size, nsplit=nsplit)
    st = lib.sparse_mla_decode_static_scratch(ctypes.byref(shape), _ptr(q), _ptr(kv), _ptr(kv_row_scale),
                                              _ptr(page_table), _ptr(indices), float(scale), _ptr(out),
                                              _ptr(lse), _stream(q.device))
    if st != 0:
        raise SmlaError(st, "sparse_mla_decode_static_scratch")
    return out, lse


def decode_split(q, kv, indices, scale: float, *, kv_row_scale=None, page_table=None,
                 page_size: int = 0, nsplit: int = 0, out=None, lse=None, workspace=None):
    """The split kernel alone.  Returns (nsplit, out, lse, workspace); with
    nsplit > 1 the partial results are in the workspace (see the header)."""
    _check_inputs(q, kv, indices, kv_row_scale, page_table, page_size)
    shape = shape_for(q, kv, indices, page_table=page_table, page_size=page_size, nsplit=nsplit)
    dev = q.device
    o_shape, l_shape = _result_shapes(q)
    if out is None:
        out = torch.empty(o_shape, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(l_shape, dtype=torch.float32, device=dev)
    nplan = plan_nsplit(shape)
    ws_bytes = partials_size(q.shape[0] * _tokens(q), nplan) if nplan > 1 else 0
    if workspace is None and ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    n = ctypes.c_int32(0)
    st = lib.sparse_mla_decode_split(ctypes.byref(shape), _ptr(q), _ptr(kv), _ptr(kv_row_scale),
                                     _ptr(page_table), _ptr(indices), float(scale), _ptr(out),
                                     _ptr(lse), _ptr(workspace),
                                     0 if workspace is None else workspace.numel(), ctypes.byref(n),
                                     _stream(dev))
    if st != 0:
        raise SmlaError(st, "sparse_mla_decode_split")
    return n.value, out, lse, workspace


def partials_size(batch: int, nsplit: int) -> int:
    """Workspace bytes sparse_mla_decode_split needs to hold the partials of
    `nsplit` splits (fp32 O and lse), rounded up to 256."""
    b = batch * nsplit * H * (D_V + 1) * 4
    return (b + 255) // 256 * 256


def partial_views(workspace, batch: int, nsplit: int):
    """(partial_o [B, nsplit, 64, 512] fp32, partial_lse [B, nsplit, 64] fp32)
    views of a split workspace."""
    n_o = batch * nsplit * H * D_V
    f = workspace.view(torch.float32)
    return f[:n_o].view(batch, nsplit, H, D_V), f[n_o:n_o + batch * nsplit * H].view(batch, nsplit, H)


def combine(partial_o, partial_lse, out=None, lse=None):
    """out, lse = log-sum-exp combine of per-split partials (sparse_mla_combine)."""
    B, n, h, dv = partial_o.shape
    dev = partial_o.device
    if out is None:
        out = torch.empty((B, h, dv), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, h), dtype=torch.float32, device=dev)
    st = lib.sparse_mla_combine(B, h, dv, n, _ptr(partial_o), _ptr(partial_lse), _ptr(out), _ptr(lse),
                                _stream(dev))
    if st != 0:
        raise SmlaError(st, "sparse_mla_combine")
    return out, lse


def decode_stalled(q, kv, indices, scale: float, wait_limit_cycles: int, out=None, lse=None):
    """sparse_mla_decode_stalled (a test hook): launches the decode kernel
    on a flat bf16 cache with the score-MMA warp waiting on a barrier that
    nothing arrives on and every pipeline wait limited to
    ``wait_limit_cycles``.  Every wait runs out and the kernel sets the
    device error word's timeout bit; ``out`` and ``lse`` are left
    unwritten.  Returns (out, lse)."""
    _check_inputs(q, kv, indices, None, None, 0)
    shape = shape_for(q, kv, indices)
    dev = q.device
    o_shape, l_shape = _result_shapes(q)
    if out is None:
        out = torch.empty(o_shape, dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty(l_shape, dtype=torch.float32, device=dev)
    st = lib.sparse_mla_decode_stalled(ctypes.byref(shape), _ptr(q), _ptr(kv), _ptr(indices), float(scale),
                                       _ptr(out), _ptr(lse), int(wait_limit_cycles), _stream(dev))
    if st != 0:
        raise SmlaError(st, "sparse_mla_decode_stalled")
    return out, lse


def device_error() -> int:
    """Reads and clears the device error word (synchronous)."""
    code = ctypes.c_uint32(0)
    st = lib.sparse_mla_get_device_error(ctypes.byref(code))
    if st not in (0, 5, 6, 7):
        raise SmlaError(st, "sparse_mla_get_device_error")
    return code.value


class DecodePlan:
    """A decode call with its arguments marshalled once.

    For repeated calls on fixed buffers (serving loops, CUDA-graph capture,
    benchmarking): run() is a single call into the library with no
    per-call Python-side checks.  The tensors must stay alive and keep their
    addresses while the plan is in use.
    """

    def __init__(self, q, kv, indices, scale: float, *, kv_row_scale=None, page_table=None,
                 page_size: int = 0, nsplit: int = 0, out=None, lse=None, workspace=None):
        _check_inputs(q, kv, indices, kv_row_scale, page_table, page_size)
        self.shape = shape_for(q, kv, indices, page_table=page_table, page_size=page_size, nsplit=nsplit)
        dev = q.device
        self.nsplit = plan_nsplit(self.shape)
        self.merge = plan_merge(self.shape)
        # the splits merge inside the split kernel (one launch, no combine):
        # in a thread-block cluster, or (stream-K) by the last CTA of a row
        self.clustered = self.merge == 1
        self.streamk = self.merge == 3
        o_shape, l_shape = _result_shapes(q)
        self.out = out if out is not None else torch.empty(o_shape, dtype=torch.bfloat16, device=dev)
        self.lse = lse if lse is not None else torch.empty(l_shape, dtype=torch.float32, device=dev)
        ws = workspace_size(self.shape)
        self.workspace = workspace if workspace is not None or ws == 0 else \
            torch.empty(ws, dtype=torch.uint8, device=dev)
        self._keep = (q, kv, indices, kv_row_scale, page_table)
        wsp = _ptr(self.workspace)
        wsn = 0 if self.workspace is None else self.workspace.numel()
        self._stream = _stream(dev)
        self._args = (ctypes.byref(self.shape), _ptr(q), _ptr(kv), _ptr(kv_row_scale), _ptr(page_table),
                      _ptr(indices), float(scale), _ptr(self.out), _ptr(self.lse), wsp, wsn)
        self._split_args = self._args + (None,)
        if self.nsplit > 1 and not self.clustered:
            rows = q.shape[0] * _tokens(q)
            po, pl = partial_views(self.workspace, rows, self.nsplit)
            self._combine_args = (rows, H, D_V, self.nsplit, _ptr(po), _ptr(pl), _ptr(self.out),
                                  _ptr(self.lse))
        else:
            self._combine_args = None

    def run(self, stream=None):
        st = lib.sparse_mla_decode(*self._args, self._stream if stream is None else stream)
        if st != 0:
            raise SmlaError(st, "sparse_mla_decode")

    def run_split(self, stream=None):
        """The split kernel of run(): all of run() when the splits reduce on chip."""
        if self.clustered or self.streamk:
            return self.run(stream)
        st = lib.sparse_mla_decode_split(*self._split_args, self._stream if stream is None else stream)
        if st != 0:
            raise SmlaError(st, "sparse_mla_decode_split")

    def run_combine(self, stream=None):
        if self._combine_args is None:
            return
        st = lib.sparse_mla_combine(*self._combine_args, self._stream if stream is None else stream)
        if st != 0:
            raise SmlaError(st, "sparse_mla_combine")


# ------------------------------------------------- per-step tensors on the host
def host_staging_size(shape: SmlaShape) -> int:
    """Device staging bytes of sparse_mla_decode_host for ``shape``."""
    return lib.sparse_mla_host_staging_size(ctypes.byref(shape))


def _check_host_inputs(q_host, kv, indices_host, kv_row_scale, page_table_host, page_size, out_host, lse_host):
    dsv4 = is_dsv4(kv)
    d_qk = DSV4_D_QK if dsv4 else D_QK
    for name, t in (("q_host", q_host), ("indices_host", indices_host), ("page_table_host", page_table_host),
                    ("out_host", out_host), ("lse_host", lse_host)):
        if t is not None and (t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous host tensor")
    for name, t in (("kv", kv), ("kv_row_scale", kv_row_scale)):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if q_host.dtype != torch.bfloat16 or q_host.dim() not in (3, 4) or q_host.shape[-2:] != (H, d_qk):
        raise ValueError(f"q_host must be bf16 [B, 64, {d_qk}] or [B, T, 64, {d_qk}]")
    if (indices_host.dtype != torch.int32 or indices_host.dim() != q_host.dim() - 1
            or indices_host.shape[:-1] != q_host.shape[:-2]):
        raise ValueError("indices_host must be int32 [B, topk] ([B, T, topk] for q [B, T, 64, d])")
    if page_size and (page_table_host is None or page_table_host.dtype != torch.int32):
        raise ValueError("paged cache needs int32 page_table_host [B, pages_per_seq]")
    o_shape, l_shape = _result_shapes(q_host)
    if out_host.dtype != torch.bfloat16 or tuple(out_host.shape) != o_shape:
        raise ValueError("out_host must be bf16 [B, (T,) 64, 512]")
    if lse_host.dtype != torch.float32 or tuple(lse_host.shape) != l_shape:
        raise ValueError("lse_host must be float32 [B, (T,) 64]")


class HostDecodePlan:
    """sparse_mla_decode_host with its arguments marshalled once.

    q_host, indices_host (and page_table_host) are host tensors the caller
    refills between steps; out_host and lse_host receive each step's
    results.  Pinned host tensors make the copies asynchronous.  kv and
    kv_row_scale are device tensors.  run(stream) enqueues one step (copies
    in, decode, copies out) on ``stream`` (default: the current stream) and
    returns; the results are ready once that stream has reached it.  Plans
    used on different streams at the same time need their own staging,
    which each plan allocates unless one is given."""

    def __init__(self, q_host, kv, indices_host, scale: float, *, kv_row_scale=None, page_table_host=None,
                 page_size: int = 0, nsplit: int = 0, out_host=None, lse_host=None, staging=None):
        pin = q_host.is_pinned()
        o_shape, l_shape = _result_shapes(q_host)
        if out_host is None:
            out_host = torch.empty(o_shape, dtype=torch.bfloat16, pin_memory=pin)
        if lse_host is None:
            lse_host = torch.empty(l_shape, dtype=torch.float32, pin_memory=pin)
        _check_host_inputs(q_host, kv, indices_host, kv_row_scale, page_table_host, page_size, out_host,
                           lse_host)
        if is_dsv4(kv):
            if kv_row_scale is not None or page_size != 64:
                raise ValueError("DeepSeek-V4 pages: no kv_row_scale, page_size 64")
        elif (kv.dtype == torch.uint8) != (kv_row_scale is not None):
            raise ValueError("an fp8 cache needs kv_row_scale, a bf16 cache none")
        self.shape = shape_for(q_host, kv, indices_host, page_table=page_table_host, page_size=page_size,
                               nsplit=nsplit)
        need = host_staging_size(self.shape)
        if staging is None:
            staging = torch.empty(need, dtype=torch.uint8, device=kv.device)
        self.out_host, self.lse_host, self.staging = out_host, lse_host, staging
        self._keep = (q_host, kv, indices_host, kv_row_scale, page_table_host)
        self._device = kv.device
        self._args = (ctypes.byref(self.shape), _ptr(q_host), _ptr(kv), _ptr(kv_row_scale), _ptr(page_table_host),
                      _ptr(indices_host), float(scale), _ptr(out_host), _ptr(lse_host), _ptr(staging),
                      staging.numel())

    def run(self, stream=None):
        s = _stream(self._device) if stream is None else (stream.cuda_stream if hasattr(stream, "cuda_stream")
                                                          else stream)
        st = lib.sparse_mla_decode_host(*self._args, s)
        if st != 0:
            raise SmlaError(st, "sparse_mla_decode_host")


def decode_host(q_host, kv, indices_host, scale: float, *, kv_row_scale=None, page_table_host=None,
                page_size: int = 0, nsplit: int = 0, out_host=None, lse_host=None):
    """One decode step with the per-step tensors on the host: returns
    (out_host, lse_host) after synchronising the current stream."""
    plan = HostDecodePlan(q_host, kv, indices_host, scale, kv_row_scale=kv_row_scale,
                          page_table_host=page_table_host, page_size=page_size, nsplit=nsplit,
                          out_host=out_host, lse_host=lse_host)
    plan.run()
    torch.cuda.current_stream(kv.device).synchronize()
    return plan.out_host, plan.lse_host


# ------------------------------------------------------------------ indexer
def indexer_shape(batch: int, topk: int, max_ctx: int, pages_per_seq: int, num_key_rows: int) -> IndexerShape:
    return IndexerShape(batch, IX_HEADS, IX_DIM, topk, max_ctx, 64, pages_per_seq, 0, num_key_rows)


def _check_indexer(q, w, k_cache, page_table, ctx_len):
    for name, t in (("q", q), ("w", w), ("k_cache", k_cache), ("page_table", page_table), ("ctx_len", ctx_len)):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if q.dtype != torch.bfloat16 or q.dim() != 3 or q.shape[1:] != (IX_HEADS, IX_DIM):
        raise ValueError("q must be bf16 [B, 64, 128]")
    B = q.shape[0]
    if w.dtype != torch.float32 or tuple(w.shape) != (B, IX_HEADS):
        raise ValueError("w must be float32 [B, 64]")
    if k_cache.dtype != torch.bfloat16 or k_cache.dim() != 2 or k_cache.shape[1] != IX_DIM:
        raise ValueError("k_cache must be bf16 [rows, 128]")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be int32 [B, pages_per_seq]")
    if ctx_len.dtype != torch.int32 or tuple(ctx_len.shape) != (B,):
        raise ValueError("ctx_len must be int32 [B]")


class IndexerPlan:
    """The indexer step with its arguments marshalled once: scores
    ([B, max_ctx] fp32) and the top-k positions ([B, topk] int32) into
    buffers the plan owns (or the caller gives).  run() is one call into
    the library (two launches)."""

    def __init__(self, q, w, k_cache, page_table, ctx_len, topk: int, *, max_ctx: int | None = None,
                 scores=None, indices=None):
        _check_indexer(q, w, k_cache, page_table, ctx_len)
        B = q.shape[0]
        if max_ctx is None:
            max_ctx = page_table.shape[1] * 64
        self.shape = indexer_shape(B, topk, max_ctx, page_table.shape[1], k_cache.shape[0])
        dev = q.device
        self.scores = scores if scores is not None else torch.empty((B, max_ctx), dtype=torch.float32, device=dev)
        self.indices = indices if indices is not None else torch.empty((B, topk), dtype=torch.int32, device=dev)
        self._keep = (q, w, k_cache, page_table, ctx_len)
        self._stream = _stream(dev)
        self._args = (ctypes.byref(self.shape), _ptr(q), _ptr(w), _ptr(k_cache), _ptr(page_table), _ptr(ctx_len),
                      _ptr(self.scores), _ptr(self.indices))

    def run(self, stream=None):
        st = lib.sparse_mla_indexer(*self._args, self._stream if stream is None else stream)
        if st != 0:
            raise SmlaError(st, "sparse_mla_indexer")

    def run_scores(self, stream=None):
        st = lib.sparse_mla_indexer_scores(*self._args[:7], self._stream if stream is None else stream)
        if st != 0:
            raise SmlaError(st, "sparse_mla_indexer_scores")

    def run_topk(self, stream=None):
        st = lib.sparse_mla_indexer_topk(self._args[0], self._args[6], self._args[5], self._args[7],
                                         self._stream if stream is None else stream)
        if st != 0:
            raise SmlaError(st, "sparse_mla_indexer_topk")


def indexer(q, w, k_cache, page_table, ctx_len, topk: int, *, max_ctx: int | None = None):
    """One indexer step: returns (indices [B, topk] int32, scores [B, max_ctx]
    fp32), enqueued on the current stream."""
    plan = IndexerPlan(q, w, k_cache, page_table, ctx_len, topk, max_ctx=max_ctx)
    plan.run()
    return plan.indices, plan.scores


# ------------------------------------------- around the decode: common parts
def _check_device(dev, **tensors):
    """Every given tensor lies on the CUDA device ``dev``."""
    for name, t in tensors.items():
        if t is not None and (not t.is_cuda or t.device != dev):
            raise ValueError(f"{name} must be a CUDA tensor on {dev}")


def _check_tensor(name, t, dtype, shape):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")


# handle of a device's current stream, without building a Stream object for it
# (0.1 us instead of 2.2)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


class _Plan:
    """A call with its arguments marshalled once.  run() is one call into the
    library, on the current stream of the tensors' device unless a stream is
    given.  The tensors must stay alive and keep their addresses while the
    plan is in use; the plan holds references to them."""

    _call = None        # name of the entry point
    _empty = False      # nothing to do (no tokens)

    def _ready(self, dev, args, keep):
        self._device, self._args, self._keep = dev, args, keep
        self._fn = getattr(lib, self._call)

    def run(self, stream=None):
        if self._empty:
            return
        dev = self._device
        if stream is None:
            stream = _current_stream(dev.index)
        elif hasattr(stream, "cuda_stream"):
            stream = stream.cuda_stream
        if torch.cuda.current_device() == dev.index:
            st = self._fn(*self._args, stream)
        else:
            with torch.cuda.device(dev):
                st = self._fn(*self._args, stream)
        if st != 0:
            raise SmlaError(st, self._call)


def _cache_kind(kv):
    """smla_kv_dtype of a cache tensor, as decode() reads it."""
    if is_dsv4(kv):
        return KV_DSV4_PAGED
    if kv.dim() != 2 or kv.shape[1] != D_QK or kv.dtype not in (torch.bfloat16, torch.uint8):
        raise ValueError("kv must be [N, 576] bf16 or uint8 (fp8 e4m3fn codes), or uint8 [pages, 37376] "
                         "DeepSeek-V4 pages")
    return KV_FP8_E4M3_ROWSCALE if kv.dtype == torch.uint8 else KV_BF16


def _check_cache(kv, kv_row_scale):
    kind = _cache_kind(kv)
    if not kv.is_contiguous():
        raise ValueError("kv must be contiguous")
    if (kind == KV_FP8_E4M3_ROWSCALE) != (kv_row_scale is not None):
        raise ValueError("an fp8 cache needs kv_row_scale, the other caches none")
    if kv_row_scale is not None:
        _check_tensor("kv_row_scale", kv_row_scale, torch.float32, (kv.shape[0],))
    return kind


# ------------------------------------------------------------------ rotary
class RopeTable:
    """Frequencies of a rotary embedding over ``rope_dim`` dims, for rope()
    and cache_append().  ``interleaved``: pairs (2 i, 2 i + 1), else (i, i +
    rope_dim / 2).  ``scaling``: None, "linear" (positions divided by
    ``factor``) or "yarn" (``factor``, ``original_ctx``, ``beta_fast``,
    ``beta_slow``).  ``mscale`` multiplies cos and sin.  Host data only."""

    def __init__(self, rope_dim: int = 64, *, base: float = 10000.0, interleaved: bool = True,
                 scaling: str | None = None, factor: float = 1.0, original_ctx: int = 0, beta_fast: float = 32.0,
                 beta_slow: float = 1.0, mscale: float = 1.0):
        kinds = {None: 0, "linear": 1, "yarn": 2}
        if scaling not in kinds:
            raise ValueError('scaling must be None, "linear" or "yarn"')
        cfg = RopeConfig(rope_dim, 0 if interleaved else 1, kinds[scaling], original_ctx, base, factor, beta_fast,
                         beta_slow, mscale)
        self.data = RopeTableData()
        st = lib.sparse_mla_rope_init(ctypes.byref(cfg), ctypes.byref(self.data))
        if st != 0:
            raise SmlaError(st, "sparse_mla_rope_init")
        self.rope_dim, self.interleaved, self.mscale = rope_dim, interleaved, mscale

    def turns(self):
        """Fraction of a turn per position of each pair (float64)."""
        return [self.data.step[i] / 2.0 ** 64 for i in range(self.rope_dim // 2)]


def _token_stride(name, t):
    """Stride between tokens of a [..., heads, dim] tensor whose leading dims
    walk memory evenly."""
    lead, strides = t.shape[:-2], t.stride()[:-2]
    if not lead:
        return 0
    stride, size = None, 1
    for n, st in zip(reversed(lead), reversed(strides)):
        if n == 1:
            continue
        if stride is None:
            stride, size = st, n
        elif st != stride * size:
            raise ValueError(f"{name}: the token dims must be evenly strided")
        else:
            size *= n
    return 0 if stride is None else stride


class RopePlan(_Plan):
    """rope() with its arguments marshalled once; the result is ``out``."""

    _call = "sparse_mla_rope"

    def __init__(self, x, positions, table: RopeTable, *, offset: int | None = None, transpose: bool = False, out=None):
        if x.dim() < 2 or x.dtype not in DTYPES:
            raise ValueError("x must be [..., heads, dim] bf16, fp16 or fp32")
        heads, dim = x.shape[-2:]
        lead = tuple(x.shape[:-2])
        if offset is None:
            offset = dim - table.rope_dim
        if offset < 0 or offset + table.rope_dim > dim:
            raise ValueError("the rotated dims must lie inside the head")
        if positions.dtype != torch.int32 or tuple(positions.shape) != lead or not positions.is_contiguous():
            raise ValueError("positions must be contiguous int32 of x's leading shape")
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if out.dtype != x.dtype or out.shape != x.shape:
            raise ValueError("out must have x's shape and dtype")
        _check_device(x.device, x=x, positions=positions, out=out)
        for name, t in (("x", x), ("out", out)):
            if dim > 1 and t.stride(-1) != 1:
                raise ValueError(f"{name}: the dims of a head must be contiguous")
        self.out = out
        self._empty = x.numel() == 0
        self.shape = RopeShape(positions.numel(), heads, dim, offset, DTYPES[x.dtype], int(transpose), 0,
                               _token_stride("x", x), x.stride(-2), _token_stride("out", out), out.stride(-2))
        self._ready(x.device, (ctypes.byref(self.shape), ctypes.byref(table.data), _ptr(x), _ptr(positions), _ptr(out)),
                    (x, positions, table, out))


def rope(x, positions, table: RopeTable, *, offset: int | None = None, transpose: bool = False, out=None):
    """x [..., heads, dim] with dims [offset, offset + rope_dim) of every head
    (default: the last ones) turned by the token's position; positions
    [...] int32.  ``out`` may be x (in place), or a view such as the rotary
    part of a larger query.  ``transpose``: the gradient of the rotation with
    respect to x, given the gradient of its result (for mscale 1 also its
    inverse)."""
    plan = RopePlan(x, positions, table, offset=offset, transpose=transpose, out=out)
    plan.run()
    return plan.out


# ------------------------------------------------------------------ append
class CacheAppendPlan(_Plan):
    """cache_append() with its arguments marshalled once."""

    _call = "sparse_mla_cache_append"

    def __init__(self, x, kv, slots, *, kv_row_scale=None, page_table=None, page_size: int = 0, seq=None,
                 norm_weight=None, eps: float = 1e-6, rope: RopeTable | None = None, positions=None):
        kind = _check_cache(kv, kv_row_scale)
        width = D_V if kind == KV_DSV4_PAGED else D_QK
        if x.dim() != 2 or x.shape[1] != width or x.dtype not in DTYPES or x.stride(1) != 1:
            raise ValueError(f"x must be [tokens, {width}] bf16, fp16 or fp32 with contiguous rows")
        n = x.shape[0]
        _check_tensor("slots", slots, torch.int32, (n,))
        if (page_size != 0) != (page_table is not None):
            raise ValueError("page_size and page_table go together")
        if kind == KV_DSV4_PAGED and page_size != 64:
            raise ValueError("DeepSeek-V4 pages are paged: page_size must be 64")
        if page_table is not None and (page_table.dtype != torch.int32 or page_table.dim() != 2
                                       or not page_table.is_contiguous()):
            raise ValueError("page_table must be contiguous int32 [B, pages_per_seq]")
        if seq is not None:
            if page_table is None:
                raise ValueError("seq goes with a page_table")
            _check_tensor("seq", seq, torch.int32, (n,))
        if norm_weight is not None:
            _check_tensor("norm_weight", norm_weight, torch.float32, (D_V,))
        if (rope is None) != (positions is None):
            raise ValueError("rope and positions go together")
        if positions is not None:
            _check_tensor("positions", positions, torch.int32, (n,))
        _check_device(kv.device, x=x, kv=kv, slots=slots, kv_row_scale=kv_row_scale, page_table=page_table, seq=seq,
                      norm_weight=norm_weight, positions=positions)
        B, pps = (0, 0) if page_table is None else page_table.shape
        self.shape = AppendShape(n, x.stride(0) if n > 1 else width, kv.shape[0] * (64 if kind == KV_DSV4_PAGED else 1),
                                 DTYPES[x.dtype], kind, page_size, pps, B, eps, 0)
        self._ready(kv.device, (ctypes.byref(self.shape), _ptr(x), _ptr(norm_weight),
                                None if rope is None else ctypes.byref(rope.data), _ptr(positions), _ptr(slots),
                                _ptr(seq), _ptr(page_table), _ptr(kv), _ptr(kv_row_scale)),
                    (x, kv, slots, kv_row_scale, page_table, seq, norm_weight, rope, positions))


def cache_append(x, kv, slots, *, kv_row_scale=None, page_table=None, page_size: int = 0, seq=None, norm_weight=None,
                 eps: float = 1e-6, rope: RopeTable | None = None, positions=None):
    """Writes the rows x [n, 576] ([n, 512] for DeepSeek-V4 pages) of n new
    tokens into the cache ``kv``: RMS norm of the first 512 dims (with
    ``norm_weight`` [512] fp32), rotation of the last 64 by ``positions`` (with
    ``rope``, a 64-dim table), encoding in the cache's layout.  slots [n] int32:
    physical rows (flat pool), or logical positions of the token's sequence
    (paged); negative: skipped.  seq [n] int32 names the sequences; without
    it the tokens are equal runs, sequence by sequence."""
    CacheAppendPlan(x, kv, slots, kv_row_scale=kv_row_scale, page_table=page_table, page_size=page_size, seq=seq,
                    norm_weight=norm_weight, eps=eps, rope=rope, positions=positions).run()


# ------------------------------------------------------- attention weights
class AttentionWeightsPlan(_Plan):
    """attention_weights() with its arguments marshalled once; the result is
    ``out``."""

    _call = "sparse_mla_attn_weights"

    def __init__(self, q, kv, indices, lse, scale: float, *, kv_row_scale=None, page_table=None, page_size: int = 0,
                 out=None):
        _check_inputs(q, kv, indices, kv_row_scale, page_table, page_size)
        _check_cache(kv, kv_row_scale)
        _check_tensor("lse", lse, torch.float32, q.shape[:-1])
        if page_table is not None and (page_table.dim() != 2 or page_table.shape[0] != q.shape[0]):
            raise ValueError("page_table must be [B, pages_per_seq]")
        if out is None:
            out = torch.empty(indices.shape, dtype=torch.float32, device=q.device)
        _check_tensor("out", out, torch.float32, indices.shape)
        _check_device(q.device, q=q, kv=kv, indices=indices, lse=lse, kv_row_scale=kv_row_scale, page_table=page_table,
                      out=out)
        self.out = out
        self.shape = shape_for(q, kv, indices, page_table=page_table, page_size=page_size)
        self._ready(q.device, (ctypes.byref(self.shape), _ptr(q), _ptr(kv), _ptr(kv_row_scale),
                               _ptr(page_table) if page_size else None, _ptr(indices), _ptr(lse), float(scale),
                               _ptr(out)),
                    (q, kv, indices, lse, kv_row_scale, page_table, out))


def attention_weights(q, kv, indices, lse, scale: float, *, kv_row_scale=None, page_table=None, page_size: int = 0,
                      out=None):
    """The attention each listed row received in the decode that returned
    ``lse``, summed over the heads: float32 of indices' shape, 0 for padding.
    Arguments as for decode()."""
    plan = AttentionWeightsPlan(q, kv, indices, lse, scale, kv_row_scale=kv_row_scale, page_table=page_table,
                                page_size=page_size, out=out)
    plan.run()
    return plan.out


class AccumulateWeightsPlan(_Plan):
    """accumulate_weights() with its arguments marshalled once."""

    _call = "sparse_mla_accumulate_weights"

    def __init__(self, acc, indices, weights, *, decay: float = 1.0):
        if acc.dtype != torch.float32 or acc.dim() != 2 or not acc.is_contiguous():
            raise ValueError("acc must be contiguous float32 [B, max_ctx]")
        B, max_ctx = acc.shape
        if indices.dtype != torch.int32 or indices.dim() not in (2, 3) or indices.shape[0] != B \
                or not indices.is_contiguous():
            raise ValueError("indices must be contiguous int32 [B, topk] or [B, T, topk]")
        _check_tensor("weights", weights, torch.float32, indices.shape)
        _check_device(acc.device, acc=acc, indices=indices, weights=weights)
        self._ready(acc.device, (B, indices.numel() // max(B, 1), max_ctx, _ptr(indices), _ptr(weights), float(decay),
                                 _ptr(acc)), (acc, indices, weights))


def accumulate_weights(acc, indices, weights, *, decay: float = 1.0):
    """acc [B, max_ctx] float32 = decay * acc + the weights summed onto their
    logical positions: indices and weights [B, topk] or [B, T, topk].  A
    position may be listed any number of times; the result does not depend
    on the order.  Returns acc."""
    AccumulateWeightsPlan(acc, indices, weights, decay=decay).run()
    return acc


# ---------------------------------------------------------------- eviction
class EvictPlan(_Plan):
    """evict() with its arguments marshalled once; the results are ``kept``,
    ``new_len`` and ``acc_out``."""

    _call = "sparse_mla_evict"

    def __init__(self, acc, ctx_len, budget: int, *, page_table, kv, kv_row_scale=None, k_cache=None, sinks: int = 0,
                 recent: int = 0, new_page_table=None, kept=None, new_len=None, acc_out=None):
        kind = _check_cache(kv, kv_row_scale)
        if acc.dtype != torch.float32 or acc.dim() != 2 or not acc.is_contiguous():
            raise ValueError("acc must be contiguous float32 [B, max_ctx]")
        B, max_ctx = acc.shape
        dev = acc.device
        for name, t in (("page_table", page_table), ("new_page_table", new_page_table)):
            if t is not None and (t.dtype != torch.int32 or t.dim() != 2 or t.shape[0] != B or not t.is_contiguous()):
                raise ValueError(f"{name} must be contiguous int32 [B, pages_per_seq]")
        if k_cache is not None and (k_cache.dtype != torch.bfloat16 or k_cache.dim() != 2
                                    or k_cache.shape[1] != IX_DIM or not k_cache.is_contiguous()):
            raise ValueError("k_cache must be contiguous bf16 [rows, 128]")
        if kept is None:
            kept = torch.empty((B, max(budget, 0)), dtype=torch.int32, device=dev)
        if new_len is None:
            new_len = torch.empty_like(ctx_len)
        if acc_out is None:
            acc_out = acc
        _check_tensor("ctx_len", ctx_len, torch.int32, (B,))
        _check_tensor("new_len", new_len, torch.int32, (B,))
        _check_tensor("kept", kept, torch.int32, (B, budget))
        _check_tensor("acc_out", acc_out, torch.float32, (B, max_ctx))
        _check_device(dev, acc=acc, ctx_len=ctx_len, page_table=page_table, kv=kv, kv_row_scale=kv_row_scale,
                      k_cache=k_cache, new_page_table=new_page_table, kept=kept, new_len=new_len, acc_out=acc_out)
        self.kept, self.new_len, self.acc_out = kept, new_len, acc_out
        self.shape = EvictShape(B, max_ctx, budget, sinks, recent, kind, page_table.shape[1],
                                0 if new_page_table is None else new_page_table.shape[1],
                                kv.shape[0] * (64 if kind == KV_DSV4_PAGED else 1),
                                0 if k_cache is None else k_cache.shape[0])
        self._ready(dev, (ctypes.byref(self.shape), _ptr(acc), _ptr(ctx_len), _ptr(kept), _ptr(new_len), _ptr(acc_out),
                          _ptr(page_table), _ptr(new_page_table), _ptr(kv), _ptr(kv_row_scale), _ptr(k_cache)),
                    (acc, ctx_len, page_table, kv, kv_row_scale, k_cache, new_page_table, kept, new_len, acc_out))


def evict(acc, ctx_len, budget: int, *, page_table, kv, kv_row_scale=None, k_cache=None, sinks: int = 0,
          recent: int = 0, new_page_table=None, kept=None, new_len=None, acc_out=None):
    """Keeps at most ``budget`` positions of each sequence -- the first
    ``sinks``, the last ``recent`` and those with the largest acc [B, max_ctx] --
    and compacts the paged caches (kv, kv_row_scale, k_cache) to them, in place
    or into the pages of ``new_page_table``.  Returns (kept [B, budget] int32,
    -1 after the last, new_len [B] int32, acc_out), acc_out being acc unless
    given; new_len may be given as ctx_len."""
    plan = EvictPlan(acc, ctx_len, budget, page_table=page_table, kv=kv, kv_row_scale=kv_row_scale, k_cache=k_cache,
                     sinks=sinks, recent=recent, new_page_table=new_page_table, kept=kept, new_len=new_len,
                     acc_out=acc_out)
    plan.run()
    return plan.kept, plan.new_len, plan.acc_out
