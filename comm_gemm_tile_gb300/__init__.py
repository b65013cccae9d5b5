"""Python binding of libmk.so: tile-pipelined fused collective + GEMM on one GB300.

Argument marshalling only.  Every step of every op runs in the CUDA library
(include/mk.h); PyTorch provides device memory and streams.  If the library is
missing the calls raise -- there is no fallback path.

The R virtual ranks of an op are R separate device buffers on one GPU.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import dataclasses
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmk.so")

MK_OK, MK_ERR_INVALID, MK_ERR_UNSUPPORTED, MK_ERR_CUDA, MK_ERR_TIMEOUT, MK_ERR_CAPACITY = range(6)
MK_BF16, MK_F32, MK_F16, MK_E4M3 = 0, 1, 2, 3
OP_AG_GEMM, OP_GEMM_RS, OP_GEMM_AR, OP_MOE = 0, 1, 2, 3
MODE_FUSED, MODE_GEMM_ONLY, MODE_UNFUSED = 0, 1, 2
REDUCE_AUTO, REDUCE_RUNNING_SUM, REDUCE_LAST_ARRIVAL, REDUCE_ATOMIC, REDUCE_SLICED = 0, 1, 2, 3, 4
WIRE_F32, WIRE_BF16 = 0, 1
OPERAND_BF16, OPERAND_FP8 = 0, 1
FP8 = torch.float8_e4m3fn
# columns of trace_records()
(TRACE_START, TRACE_INPUTS, TRACE_ISSUED, TRACE_READY, TRACE_END, TRACE_CLK_START,
 TRACE_CLK_READY, TRACE_ID) = range(8)
TRACE_WORDS = 8
TRACE_COPY_RECORDS = 1024


def _with_operand(cfg, t):
    """The config for operands of t's dtype: fp8 e4m3 tensors set operand = 1."""
    if t.dtype != FP8:
        return cfg
    c = dataclasses.replace(cfg) if cfg is not None else Config()
    c.operand = OPERAND_FP8
    return c
PAIR_AUTO, PAIR_OFF, PAIR_ON = 0, 1, 2
MAX_RANKS = 16


class MkError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


class _Cfg(ctypes.Structure):
    _fields_ = [("n_copy_ctas", ctypes.c_int), ("n_reduce_ctas", ctypes.c_int),
                ("max_ctas", ctypes.c_int), ("group_m", ctypes.c_int), ("split_k", ctypes.c_int),
                ("mode", ctypes.c_int), ("wait_limit_ns", ctypes.c_longlong),
                ("inject", ctypes.c_int), ("reduce", ctypes.c_int), ("cta_pair", ctypes.c_int),
                ("wire", ctypes.c_int), ("operand", ctypes.c_int), ("trace", ctypes.c_int)]


@dataclasses.dataclass
class Config:
    """Tuning / test knobs (mk_config); 0 means the library's own choice."""
    n_copy_ctas: int = 0
    n_reduce_ctas: int = 0
    max_ctas: int = 0
    group_m: int = 0
    split_k: int = 0
    mode: int = MODE_FUSED
    wait_limit_ns: int = 0
    inject: int = 0
    reduce: int = 0
    cta_pair: int = 0
    wire: int = 0
    operand: int = 0
    trace: int = 0

    def c(self) -> _Cfg:
        return _Cfg(self.n_copy_ctas, self.n_reduce_ctas, self.max_ctas, self.group_m,
                    self.split_k, self.mode, self.wait_limit_ns, self.inject, self.reduce,
                    self.cta_pair, self.wire, self.operand, self.trace)


_lib = None
_lib_lock = threading.Lock()


LIB_DEBUG_PATH = os.path.join(_HERE, "libmk_debug.so")


def lib() -> ctypes.CDLL:
    """Load libmk.so (built in-tree by build.py).  Raises if it is missing."""
    global _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        _lib = load_library(LIB_PATH)
        return _lib


class _Rotation(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("start", ctypes.c_longlong),
                ("positions_64", ctypes.c_int), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("inverse", ctypes.c_int), ("magnitude", ctypes.c_float)]


class _Seqs(ctypes.Structure):
    _fields_ = [("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("pages", ctypes.c_void_p),
                ("pages_stride", ctypes.c_longlong), ("batch", ctypes.c_int), ("max_pages", ctypes.c_int)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong), ("slot_stride", ctypes.c_longlong),
                ("n_pages", ctypes.c_longlong), ("dtype", ctypes.c_int), ("heads", ctypes.c_int),
                ("d", ctypes.c_int), ("page_size", ctypes.c_int)]


class _Rows(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("token", ctypes.c_longlong), ("head", ctypes.c_longlong)]


class _W4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
                ("n", ctypes.c_longlong), ("k", ctypes.c_longlong), ("group", ctypes.c_int), ("dtype", ctypes.c_int)]


class use_library:
    """Context manager: every op of this module calls the given library (for
    example the bounds-checking LIB_DEBUG_PATH) instead of libmk.so."""

    def __init__(self, path: str):
        self.path = path

    def __enter__(self):
        global _lib
        self.prev = lib()
        with _lib_lock:
            _lib = load_library(self.path)
        return _lib

    def __exit__(self, *exc):
        global _lib
        with _lib_lock:
            _lib = self.prev
        return False


def load_library(path: str) -> ctypes.CDLL:
    """Open a build of the library and declare its C ABI."""
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run comm_gemm_tile_gb300/build.py "
                           "(or __graft_entry__.build())")
    L = ctypes.CDLL(path)
    vp, sz, ll, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_longlong, ctypes.c_int
    P = ctypes.POINTER
    L.mk_version.restype = i
    L.mk_device_sm_count.restype = i
    L.mk_status_string.restype = ctypes.c_char_p
    L.mk_status_string.argtypes = [i]
    L.mk_workspace_size.restype = sz
    L.mk_workspace_size.argtypes = [i, i, ll, ll, ll, P(_Cfg)]
    L.mk_trace_entries.restype = sz
    L.mk_trace_entries.argtypes = [i, i, ll, ll, ll, P(_Cfg), P(sz)]
    L.mk_moe_trace_entries.restype = sz
    L.mk_moe_trace_entries.argtypes = [i, i, i, ll, ll, ll, ll, P(_Cfg), P(sz)]
    L.mk_mlp_trace_entries.restype = sz
    L.mk_mlp_trace_entries.argtypes = [i, ll, ll, ll, P(_Cfg), P(sz)]
    L.mk_moe_workspace_size.restype = sz
    L.mk_moe_workspace_size.argtypes = [i, i, i, ll, ll, ll, ll, P(_Cfg)]
    L.mk_get_device_status.restype = i
    L.mk_get_device_status.argtypes = [vp, vp, P(ll)]
    L.mk_ag_gemm.restype = i
    L.mk_ag_gemm.argtypes = [P(vp), vp, vp, vp, i, i, i, ll, ll, ll, vp, sz, P(_Cfg), vp]
    for name in ("mk_gemm_rs", "mk_gemm_ar"):
        f = getattr(L, name)
        f.restype = i
        f.argtypes = [P(vp), P(vp), P(vp), i, i, ll, ll, ll, vp, sz, P(_Cfg), vp]
    L.mk_ag_gemm_noalloc.restype = i
    L.mk_ag_gemm_noalloc.argtypes = [P(vp), vp, vp, vp, i, i, i, ll, ll, ll, vp, P(_Cfg), vp]
    L.mk_moe_combine_workspace_size.restype = sz
    L.mk_moe_combine_workspace_size.argtypes = [i, i, i, ll, ll, ll, ll, P(_Cfg)]
    L.mk_moe_combine.restype = i
    L.mk_moe_combine.argtypes = [P(vp), P(vp), P(vp), P(vp), vp, i, i, i, ll, ll, ll, ll,
                                 P(vp), P(vp), vp, sz, P(_Cfg), vp]
    L.mk_mlp_workspace_size.restype = sz
    L.mk_mlp_workspace_size.argtypes = [i, ll, ll, ll, P(_Cfg)]
    L.mk_mlp_ag_rs.restype = i
    L.mk_mlp_ag_rs.argtypes = [P(vp), P(vp), P(vp), i, ll, ll, ll, vp, P(vp), P(vp), vp, sz,
                               P(_Cfg), vp]
    L.mk_ring_attention_workspace_size.restype = sz
    L.mk_ring_attention_workspace_size.argtypes = [i, i, ll, i, i, P(_Cfg)]
    L.mk_ring_attention.restype = i
    L.mk_ring_attention.argtypes = [P(vp), P(vp), P(vp), i, i, ll, i, i, ctypes.c_float, P(vp),
                                    P(vp), P(vp), vp, sz, P(_Cfg), vp]
    L.mk_moe_dispatch_gemm.restype = i
    L.mk_moe_dispatch_gemm.argtypes = [P(vp), P(vp), P(vp), i, i, i, ll, ll, ll, ll, vp, vp,
                                       P(vp), vp, P(vp), P(vp), vp, sz, P(_Cfg), vp]
    f32 = ctypes.c_float
    L.mk_rope.restype = i
    L.mk_rope.argtypes = [vp, vp, i, ll, i, i, ll, ll, ll, ll, P(_Rotation), vp]
    L.mk_kv_append.restype = i
    L.mk_kv_append.argtypes = [P(_Cache), vp, vp, i, ll, ll, ll, ll, ll, vp, vp, i, ll, ll, ll, ll, P(_Seqs),
                               P(_Rotation), vp, sz, vp]
    L.mk_paged_attention_workspace_size.restype = sz
    L.mk_paged_attention_workspace_size.argtypes = [ll, i, i, i, i]
    L.mk_paged_attention.restype = i
    L.mk_paged_attention.argtypes = [vp, vp, vp, i, ll, i, ll, ll, ll, ll, P(_Cache), P(_Seqs), f32, i, i, i, i,
                                     vp, sz, P(_Cfg), vp]
    rows = P(_Rows)
    L.mk_rms_norm.restype = i
    L.mk_rms_norm.argtypes = [rows, rows, vp, rows, rows, vp, i, i, i, ll, i, i, f32, vp]
    L.mk_rms_norm_backward_workspace_size.restype = sz
    L.mk_rms_norm_backward_workspace_size.argtypes = [ll, i, i]
    L.mk_rms_norm_backward.restype = i
    L.mk_rms_norm_backward.argtypes = [rows, rows, rows, vp, rows, vp, i, i, ll, i, i, f32, vp, sz, vp]
    L.mk_moe_route_workspace_size.restype = sz
    L.mk_moe_route_workspace_size.argtypes = [ll, i]
    L.mk_moe_route.restype = i
    L.mk_moe_route.argtypes = [vp, i, ll, i, ll, i, i, f32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.mk_moe_route_backward.restype = i
    L.mk_moe_route_backward.argtypes = [vp, i, ll, i, ll, i, i, f32, vp, vp, vp, vp, vp, vp, vp, ll, vp]
    L.mk_w4_gemm_scratch_size.restype = sz
    L.mk_w4_gemm_scratch_size.argtypes = [P(_W4), ll]
    L.mk_w4_gemm.restype = i
    L.mk_w4_gemm.argtypes = [vp, ll, P(_W4), vp, ll, i, i, ll, vp, sz, vp, sz, P(_Cfg), vp]
    return L


def status_string(s: int) -> str:
    return lib().mk_status_string(int(s)).decode()


def _ptrs(ts) -> ctypes.Array:
    arr = (ctypes.c_void_p * len(ts))()
    for j, t in enumerate(ts):
        arr[j] = t.data_ptr() if isinstance(t, torch.Tensor) else t
    return arr


def _cfgp(cfg: Config | None):
    return ctypes.byref(cfg.c()) if cfg is not None else None


def _stream(stream, device) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dt(dtype) -> int:
    if dtype == torch.bfloat16:
        return MK_BF16
    if dtype == torch.float32:
        return MK_F32
    raise ValueError(f"unsupported output dtype {dtype}")


def _check(st: int, what: str):
    if st != MK_OK:
        raise MkError(st, what)


# ------------------------------------------------------------------ workspaces

class Workspace:
    """A device workspace, zero-filled once at (re)allocation as the library requires, before any stream uses
    it.  A buffer stays allocated when a larger one takes its place, since calls in flight on any stream and
    graphs keep its address; buffers at least double, so that those kept are no more than the last.  A buffer made
    while capturing is filled by every captured call that uses it, until a call outside has filled it: graphs may be
    replayed in any order.  Calls whose scratch holds nothing from one call to the next (moe_route,
    rms_norm_backward) have a buffer apart, so that they leave the others' flags and status alone."""

    def __init__(self, device=None):
        self.device = torch.device(device or "cuda")
        self.buf = None
        self.apart = None          # the Workspace of scratch
        self.kept = []             # outgrown buffers
        self.filled = True         # False: allocated while capturing, so that only a replay would fill it

    def get(self, nbytes: int, stream=None) -> torch.Tensor:
        """A buffer of at least nbytes for a call on the given stream (None: the current one)."""
        nbytes = max(int(nbytes), 256)
        large = self.buf is not None and self.buf.numel() >= nbytes
        if large and self.filled:
            return self.buf
        capturing = torch._C._cuda_isCurrentStreamCapturing()
        with contextlib.nullcontext() if stream is None else _on(stream, self.device):
            capturing = capturing or torch._C._cuda_isCurrentStreamCapturing()
            if large:
                self.buf.zero_()
            else:
                if self.buf is not None:
                    self.kept.append(self.buf)
                    nbytes = max(nbytes, 2 * self.buf.numel())
                self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
            self.filled = not capturing
            if not capturing:
                torch.cuda.current_stream(self.device).synchronize()
        return self.buf

    def scratch(self, nbytes: int, stream=None) -> torch.Tensor:
        """Memory that no other operator's call expects to find as it left it."""
        if self.apart is None:
            self.apart = Workspace(self.device)
        return self.apart.get(nbytes, stream)


_default_ws: dict = {}
_default_paged_ws: dict = {}   # paged attention's partial results must not meet the other ops' ready flags


def _ws(workspace, device, default=_default_ws) -> Workspace:
    if workspace is not None:
        return workspace
    key = torch.device(device).index if torch.device(device).index is not None else \
        torch.cuda.current_device()
    if key not in default:
        default[key] = Workspace(torch.device("cuda", key))
    return default[key]


def workspace_size(op: int, R: int, m: int, n: int, k: int, cfg: Config | None = None) -> int:
    return int(lib().mk_workspace_size(op, R, m, n, k, _cfgp(cfg)))


def device_status(workspace: Workspace | None = None, stream=None, device=None):
    """Synchronise the stream and read-and-clear the workspace's device status.
    Returns (status, detail).  Without a workspace: that of the device's default
    workspaces (paged attention has one of its own)."""
    ws = _ws(workspace, device or "cuda")
    spaces = [ws]
    if workspace is None and ws.device.index in _default_paged_ws:
        spaces.append(_default_paged_ws[ws.device.index])
    first = (MK_OK, 0)
    for w in spaces:
        detail = ctypes.c_longlong(0)
        st = lib().mk_get_device_status(ctypes.c_void_p(w.get(256, stream).data_ptr()),
                                        ctypes.c_void_p(_stream(stream, w.device)), ctypes.byref(detail))
        if first[0] == MK_OK:
            first = (int(st), int(detail.value))
    return first


# ------------------------------------------------------------------ ops

def ag_gemm(a_shards, b, *, local_rank: int = 0, out_dtype=torch.bfloat16, a_gathered=None,
            c=None, cfg: Config | None = None, workspace: Workspace | None = None, stream=None):
    """AllGather + GEMM: returns (a_gathered = [A_0; ...; A_{R-1}], c = a_gathered @ b).
    With fp8 e4m3 operands b is B^T ([n x k]) and c = a_gathered @ b.T."""
    R = len(a_shards)
    m_r, k = a_shards[0].shape
    cfg = _with_operand(cfg, a_shards[0])
    n = b.shape[0] if a_shards[0].dtype == FP8 else b.shape[1]
    dev = b.device
    if a_gathered is None:
        a_gathered = torch.empty((R * m_r, k), dtype=a_shards[0].dtype, device=dev)
    if c is None:
        c = torch.empty((R * m_r, n), dtype=out_dtype, device=dev)
    ws = _ws(workspace, dev)
    nb = workspace_size(OP_AG_GEMM, R, m_r, n, k, cfg)
    if nb == 0:
        raise MkError(MK_ERR_INVALID, "mk_workspace_size(AG)")
    buf = ws.get(nb, stream)
    st = lib().mk_ag_gemm(_ptrs(a_shards), b.data_ptr(), a_gathered.data_ptr(), c.data_ptr(),
                          _dt(c.dtype), R, local_rank, m_r, n, k, buf.data_ptr(), buf.numel(),
                          _cfgp(cfg), _stream(stream, dev))
    _check(st, "mk_ag_gemm")
    return a_gathered, c


def _rs_ar(fn, op, a, b, outs, R, m, n, k, cfg, workspace, stream, what):
    dev = a[0].device
    ws = _ws(workspace, dev)
    nb = workspace_size(op, R, m, n, k, cfg)
    if nb == 0:
        raise MkError(MK_ERR_INVALID, f"mk_workspace_size({what})")
    buf = ws.get(nb, stream)
    st = fn(_ptrs(a), _ptrs(b), _ptrs(outs), _dt(outs[0].dtype), R, m, n, k, buf.data_ptr(),
            buf.numel(), _cfgp(cfg), _stream(stream, dev))
    _check(st, what)
    return outs


def gemm_rs(a, b, *, out_dtype=torch.bfloat16, c_blocks=None, cfg: Config | None = None,
            workspace: Workspace | None = None, stream=None):
    """GEMM + ReduceScatter: S = sum_r a[r] @ b[r]; returns R row blocks of S.
    With fp8 e4m3 operands b[r] is B_r^T ([n x k]) and S = sum_r a[r] @ b[r].T."""
    R = len(a)
    m, k = a[0].shape
    cfg = _with_operand(cfg, a[0])
    n = b[0].shape[0] if a[0].dtype == FP8 else b[0].shape[1]
    if c_blocks is None:
        c_blocks = [torch.empty((m // R, n), dtype=out_dtype, device=a[0].device) for _ in range(R)]
    return _rs_ar(lib().mk_gemm_rs, OP_GEMM_RS, a, b, c_blocks, R, m, n, k, cfg, workspace, stream,
                  "mk_gemm_rs")


def gemm_ar(a, b, *, out_dtype=torch.bfloat16, c_replicas=None, cfg: Config | None = None,
            workspace: Workspace | None = None, stream=None):
    """GEMM + AllReduce: S = sum_r a[r] @ b[r]; returns R identical replicas of S.
    With fp8 e4m3 operands b[r] is B_r^T ([n x k]) and S = sum_r a[r] @ b[r].T."""
    R = len(a)
    m, k = a[0].shape
    cfg = _with_operand(cfg, a[0])
    n = b[0].shape[0] if a[0].dtype == FP8 else b[0].shape[1]
    if c_replicas is None:
        c_replicas = [torch.empty((m, n), dtype=out_dtype, device=a[0].device) for _ in range(R)]
    return _rs_ar(lib().mk_gemm_ar, OP_GEMM_AR, a, b, c_replicas, R, m, n, k, cfg, workspace,
                  stream, "mk_gemm_ar")


def trace_records(workspace: Workspace, op: int, R, m, n, k, cfg: Config):
    """The in-kernel trace of the last AG / RS / AR call made on `workspace` with
    cfg.trace = 1 and these arguments (m = rows per shard for AG, as for
    workspace_size): an int64 tensor [records x 8], record 2*i + c for work item i
    on the CTA of pair rank c.  Columns (TRACE_* below): ns stamps when the
    producer takes the item, its inputs are ready, its last load is issued, the
    accumulator is ready, the epilogue is done; the SM's clock64 at the first and
    fourth stamps; epoch << 32 | CTA << 1 | pair rank.  Records the call did not
    write keep older contents (another epoch) or zeros."""
    off = ctypes.c_size_t(0)
    n_rec = int(lib().mk_trace_entries(op, R, m, n, k, _cfgp(cfg), ctypes.byref(off)))
    if n_rec == 0:
        return torch.zeros((0, TRACE_WORDS), dtype=torch.int64)
    nb = n_rec * TRACE_WORDS * 8
    buf = workspace.get(int(off.value) + nb)
    raw = buf[int(off.value):int(off.value) + nb]
    return raw.view(torch.int64).view(n_rec, TRACE_WORDS).cpu()


def trace_copy_records(workspace: Workspace, op: int, R, m, n, k, cfg: Config):
    """The copy-warp records that follow the item records: int64 [TRACE_COPY_RECORDS x 8],
    record w for copy worker w: start ns, end ns, pieces, bytes, 0, 0, 0,
    epoch << 32 | w.  Only an AllGather copy-in by copy warps writes them."""
    off = ctypes.c_size_t(0)
    n_rec = int(lib().mk_trace_entries(op, R, m, n, k, _cfgp(cfg), ctypes.byref(off)))
    if n_rec == 0:
        return torch.zeros((0, TRACE_WORDS), dtype=torch.int64)
    o = int(off.value) + n_rec * TRACE_WORDS * 8
    nb = TRACE_COPY_RECORDS * TRACE_WORDS * 8
    buf = workspace.get(o + nb)
    return buf[o:o + nb].view(torch.int64).view(TRACE_COPY_RECORDS, TRACE_WORDS).cpu()


def moe_trace_records(workspace: Workspace, R, E_loc, topk, T, H, N, cap_rows, cfg: Config):
    """The in-kernel trace of the last MoE dispatch + grouped GEMM call made on
    `workspace` with cfg.trace = 1 and these arguments (cap_rows as the call used it):
    (item records [2 x tile-table entries x 8], the reserved copy-warp records), int64,
    with the words of trace_records.  The dispatch copy writes no copy-warp records."""
    off = ctypes.c_size_t(0)
    n_rec = int(lib().mk_moe_trace_entries(R, E_loc, topk, T, H, N, cap_rows, _cfgp(cfg),
                                           ctypes.byref(off)))
    if n_rec == 0:
        z = torch.zeros((0, TRACE_WORDS), dtype=torch.int64)
        return z, z
    o = int(off.value)
    nb = (n_rec + TRACE_COPY_RECORDS) * TRACE_WORDS * 8
    raw = workspace.get(o + nb)[o:o + nb].view(torch.int64).view(-1, TRACE_WORDS).cpu()
    return raw[:n_rec], raw[n_rec:]


def mlp_trace_records(workspace: Workspace, R, m, h, f_r, cfg: Config):
    """The in-kernel trace of the last chained MLP call made on `workspace` with
    cfg.trace = 1 and these arguments: (item records, copy-warp records), int64 with
    the words of trace_records; item i < R * row tiles * f_r column tiles is an
    up-projection tile, the rest are down-projection items."""
    off = ctypes.c_size_t(0)
    n_rec = int(lib().mk_mlp_trace_entries(R, m, h, f_r, _cfgp(cfg), ctypes.byref(off)))
    if n_rec == 0:
        z = torch.zeros((0, TRACE_WORDS), dtype=torch.int64)
        return z, z
    o = int(off.value)
    nb = (n_rec + TRACE_COPY_RECORDS) * TRACE_WORDS * 8
    raw = workspace.get(o + nb)[o:o + nb].view(torch.int64).view(-1, TRACE_WORDS).cpu()
    return raw[:n_rec], raw[n_rec:]


def moe_workspace_size(R, E_loc, topk, T, H, N, cap_rows, cfg: Config | None = None) -> int:
    return int(lib().mk_moe_workspace_size(R, E_loc, topk, T, H, N, cap_rows, _cfgp(cfg)))


def moe_dispatch_gemm(x, logits, w, *, E_loc: int, topk: int = 2, cap_rows: int | None = None,
                      out=None, cfg: Config | None = None, workspace: Workspace | None = None,
                      stream=None):
    """MoE dispatch + grouped GEMM over R virtual ranks.

    x[r]: [T x H] bf16 tokens; logits[r]: [T x E] fp32 (E = R*E_loc); w[d]: [E_loc x H x N] bf16.
    Returns a dict with topk_idx [R*T x topk], counts [R x E], recv_src[d] [cap],
    recv_counts [R] (int32) and recv_x[d] [cap x H], y[d] [cap x N] (bf16); rows of rank d
    past recv_counts[d] are left as they were.  `out` may pass preallocated buffers.
    """
    R = len(x)
    T, H = x[0].shape
    N = w[0].shape[2]
    E = R * E_loc
    cap = cap_rows if cap_rows is not None else R * T * topk
    dev = x[0].device
    o = dict(out or {})
    i32 = torch.int32
    o.setdefault("topk_idx", torch.empty((R * T, topk), dtype=i32, device=dev))
    o.setdefault("counts", torch.empty((R, E), dtype=i32, device=dev))
    o.setdefault("recv_counts", torch.empty((R,), dtype=i32, device=dev))
    o.setdefault("recv_src", [torch.empty((cap,), dtype=i32, device=dev) for _ in range(R)])
    o.setdefault("recv_x", [torch.empty((cap, H), dtype=torch.bfloat16, device=dev) for _ in range(R)])
    o.setdefault("y", [torch.empty((cap, N), dtype=torch.bfloat16, device=dev) for _ in range(R)])
    ws = _ws(workspace, dev)
    nb = moe_workspace_size(R, E_loc, topk, T, H, N, cap, cfg)
    if nb == 0:
        raise MkError(MK_ERR_INVALID, "mk_moe_workspace_size")
    buf = ws.get(nb, stream)
    st = lib().mk_moe_dispatch_gemm(_ptrs(x), _ptrs(logits), _ptrs(w), R, E_loc, topk, T, H, N, cap,
                                    o["topk_idx"].data_ptr(), o["counts"].data_ptr(),
                                    _ptrs(o["recv_src"]), o["recv_counts"].data_ptr(),
                                    _ptrs(o["recv_x"]), _ptrs(o["y"]), buf.data_ptr(), buf.numel(),
                                    _cfgp(cfg), _stream(stream, dev))
    _check(st, "mk_moe_dispatch_gemm")
    return o


def moe_combine_workspace_size(R, E_loc, topk, T, N, H, cap_rows, cfg: Config | None = None) -> int:
    return int(lib().mk_moe_combine_workspace_size(R, E_loc, topk, T, N, H, cap_rows, _cfgp(cfg)))


def moe_combine(h, w2, gates, recv_src, counts, *, E_loc: int, topk: int = 2,
                cap_rows: int | None = None, out=None, cfg: Config | None = None,
                workspace: Workspace | None = None, stream=None):
    """MoE combine over R virtual ranks: down-projection of every expert's rows,
    return of the rows to their source ranks, gate-weighted sum over the top-k.

    h[d]: [cap x N] bf16 expert hidden rows in dispatch order; w2[d]: [E_loc x N x H] bf16;
    gates[r]: [T x topk] fp32; recv_src[d]: [cap] int32 and counts: [R x E] int32 from the
    dispatch.  Returns a dict with ret[r] [T x topk x H] (the returned expert rows) and
    out[r] [T x H] (bf16).  `out` may pass preallocated buffers.
    """
    R = len(h)
    cap = cap_rows if cap_rows is not None else h[0].shape[0]
    N = h[0].shape[1]
    H = w2[0].shape[2]
    T = gates[0].shape[0]
    dev = h[0].device
    o = dict(out or {})
    o.setdefault("ret", [torch.empty((T, topk, H), dtype=torch.bfloat16, device=dev) for _ in range(R)])
    o.setdefault("out", [torch.empty((T, H), dtype=torch.bfloat16, device=dev) for _ in range(R)])
    ws = _ws(workspace, dev)
    nb = moe_combine_workspace_size(R, E_loc, topk, T, N, H, cap, cfg)
    if nb == 0:
        raise MkError(MK_ERR_INVALID, "mk_moe_combine_workspace_size")
    buf = ws.get(nb, stream)
    st = lib().mk_moe_combine(_ptrs(h), _ptrs(w2), _ptrs(gates), _ptrs(recv_src), counts.data_ptr(),
                              R, E_loc, topk, T, N, H, cap, _ptrs(o["ret"]), _ptrs(o["out"]),
                              buf.data_ptr(), buf.numel(), _cfgp(cfg), _stream(stream, dev))
    _check(st, "mk_moe_combine")
    return o


def mlp_workspace_size(R, m, h, f_r, cfg: Config | None = None) -> int:
    return int(lib().mk_mlp_workspace_size(R, m, h, f_r, _cfgp(cfg)))


def mlp_ag_rs(x_shards, w1, w2, *, x_gathered=None, hid=None, y_blocks=None,
              cfg: Config | None = None, workspace: Workspace | None = None, stream=None):
    """Chained tensor-parallel MLP over R virtual ranks: AllGather + GEMM (w1[r]) ->
    ReLU -> GEMM (w2[r]) + ReduceScatter.  x_shards[r]: [m x h]; w1[r]: [h x f_r];
    w2[r]: [f_r x h] (bf16).  Returns (x_gathered [R*m x h], hid [R x [R*m x f_r]],
    y_blocks [R x [m x h]])."""
    R = len(x_shards)
    m, h = x_shards[0].shape
    f_r = w1[0].shape[1]
    dev = x_shards[0].device
    bf = torch.bfloat16
    if x_gathered is None:
        x_gathered = torch.empty((R * m, h), dtype=bf, device=dev)
    if hid is None:
        hid = [torch.empty((R * m, f_r), dtype=bf, device=dev) for _ in range(R)]
    if y_blocks is None:
        y_blocks = [torch.empty((m, h), dtype=bf, device=dev) for _ in range(R)]
    ws = _ws(workspace, dev)
    nb = mlp_workspace_size(R, m, h, f_r, cfg)
    if nb == 0:
        raise MkError(MK_ERR_INVALID, "mk_mlp_workspace_size")
    buf = ws.get(nb, stream)
    st = lib().mk_mlp_ag_rs(_ptrs(x_shards), _ptrs(w1), _ptrs(w2), R, m, h, f_r, x_gathered.data_ptr(),
                            _ptrs(hid), _ptrs(y_blocks), buf.data_ptr(), buf.numel(), _cfgp(cfg),
                            _stream(stream, dev))
    _check(st, "mk_mlp_ag_rs")
    return x_gathered, hid, y_blocks


def ring_attention(q, k, v, *, causal: bool = False, scale: float | None = None, out=None,
                   k_recv=None, v_recv=None, cfg: Config | None = None,
                   workspace: Workspace | None = None, stream=None):
    """Ring attention over R virtual ranks.  q[r], k[r], v[r]: [heads x s_r x d] bf16
    (d = 128), rank r holding positions [r*s_r, (r+1)*s_r).  Returns out[r] (same shape)
    = softmax(scale * Q_r K^T (+ causal mask)) V over the whole sequence."""
    R = len(q)
    heads, s_r, d = q[0].shape
    dev = q[0].device
    bf = torch.bfloat16
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = [torch.empty((heads, s_r, d), dtype=bf, device=dev) for _ in range(R)]
    mode = cfg.mode if cfg is not None else MODE_FUSED
    if R > 1 and mode != MODE_GEMM_ONLY:
        if k_recv is None:
            k_recv = [torch.empty(((R - 1) * heads, s_r, d), dtype=bf, device=dev) for _ in range(R)]
        if v_recv is None:
            v_recv = [torch.empty(((R - 1) * heads, s_r, d), dtype=bf, device=dev) for _ in range(R)]
    kr = _ptrs(k_recv) if k_recv is not None else None
    vr = _ptrs(v_recv) if v_recv is not None else None
    ws = _ws(workspace, dev)
    nb = int(lib().mk_ring_attention_workspace_size(R, heads, s_r, d, int(causal), _cfgp(cfg)))
    if nb == 0:
        raise MkError(MK_ERR_INVALID, "mk_ring_attention_workspace_size")
    buf = ws.get(nb, stream)
    st = lib().mk_ring_attention(_ptrs(q), _ptrs(k), _ptrs(v), R, heads, s_r, d, int(causal),
                                 float(scale), kr, vr, _ptrs(out), buf.data_ptr(), buf.numel(),
                                 _cfgp(cfg), _stream(stream, dev))
    _check(st, "mk_ring_attention")
    return out


# ------------------------------------------------------------------ rotary positions and the paged cache

_bound = None


def _bind():
    """The native marshalling module (csrc/mk_bind.c), built in-tree like the library."""
    global _bound
    if _bound is None:
        try:
            from . import _mkbind
        except ImportError as e:
            raise RuntimeError("_mkbind.so is not built; run comm_gemm_tile_gb300/build.py "
                               "(or __graft_entry__.build())") from e
        _mkbind.setup((torch.bfloat16, torch.float32, torch.float16, FP8, torch.int32, torch.int64, torch.float64,
                       torch.uint8, torch.bool),
                      torch._C._cuda_getCurrentRawStream, torch.empty, torch._C._cuda_getDevice)
        _bound = _mkbind
    return _bound


def _address(name: str) -> int:
    """Address of an entry point of the library in use."""
    L = _lib or lib()
    found = L.__dict__.setdefault("_addresses", {})
    if name not in found:
        found[name] = ctypes.cast(getattr(L, name), ctypes.c_void_p).value
    return found[name]


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _on(stream, device):
    """A context in which outputs of a call on a given stream come from that stream's pool."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


_increment_version = torch.autograd.graph.increment_version


def _written(*given):
    """Tells autograd of the outputs that a call was given: a graph that has saved one may not use what it holds now."""
    _increment_version([t for t in given if t is not None and isinstance(t, torch.Tensor)])


def _new(shape, dtype, device, stream):
    with _on(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


def _raw(stream):
    return None if stream is None else stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def rope_freqs(rot: int, *, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
               original_length: int = 4096, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """(frequencies, magnitude) for rope / kv_append: float64 [rot / 2] and a factor.

    Unscaled, frequency i is base^(-2 i / rot).  scaling, for contexts `factor` times as
    long as the `original_length` a model was trained on:
      "linear"    every frequency divided by factor (positions interpolated);
      "ntk"       base grown to base * factor^(rot / (rot - 2)): the fastest frequency stays,
                  the slowest is divided by factor;
      "by_parts"  frequencies that turn at least `fast` times over original_length stay, those
                  that turn at most `slow` times are divided by factor, a linear blend in the
                  number of turns between; magnitude 1 + 0.1 ln(factor).
    """
    _need(rot >= 0 and rot % 2 == 0, "rot must be even")
    _need(scaling in (None, "linear", "ntk", "by_parts"), f"unknown scaling {scaling!r}")
    _need(base > 0 and factor >= 1 and fast > slow, "base, factor or the turns' bounds are out of range")
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    magnitude = 1.0
    if scaling == "ntk":
        _need(rot > 2, "ntk scaling needs rot > 2")
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-i / max(rot, 1))
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        keep = ((original_length * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        magnitude = 1.0 + 0.1 * math.log(factor)
    return f.to(device), magnitude


def _used_here(other, *tensors):
    """Of tensors that forward used on a stream it was given (`other`) and backward reads on the current one: their memory
    goes back to that stream's pool only when the current one is done with it."""
    if not other:
        return
    for t in tensors:
        if t is not None:
            t.record_stream(torch.cuda.current_stream(t.device))


class _Rope(torch.autograd.Function):
    """rope under autograd: the gradient is the inverse rotation, through rope again, so that it has one too."""

    @staticmethod
    def forward(ctx, x, freqs, positions, how, stream):
        y = rope(x, freqs, positions, **how, stream=stream)
        ctx.how, ctx.other = how, stream is not None
        ctx.save_for_backward(freqs, positions)
        return y

    @staticmethod
    def backward(ctx, dy):
        freqs, positions = ctx.saved_tensors
        _used_here(ctx.other, freqs, positions)
        if dy.stride(-1) != 1:      # the gradient of a sum, for one, is expanded
            dy = dy.contiguous()
        # (autograd runs this on the stream that was current in forward, and orders it)
        return rope(dy, freqs, positions, **{**ctx.how, "inverse": not ctx.how["inverse"]}), None, None, None, None


def rope(x, freqs, positions=None, *, start: int = 0, interleaved: bool = False, inverse: bool = False,
         magnitude: float = 1.0, out=None, stream=None):
    """Rotary positions.  x: [tokens x heads x d] (bf16, fp16 or fp32, any strides with d
    contiguous; a [heads x s x d] tensor of ring_attention is passed as x.transpose(0, 1)).
    The first 2 * len(freqs) elements of every head are turned by positions[t] * freqs (or
    (start + t) * freqs) and scaled by magnitude; interleaved pairs neighbours instead of
    halves.  inverse=True is the gradient: rope(dy, ..., inverse=True) = dx; where x requires a
    gradient, autograd takes it (not through an `out` of the caller's: that is refused).
    Returns out (unless given: of x's shape and memory order, dense; out=x works in place)."""
    if _forward_ad._current_level >= 0:
        _no_tangents(x)
    if torch.is_grad_enabled() and getattr(x, "requires_grad", False):
        _need(out is None, "x requires a gradient: rope cannot write it to a given out")
        return _Rope.apply(x, freqs, positions, dict(start=start, interleaved=interleaved, inverse=inverse,
                                                     magnitude=magnitude), stream)
    given = out
    if out is None:
        _need(isinstance(x, torch.Tensor), "x is not a tensor")
        if stream is None:
            out = torch.empty_like(x)
        else:
            with _on(stream, x.device):
                out = torch.empty_like(x)
    st = _bind().rope(_address("mk_rope"), x, out, freqs, positions, start, interleaved, inverse, magnitude, _raw(stream))
    if st:
        _check(st, "mk_rope")
    if given is not None:
        _written(given)
    return out


class KVCache:
    """A paged key / value cache: k, v [n_pages x heads x page_size x d] (any strides with d
    contiguous, the same for both; a cache laid out [n_pages x page_size x heads x d] is passed
    as k.transpose(1, 2)) in bf16, fp16 or float8_e4m3fn, the latter with k_scale, v_scale
    [n_pages x heads] fp32, not negative.  KVCache.empty allocates one.  The tensors and their memory are the
    cache's for good: a larger one is another KVCache, and one of whose tensors has been given other memory is refused."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        self._c, self._device = _bind().cache(k, v, k_scale, v_scale)   # the bytes of an mk_kv_cache
        self._tensors = k, v, k_scale, v_scale

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])

    @staticmethod
    def empty(n_pages: int, heads: int, page_size: int, d: int, dtype=torch.bfloat16, device="cuda"):
        """A cache of zeros."""
        make = lambda s, t: torch.zeros(s, dtype=t, device=device)   # noqa: E731
        shape = (n_pages, heads, page_size, d)
        scales = [make((n_pages, heads), torch.float32) for _ in range(2)] if dtype == FP8 else [None, None]
        return KVCache(make(shape, dtype), make(shape, dtype), *scales)


def kv_append(cache: KVCache, k, v, cu_q, kv_len, pages, *, q=None, freqs=None, positions=None,
              interleaved: bool = False, magnitude: float = 1.0, q_out=None, workspace: Workspace | None = None,
              stream=None):
    """Append a step's keys (rotated) and values to the cache, and rotate its queries.

    k, v: [tokens x heads x d], q: [tokens x heads_q x d]; cu_q [B+1]: sequence b has the tokens
    cu_q[b] .. cu_q[b+1]-1; kv_len [B]: its length with them; pages [B x max_pages]: its pages
    (all int32, on the device).  A token's rotary position is its position in the sequence
    unless `positions` gives another; freqs=None stores k as it is.  8-bit caches are
    quantised with a power-of-two scale for each page and head (see include/mk.h).
    Returns q_out (None without q).  Tokens without a slot set the device status.  For serving:
    no gradient comes through it (rope has one)."""
    _need(isinstance(cache, KVCache), "cache is not a KVCache")
    given = q_out
    if q is not None and q_out is None and stream is not None:
        q_out = _new(q.shape, q.dtype, q.device, stream)
    st, q_out = _bind().append(_address("mk_kv_append"), cache._c, cache._device, k, v, cu_q, kv_len, pages, q, q_out,
                               freqs, positions, interleaved, magnitude, (workspace or _default_ws.get(cache._device) or _ws(None, cache.k.device)).get(256, stream),
                               _raw(stream), cache._tensors)
    if st:
        _check(st, "mk_kv_append")
    if given is not None:
        _written(given)
    return q_out


def paged_attention_workspace_size(tokens: int, heads_q: int, heads: int, d: int, batch: int) -> int:
    return int(lib().mk_paged_attention_workspace_size(tokens, heads_q, heads, d, batch))


def paged_attention(q, cache: KVCache, cu_q, kv_len, pages, *, causal: bool = True, window: int = 0, sinks: int = 0,
                    scale: float | None = None, max_q: int = 0, out=None, return_lse: bool = False,
                    cfg: Config | None = None, workspace: Workspace | None = None, stream=None):
    """Attention of the new tokens of a batch of sequences over a paged cache (after kv_append).

    q: [tokens x heads_q x d] (bf16 or fp16, d = 64 or 128, heads_q a multiple of the cache's
    heads); cu_q, kv_len, pages as for kv_append.  The token at position p sees the keys
    j <= p (all of them with causal=False) that are among the last `window` (0: no window) or
    the first `sinks`.  max_q: an upper bound on a sequence's new tokens, if the caller knows
    one.  Returns out, or (out, lse) with return_lse; rows that see nothing are 0 (-inf).  For
    serving: no gradient comes through it.
    Calls that may run at the same time (on several streams) need a workspace each, and not one of the
    collective calls (ag_gemm and so on)."""
    _need(isinstance(cache, KVCache), "cache is not a KVCache")
    lse, given = True if return_lse else None, out
    if stream is not None:
        _need(isinstance(q, torch.Tensor) and q.dim() == 3, "q must be a [tokens x heads x d] CUDA tensor")
        if out is None:
            out = _new(q.shape, q.dtype, q.device, stream)
        if return_lse:
            lse = _new(q.shape[:2], torch.float32, q.device, stream)
    c = cfg.c() if cfg is not None else None
    get = (workspace or _default_paged_ws.get(cache._device) or _ws(None, cache.k.device, _default_paged_ws)).get
    if stream is not None:
        get = functools.partial(get, stream=stream)
    st, out, lse = _bind().attention(_address("mk_paged_attention"), _address("mk_paged_attention_workspace_size"),
                                     get, q, cache._c, cache._device, cu_q, kv_len, pages, causal, window, sinks, scale,
                                     max_q, out, lse,
                                     ctypes.addressof(c) if c is not None else None, _raw(stream), cache._tensors)
    if st:
        _check(st, "mk_paged_attention")
    if given is not None:
        _written(given)
    return (out, lse) if return_lse else out


# ------------------------------------------------------------------ norm, router, 4-bit weights

_NULL = contextlib.nullcontext()


def _on_given(stream, x):
    """A context in which the outputs and scratch of a call come from the pool of the stream it is given."""
    if stream is None:
        return _NULL
    _need(isinstance(x, torch.Tensor) and x.is_cuda, "the first argument is not a CUDA tensor")
    return _on(stream, x.device)


def _getter(workspace, stream):
    return None if workspace is None else functools.partial(getattr(workspace, "scratch", workspace.get), stream=stream)


def _wants_gradient(*tensors):
    for t in tensors:
        if getattr(t, "requires_grad", False):
            return torch.is_grad_enabled()
    return False


_forward_ad = torch.autograd.forward_ad      # (_current_level: -1 outside of forward-mode differentiation)


def _no_tangents(*tensors):
    """Refuses tensors of forward-mode differentiation, whose tangents would be lost."""
    for t in tensors:
        _need(not isinstance(t, torch.Tensor) or _forward_ad.unpack_dual(t).tangent is None,
              "an input has a tangent of forward-mode differentiation: there is none of this call")


def _rows_gradient(g):
    """A gradient as the calls read it: the one of a sum, for one, is expanded."""
    return g if g is None or g.stride(-1) == 1 else g.contiguous()


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps, stream):
        ctx.set_materialize_grads(False)
        y = rms_norm(x, weight, residual=residual, eps=eps, stream=stream)
        ctx.eps, ctx.residual, ctx.other = eps, residual is not None, stream is not None
        ctx.save_for_backward(y[1] if ctx.residual else x, weight)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight = ctx.saved_tensors
        _used_here(ctx.other, h, weight)
        dx = dh
        dw = None
        if dy is not None:       # (autograd runs this on the stream that was current in forward, and orders it)
            dx, dw = rms_norm_backward(_rows_gradient(dy), h, weight, dh=_rows_gradient(dh), eps=ctx.eps,
                                       weight_gradient=ctx.needs_input_grad[1])
        return dx, dw, dx if ctx.residual else None, None, None


def rms_norm(x, weight=None, *, residual=None, eps: float = 1e-6, out_dtype=None, out=None, scale_out=None, h_out=None,
             stream=None):
    """Root-mean-square norm of every row: y = h / sqrt(mean(h^2) + eps) * weight with h = x, or with
    a residual h = x + residual rounded to x's type (the residual stream that goes on).

    x, residual: [rows x n] or [tokens x heads x n] (bf16, fp16 or fp32, any strides with n
    contiguous, n <= 16384); weight: [n] of x's type or fp32, None for ones.  out_dtype: x's type,
    or float8_e4m3fn: then a row's scale is max(amax / 448, 2^-100) and y is the codes of
    y / scale, an operand of ag_gemm whose rows of c are multiplied by scale.
    Returns y, followed by scale (8 bits) and h (with a residual).  Outputs may be given: out,
    scale_out, h_out (h_out=residual updates the stream in place).  Where x, weight or residual
    requires a gradient, autograd takes it (not through an 8-bit output or outputs of the
    caller's: those are refused)."""
    e4m3 = out_dtype == FP8
    _need(out_dtype is None or e4m3 or out_dtype == getattr(x, "dtype", None), "out_dtype is x's type or float8_e4m3fn")
    if _forward_ad._current_level >= 0:
        _no_tangents(x, weight, residual)
    if _wants_gradient(x, weight, residual):
        _need(not e4m3, "an input requires a gradient: an 8-bit output has none")
        _need(out is None and scale_out is None and h_out is None, "an input requires a gradient: rms_norm cannot write to a given out")
        return _RmsNorm.apply(x, weight, residual, eps, stream)
    with _on_given(stream, x):
        st, y, scale, h = _bind().rms_norm(_address("mk_rms_norm"), x, residual, weight, out, scale_out, h_out, e4m3, eps,
                                           _raw(stream))
    if st:
        _check(st, "mk_rms_norm")
    if out is not None or scale_out is not None or h_out is not None:
        _written(out, scale_out, h_out)
    if residual is not None:
        return (y, scale, h) if e4m3 else (y, h)
    return (y, scale) if e4m3 else y


def rms_norm_backward(dy, h, weight=None, *, dh=None, eps: float = 1e-6, weight_gradient: bool = True, out=None,
                      workspace: Workspace | None = None, stream=None):
    """The gradient of rms_norm: (dx, dweight) for dy, the gradient of y, and dh, that of the h it returned.

    h: what was normalised (x, or the returned h).  dx is the gradient of x and of the residual
    alike (out: where to write it, dy and dh too).  dweight is None without a weight or with
    weight_gradient=False.  Scratch comes from the stream's memory unless a workspace is given
    (calls that may run at the same time need one each)."""
    if _forward_ad._current_level >= 0:
        _no_tangents(dy, h, weight, dh)
    wants = True if weight is not None and weight_gradient else None
    with _on_given(stream, dy):
        st, dx, dw = _bind().rms_norm_backward(_address("mk_rms_norm_backward"),
                                               _address("mk_rms_norm_backward_workspace_size"),
                                               _getter(workspace, stream), dy, dh, h, weight, out, wants, eps, _raw(stream))
    if st:
        _check(st, "mk_rms_norm_backward")
    if out is not None:
        _written(out)
    return dx, dw


_ROUTE = ("topk_idx", "gates", "counts", "tokens", "balance_loss", "z_loss")
_NONE = (None,) * len(_ROUTE)


class _MoeRoute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, topk, how, mask, workspace, stream):
        ctx.set_materialize_grads(False)
        r = moe_route(logits, topk, mask=mask, workspace=workspace, stream=stream, **how)
        ctx.how, ctx.other = how, stream is not None
        ctx.save_for_backward(logits, r["topk_idx"], r["counts"], r["tokens"])
        ctx.mark_non_differentiable(r["topk_idx"], r["counts"], r["tokens"])
        return tuple(r[name] for name in _ROUTE)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _idx, dgates, _counts, _tokens, dbalance, dz):
        logits, idx, counts, tokens = ctx.saved_tensors
        if dgates is None and dbalance is None and dz is None:
            return (None,) * 6
        _used_here(ctx.other, logits, idx, counts, tokens)
        route = {"topk_idx": idx, "counts": counts, "tokens": tokens}
        if dgates is not None:
            dgates = dgates.contiguous()
        return moe_route_backward(logits, route, dgates, dbalance, dz, **ctx.how), None, None, None, None, None


def moe_route(logits, topk: int, *, normalize: bool = True, scale: float = 1.0, mask=None, out=None,
              workspace: Workspace | None = None, stream=None):
    """Expert choice for the tokens of logits [T x E] (fp32, bf16 or fp16; E <= 256, topk <= 8).

    Returns a dict: topk_idx [T x topk] int32, the experts moe_dispatch_gemm chooses for these
    logits; gates [T x topk] fp32 for moe_combine: scale * softmax(logits) of those, over their
    sum if normalize; counts [E] int32, the tokens of each expert; tokens, how many count (N); and
    balance_loss = E * sum_e counts_e / (topk N) * mean p_e and z_loss = mean logsumexp^2 (fp32).
    mask [T] bool: False leaves a token out (ids -1, gates 0, counted nowhere), as tokens whose
    logits are all -inf are; an expert with a logit of -inf is not chosen.  `out` may pass
    preallocated buffers.  Where logits requires a gradient, autograd takes that of the gates and
    both losses (not into buffers of the caller's: those are refused).  Scratch as for rms_norm_backward."""
    o = out or {}
    if _forward_ad._current_level >= 0:
        _no_tangents(logits)
    if _wants_gradient(logits):
        _need(not o, "logits requires a gradient: moe_route cannot write to given outputs")
        return dict(zip(_ROUTE, _MoeRoute.apply(logits, topk, dict(normalize=normalize, scale=scale), mask, workspace, stream)))
    with _on_given(stream, logits):
        st, *got = _bind().route(_address("mk_moe_route"), _address("mk_moe_route_workspace_size"), _getter(workspace, stream),
                                 logits, topk, normalize, scale, mask, tuple(map(o.get, _ROUTE)) if o else _NONE, _raw(stream))
    if st:
        _check(st, "mk_moe_route")
    if o:
        _written(*o.values())
    return dict(zip(_ROUTE, got))


def moe_route_backward(logits, route, dgates=None, dbalance=None, dz=None, *, normalize: bool = True, scale: float = 1.0,
                       out=None, stream=None):
    """The gradient of moe_route with respect to the logits, for the gradients of its gates [T x topk],
    balance_loss and z_loss (fp32 on the device; None: none).  route: what moe_route returned for these logits,
    normalize and scale as it had them.  The counts are constants."""
    if _forward_ad._current_level >= 0:
        _no_tangents(logits, dgates, dbalance, dz)
    with _on_given(stream, logits):
        st, dl = _bind().route_backward(_address("mk_moe_route_backward"), logits, route["topk_idx"], route["counts"],
                                        route["tokens"], dgates, dbalance, dz, normalize, scale, out, _raw(stream))
    if st:
        _check(st, "mk_moe_route_backward")
    if out is not None:
        _written(out)
    return dl


class W4Weight:
    """A matrix of 4-bit weights [n x k], W[i][j] = scales[i][j / group] * (code[i][j] - zeros[i][j / group]):
    codes [n x k / 2] uint8 (the code of an even j in the lower four bits), scales and zeros [n x k / group]
    bf16 or fp16, all contiguous; without zeros 8 takes their place.  Groups have 32, 64 or 128 weights.
    W4Weight.quantize makes one.  What the tensors hold may change, their memory may not: w4_gemm refuses a weight
    one of whose tensors has been given other memory."""

    def __init__(self, codes, scales, zeros=None):
        self._w, self._device = _bind().w4(codes, scales, zeros)   # the bytes of an mk_w4_weight
        self._tensors = codes, scales, zeros

    codes = property(lambda self: self._tensors[0])
    scales = property(lambda self: self._tensors[1])
    zeros = property(lambda self: self._tensors[2])

    @staticmethod
    def pack(w, *, group: int = 128, symmetric: bool = True, dtype=torch.bfloat16):
        """(codes, scales, zeros) of w [n x k], on its device: by group, symmetric scale amax / 7 and codes 1 .. 15
        around 8, else scale (max - min) / 15 and the zero point of the least weight."""
        _need(w.dim() == 2 and group in (32, 64, 128) and w.shape[1] % group == 0, "w must be [n x k], k whole groups of 32, 64 or 128")
        _need(dtype in (torch.bfloat16, torch.float16), "scales are bf16 or fp16")
        n, k = w.shape
        f = w.detach().float().view(n, k // group, group)
        if symmetric:
            scale, zero = f.abs().amax(dim=-1) / 7, None
        else:
            lo, hi = f.amin(dim=-1).clamp_max(0), f.amax(dim=-1).clamp_min(0)
            scale = (hi - lo) / 15
        scale = scale.to(dtype)
        by = torch.where(scale == 0, torch.inf, scale.float())[..., None]
        if not symmetric:
            zero = (-lo / by[..., 0]).round().clamp(0, 15).to(dtype)
        code = (f / by).round() + (8 if symmetric else zero.float()[..., None])
        code = code.clamp(0, 15).to(torch.uint8).view(n, k // 2, 2)
        return code[..., 0] | (code[..., 1] << 4), scale, zero

    @staticmethod
    def quantize(w, *, group: int = 128, symmetric: bool = True, dtype=torch.bfloat16):
        """The 4-bit form of w [n x k] (once, when a model is loaded: plain tensor operations)."""
        return W4Weight(*W4Weight.pack(w, group=group, symmetric=symmetric, dtype=dtype))

    def dequantize(self, dtype=None):
        """W [n x k] in the scales' type, or another (plain tensor operations): for checks, or for the 16-bit
        products of prompts."""
        c, s, z = self._tensors
        code = torch.stack((c & 15, c >> 4), dim=-1).view(*s.shape, 2 * c.shape[1] // s.shape[1]).float()
        w = (code - (8.0 if z is None else z.float()[..., None])) * s.float()[..., None]
        return w.flatten(1).to(dtype or s.dtype)


def w4_gemm(x, w: W4Weight, *, out_dtype=None, out=None, cfg: Config | None = None, workspace: Workspace | None = None,
            stream=None):
    """y = x @ W^T for the rows of a decode step: x [m x k] of the weight's 16-bit type, y [m x n] in it or fp32
    (out_dtype).  Codes are multiplied as whole numbers, groups scaled and summed in fp32, y is rounded once.
    x's rows start on whole 16-byte pieces.  Any m is taken; for long prompts the 16-bit products are faster.  For serving: an
    x, scales or zero points that require a gradient are refused.  Calls of many rows or large matrices take scratch from the stream's
    memory; a wait that runs out there sets the device status."""
    _need(isinstance(w, W4Weight), "w is not a W4Weight")
    _need(out_dtype in (None, torch.float32) or out_dtype == getattr(x, "dtype", None), "out_dtype is x's type or fp32")
    if _forward_ad._current_level >= 0:
        _no_tangents(x, w.scales, w.zeros)
    tensors = w._tensors
    _need(not _wants_gradient(x, tensors[1], tensors[2]), "x, scales or zero points require a gradient: w4_gemm has none (use torch.no_grad)")
    c = cfg.c() if cfg is not None else None
    get = (workspace or _default_ws.get(w._device) or _ws(None, w.codes.device)).get
    if stream is not None:
        get = functools.partial(get, stream=stream)
    with _on_given(stream, x):
        st, y = _bind().w4_gemm(_address("mk_w4_gemm"), _address("mk_w4_gemm_scratch_size"), get, x, w._w, w._device, out,
                                out_dtype == torch.float32, ctypes.addressof(c) if c is not None else None, _raw(stream), tensors)
    if st:
        _check(st, "mk_w4_gemm")
    if out is not None:
        _written(out)
    return y


__all__ = ["Config", "MkError", "Workspace", "ag_gemm", "gemm_rs", "gemm_ar", "device_status",
           "workspace_size", "lib", "status_string", "MODE_FUSED", "MODE_GEMM_ONLY",
           "MODE_UNFUSED", "moe_dispatch_gemm", "moe_workspace_size", "moe_combine",
           "moe_combine_workspace_size", "mlp_ag_rs", "mlp_workspace_size", "ring_attention", "rope_freqs", "rope",
           "KVCache", "kv_append", "paged_attention", "paged_attention_workspace_size", "rms_norm", "rms_norm_backward",
           "moe_route", "moe_route_backward", "W4Weight", "w4_gemm"]
