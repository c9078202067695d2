"""Thin ctypes binding over the C ABI in include/ep.h (argument marshalling only).

Every step of the path runs in libep.so's CUDA kernels; this module only
allocates torch tensors for outputs the caller did not pass, fills the
``ep_layout_t`` struct and forwards raw pointers plus torch's current CUDA
stream.  There is no CPU fallback: if libep.so is missing or a tensor is not on
a CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libep.so")

(EP_OK, EP_ERR_INVALID_ARG, EP_ERR_CAPACITY, EP_ERR_BAD_EXPERT_ID, EP_ERR_CUDA, EP_ERR_UNSUPPORTED,
 EP_ERR_TIMEOUT) = range(7)
LAYOUT_KIND = {"contig": 0, "masked": 1}
QUANT = {"none": 0, "fp8_f32": 1, "fp8_ue8m0": 2, "mxfp8": 3, "fp8_ue8m0_mn": 4}
MAX_TOPK, MAX_EXPERTS, MAX_ALIGN = 32, 1024, 128


class EPError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"{what}: {status_str(code)}" if what else status_str(code))


class _Layout(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int32),
        ("num_topk", ctypes.c_int32),
        ("num_experts", ctypes.c_int32),
        ("num_ranks", ctypes.c_int32),
        ("kind", ctypes.c_int32),
        ("align", ctypes.c_int32),
        ("capacity", ctypes.c_int32),
        ("max_tokens", ctypes.c_int32),
        ("dst_row", ctypes.c_void_p),
        ("row_src", ctypes.c_void_p),
        ("expert_count", ctypes.c_void_p),
        ("expert_offset", ctypes.c_void_p),
        ("rank_rows", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
    ]


_lib = None

EXPORTS = ("ep_status_str", "ep_rows_capacity", "ep_scale_cols", "ep_scale_words",
           "ep_layout_workspace_bytes",
           "ep_layout", "ep_dispatch", "ep_layout_dispatch", "ep_combine", "ep_masked_repack",
           "ep_layout_noalloc", "ep_selftest_bounded_wait", "ep_selftest_cluster_wait",
           "ep_rank_layout", "ep_rank_expand", "ep_route_topk", "ep_rmsnorm", "ep_expert_gemm",
           "ep_expert_swiglu", "ep_moe_decode", "ep_moe_decode_workspace_bytes")
NOALLOC_SCRATCH_BYTES = 256 * 1024


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libep.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(path)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    LP = ctypes.POINTER(_Layout)
    L.ep_status_str.restype = ctypes.c_char_p
    L.ep_status_str.argtypes = [ctypes.c_int]
    L.ep_rows_capacity.restype = I64
    L.ep_rows_capacity.argtypes = [LP]
    L.ep_scale_cols.restype = I64
    L.ep_scale_cols.argtypes = [I32, ctypes.c_int]
    L.ep_scale_words.restype = I64
    L.ep_scale_words.argtypes = [LP, I32, ctypes.c_int]
    L.ep_layout_workspace_bytes.restype = SZ
    L.ep_layout_workspace_bytes.argtypes = [LP]
    L.ep_layout.restype = ctypes.c_int
    L.ep_layout.argtypes = [P, LP, P, SZ, P]
    L.ep_dispatch.restype = ctypes.c_int
    L.ep_dispatch.argtypes = [LP, P, I32, ctypes.c_int, P, P, P, P, P]
    L.ep_layout_dispatch.restype = ctypes.c_int
    L.ep_layout_dispatch.argtypes = [P, LP, P, SZ, P, I32, ctypes.c_int, P, P, P, P, P]
    L.ep_combine.restype = ctypes.c_int
    L.ep_combine.argtypes = [LP, P, I32, P, P, P]
    L.ep_masked_repack.restype = ctypes.c_int
    L.ep_masked_repack.argtypes = [LP, P, P, I32, ctypes.c_int, I32, P, P, P, P]
    L.ep_route_topk.restype = ctypes.c_int
    L.ep_route_topk.argtypes = [P, P, I32, I32, I32, ctypes.c_int, I32, I32, P, P, P]
    L.ep_rank_layout.restype = ctypes.c_int
    L.ep_rank_layout.argtypes = [P, I32, P, LP, P, SZ, P]
    L.ep_rank_expand.restype = ctypes.c_int
    L.ep_rank_expand.argtypes = [LP, LP, P, I32, ctypes.c_int, P, P, P, P, P]
    L.ep_selftest_bounded_wait.restype = ctypes.c_int
    L.ep_selftest_bounded_wait.argtypes = [P, I64, P]
    L.ep_selftest_cluster_wait.restype = ctypes.c_int
    L.ep_selftest_cluster_wait.argtypes = [P, I64, P]
    L.ep_layout_noalloc.restype = ctypes.c_int
    L.ep_layout_noalloc.argtypes = [P, LP, P]
    Q = ctypes.c_int
    L.ep_rmsnorm.restype = ctypes.c_int
    L.ep_rmsnorm.argtypes = [P, P, P, ctypes.c_float, I32, I32, Q, P, P, P, P, P]
    L.ep_expert_gemm.restype = ctypes.c_int
    L.ep_expert_gemm.argtypes = [LP, P, P, I32, Q, P, P, I32, P, P]
    L.ep_expert_swiglu.restype = ctypes.c_int
    L.ep_expert_swiglu.argtypes = [LP, P, P, I32, Q, P, P, I32, Q, P, P, P]
    L.ep_moe_decode_workspace_bytes.restype = SZ
    L.ep_moe_decode_workspace_bytes.argtypes = [I32] * 5
    L.ep_moe_decode.restype = ctypes.c_int
    L.ep_moe_decode.argtypes = [P, P, Q, P, P, I32, I32, I32, I32, I32, P, P, P, P, P, P, P, SZ, P]
    if path == LIB_PATH:
        _lib = L
    return L


def status_str(code: int) -> str:
    try:
        return load_library().ep_status_str(int(code)).decode()
    except RuntimeError:
        return f"ep_status_t {code}"


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libep works on CUDA tensors only")
    if not t.is_contiguous():
        raise ValueError("libep needs contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(code: int, what: str):
    if code != EP_OK:
        raise EPError(code, what)


@dataclass
class Layout:
    """Shape + device arrays of one layout (the dispatch "handle")."""

    num_tokens: int
    num_topk: int
    num_experts: int
    num_ranks: int
    kind: str
    align: int
    capacity: int
    max_tokens: int
    dst_row: torch.Tensor
    row_src: Optional[torch.Tensor]
    expert_count: torch.Tensor
    expert_offset: torch.Tensor
    rank_rows: Optional[torch.Tensor]
    status: torch.Tensor
    workspace: Optional[torch.Tensor] = None
    _c: _Layout = field(default=None, repr=False)

    def struct(self) -> _Layout:
        c = _Layout()
        c.num_tokens, c.num_topk, c.num_experts = self.num_tokens, self.num_topk, self.num_experts
        c.num_ranks, c.kind, c.align = self.num_ranks, LAYOUT_KIND[self.kind], self.align
        c.capacity, c.max_tokens = self.capacity, self.max_tokens
        c.dst_row = _ptr(self.dst_row).value
        c.row_src = _ptr(self.row_src).value if self.row_src is not None else None
        c.expert_count = _ptr(self.expert_count).value
        c.expert_offset = _ptr(self.expert_offset).value
        c.rank_rows = _ptr(self.rank_rows).value if self.rank_rows is not None else None
        c.status = _ptr(self.status).value
        self._c = c
        return c

    @property
    def rows_capacity(self) -> int:
        return ep_rows_capacity(self)

    def check_status(self) -> None:
        """Synchronise and raise EPError if a device-side error was recorded."""
        st = int(self.status.item())
        if st != EP_OK:
            raise EPError(st, "device status")


def new_layout(num_tokens: int, num_topk: int, num_experts: int, kind: str = "contig",
               align: int = 128, capacity: int = 0, num_ranks: int = 1, max_tokens: int = 0,
               with_row_src: bool = True, device=None) -> Layout:
    """Allocate the arrays of a layout (uninitialised; ep_layout fills them)."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    i32 = dict(dtype=torch.int32, device=dev)
    L = Layout(num_tokens, num_topk, num_experts, num_ranks, kind, align, capacity, max_tokens,
               dst_row=torch.empty(max(num_tokens * num_topk, 1), **i32),
               row_src=None, expert_count=torch.empty(num_experts, **i32),
               expert_offset=torch.empty(num_experts + 1, **i32),
               rank_rows=torch.empty(num_ranks, **i32), status=torch.zeros(1, **i32))
    rows = ep_rows_capacity(L)
    if rows < 0:
        raise EPError(EP_ERR_INVALID_ARG, "layout shape")
    if with_row_src:
        L.row_src = torch.empty(max(rows, 1), **i32)
    ws = ep_layout_workspace_bytes(L)
    if ws:
        L.workspace = torch.empty((ws + 3) // 4, **i32)
    return L


# ------------------------------------------------------------- C ABI mirrors
def ep_rows_capacity(layout: Layout) -> int:
    c = _Layout()
    c.num_tokens, c.num_topk, c.num_experts = layout.num_tokens, layout.num_topk, layout.num_experts
    c.num_ranks, c.kind, c.align = layout.num_ranks, LAYOUT_KIND[layout.kind], layout.align
    c.capacity, c.max_tokens = layout.capacity, layout.max_tokens
    return int(load_library().ep_rows_capacity(ctypes.byref(c)))


def ep_scale_cols(hidden: int, quant: str) -> int:
    return int(load_library().ep_scale_cols(hidden, QUANT[quant]))


def _shape_struct(layout: Layout) -> _Layout:
    c = _Layout()
    c.num_tokens, c.num_topk, c.num_experts = layout.num_tokens, layout.num_topk, layout.num_experts
    c.num_ranks, c.kind, c.align = layout.num_ranks, LAYOUT_KIND[layout.kind], layout.align
    c.capacity, c.max_tokens = layout.capacity, layout.max_tokens
    return c


def ep_scale_words(layout: Layout, hidden: int, quant: str) -> int:
    return int(load_library().ep_scale_words(ctypes.byref(_shape_struct(layout)), hidden,
                                             QUANT[quant]))


def scale_buffer(layout: Layout, hidden: int, quant: str, device=None) -> Optional[torch.Tensor]:
    """An uninitialised scale buffer shaped for ``quant`` on this layout."""
    if quant == "none":
        return None
    dev = device if device is not None else layout.dst_row.device
    cols = ep_scale_cols(hidden, quant)
    if quant == "fp8_ue8m0_mn":
        if layout.kind == "masked":
            shape = (layout.num_experts, cols, (layout.capacity + 3) // 4 * 4)
        else:
            shape = (cols, (max(layout.rows_capacity, 1) + 3) // 4 * 4)
        return torch.empty(shape, device=dev, dtype=torch.int32)
    return torch.empty((max(layout.rows_capacity, 1), cols), device=dev,
                       dtype=torch.float32 if quant == "fp8_f32" else torch.int32)


def ep_layout_workspace_bytes(layout: Layout) -> int:
    c = _Layout()
    c.num_tokens, c.num_topk, c.num_experts = layout.num_tokens, layout.num_topk, layout.num_experts
    c.num_ranks, c.kind, c.align = layout.num_ranks, LAYOUT_KIND[layout.kind], layout.align
    c.capacity, c.max_tokens = layout.capacity, layout.max_tokens
    return int(load_library().ep_layout_workspace_bytes(ctypes.byref(c)))


def ep_layout(topk_idx: torch.Tensor, num_experts: int, kind: str = "contig", align: int = 128,
              capacity: int = 0, num_ranks: int = 1, max_tokens: int = 0,
              with_row_src: bool = True, out: Optional[Layout] = None, stream=None) -> Layout:
    """Expert histogram, padded scan and stable slots for topk_idx (int32 [T, K])."""
    if topk_idx.dtype != torch.int32 or topk_idx.dim() != 2:
        raise ValueError("topk_idx must be int32 [T, K]")
    T, K = topk_idx.shape
    L = out if out is not None else new_layout(T, K, num_experts, kind, align, capacity,
                                               num_ranks, max_tokens, with_row_src,
                                               device=topk_idx.device)
    if (L.num_tokens, L.num_topk) != (T, K):
        raise ValueError("layout shape does not match topk_idx")
    ws = L.workspace
    nbytes = ws.numel() * 4 if ws is not None else 0
    code = load_library().ep_layout(_ptr(topk_idx) if T * K else None, ctypes.byref(L.struct()),
                                    _ptr(ws), nbytes, _stream(stream))
    _check(code, "ep_layout")
    return L


def ep_dispatch(layout: Layout, x: torch.Tensor, quant: str = "none",
                out_rows: Optional[torch.Tensor] = None, out_scales: Optional[torch.Tensor] = None,
                topk_w: Optional[torch.Tensor] = None, row_w: Optional[torch.Tensor] = None,
                stream=None):
    """Scatter (and quantise) x (bf16 [T, H]) into the layout's rows.

    Returns (out_rows, out_scales, row_w).  out_rows is bf16 [rows, H] or uint8
    E4M3 bytes; out_scales fp32 [rows, H/128] (fp8_f32), int32 [rows, ceil(H/512)]
    (fp8_ue8m0) or int32 [rows, H/128] holding H/32 E8M0 bytes (mxfp8).
    """
    T, H = x.shape
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16")
    rows = layout.rows_capacity
    dev = x.device
    if out_rows is None:
        out_rows = torch.empty((max(rows, 1), H), device=dev,
                               dtype=torch.bfloat16 if quant == "none" else torch.uint8)
    if quant != "none" and out_scales is None:
        out_scales = scale_buffer(layout, H, quant, device=dev)
    if topk_w is not None and row_w is None:
        row_w = torch.empty(max(rows, 1), device=dev, dtype=torch.float32)
    code = load_library().ep_dispatch(ctypes.byref(layout.struct()), _ptr(x), H, QUANT[quant],
                                      _ptr(out_rows), _ptr(out_scales), _ptr(topk_w), _ptr(row_w),
                                      _stream(stream))
    _check(code, "ep_dispatch")
    return out_rows, out_scales, row_w


def ep_layout_dispatch(topk_idx: torch.Tensor, layout: Layout, x: torch.Tensor,
                       quant: str = "none", out_rows: Optional[torch.Tensor] = None,
                       out_scales: Optional[torch.Tensor] = None,
                       topk_w: Optional[torch.Tensor] = None, row_w: Optional[torch.Tensor] = None,
                       stream=None):
    """ep_layout into ``layout`` and ep_dispatch of x, in one call (the two
    kernels back to back).  Returns (out_rows, out_scales, row_w) like ep_dispatch."""
    if topk_idx.dtype != torch.int32 or topk_idx.dim() != 2:
        raise ValueError("topk_idx must be int32 [T, K]")
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16")
    T, K = topk_idx.shape
    if (layout.num_tokens, layout.num_topk) != (T, K):
        raise ValueError("layout shape does not match topk_idx")
    H = x.shape[1]
    rows = layout.rows_capacity
    dev = x.device
    if out_rows is None:
        out_rows = torch.empty((max(rows, 1), H), device=dev,
                               dtype=torch.bfloat16 if quant == "none" else torch.uint8)
    if quant != "none" and out_scales is None:
        out_scales = scale_buffer(layout, H, quant, device=dev)
    if topk_w is not None and row_w is None:
        row_w = torch.empty(max(rows, 1), device=dev, dtype=torch.float32)
    ws = layout.workspace
    code = load_library().ep_layout_dispatch(
        _ptr(topk_idx) if T * K else None, ctypes.byref(layout.struct()), _ptr(ws),
        ws.numel() * 4 if ws is not None else 0, _ptr(x), H, QUANT[quant], _ptr(out_rows),
        _ptr(out_scales), _ptr(topk_w), _ptr(row_w), _stream(stream))
    _check(code, "ep_layout_dispatch")
    return out_rows, out_scales, row_w


def ep_combine(layout: Layout, y: torch.Tensor, topk_w: torch.Tensor,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = bf16(sum_k topk_w[t,k] * y[dst_row[t,k]]), fp32 accumulation."""
    H = y.shape[-1]
    if y.dtype != torch.bfloat16 or topk_w.dtype != torch.float32:
        raise ValueError("y must be bf16 and topk_w fp32")
    if out is None:
        out = torch.empty((layout.num_tokens, H), device=y.device, dtype=torch.bfloat16)
    code = load_library().ep_combine(ctypes.byref(layout.struct()), _ptr(y), H, _ptr(topk_w),
                                     _ptr(out), _stream(stream))
    _check(code, "ep_combine")
    return out


def ep_masked_repack(layout: Layout, rows: torch.Tensor, row_scales: Optional[torch.Tensor],
                     quant: str, capacity: int, slab: Optional[torch.Tensor] = None,
                     slab_scales: Optional[torch.Tensor] = None,
                     masked_m: Optional[torch.Tensor] = None, stream=None):
    """Contiguous layout rows -> masked slab [E, capacity, ...]; returns (slab, slab_scales, masked_m)."""
    E = layout.num_experts
    H = rows.shape[-1]
    dev = rows.device
    if slab is None:
        slab = torch.empty((E, capacity, H), device=dev, dtype=rows.dtype)
    if row_scales is not None and slab_scales is None:
        if quant == "fp8_ue8m0_mn":
            slab_scales = torch.empty((E, ep_scale_cols(H, quant), (capacity + 3) // 4 * 4),
                                      device=dev, dtype=row_scales.dtype)
        else:
            slab_scales = torch.empty((E, capacity, row_scales.shape[-1]), device=dev,
                                      dtype=row_scales.dtype)
    if masked_m is None:
        masked_m = torch.empty(E, device=dev, dtype=torch.int32)
    code = load_library().ep_masked_repack(ctypes.byref(layout.struct()), _ptr(rows),
                                           _ptr(row_scales), H, QUANT[quant], capacity, _ptr(slab),
                                           _ptr(slab_scales), _ptr(masked_m), _stream(stream))
    _check(code, "ep_masked_repack")
    return slab, slab_scales, masked_m


def ep_selftest_bounded_wait(status: torch.Tensor, limit_clocks: int, stream=None) -> None:
    """Make one bounded device wait run out; EP_ERR_TIMEOUT lands in ``status``."""
    if status.dtype != torch.int32 or not status.is_cuda:
        raise ValueError("status must be a device int32 tensor")
    _check(load_library().ep_selftest_bounded_wait(_ptr(status), int(limit_clocks),
                                                    _stream(stream)), "ep_selftest_bounded_wait")


def ep_selftest_cluster_wait(status: torch.Tensor, limit_clocks: int, stream=None) -> None:
    """Make the cluster exchange's bounded wait run out in a 2-CTA cluster;
    EP_ERR_TIMEOUT lands in ``status``."""
    if status.dtype != torch.int32 or not status.is_cuda:
        raise ValueError("status must be a device int32 tensor")
    _check(load_library().ep_selftest_cluster_wait(_ptr(status), int(limit_clocks),
                                                    _stream(stream)), "ep_selftest_cluster_wait")


def ep_layout_noalloc(topk_idx: torch.Tensor, out: Layout, stream=None) -> Layout:
    """ep_layout with the library's fixed scratch array instead of a workspace.

    For callers that cannot allocate device memory; ``out`` must be a layout
    whose arrays the caller already owns (``out.workspace`` is ignored).  Calls
    share the library's one scratch array, so calls that overlap on the GPU race.
    """
    if topk_idx.dtype != torch.int32 or topk_idx.dim() != 2:
        raise ValueError("topk_idx must be int32 [T, K]")
    T, K = topk_idx.shape
    if (out.num_tokens, out.num_topk) != (T, K):
        raise ValueError("layout shape does not match topk_idx")
    code = load_library().ep_layout_noalloc(_ptr(topk_idx) if T * K else None,
                                            ctypes.byref(out.struct()), _stream(stream))
    _check(code, "ep_layout_noalloc")
    return out


def ep_rank_layout(topk_idx: torch.Tensor, num_experts: int, num_ranks: int, align: int = 1,
                   out: Optional[Layout] = None, rank_idx: Optional[torch.Tensor] = None,
                   stream=None):
    """Per-rank deduplicated send layout; returns (rank Layout, rank_idx [T, K])."""
    if topk_idx.dtype != torch.int32 or topk_idx.dim() != 2:
        raise ValueError("topk_idx must be int32 [T, K]")
    T, K = topk_idx.shape
    RL = out if out is not None else new_layout(T, K, num_ranks, "contig", align=align,
                                                device=topk_idx.device)
    if rank_idx is None:
        rank_idx = torch.empty((T, K), dtype=torch.int32, device=topk_idx.device)
    ws = RL.workspace
    code = load_library().ep_rank_layout(_ptr(topk_idx) if T * K else None, num_experts,
                                         _ptr(rank_idx) if T * K else None,
                                         ctypes.byref(RL.struct()), _ptr(ws),
                                         ws.numel() * 4 if ws is not None else 0, _stream(stream))
    _check(code, "ep_rank_layout")
    return RL, rank_idx


def ep_rank_expand(rank_layout: Layout, layout: Layout, topk_idx: torch.Tensor, quant: str,
                   send_rows: torch.Tensor, send_scales: Optional[torch.Tensor],
                   out_rows: Optional[torch.Tensor] = None,
                   out_scales: Optional[torch.Tensor] = None, stream=None):
    """Send buffer -> per-expert rows (and scale rows); returns (out_rows, out_scales)."""
    H = send_rows.shape[-1]
    dev = send_rows.device
    rows = layout.rows_capacity
    if out_rows is None:
        out_rows = torch.empty((max(rows, 1), H), device=dev, dtype=send_rows.dtype)
    if send_scales is not None and out_scales is None:
        out_scales = torch.empty((max(rows, 1), send_scales.shape[-1]), device=dev,
                                 dtype=send_scales.dtype)
    code = load_library().ep_rank_expand(ctypes.byref(rank_layout.struct()),
                                         ctypes.byref(layout.struct()), _ptr(topk_idx), H,
                                         QUANT[quant], _ptr(send_rows), _ptr(send_scales),
                                         _ptr(out_rows), _ptr(out_scales), _stream(stream))
    _check(code, "ep_rank_expand")
    return out_rows, out_scales


ROUTE = {"softmax": 0, "grouped_sigmoid": 1}


def ep_route_topk(logits: torch.Tensor, num_topk: int, mode: str = "softmax",
                  bias: Optional[torch.Tensor] = None, n_group: int = 1, topk_group: int = 1,
                  topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
                  stream=None):
    """Router top-k from fp32 logits [T, E]; returns (topk_idx int32, topk_w fp32) [T, K]."""
    if logits.dtype != torch.float32 or logits.dim() != 2:
        raise ValueError("logits must be fp32 [T, E]")
    T, E = logits.shape
    dev = logits.device
    if topk_idx is None:
        topk_idx = torch.empty((T, num_topk), dtype=torch.int32, device=dev)
    if topk_w is None:
        topk_w = torch.empty((T, num_topk), dtype=torch.float32, device=dev)
    code = load_library().ep_route_topk(_ptr(logits), _ptr(bias), T, E, num_topk, ROUTE[mode],
                                        n_group, topk_group, _ptr(topk_idx), _ptr(topk_w),
                                        _stream(stream))
    _check(code, "ep_route_topk")
    return topk_idx, topk_w


# ------------------------------------------------------- norm, experts, decode
_E4M3 = (torch.uint8, torch.float8_e4m3fn)
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _refuse(t, name: str, dtypes, shape, dev: int):
    """The error for a tensor that _want did not take."""
    if t is None:
        raise ValueError(f"{name} is missing")
    if not t.is_cuda:
        raise ValueError("libep works on CUDA tensors only")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} is not accepted")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{dev}")
    raise ValueError("libep needs contiguous tensors")


def _want(t: torch.Tensor, name: str, dtypes, shape, dev: int) -> int:
    """Address of a tensor argument of one of `dtypes`, `shape`, contiguous on device `dev`."""
    if t is None or t.dtype not in dtypes or t.shape != shape or t.get_device() != dev \
            or not t.is_contiguous():
        _refuse(t, name, dtypes, shape, dev)
    return t.data_ptr()


def _rows_of(t: torch.Tensor, name: str, dims: int = 2) -> int:
    """Device index of a call's first tensor, a CUDA tensor of `dims` dimensions."""
    if not t.is_cuda:
        raise ValueError("libep works on CUDA tensors only")
    if t.dim() != dims:
        raise ValueError(f"{name}: {t.dim()} dimensions, expected {dims}")
    return t.get_device()


def _on(stream, dev: int) -> int:
    """The stream a call runs on: `stream`, or device `dev`'s current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device.index != dev:
        raise ValueError(f"stream on {stream.device}, tensors on cuda:{dev}")
    return stream.cuda_stream


def _empty(shape, dtype, dev: int, stream) -> torch.Tensor:
    """An output that belongs to the call's stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", dev))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", dev))


def _call(fn, name: str, dev: int, *args) -> None:
    if dev == torch.cuda.current_device():
        code = fn(*args)
    else:
        with torch.cuda.device(dev):
            code = fn(*args)
    if code != EP_OK:
        raise EPError(code, name)


def _scale_shape(rows: int, hidden: int, quant: str, slab=None):
    """(dtypes, shape) of the scales of `rows` rows; slab = (E, capacity) of a masked layout."""
    if quant == "fp8_f32" and hidden % 128 == 0:
        return (_F32,), (rows, hidden // 128)
    cols = ep_scale_cols(hidden, quant)
    if cols < 0:
        raise EPError(EP_ERR_INVALID_ARG, f"hidden {hidden} for {quant}")
    if quant == "fp8_ue8m0_mn":
        if slab is not None:
            return (_I32,), (slab[0], cols, (slab[1] + 3) // 4 * 4)
        return (_I32,), (cols, (rows + 3) // 4 * 4)
    return (_I32,), (rows, cols)


def ep_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
               residual: Optional[torch.Tensor] = None, quant: str = "none",
               out: Optional[torch.Tensor] = None, out_rows: Optional[torch.Tensor] = None,
               out_scales: Optional[torch.Tensor] = None,
               residual_out: Optional[torch.Tensor] = None, with_out: bool = True, stream=None):
    """RMS norm of x + residual (bf16 [T, H]), as bf16 and / or 8-bit rows.

    Returns (out, out_rows, out_scales, residual_out): out is None with
    ``with_out=False`` (8-bit rows only), out_rows and out_scales are None for
    quant "none", residual_out (the sum; may be ``residual`` or ``x`` itself) is
    None without a residual unless a tensor is passed for it.
    """
    lib = load_library()
    dev = _rows_of(x, "x")
    shape = x.shape
    T, H = shape
    px = _want(x, "x", (_BF16,), shape, dev)
    pw = _want(weight, "weight", (_BF16,), (H,), dev)
    pr = po = pq = ps = pro = None
    if residual is not None:
        pr = _want(residual, "residual", (_BF16,), shape, dev)
        if residual_out is None:
            residual_out = _empty(shape, _BF16, dev, stream)
    if residual_out is not None:
        pro = _want(residual_out, "residual_out", (_BF16,), shape, dev)
    if out is None and with_out:
        out = _empty(shape, _BF16, dev, stream)
    if out is not None:
        po = _want(out, "out", (_BF16,), shape, dev)
    if quant != "none":
        sdt, sshape = _scale_shape(T, H, quant)
        if out_rows is None:
            out_rows = _empty(shape, torch.uint8, dev, stream)
        if out_scales is None:
            out_scales = _empty(sshape, sdt[0], dev, stream)
        pq = _want(out_rows, "out_rows", _E4M3, shape, dev)
        ps = _want(out_scales, "out_scales", sdt, sshape, dev)
    elif out_rows is not None or out_scales is not None:
        raise ValueError('out_rows and out_scales belong to an 8-bit quant, not "none"')
    _call(lib.ep_rmsnorm, "ep_rmsnorm", dev, px, pr, pw, eps, T, H, QUANT[quant], pro, po, pq, ps,
          _on(stream, dev))
    return out, out_rows, out_scales, residual_out


def _layout_arg(layout: Layout, dev: int) -> _Layout:
    """The C struct of a layout on device `dev` for the experts' products.  Of a
    masked one, which may be made up, they read only the counts and the status."""
    E = layout.num_experts
    count = _want(layout.expert_count, "layout.expert_count", (_I32,), (E,), dev)
    status = _want(layout.status, "layout.status", (_I32,), (1,), dev)
    if layout.kind == "masked":
        return _Layout(num_experts=E, kind=LAYOUT_KIND["masked"], capacity=layout.capacity,
                       expert_count=count, status=status)
    rr, rs = layout.rank_rows, layout.row_src
    return _Layout(layout.num_tokens, layout.num_topk, E, layout.num_ranks,
                   LAYOUT_KIND[layout.kind], layout.align, layout.capacity, layout.max_tokens,
                   layout.dst_row.data_ptr(), rs.data_ptr() if rs is not None else None, count,
                   _want(layout.expert_offset, "layout.expert_offset", (_I32,), (E + 1,), dev),
                   rr.data_ptr() if rr is not None else None, status)


def _slab_rows(t: torch.Tensor) -> torch.Tensor:
    """A slab [E, capacity, n] as its rows [E * capacity, n], in the same memory
    (flatten would copy another one, into a tensor that is gone before the launch)."""
    if not t.is_contiguous():
        raise ValueError("libep needs contiguous tensors")
    return t.flatten(0, 1)


def _expert_args(lib, layout: Layout, rows, row_scales, weights, weight_scales, quant: str):
    """Shared argument checks of the experts' products: (device index, C layout,
    rows of the row space, slab, N, K, the four addresses)."""
    slab = (layout.num_experts, layout.capacity) if layout.kind == "masked" else None
    if slab is not None:  # [E, capacity, ...], as ep_masked_repack returns it
        if rows.dim() == 3:
            rows = _slab_rows(rows)
        if row_scales is not None and row_scales.dim() == 3 and quant != "fp8_ue8m0_mn":
            row_scales = _slab_rows(row_scales)
    dev = _rows_of(rows, "rows")
    c = _layout_arg(layout, dev)
    cap = slab[0] * slab[1] if slab is not None else lib.ep_rows_capacity(ctypes.byref(c))
    if cap < 0:
        raise EPError(EP_ERR_INVALID_ARG, "layout shape")
    if cap == 0:
        cap = 1
    E, K = layout.num_experts, rows.shape[1]
    px = _want(rows, "rows", _E4M3, (cap, K), dev)
    if quant == "none" or quant == "mxfp8":
        raise EPError(EP_ERR_UNSUPPORTED, f"expert products of {quant} rows")
    sdt, sshape = _scale_shape(cap, K, quant, slab)
    ps = _want(row_scales, "row_scales", sdt, sshape, dev)
    N = weights.shape[1] if weights is not None and weights.dim() == 3 else 0
    pw = _want(weights, "weights", _E4M3, (E, N, K), dev)
    pws = _want(weight_scales, "weight_scales", (_F32,), (E, (N + 127) // 128, K // 128), dev)
    return dev, c, cap, slab, N, K, px, ps, pw, pws


def ep_expert_gemm(layout: Layout, rows: torch.Tensor, row_scales: torch.Tensor,
                   weights: torch.Tensor, weight_scales: torch.Tensor, quant: str = "fp8_f32",
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Each expert's block-scaled product on its rows: bf16 [rows, N].

    rows / row_scales as ep_dispatch (or ep_masked_repack) wrote them; weights
    E4M3 [E, N, K], weight_scales fp32 [E, ceil(N/128), K/128].  Rows of the
    layout that no entry fills are not written.
    """
    lib = load_library()
    dev, c, cap, _, N, K, px, ps, pw, pws = _expert_args(lib, layout, rows, row_scales, weights,
                                                         weight_scales, quant)
    if out is None:
        out = _empty((cap, N), _BF16, dev, stream)
    po = _want(out, "out", (_BF16,), (cap, N), dev)
    _call(lib.ep_expert_gemm, "ep_expert_gemm", dev, ctypes.byref(c), px, ps, K, QUANT[quant], pw,
          pws, N, po, _on(stream, dev))
    return out


def ep_expert_swiglu(layout: Layout, rows: torch.Tensor, row_scales: torch.Tensor,
                     weights: torch.Tensor, weight_scales: torch.Tensor, quant: str = "fp8_f32",
                     out_quant: str = "fp8_f32", out_rows: Optional[torch.Tensor] = None,
                     out_scales: Optional[torch.Tensor] = None, stream=None):
    """Gate and up products (weights E4M3 [E, 2I, K], gate rows first) with the
    gated SiLU; returns (out_rows, out_scales) of [rows, I] in ``out_quant``, as
    ep_expert_gemm takes them (bf16 and None for "none")."""
    lib = load_library()
    dev, c, cap, slab, N, K, px, ps, pw, pws = _expert_args(lib, layout, rows, row_scales, weights,
                                                            weight_scales, quant)
    if N % 256:
        raise EPError(EP_ERR_INVALID_ARG, "weights must have 2*I rows, I a multiple of 128")
    inter = N // 2
    if out_quant == "mxfp8":
        raise EPError(EP_ERR_UNSUPPORTED, "gated SiLU in mxfp8")
    plain = out_quant == "none"
    if out_rows is None:
        out_rows = _empty((cap, inter), _BF16 if plain else torch.uint8, dev, stream)
    po = _want(out_rows, "out_rows", (_BF16,) if plain else _E4M3, (cap, inter), dev)
    pos = None
    if not plain:
        sdt, sshape = _scale_shape(cap, inter, out_quant, slab)
        if out_scales is None:
            out_scales = _empty(sshape, sdt[0], dev, stream)
        pos = _want(out_scales, "out_scales", sdt, sshape, dev)
    elif out_scales is not None:
        raise ValueError('out_scales belong to an 8-bit out_quant, not "none"')
    _call(lib.ep_expert_swiglu, "ep_expert_swiglu", dev, ctypes.byref(c), px, ps, K, QUANT[quant],
          pw, pws, inter, QUANT[out_quant], po, pos, _on(stream, dev))
    return out_rows, out_scales


@dataclass
class MoeWorkspace:
    """Scratch and status word of ep_moe_decode calls that do not overlap."""

    scratch: torch.Tensor
    status: torch.Tensor

    def check_status(self) -> None:
        """Synchronise and raise EPError if the last call recorded a device-side error."""
        st = int(self.status.item())
        if st != EP_OK:
            raise EPError(st, "device status")


def ep_moe_decode_workspace_bytes(num_tokens: int, num_topk: int, num_experts: int, hidden: int,
                                  inter: int) -> int:
    return int(load_library().ep_moe_decode_workspace_bytes(num_tokens, num_topk, num_experts,
                                                            hidden, inter))


def _moe_scratch_bytes(dev, *shape) -> int:
    """ep_moe_decode_workspace_bytes for device `dev`: it depends on the number of SMs."""
    with torch.cuda.device(dev):
        return ep_moe_decode_workspace_bytes(*shape)


def new_moe_workspace(num_tokens: int, num_topk: int, num_experts: int, hidden: int, inter: int,
                      device=None) -> MoeWorkspace:
    """Allocate a workspace for ep_moe_decode calls of this shape, or of fewer tokens."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    n = _moe_scratch_bytes(dev, num_tokens, num_topk, num_experts, hidden, inter)
    if n == 0 and num_tokens > 0:
        raise EPError(EP_ERR_INVALID_ARG, "ep_moe_decode shape")
    return MoeWorkspace(torch.empty(max(n, 16), dtype=torch.uint8, device=dev),
                        torch.zeros(1, dtype=torch.int32, device=dev))


def ep_moe_decode(x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                  w13: torch.Tensor, w13_scales: torch.Tensor, w2: torch.Tensor,
                  w2_scales: torch.Tensor, workspace: Optional[MoeWorkspace] = None,
                  x_scales: Optional[torch.Tensor] = None, quant: str = "none",
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """A whole mixture-of-experts layer for a few tokens: bf16 [T, H].

    x is bf16 [T, H] (quant "none"), or E4M3 rows with x_scales as ep_rmsnorm
    writes them ("fp8_f32", "fp8_ue8m0").  w13 E4M3 [E, 2I, H] (gate rows
    first), w2 E4M3 [E, H, I], both with fp32 scales of their 128x128 blocks.
    A device-side error (a bad expert id) is left in workspace.status.
    """
    lib = load_library()
    dev = _rows_of(x, "x")
    shape = x.shape
    T, H = shape
    px = _want(x, "x", (_BF16,) if quant == "none" else _E4M3, shape, dev)
    _rows_of(topk_idx, "topk_idx")
    K = topk_idx.shape[1]
    pi = _want(topk_idx, "topk_idx", (_I32,), (T, K), dev)
    pw = _want(topk_w, "topk_w", (_F32,), (T, K), dev)
    _rows_of(w13, "w13", 3)
    E, R, _ = w13.shape
    if R % 256:
        raise EPError(EP_ERR_INVALID_ARG, "w13 must have 2*I rows, I a multiple of 128")
    inter = R // 2
    p13 = _want(w13, "w13", _E4M3, (E, R, H), dev)
    p2 = _want(w2, "w2", _E4M3, (E, H, inter), dev)
    ps13 = _want(w13_scales, "w13_scales", (_F32,), (E, R // 128, H // 128), dev)
    ps2 = _want(w2_scales, "w2_scales", (_F32,), (E, H // 128, inter // 128), dev)
    psx = None
    if quant != "none":
        sdt, sshape = _scale_shape(T, H, quant)
        psx = _want(x_scales, "x_scales", sdt, sshape, dev)
    elif x_scales is not None:
        raise ValueError("x_scales given for bf16 rows")
    if workspace is None:
        n = _moe_scratch_bytes(dev, T, K, E, H, inter)
        workspace = MoeWorkspace(_empty(max(n, 16), torch.uint8, dev, stream),
                                 _empty(1, _I32, dev, stream))
    ws = workspace.scratch
    nbytes = ws.numel()
    pws = _want(ws, "workspace.scratch", (torch.uint8,), (nbytes,), dev)
    pst = _want(workspace.status, "workspace.status", (_I32,), (1,), dev)
    if out is None:
        out = _empty(shape, _BF16, dev, stream)
    po = _want(out, "out", (_BF16,), shape, dev)
    _call(lib.ep_moe_decode, "ep_moe_decode", dev, px, psx, QUANT[quant], pi, pw, T, K, E, H, inter,
          p13, ps13, p2, ps2, po, pst, pws, nbytes, _on(stream, dev))
    return out
