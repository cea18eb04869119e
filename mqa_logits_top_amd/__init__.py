"""Python binding of libidx, the MI355X dense prefill indexer (MQA logits + top-K).

Argument marshalling only: every step of the indexer runs in the HIP kernels
behind the C ABI declared in include/idx.h.  PyTorch supplies device memory
(outputs and workspace are allocated here with torch when the caller passes
none) and the current HIP stream.  There is no fallback: if libidx.so is
missing or fails to load, every call raises.

Function names match the C entry points.  Tensors must be on the GPU and
contiguous; key indices in outputs are absolute rows of k.  The operators around
the indexer (idx_rope, idx_cache_write, idx_cache_read, idx_sparse_attn,
idx_paged_attn, idx_rms_norm) check types, shapes and devices here, and take any strides the C entry points take.
They record no gradient and refuse rows that require one while autograd is on.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libidx.so")

IDX_K_FP8_E4M3 = 0
IDX_K_MXFP4 = 1
IDX_K_BF16 = 2
IDX_K_F16 = 3
IDX_K_F32 = 4
IDX_ROPE_HALF = 0
IDX_ROPE_INTERLEAVED = 1
IDX_ROPE_PLAIN = 0
IDX_ROPE_LINEAR = 1
IDX_ROPE_BASE = 2
IDX_ROPE_PARTS = 3
IDX_MAX_WRITES = 8
IDX_OP_MQA_LOGITS = 0
IDX_OP_TOPK = 1
IDX_OP_LOGITS_TOPK_FUSED = 2
IDX_OP_BLOCK_CANDIDATES = 3
IDX_OP_BLOCK_CANDIDATES_DENSE = 4
IDX_OP_GATHER_ROWS = 5

STATUS = {0: "IDX_OK", 1: "IDX_E_NULL", 2: "IDX_E_SHAPE", 3: "IDX_E_PARAM", 4: "IDX_E_FORMAT",
          5: "IDX_E_WORKSPACE", 6: "IDX_E_UNSUPPORTED", 7: "IDX_E_LAUNCH", 8: "IDX_E_ALIGN", 9: "IDX_E_DEVICE_CHECK"}

EXPORTS = ("idx_mqa_logits", "idx_mqa_logits_block", "idx_topk", "idx_logits_topk_fused",
           "idx_logits_topk_fused_paged", "idx_logits_topk_fused_blocks", "idx_logits_topk_fused_static",
           "idx_refine_topk",
           "idx_block_candidates", "idx_workspace_size", "idx_ragged_windows", "idx_ragged_windows_ratio",
           "idx_gather_rows", "idx_tail_rows", "idx_rope_freqs", "idx_rope", "idx_cache_write", "idx_cache_read",
           "idx_sparse_attn_workspace", "idx_sparse_attn", "idx_paged_attn_workspace", "idx_paged_attn", "idx_rms_norm",
           "idx_launch_timing", "idx_launch_timing_read",
           "idx_status_str")

IDX_TIMING_MAX = 1024
LAUNCH_MODES = {0: "dense", 1: "block", 2: "pool8", 4: "slab"}


class IdxError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} ({status_str(status)})")


class idx_launch_time(ctypes.Structure):
    _fields_ = [("ms", ctypes.c_float), ("mode", ctypes.c_int32), ("flagged", ctypes.c_int32),
                ("row0", ctypes.c_int32), ("nrows", ctypes.c_int32), ("key0", ctypes.c_int32),
                ("nkeys", ctypes.c_int32)]


class idx_problem(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_scale", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("k_fmt", ctypes.c_int32), ("w", ctypes.c_void_p),
                ("ks", ctypes.c_void_p), ("ke", ctypes.c_void_p), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("D", ctypes.c_int32), ("L", ctypes.c_int32), ("scale", ctypes.c_float)]


class idx_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld_t", ctypes.c_int64), ("ld_h", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("D", ctypes.c_int32)]


class idx_rotary(ctypes.Structure):
    _fields_ = [("freq", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("rot", ctypes.c_int32),
                ("rot0", ctypes.c_int32), ("layout", ctypes.c_int32), ("inverse", ctypes.c_int32),
                ("mscale", ctypes.c_double)]


class idx_cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("ld_scale", ctypes.c_int64), ("fmt", ctypes.c_int32),
                ("H", ctypes.c_int32), ("D", ctypes.c_int32)]


class idx_write(ctypes.Structure):
    _fields_ = [("x", idx_rows), ("rotary", ctypes.POINTER(idx_rotary)), ("slot", ctypes.c_void_p),
                ("to", idx_cache)]


class idx_attn(ctypes.Structure):
    _fields_ = [("q", idx_rows), ("out", idx_rows), ("k", idx_cache), ("v", idx_cache), ("sel", ctypes.c_void_p),
                ("ld_sel", ctypes.c_int64), ("n_sel", ctypes.c_int32), ("pool", ctypes.c_int32),
                ("ks", ctypes.c_void_p), ("ke", ctypes.c_void_p), ("slot_of_key", ctypes.c_void_p),
                ("L", ctypes.c_int32), ("scale", ctypes.c_float), ("lse", ctypes.c_void_p)]


class idx_paged(ctypes.Structure):
    _fields_ = [("q", idx_rows), ("out", idx_rows), ("k", idx_cache), ("v", idx_cache), ("pages", ctypes.c_void_p),
                ("ld_pages", ctypes.c_int64), ("n_pages", ctypes.c_int32), ("page", ctypes.c_int32),
                ("cu_q", ctypes.c_void_p), ("len_k", ctypes.c_void_p), ("B", ctypes.c_int32),
                ("window", ctypes.c_int32), ("first", ctypes.c_int32), ("scale", ctypes.c_float),
                ("lse", ctypes.c_void_p)]


class idx_norm(ctypes.Structure):
    _fields_ = [("x", idx_rows), ("residual", idx_rows), ("total", idx_rows), ("out", idx_rows),
                ("to", ctypes.POINTER(idx_cache)), ("weight", ctypes.c_void_p), ("weight_dtype", ctypes.c_int32),
                ("eps", ctypes.c_float)]


_lib = None


def load_library():
    """Load libidx.so (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libidx is not built ({LIB_PATH} missing); run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P, VP = ctypes.POINTER(idx_problem), ctypes.c_void_p
    i32, i64, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.idx_mqa_logits.argtypes = [P, VP, i64, i32, VP]
    lib.idx_mqa_logits_block.argtypes = [P, i32, i32, i32, i32, VP, i64, VP]
    lib.idx_topk.argtypes = [VP, i64, i32, VP, VP, VP, i64, i32, i32, i32, VP, VP, VP, sz, VP]
    lib.idx_logits_topk_fused.argtypes = [P, i32, i32, i32, VP, i64, VP, VP, VP, sz, VP]
    lib.idx_logits_topk_fused_paged.argtypes = [P, i32, i32, i32, VP, i64, VP, VP, VP, VP, VP, sz, VP]
    lib.idx_logits_topk_fused_blocks.argtypes = [P, i32, i32, i32, VP, i64, i32, i32, VP, VP, VP, sz, VP]
    lib.idx_logits_topk_fused_static.argtypes = [P, i32, i32, i32, VP, i64, VP, VP, VP]
    lib.idx_refine_topk.argtypes = [P, VP, VP, i64, i32, i32, i32, VP, VP, VP, sz, VP]
    lib.idx_block_candidates.argtypes = [P, VP, i64, i32, i32, i32, i32, VP, i64, i32, VP, VP, sz, VP]
    lib.idx_workspace_size.argtypes = [i32, P, i32, i32, i32, i32, i32, i32, ctypes.POINTER(sz)]
    lib.idx_ragged_windows.argtypes = [VP, VP, i32, i32, VP, VP, VP]
    lib.idx_ragged_windows_ratio.argtypes = [VP, VP, VP, i32, i32, i32, VP, VP, VP]
    lib.idx_gather_rows.argtypes = [P, VP, i32, P, VP, sz, VP]
    lib.idx_tail_rows.argtypes = [VP, i32, i32, VP, VP]
    f64, pf64 = ctypes.c_double, ctypes.POINTER(ctypes.c_double)
    R, C = ctypes.POINTER(idx_rows), ctypes.POINTER(idx_cache)
    lib.idx_rope_freqs.argtypes = [i32, f64, i32, f64, f64, f64, f64, pf64, pf64]
    lib.idx_rope.argtypes = [R, ctypes.POINTER(idx_rotary), R, VP]
    lib.idx_cache_write.argtypes = [ctypes.POINTER(idx_write), i32, VP]
    lib.idx_cache_read.argtypes = [C, VP, R, VP]
    lib.idx_sparse_attn_workspace.argtypes = [ctypes.POINTER(idx_attn), ctypes.POINTER(sz)]
    lib.idx_sparse_attn.argtypes = [ctypes.POINTER(idx_attn), VP, sz, VP]
    lib.idx_paged_attn_workspace.argtypes = [ctypes.POINTER(idx_paged), ctypes.POINTER(sz)]
    lib.idx_paged_attn.argtypes = [ctypes.POINTER(idx_paged), VP, sz, VP]
    lib.idx_rms_norm.argtypes = [ctypes.POINTER(idx_norm), VP]
    lib.idx_launch_timing.argtypes = [i32]
    lib.idx_launch_timing_read.argtypes = [ctypes.POINTER(idx_launch_time), i32, ctypes.POINTER(i32)]
    lib.idx_status_str.argtypes = [i32]
    lib.idx_status_str.restype = ctypes.c_char_p
    for name in EXPORTS:
        if name != "idx_status_str":
            getattr(lib, name).restype = i32
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return load_library().idx_status_str(status).decode()


def _check(fn: str, status: int):
    if status != 0:
        raise IdxError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


@dataclass
class Inputs:
    """Device tensors of one indexer call (see include/idx.h, idx_problem)."""
    q: torch.Tensor        # uint8 [T, H, D]
    q_scale: torch.Tensor  # float32 [T, H]
    k: torch.Tensor        # uint8 [L, D] (fp8) or [L, D/2] (MXFP4)
    k_scale: torch.Tensor  # float32 [L] (fp8) or uint8 [L, D/32] (MXFP4)
    w: torch.Tensor        # float32 [T, H]
    ks: torch.Tensor       # int32 [T]
    ke: torch.Tensor       # int32 [T]
    k_fmt: int = IDX_K_FP8_E4M3
    scale: float = 1.0

    @property
    def T(self):
        return int(self.q.shape[0])

    @property
    def H(self):
        return int(self.q.shape[1])

    @property
    def L(self):
        return int(self.k.shape[0])

    def struct(self) -> idx_problem:
        return idx_problem(q=self.q.data_ptr(), q_scale=self.q_scale.data_ptr(), k=self.k.data_ptr(),
                           k_scale=self.k_scale.data_ptr(), k_fmt=self.k_fmt, w=self.w.data_ptr(),
                           ks=self.ks.data_ptr(), ke=self.ke.data_ptr(), T=self.T, H=self.H,
                           D=int(self.q.shape[2]), L=self.L, scale=self.scale)

    @property
    def W(self) -> int:
        """Longest row window (max_seqlen_k), read from the device windows."""
        return int((self.ke - self.ks).max().item()) if self.T else 0

    @property
    def pairs(self) -> int:
        """In-window (row, key) pairs, read from the device windows."""
        return int((self.ke.to(torch.int64) - self.ks).sum().item()) if self.T else 0

    @staticmethod
    def from_host(p, device="cuda") -> "Inputs":
        """Copy a host problem (numpy arrays with the same field names) to the device.  A problem
        without ks / ke gives its batch as cu_q / cu_k; the windows are then built on the device
        by idx_ragged_windows."""
        t = lambda a: torch.from_numpy(a).to(device)
        if getattr(p, "ks", None) is not None:
            ks, ke = t(p.ks), t(p.ke)
        else:
            ks, ke = idx_ragged_windows(t(p.cu_q), t(p.cu_k), int(p.q.shape[0]))
        return Inputs(q=t(p.q), q_scale=t(p.q_scale), k=t(p.k), k_scale=t(p.k_scale), w=t(p.w), ks=ks,
                      ke=ke, k_fmt=int(p.k_fmt), scale=float(p.scale))


def idx_workspace_size(op: int, p: Inputs, K: int = 0, block_k: int = 0, row_chunk: int = 0, pool: int = 0,
                       n_blocks: int = 0, W: int = 0) -> int:
    n = ctypes.c_size_t(0)
    s = p.struct()
    _check("idx_workspace_size",
           load_library().idx_workspace_size(op, ctypes.byref(s), K, block_k, row_chunk, pool, n_blocks, W,
                                             ctypes.byref(n)))
    return n.value


def _workspace(nbytes: int, device) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def idx_mqa_logits(p: Inputs, W: Optional[int] = None, out: Optional[torch.Tensor] = None, stream=None):
    """Dense row-relative logits [T, W] fp32 (-inf past each row's window)."""
    if W is None:
        W = int((p.ke - p.ks).max().item()) if p.T else 0
    if out is None:
        out = torch.empty((p.T, W), dtype=torch.float32, device=p.q.device)
    s = p.struct()
    _check("idx_mqa_logits", load_library().idx_mqa_logits(ctypes.byref(s), _ptr(out), out.stride(0), W,
                                                           _stream(stream)))
    return out


def idx_mqa_logits_block(p: Inputs, row0: int, nrows: int, key0: int, nkeys: int,
                         out: Optional[torch.Tensor] = None, stream=None):
    """Logits of rows [row0, row0+nrows) x keys [key0, key0+nkeys) (in-window entries only)."""
    if out is None:
        out = torch.full((nrows, nkeys), float("nan"), dtype=torch.float32, device=p.q.device)
    s = p.struct()
    _check("idx_mqa_logits_block",
           load_library().idx_mqa_logits_block(ctypes.byref(s), row0, nrows, key0, nkeys, _ptr(out), out.stride(0),
                                               _stream(stream)))
    return out


def idx_topk(logits: torch.Tensor, ks: torch.Tensor, ke: torch.Tensor, K: int, W: Optional[int] = None,
             block_k: int = 0, mask: Optional[torch.Tensor] = None, out_idx: Optional[torch.Tensor] = None,
             out_val: Optional[torch.Tensor] = None, with_values: bool = True, stream=None):
    T = int(logits.shape[0])
    W = int(logits.shape[1]) if W is None else W
    dev = logits.device
    if out_idx is None:
        out_idx = torch.empty((T, K), dtype=torch.int32, device=dev)
    if out_val is None and with_values:
        out_val = torch.empty((T, K), dtype=torch.float32, device=dev)
    _check("idx_topk", load_library().idx_topk(
        _ptr(logits), logits.stride(0), W, _ptr(ks), _ptr(ke), _ptr(mask), mask.stride(0) if mask is not None else 0,
        T, K, block_k, _ptr(out_idx), _ptr(out_val), None, 0, _stream(stream)))
    return out_idx, out_val


def idx_logits_topk_fused(p: Inputs, K: int, block_k: int = 32768, row_chunk: int = 0,
                          mask: Optional[torch.Tensor] = None, out_idx: Optional[torch.Tensor] = None,
                          out_val: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                          with_values: bool = True, stream=None):
    dev = p.q.device
    if out_idx is None:
        out_idx = torch.empty((p.T, K), dtype=torch.int32, device=dev)
    if out_val is None and with_values:
        out_val = torch.empty((p.T, K), dtype=torch.float32, device=dev)
    if ws is None:
        ws = _workspace(idx_workspace_size(IDX_OP_LOGITS_TOPK_FUSED, p, K=K, block_k=block_k, row_chunk=row_chunk),
                        dev)
    s = p.struct()
    _check("idx_logits_topk_fused", load_library().idx_logits_topk_fused(
        ctypes.byref(s), K, block_k, row_chunk, _ptr(mask), mask.stride(0) if mask is not None else 0,
        _ptr(out_idx), _ptr(out_val), _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream)))
    return out_idx, out_val


def idx_logits_topk_fused_paged(p: Inputs, K: int, slot_of_key: torch.Tensor, block_k: int = 32768,
                                row_chunk: int = 0, mask: Optional[torch.Tensor] = None,
                                out_idx: Optional[torch.Tensor] = None, out_val: Optional[torch.Tensor] = None,
                                out_slot: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                                with_values: bool = True, stream=None):
    """idx_logits_topk_fused plus out_slot = slot_of_key[out_idx] (-1 pads), in the same final write."""
    dev = p.q.device
    if out_idx is None:
        out_idx = torch.empty((p.T, K), dtype=torch.int32, device=dev)
    if out_val is None and with_values:
        out_val = torch.empty((p.T, K), dtype=torch.float32, device=dev)
    if out_slot is None:
        out_slot = torch.empty((p.T, K), dtype=torch.int32, device=dev)
    if ws is None:
        ws = _workspace(idx_workspace_size(IDX_OP_LOGITS_TOPK_FUSED, p, K=K, block_k=block_k, row_chunk=row_chunk),
                        dev)
    s = p.struct()
    _check("idx_logits_topk_fused_paged", load_library().idx_logits_topk_fused_paged(
        ctypes.byref(s), K, block_k, row_chunk, _ptr(mask), mask.stride(0) if mask is not None else 0,
        _ptr(slot_of_key), _ptr(out_idx), _ptr(out_val), _ptr(out_slot), _ptr(ws),
        ws.numel() if ws is not None else 0, _stream(stream)))
    return out_idx, out_val, out_slot


def idx_logits_topk_fused_blocks(p: Inputs, K: int, blocks: torch.Tensor, pool: int = 8, block_k: int = 32768,
                                 row_chunk: int = 0, out_idx: Optional[torch.Tensor] = None,
                                 out_val: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                                 with_values: bool = True, stream=None):
    """idx_logits_topk_fused restricted to the candidate blocks blocks[t] ([T, n_blocks], -1 ignored)."""
    dev = p.q.device
    if out_idx is None:
        out_idx = torch.empty((p.T, K), dtype=torch.int32, device=dev)
    if out_val is None and with_values:
        out_val = torch.empty((p.T, K), dtype=torch.float32, device=dev)
    if ws is None:
        ws = _workspace(idx_workspace_size(IDX_OP_LOGITS_TOPK_FUSED, p, K=K, block_k=block_k, row_chunk=row_chunk),
                        dev)
    s = p.struct()
    _check("idx_logits_topk_fused_blocks", load_library().idx_logits_topk_fused_blocks(
        ctypes.byref(s), K, block_k, row_chunk, _ptr(blocks), blocks.stride(0), int(blocks.shape[1]), pool,
        _ptr(out_idx), _ptr(out_val), _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream)))
    return out_idx, out_val


STATIC_WS_BYTES = 128 << 20   # IDX_STATIC_WS_BYTES


def idx_logits_topk_fused_static(p: Inputs, K: int, block_k: int = 32768, row_chunk: int = 0,
                                 mask: Optional[torch.Tensor] = None, out_idx: Optional[torch.Tensor] = None,
                                 out_val: Optional[torch.Tensor] = None, with_values: bool = True, stream=None):
    """idx_logits_topk_fused on the library's static workspace: no workspace argument, and the
    library allocates nothing (the outputs are the caller's; they are allocated here only when
    not given)."""
    dev = p.q.device
    if out_idx is None:
        out_idx = torch.empty((p.T, K), dtype=torch.int32, device=dev)
    if out_val is None and with_values:
        out_val = torch.empty((p.T, K), dtype=torch.float32, device=dev)
    s = p.struct()
    _check("idx_logits_topk_fused_static", load_library().idx_logits_topk_fused_static(
        ctypes.byref(s), K, block_k, row_chunk, _ptr(mask), mask.stride(0) if mask is not None else 0,
        _ptr(out_idx), _ptr(out_val), _stream(stream)))
    return out_idx, out_val


RESERVE = 512   # extra candidates the exact boundary refinement keeps per row
REFINE_WS = 2304


def candidate_capacity(K: int) -> int:
    return min(K + RESERVE, 2560)


def idx_refine_topk(p: Inputs, cand_idx: torch.Tensor, cand_val: torch.Tensor, K: int, pool: int = 1,
                    out_idx: Optional[torch.Tensor] = None, out_val: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None, with_values: bool = True, stream=None):
    dev = cand_idx.device
    T, Kc = int(cand_idx.shape[0]), int(cand_idx.shape[1])
    if out_idx is None:
        out_idx = torch.empty((T, K), dtype=torch.int32, device=dev)
    if out_val is None and with_values:
        out_val = torch.empty((T, K), dtype=torch.float32, device=dev)
    if ws is None:
        ws = _workspace(REFINE_WS, dev)
    s = p.struct()
    _check("idx_refine_topk", load_library().idx_refine_topk(
        ctypes.byref(s), _ptr(cand_idx), _ptr(cand_val), cand_idx.stride(0), Kc, K, pool, _ptr(out_idx),
        _ptr(out_val), _ptr(ws), ws.numel(), _stream(stream)))
    return out_idx, out_val


def overflow_count(ws: torch.Tensor) -> int:
    """Rows of the last call on this workspace whose candidate list could not settle the boundary."""
    return int(ws[:4].view(torch.int32).item())


def idx_block_candidates(p: Inputs, W: int, pool: int = 8, n_blocks: int = 2048,
                         logits: Optional[torch.Tensor] = None, block_k: int = 32768, row_chunk: int = 0,
                         mask: Optional[torch.Tensor] = None, out_blocks: Optional[torch.Tensor] = None,
                         ws: Optional[torch.Tensor] = None, stream=None):
    dev = p.ks.device
    if mask is None:
        mask = torch.empty((p.T, W), dtype=torch.uint8, device=dev)
    op = IDX_OP_BLOCK_CANDIDATES_DENSE if logits is not None else IDX_OP_BLOCK_CANDIDATES
    if ws is None:
        ws = _workspace(idx_workspace_size(op, p, block_k=block_k, row_chunk=row_chunk, pool=pool,
                                           n_blocks=n_blocks, W=W), dev)
    s = p.struct()
    _check("idx_block_candidates", load_library().idx_block_candidates(
        ctypes.byref(s), _ptr(logits), logits.stride(0) if logits is not None else 0, pool, n_blocks, block_k,
        row_chunk, _ptr(mask), mask.stride(0), W, _ptr(out_blocks), _ptr(ws), ws.numel() if ws is not None else 0,
        _stream(stream)))
    return mask, out_blocks


def idx_ragged_windows(cu_q: torch.Tensor, cu_k: torch.Tensor, T: int, stream=None):
    B = int(cu_q.numel()) - 1
    ks = torch.empty(T, dtype=torch.int32, device=cu_q.device)
    ke = torch.empty(T, dtype=torch.int32, device=cu_q.device)
    _check("idx_ragged_windows", load_library().idx_ragged_windows(_ptr(cu_q), _ptr(cu_k), B, T, _ptr(ks), _ptr(ke),
                                                                   _stream(stream)))
    return ks, ke


def idx_ragged_windows_ratio(cu_q: torch.Tensor, cu_k: torch.Tensor, cu_c: torch.Tensor, ratio: int, T: int,
                             stream=None):
    """Windows over keys compressed `ratio` tokens to one (cu_c: key rows per request)."""
    B = int(cu_q.numel()) - 1
    ks = torch.empty(T, dtype=torch.int32, device=cu_q.device)
    ke = torch.empty(T, dtype=torch.int32, device=cu_q.device)
    _check("idx_ragged_windows_ratio", load_library().idx_ragged_windows_ratio(
        _ptr(cu_q), _ptr(cu_k), _ptr(cu_c), ratio, B, T, _ptr(ks), _ptr(ke), _stream(stream)))
    return ks, ke


def idx_gather_rows(p: Inputs, rows: torch.Tensor, ws: Optional[torch.Tensor] = None, stream=None) -> Inputs:
    """The problem restricted to rows[r] (-1: padding row).  The returned Inputs' row tensors
    are views of ws (the copies idx_gather_rows made); keys are shared with p."""
    R = int(rows.numel())
    if ws is None:
        ws = _workspace(idx_workspace_size(IDX_OP_GATHER_ROWS, p, K=R), p.q.device)
    s, out = p.struct(), idx_problem()
    _check("idx_gather_rows", load_library().idx_gather_rows(ctypes.byref(s), _ptr(rows), R, ctypes.byref(out),
                                                             _ptr(ws), ws.numel() if ws is not None else 0,
                                                             _stream(stream)))
    H, D = p.H, int(p.q.shape[2])

    def view(ptr, nbytes, dtype, shape):   # the array the C call placed at ptr inside ws
        if R == 0:
            return torch.empty(shape, dtype=dtype, device=p.q.device)
        o = ptr - ws.data_ptr()
        return ws[o:o + nbytes].view(dtype).view(shape)

    return Inputs(q=view(out.q, R * H * D, torch.uint8, (R, H, D)),
                  q_scale=view(out.q_scale, R * H * 4, torch.float32, (R, H)), k=p.k, k_scale=p.k_scale,
                  w=view(out.w, R * H * 4, torch.float32, (R, H)), ks=view(out.ks, R * 4, torch.int32, (R,)),
                  ke=view(out.ke, R * 4, torch.int32, (R,)), k_fmt=p.k_fmt, scale=p.scale)


def idx_tail_rows(cu_q: torch.Tensor, n: int, stream=None) -> torch.Tensor:
    """The last n rows of every request ([B * n], -1 where a request is shorter)."""
    B = int(cu_q.numel()) - 1
    rows = torch.empty(B * n, dtype=torch.int32, device=cu_q.device)
    _check("idx_tail_rows", load_library().idx_tail_rows(_ptr(cu_q), B, n, _ptr(rows), _stream(stream)))
    return rows


def idx_launch_timing(enable: bool) -> None:
    """Start (clearing the record) or stop recording the scoring launches' HIP event times."""
    _check("idx_launch_timing", load_library().idx_launch_timing(1 if enable else 0))


def idx_launch_timing_read() -> list:
    """The recorded launches, in launch order, as dicts (ms < 0: the launch failed); clears the
    record."""
    buf = (idx_launch_time * IDX_TIMING_MAX)()
    n = ctypes.c_int32()
    _check("idx_launch_timing_read", load_library().idx_launch_timing_read(buf, IDX_TIMING_MAX, ctypes.byref(n)))
    return [{"ms": e.ms, "mode": LAUNCH_MODES.get(e.mode, e.mode), "flagged": bool(e.flagged), "row0": e.row0,
             "nrows": e.nrows, "key0": e.key0, "nkeys": e.nkeys} for e in buf[:min(n.value, IDX_TIMING_MAX)]]


def idx_status_str(status: int) -> str:
    return status_str(status)


# ---- around the indexer: rotary positions, quantised caches, attention over the selection ----

_VALUE = {torch.bfloat16: IDX_K_BF16, torch.float16: IDX_K_F16, torch.float32: IDX_K_F32}
_STORED = {IDX_K_FP8_E4M3: torch.uint8, IDX_K_MXFP4: torch.uint8, IDX_K_BF16: torch.bfloat16,
           IDX_K_F16: torch.float16, IDX_K_F32: torch.float32}


def _on(t: torch.Tensor, device, dtype, what: str) -> int:
    """The tensor's address, if it is one the kernels can read as it stands."""
    if t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous {dtype} tensor on {device}, got {t.dtype} on {t.device}"
                         f"{'' if t.is_contiguous() else ', not contiguous'}")
    return t.data_ptr()


def _rows(x: torch.Tensor, what: str) -> idx_rows:
    if x.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{what} requires a gradient, and no entry point records one: call it under torch.no_grad() "
                         "or on x.detach() (idx_rope's gradient is idx_rope with inverse=True)")
    dtype, shape, ld = _VALUE.get(x.dtype), x.shape, x.stride()
    if dtype is None or not x.is_cuda or len(shape) != 3 or (ld[2] != 1 and shape[2] > 1):
        raise ValueError(f"{what}: [T, H, D] bfloat16, float16 or float32 on the GPU with a contiguous last "
                         f"dimension, got {list(shape)} {x.dtype} on {x.device}, strides {ld}")
    return idx_rows(x.data_ptr(), ld[0], ld[1], dtype, *shape)


def _new_rows(x: torch.Tensor, dtype: int, T: int, H: int, D: int) -> idx_rows:
    """Of a tensor just allocated with these sizes."""
    return idx_rows(x.data_ptr(), H * D, D, dtype, T, H, D)


def _new_like(x: torch.Tensor) -> torch.Tensor:
    """Contiguous, with x's sizes and type.  (empty_like keeps x's strides; it takes the host 0.6 us less.)"""
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


class _on_stream:
    """The calls below run on the stream given, or on the current stream of the tensors' device: outputs and
    workspaces allocated inside belong to it.  Where that is the current stream already, there is nothing to
    set (guard is None) and only its handle is looked up."""

    __slots__ = ("guard", "handle")

    def __init__(self, device: torch.device, stream):
        if stream is None:
            self.guard = None if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)
            self.handle = torch._C._cuda_getCurrentRawStream(device.index)
        else:
            if stream.device != device:
                raise ValueError(f"a stream of {stream.device} for tensors on {device}")
            self.guard, self.handle = torch.cuda.stream(stream), stream.cuda_stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def idx_rope_freqs(rot: int, base: float = 10000.0, scaling: int = IDX_ROPE_PLAIN, factor: float = 1.0,
                   original: float = 1.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """Pair frequencies (a CPU float64 tensor [rot / 2]) and the gain that goes with them."""
    out, gain = (ctypes.c_double * max(rot // 2, 1))(), ctypes.c_double()
    _check("idx_rope_freqs", load_library().idx_rope_freqs(rot, base, scaling, factor, original, beta_fast, beta_slow,
                                                           out, ctypes.byref(gain)))
    return torch.tensor(list(out), dtype=torch.float64), gain.value


class Rotary:
    """Rotary positions of dims [rot0, rot0 + 2 len(freq)) of a head; keep one and pass it to every call."""

    def __init__(self, freq: torch.Tensor, rot0: int = 0, layout: int = IDX_ROPE_HALF, mscale: float = 1.0):
        if not freq.is_cuda or freq.dim() != 1:
            raise ValueError(f"freq: one dimension, on the GPU, got {list(freq.shape)} on {freq.device}")
        self._freq, self.rot0, self.layout, self.mscale = freq, rot0, layout, mscale
        self.device = freq.device
        self._args = (_on(freq, freq.device, torch.float64, "freq"), 2 * int(freq.numel()), rot0, layout, mscale)

    @property
    def freq(self) -> torch.Tensor:
        return self._freq

    @staticmethod
    def make(rot: int, device="cuda", rot0: int = 0, layout: int = IDX_ROPE_HALF, **scaling) -> "Rotary":
        """From idx_rope_freqs's arguments."""
        freq, mscale = idx_rope_freqs(rot, **scaling)
        return Rotary(freq.to(device), rot0=rot0, layout=layout, mscale=mscale)

    def struct(self, pos: torch.Tensor, x: torch.Tensor, inverse: bool = False) -> idx_rotary:
        freq, rot, rot0, layout, mscale = self._args
        if pos is None or pos.shape != x.shape[:1]:
            raise ValueError("pos: [T], one position a row")
        if self.device != x.device:
            raise ValueError(f"a Rotary on {self.device} for rows on {x.device}")
        return idx_rotary(freq, _on(pos, self.device, torch.int32, "pos"), rot, rot0, layout, inverse, mscale)


class Cache:
    """A cache of slots of H heads of D values (include/idx.h, idx_cache); keep one and pass it to
    every call.  data: [slots, H, D] of the format's type, MXFP4 uint8 [slots, H, D / 2]; scale:
    float32 [slots, H] for E4M3, uint8 [slots, H, D / 32] for MXFP4, else None.  A head's values
    follow each other, and so do a slot's heads; slots may be further apart."""

    def __init__(self, data: torch.Tensor, scale: Optional[torch.Tensor] = None, D: Optional[int] = None,
                 fmt: int = IDX_K_FP8_E4M3):
        if fmt not in _STORED:
            raise ValueError(f"unknown cache format {fmt}")
        if not data.is_cuda or data.dim() != 3 or data.dtype != _STORED[fmt]:
            raise ValueError(f"cache data: [slots, H, D] {_STORED[fmt]} on the GPU, got {list(data.shape)} "
                             f"{data.dtype} on {data.device}")
        rows, H, width = data.shape
        D = width * (2 if fmt == IDX_K_MXFP4 else 1) if D is None else D
        if width != (D // 2 if fmt == IDX_K_MXFP4 else D):
            raise ValueError(f"cache data: {width} wide for D = {D}")
        if (width > 1 and data.stride(2) != 1) or (H > 1 and data.stride(1) != width):
            raise ValueError(f"cache data: a slot's heads, and a head's values, follow each other; strides "
                             f"{data.stride()}")
        ld_scale, shape = 0, {IDX_K_FP8_E4M3: (rows, H), IDX_K_MXFP4: (rows, H, D // 32)}.get(fmt)
        if shape is None:
            if scale is not None:
                raise ValueError("a 16- or 32-bit cache has no scale")
        else:
            want = torch.float32 if fmt == IDX_K_FP8_E4M3 else torch.uint8
            if scale is None or scale.device != data.device or scale.dtype != want or tuple(scale.shape) != shape:
                raise ValueError(f"cache scale: {list(shape)} {want} on {data.device}")
            if rows and not scale[:1].is_contiguous():
                raise ValueError(f"cache scale: a slot's scales follow each other; strides {scale.stride()}")
            ld_scale = scale.stride(0)
        self._data, self._scale, self.fmt, self.D = data, scale, fmt, D
        self.rows, self.H, self.device = rows, H, data.device
        ld = data.stride(0) * (2 if fmt == IDX_K_MXFP4 else 1)
        self._struct = idx_cache(data.data_ptr(), None if scale is None else scale.data_ptr(), rows, ld, ld_scale,
                                 fmt, H, D)

    @staticmethod
    def empty(rows: int, H: int, D: int, fmt: int = IDX_K_FP8_E4M3, device="cuda") -> "Cache":
        """A cache of zeros."""
        if fmt not in _STORED:
            raise ValueError(f"unknown cache format {fmt}")
        data = torch.zeros((rows, H, D // 2 if fmt == IDX_K_MXFP4 else D), dtype=_STORED[fmt], device=device)
        scale = None
        if fmt == IDX_K_FP8_E4M3:
            scale = torch.ones((rows, H), dtype=torch.float32, device=device)
        elif fmt == IDX_K_MXFP4:
            scale = torch.zeros((rows, H, D // 32), dtype=torch.uint8, device=device)
        return Cache(data, scale, D=D, fmt=fmt)

    # the tensors of a handle stay the ones its struct points to
    @property
    def data(self) -> torch.Tensor:
        return self._data

    @property
    def scale(self) -> Optional[torch.Tensor]:
        return self._scale

    def struct(self) -> idx_cache:
        return self._struct


@dataclass
class Write:
    """One array of rows [T, H, D] on its way into a cache (include/idx.h, idx_write)."""
    x: torch.Tensor
    cache: Cache
    slot: Optional[torch.Tensor] = None     # int32 [T]; None: row t to slot t
    rotary: Optional[Rotary] = None
    pos: Optional[torch.Tensor] = None      # int32 [T], with a rotary
    inverse: bool = False


def idx_rope(x: torch.Tensor, pos: torch.Tensor, rotary: Rotary, out: Optional[torch.Tensor] = None,
             inverse: bool = False, stream=None) -> torch.Tensor:
    """x [T, H, D] rotated to positions pos [T]; out may be x."""
    rows, r = _rows(x, "x"), rotary.struct(pos, x, inverse)
    device = rotary.device
    with _on_stream(device, stream) as st:
        if out is None:
            out = x.new_empty(x.shape)
            to = _new_rows(out, rows.dtype, *x.shape)
        elif out.device != device:
            raise ValueError(f"out on {out.device} for x on {device}")
        else:
            to = _rows(out, "out")
        s = load_library().idx_rope(rows, r, to, st)
    if s:
        raise IdxError("idx_rope", s)
    return out


def idx_cache_write(writes, stream=None) -> None:
    """Rotate (where asked), quantise and store every Write's rows, in one launch."""
    n = len(writes)
    if n > IDX_MAX_WRITES:
        raise ValueError(f"{n} writes in a call, at most {IDX_MAX_WRITES}")
    if n == 0:
        return
    device = writes[0].cache.device
    args, keep = (idx_write * n)(), []
    for a, w in zip(args, writes):
        x, cache = w.x, w.cache
        a.x, a.to = _rows(x, "x"), cache._struct
        if x.device != device or cache.device != device:
            raise ValueError("every row array and cache of a call on one device")
        if w.rotary is not None:
            keep.append(w.rotary.struct(w.pos, x, w.inverse))
            a.rotary = ctypes.pointer(keep[-1])
        elif w.pos is not None:
            raise ValueError("pos without a rotary")
        if w.slot is not None:
            if w.slot.shape != x.shape[:1]:
                raise ValueError("slot: [T], one slot a row")
            a.slot = _on(w.slot, device, torch.int32, "slot")
    with _on_stream(device, stream) as st:
        s = load_library().idx_cache_write(args, n, st)
    if s:
        raise IdxError("idx_cache_write", s)


def idx_cache_read(cache: Cache, rows: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """Values [N, H, D] of the slots rows [N] (None: every slot in order); zeros for a slot outside the cache."""
    device, at, n = cache.device, None, cache.rows
    if rows is not None:
        if rows.dim() != 1:
            raise ValueError("rows: one dimension")
        at, n = _on(rows, device, torch.int32, "rows"), rows.shape[0]
    with _on_stream(device, stream) as st:
        if out is None:
            if dtype not in _VALUE:
                raise ValueError(f"dtype: bfloat16, float16 or float32, got {dtype}")
            out = cache._data.new_empty((n, cache.H, cache.D), dtype=dtype)
            to = _new_rows(out, _VALUE[dtype], n, cache.H, cache.D)
        elif out.device != device or out.shape[0] != n:
            raise ValueError(f"out: {n} rows on {device}")
        else:
            to = _rows(out, "out")
        s = load_library().idx_cache_read(cache._struct, at, to, st)
    if s:
        raise IdxError("idx_cache_read", s)
    return out


def idx_sparse_attn(q: torch.Tensor, k: Cache, v: Cache, sel: torch.Tensor, scale: float, pool: int = 1,
                    ks: Optional[torch.Tensor] = None, ke: Optional[torch.Tensor] = None,
                    slot_of_key: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, with_lse: bool = True,
                    stream=None):
    """Attention of q [T, Hq, D] over the keys (pool 1) or blocks of keys that sel [T, n] lists; (out, lse)."""
    device, rows = k.device, _rows(q, "q")
    T, Hq = rows.T, rows.H
    if q.device != device or v.device != device:
        raise ValueError(f"caches on {k.device} and {v.device} for q on {q.device}")
    if (sel.dtype is not torch.int32 or sel.device != device or sel.dim() != 2 or sel.shape[0] != T
            or (sel.stride(1) != 1 and sel.shape[1] > 1)):
        raise ValueError(f"sel: [T, n] int32 on {device} with a contiguous last dimension, got {list(sel.shape)} "
                         f"{sel.dtype} on {sel.device}")
    a_ks = a_ke = table = None
    L = k.rows
    if ks is not None or ke is not None:
        if ks is None or ke is None or ks.shape != (T,) or ke.shape != (T,):
            raise ValueError("ks and ke: [T] both")
        a_ks, a_ke = _on(ks, device, torch.int32, "ks"), _on(ke, device, torch.int32, "ke")
    if slot_of_key is not None:
        if slot_of_key.dim() != 1:
            raise ValueError("slot_of_key: one dimension")
        L, table = slot_of_key.shape[0], _on(slot_of_key, device, torch.int32, "slot_of_key")
    lib = load_library()
    with _on_stream(device, stream) as st:
        if out is None:
            out = q.new_empty(q.shape)
            to = _new_rows(out, rows.dtype, *q.shape)
        elif out.device != device:
            raise ValueError(f"out on {out.device} for q on {device}")
        else:
            to = _rows(out, "out")
        if lse is None:
            if with_lse:
                lse = q.new_empty((T, Hq), dtype=torch.float32)
        elif lse.shape != (T, Hq):
            raise ValueError(f"lse: {[T, Hq]}")
        a = idx_attn(rows, to, k._struct, v._struct, sel.data_ptr(), sel.stride(0), sel.shape[1], pool,
                     a_ks, a_ke, table, L, scale, None if lse is None else _on(lse, device, torch.float32, "lse"))
        at, size = None, 0
        if ws is None:
            need = ctypes.c_size_t()
            s = lib.idx_sparse_attn_workspace(a, need)
            if s:
                raise IdxError("idx_sparse_attn_workspace", s)
            size = need.value
            if size:
                ws = torch.empty(size, dtype=torch.uint8, device=device)
        else:
            size = ws.numel()
        if ws is not None:
            at = _on(ws, device, torch.uint8, "ws")
        s = lib.idx_sparse_attn(a, at, size, st)
    if s:
        raise IdxError("idx_sparse_attn", s)
    return out, lse


def idx_paged_attn(q: torch.Tensor, k: Cache, v: Cache, pages: torch.Tensor, cu_q: torch.Tensor, len_k: torch.Tensor,
                   scale: float, page: int, window: int = 0, first: int = 0, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, with_lse: bool = True,
                   stream=None):
    """Attention of the new rows q [T, Hq, D] of a batch over the keys of their requests, or over the last `window`
    and the `first` of them; (out, lse).  Request b has the rows cu_q[b] .. cu_q[b + 1] - 1, the last of its len_k[b]
    keys, which lie in the slots pages[b] names, `page` to a page."""
    device, rows = k.device, _rows(q, "q")
    T, Hq = rows.T, rows.H
    if q.device != device or v.device != device:
        raise ValueError(f"caches on {k.device} and {v.device} for q on {q.device}")
    if (pages.dtype is not torch.int32 or pages.device != device or pages.dim() != 2
            or (pages.stride(1) != 1 and pages.shape[1] > 1)):
        raise ValueError(f"pages: [B, n] int32 on {device} with a contiguous last dimension, got {list(pages.shape)} "
                         f"{pages.dtype} on {pages.device}")
    if not (0 <= page < 1 << 31 and 0 <= window < 1 << 31 and 0 <= first < 1 << 31):
        raise ValueError(f"page, window and first from 0 to 2^31 - 1, got {page}, {window}, {first}")
    B = pages.shape[0]
    if cu_q.shape != (B + 1,) or len_k.shape != (B,):
        raise ValueError(f"cu_q: [{B + 1}] and len_k: [{B}] for {B} rows of pages, got {list(cu_q.shape)} and "
                         f"{list(len_k.shape)}")
    a_cu, a_len = _on(cu_q, device, torch.int32, "cu_q"), _on(len_k, device, torch.int32, "len_k")
    lib = load_library()
    with _on_stream(device, stream) as st:
        if out is None:
            out = _new_like(q)
            to = _new_rows(out, rows.dtype, *q.shape)
        elif out.device != device:
            raise ValueError(f"out on {out.device} for q on {device}")
        else:
            to = _rows(out, "out")
        if lse is None:
            if with_lse:
                lse = q.new_empty((T, Hq), dtype=torch.float32)
        elif lse.shape != (T, Hq):
            raise ValueError(f"lse: {[T, Hq]}")
        a = idx_paged(rows, to, k._struct, v._struct, pages.data_ptr(), pages.stride(0), pages.shape[1], page, a_cu, a_len,
                      B, window, first, scale, None if lse is None else _on(lse, device, torch.float32, "lse"))
        at, size = None, 0
        if ws is None:
            need = ctypes.c_size_t()
            s = lib.idx_paged_attn_workspace(a, need)
            if s:
                raise IdxError("idx_paged_attn_workspace", s)
            size = need.value
            if size:
                ws = torch.empty(size, dtype=torch.uint8, device=device)
        else:
            size = ws.numel()
        if ws is not None:
            at = _on(ws, device, torch.uint8, "ws")
        s = lib.idx_paged_attn(a, at, size, st)
    if s:
        raise IdxError("idx_paged_attn", s)
    return out, lse


def _norm_rows(x: torch.Tensor, what: str) -> idx_rows:
    """Rows [T, H, D], or hidden rows [T, D] as one head."""
    if x.dim() != 2:
        return _rows(x, what)
    if x.requires_grad and torch.is_grad_enabled():
        return _rows(x.unsqueeze(1), what)          # refuses them
    dtype, (T, D), ld = _VALUE.get(x.dtype), x.shape, x.stride()
    if dtype is None or not x.is_cuda or (ld[1] != 1 and D > 1):
        raise ValueError(f"{what}: [T, D] or [T, H, D] bfloat16, float16 or float32 on the GPU with a contiguous last "
                         f"dimension, got {[T, D]} {x.dtype} on {x.device}, strides {ld}")
    return idx_rows(x.data_ptr(), ld[0], D, dtype, T, 1, D)


def idx_rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 residual: Optional[torch.Tensor] = None, total: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, to: Optional[Cache] = None, with_out: bool = True, stream=None):
    """RMS norm of each row of x [T, D], or of each head of x [T, H, D], times weight [D]; returns out (None where
    with_out is False).  residual: added before the norm, the sum written to `total`, or to the residual itself where that
    is None.  to: an E4M3 cache of T slots or more that receives the result with a scale for each of its heads, which for
    x [T, D] may be groups of D."""
    rows, device, shape = _norm_rows(x, "x"), x.device, x.shape
    n = idx_norm()
    n.x, n.eps, n.weight_dtype = rows, eps, IDX_K_F32
    if residual is not None:
        if residual.shape != shape or residual.device != device:
            raise ValueError(f"residual: {list(shape)} on {device} as x, got {list(residual.shape)} on {residual.device}")
        n.residual = r = _norm_rows(residual, "residual")
        if total is None or total is residual:
            n.total = r
        elif total.shape != shape or total.device != device:
            raise ValueError(f"total: {list(shape)} on {device} as x, got {list(total.shape)} on {total.device}")
        else:
            n.total = _norm_rows(total, "total")
    elif total is not None:
        raise ValueError("total without a residual")
    if weight is not None:
        if weight.requires_grad and torch.is_grad_enabled():
            raise ValueError("weight requires a gradient, and no entry point records one: call it under torch.no_grad() "
                             "or on weight.detach()")
        if weight.shape != shape[-1:] or weight.dtype not in _VALUE:
            raise ValueError(f"weight: {list(shape[-1:])} bfloat16, float16 or float32, got {list(weight.shape)} "
                             f"{weight.dtype}")
        n.weight, n.weight_dtype = _on(weight, device, weight.dtype, "weight"), _VALUE[weight.dtype]
    if to is not None:
        if to.device != device:
            raise ValueError(f"a cache on {to.device} for x on {device}")
        n.to = ctypes.pointer(to._struct)
    with _on_stream(device, stream) as st:
        if out is not None:
            if out.device != device or out.shape != shape:
                raise ValueError(f"out: {list(shape)} on {device}, got {list(out.shape)} on {out.device}")
            n.out = _norm_rows(out, "out")
        elif with_out:
            out = _new_like(x)
            n.out = _new_rows(out, rows.dtype, rows.T, rows.H, rows.D)
        s = load_library().idx_rms_norm(n, st)
    if s:
        raise IdxError("idx_rms_norm", s)
    return out
