"""ctypes binding of libsge.so: argument marshalling only.

Each function has the name of the C entry point it calls and takes torch
tensors on a CUDA device; outputs not given are allocated with torch (device
memory is the only thing PyTorch provides here) and returned.  Launches go on
the current torch stream of the tensors' device unless ``stream`` is given.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

SGE_F32, SGE_BF16 = 0, 1
_DTYPES = {torch.float32: SGE_F32, torch.bfloat16: SGE_BF16}

_HERE = os.path.dirname(os.path.abspath(__file__))
# SGE_DEBUG=1 loads the debug build (index checks in every kernel, read with
# debug_flags); it is built by ``python -m activation_sparse_gated_epilogue_b200.build --debug``
_LIB_PATH = os.path.join(_HERE, "libsge_debug.so" if os.environ.get("SGE_DEBUG") == "1" else "libsge.so")
_lib = None


class _SgeHybrid(ctypes.Structure):
    """Mirror of `sge_hybrid` in include/sge.h."""
    _fields_ = [("n_tokens", ctypes.c_int64), ("d_ff", ctypes.c_int64),
                ("ell_cap", ctypes.c_int32), ("s_max", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("row_nnz", ctypes.c_void_p), ("spill_slot", ctypes.c_void_p),
                ("spill_rows", ctypes.c_void_p), ("n_spill", ctypes.c_void_p),
                ("ell_idx", ctypes.c_void_p), ("ell_a", ctypes.c_void_p),
                ("ell_u", ctypes.c_void_p), ("spill_a", ctypes.c_void_p),
                ("spill_u", ctypes.c_void_p)]


class LibraryError(RuntimeError):
    """A C entry point returned an error code (message from sge_last_error)."""

    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed (code {code}): {msg}")
        self.code = code


def library_path() -> str:
    return _LIB_PATH


def library() -> ctypes.CDLL:
    """Load libsge.so (built in-tree by ``python -m
    activation_sparse_gated_epilogue_b200.build``); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                               "`python -m activation_sparse_gated_epilogue_b200.build`")
        lib = ctypes.CDLL(_LIB_PATH)
        P, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        sigs = {
            "sge_version": (I, []),
            "sge_debug_flags": (I, [I]),
            "sge_last_error": (ctypes.c_char_p, []),
            "twell_gate_pack": (I, [P, P, I64, I64, I64, I, I, I, P, P, P, P, P]),
            "twell_fused_up_down_workspace_bytes": (ctypes.c_size_t, [I64, I64]),
            "twell_fused_up_down": (I, [P, P, P, P, P, P, I64, P, I64, I64, I64, I, I, I, P,
                                        ctypes.c_size_t, P, P]),
            "twell_fused_up_down_noalloc": (I, [P, P, P, P, P, P, I64, P, I64, I64, I64, I, I, I,
                                                P, P]),
            "sge_interleave_up_down": (I, [P, P, P, I64, I64, I, P]),
            "twell_hybrid_up_down_workspace_bytes": (ctypes.c_size_t, [I64, I64, I64, I]),
            "twell_hybrid_up_down": (I, [P, P, P, P, P, P, I64, P, P, I64, I64, I64, I, I, I, I, P,
                                         ctypes.c_size_t, P, P]),
            "twell_fused_up_down_noalloc_max_tokens": (I64, []),
            "dense_ffn_fwd": (I, [P, P, P, P, P, P, I64, I64, I64, P, P]),
            "hybrid_pack": (I, [P, P, P, I, I, ctypes.POINTER(_SgeHybrid), P, P]),
            "hybrid_ffn_fwd_workspace_bytes": (ctypes.c_size_t, [I64, I64, I]),
            "hybrid_ffn_fwd": (I, [P, ctypes.POINTER(_SgeHybrid), P, P, P, P, P, I64, P,
                                   ctypes.c_size_t, P]),
            "hybrid_ffn_bwd_workspace_bytes": (ctypes.c_size_t, [I64, I64, I64, I, I]),
            "hybrid_ffn_bwd": (I, [P, P, ctypes.POINTER(_SgeHybrid), P, P, P, P, P, P, P, P, I64, P,
                                   ctypes.c_size_t, P]),
            "sge_transpose_up_gate": (I, [P, P, P, I64, I64, P]),
            "int8_quant_rows": (I, [P, I64, I64, I64, I, P, I64, P, P]),
            "int8_linear": (I, [P, I64, P, P, I64, P, P, I64, I64, I64, I, P, P]),
            "moe_route_workspace_bytes": (ctypes.c_size_t, [I64, I]),
            "moe_route_fwd": (I, [P, P, I64, I, I, I, I, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]),
            "moe_route_bwd": (I, [P, P, I64, I, I, I, I, P, P, P, P, P, P, P, P, P]),
            "int8_ffn_workspace_bytes": (ctypes.c_size_t, [I64, I64, I64, I, I, I]),
            "int8_ffn_fwd": (I, [P] * 8 + [I64, I64, I64, I, P, ctypes.c_size_t, P, P]),
            "moe_int8_ffn_fwd": (I, [P] * 11 + [I64, I64, I64, I, I, I, P, ctypes.c_size_t, P, P]),
            "twell_gate_pack_int8": (I, [P, I64, P, P, I64, P, I64, I64, I64, I, I, P, P, P, P, P]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def debug_flags(clear: bool = True) -> int:
    """OR of the SGE_FLAG_* bits the debug build's index checks raised since
    the last clear (synchronises the device); -1 with the release build."""
    r = library().sge_debug_flags(1 if clear else 0)
    if r == -2:
        raise LibraryError("sge_debug_flags", 3, library().sge_last_error().decode())
    return r


def _call(name: str, *args) -> None:
    lib = library()
    rc = getattr(lib, name)(*args)
    if rc != 0:
        raise LibraryError(name, rc, lib.sge_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t: torch.Tensor, name: str, dtype=None, shape=None) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _check_rows(t: torch.Tensor, name: str, dtype, shape) -> int:
    """A 2-D matrix of `shape` whose rows are contiguous (any row stride);
    returns the row stride in elements."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _stream(dev: torch.device, stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream(dev) if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return _DTYPES[t.dtype]


def new_diag(device) -> torch.Tensor:
    """A zeroed int32[4] diagnostics word (see include/sge.h)."""
    return torch.zeros(4, dtype=torch.int32, device=device)


@dataclass
class TwELL:
    """Device TwELL buffers: count [N][F/T] u8, idx [N][F/T][C] u8,
    val [N][F/T][C] in the activation dtype."""
    count: torch.Tensor
    idx: torch.Tensor
    val: torch.Tensor
    tile: int
    cap: int

    @property
    def n_rows(self) -> int:
        return self.count.shape[0]

    @property
    def n_cols(self) -> int:
        return self.count.shape[1] * self.tile

    @staticmethod
    def empty(n: int, f: int, tile: int, cap: int, dtype, device) -> "TwELL":
        nt = f // tile
        return TwELL(torch.empty((n, nt), dtype=torch.uint8, device=device),
                     torch.empty((n, nt, cap), dtype=torch.uint8, device=device),
                     torch.empty((n, nt, cap), dtype=dtype, device=device), tile, cap)


def twell_gate_pack(x: torch.Tensor, wg_t: torch.Tensor, tile: int, cap: int,
                    out: Optional[TwELL] = None, diag: Optional[torch.Tensor] = None,
                    stream=None) -> TwELL:
    """TwELL of ReLU(x W_gate), produced in the gate GEMM's epilogue."""
    _check(x, "x")
    n, d = x.shape
    f = wg_t.shape[0]
    _check(wg_t, "wg_t", x.dtype, (f, d))
    if out is None:
        out = TwELL.empty(n, f, tile, cap, x.dtype, x.device)
    else:
        _check(out.count, "count", torch.uint8, (n, f // tile))
        _check(out.idx, "idx", torch.uint8, (n, f // tile, cap))
        _check(out.val, "val", x.dtype, (n, f // tile, cap))
    if diag is not None:
        _check(diag, "diag", torch.int32, (4,))
    _call("twell_gate_pack", _ptr(x), _ptr(wg_t), n, d, f, _dtype_code(x), tile, cap,
          _ptr(out.count), _ptr(out.idx), _ptr(out.val), _ptr(diag), _stream(x.device, stream))
    return out


def fused_workspace(n_tokens: int, d_model: int, device) -> torch.Tensor:
    """Scratch for twell_fused_up_down (entry counts, job lists, fp32 partial
    outputs of split heavy tokens, counters)."""
    nbytes = library().twell_fused_up_down_workspace_bytes(n_tokens, d_model)
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


def interleave_up_down(wu_t: torch.Tensor, wd: torch.Tensor, stream=None):
    """The interleaved weight layout twell_fused_up_down streams fastest:
    returns (w_ud, wu_view, wd_view), w_ud [F][2d] with row j = wu_t[j] then
    wd[j], and the two [F][d] views of it (row stride 2d) to pass as wu_t and
    wd.  A weight-loading step, done once."""
    _check(wu_t, "wu_t")
    f, d = wu_t.shape
    _check(wd, "wd", wu_t.dtype, (f, d))
    w_ud = torch.empty((f, 2 * d), dtype=wu_t.dtype, device=wu_t.device)
    _call("sge_interleave_up_down", _ptr(wu_t), _ptr(wd), _ptr(w_ud), f, d, _dtype_code(wu_t),
          _stream(wu_t.device, stream))
    return w_ud, w_ud[:, :d], w_ud[:, d:]


def twell_fused_up_down(x: torch.Tensor, tw: TwELL, wu_t: torch.Tensor, wd: torch.Tensor,
                        y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        diag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = sum over TwELL entries of a * (x . W_up[:, j]) * W_down[j] (h never stored).
    wu_t and wd may be row-strided views with one row stride, e.g. the two
    halves of interleave_up_down's matrix."""
    _check(x, "x")
    n, d = x.shape
    f = wu_t.shape[0]
    ldw = _check_rows(wu_t, "wu_t", x.dtype, (f, d))
    if _check_rows(wd, "wd", x.dtype, (f, d)) != ldw:
        raise ValueError("wu_t and wd must have the same row stride")
    _check(tw.count, "count", torch.uint8, (n, f // tw.tile))
    _check(tw.idx, "idx", torch.uint8, (n, f // tw.tile, tw.cap))
    _check(tw.val, "val", x.dtype, (n, f // tw.tile, tw.cap))
    if y is None:
        y = torch.empty_like(x)
    _check(y, "y", x.dtype, (n, d))
    if workspace is None:
        workspace = fused_workspace(n, d, x.device)
    _check(workspace, "workspace", torch.uint8)
    if diag is not None:
        _check(diag, "diag", torch.int32, (4,))
    _call("twell_fused_up_down", _ptr(x), _ptr(tw.count), _ptr(tw.idx), _ptr(tw.val),
          _ptr(wu_t), _ptr(wd), ldw, _ptr(y), n, d, f, _dtype_code(x), tw.tile, tw.cap,
          _ptr(workspace), workspace.numel(), _ptr(diag), _stream(x.device, stream))
    return y


def routed_workspace(n_tokens: int, d_model: int, d_ff: int, s_max: int, device) -> torch.Tensor:
    """Scratch for twell_hybrid_up_down (the caching allocator's blocks are
    512-byte aligned; 256 are needed)."""
    nbytes = library().twell_hybrid_up_down_workspace_bytes(n_tokens, d_model, d_ff, s_max)
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def twell_hybrid_up_down(x: torch.Tensor, tw: TwELL, wu_t: torch.Tensor, wd: torch.Tensor,
                         wd_t: Optional[torch.Tensor], ell_cap: int, s_max: int,
                         y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                         diag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y from TwELL with tokens of more than ell_cap stored entries (the first
    s_max of them) on the tensor-core spill GEMMs and the others per entry on
    CUDA cores (batches of at most 64 tokens: every token per entry).  bf16.  ``wd_t`` is W_down transposed, [d][F]
    (None only when s_max == 0); wu_t and wd may be the row-strided halves of
    interleave_up_down's matrix."""
    _check(x, "x", torch.bfloat16)
    n, d = x.shape
    f = wu_t.shape[0]
    ldw = _check_rows(wu_t, "wu_t", x.dtype, (f, d))
    if _check_rows(wd, "wd", x.dtype, (f, d)) != ldw:
        raise ValueError("wu_t and wd must have the same row stride")
    if wd_t is None:
        if s_max > 0:
            raise ValueError("wd_t (W_down transposed, [d][F]) is required when s_max > 0")
    else:
        _check(wd_t, "wd_t", torch.bfloat16, (d, f))
    _check(tw.count, "count", torch.uint8, (n, f // tw.tile))
    _check(tw.idx, "idx", torch.uint8, (n, f // tw.tile, tw.cap))
    _check(tw.val, "val", x.dtype, (n, f // tw.tile, tw.cap))
    if y is None:
        y = torch.empty_like(x)
    _check(y, "y", x.dtype, (n, d))
    if workspace is None:
        workspace = routed_workspace(n, d, f, s_max, x.device)
    _check(workspace, "workspace", torch.uint8)
    if diag is not None:
        _check(diag, "diag", torch.int32, (4,))
    _call("twell_hybrid_up_down", _ptr(x), _ptr(tw.count), _ptr(tw.idx), _ptr(tw.val), _ptr(wu_t),
          _ptr(wd), ldw, _ptr(wd_t), _ptr(y), n, d, f, tw.tile, tw.cap, ell_cap, s_max,
          _ptr(workspace), workspace.numel(), _ptr(diag), _stream(x.device, stream))
    return y


def twell_ffn_forward(x, wg_t, wu_t, wd, tile: int, cap: int, tw: Optional[TwELL] = None,
                      y: Optional[torch.Tensor] = None, diag: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None):
    """The sparse inference forward: gate GEMM + TwELL epilogue, then the
    fused up/down kernel.  Returns (y, twell)."""
    tw = twell_gate_pack(x, wg_t, tile, cap, out=tw, diag=diag, stream=stream)
    y = twell_fused_up_down(x, tw, wu_t, wd, y=y, workspace=workspace, diag=diag, stream=stream)
    return y, tw


def dense_ffn_fwd(x: torch.Tensor, wg_t: torch.Tensor, wu_t: torch.Tensor, wd_t: torch.Tensor,
                  h: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                  diag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Dense bf16 gated FFN (baseline).  ``wd_t`` is W_down transposed, [d][F]."""
    _check(x, "x", torch.bfloat16)
    n, d = x.shape
    f = wg_t.shape[0]
    _check(wg_t, "wg_t", torch.bfloat16, (f, d))
    _check(wu_t, "wu_t", torch.bfloat16, (f, d))
    _check(wd_t, "wd_t", torch.bfloat16, (d, f))
    if h is None:
        h = torch.empty((n, f), dtype=torch.bfloat16, device=x.device)
    if y is None:
        y = torch.empty_like(x)
    _check(h, "h", torch.bfloat16, (n, f))
    _check(y, "y", torch.bfloat16, (n, d))
    _call("dense_ffn_fwd", _ptr(x), _ptr(wg_t), _ptr(wu_t), _ptr(wd_t), _ptr(h), _ptr(y),
          n, d, f, _ptr(diag), _stream(x.device, stream))
    return y


@dataclass
class Hybrid:
    """Device buffers of the hybrid format (see `sge_hybrid` in include/sge.h)."""
    n_tokens: int
    d_ff: int
    ell_cap: int
    s_max: int
    row_nnz: torch.Tensor
    spill_slot: torch.Tensor
    spill_rows: torch.Tensor
    n_spill: torch.Tensor
    ell_idx: torch.Tensor
    ell_a: torch.Tensor
    ell_u: torch.Tensor
    spill_a: torch.Tensor
    spill_u: torch.Tensor

    @staticmethod
    def empty(n: int, f: int, ell_cap: int, s_max: int, device) -> "Hybrid":
        kk, ss = max(ell_cap, 1), max(s_max, 1)
        z = lambda *shape, dt: torch.empty(shape, dtype=dt, device=device)
        return Hybrid(n, f, ell_cap, s_max, z(n, dt=torch.int32), z(n, dt=torch.int32),
                      z(ss, dt=torch.int32), z(1, dt=torch.int32), z(n, kk, dt=torch.uint16),
                      z(n, kk, dt=torch.bfloat16), z(n, kk, dt=torch.bfloat16),
                      z(ss, f, dt=torch.bfloat16), z(ss, f, dt=torch.bfloat16))

    def c_struct(self) -> _SgeHybrid:
        for name in ("row_nnz", "spill_slot", "spill_rows", "n_spill", "ell_idx", "ell_a", "ell_u",
                     "spill_a", "spill_u"):
            _check(getattr(self, name), name)
        return _SgeHybrid(self.n_tokens, self.d_ff, self.ell_cap, self.s_max, SGE_BF16, 0,
                          self.row_nnz.data_ptr(), self.spill_slot.data_ptr(),
                          self.spill_rows.data_ptr(), self.n_spill.data_ptr(),
                          self.ell_idx.data_ptr(), self.ell_a.data_ptr(), self.ell_u.data_ptr(),
                          self.spill_a.data_ptr(), self.spill_u.data_ptr())


def hybrid_pack(tw: TwELL, ell_cap: int, s_max: int, out: Optional[Hybrid] = None,
                diag: Optional[torch.Tensor] = None, stream=None) -> Hybrid:
    """Route each row of a bf16 TwELL to the ELL part (nnz <= K) or the dense spill."""
    _check(tw.count, "count", torch.uint8)
    _check(tw.val, "val", torch.bfloat16)
    n, f = tw.n_rows, tw.n_cols
    if out is None:
        out = Hybrid.empty(n, f, ell_cap, s_max, tw.count.device)
    cs = out.c_struct()
    _call("hybrid_pack", _ptr(tw.count), _ptr(tw.idx), _ptr(tw.val), tw.tile, tw.cap,
          ctypes.byref(cs), _ptr(diag), _stream(tw.count.device, stream))
    return out


def hybrid_fwd_workspace(d_model: int, d_ff: int, s_max: int, device) -> torch.Tensor:
    nbytes = library().hybrid_ffn_fwd_workspace_bytes(d_model, d_ff, s_max)
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


def hybrid_ffn_fwd(x: torch.Tensor, hy: Hybrid, wu_t: torch.Tensor, wd: torch.Tensor,
                   wd_t: Optional[torch.Tensor], y: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None,
                   wg_t: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y from the hybrid form; fills hy.ell_u and hy.spill_u.  ``wd_t`` is
    W_down transposed, [d][F] (a weight layout the caller builds once; None
    only when hy.s_max == 0).  With wg_t the spill rows' activations are
    recomputed from the gate (and written to hy.spill_a), so rows that
    reached the spill through an overflowing TwELL tile come out exact."""
    _check(x, "x", torch.bfloat16)
    n, d = x.shape
    f = hy.d_ff
    _check(wu_t, "wu_t", torch.bfloat16, (f, d))
    _check(wd, "wd", torch.bfloat16, (f, d))
    if wd_t is None:
        if hy.s_max > 0:
            raise ValueError("wd_t (W_down transposed, [d][F]) is required when s_max > 0")
    else:
        _check(wd_t, "wd_t", torch.bfloat16, (d, f))
    if wg_t is not None:
        _check(wg_t, "wg_t", torch.bfloat16, (f, d))
    if y is None:
        y = torch.empty_like(x)
    if workspace is None:
        workspace = hybrid_fwd_workspace(d, f, hy.s_max, x.device)
    cs = hy.c_struct()
    _call("hybrid_ffn_fwd", _ptr(x), ctypes.byref(cs), _ptr(wu_t), _ptr(wd), _ptr(wd_t),
          _ptr(wg_t) if wg_t is not None else None, _ptr(y), d,
          _ptr(workspace), workspace.numel(), _stream(x.device, stream))
    return y


def hybrid_bwd_workspace(n_tokens: int, d_model: int, d_ff: int, ell_cap: int, s_max: int,
                         device) -> torch.Tensor:
    nbytes = library().hybrid_ffn_bwd_workspace_bytes(n_tokens, d_model, d_ff, ell_cap, s_max)
    # 256-byte alignment: the caching allocator hands out 512-byte aligned blocks
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def transpose_up_gate(wu_t: torch.Tensor, wg_t: torch.Tensor, stream=None) -> torch.Tensor:
    """w_ug [d][2F] = [W_up | W_gate], hybrid_ffn_bwd's dX operand; a
    weight-loading step, done once per weight update."""
    _check(wu_t, "wu_t", torch.bfloat16)
    f, d = wu_t.shape
    _check(wg_t, "wg_t", torch.bfloat16, (f, d))
    w_ug = torch.empty((d, 2 * f), dtype=torch.bfloat16, device=wu_t.device)
    _call("sge_transpose_up_gate", _ptr(wu_t), _ptr(wg_t), _ptr(w_ug), f, d, _stream(wu_t.device, stream))
    return w_ug


def hybrid_ffn_bwd(x: torch.Tensor, dy: torch.Tensor, hy: Hybrid, wg_t: torch.Tensor,
                   wu_t: torch.Tensor, wd: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                   stream=None, w_ug: Optional[torch.Tensor] = None, out=None):
    """Returns (dx bf16 [N][d], dwg_t, dwu_t, dwd fp32 [F][d]).  ``w_ug`` is
    transpose_up_gate's [W_up | W_gate] (None: built in the workspace per
    call); ``out`` optionally gives the four output tensors."""
    _check(x, "x", torch.bfloat16)
    n, d = x.shape
    f = hy.d_ff
    _check(dy, "dy", torch.bfloat16, (n, d))
    for name, w in (("wg_t", wg_t), ("wu_t", wu_t), ("wd", wd)):
        _check(w, name, torch.bfloat16, (f, d))
    if w_ug is not None:
        _check(w_ug, "w_ug", torch.bfloat16, (d, 2 * f))
    if out is None:
        out = (torch.empty_like(x),) + tuple(torch.empty((f, d), dtype=torch.float32, device=x.device)
                                              for _ in range(3))
    dx, dwg, dwu, dwd = out
    if workspace is None:
        workspace = hybrid_bwd_workspace(n, d, f, hy.ell_cap, hy.s_max, x.device)
    cs = hy.c_struct()
    _call("hybrid_ffn_bwd", _ptr(x), _ptr(dy), ctypes.byref(cs), _ptr(wg_t), _ptr(wu_t), _ptr(wd),
          _ptr(w_ug), _ptr(dx), _ptr(dwg), _ptr(dwu), _ptr(dwd), d, _ptr(workspace),
          workspace.numel(), _stream(x.device, stream))
    return dx, dwg, dwu, dwd


# ------------------------------------------------- 8-bit integer products


# A decode step makes many small calls, so the checks below read each property
# of a tensor once and form no message unless one fails.


def _launch(name: str, index: int, stream, *args) -> None:
    """Call `name` with the stream appended, on CUDA device `index`."""
    lib = _lib or library()
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            rc = getattr(lib, name)(*args, _raw_stream(index, stream))
    else:
        rc = getattr(lib, name)(*args, _raw_stream(index, stream))
    if rc != 0:
        raise LibraryError(name, rc, lib.sge_last_error().decode())


def _raw_stream(index: int, stream) -> int:
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _device_of(t: torch.Tensor, name: str) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    return index


def _operand(t: torch.Tensor, name: str, index: int, dtype, shape) -> int:
    """The address of a contiguous tensor of this dtype and shape on device `index`."""
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()):
        _check(t, name, dtype, shape)
        raise ValueError(f"{name} is on {t.device}, other operands on cuda:{index}")
    return t.data_ptr()


def _scratch(t: torch.Tensor, index: int) -> int:
    return _operand(t, "workspace", index, torch.uint8, (t.numel(),))


def _diag_ptr(diag: Optional[torch.Tensor], index: int) -> Optional[int]:
    return None if diag is None else _operand(diag, "diag", index, torch.int32, (4,))


def _allocate(stream, make, *args):
    """Tensors made for a call on `stream` come from that stream's pool: one
    from the current stream's could still be in use there."""
    if stream is None:
        return make(*args)
    with torch.cuda.stream(stream):
        return make(*args)


def _empty(shape, dtype, index: int) -> torch.Tensor:
    return torch.empty(shape, dtype=dtype, device=torch.device("cuda", index))


class Int8Rows:
    """An 8-bit matrix: q int8 [rows][pitch] (pitch a multiple of 16, bytes
    past `cols` are padding) and one fp32 scale per row.  Weights of E experts
    are E blocks of rows."""
    __slots__ = ("cols", "_q", "_scale", "_buffer", "_shape")

    def __init__(self, q: torch.Tensor, scale: torch.Tensor, cols: int):
        self._q, self._scale, self.cols, self._buffer = q, scale, cols, None

    @staticmethod
    def empty(rows: int, cols: int, device) -> "Int8Rows":
        """Uninitialised rows, the scales behind them in one allocation."""
        out = Int8Rows.__new__(Int8Rows)
        pitch = (cols + 15) & ~15
        out.cols, out._shape = cols, (rows, pitch)
        out._q = out._scale = None
        out._buffer = torch.empty(rows * (pitch + 4), dtype=torch.int8, device=device)
        return out

    @property
    def q(self) -> torch.Tensor:
        if self._q is None:
            n, pitch = self._shape
            self._q = self._buffer[:n * pitch].view(n, pitch)
        return self._q

    @property
    def scale(self) -> torch.Tensor:
        if self._scale is None:
            n, pitch = self._shape
            self._scale = self._buffer[n * pitch:].view(torch.float32)
        return self._scale

    @property
    def rows(self) -> int:
        return self.q.shape[0] if self._buffer is None else self._shape[0]

    def _operands(self, name: str, index: int, rows: Optional[int] = None, cols: Optional[int] = None):
        """(address of q, pitch, address of scale, rows), checked."""
        buffer = self._buffer
        if buffer is not None:  # made by empty(): only its device and rows are in question
            n, pitch = self._shape
            if buffer.get_device() != index:
                raise ValueError(f"{name} is on {buffer.device}, other operands on cuda:{index}")
            q = buffer.data_ptr()
            scale = q + n * pitch
        else:
            t = self._q
            if t.dim() != 2 or t.shape[1] % 16 or not 1 <= self.cols <= t.shape[1]:
                raise ValueError(f"{name}.q must be [rows][pitch], pitch a multiple of 16, at least cols")
            n, pitch = t.shape
            q = _operand(t, f"{name}.q", index, torch.int8, (n, pitch))
            scale = _operand(self._scale, f"{name}.scale", index, torch.float32, (n,))
        if rows is not None and n != rows:
            raise ValueError(f"{name} must have {rows} rows, got {n}")
        if cols is not None and self.cols != cols:
            raise ValueError(f"{name} must have {cols} columns, got {self.cols}")
        return q, pitch, scale, n

    def _index(self, name: str) -> int:
        return _device_of(self._q if self._buffer is None else self._buffer, name)


def int8_quant_rows(x: torch.Tensor, out: Optional[Int8Rows] = None, stream=None) -> Int8Rows:
    """The rows of a bf16 or fp32 matrix as 8-bit integers with a scale each
    (activations per token; weights per output channel, done once when they
    are loaded).  x may be a row-strided view."""
    index = _device_of(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    n, d = x.shape
    if d > 1 and x.stride(1) != 1:
        raise ValueError("x must have contiguous rows")
    ldx = x.stride(0) if n > 1 else d
    if out is None:
        out = _allocate(stream, Int8Rows.empty, n, d, x.device)
    q, ldq, scale, _ = out._operands("out", index, n, d)
    _launch("int8_quant_rows", index, stream, x.data_ptr(), ldx, n, d, _dtype_code(x), q, ldq, scale)
    return out


def int8_linear(xq: Int8Rows, wq: Int8Rows, dtype: torch.dtype = torch.bfloat16,
                y: Optional[torch.Tensor] = None, diag: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """y[n][m] = (sum over k of xq[n][k] * wq[m][k]) * xq.scale[n] * wq.scale[m]
    with exact integer sums, in bf16 or fp32."""
    index = xq._index("xq")
    k = xq.cols
    x, ldx, sx, n = xq._operands("xq", index)
    w, ldw, sw, m = wq._operands("wq", index, cols=k)
    if y is None:
        y = _allocate(stream, _empty, (n, m), dtype, index)
    _launch("int8_linear", index, stream, x, ldx, sx, w, ldw, sw, _operand(y, "y", index, dtype, (n, m)), n, m, k,
            _dtype_code(y), _diag_ptr(diag, index))
    return y


def twell_gate_pack_int8(xq: Int8Rows, wg_q: Int8Rows, tile: int, cap: int, out: Optional[TwELL] = None,
                         diag: Optional[torch.Tensor] = None, stream=None) -> TwELL:
    """twell_gate_pack with the gate projection in 8-bit integers: TwELL
    (bf16 values) of ReLU of int8_linear's product."""
    index = xq._index("xq")
    k = xq.cols
    x, ldx, sx, n = xq._operands("xq", index)
    w, ldw, sw, f = wg_q._operands("wg_q", index, cols=k)
    if tile < 1 or cap < 1:
        raise ValueError(f"tile {tile} and cap {cap} must be at least 1")
    if out is None:
        out = _allocate(stream, TwELL.empty, n, f, tile, cap, torch.bfloat16, torch.device("cuda", index))
    _launch("twell_gate_pack_int8", index, stream, x, ldx, sx, w, ldw, sw, n, k, f, tile, cap,
            _operand(out.count, "count", index, torch.uint8, (n, f // tile)),
            _operand(out.idx, "idx", index, torch.uint8, (n, f // tile, cap)),
            _operand(out.val, "val", index, torch.bfloat16, (n, f // tile, cap)), _diag_ptr(diag, index))
    return out


# ------------------------------------------------------------ expert router


class MoeRoute:
    """What moe_route_fwd gives (see include/sge.h): ids, w, pos [N][k]; order
    [N * k]; counts [E]; offsets [E + 1]; loss, n_live [1]; and the settings
    that its gradient needs again."""
    NAMES = ("ids", "w", "counts", "offsets", "pos", "order", "loss", "n_live")
    __slots__ = ("renorm", "_tensors", "_buffer", "_sizes", "_at")

    def __init__(self, ids, w, counts, offsets, pos, order, loss, n_live, renorm: bool = True):
        self._tensors = [ids, w, counts, offsets, pos, order, loss, n_live]
        self._buffer = None
        self.renorm = renorm

    @staticmethod
    def empty(n_tokens: int, n_experts: int, top_k: int, device) -> "MoeRoute":
        """Uninitialised tensors, views of one allocation."""
        out = MoeRoute.__new__(MoeRoute)
        out.renorm = True
        out._tensors = [None] * 8
        out._sizes = (n_tokens, n_experts, top_k)
        nk = n_tokens * top_k
        at, end = [], 0
        for count in (nk, nk, n_experts, n_experts + 1, nk, nk, 1, 1):
            at.append(end)
            end += (count + 3) & ~3      # 16-byte aligned parts
        out._at = at
        out._buffer = torch.empty(end, dtype=torch.int32, device=device)
        return out

    def _tensor(self, i: int) -> torch.Tensor:
        t = self._tensors[i]
        if t is None:
            n, e, k = self._sizes
            shape = ((n, k), (n, k), (e,), (e + 1,), (n, k), (n * k,), (1,), (1,))[i]
            size = shape[0] * shape[1] if len(shape) == 2 else shape[0]
            t = self._buffer[self._at[i]:self._at[i] + size].view(shape)
            if i in (1, 6):
                t = t.view(torch.float32)
            self._tensors[i] = t
        return t

    ids = property(lambda self: self._tensor(0))
    w = property(lambda self: self._tensor(1))
    counts = property(lambda self: self._tensor(2))
    offsets = property(lambda self: self._tensor(3))
    pos = property(lambda self: self._tensor(4))
    order = property(lambda self: self._tensor(5))
    loss = property(lambda self: self._tensor(6))
    n_live = property(lambda self: self._tensor(7))

    @property
    def top_k(self) -> int:
        return self._tensors[0].shape[1] if self._buffer is None else self._sizes[2]

    def _operands(self, index: int, n: int, e: int, k: int):
        """The eight addresses in the order of NAMES, checked."""
        buffer = self._buffer
        if buffer is not None:  # made by empty(): only its device and sizes are in question
            if self._sizes != (n, e, k):
                raise ValueError(f"route has the shape (tokens, experts, top_k) = {self._sizes}, not {(n, e, k)}")
            if buffer.get_device() != index:
                raise ValueError(f"route is on {buffer.device}, the logits on cuda:{index}")
            base = buffer.data_ptr()
            return [base + 4 * at for at in self._at]
        i32, f32, nk = torch.int32, torch.float32, (n, k)
        return [_operand(t, name, index, dtype, shape) for t, name, dtype, shape in zip(
            self._tensors, MoeRoute.NAMES, (i32, f32, i32, i32, i32, i32, f32, i32),
            (nk, nk, (e,), (e + 1,), nk, (n * k,), (1,), (1,)))]


def moe_route_workspace(n_tokens: int, n_experts: int, top_k: int, device) -> torch.Tensor:
    """Scratch for moe_route_fwd (each block's counts and probability sums), for
    batches of at most n_tokens; the same for every top_k."""
    nbytes = library().moe_route_workspace_bytes(n_tokens, n_experts)
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _logits_operands(logits: torch.Tensor, mask: Optional[torch.Tensor]):
    """(device, tokens, experts, address of the logits, of the mask), checked."""
    index = _device_of(logits, "logits")
    if logits.dim() != 2 or not logits.is_contiguous():
        raise ValueError("logits must be [tokens][experts], contiguous")
    n, e = logits.shape
    if mask is None:
        return index, n, e, logits.data_ptr(), None
    if mask.dtype not in (torch.uint8, torch.bool):
        raise ValueError(f"mask must be uint8 or bool, got {mask.dtype}")
    return index, n, e, logits.data_ptr(), _operand(mask, "mask", index, mask.dtype, (n,))


def moe_route_fwd(logits: torch.Tensor, top_k: int, renorm: bool = True, mask: Optional[torch.Tensor] = None,
                  out: Optional[MoeRoute] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> MoeRoute:
    """Top-k experts and weights of each token, assignments per expert, their
    expert order, and the balance loss.  ``mask`` [N]: 0 for padding tokens."""
    index, n, e, x, m = _logits_operands(logits, mask)
    if out is None:
        out = _allocate(stream, MoeRoute.empty, n, e, max(top_k, 0), logits.device)
    renorm = bool(renorm)
    if workspace is None:
        workspace = _allocate(stream, moe_route_workspace, n, e, top_k, logits.device)
    _launch("moe_route_fwd", index, stream, x, m, n, e, top_k, int(renorm), _dtype_code(logits),
            *out._operands(index, n, e, top_k), _scratch(workspace, index), workspace.numel())
    out.renorm = renorm  # a refused call leaves `out` as it was
    return out


def moe_route_bwd(logits: torch.Tensor, route: MoeRoute, dloss: Optional[torch.Tensor] = None,
                  dw: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dlogits from the gradients of the balance loss (fp32 [1]) and of the
    weights (fp32 [N][k]); logits and mask as in the forward that gave route."""
    index, n, e, x, m = _logits_operands(logits, mask)
    k = route.top_k
    if out is None:
        out = _allocate(stream, torch.empty_like, logits)
    ids, w, counts, offsets, _, _, _, n_live = route._operands(index, n, e, k)
    _launch("moe_route_bwd", index, stream, x, m, n, e, k, int(route.renorm), _dtype_code(logits), ids, w, counts,
            offsets, n_live,
            None if dloss is None else _operand(dloss, "dloss", index, torch.float32, (1,)),
            None if dw is None else _operand(dw, "dw", index, torch.float32, (n, k)),
            _operand(out, "out", index, logits.dtype, (n, e)))
    return out


# --------------------------------------- feed-forward block on 8-bit weights


def int8_ffn_workspace(n_tokens: int, d_model: int, d_ff: int, n_experts: int, top_k: int, dtype: torch.dtype,
                       device) -> torch.Tensor:
    """Scratch for int8_ffn_fwd (n_experts = top_k = 1) and moe_int8_ffn_fwd, for
    batches of at most n_tokens."""
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    nbytes = library().int8_ffn_workspace_bytes(n_tokens, d_model, d_ff, n_experts, top_k, _DTYPES[dtype])
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _ffn_operands(x, index, wg_q, wu_q, wd_t_q, e, k, y, workspace, stream):
    """Checked operands of the two calls: (n, d, f, addresses of the weights
    and scales, y, workspace)."""
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be [tokens][d_model], contiguous")
    n, d = x.shape
    if wg_q.rows % e:
        raise ValueError(f"wg_q must have a multiple of {e} rows, got {wg_q.rows}")
    f = wg_q.rows // e
    weights = []
    for name, m, rows, cols in (("wg_q", wg_q, e * f, d), ("wu_q", wu_q, e * f, d), ("wd_t_q", wd_t_q, e * d, f)):
        q, pitch, scale, _ = m._operands(name, index, rows, cols)
        if pitch != (cols + 15) // 16 * 16:
            raise ValueError(f"{name}.q must have rows of {(cols + 15) // 16 * 16} bytes, got {pitch}")
        weights += (q, scale)
    if y is None:
        y = _allocate(stream, torch.empty_like, x)
    if workspace is None:
        workspace = _allocate(stream, int8_ffn_workspace, n, d, f, e, k, x.dtype, x.device)
    return n, d, f, weights, y, workspace


def int8_ffn_fwd(x: torch.Tensor, wg_q: Int8Rows, wu_q: Int8Rows, wd_t_q: Int8Rows,
                 y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 diag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gated feed-forward block on 8-bit weights.  ``wd_t_q`` is
    int8_quant_rows of W_down transposed, [d][F]."""
    index = _device_of(x, "x")
    n, d, f, weights, y, workspace = _ffn_operands(x, index, wg_q, wu_q, wd_t_q, 1, 1, y, workspace, stream)
    _launch("int8_ffn_fwd", index, stream, x.data_ptr(), *weights, _operand(y, "y", index, x.dtype, (n, d)), n, d, f,
            _dtype_code(x), _scratch(workspace, index), workspace.numel(), _diag_ptr(diag, index))
    return y


def moe_int8_ffn_fwd(x: torch.Tensor, wg_q: Int8Rows, wu_q: Int8Rows, wd_t_q: Int8Rows, w: torch.Tensor,
                     offsets: torch.Tensor, pos: torch.Tensor, y: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, diag: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """The experts' blocks on 8-bit weights (expert by expert in the rows of
    wg_q, wu_q and wd_t_q), each token's summed with its weights; w, offsets
    and pos are moe_route_fwd's."""
    index = _device_of(x, "x")
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must be [experts + 1]")
    if w.dim() != 2:
        raise ValueError("w must be [tokens][top_k]")
    e, k = offsets.shape[0] - 1, w.shape[1]
    n, d, f, weights, y, workspace = _ffn_operands(x, index, wg_q, wu_q, wd_t_q, e, k, y, workspace, stream)
    _launch("moe_int8_ffn_fwd", index, stream, x.data_ptr(), *weights,
            _operand(w, "w", index, torch.float32, (n, k)),
            _operand(offsets, "offsets", index, torch.int32, (e + 1,)),
            _operand(pos, "pos", index, torch.int32, (n, k)), _operand(y, "y", index, x.dtype, (n, d)), n, d, f, e, k,
            _dtype_code(x), _scratch(workspace, index), workspace.numel(), _diag_ptr(diag, index))
    return y
