"""GB300-native Flash-Overlap: Python binding of the C ABI in include/fo.h.

This module only marshals arguments (tensor pointers, shapes, the current CUDA
stream) into the C entry points of ``libfo.so``; every step of the hot path
runs in the library's own CUDA kernels.  There is no fallback: if the library
is missing, importing :func:`load` raises.

Method: "FlashOverlap: Minimizing Tail Latency in Communication Overlap for
Distributed LLM Training" (technical summary, section 2): Flash-AG,
Flash-RS with rank-adaptive order, query-split attention -- here with all P
ranks on one GPU.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfo.so")

(FO_OK, FO_ERR_INVALID_ARG, FO_ERR_SHAPE, FO_ERR_UNSUPPORTED, FO_ERR_CUDA, FO_ERR_TIMEOUT, FO_ERR_OOM,
 FO_ERR_RANGE, FO_ERR_INTERNAL) = range(9)
STATUS_NAMES = ["FO_OK", "FO_ERR_INVALID_ARG", "FO_ERR_SHAPE", "FO_ERR_UNSUPPORTED", "FO_ERR_CUDA",
                "FO_ERR_TIMEOUT", "FO_ERR_OOM", "FO_ERR_RANGE", "FO_ERR_INTERNAL"]
FO_BF16, FO_F32 = 0, 1
ORDERS = {"flash": 0, "naive": 1, "slicing": 2, "serial": 3}
LINKS = {"default": 0, "ce": 1, "push": 2}
FAULTS = {"none": 0, "skip_hop": 1}
EPILOGUES = {"plain": 0, "silu": 1}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {None: 0, "linear": 1, "banded": 2, "ramped": 3}
ROPE_MAX_PAIRS = 256

# Every entry point declared in include/fo.h.
ABI_SYMBOLS = ("fo_version", "fo_last_error_string", "fo_ctx_create", "fo_ctx_destroy", "fo_ctx_poll",
               "fo_ctx_phase_ms", "fo_gemm", "fo_ag_gemm", "fo_gemm_rs", "fo_silu_mul", "fo_mlp_layer",
               "fo_mlp_layer_host", "fo_qsplit_attn", "fo_attn_layer", "fo_gemm_a2a", "fo_a2a_gemm", "fo_col_linear_backward",
               "fo_row_linear_backward", "fo_step_order",
               "fo_gemm_rs_noalloc", "fo_attn_forward", "fo_attn_backward", "fo_norm_residual",
               "fo_norm_residual_backward", "fo_rope_table_init", "fo_rope", "fo_rope_backward")


class FoMat(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld", ctypes.c_int64)]


class FoOpts(ctypes.Structure):
    _fields_ = [("order", ctypes.c_int32), ("link", ctypes.c_int32), ("n_slices", ctypes.c_int32),
                ("timeout_us", ctypes.c_uint32), ("causal_prune", ctypes.c_int32), ("num_sms", ctypes.c_int32),
                ("fault", ctypes.c_int32), ("epilogue", ctypes.c_int32), ("sm_pairs", ctypes.c_int32),
                ("compute_only", ctypes.c_int32), ("split_layer", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class FoAttnMask(ctypes.Structure):
    _fields_ = [("causal", ctypes.c_int32), ("num_seqs", ctypes.c_int32), ("q_offsets", ctypes.c_void_p),
                ("k_offsets", ctypes.c_void_p), ("scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class FoNormParams(ctypes.Structure):
    _fields_ = [("w_post", ctypes.POINTER(FoMat)), ("w_pre", ctypes.POINTER(FoMat)),
                ("gate", ctypes.POINTER(FoMat)), ("gate_per_token", ctypes.c_int32),
                ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32)]


class FoNormGrads(ctypes.Structure):
    _fields_ = [("w_post", ctypes.POINTER(FoMat)), ("w_pre", ctypes.POINTER(FoMat)),
                ("gate", ctypes.POINTER(FoMat))]


class FoRopeTable(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("amplitude", ctypes.c_float),
                ("turns", ctypes.c_uint64 * ROPE_MAX_PAIRS)]


class FoRopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("reserved", ctypes.c_int32), ("factor", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("original_length", ctypes.c_int64)]


class FoError(RuntimeError):
    def __init__(self, status: int, message: str):
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else str(status)
        super().__init__(f"{name}: {message}")
        self.status = status


_lib = None


def load() -> ctypes.CDLL:
    """Loads libfo.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with overlapped_tensor_gemm_gb300._build.build()")
        lib = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        vp = ctypes.c_void_p
        lib.fo_version.restype = ctypes.c_int
        lib.fo_step_order.restype = ctypes.c_int
        lib.fo_last_error_string.restype = ctypes.c_char_p
        lib.fo_ctx_create.argtypes = [ctypes.c_int, P(vp)]
        lib.fo_ctx_destroy.argtypes = [vp]
        lib.fo_ctx_poll.argtypes = [vp]
        lib.fo_ctx_phase_ms.argtypes = [vp, P(ctypes.c_float), P(ctypes.c_float)]
        lib.fo_gemm.argtypes = [vp, P(FoMat), P(FoMat), P(FoMat), P(FoOpts), vp]
        for name in ("fo_ag_gemm", "fo_gemm_rs", "fo_gemm_a2a", "fo_a2a_gemm"):
            getattr(lib, name).argtypes = [vp, P(FoMat), P(FoMat), ctypes.c_int, P(FoMat), P(FoOpts), vp]
        lib.fo_silu_mul.argtypes = [vp, P(FoMat), ctypes.c_int, P(FoMat), vp]
        for name in ("fo_mlp_layer", "fo_mlp_layer_host"):
            getattr(lib, name).argtypes = [vp, P(FoMat), P(FoMat), P(FoMat), ctypes.c_int, ctypes.c_int,
                                           P(FoMat), P(FoOpts), vp]
        lib.fo_qsplit_attn.argtypes = [vp, P(FoMat), P(FoMat), P(FoMat), ctypes.c_int, ctypes.c_int,
                                       ctypes.c_int, ctypes.c_int, P(FoMat), P(FoOpts), vp]
        lib.fo_attn_layer.argtypes = [vp, P(FoMat), P(FoMat), P(FoMat), ctypes.c_int, ctypes.c_int,
                                      ctypes.c_int, ctypes.c_int, P(FoMat), P(FoOpts), vp]
        for name in ("fo_col_linear_backward", "fo_row_linear_backward"):
            getattr(lib, name).argtypes = [vp, P(FoMat), P(FoMat), P(FoMat), ctypes.c_int, P(FoMat), P(FoMat),
                                           P(FoOpts), vp]
        lib.fo_step_order.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, P(ctypes.c_int32),
                                      P(ctypes.c_int32), ctypes.c_int]
        ci, i64 = ctypes.c_int, ctypes.c_int64
        lib.fo_attn_forward.argtypes = [vp, P(FoMat), P(FoMat), P(FoMat), ci, ci, ci, ci, P(FoAttnMask), P(FoMat),
                                        P(FoMat), P(FoOpts), vp]
        lib.fo_attn_backward.argtypes = [vp, P(FoMat), P(FoMat), P(FoMat), P(FoMat), P(FoMat), P(FoMat), ci, ci, ci,
                                         ci, P(FoAttnMask), P(FoMat), P(FoMat), P(FoMat), P(FoOpts), vp]
        lib.fo_norm_residual.argtypes = [vp, P(FoMat), P(FoMat), ci, P(FoNormParams), P(FoMat), P(FoMat), vp]
        lib.fo_norm_residual_backward.argtypes = [vp, P(FoMat), P(FoMat), P(FoMat), P(FoMat), ci, P(FoNormParams),
                                                  P(FoMat), P(FoMat), P(FoNormGrads), vp]
        lib.fo_rope_table_init.argtypes = [P(FoRopeTable), ci, ctypes.c_double, P(FoRopeScaling)]
        for name in ("fo_rope", "fo_rope_backward"):
            getattr(lib, name).argtypes = [vp, P(FoMat), ci, P(FoRopeTable), ci, ci, P(vp), i64, i64, P(FoMat), vp]
        lib.fo_gemm_rs_noalloc.argtypes = [P(FoMat), P(FoMat), ctypes.c_int, P(FoMat), ctypes.c_uint32,
                                           vp, vp]
        for name in ABI_SYMBOLS:
            if name not in ("fo_version", "fo_last_error_string", "fo_step_order"):
                getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


def _check(status: int) -> None:
    if status != FO_OK:
        msg = load().fo_last_error_string().decode(errors="replace")
        raise FoError(status, msg)


def mat(t) -> FoMat:
    """fo_mat view of a 2-D (or [rows, a, b] contiguous-inner) torch tensor."""
    import torch
    if t.dim() > 2:
        t = t.reshape(t.shape[0], -1) if t[0].is_contiguous() else None
        if t is None:
            raise ValueError("inner dimensions must be contiguous")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("need a row-major 2-D view (unit column stride)")
    if t.dtype == torch.bfloat16:
        dt = FO_BF16
    elif t.dtype == torch.float32:
        dt = FO_F32
    else:
        raise TypeError(f"unsupported dtype {t.dtype}")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if ld < t.shape[1]:
        raise ValueError(f"rows {ld} elements apart share memory (an expanded view?): need {t.shape[1]} or more")
    return FoMat(t.data_ptr(), dt, 0, t.shape[0], t.shape[1], ld)


_MAT_ARRAYS = [FoMat * n for n in range(65)]  # array types by length
_MAT_BYTES = ctypes.sizeof(FoMat)
_PACK_MAT = struct.Struct("@Piiqqq").pack_into  # FoMat's fields
assert struct.calcsize("@Piiqqq") == _MAT_BYTES
_DTYPE_CODES: dict = {}


def _dtype_codes() -> dict:
    if not _DTYPE_CODES:
        import torch
        _DTYPE_CODES.update({torch.bfloat16: FO_BF16, torch.float32: FO_F32})
    return _DTYPE_CODES


def _mats(ts: Sequence) -> ctypes.Array:
    arr = (FoMat * len(ts))()
    for i, t in enumerate(ts):
        arr[i] = mat(t)
    return arr


def opts(order: str = "flash", link: str = "default", n_slices: int = 0, timeout_us: int = 0,
         causal_prune: bool = False, num_sms: int = 0, fault: str = "none", epilogue: str = "plain",
         single_sm: bool = False, compute_only: bool = False, split_layer: bool = False,
         pairs: bool = False) -> FoOpts:
    tiles = 2 if pairs else int(single_sm)  # fo_opts.sm_pairs
    return FoOpts(ORDERS[order], LINKS[link], n_slices, timeout_us, int(causal_prune), num_sms, FAULTS[fault],
                  EPILOGUES[epilogue], tiles, int(compute_only), int(split_layer), 0)


def _stream(stream) -> ctypes.c_void_p:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


class RopeTable:
    """Frequencies of rotary positions: pair i turns by base^(-2i/rot_dim) radians per position, scaled for a
    longer context by ``scaling`` ("linear": all by 1/factor; "banded": pairs that turn fewer than low_factor
    times over original_length positions by 1/factor, more than high_factor times not; "ramped": by pair index
    between those that turn beta_fast and beta_slow times, with an amplitude).  Host only."""

    def __init__(self, rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                 low_factor: float = 1.0, high_factor: float = 4.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 original_length: int = 0):
        low, high = (beta_slow, beta_fast) if scaling == "ramped" else (low_factor, high_factor)
        how = FoRopeScaling(ROPE_SCALINGS[scaling], 0, factor, low, high, original_length)
        self.c = FoRopeTable()
        _check(load().fo_rope_table_init(ctypes.byref(self.c), rot_dim, base, ctypes.byref(how)))

    @property
    def rot_dim(self) -> int:
        return self.c.rot_dim


class Context:
    """Owns one fo_ctx (link streams, ring workspace, flags) on one device."""

    def __init__(self, device: int = 0):
        self._lib = load()
        self._h = ctypes.c_void_p()
        _check(self._lib.fo_ctx_create(device, ctypes.byref(self._h)))
        self.device = device

    def close(self) -> None:
        if self._h:
            self._lib.fo_ctx_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def poll(self) -> None:
        """Raises FoError if a device wait of an earlier (synchronised) call gave up."""
        _check(self._lib.fo_ctx_poll(self._h))

    def phase_ms(self) -> tuple[float, float]:
        """(collective_ms, gemm_ms) of the last serial-baseline call."""
        a, b = ctypes.c_float(), ctypes.c_float()
        _check(self._lib.fo_ctx_phase_ms(self._h, ctypes.byref(a), ctypes.byref(b)))
        return a.value, b.value

    def gemm(self, A, B, C, stream=None, **kw) -> None:
        o = opts(**kw)
        _check(self._lib.fo_gemm(self._h, ctypes.byref(mat(A)), ctypes.byref(mat(B)), ctypes.byref(mat(C)),
                                 ctypes.byref(o), _stream(stream)))

    def ag_gemm(self, X_shards, W_col, Y, stream=None, **kw) -> None:
        P = len(X_shards)
        o = opts(**kw)
        _check(self._lib.fo_ag_gemm(self._h, _mats(X_shards), _mats(W_col), P, _mats(Y), ctypes.byref(o),
                                    _stream(stream)))

    def gemm_rs(self, X, W_row, Y, stream=None, **kw) -> None:
        P = len(X)
        o = opts(**kw)
        _check(self._lib.fo_gemm_rs(self._h, _mats(X), _mats(W_row), P, _mats(Y), ctypes.byref(o),
                                    _stream(stream)))

    def gemm_a2a(self, X_shards, W, Y, stream=None, **kw) -> None:
        """Y[d][rows r*m..] = X_shards[r] W[r][rows d*Nb..]^T (the all-to-all's producer GEMM)."""
        P = len(X_shards)
        o = opts(**kw)
        _check(self._lib.fo_gemm_a2a(self._h, _mats(X_shards), _mats(W), P, _mats(Y), ctypes.byref(o),
                                     _stream(stream)))

    def a2a_gemm(self, C, W, Y, stream=None, **kw) -> None:
        """Y[d] = [C[0] rows d*m.. | ... | C[P-1] rows d*m..] W[d]^T (the all-to-all's consumer GEMM)."""
        P = len(C)
        o = opts(**kw)
        _check(self._lib.fo_a2a_gemm(self._h, _mats(C), _mats(W), P, _mats(Y), ctypes.byref(o), _stream(stream)))

    def col_linear_backward(self, X_shards, W_col, dY, dX, dW, stream=None, **kw) -> None:
        """Backward of Y[r] = AG(X) W_col[r]^T: dX (token slices, Flash-RS) and dW (per rank)."""
        P = len(X_shards)
        o = opts(**kw)
        _check(self._lib.fo_col_linear_backward(self._h, _mats(X_shards), _mats(W_col), _mats(dY), P, _mats(dX),
                                                _mats(dW), ctypes.byref(o), _stream(stream)))

    def row_linear_backward(self, H, W_row, dZ_shards, dH, dW, stream=None, **kw) -> None:
        """Backward of Z = RS(H[r] W_row[r]^T): dH (Flash-AG) and dW (per rank)."""
        P = len(H)
        o = opts(**kw)
        _check(self._lib.fo_row_linear_backward(self._h, _mats(H), _mats(W_row), _mats(dZ_shards), P, _mats(dH),
                                                _mats(dW), ctypes.byref(o), _stream(stream)))

    def silu_mul(self, GU, H, stream=None) -> None:
        _check(self._lib.fo_silu_mul(self._h, _mats(GU), len(GU), _mats(H), _stream(stream)))

    def mlp_layer(self, X_shards, W_col, W_row, Z, gated: bool, stream=None, **kw) -> None:
        P = len(X_shards)
        o = opts(**kw)
        _check(self._lib.fo_mlp_layer(self._h, _mats(X_shards), _mats(W_col), _mats(W_row), P, int(gated),
                                      _mats(Z), ctypes.byref(o), _stream(stream)))

    def mlp_layer_host(self, X_shards, W_col, W_row, Z, gated: bool, stream=None, **kw) -> None:
        """X_shards and Z are CPU tensors (pinned for asynchronous copies)."""
        P = len(X_shards)
        o = opts(**kw)
        _check(self._lib.fo_mlp_layer_host(self._h, _mats(X_shards), _mats(W_col), _mats(W_row), P, int(gated),
                                           _mats(Z), ctypes.byref(o), _stream(stream)))

    def qsplit_attn(self, Q, K, V, O, heads: int, head_dim: int, causal: bool = True, stream=None, **kw) -> None:
        P = len(Q)
        o = opts(**kw)
        _check(self._lib.fo_qsplit_attn(self._h, _mats(Q), _mats(K), _mats(V), P, heads, head_dim, int(causal),
                                        _mats(O), ctypes.byref(o), _stream(stream)))

    def attn_layer(self, X_shards, W_qkv, W_o, Z, heads: int, head_dim: int = 128, causal: bool = True,
                   stream=None, **kw) -> None:
        """Flash-AG QKV projection -> per-rank causal attention -> Flash-RS output projection."""
        P = len(X_shards)
        o = opts(**kw)
        _check(self._lib.fo_attn_layer(self._h, _mats(X_shards), _mats(W_qkv), _mats(W_o), P, heads, head_dim,
                                       int(causal), _mats(Z), ctypes.byref(o), _stream(stream)))


    # -- training operators ------------------------------------------------------------------

    def _list(self, ts, P: int, what: str):
        """P matrices on the context's device (None stays None)."""
        if ts is None:
            return None
        if len(ts) != P or P >= len(_MAT_ARRAYS):
            raise ValueError(f"{what}: {len(ts)} matrices for {P} ranks")
        arr = _MAT_ARRAYS[P]()
        at = 0
        codes = _DTYPE_CODES or _dtype_codes()
        for t in ts:
            if t.get_device() != self.device:
                self._here(t, what)
            dt, shape, stride = codes.get(t.dtype), t.shape, t.stride()
            if dt is None or len(shape) != 2 or (stride[1] != 1 and shape[1] > 1) or stride[0] < shape[1]:
                m = mat(t)
                ptr, dt, rows, cols, ld = m.ptr, m.dtype, m.rows, m.cols, m.ld
            else:
                ptr, (rows, cols), ld = t.data_ptr(), shape, stride[0]
            if rows <= 1:  # the row pitch of one row is not used: any whole number of 16 bytes
                ld = cols + 7 & -8
            _PACK_MAT(arr, at, ptr or 0, dt, 0, rows, cols, ld)
            at += _MAT_BYTES
        return arr

    def _here(self, t, what: str) -> None:
        if t.device.type != "cuda" or t.device.index != self.device:
            raise ValueError(f"{what} is on {t.device}, the context on cuda:{self.device}")

    def _vector(self, t, what: str):
        """[1, H] matrix of a vector (None stays None)."""
        if t is None:
            return None
        dt = (_DTYPE_CODES or _dtype_codes()).get(t.dtype)
        if dt is None or t.dim() != 1 or (t.stride(0) != 1 and t.shape[0] > 1):
            raise ValueError(f"{what} must be a contiguous bf16 or fp32 vector")
        if t.get_device() != self.device:
            self._here(t, what)
        arr, n = _MAT_ARRAYS[1](), t.shape[0]
        _PACK_MAT(arr, 0, t.data_ptr(), dt, 0, 1, n, n + 7 & -8)
        return arr

    def _own_stream(self, stream):
        if stream is None:
            import torch
            stream = torch.cuda.current_stream(self.device)
        return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))

    def _mask(self, causal, scale, q_offsets, k_offsets):
        import torch
        if q_offsets is None and k_offsets is not None:
            raise ValueError("k_offsets without q_offsets")
        for t, what in ((q_offsets, "q_offsets"), (k_offsets, "k_offsets")):
            if t is None:
                continue
            self._here(t, what)
            if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.numel() < 2:
                raise ValueError(f"{what} must be a contiguous int32 vector of num_seqs + 1 entries")
            if t.numel() != q_offsets.numel():
                raise ValueError("q_offsets and k_offsets must have one length")
        if scale is not None and not scale > 0:
            raise ValueError("scale must be positive")
        return FoAttnMask(int(causal), 0 if q_offsets is None else q_offsets.numel() - 1,
                          None if q_offsets is None else q_offsets.data_ptr(),
                          None if k_offsets is None else k_offsets.data_ptr(), 0.0 if scale is None else scale, 0)

    def attn_forward(self, Q, K, V, O, LSE, heads: int, kv_heads: int | None = None, head_dim: int = 128,
                     causal: bool = True, scale: float | None = None, q_offsets=None, k_offsets=None, stream=None,
                     **kw) -> None:
        """O = softmax(scale Q K^T) V per rank and head, LSE [heads, tokens] its row statistics.  kv_heads < heads:
        shared key/value heads.  q_offsets / k_offsets: int32 tensors, boundaries of packed sequences."""
        P = len(Q)
        m = self._mask(causal, scale, q_offsets, k_offsets)
        o = opts(**kw)
        _check(self._lib.fo_attn_forward(
            self._h, self._list(Q, P, "Q"), self._list(K, P, "K"), self._list(V, P, "V"), P, heads,
            heads if kv_heads is None else kv_heads, head_dim, ctypes.byref(m), self._list(O, P, "O"),
            self._list(LSE, P, "LSE"), ctypes.byref(o), self._own_stream(stream)))

    def attn_backward(self, Q, K, V, O, LSE, dO, dQ, dK, dV, heads: int, kv_heads: int | None = None,
                      head_dim: int = 128, causal: bool = True, scale: float | None = None, q_offsets=None,
                      k_offsets=None, stream=None, **kw) -> None:
        """Gradients dQ, dK, dV of attn_forward from its inputs, its O and LSE, and dO."""
        P = len(Q)
        m = self._mask(causal, scale, q_offsets, k_offsets)
        o = opts(**kw)
        _check(self._lib.fo_attn_backward(
            self._h, self._list(Q, P, "Q"), self._list(K, P, "K"), self._list(V, P, "V"), self._list(O, P, "O"),
            self._list(LSE, P, "LSE"), self._list(dO, P, "dO"), P, heads, heads if kv_heads is None else kv_heads,
            head_dim, ctypes.byref(m), self._list(dQ, P, "dQ"), self._list(dK, P, "dK"), self._list(dV, P, "dV"),
            ctypes.byref(o), self._own_stream(stream)))

    def _norm_params(self, P, w_post, gate, w_pre, residual_scale, eps, what="gate"):
        token = gate is not None and isinstance(gate, (list, tuple))
        g = self._list(gate, P, what) if token else self._vector(gate, what)
        return FoNormParams(self._vector(w_post, "w_post"), self._vector(w_pre, "w_pre"), g, int(token),
                            residual_scale, eps, 0)

    def norm_residual(self, R, Y, R_out, X, w_post=None, gate=None, w_pre=None, residual_scale: float = 1.0,
                      eps: float = 1e-6, stream=None) -> None:
        """R_out = residual_scale R + gate (w_post Y / rms(Y)); X = w_pre R_out / rms(R_out), per rank's token slice.
        gate: None, a vector, or a list of P matrices (per token).  Y and R_out None: X from R alone.  X None: no
        norm behind (w_pre None)."""
        P = len(R)
        prm = self._norm_params(P, w_post, gate, w_pre, residual_scale, eps)
        _check(self._lib.fo_norm_residual(self._h, self._list(R, P, "R"), self._list(Y, P, "Y"), P, ctypes.byref(prm),
                                          self._list(R_out, P, "R_out"), self._list(X, P, "X"),
                                          self._own_stream(stream)))

    def norm_residual_backward(self, R_out, Y, dX, dR_out, dR, dY, w_post=None, gate=None, w_pre=None, dw_post=None,
                               dgate=None, dw_pre=None, residual_scale: float = 1.0, eps: float = 1e-6,
                               stream=None) -> None:
        """Backward of norm_residual: dR, dY and the parameters' gradients (vectors summed over all ranks' tokens;
        a per-token gate's as a list of P matrices)."""
        P = len(R_out)
        prm = self._norm_params(P, w_post, gate, w_pre, residual_scale, eps)
        got = self._norm_params(P, dw_post, dgate, dw_pre, residual_scale, eps, "dgate")
        if (dgate is not None) != (gate is not None) or got.gate_per_token != prm.gate_per_token:
            raise ValueError("dgate must have gate's form")
        grads = FoNormGrads(got.w_post, got.w_pre, got.gate)
        _check(self._lib.fo_norm_residual_backward(
            self._h, self._list(R_out, P, "R_out"), self._list(Y, P, "Y"), self._list(dX, P, "dX"),
            self._list(dR_out, P, "dR_out"), P, ctypes.byref(prm), self._list(dR, P, "dR"), self._list(dY, P, "dY"),
            ctypes.byref(grads), self._own_stream(stream)))

    def _rope(self, call, X, Y, table, head_dim, layout, positions, start, rank_stride, stream) -> None:
        import torch
        P = len(X)
        pos = None
        if positions is not None:
            if len(positions) != P:
                raise ValueError(f"positions: {len(positions)} vectors for {P} ranks")
            for t, x in zip(positions, X):
                self._here(t, "positions")
                if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.numel() != x.shape[0]:
                    raise ValueError("positions must be contiguous int32 vectors, one entry per row")
            pos = (ctypes.c_void_p * P)(*(t.data_ptr() for t in positions))
        _check(call(self._h, self._list(X, P, "X"), P, ctypes.byref(table.c),
                    table.rot_dim if head_dim is None else head_dim, ROPE_LAYOUTS[layout], pos, start, rank_stride,
                    self._list(Y, P, "Y"), self._own_stream(stream)))

    def rope(self, X, Y, table: RopeTable, head_dim: int | None = None, layout: str = "half", positions=None,
             start: int = 0, rank_stride: int = 0, stream=None) -> None:
        """Turns the heads of X into Y (Y may be X).  Row i of rank r is at positions[r][i], or at
        start + r * rank_stride + i."""
        self._rope(self._lib.fo_rope, X, Y, table, head_dim, layout, positions, start, rank_stride, stream)

    def rope_backward(self, dY, dX, table: RopeTable, head_dim: int | None = None, layout: str = "half",
                      positions=None, start: int = 0, rank_stride: int = 0, stream=None) -> None:
        """dX from the gradient dY of rope's output (dX may be dY)."""
        self._rope(self._lib.fo_rope_backward, dY, dX, table, head_dim, layout, positions, start, rank_stride, stream)


def step_order(op: str, P: int, order: str = "flash") -> list[list[tuple[int, int]]]:
    """The library's launch order: per step, (rank, slice or chunk) of each unit."""
    lib = load()
    n = P * P
    rank = (ctypes.c_int32 * n)()
    item = (ctypes.c_int32 * n)()
    got = lib.fo_step_order({"ag": 0, "rs": 1, "gemm_a2a": 2, "a2a_gemm": 3}[op], P, ORDERS[order], rank, item, n)
    if got != n:
        raise FoError(FO_ERR_INVALID_ARG, "bad step-order request")
    return [[(rank[t * P + i], item[t * P + i]) for i in range(P)] for t in range(P)]
