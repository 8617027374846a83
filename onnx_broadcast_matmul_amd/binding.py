"""ctypes binding of libmm.so (argument marshalling only).

Every computation runs in the HIP kernels behind the C ABI declared in
``include/mm.h``; this module converts shapes and torch tensors to the plain
pointers and sizes the ABI takes, and raises on error statuses.  There is no
fallback: if ``libmm.so`` is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Optional, Sequence, Tuple

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmm.so")

FLOAT, FLOAT16, DOUBLE, BFLOAT16 = 1, 10, 11, 16
UINT8, INT8, INT32 = 2, 3, 6
ZP_NONE, ZP_SCALAR, ZP_VECTOR = 0, 1, 2
ACT_NONE = 0
ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_RELU, ACT_SIGMOID = 1, 2, 3, 4, 5
ACTIVATIONS = {"silu": ACT_SILU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH, "relu": ACT_RELU,
               "sigmoid": ACT_SIGMOID}
NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
NORM_MAX_COLS = 16384
MAX_BATCH_DIMS = 8
MAX_RANK = MAX_BATCH_DIMS + 2

ALGO_AUTO, ALGO_EMPTY, ALGO_ZERO_FILL, ALGO_DIRECT = 0, 1, 2, 3
ALGO_SKINNY_M, ALGO_SKINNY_N, ALGO_SPLIT_K, ALGO_GENERAL = 4, 5, 6, 7
ALGO_NAMES = {0: "auto", 1: "empty", 2: "zero_fill", 3: "direct", 4: "skinny_m", 5: "skinny_n",
              6: "split_k", 7: "general"}

ERR_NULL_ARG, ERR_RANK, ERR_NEG_DIM, ERR_K_MISMATCH, ERR_BROADCAST = 1, 2, 3, 4, 5
ERR_DTYPE, ERR_BAD_OPTION, ERR_TOO_LARGE, ERR_ALLOC, ERR_HIP = 6, 7, 8, 9, 10
ERR_SIZE, ERR_NO_CONSTANT_B = 11, 12


class MMError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"mm status {status}: {detail}")
        self.status = status
        self.detail = detail


class PlanOptions(ctypes.Structure):
    _fields_ = [("force_algo", ctypes.c_int32), ("tile", ctypes.c_int32), ("split_k", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class PlanInfo(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("algo", ctypes.c_int32),
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("batch", ctypes.c_int64), ("kernel_m", ctypes.c_int64),
        ("folded", ctypes.c_int32), ("batch_rank", ctypes.c_int32),
        ("batch_dims", ctypes.c_int64 * MAX_BATCH_DIMS),
        ("a_batch_strides", ctypes.c_int64 * MAX_BATCH_DIMS),
        ("b_batch_strides", ctypes.c_int64 * MAX_BATCH_DIMS),
        ("tile", ctypes.c_int32), ("split_k", ctypes.c_int32),
        ("k_chunk", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
        ("flops", ctypes.c_double), ("min_bytes", ctypes.c_double),
        ("tail_col", ctypes.c_int64), ("tail_tile", ctypes.c_int32), ("constant_b_packed", ctypes.c_int32),
    ]


class GemmDesc(ctypes.Structure):
    _fields_ = [
        ("a_rows", ctypes.c_int64), ("a_cols", ctypes.c_int64),
        ("b_rows", ctypes.c_int64), ("b_cols", ctypes.c_int64),
        ("trans_a", ctypes.c_int32), ("trans_b", ctypes.c_int32),
        ("c_rank", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("c_shape", ctypes.c_int64 * 2),
        ("alpha", ctypes.c_float), ("beta", ctypes.c_float),
    ]


class ScaledIntDesc(ctypes.Structure):
    _fields_ = [("a_type", ctypes.c_int32), ("out_type", ctypes.c_int32), ("trans_b", ctypes.c_int32),
                ("has_bias", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class GluDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("in_features", ctypes.c_int64), ("hidden", ctypes.c_int64),
                ("w_pitch", ctypes.c_int64), ("trans_w", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("training", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class GluOptions(ctypes.Structure):
    _fields_ = [("kept_type", ctypes.c_int32), ("dx_tile", ctypes.c_int32), ("dx_split_k", ctypes.c_int32),
                ("dw_tile", ctypes.c_int32), ("dw_split_k", ctypes.c_int32)]


class LinearDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("in_features", ctypes.c_int64), ("out_features", ctypes.c_int64),
                ("w_pitch", ctypes.c_int64), ("trans_w", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("has_bias", ctypes.c_int32), ("has_residual", ctypes.c_int32), ("training", ctypes.c_int32),
                ("z_type", ctypes.c_int32), ("x_type", ctypes.c_int32), ("x_activation", ctypes.c_int32),
                ("dx_tile", ctypes.c_int32), ("dx_split_k", ctypes.c_int32), ("dw_tile", ctypes.c_int32),
                ("dw_split_k", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class LinearTails(ctypes.Structure):
    _fields_ = [("dx_col", ctypes.c_int64), ("dw_col", ctypes.c_int64), ("dx_tile", ctypes.c_int32),
                ("dw_tile", ctypes.c_int32)]


class NormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("gate_rows", ctypes.c_int64),
                ("post_norm", ctypes.c_int32), ("pre_norm", ctypes.c_int32), ("post_eps", ctypes.c_float),
                ("pre_eps", ctypes.c_float), ("residual_scale", ctypes.c_float), ("has_block", ctypes.c_int32),
                ("post_weight", ctypes.c_int32), ("post_bias", ctypes.c_int32), ("pre_weight", ctypes.c_int32),
                ("pre_bias", ctypes.c_int32), ("training", ctypes.c_int32), ("kept_type", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class NormForwardArgs(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in
                ("residual", "block", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias", "sum", "out",
                 "stats", "sum_f32", "sum_q", "sum_scale", "block_q", "block_scale", "out_q", "out_scale")]


class NormBackwardArgs(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in
                ("stats", "sum", "sum_scale", "block", "block_scale", "gate", "post_weight", "post_bias", "pre_weight",
                 "dout", "dsum", "dresidual", "dblock", "dgate", "dpost_weight", "dpost_bias", "dpre_weight",
                 "dpre_bias")]


_lib = None
_lib_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """Load libmm.so (raises if it has not been built)."""
    global _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "or python -m onnx_broadcast_matmul_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        i64p = ctypes.POINTER(ctypes.c_int64)
        vp = ctypes.c_void_p
        L.mm_plan_create.argtypes = [i64p, ctypes.c_int, i64p, ctypes.c_int, ctypes.c_int, ctypes.POINTER(vp)]
        L.mm_plan_create.restype = ctypes.c_int
        L.mm_plan_create_ex.argtypes = [i64p, ctypes.c_int, i64p, ctypes.c_int, ctypes.c_int,
                                        ctypes.POINTER(PlanOptions), ctypes.POINTER(vp)]
        L.mm_plan_create_ex.restype = ctypes.c_int
        L.mm_plan_destroy.argtypes = [vp]
        L.mm_plan_destroy.restype = None
        L.mm_execute.argtypes = [vp, vp, vp, vp, vp]
        L.mm_execute.restype = ctypes.c_int
        L.mm_execute_noalloc.argtypes = [vp, vp, vp, vp, vp]
        L.mm_execute_noalloc.restype = ctypes.c_int
        L.mm_plan_output_shape.argtypes = [vp, i64p, ctypes.POINTER(ctypes.c_int)]
        L.mm_plan_output_shape.restype = ctypes.c_int
        L.mm_plan_output_numel.argtypes = [vp]
        L.mm_plan_output_numel.restype = ctypes.c_int64
        L.mm_plan_algo.argtypes = [vp]
        L.mm_plan_algo.restype = ctypes.c_int
        L.mm_plan_workspace_bytes.argtypes = [vp]
        L.mm_plan_workspace_bytes.restype = ctypes.c_size_t
        L.mm_plan_get_info.argtypes = [vp, ctypes.POINTER(PlanInfo)]
        L.mm_plan_get_info.restype = ctypes.c_int
        L.mm_tile_count.argtypes = [ctypes.c_int]
        L.mm_tile_count.restype = ctypes.c_int
        L.mm_tile_config.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                     ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
        L.mm_tile_config.restype = ctypes.c_int
        L.mm_plan_set_constant_b.argtypes = [vp, vp, ctypes.c_int64, vp]
        L.mm_plan_set_constant_b.restype = ctypes.c_int
        L.mm_plan_has_constant_b.argtypes = [vp]
        L.mm_plan_has_constant_b.restype = ctypes.c_int
        L.mm_execute_constant_b.argtypes = [vp, vp, vp, vp]
        L.mm_execute_constant_b.restype = ctypes.c_int
        L.mm_gemm_plan_create.argtypes = [ctypes.POINTER(GemmDesc), ctypes.c_int, ctypes.POINTER(PlanOptions),
                                           ctypes.POINTER(vp)]
        L.mm_gemm_plan_create.restype = ctypes.c_int
        L.mm_gemm_execute.argtypes = [vp, vp, vp, vp, vp, vp]
        L.mm_gemm_execute.restype = ctypes.c_int
        L.mm_int_plan_create.argtypes = [i64p, ctypes.c_int, i64p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                          ctypes.c_int, ctypes.c_int, ctypes.POINTER(PlanOptions), ctypes.POINTER(vp)]
        L.mm_int_plan_create.restype = ctypes.c_int
        L.mm_int_execute.argtypes = [vp, vp, vp, vp, vp, vp, vp]
        L.mm_int_execute.restype = ctypes.c_int
        L.mm_scaled_int_plan_create.argtypes = [i64p, ctypes.c_int, i64p, ctypes.c_int, ctypes.POINTER(ScaledIntDesc),
                                                 ctypes.POINTER(PlanOptions), ctypes.POINTER(vp)]
        L.mm_scaled_int_plan_create.restype = ctypes.c_int
        L.mm_scaled_int_execute.argtypes = [vp] * 8
        L.mm_scaled_int_execute.restype = ctypes.c_int
        L.mm_quantize_rows.argtypes = [vp, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, vp, vp, vp]
        L.mm_quantize_rows.restype = ctypes.c_int
        L.mm_glu_plan_create.argtypes = [ctypes.POINTER(GluDesc), ctypes.c_int, ctypes.POINTER(PlanOptions),
                                         ctypes.POINTER(vp)]
        L.mm_glu_plan_create.restype = ctypes.c_int
        L.mm_glu_plan_create_ex.argtypes = [ctypes.POINTER(GluDesc), ctypes.c_int, ctypes.POINTER(PlanOptions),
                                            ctypes.POINTER(GluOptions), ctypes.POINTER(vp)]
        L.mm_glu_plan_create_ex.restype = ctypes.c_int
        L.mm_glu_get_options.argtypes = [vp, ctypes.POINTER(GluOptions)]
        L.mm_glu_get_options.restype = ctypes.c_int
        L.mm_glu_execute.argtypes = [vp] * 8
        L.mm_glu_execute.restype = ctypes.c_int
        L.mm_glu_backward.argtypes = [vp] * 11
        L.mm_glu_backward.restype = ctypes.c_int
        L.mm_checkpoint_blocks.argtypes = [ctypes.c_int64]
        L.mm_checkpoint_blocks.restype = ctypes.c_int64
        L.mm_checkpoint_pack.argtypes = [vp, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, vp, vp, vp]
        L.mm_checkpoint_pack.restype = ctypes.c_int
        L.mm_checkpoint_unpack.argtypes = [vp, vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, vp, vp]
        L.mm_checkpoint_unpack.restype = ctypes.c_int
        L.mm_linear_plan_create.argtypes = [ctypes.POINTER(LinearDesc), ctypes.c_int, ctypes.POINTER(PlanOptions),
                                            ctypes.POINTER(vp)]
        L.mm_linear_plan_create.restype = ctypes.c_int
        L.mm_linear_get_desc.argtypes = [vp, ctypes.POINTER(LinearDesc)]
        L.mm_linear_get_desc.restype = ctypes.c_int
        L.mm_linear_get_tails.argtypes = [vp, ctypes.POINTER(LinearTails)]
        L.mm_linear_get_tails.restype = ctypes.c_int
        L.mm_linear_execute.argtypes = [vp] * 9
        L.mm_linear_execute.restype = ctypes.c_int
        L.mm_linear_backward.argtypes = [vp] * 11
        L.mm_linear_backward.restype = ctypes.c_int
        L.mm_norm_plan_create.argtypes = [ctypes.POINTER(NormDesc), ctypes.c_int, ctypes.POINTER(vp)]
        L.mm_norm_plan_create.restype = ctypes.c_int
        L.mm_norm_execute.argtypes = [vp, ctypes.POINTER(NormForwardArgs), vp]
        L.mm_norm_execute.restype = ctypes.c_int
        L.mm_norm_backward.argtypes = [vp, ctypes.POINTER(NormBackwardArgs), vp]
        L.mm_norm_backward.restype = ctypes.c_int
        L.mm_status_string.argtypes = [ctypes.c_int]
        L.mm_status_string.restype = ctypes.c_char_p
        L.mm_last_error.argtypes = []
        L.mm_last_error.restype = ctypes.c_char_p
        _lib = L
        return L


def _check(status: int) -> None:
    if status != 0:
        L = lib()
        detail = (L.mm_last_error() or b"").decode() or L.mm_status_string(status).decode()
        raise MMError(status, detail)


def _shape(shape: Sequence[int]):
    return (ctypes.c_int64 * max(1, len(shape)))(*[int(d) for d in shape])


_dtype_codes = {}


def torch_dtype_code(dt) -> int:
    code = _dtype_codes.get(dt)
    if code is None:
        import torch

        _dtype_codes.update({torch.float32: FLOAT, torch.float16: FLOAT16, torch.bfloat16: BFLOAT16,
                             torch.float64: DOUBLE})
        code = _dtype_codes.get(dt)
        if code is None:
            raise TypeError(f"unsupported tensor dtype {dt}")
    return code


def torch_dtype(code: int):
    import torch

    return {FLOAT: torch.float32, FLOAT16: torch.float16, BFLOAT16: torch.bfloat16, DOUBLE: torch.float64,
            INT32: torch.int32, INT8: torch.int8, UINT8: torch.uint8}[code]


def tile_configs(dtype: int):
    L = lib()
    out = []
    for i in range(L.mm_tile_count(dtype)):
        bm, bn, bk = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
        _check(L.mm_tile_config(dtype, i, ctypes.byref(bm), ctypes.byref(bn), ctypes.byref(bk)))
        out.append((bm.value, bn.value, bk.value))
    return out


class Plan:
    """mm_plan_create / mm_execute / mm_plan_destroy for one (A shape, B shape, dtype)."""

    def __init__(self, a_shape: Sequence[int], b_shape: Sequence[int], dtype: int, force_algo: int = 0,
                 tile: int = 0, split_k: int = 0):
        L = lib()
        self._handle = ctypes.c_void_p()
        self.a_shape = tuple(int(d) for d in a_shape)
        self.b_shape = tuple(int(d) for d in b_shape)
        self.dtype = int(dtype)
        if force_algo or tile or split_k:
            opt = PlanOptions(force_algo, tile, split_k, 0)
            st = L.mm_plan_create_ex(_shape(self.a_shape), len(self.a_shape), _shape(self.b_shape),
                                     len(self.b_shape), self.dtype, ctypes.byref(opt), ctypes.byref(self._handle))
        else:
            st = L.mm_plan_create(_shape(self.a_shape), len(self.a_shape), _shape(self.b_shape),
                                  len(self.b_shape), self.dtype, ctypes.byref(self._handle))
        _check(st)
        self._lock = threading.Lock()

    def close(self) -> None:
        """mm_plan_destroy (the caller makes sure no execution is in flight)."""
        h = getattr(self, "_handle", None)
        if h is not None and h.value and _lib is not None:
            _lib.mm_plan_destroy(h)
            self._handle = ctypes.c_void_p()

    def __del__(self):
        self.close()

    @property
    def handle(self) -> ctypes.c_void_p:
        return self._handle

    @property
    def output_shape(self) -> Tuple[int, ...]:
        shp = (ctypes.c_int64 * MAX_RANK)()
        rank = ctypes.c_int()
        _check(lib().mm_plan_output_shape(self._handle, shp, ctypes.byref(rank)))
        return tuple(shp[i] for i in range(rank.value))

    @property
    def output_numel(self) -> int:
        return int(lib().mm_plan_output_numel(self._handle))

    @property
    def algo(self) -> int:
        return int(lib().mm_plan_algo(self._handle))

    @property
    def workspace_bytes(self) -> int:
        return int(lib().mm_plan_workspace_bytes(self._handle))

    def info(self) -> dict:
        inf = PlanInfo()
        _check(lib().mm_plan_get_info(self._handle, ctypes.byref(inf)))
        nb = inf.batch_rank
        return {
            "dtype": inf.dtype, "algo": inf.algo, "algo_name": ALGO_NAMES.get(inf.algo, "?"),
            "M": inf.M, "N": inf.N, "K": inf.K, "batch": inf.batch, "kernel_m": inf.kernel_m,
            "folded": bool(inf.folded), "batch_dims": tuple(inf.batch_dims[:nb]),
            "a_batch_strides": tuple(inf.a_batch_strides[:nb]), "b_batch_strides": tuple(inf.b_batch_strides[:nb]),
            "tile": inf.tile, "split_k": inf.split_k, "k_chunk": inf.k_chunk,
            "workspace_bytes": inf.workspace_bytes, "flops": inf.flops, "min_bytes": inf.min_bytes,
            "tail_col": inf.tail_col, "tail_tile": inf.tail_tile, "constant_b_packed": inf.constant_b_packed,
        }

    def execute_ptr(self, A: int, B: int, Y: int, stream: int = 0) -> None:
        """mm_execute on raw device pointers and a raw hipStream_t."""
        _check(lib().mm_execute(self._handle, ctypes.c_void_p(A), ctypes.c_void_p(B), ctypes.c_void_p(Y),
                                ctypes.c_void_p(stream)))

    def execute_noalloc_ptr(self, A: int, B: int, Y: int, stream: int = 0) -> None:
        """mm_execute_noalloc on raw device pointers and a raw hipStream_t."""
        _check(lib().mm_execute_noalloc(self._handle, ctypes.c_void_p(A), ctypes.c_void_p(B), ctypes.c_void_p(Y),
                                        ctypes.c_void_p(stream)))

    def execute_noalloc(self, A, B, Y, stream=None) -> None:
        """mm_execute_noalloc on torch device tensors (checked as in execute)."""
        self.execute(A, B, Y, stream, _entry=self.execute_noalloc_ptr)

    def execute(self, A, B, Y, stream=None, _entry=None) -> None:
        """mm_execute on torch device tensors; ``stream`` is a torch.cuda.Stream
        (default: the current stream of Y's device)."""
        import torch

        want = torch_dtype(self.dtype)
        for name, t, shape in (("A", A, self.a_shape), ("B", B, self.b_shape), ("Y", Y, self.output_shape)):
            if t.dtype != want:
                raise TypeError(f"{name} has dtype {t.dtype}, plan expects {want}")
            if tuple(t.shape) != tuple(shape):
                raise ValueError(f"{name} has shape {tuple(t.shape)}, plan expects {tuple(shape)}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            if t.numel() and not t.is_cuda:
                raise ValueError(f"{name} must be a device tensor")
        if stream is None:
            stream = torch.cuda.current_stream(Y.device)
        with self._lock:
            (_entry or self.execute_ptr)(A.data_ptr(), B.data_ptr(), Y.data_ptr(), stream.cuda_stream)

    # ---- plan-owned constant B
    def set_constant_b_ptr(self, B: int, numel: int, stream: int = 0) -> None:
        """mm_plan_set_constant_b on a raw device pointer (copy completes before return)."""
        _check(lib().mm_plan_set_constant_b(self._handle, ctypes.c_void_p(B), ctypes.c_int64(numel),
                                            ctypes.c_void_p(stream)))

    def set_constant_b(self, B, stream=None) -> None:
        """Copy the device tensor B (the planned B shape and type) into plan-owned storage."""
        import torch

        if B.dtype != torch_dtype(self.dtype) or tuple(B.shape) != self.b_shape or not B.is_contiguous():
            raise ValueError(f"B must be a contiguous {torch_dtype(self.dtype)} tensor of shape {self.b_shape}")
        if stream is None:
            stream = torch.cuda.current_stream(B.device)
        with self._lock:
            self.set_constant_b_ptr(B.data_ptr(), B.numel(), stream.cuda_stream)

    @property
    def has_constant_b(self) -> bool:
        return bool(lib().mm_plan_has_constant_b(self._handle))

    def execute_constant_b_ptr(self, A: int, Y: int, stream: int = 0) -> None:
        """mm_execute_constant_b on raw device pointers."""
        _check(lib().mm_execute_constant_b(self._handle, ctypes.c_void_p(A), ctypes.c_void_p(Y),
                                           ctypes.c_void_p(stream)))

    def execute_constant_b(self, A, Y, stream=None) -> None:
        """mm_execute_constant_b on torch device tensors (B is the plan's own)."""
        import torch

        want = torch_dtype(self.dtype)
        for name, t, shape in (("A", A, self.a_shape), ("Y", Y, self.output_shape)):
            if t.dtype != want or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {want} tensor of shape {tuple(shape)}")
        if stream is None:
            stream = torch.cuda.current_stream(Y.device)
        with self._lock:
            self.execute_constant_b_ptr(A.data_ptr(), Y.data_ptr(), stream.cuda_stream)


class GemmPlan(Plan):
    """mm_gemm_plan_create / mm_gemm_execute: ONNX Gemm of rank-2 A, B with
    transA / transB, alpha, beta and an optional C broadcast to [M, N]."""

    def __init__(self, a_shape, b_shape, dtype: int, trans_a: bool = False, trans_b: bool = False,
                 c_shape=None, alpha: float = 1.0, beta: float = 1.0, force_algo: int = 0, tile: int = 0,
                 split_k: int = 0):
        L = lib()
        self._handle = ctypes.c_void_p()
        self.a_shape = tuple(int(d) for d in a_shape)
        self.b_shape = tuple(int(d) for d in b_shape)
        self.c_shape = None if c_shape is None else tuple(int(d) for d in c_shape)
        self.dtype = int(dtype)
        if len(self.a_shape) != 2 or len(self.b_shape) != 2:
            raise ValueError("Gemm takes rank-2 A and B")
        d = GemmDesc()
        d.a_rows, d.a_cols = self.a_shape
        d.b_rows, d.b_cols = self.b_shape
        d.trans_a, d.trans_b = int(trans_a), int(trans_b)
        d.c_rank = -1 if self.c_shape is None else len(self.c_shape)
        for i, v in enumerate(self.c_shape or ()):
            d.c_shape[i] = v
        d.alpha, d.beta = float(alpha), float(beta)
        opt = PlanOptions(force_algo, tile, split_k, 0)
        _check(L.mm_gemm_plan_create(ctypes.byref(d), self.dtype, ctypes.byref(opt), ctypes.byref(self._handle)))
        self._lock = threading.Lock()

    def execute_ptr(self, A: int, B: int, Y: int, stream: int = 0, C: int = 0) -> None:
        _check(lib().mm_gemm_execute(self._handle, ctypes.c_void_p(A), ctypes.c_void_p(B), ctypes.c_void_p(C),
                                     ctypes.c_void_p(Y), ctypes.c_void_p(stream)))

    def execute(self, A, B, Y, C=None, stream=None) -> None:
        import torch

        want = torch_dtype(self.dtype)
        checks = [("A", A, self.a_shape), ("B", B, self.b_shape), ("Y", Y, self.output_shape)]
        if self.c_shape is not None:
            if C is None:
                raise ValueError("this Gemm plan has a C")
            checks.append(("C", C, self.c_shape))
        for name, t, shape in checks:
            if t.dtype != want or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {want} tensor of shape {tuple(shape)}")
        if stream is None:
            stream = torch.cuda.current_stream(Y.device)
        with self._lock:
            self.execute_ptr(A.data_ptr(), B.data_ptr(), Y.data_ptr(), stream.cuda_stream,
                             C.data_ptr() if C is not None else 0)


def torch_int_code(dt) -> int:
    import torch

    codes = {torch.uint8: UINT8, torch.int8: INT8}
    if dt not in codes:
        raise TypeError(f"MatMulInteger takes uint8 / int8 tensors, not {dt}")
    return codes[dt]


class IntPlan(Plan):
    """mm_int_plan_create / mm_int_execute: ONNX MatMulInteger (UINT8 / INT8
    operands, optional scalar or per-row / per-column zero points, INT32
    output modulo 2^32)."""

    def __init__(self, a_shape, b_shape, a_type: int, b_type: int, a_zp: int = ZP_NONE, b_zp: int = ZP_NONE,
                 force_algo: int = 0, tile: int = 0, split_k: int = 0):
        L = lib()
        self._handle = ctypes.c_void_p()
        self.a_shape = tuple(int(d) for d in a_shape)
        self.b_shape = tuple(int(d) for d in b_shape)
        self.a_type, self.b_type = int(a_type), int(b_type)
        self.a_zp, self.b_zp = int(a_zp), int(b_zp)
        self.dtype = INT32
        opt = PlanOptions(force_algo, tile, split_k, 0)
        _check(L.mm_int_plan_create(_shape(self.a_shape), len(self.a_shape), _shape(self.b_shape), len(self.b_shape),
                                    self.a_type, self.b_type, self.a_zp, self.b_zp, ctypes.byref(opt),
                                    ctypes.byref(self._handle)))
        self._lock = threading.Lock()

    def zero_point_numel(self, which: str) -> int:
        """Elements the plan reads from the A or B zero point (0 for none)."""
        kind = self.a_zp if which == "a" else self.b_zp
        if kind == ZP_NONE:
            return 0
        if kind == ZP_SCALAR:
            return 1
        inf = self.info()
        return inf["M"] if which == "a" else inf["N"]

    def execute_ptr(self, A: int, B: int, Y: int, stream: int = 0, a_zp: int = 0, b_zp: int = 0) -> None:
        _check(lib().mm_int_execute(self._handle, ctypes.c_void_p(A), ctypes.c_void_p(B), ctypes.c_void_p(a_zp),
                                    ctypes.c_void_p(b_zp), ctypes.c_void_p(Y), ctypes.c_void_p(stream)))

    def execute(self, A, B, Y, a_zp=None, b_zp=None, stream=None) -> None:
        import torch

        tdt = {UINT8: torch.uint8, INT8: torch.int8}
        checks = [("A", A, self.a_shape, tdt[self.a_type]), ("B", B, self.b_shape, tdt[self.b_type]),
                  ("Y", Y, self.output_shape, torch.int32)]
        for which, zp, typ in (("a", a_zp, self.a_type), ("b", b_zp, self.b_type)):
            n = self.zero_point_numel(which)
            if (zp is None) != (n == 0):
                raise ValueError(f"{which}_zp: the plan expects {'none' if n == 0 else f'{n} value(s)'}")
            if zp is not None:
                if zp.numel() != n:
                    raise ValueError(f"{which}_zp has {zp.numel()} elements, the plan reads {n}")
                checks.append((f"{which}_zp", zp, tuple(zp.shape), tdt[typ]))
        for name, t, shape, want in checks:
            if t.dtype != want or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {want} tensor of shape {tuple(shape)}")
        if stream is None:
            stream = torch.cuda.current_stream(Y.device)
        with self._lock:
            self.execute_ptr(A.data_ptr(), B.data_ptr(), Y.data_ptr(), stream.cuda_stream,
                             a_zp.data_ptr() if a_zp is not None else 0, b_zp.data_ptr() if b_zp is not None else 0)


def _wrong(name, t, dt, shape, dev) -> None:
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the output on GPU {dev}")
    raise ValueError(f"{name} must be a contiguous {dt} tensor of shape {tuple(shape)}")


def _dense(name, t, dt, shape, dev) -> int:
    """t's address, if it is dense, of that type and shape, on GPU `dev`."""
    if t.dtype is not dt or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _wrong(name, t, dt, shape, dev)
    return t.data_ptr()


def _device_of(t) -> int:
    """The index of the GPU that holds the output t."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("the tensors must be device tensors")
    return dev


def _run(dev, stream, fn, *args) -> None:
    """fn(*args, raw stream) with GPU `dev` current; stream defaults to its current stream."""
    import torch

    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return _run(dev, stream, fn, *args)
    if stream is not None:
        raw = stream.cuda_stream
    else:
        # The handle alone where torch offers it: building the Stream object
        # takes 1 us of the call's 6.
        get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        raw = get(dev) if get else torch.cuda.current_stream(dev).cuda_stream
    st = fn(*args, raw)
    if st:
        _check(st)


def _empty(shape, dt, device, stream):
    """A result that is made on `stream` (None: the current one)."""
    import torch

    if stream is None:
        return torch.empty(shape, dtype=dt, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dt, device=device)


def quantize_rows(X, q=None, scale=None, stream=None):
    """mm_quantize_rows: (q, scale) of X's rows (its last dimension), q INT8 of
    X's shape, scale FP32 of X's shape without the last dimension.  Those that
    are not given are made on ``stream`` (default: the current stream), as if
    it were current: memory that another stream's queued work still uses does
    not come into them."""
    import torch

    code = torch_dtype_code(X.dtype)
    if X.dim() < 1:
        raise ValueError("X needs at least one dimension")
    dev = _device_of(X)
    if q is None:
        q = _empty(X.shape, torch.int8, X.device, stream)
    if scale is None:
        scale = _empty(X.shape[:-1], torch.float32, X.device, stream)
    xp = _dense("X", X, X.dtype, X.shape, dev)
    qp = _dense("q", q, torch.int8, X.shape, dev)
    sp = _dense("scale", scale, torch.float32, X.shape[:-1], dev)
    cols = X.shape[-1]
    rows = 1
    for d in X.shape[:-1]:
        rows *= d
    _run(dev, stream, lib().mm_quantize_rows, xp, code, rows, cols, qp, sp)
    return q, scale


class ScaledIntPlan(Plan):
    """mm_scaled_int_plan_create / mm_scaled_int_execute: INT8 product with a
    scale for each row of A and each column of B.  a_type is INT8, or the
    float type of an A that every execution quantizes by rows first."""

    def __init__(self, a_shape, b_shape, out_type: int, a_type: int = INT8, trans_b: bool = False, bias: bool = False,
                 force_algo: int = 0, tile: int = 0, split_k: int = 0):
        import torch

        L = lib()
        self._handle = ctypes.c_void_p()
        self.a_shape = torch.Size(int(d) for d in a_shape)
        self.b_shape = torch.Size(int(d) for d in b_shape)
        self.a_type, self.dtype = int(a_type), int(out_type)
        self.trans_b, self.bias = bool(trans_b), bool(bias)
        desc = ScaledIntDesc(self.a_type, self.dtype, int(self.trans_b), int(self.bias), 0)
        opt = PlanOptions(force_algo, tile, split_k, 0)
        _check(L.mm_scaled_int_plan_create(_shape(self.a_shape), len(self.a_shape), _shape(self.b_shape),
                                           len(self.b_shape), ctypes.byref(desc), ctypes.byref(opt),
                                           ctypes.byref(self._handle)))
        self._lock = threading.Lock()
        self._execute = L.mm_scaled_int_execute
        self._i8, self._f32 = torch.int8, torch.float32
        self._a_dt, self._out_dt = torch_dtype(self.a_type), torch_dtype(self.dtype)
        self._y_shape = torch.Size(self.output_shape)
        n = 1 if len(self.b_shape) == 1 else self.b_shape[-2 if self.trans_b else -1]
        self._bias_shape = torch.Size((n,))
        self.a_scale_shape = self.a_shape[:-1]
        self.b_scale_shape = torch.Size(()) if len(self.b_shape) == 1 else self.b_shape[:-2] + self._bias_shape

    def execute_ptr(self, A: int, B: int, Y: int, stream: int = 0, a_scale: int = 0, b_scale: int = 0,
                    bias: int = 0) -> None:
        _check(lib().mm_scaled_int_execute(self._handle, A, B, a_scale, b_scale, bias, Y, stream))

    def execute(self, A, B, Y, a_scale=None, b_scale=None, bias=None, stream=None) -> None:
        """a_scale: FP32, A's shape without K (None where the plan quantizes
        A); b_scale: FP32, B's batch dimensions and N; bias: N values of Y's type."""
        if (a_scale is None) != (self.a_type != INT8):
            raise ValueError("a_scale: " + ("the plan quantizes A itself" if a_scale is not None
                                            else "an INT8 A needs its scales"))
        if b_scale is None:
            raise ValueError("b_scale is missing")
        if (bias is None) == self.bias:
            raise ValueError("bias: the plan has " + ("one" if self.bias else "none"))
        dev = _device_of(Y)
        ap = _dense("A", A, self._a_dt, self.a_shape, dev)
        bp = _dense("B", B, self._i8, self.b_shape, dev)
        yp = _dense("Y", Y, self._out_dt, self._y_shape, dev)
        bsp = _dense("b_scale", b_scale, self._f32, self.b_scale_shape, dev)
        asp = None if a_scale is None else _dense("a_scale", a_scale, self._f32, self.a_scale_shape, dev)
        biasp = None if bias is None else _dense("bias", bias, self._out_dt, self._bias_shape, dev)
        with self._lock:
            _run(dev, stream, self._execute, self._handle, ap, bp, asp, bsp, biasp, yp)


class GluPlan(Plan):
    """mm_glu_plan_create_ex / mm_glu_execute / mm_glu_backward: the gated
    feed-forward block H = f(X Wg) * (X Wu) and its gradients.  The weights are
    [in_features, hidden], or [hidden, in_features] with trans_w; they may be
    views of a merged matrix (rows w_pitch elements apart).  kept_type is the
    type of G and U (0: the plan's; FLOAT keeps their FP32 sums).  tile and
    split_k override the forward pass's choices, dx_* and dw_* the backward
    pass's."""

    def __init__(self, rows: int, in_features: int, hidden: int, dtype: int, activation: int = ACT_SILU,
                 trans_w: bool = False, training: bool = False, w_pitch: int = 0, force_algo: int = 0, tile: int = 0,
                 split_k: int = 0, kept_type: int = 0, dx_tile: int = 0, dx_split_k: int = 0, dw_tile: int = 0,
                 dw_split_k: int = 0):
        import torch

        L = lib()
        self._handle = ctypes.c_void_p()
        self.dtype = int(dtype)
        self.rows, self.in_features, self.hidden = int(rows), int(in_features), int(hidden)
        self.trans_w, self.training = bool(trans_w), bool(training)
        desc = GluDesc(self.rows, self.in_features, self.hidden, int(w_pitch), int(self.trans_w), int(activation),
                       int(self.training), 0)
        opt = PlanOptions(force_algo, tile, split_k, 0)
        glu = GluOptions(int(kept_type), dx_tile, dx_split_k, dw_tile, dw_split_k)
        _check(L.mm_glu_plan_create_ex(ctypes.byref(desc), self.dtype, ctypes.byref(opt), ctypes.byref(glu),
                                       ctypes.byref(self._handle)))
        self._lock = threading.Lock()
        self._dt = torch_dtype(self.dtype)
        self._kept = torch_dtype(int(kept_type) or self.dtype)
        self._x = torch.Size((self.rows, self.in_features))
        self._h = torch.Size((self.rows, self.hidden))
        self._w = torch.Size((self.hidden, self.in_features) if self.trans_w else (self.in_features, self.hidden))
        self._pitch = int(w_pitch) or self._w[1]
        self._execute, self._backward = L.mm_glu_execute, L.mm_glu_backward

    def options(self) -> dict:
        """mm_glu_get_options: the type of G and U, and the tile entry and K
        partitions of a training plan's dX and of dWg, dWu."""
        t = GluOptions()
        _check(lib().mm_glu_get_options(self._handle, ctypes.byref(t)))
        return {name: getattr(t, name) for name, _ in t._fields_}

    def _weight(self, name, t, dev) -> int:
        """t's address, if it is a weight of this plan on GPU `dev`."""
        ok = t.dtype is self._dt and t.shape == self._w and t.get_device() == dev
        if ok and not (t.is_contiguous() and self._pitch == self._w[1]) and t.numel():
            ok = (t.stride(1) == 1 or t.shape[1] == 1) and (t.stride(0) == self._pitch or t.shape[0] == 1)
        if not ok:
            raise ValueError(f"{name} must be a {self._dt} tensor of shape {tuple(self._w)} with rows {self._pitch} "
                             f"elements apart on the output's GPU")
        return t.data_ptr()

    def execute_ptr(self, X: int, Wg: int, Wu: int, H: int, G: int = 0, U: int = 0, stream: int = 0) -> None:
        _check(lib().mm_glu_execute(self._handle, X, Wg, Wu, H, G, U, stream))

    def execute(self, X, Wg, Wu, H, G=None, U=None, stream=None) -> None:
        """The forward pass; G and U (both or neither) keep X Wg and X Wu."""
        if (G is None) != (U is None):
            raise ValueError("G and U are given together or not at all")
        dt, h = self._dt, self._h
        dev = _device_of(H)
        xp = _dense("X", X, dt, self._x, dev)
        gp, up = self._weight("Wg", Wg, dev), self._weight("Wu", Wu, dev)
        hp = _dense("H", H, dt, h, dev)
        kg = None if G is None else _dense("G", G, self._kept, h, dev)
        ku = None if U is None else _dense("U", U, self._kept, h, dev)
        with self._lock:
            _run(dev, stream, self._execute, self._handle, xp, gp, up, hp, kg, ku)

    def backward(self, X, Wg, Wu, G, U, dH, dX=None, dWg=None, dWu=None, stream=None) -> None:
        """The backward pass into dX and / or dWg and dWu (overwritten)."""
        if (dWg is None) != (dWu is None):
            raise ValueError("dWg and dWu are given together or not at all")
        dt, h = self._dt, self._h
        dev = _device_of(dH)
        ptrs = (_dense("X", X, dt, self._x, dev), self._weight("Wg", Wg, dev), self._weight("Wu", Wu, dev),
                _dense("G", G, self._kept, h, dev), _dense("U", U, self._kept, h, dev), _dense("dH", dH, dt, h, dev),
                None if dX is None else _dense("dX", dX, dt, self._x, dev),
                None if dWg is None else self._weight("dWg", dWg, dev),
                None if dWu is None else self._weight("dWu", dWu, dev))
        with self._lock:
            _run(dev, stream, self._backward, self._handle, *ptrs)


CHECKPOINT_BLOCK = 32


def checkpoint_blocks(cols: int) -> int:
    """Scale bytes of a checkpoint row of ``cols`` elements."""
    return -(-int(cols) // CHECKPOINT_BLOCK)


def _checkpoint(name, q, scale, shape, dev):
    """The addresses of a checkpoint of a tensor of `shape` on GPU `dev`."""
    import torch

    *lead, cols = shape
    return (_dense(name, q, torch.int8, shape, dev),
            _dense(f"{name}'s scale", scale, torch.uint8, (*lead, -(-cols // CHECKPOINT_BLOCK)), dev))


def _rows_cols(shape) -> Tuple[int, int]:
    if not shape:
        raise ValueError("a tensor of at least one dimension is needed")
    *lead, cols = shape
    return math.prod(lead), cols


def checkpoint_pack(X, q=None, scale=None, stream=None):
    """mm_checkpoint_pack: (q, scale), the 8-bit checkpoint of X's rows (its
    last dimension): q INT8 of X's shape, scale UINT8 with a byte for each block
    of CHECKPOINT_BLOCK elements.  Those that are not given are made on ``stream``
    (default: the current stream), as if it were current."""
    import torch

    dt, shape = X.dtype, X.shape
    code = torch_dtype_code(dt)
    rows, cols = _rows_cols(shape)
    dev = _device_of(X)
    if q is None:
        q = _empty(shape, torch.int8, X.device, stream)
    if scale is None:
        scale = _empty(shape[:-1] + (checkpoint_blocks(cols),), torch.uint8, X.device, stream)
    xp = _dense("X", X, dt, shape, dev)
    qp, sp = _checkpoint("q", q, scale, shape, dev)
    _run(dev, stream, (_lib or lib()).mm_checkpoint_pack, xp, code, rows, cols, qp, sp)
    return q, scale


def checkpoint_unpack(q, scale, out, stream=None):
    """mm_checkpoint_unpack: the checkpoint's values into ``out`` (q's shape), or
    into a new tensor of ``out`` if that is a torch dtype."""
    import torch

    shape = q.shape
    rows, cols = _rows_cols(shape)
    dev = _device_of(q)
    if isinstance(out, torch.dtype):
        torch_dtype_code(out)
        out = _empty(shape, out, q.device, stream)
    dt = out.dtype
    code = torch_dtype_code(dt)
    qp, sp = _checkpoint("q", q, scale, shape, dev)
    op = _dense("out", out, dt, shape, dev)
    _run(dev, stream, (_lib or lib()).mm_checkpoint_unpack, qp, sp, rows, cols, code, op)
    return out


class LinearPlan(Plan):
    """mm_linear_plan_create / mm_linear_execute / mm_linear_backward: the linear
    layer Y = f(X W + bias) + residual and its gradients.  The weights are
    [in_features, out_features], or [out_features, in_features] with trans_w;
    they may be a view of a wider matrix (rows w_pitch elements apart).  A
    training plan with an activation keeps Z = X W + bias in z_type (0: the
    plan's type; FLOAT; INT8: a checkpoint) and takes X for the backward pass as
    x_type says (INT8: a checkpoint, to whose values x_activation is applied).
    tile and split_k override the forward pass's choices, dx_* and dw_* the
    backward pass's."""

    def __init__(self, rows: int, in_features: int, out_features: int, dtype: int, activation: int = ACT_NONE,
                 trans_w: bool = False, bias: bool = False, residual: bool = False, training: bool = False,
                 z_type: int = 0, x_type: int = 0, x_activation: int = ACT_NONE, w_pitch: int = 0, force_algo: int = 0,
                 tile: int = 0, split_k: int = 0, dx_tile: int = 0, dx_split_k: int = 0, dw_tile: int = 0,
                 dw_split_k: int = 0):
        import torch

        L = lib()
        self._handle = ctypes.c_void_p()
        self.dtype = int(dtype)
        self.rows, self.in_features, self.out_features = int(rows), int(in_features), int(out_features)
        self.trans_w, self.bias, self.residual = bool(trans_w), bool(bias), bool(residual)
        self.training, self.activation = bool(training), int(activation)
        desc = LinearDesc(self.rows, self.in_features, self.out_features, int(w_pitch), int(self.trans_w),
                          self.activation, int(self.bias), int(self.residual), int(self.training), int(z_type),
                          int(x_type), int(x_activation), dx_tile, dx_split_k, dw_tile, dw_split_k, 0)
        opt = PlanOptions(force_algo, tile, split_k, 0)
        _check(L.mm_linear_plan_create(ctypes.byref(desc), self.dtype, ctypes.byref(opt), ctypes.byref(self._handle)))
        self._lock = threading.Lock()
        self._dt = torch_dtype(self.dtype)
        kept = self.training and self.activation != ACT_NONE
        self._z_dt = torch_dtype(int(z_type) or self.dtype) if kept else None
        self._z8, self._x8 = kept and int(z_type) == INT8, int(x_type) == INT8
        self._x = torch.Size((self.rows, self.in_features))
        self._y = torch.Size((self.rows, self.out_features))
        self._b = torch.Size((self.out_features,))
        self._w = torch.Size((self.out_features, self.in_features) if self.trans_w else
                             (self.in_features, self.out_features))
        self._pitch = int(w_pitch) or self._w[1]
        self._execute, self._backward = L.mm_linear_execute, L.mm_linear_backward

    def desc(self) -> dict:
        """mm_linear_get_desc: what the plan resolved, the backward products'
        tile entries and K partitions among it."""
        d = LinearDesc()
        _check(lib().mm_linear_get_desc(self._handle, ctypes.byref(d)))
        return {name: getattr(d, name) for name, _ in d._fields_ if name != "reserved"}

    def tails(self) -> dict:
        """mm_linear_get_tails: the columns from which a training plan's dX and
        dW run as second launches, and their tile entries (0: they do not)."""
        t = LinearTails()
        _check(lib().mm_linear_get_tails(self._handle, ctypes.byref(t)))
        return {name: getattr(t, name) for name, _ in t._fields_}

    _weight = GluPlan._weight

    def _kept(self, Z, z_scale, dev):
        """The addresses of Z and of its scale."""
        if Z is None:
            if z_scale is not None:
                raise ValueError("z_scale is given without Z")
            return None, None
        if self._z_dt is None:
            raise ValueError("the plan keeps no Z")
        if self._z8:
            if z_scale is None:
                raise ValueError("Z is a checkpoint: z_scale is missing")
            return _checkpoint("Z", Z, z_scale, self._y, dev)
        if z_scale is not None:
            raise ValueError("z_scale: the plan keeps Z whole")
        return _dense("Z", Z, self._z_dt, self._y, dev), None

    def execute_ptr(self, X: int, W: int, Y: int, stream: int = 0, bias: int = 0, residual: int = 0, Z: int = 0,
                    z_scale: int = 0) -> None:
        _check(lib().mm_linear_execute(self._handle, X, W, bias, residual, Y, Z, z_scale, stream))

    def execute(self, X, W, Y, bias=None, residual=None, Z=None, z_scale=None, stream=None) -> None:
        """The forward pass; Z (and z_scale, for a checkpoint) keeps what the
        backward pass needs.  Y may be the residual itself."""
        if (bias is None) == self.bias:
            raise ValueError("bias: the plan has " + ("one" if self.bias else "none"))
        if (residual is None) == self.residual:
            raise ValueError("residual: the plan has " + ("one" if self.residual else "none"))
        dt = self._dt
        dev = _device_of(Y)
        xp = _dense("X", X, dt, self._x, dev)
        wp = self._weight("W", W, dev)
        yp = _dense("Y", Y, dt, self._y, dev)
        bp = None if bias is None else _dense("bias", bias, dt, self._b, dev)
        rp = None if residual is None else _dense("residual", residual, dt, self._y, dev)
        zp, sp = self._kept(Z, z_scale, dev)
        with self._lock:
            _run(dev, stream, self._execute, self._handle, xp, wp, bp, rp, yp, zp, sp)

    def backward(self, X, W, dY, Z=None, z_scale=None, x_scale=None, dX=None, dW=None, dbias=None, stream=None) -> None:
        """The backward pass into those of dX, dW and dbias that are given
        (overwritten).  X may be None without dW, W without dX."""
        dt = self._dt
        dev = _device_of(dY)
        if X is not None and self._x8:
            if x_scale is None:
                raise ValueError("X is a checkpoint: x_scale is missing")
            xp, xsp = _checkpoint("X", X, x_scale, self._x, dev)
        else:
            if x_scale is not None:
                raise ValueError("x_scale: " + ("X is missing" if self._x8 else "the plan takes X whole"))
            xp, xsp = None if X is None else _dense("X", X, dt, self._x, dev), None
        zp, zsp = self._kept(Z, z_scale, dev)
        if dbias is not None and not self.bias:
            raise ValueError("dbias: the plan has no bias")
        ptrs = (xp, xsp, None if W is None else self._weight("W", W, dev), zp, zsp, _dense("dY", dY, dt, self._y, dev),
                None if dX is None else _dense("dX", dX, dt, self._x, dev),
                None if dW is None else self._weight("dW", dW, dev),
                None if dbias is None else _dense("dbias", dbias, dt, self._b, dev))
        with self._lock:
            _run(dev, stream, self._backward, self._handle, *ptrs)


class NormPlan(Plan):
    """mm_norm_plan_create / mm_norm_execute / mm_norm_backward: the norms on
    both sides of a block's end, fused with its gate and residual scale,

        sum = X + residual_scale * gate * n1,  n1 = post(block) * post_weight + post_bias (post NORM_NONE: block)
        out = pre(sum) * pre_weight + pre_bias                                             (pre NORM_NONE: none)

    and their gradients.  block=False: sum is X, out its norm.  gate_rows: row m
    takes gate row m // gate_rows (0: no gate).  kept_type: the backward pass is
    given sum and block (0), sum in FP32 as the forward pass kept it in sum_f32
    (FLOAT), or checkpoints of both (INT8)."""

    def __init__(self, rows: int, cols: int, dtype: int, pre: int = NORM_RMS, post: int = NORM_NONE, block: bool = True,
                 pre_weight: bool = True, pre_bias: bool = False, post_weight: bool = False, post_bias: bool = False,
                 gate_rows: int = 0, residual_scale: float = 1.0, pre_eps: float = 1e-6, post_eps: float = 1e-6,
                 training: bool = False, kept_type: int = 0):
        import torch

        L = lib()
        self._handle = ctypes.c_void_p()
        self.dtype, self.rows, self.cols = int(dtype), int(rows), int(cols)
        self.training, self.pre, self.post, self.block = bool(training), int(pre), int(post), bool(block)
        desc = NormDesc(self.rows, self.cols, int(gate_rows), self.post, self.pre, post_eps, pre_eps, residual_scale,
                        int(self.block), int(post_weight), int(post_bias), int(pre_weight), int(pre_bias),
                        int(self.training), int(kept_type), 0)
        _check(L.mm_norm_plan_create(ctypes.byref(desc), self.dtype, ctypes.byref(self._handle)))
        self._lock = threading.Lock()
        self._dt, self._f32 = torch_dtype(self.dtype), torch.float32
        self._kept8 = int(kept_type) == INT8
        self._sum_dt = self._f32 if int(kept_type) == FLOAT else self._dt
        self._x = torch.Size((self.rows, self.cols))
        self._w = torch.Size((self.cols,))
        self._g = torch.Size((-(-self.rows // gate_rows), self.cols)) if gate_rows else None
        self._stats = torch.Size((self.rows, 4))
        self._execute, self._backward = L.mm_norm_execute, L.mm_norm_backward

    def _one(self, name, t, dev, shape):
        return None if t is None else _dense(name, t, self._dt, shape, dev)

    def _gate(self, name, t, dev):
        if t is None:
            return None
        if self._g is None:
            raise ValueError(f"{name}: the plan has no gate")
        return _dense(name, t, self._dt, self._g, dev)

    def _pair(self, name, pair, dev):
        return (None, None) if pair is None else _checkpoint(name, pair[0], pair[1], self._x, dev)

    def execute(self, X, out=None, block=None, sum=None, gate=None, pre_weight=None, pre_bias=None, post_weight=None,
                post_bias=None, stats=None, sum_f32=None, sum_checkpoint=None, block_checkpoint=None,
                out_checkpoint=None, stream=None) -> None:
        """The forward pass into sum (None: not written) and out.  A training
        plan's stats (FP32 [rows, 4]) and sum_f32 or checkpoints, pairs (q,
        scale), keep what the backward pass needs.  sum may be X itself, out the block."""
        dev = _device_of(X)
        x, w = self._x, self._w
        args = NormForwardArgs(
            _dense("X", X, self._dt, x, dev), self._one("block", block, dev, x), self._gate("gate", gate, dev),
            self._one("post_weight", post_weight, dev, w), self._one("post_bias", post_bias, dev, w),
            self._one("pre_weight", pre_weight, dev, w), self._one("pre_bias", pre_bias, dev, w),
            self._one("sum", sum, dev, x), self._one("out", out, dev, x),
            None if stats is None else _dense("stats", stats, self._f32, self._stats, dev),
            None if sum_f32 is None else _dense("sum_f32", sum_f32, self._f32, x, dev))
        if sum_checkpoint is not None:
            args.sum_q, args.sum_scale = _checkpoint("sum_checkpoint", *sum_checkpoint, x, dev)
        if block_checkpoint is not None:
            args.block_q, args.block_scale = _checkpoint("block_checkpoint", *block_checkpoint, x, dev)
        if out_checkpoint is not None:
            args.out_q, args.out_scale = _checkpoint("out_checkpoint", *out_checkpoint, x, dev)
        with self._lock:
            _run(dev, stream, self._execute, self._handle, args)

    def backward(self, stats, sum=None, block=None, dout=None, dsum=None, gate=None, pre_weight=None, post_weight=None,
                 post_bias=None, dX=None, dblock=None, dgate=None, dpre_weight=None, dpre_bias=None, dpost_weight=None,
                 dpost_bias=None, stream=None) -> None:
        """The backward pass into those results that are given (overwritten).
        sum and block are tensors, or pairs (q, scale) with kept_type INT8.  dX may
        be dsum itself, dblock dout."""
        dev = _device_of(stats)
        x, w = self._x, self._w

        def kept(name, t, dt):
            if self._kept8:
                return self._pair(name, t, dev)
            return None if t is None else _dense(name, t, dt, x, dev), None

        args = NormBackwardArgs(
            _dense("stats", stats, self._f32, self._stats, dev), *kept("sum", sum, self._sum_dt),
            *kept("block", block, self._dt),
            self._gate("gate", gate, dev), self._one("post_weight", post_weight, dev, w),
            self._one("post_bias", post_bias, dev, w), self._one("pre_weight", pre_weight, dev, w),
            self._one("dout", dout, dev, x), self._one("dsum", dsum, dev, x), self._one("dX", dX, dev, x),
            self._one("dblock", dblock, dev, x), self._gate("dgate", dgate, dev),
            self._one("dpost_weight", dpost_weight, dev, w), self._one("dpost_bias", dpost_bias, dev, w),
            self._one("dpre_weight", dpre_weight, dev, w), self._one("dpre_bias", dpre_bias, dev, w))
        with self._lock:
            _run(dev, stream, self._backward, self._handle, args)


_plan_cache = {}
_plan_cache_lock = threading.Lock()


def matmul(A, B, out=None, stream=None):
    """Y = MatMul(A, B) (ONNX semantics) on ``stream`` (default: the current
    stream of A's device).  Plans are cached per (shapes, dtype, stream), so a
    plan's split-K workspace is never shared by two streams."""
    import torch

    code = torch_dtype_code(A.dtype)
    if B.dtype != A.dtype:
        raise TypeError(f"mixed input types {A.dtype} and {B.dtype}")
    if stream is None:
        stream = torch.cuda.current_stream(A.device)
    key = (tuple(A.shape), tuple(B.shape), code, A.device.index, stream.cuda_stream)
    with _plan_cache_lock:
        plan = _plan_cache.get(key)
        if plan is None:
            plan = Plan(A.shape, B.shape, code)
            _plan_cache[key] = plan
    if out is None:
        out = torch.empty(plan.output_shape, dtype=A.dtype, device=A.device)
    plan.execute(A, B, out, stream)
    return out
