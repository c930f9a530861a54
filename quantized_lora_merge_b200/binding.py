"""Thin ctypes binding of libintlora.so (the C ABI in include/intlora.h).

Argument marshalling only: torch tensors are passed as device pointers and
every step of the computation runs in the library's CUDA kernels. Function
names match the C entry points. Importing works without a GPU; the first call
loads the library and raises ``IntLoRAError``/``OSError`` if it is missing or a
call fails (there is no fallback of any kind).
"""
from __future__ import annotations

import ctypes
import re
from dataclasses import dataclass
from pathlib import Path
from typing import Optional, Sequence

PKG = Path(__file__).resolve().parent
LIB_PATH = PKG / "libintlora.so"
HEADER = PKG.parent / "include" / "intlora.h"

_c_i64, _c_i32, _c_u64, _c_u32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64, ctypes.c_uint32
_c_f32, _c_ptr, _c_size = ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t

DIST_LAPLACE, DIST_GAUSSIAN, DIST_CAUCHY, DIST_STUDENT_T2 = 0, 1, 2, 3   # INTLORA_DIST_*

TYPE_F32, TYPE_BF16, TYPE_F16 = 0, 1, 2             # INTLORA_TYPE_*

STATUS = {0: "INTLORA_OK", 1: "INTLORA_ERR_INVALID_ARG", 2: "INTLORA_ERR_UNSUPPORTED",
          3: "INTLORA_ERR_WORKSPACE", 4: "INTLORA_ERR_CUDA", 5: "INTLORA_ERR_TIMEOUT"}


class IntLoRAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class intlora_aux_job(ctypes.Structure):
    _fields_ = [("W", _c_ptr), ("d", _c_i64), ("n", _c_i64), ("seed", _c_u64),
                ("stream_id", _c_u32), ("alpha", _c_f32), ("w_bits", _c_i32),
                ("sigma_w_out", _c_ptr), ("sigma_r_out", _c_ptr), ("r_star_out", _c_ptr),
                ("w_round_out", _c_ptr), ("ld_w_out", _c_i64), ("s_out", _c_ptr),
                ("z_out", _c_ptr), ("distribution", _c_i32)]


class intlora_layer(ctypes.Structure):
    _fields_ = [("d", _c_i64), ("n", _c_i64), ("r", _c_i32), ("w_bits", _c_i32),
                ("w_round", _c_ptr), ("ld_w", _c_i64), ("s", _c_ptr), ("z", _c_ptr),
                ("A", _c_ptr), ("B", _c_ptr), ("seed", _c_u64), ("stream_id", _c_u32),
                ("alpha", _c_f32), ("sigma_w", _c_ptr), ("sigma_r", _c_ptr),
                ("distribution", _c_i32)]


class intlora_merge_out(ctypes.Structure):
    _fields_ = [("out", _c_ptr), ("sbar", _c_ptr), ("zbar", _c_ptr), ("code", _c_ptr)]


class intlora_ste_job(ctypes.Structure):
    _fields_ = [("G", _c_ptr), ("A", _c_ptr), ("B", _c_ptr), ("d", _c_i64), ("n", _c_i64),
                ("r", _c_i32), ("dA", _c_ptr), ("dB", _c_ptr), ("mask_codes", _c_ptr),
                ("mask_ld", _c_i64), ("mask_bits", _c_i32), ("mask_z", _c_ptr)]


class intlora_fakequant_job(ctypes.Structure):
    _fields_ = [("q", _c_ptr), ("q_bytes", _c_i32), ("sbar", _c_ptr), ("d", _c_i64), ("n", _c_i64),
                ("w_out", _c_ptr)]


class intlora_linear_job(ctypes.Structure):
    _fields_ = [("X", _c_ptr), ("W", _c_ptr), ("tokens", _c_i64), ("d", _c_i64), ("n", _c_i64),
                ("Y", _c_ptr), ("y_bf16", _c_i32)]


class intlora_train_backward_job(ctypes.Structure):
    _fields_ = [("X", _c_ptr), ("dY", _c_ptr), ("W", _c_ptr), ("A", _c_ptr), ("B", _c_ptr),
                ("tokens", _c_i64), ("d", _c_i64), ("n", _c_i64), ("r", _c_i32),
                ("dX", _c_ptr), ("dA", _c_ptr), ("dB", _c_ptr)]


class intlora_int_gemm_job(ctypes.Structure):
    _fields_ = [("X", _c_ptr), ("x_scale", _c_ptr), ("W", _c_ptr), ("w_scale", _c_ptr),
                ("tokens", _c_i64), ("d", _c_i64), ("n", _c_i64), ("Y", _c_ptr),
                ("y_bf16", _c_i32)]


class intlora_layer_norm_job(ctypes.Structure):
    _fields_ = [("x", _c_ptr), ("weight", _c_ptr), ("bias", _c_ptr), ("y", _c_ptr),
                ("mean", _c_ptr), ("rstd", _c_ptr), ("tokens", _c_i64), ("n", _c_i64),
                ("ld_x", _c_i64), ("ld_y", _c_i64), ("x_type", _c_i32), ("param_type", _c_i32),
                ("y_type", _c_i32), ("eps", _c_f32)]


class intlora_layer_norm_backward_job(ctypes.Structure):
    _fields_ = [("dy", _c_ptr), ("x", _c_ptr), ("weight", _c_ptr), ("mean", _c_ptr),
                ("rstd", _c_ptr), ("dx", _c_ptr), ("dweight", _c_ptr), ("dbias", _c_ptr),
                ("tokens", _c_i64), ("n", _c_i64), ("ld_dy", _c_i64), ("ld_x", _c_i64),
                ("ld_dx", _c_i64), ("dy_type", _c_i32), ("x_type", _c_i32),
                ("param_type", _c_i32), ("dx_type", _c_i32), ("accumulate", _c_i32)]


class intlora_embedding_job(ctypes.Structure):
    _fields_ = [("table", _c_ptr), ("ids", _c_ptr), ("y", _c_ptr), ("invalid", _c_ptr),
                ("vocab", _c_i64), ("n", _c_i64), ("tokens", _c_i64), ("ld_table", _c_i64),
                ("ld_y", _c_i64), ("table_type", _c_i32), ("y_type", _c_i32),
                ("id_bytes", _c_i32), ("scale", _c_f32)]


class intlora_embedding_backward_job(ctypes.Structure):
    _fields_ = [("dy", _c_ptr), ("ids", _c_ptr), ("dtable", _c_ptr), ("invalid", _c_ptr),
                ("vocab", _c_i64), ("n", _c_i64), ("tokens", _c_i64), ("padding_id", _c_i64),
                ("ld_dy", _c_i64), ("ld_dtable", _c_i64), ("dy_type", _c_i32),
                ("dtable_type", _c_i32), ("id_bytes", _c_i32), ("accumulate", _c_i32),
                ("scale", _c_f32)]


class intlora_grad_job(ctypes.Structure):
    _fields_ = [("g", _c_ptr), ("count", _c_i64), ("type", _c_i32)]


_P = ctypes.POINTER
_SIGNATURES = {
    "intlora_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "intlora_last_error": (ctypes.c_char_p, []),
    "intlora_version": (ctypes.c_int, []),
    "intlora_device_timeouts": (_c_u32, []),
    "intlora_kernel_launches": (_c_u64, []),
    "intlora_device_status": (ctypes.c_int, []),
    "intlora_selftest_bounded_wait": (ctypes.c_int, [_c_u32, _c_ptr]),
    "intlora_merge_out_bytes": (_c_i32, [_c_i32, _c_i32, _c_i32]),
    "intlora_gen_aux_workspace_size": (_c_size, [_P(intlora_aux_job), _c_i32]),
    "intlora_gen_aux": (ctypes.c_int, [_c_ptr, _c_i64, _c_i64, _c_u64, _c_u32, _c_f32, _c_i32,
                                       _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_i64, _c_ptr, _c_ptr,
                                       _c_ptr, _c_size, _c_ptr]),
    "intlora_gen_aux_batched": (ctypes.c_int, [_P(intlora_aux_job), _c_i32, _c_ptr, _c_size,
                                               _c_ptr]),
    "intlora_gen_aux_noalloc": (ctypes.c_int, [_c_ptr, _c_i64, _c_i64, _c_u64, _c_u32, _c_f32,
                                               _c_i32, _c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_i64,
                                               _c_ptr, _c_ptr, _c_ptr]),
    "intlora_merge_workspace_size": (_c_size, [_P(intlora_layer), _c_i32]),
    "intlora_merge_mul": (ctypes.c_int, [_P(intlora_layer), _c_i32, _c_ptr, _c_ptr, _c_ptr,
                                         _c_ptr, _c_ptr, _c_size, _c_ptr]),
    "intlora_merge_shift": (ctypes.c_int, [_P(intlora_layer), _c_i32, _c_ptr, _c_ptr, _c_ptr,
                                           _c_ptr, _c_size, _c_ptr]),
    "intlora_merge_mul_batched": (ctypes.c_int, [_P(intlora_layer), _P(intlora_merge_out),
                                                 _c_i32, _c_i32, _c_ptr, _c_size, _c_ptr]),
    "intlora_merge_shift_batched": (ctypes.c_int, [_P(intlora_layer), _P(intlora_merge_out),
                                                   _c_i32, _c_i32, _c_ptr, _c_size, _c_ptr]),
    "intlora_ste_workspace_size": (_c_size, [_P(intlora_ste_job), _c_i32]),
    "intlora_ste_backward": (ctypes.c_int, [_c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_i32,
                                            _c_ptr, _c_ptr, _c_ptr, _c_size, _c_ptr]),
    "intlora_ste_backward_batched": (ctypes.c_int, [_P(intlora_ste_job), _c_i32, _c_ptr,
                                                    _c_size, _c_ptr]),
    "intlora_int_planes": (_c_i32, [_c_i64]),
    "intlora_fakequant_bf16": (ctypes.c_int, [_c_ptr, _c_i32, _c_ptr, _c_i64, _c_i64, _c_ptr,
                                              _c_ptr]),
    "intlora_linear_bf16_batched": (ctypes.c_int, [_P(intlora_linear_job), _c_i32, _c_ptr]),
    "intlora_train_backward_workspace_size": (_c_size, [_P(intlora_train_backward_job), _c_i32]),
    "intlora_train_backward_batched": (ctypes.c_int, [_P(intlora_train_backward_job), _c_i32,
                                                      _c_ptr, _c_size, _c_ptr]),
    "intlora_fakequant_bf16_batched": (ctypes.c_int, [_P(intlora_fakequant_job), _c_i32, _c_ptr]),
    "intlora_int_pack": (ctypes.c_int, [_c_ptr, _c_i32, _c_i64, _c_i64, _c_i32, _c_ptr, _c_ptr,
                                        _c_ptr]),
    "intlora_int_gemm_batched": (ctypes.c_int, [_P(intlora_int_gemm_job), _c_i32, _c_i32,
                                                _c_ptr]),
    "intlora_layer_norm_batched": (ctypes.c_int, [_P(intlora_layer_norm_job), _c_i32, _c_ptr]),
    "intlora_layer_norm_backward_workspace_size": (_c_size, [_P(intlora_layer_norm_backward_job),
                                                             _c_i32]),
    "intlora_layer_norm_backward_batched": (ctypes.c_int, [_P(intlora_layer_norm_backward_job),
                                                           _c_i32, _c_ptr, _c_size, _c_ptr]),
    "intlora_embedding_batched": (ctypes.c_int, [_P(intlora_embedding_job), _c_i32, _c_ptr]),
    "intlora_embedding_backward_workspace_size": (_c_size, [_P(intlora_embedding_backward_job),
                                                            _c_i32]),
    "intlora_embedding_backward_batched": (ctypes.c_int, [_P(intlora_embedding_backward_job),
                                                          _c_i32, _c_ptr, _c_size, _c_ptr]),
    "intlora_grad_norm_workspace_size": (_c_size, [_P(intlora_grad_job), _c_i32]),
    "intlora_grad_norm_batched": (ctypes.c_int, [_P(intlora_grad_job), _c_i32, _c_ptr, _c_ptr,
                                                 _c_size, _c_ptr]),
    "intlora_grad_clip_batched": (ctypes.c_int, [_P(intlora_grad_job), _c_i32, _c_f32, _c_ptr,
                                                 _c_ptr]),
    "intlora_clip_grad_norm_batched": (ctypes.c_int, [_P(intlora_grad_job), _c_i32, _c_f32, _c_ptr,
                                                      _c_ptr, _c_size, _c_ptr]),
    "intlora_int_gemm": (ctypes.c_int, [_c_ptr, _c_ptr, _c_ptr, _c_ptr, _c_i64, _c_i64, _c_i64,
                                        _c_i32, _c_ptr, _c_ptr]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load libintlora.so (fails loudly when it has not been built)."""
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise OSError(f"{LIB_PATH} is missing: build it with "
                          "`python -m quantized_lora_merge_b200.build`")
        L = ctypes.CDLL(str(LIB_PATH))
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of every function the public header declares."""
    text = HEADER.read_text()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(intlora_[a-z0-9_]+)\s*\(", text)))


def _check(status: int) -> None:
    if status != 0:
        raise IntLoRAError(status, lib().intlora_last_error().decode())


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        # the handle alone: building a Stream object takes longer than a launch
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return getattr(stream, "cuda_stream", stream)


def _ws(ws):
    if ws is None:
        return None, 0
    return ws.data_ptr(), ws.numel() * ws.element_size()


# ---------------------------------------------------------------------------
# descriptors (torch tensors + scalars)
# ---------------------------------------------------------------------------
@dataclass
class AuxJob:
    W: object
    seed: int
    stream_id: int
    alpha: float
    w_bits: int
    sigma_w: object                 # device float64 scalar (output)
    sigma_r: object                 # device float64 scalar (output)
    r_star: object = None
    w_round: object = None          # uint8 [d, ld]
    s: object = None
    z: object = None
    distribution: int = 0           # INTLORA_DIST_*

    def to_c(self) -> intlora_aux_job:
        d, n = self.W.shape
        ld = self.w_round.shape[1] if self.w_round is not None else 0
        return intlora_aux_job(_ptr(self.W), d, n, self.seed, self.stream_id, self.alpha,
                               self.w_bits, _ptr(self.sigma_w), _ptr(self.sigma_r),
                               _ptr(self.r_star), _ptr(self.w_round), ld, _ptr(self.s),
                               _ptr(self.z), self.distribution)


@dataclass
class Layer:
    w_round: object                 # uint8 [d, ld_w] codes
    n: int
    w_bits: int
    s: object
    z: object
    A: object                       # fp32 [d, r]
    B: object                       # fp32 [r, n]
    seed: int
    stream_id: int
    alpha: float
    sigma_w: object
    sigma_r: object = None
    distribution: int = 0           # INTLORA_DIST_*

    def to_c(self) -> intlora_layer:
        d = self.w_round.shape[0]
        return intlora_layer(d, self.n, self.A.shape[1], self.w_bits, _ptr(self.w_round),
                             self.w_round.shape[1], _ptr(self.s), _ptr(self.z), _ptr(self.A),
                             _ptr(self.B), self.seed, self.stream_id, self.alpha,
                             _ptr(self.sigma_w), _ptr(self.sigma_r), self.distribution)


@dataclass
class MergeOut:
    out: object
    sbar: object
    zbar: object = None
    code: object = None

    def to_c(self) -> intlora_merge_out:
        return intlora_merge_out(_ptr(self.out), _ptr(self.sbar), _ptr(self.zbar),
                                 _ptr(self.code))


@dataclass
class SteJob:
    G: object                       # bf16 [d, n]
    A: object                       # bf16 [d, r]
    B: object                       # bf16 [r, n]
    dA: object                      # fp32 [d, r]
    dB: object                      # fp32 [r, n]
    mask_codes: object = None       # masked STE: W_round uint8 [d, ld] (None: plain STE)
    mask_bits: int = 0
    mask_z: object = None           # int32 [d]

    def to_c(self) -> intlora_ste_job:
        d, n = self.G.shape
        ld = self.mask_codes.shape[1] if self.mask_codes is not None else 0
        return intlora_ste_job(_ptr(self.G), _ptr(self.A), _ptr(self.B), d, n, self.A.shape[1],
                               _ptr(self.dA), _ptr(self.dB), _ptr(self.mask_codes), ld,
                               self.mask_bits, _ptr(self.mask_z))


@dataclass
class IntGemmJob:
    X: object                       # int8 [tokens, n]
    x_scale: object                 # fp32 [tokens]
    W: object                       # int8 [d, planes, n] digit planes
    w_scale: object                 # fp32 [d]
    Y: object                       # fp32 or bf16 [tokens, d]

    def to_c(self) -> intlora_int_gemm_job:
        import torch
        tokens, n = self.X.shape
        return intlora_int_gemm_job(_ptr(self.X), _ptr(self.x_scale), _ptr(self.W),
                                    _ptr(self.w_scale), tokens, self.W.shape[0], n, _ptr(self.Y),
                                    int(self.Y.dtype == torch.bfloat16))


@dataclass
class FakeQuantJob:
    q: object                       # merged integer weights [d, n] (int8/int16/int32)
    sbar: object                    # fp32 [d]
    w_out: object                   # bf16 [d, n]

    def to_c(self) -> intlora_fakequant_job:
        d, n = self.q.shape
        return intlora_fakequant_job(_ptr(self.q), self.q.element_size(), _ptr(self.sbar), d, n,
                                     _ptr(self.w_out))


@dataclass
class LinearJob:
    X: object                       # bf16 [tokens, n]
    W: object                       # bf16 [d, n]
    Y: object                       # fp32 or bf16 [tokens, d]

    def to_c(self) -> intlora_linear_job:
        import torch
        tokens, n = self.X.shape
        return intlora_linear_job(_ptr(self.X), _ptr(self.W), tokens, self.W.shape[0], n,
                                  _ptr(self.Y), int(self.Y.dtype == torch.bfloat16))


@dataclass
class TrainBackwardJob:
    X: object                       # bf16 [tokens, n]
    dY: object                      # bf16 [tokens, d]
    W: object                       # bf16 [d, n] (fake-quantized merged weight)
    A: object                       # bf16 [d, r]
    B: object                       # bf16 [r, n]
    dX: object                      # fp32 [tokens, n]
    dA: object                      # fp32 [d, r]
    dB: object                      # fp32 [r, n]

    def to_c(self) -> intlora_train_backward_job:
        tokens, n = self.X.shape
        d, r = self.A.shape
        return intlora_train_backward_job(_ptr(self.X), _ptr(self.dY), _ptr(self.W), _ptr(self.A),
                                          _ptr(self.B), tokens, d, n, r, _ptr(self.dX),
                                          _ptr(self.dA), _ptr(self.dB))


# ---------------------------------------------------------------------------
# descriptors of the operators around the linears. Element types, shapes and
# strides travel to the library from the tensors, so they are checked here.
# ---------------------------------------------------------------------------
def _elem_type(name, t) -> int:
    import torch
    types = {torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16, torch.float16: TYPE_F16}
    if t.dtype not in types:
        raise TypeError(f"{name} must be fp32, bf16 or fp16, got {t.dtype}")
    return types[t.dtype]


def _matrix(name, t, rows=None, cols=None) -> int:
    """Row stride of a 2-D tensor whose rows are contiguous."""
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or \
            (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name} must be 2-D, {rows if rows is not None else 'any'} x "
                         f"{cols if cols is not None else 'any'}, got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _vector(name, t, count, dtype=None) -> None:
    if t is None:
        return
    if t.dim() != 1 or t.shape[0] != count or (count > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {count}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _one_device(*tensors):
    """The CUDA device that all tensors are on."""
    devices = {t.device for t in tensors if t is not None}
    if len(devices) != 1 or next(iter(devices)).type != "cuda":
        raise ValueError("tensors must be on one CUDA device, got "
                         f"{', '.join(sorted(str(d) for d in devices))}")
    return next(iter(devices))


def _counter(name, t) -> None:
    import torch
    if t is not None and (t.dtype != torch.int32 or t.numel() < 1):
        raise TypeError(f"{name} must be an int32 tensor")


def _ids(t) -> int:
    import torch
    if t.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, got {t.dtype}")
    return t.element_size()


@dataclass
class LayerNormJob:
    x: object                       # fp32, bf16 or fp16 [tokens, n]
    weight: object                  # [n] or None
    bias: object                    # [n], the weight's type, or None
    y: object                       # [tokens, n]
    mean: object = None             # fp32 [tokens]
    rstd: object = None             # fp32 [tokens]
    eps: float = 1e-5

    def to_c(self) -> intlora_layer_norm_job:
        import torch
        _one_device(self.x, self.weight, self.bias, self.y, self.mean, self.rstd)
        ld_x = _matrix("x", self.x)
        tokens, n = self.x.shape
        ld_y = _matrix("y", self.y, tokens, n)
        _vector("weight", self.weight, n)
        _vector("bias", self.bias, n, None if self.weight is None else self.weight.dtype)
        _vector("mean", self.mean, tokens, torch.float32)
        _vector("rstd", self.rstd, tokens, torch.float32)
        param = self.weight if self.weight is not None else self.bias
        return intlora_layer_norm_job(_ptr(self.x), _ptr(self.weight), _ptr(self.bias),
                                      _ptr(self.y), _ptr(self.mean), _ptr(self.rstd), tokens, n,
                                      ld_x, ld_y, _elem_type("x", self.x),
                                      TYPE_F32 if param is None else _elem_type("weight", param),
                                      _elem_type("y", self.y), self.eps)

    def device(self):
        return self.x.device


@dataclass
class LayerNormBackwardJob:
    dy: object                      # fp32, bf16 or fp16 [tokens, n]
    x: object                       # [tokens, n], the forward's input
    weight: object                  # [n] or None
    mean: object                    # fp32 [tokens], from the forward
    rstd: object                    # fp32 [tokens], from the forward
    dx: object = None               # [tokens, n]
    dweight: object = None          # fp32 [n]
    dbias: object = None            # fp32 [n]
    accumulate: bool = False        # add to dweight and dbias

    def to_c(self) -> intlora_layer_norm_backward_job:
        import torch
        _one_device(self.dy, self.x, self.weight, self.mean, self.rstd, self.dx, self.dweight,
                    self.dbias)
        ld_x = _matrix("x", self.x)
        tokens, n = self.x.shape
        ld_dy = _matrix("dy", self.dy, tokens, n)
        ld_dx = _matrix("dx", self.dx, tokens, n) if self.dx is not None else n
        _vector("weight", self.weight, n)
        _vector("mean", self.mean, tokens, torch.float32)
        _vector("rstd", self.rstd, tokens, torch.float32)
        _vector("dweight", self.dweight, n, torch.float32)
        _vector("dbias", self.dbias, n, torch.float32)
        return intlora_layer_norm_backward_job(
            _ptr(self.dy), _ptr(self.x), _ptr(self.weight), _ptr(self.mean), _ptr(self.rstd),
            _ptr(self.dx), _ptr(self.dweight), _ptr(self.dbias), tokens, n, ld_dy, ld_x, ld_dx,
            _elem_type("dy", self.dy), _elem_type("x", self.x),
            TYPE_F32 if self.weight is None else _elem_type("weight", self.weight),
            TYPE_F32 if self.dx is None else _elem_type("dx", self.dx), int(self.accumulate))

    def device(self):
        return self.x.device


@dataclass
class EmbeddingJob:
    table: object                   # fp32, bf16 or fp16 [vocab, n]
    ids: object                     # int32 or int64 [tokens]
    y: object                       # [tokens, n]
    scale: float = 1.0
    invalid: object = None          # int32 counter of ids outside the table

    def to_c(self) -> intlora_embedding_job:
        _one_device(self.table, self.ids, self.y, self.invalid)
        ld_table = _matrix("table", self.table)
        vocab, n = self.table.shape
        id_bytes = _ids(self.ids)
        _vector("ids", self.ids, self.ids.numel())
        tokens = self.ids.numel()
        ld_y = _matrix("y", self.y, tokens, n)
        _counter("invalid", self.invalid)
        return intlora_embedding_job(_ptr(self.table), _ptr(self.ids), _ptr(self.y),
                                     _ptr(self.invalid), vocab, n, tokens, ld_table, ld_y,
                                     _elem_type("table", self.table), _elem_type("y", self.y),
                                     id_bytes, self.scale)

    def device(self):
        return self.table.device


@dataclass
class EmbeddingBackwardJob:
    dy: object                      # fp32, bf16 or fp16 [tokens, n]
    ids: object                     # int32 or int64 [tokens]
    dtable: object                  # [vocab, n]
    scale: float = 1.0
    padding_id: int = -1            # its row gets no gradient (-1: none)
    accumulate: bool = False        # add to the rows that have tokens; False: write all of dtable
    invalid: object = None          # int32 counter of ids outside the table

    def to_c(self) -> intlora_embedding_backward_job:
        _one_device(self.dy, self.ids, self.dtable, self.invalid)
        ld_dtable = _matrix("dtable", self.dtable)
        vocab, n = self.dtable.shape
        id_bytes = _ids(self.ids)
        _vector("ids", self.ids, self.ids.numel())
        tokens = self.ids.numel()
        ld_dy = _matrix("dy", self.dy, tokens, n)
        _counter("invalid", self.invalid)
        return intlora_embedding_backward_job(
            _ptr(self.dy), _ptr(self.ids), _ptr(self.dtable), _ptr(self.invalid), vocab, n, tokens,
            self.padding_id, ld_dy, ld_dtable, _elem_type("dy", self.dy),
            _elem_type("dtable", self.dtable), id_bytes, int(self.accumulate), self.scale)

    def device(self):
        return self.dtable.device


@dataclass
class GradJob:
    g: object                       # fp32, bf16 or fp16, contiguous, any shape

    def to_c(self) -> intlora_grad_job:
        _one_device(self.g)
        if not self.g.is_contiguous():
            raise ValueError("g must be contiguous")
        return intlora_grad_job(_ptr(self.g), self.g.numel(), _elem_type("g", self.g))

    def device(self):
        return self.g.device


def _array(struct, items):
    if isinstance(items, Descriptors):
        if items.struct is not struct:
            raise TypeError(f"descriptors of {items.struct.__name__}, expected {struct.__name__}")
        return items.arr
    arr = (struct * max(1, len(items)))()
    for k, it in enumerate(items):
        arr[k] = it.to_c()
    return arr


def _device_index(jobs) -> int:
    indices = {j.device().index for j in jobs}
    if len(indices) != 1:
        raise ValueError(f"the jobs of a call must be on one device, got {sorted(indices)}")
    return indices.pop()


def _here(jobs, *others) -> None:
    """The library launches on the current device: the tensors must be there,
    the workspace and the norm (`others`, None left out) too."""
    import torch
    if isinstance(jobs, Descriptors):
        index = jobs.device_index
    else:
        index = _device_index(jobs) if len(jobs) else None
    for t in others:
        if t is None:
            continue
        at = t.get_device()
        if at < 0 or not t.is_contiguous():
            raise ValueError("workspace and norm must be contiguous and on a CUDA device")
        if index is None:
            index = at
        elif at != index:
            raise ValueError(f"workspace or norm is on cuda:{at}, other tensors on cuda:{index}")
    if index is not None and index != torch.cuda.current_device():
        raise ValueError(f"tensors are on cuda:{index}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")


def _norm_scalar(norm) -> int:
    import torch
    if norm.dtype != torch.float32 or norm.numel() != 1 or not norm.is_cuda:
        raise TypeError("norm must be one fp32 element on a CUDA device")
    return norm.data_ptr()


class Descriptors:
    """A list of descriptors converted to their C structs once, for calls that
    repeat on the same buffers (the per-call conversion of a 128-layer list
    costs milliseconds of Python). Pass it wherever a list is accepted. The
    structs hold addresses, so the descriptors, and with them their tensors, live
    as long as this does."""

    _STRUCT = {}

    def __init__(self, items):
        items = list(items)
        if not items:
            raise ValueError("empty descriptor list")
        self.struct = self._STRUCT[type(items[0])]
        self.arr = (self.struct * len(items))()
        for k, it in enumerate(items):
            if type(it) is not type(items[0]):
                raise TypeError("mixed descriptor types")
            self.arr[k] = it.to_c()
        self.items = items
        self.count = len(items)
        self.device_index = _device_index(items) if hasattr(items[0], "device") else None

    def __len__(self):
        return self.count


Descriptors._STRUCT = {AuxJob: intlora_aux_job, Layer: intlora_layer,
                       MergeOut: intlora_merge_out, SteJob: intlora_ste_job,
                       IntGemmJob: intlora_int_gemm_job, LinearJob: intlora_linear_job,
                       FakeQuantJob: intlora_fakequant_job,
                       TrainBackwardJob: intlora_train_backward_job,
                       LayerNormJob: intlora_layer_norm_job,
                       LayerNormBackwardJob: intlora_layer_norm_backward_job,
                       EmbeddingJob: intlora_embedding_job,
                       EmbeddingBackwardJob: intlora_embedding_backward_job,
                       GradJob: intlora_grad_job}


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def intlora_version() -> int:
    return lib().intlora_version()


def intlora_device_timeouts() -> int:
    """Bounded device waits that gave up since the library was loaded."""
    return lib().intlora_device_timeouts()


def intlora_device_status() -> int:
    """INTLORA_OK, or INTLORA_ERR_TIMEOUT when bounded device waits gave up
    since the last check (synchronizes the device). Returns the status code
    (no exception), so callers can tell the two apart."""
    return lib().intlora_device_status()


def intlora_selftest_bounded_wait(limit_us: int, stream=None) -> None:
    """Enqueues the self-test kernel whose bounded wait runs out."""
    _check(lib().intlora_selftest_bounded_wait(limit_us, _stream(stream)))


def intlora_kernel_launches() -> int:
    """Kernels the library has enqueued since it was loaded (host counter)."""
    return lib().intlora_kernel_launches()


def intlora_merge_out_bytes(variant: int, w_bits: int, out_bits: int) -> int:
    return lib().intlora_merge_out_bytes(variant, w_bits, out_bits)


def intlora_gen_aux_workspace_size(jobs: Sequence[AuxJob]) -> int:
    return lib().intlora_gen_aux_workspace_size(_array(intlora_aux_job, jobs), len(jobs))


def intlora_gen_aux_batched(jobs: Sequence[AuxJob], ws=None, stream=None) -> None:
    p, nb = _ws(ws)
    _check(lib().intlora_gen_aux_batched(_array(intlora_aux_job, jobs), len(jobs), p, nb,
                                         _stream(stream)))


def intlora_gen_aux(job: AuxJob, ws=None, stream=None) -> None:
    c = job.to_c()
    p, nb = _ws(ws)
    _check(lib().intlora_gen_aux(c.W, c.d, c.n, c.seed, c.stream_id, c.alpha, c.w_bits,
                                 c.sigma_w_out, c.sigma_r_out, c.r_star_out, c.w_round_out,
                                 c.ld_w_out, c.s_out, c.z_out, p, nb, _stream(stream)))


def intlora_gen_aux_noalloc(job: AuxJob, stream=None) -> None:
    """Layer preparation with the library's built-in scratch (no workspace)."""
    c = job.to_c()
    _check(lib().intlora_gen_aux_noalloc(c.W, c.d, c.n, c.seed, c.stream_id, c.alpha, c.w_bits,
                                         c.sigma_w_out, c.sigma_r_out, c.r_star_out,
                                         c.w_round_out, c.ld_w_out, c.s_out, c.z_out,
                                         _stream(stream)))


def intlora_merge_workspace_size(layers: Sequence[Layer]) -> int:
    return lib().intlora_merge_workspace_size(_array(intlora_layer, layers), len(layers))


def intlora_merge_mul(layer: Layer, u_bits: int, out: MergeOut, ws=None, stream=None) -> None:
    p, nb = _ws(ws)
    c = layer.to_c()
    _check(lib().intlora_merge_mul(ctypes.byref(c), u_bits, _ptr(out.out), _ptr(out.sbar),
                                   _ptr(out.zbar), _ptr(out.code), p, nb, _stream(stream)))


def intlora_merge_shift(layer: Layer, shift_bits: int, out: MergeOut, ws=None,
                        stream=None) -> None:
    p, nb = _ws(ws)
    c = layer.to_c()
    _check(lib().intlora_merge_shift(ctypes.byref(c), shift_bits, _ptr(out.out), _ptr(out.sbar),
                                     _ptr(out.code), p, nb, _stream(stream)))


def intlora_merge_mul_batched(layers: Sequence[Layer], outs: Sequence[MergeOut], u_bits: int,
                              ws=None, stream=None) -> None:
    p, nb = _ws(ws)
    _check(lib().intlora_merge_mul_batched(_array(intlora_layer, layers),
                                           _array(intlora_merge_out, outs), len(layers), u_bits,
                                           p, nb, _stream(stream)))


def intlora_merge_shift_batched(layers: Sequence[Layer], outs: Sequence[MergeOut],
                                shift_bits: int, ws=None, stream=None) -> None:
    p, nb = _ws(ws)
    _check(lib().intlora_merge_shift_batched(_array(intlora_layer, layers),
                                             _array(intlora_merge_out, outs), len(layers),
                                             shift_bits, p, nb, _stream(stream)))


def intlora_ste_workspace_size(jobs: Sequence[SteJob]) -> int:
    return lib().intlora_ste_workspace_size(_array(intlora_ste_job, jobs), len(jobs))


def intlora_ste_backward(job: SteJob, ws=None, stream=None) -> None:
    c = job.to_c()
    p, nb = _ws(ws)
    _check(lib().intlora_ste_backward(c.G, c.A, c.B, c.d, c.n, c.r, c.dA, c.dB, p, nb,
                                      _stream(stream)))


def intlora_ste_backward_batched(jobs: Sequence[SteJob], ws=None, stream=None) -> None:
    p, nb = _ws(ws)
    _check(lib().intlora_ste_backward_batched(_array(intlora_ste_job, jobs), len(jobs), p, nb,
                                              _stream(stream)))


def intlora_int_planes(max_abs: int) -> int:
    return lib().intlora_int_planes(max_abs)


def intlora_int_pack(q, planes: int, packed, overflow=None, stream=None) -> None:
    """Packs the merged integer weights q (int8/int16/int32 [d, n]) into
    base-128 digit planes packed (int8 [d, planes, n])."""
    d, n = q.shape
    _check(lib().intlora_int_pack(_ptr(q), q.element_size(), d, n, planes, _ptr(packed),
                                  _ptr(overflow), _stream(stream)))


def intlora_int_gemm_batched(jobs: Sequence[IntGemmJob], planes: int, stream=None) -> None:
    _check(lib().intlora_int_gemm_batched(_array(intlora_int_gemm_job, jobs), len(jobs), planes,
                                          _stream(stream)))


def intlora_int_gemm(job: IntGemmJob, planes: int, stream=None) -> None:
    """Single-layer call (fp32 Y; a bf16 Y goes through intlora_int_gemm_batched)."""
    c = job.to_c()
    if c.y_bf16:
        raise TypeError("intlora_int_gemm writes fp32 Y; use intlora_int_gemm_batched for bf16 Y")
    _check(lib().intlora_int_gemm(c.X, c.x_scale, c.W, c.w_scale, c.tokens, c.d, c.n, planes,
                                  c.Y, _stream(stream)))


def intlora_fakequant_bf16(q, sbar, w_out, stream=None) -> None:
    """w_out (bf16 [d, n]) = bf16(fp32(sbar_i) * q_ij) for merged weights q."""
    d, n = q.shape
    _check(lib().intlora_fakequant_bf16(_ptr(q), q.element_size(), _ptr(sbar), d, n, _ptr(w_out),
                                        _stream(stream)))


def intlora_linear_bf16_batched(jobs: Sequence[LinearJob], stream=None) -> None:
    _check(lib().intlora_linear_bf16_batched(_array(intlora_linear_job, jobs), len(jobs),
                                             _stream(stream)))


def intlora_train_backward_workspace_size(jobs: Sequence[TrainBackwardJob]) -> int:
    return lib().intlora_train_backward_workspace_size(_array(intlora_train_backward_job, jobs),
                                                       len(jobs))


def intlora_train_backward_batched(jobs: Sequence[TrainBackwardJob], ws=None, stream=None) -> None:
    p, nb = _ws(ws)
    _check(lib().intlora_train_backward_batched(_array(intlora_train_backward_job, jobs), len(jobs),
                                                p, nb, _stream(stream)))


def intlora_fakequant_bf16_batched(jobs: Sequence[FakeQuantJob], stream=None) -> None:
    _check(lib().intlora_fakequant_bf16_batched(_array(intlora_fakequant_job, jobs), len(jobs),
                                                _stream(stream)))


def intlora_layer_norm_batched(jobs: Sequence[LayerNormJob], stream=None) -> None:
    arr = _array(intlora_layer_norm_job, jobs)
    _here(jobs)
    _check(lib().intlora_layer_norm_batched(arr, len(jobs), _stream(stream)))


def intlora_layer_norm_backward_workspace_size(jobs: Sequence[LayerNormBackwardJob]) -> int:
    return lib().intlora_layer_norm_backward_workspace_size(
        _array(intlora_layer_norm_backward_job, jobs), len(jobs))


def intlora_layer_norm_backward_batched(jobs: Sequence[LayerNormBackwardJob], ws=None,
                                        stream=None) -> None:
    arr = _array(intlora_layer_norm_backward_job, jobs)
    _here(jobs, ws)
    p, nb = _ws(ws)
    _check(lib().intlora_layer_norm_backward_batched(arr, len(jobs), p, nb, _stream(stream)))


def intlora_embedding_batched(jobs: Sequence[EmbeddingJob], stream=None) -> None:
    arr = _array(intlora_embedding_job, jobs)
    _here(jobs)
    _check(lib().intlora_embedding_batched(arr, len(jobs), _stream(stream)))


def intlora_embedding_backward_workspace_size(jobs: Sequence[EmbeddingBackwardJob]) -> int:
    return lib().intlora_embedding_backward_workspace_size(
        _array(intlora_embedding_backward_job, jobs), len(jobs))


def intlora_embedding_backward_batched(jobs: Sequence[EmbeddingBackwardJob], ws=None,
                                       stream=None) -> None:
    arr = _array(intlora_embedding_backward_job, jobs)
    _here(jobs, ws)
    p, nb = _ws(ws)
    _check(lib().intlora_embedding_backward_batched(arr, len(jobs), p, nb, _stream(stream)))


def intlora_grad_norm_workspace_size(jobs: Sequence[GradJob]) -> int:
    return lib().intlora_grad_norm_workspace_size(_array(intlora_grad_job, jobs), len(jobs))


def intlora_grad_norm_batched(jobs: Sequence[GradJob], norm, ws=None, stream=None) -> None:
    """norm (fp32, one element) = sqrt(sum of g^2 over all jobs)."""
    arr = _array(intlora_grad_job, jobs)
    _here(jobs, ws, norm)
    p, nb = _ws(ws)
    _check(lib().intlora_grad_norm_batched(arr, len(jobs), _norm_scalar(norm), p, nb,
                                           _stream(stream)))


def intlora_grad_clip_batched(jobs: Sequence[GradJob], max_norm: float, norm, stream=None) -> None:
    """g *= min(1, max_norm / (norm + 1e-6)) in place, norm as given."""
    arr = _array(intlora_grad_job, jobs)
    _here(jobs, norm)
    _check(lib().intlora_grad_clip_batched(arr, len(jobs), max_norm, _norm_scalar(norm),
                                           _stream(stream)))


def intlora_clip_grad_norm_batched(jobs: Sequence[GradJob], max_norm: float, norm, ws=None,
                                   stream=None) -> None:
    """Both: norm is written, and the gradients are clipped by it in place."""
    arr = _array(intlora_grad_job, jobs)
    _here(jobs, ws, norm)
    p, nb = _ws(ws)
    _check(lib().intlora_clip_grad_norm_batched(arr, len(jobs), max_norm, _norm_scalar(norm), p, nb,
                                                _stream(stream)))
