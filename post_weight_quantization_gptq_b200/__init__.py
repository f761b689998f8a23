"""Python binding of the sm_100a GPTQ layer quantizer (libgptq_b200.so).

Argument marshalling only: every function below forwards torch CUDA tensors
as raw device pointers (and the current CUDA stream) to the C ABI declared in
``include/gptq.h`` under the same name.  All arithmetic runs in the library's
CUDA kernels; there is no CPU path.  Importing this package fails loudly when
the library has not been built (``python
post_weight_quantization_gptq_b200/build.py``).

Stages (see the header for the exact contracts):

* ``gptq_hessian_accumulate``  H += 2 X^T X            (tcgen05 bf16 GEMM)
* ``gptq_hessian_accumulate_host``  the same with X in host memory, copies
  overlapped with the GEMM through a two-slot device staging buffer
* ``gptq_prepare_hinv``        dead columns, act-order, damping, U = chol-inverse factor
* ``gptq_quantize_layer``      column walk with OBQ error feedback and lazy updates
* ``gptq_pack``                codes -> uint32 bit stream (8 codes per word at 4 bits)
* ``gptq_dequant_matmul``      Y = X W_hat^T from the packed layer (decode form)
* ``gptq_dequant_gemm``        the same for many tokens on the tensor cores (bf16 W_hat)
* ``gptq_dequant_matmul_linear`` / ``_gated``  the decode form with its epilogue, bf16 Y:
  act(X W^T + bias) + residual, and act(X Wg^T) * (X Wu^T) for a gated feed-forward block
* ``gptq_dequant_gemm_linear`` / ``_gated``  the same for many tokens on the tensor cores
* ``gptq_dequant_gemm_linear_backward`` / ``_gated_backward``  their gradients
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "GPTQConfig", "GPTQError", "gptq_hessian_accumulate", "gptq_hessian_accumulate_host",
    "gptq_hessian_staging_size", "gptq_prepare_hinv", "gptq_dequant_matmul", "gptq_dequant_matmul_workspace_size",
    "gptq_dequant_gemm", "gptq_dequant_gemm_workspace_size",
    "gptq_dequant_matmul_linear", "gptq_dequant_matmul_linear_workspace_size",
    "gptq_dequant_matmul_gated", "gptq_dequant_matmul_gated_workspace_size", "ACTIVATIONS",
    "gptq_dequant_gemm_linear", "gptq_dequant_gemm_linear_workspace_size",
    "gptq_dequant_gemm_gated", "gptq_dequant_gemm_gated_workspace_size",
    "gptq_dequant_gemm_linear_backward", "gptq_dequant_gemm_linear_backward_workspace_size",
    "gptq_dequant_gemm_gated_backward", "gptq_dequant_gemm_gated_backward_workspace_size",
    "gptq_quantize_layer", "gptq_quantize_layer_noalloc", "gptq_noalloc_scratch_bytes", "gptq_pack", "gptq_workspace_size", "gptq_sync_status",
    "gptq_status_string", "gptq_version", "gptq_launch_counter", "gptq_debug_arm_wait_probe",
    "library_path", "n_groups", "packed_words",
    "STATUS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libgptq_b200.so")

STATUS = {0: "GPTQ_OK", 1: "GPTQ_ERR_INVALID_ARG", 2: "GPTQ_ERR_UNSUPPORTED",
          3: "GPTQ_ERR_NOT_PD", 4: "GPTQ_ERR_TIMEOUT", 5: "GPTQ_ERR_CUDA",
          6: "GPTQ_ERR_WORKSPACE"}

# gptq_activation, by name
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


class GPTQConfig(ctypes.Structure):
    """Mirror of ``gptq_config``: bits, group_size (-1 = one group per row),
    block_size (128), desc_act, damp (lambda = damp * mean(diag H)),
    pure_minmax (each group's own [min, max] instead of the range widened to
    contain 0)."""
    _fields_ = [("bits", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("desc_act", ctypes.c_int32),
                ("damp", ctypes.c_float), ("pure_minmax", ctypes.c_int32)]

    def __init__(self, bits=4, group_size=128, desc_act=False, damp=0.01, block_size=128,
                 pure_minmax=False):
        super().__init__(int(bits), int(group_size), int(block_size), int(bool(desc_act)),
                         float(damp), int(bool(pure_minmax)))


class GPTQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {STATUS.get(self.status, self.status)} "
                         f"({gptq_status_string(self.status)})")


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is missing: build the CUDA library first "
            "(python post_weight_quantization_gptq_b200/build.py)")
    lib = ctypes.CDLL(_LIB_PATH)
    P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    cfgp = ctypes.POINTER(GPTQConfig)
    sig = {
        "gptq_status_string": ([i32], ctypes.c_char_p),
        "gptq_version": ([], i32),
        "gptq_launch_counter": ([], ctypes.c_int64),
        "gptq_workspace_size": ([cfgp, i64, i64, ctypes.POINTER(ctypes.c_size_t)], ctypes.c_int),
        "gptq_hessian_accumulate": ([P, i64, i64, i64, P, i64, P, P, ctypes.c_size_t, P],
                                    ctypes.c_int),
        "gptq_hessian_accumulate_host": ([P, i64, i64, i64, P, i64, P, P, ctypes.c_size_t, P],
                                         ctypes.c_int),
        "gptq_hessian_staging_size": ([i64, i64], ctypes.c_size_t),
        "gptq_prepare_hinv": ([P, i64, i64, cfgp, P, P, P, P, P, ctypes.c_size_t, P],
                              ctypes.c_int),
        "gptq_quantize_layer": ([P, i64, i64, i64, P, P, P, cfgp, P, P, P, P, P,
                                 ctypes.c_size_t, P], ctypes.c_int),
        "gptq_pack": ([P, i64, i64, i32, P, P], ctypes.c_int),
        "gptq_dequant_matmul": ([P, i64, i64, i64, P, P, P, P, i64, i32, i32, P, i64, P,
                                 ctypes.c_size_t, P], ctypes.c_int),
        "gptq_dequant_matmul_workspace_size": ([i64, i64], ctypes.c_size_t),
        "gptq_dequant_gemm": ([P, i64, i64, i64, P, P, P, P, i64, i32, i32, P, i64, P, P,
                               ctypes.c_size_t, P], ctypes.c_int),
        "gptq_dequant_gemm_workspace_size": ([i64, i64], ctypes.c_size_t),
        "gptq_dequant_matmul_linear": ([P, i64, i64, i64, P, P, P, P, i64, i32, i32, P, i32, P, i64,
                                        P, i64, P, P, ctypes.c_size_t, P], ctypes.c_int),
        "gptq_dequant_matmul_linear_workspace_size": ([i64, i64], ctypes.c_size_t),
        "gptq_dequant_matmul_gated": ([P, i64, i64, i64, P, P, P, P, P, P, P, i64, i32, i32, i32,
                                       P, i64, P, P, ctypes.c_size_t, P], ctypes.c_int),
        "gptq_dequant_matmul_gated_workspace_size": ([i64, i64], ctypes.c_size_t),
        "gptq_dequant_gemm_linear": ([P, i64, i64, i64, P, P, P, P, i64, i32, i32, P, i32, P, i64,
                                      P, i64, P, i64, P, P, ctypes.c_size_t, P], ctypes.c_int),
        "gptq_dequant_gemm_gated": ([P, i64, i64, i64, P, P, P, P, P, P, P, i64, i32, i32, i32,
                                     P, i64, P, i64, P, i64, P, P, ctypes.c_size_t, P],
                                    ctypes.c_int),
        "gptq_dequant_gemm_linear_backward": ([P, i64, i64, i64, P, P, P, P, i64, i32, i32, i32, P,
                                               i64, P, i64, P, P, i64, P, P, ctypes.c_size_t, P],
                                              ctypes.c_int),
        "gptq_dequant_gemm_gated_backward": ([P, i64, i64, i64, P, i64, P, i64, P, P, P, P, P, P, P,
                                              i64, i32, i32, i32, P, i64, P, i64, P, i64, P, P,
                                              ctypes.c_size_t, P], ctypes.c_int),
        "gptq_dequant_gemm_linear_workspace_size": ([i64, i64, i64], ctypes.c_size_t),
        "gptq_dequant_gemm_gated_workspace_size": ([i64, i64, i64], ctypes.c_size_t),
        "gptq_dequant_gemm_linear_backward_workspace_size": ([i64, i64, i64], ctypes.c_size_t),
        "gptq_dequant_gemm_gated_backward_workspace_size": ([i64, i64, i64], ctypes.c_size_t),
        "gptq_quantize_layer_noalloc": ([P, i64, i64, i64, P, P, P, cfgp, P, P, P, P, P],
                                        ctypes.c_int),
        "gptq_noalloc_scratch_bytes": ([], ctypes.c_size_t),
        "gptq_sync_status": ([P, P, ctypes.POINTER(i32)], ctypes.c_int),
        "gptq_debug_arm_wait_probe": ([i32, i64], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()


def library_path() -> str:
    return _LIB_PATH


def gptq_status_string(status: int) -> str:
    return _lib.gptq_status_string(int(status)).decode()


def gptq_version() -> int:
    return int(_lib.gptq_version())


def gptq_launch_counter() -> int:
    """Kernels launched by the library in this process so far."""
    return int(_lib.gptq_launch_counter())


def n_groups(d_col: int, group_size: int) -> int:
    g = d_col if group_size == -1 or group_size > d_col else group_size
    return -(-d_col // g)


def packed_words(d_col: int, bits: int) -> int:
    return -(-(d_col * bits) // 32)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return getattr(stream, "cuda_stream", stream)


def _check(status: int, where: str) -> None:
    if status != 0:
        raise GPTQError(status, where)


def _cuda(t: torch.Tensor, name: str, dtype=None) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _row_major(t: torch.Tensor, name: str) -> int:
    """Leading dimension of a 2-D tensor with unit column stride."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], t.stride(0))


def _same_device(ref: torch.Tensor, ref_name: str, *others) -> None:
    """Every (tensor, name, dtype) of ``others`` that is given lives on ref's
    device, and that device is the current one: the library launches on the
    current device and its kernels dereference every pointer there, so a
    buffer elsewhere (host memory, another GPU) is refused here instead of
    being read by a kernel.  dtype None accepts any element type."""
    for t, name, dtype in others:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != ref.device:
            where = t.device if isinstance(t, torch.Tensor) else type(t).__name__
            raise ValueError(f"{name} must be on {ref.device} like {ref_name}, not on {where}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ref.device.index != torch.cuda.current_device():
        raise ValueError(f"{ref_name} is on {ref.device} but cuda:{torch.cuda.current_device()} "
                         "is current: make its device current (torch.cuda.device(...))")


def gptq_workspace_size(cfg: GPTQConfig, d_row: int, d_col: int) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.gptq_workspace_size(ctypes.byref(cfg), int(d_row), int(d_col), ctypes.byref(out)),
           "gptq_workspace_size")
    return int(out.value)


def gptq_hessian_accumulate(X: torch.Tensor, H: torch.Tensor, dev_status: torch.Tensor | None = None,
                            ws: torch.Tensor | None = None, stream=None) -> None:
    """H += 2 X^T X (X: n x d bf16, H: d x d fp32, both CUDA, row-major)."""
    _cuda(X, "X", torch.bfloat16)
    _cuda(H, "H", torch.float32)
    _same_device(X, "X", (H, "H", torch.float32), (dev_status, "dev_status", torch.int32),
                 (ws, "ws", None))
    n, d = X.shape
    ldx = _row_major(X, "X")
    ldh = _row_major(H, "H")
    _check(_lib.gptq_hessian_accumulate(_ptr(X), n, d, ldx, _ptr(H), ldh, _ptr(dev_status),
                                        _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                        _stream(stream)), "gptq_hessian_accumulate")


def gptq_hessian_accumulate_host(X: torch.Tensor, H: torch.Tensor, staging: torch.Tensor,
                                 dev_status: torch.Tensor | None = None, stream=None) -> None:
    """H += 2 X^T X with X (n x d bf16) in HOST memory, streamed through the
    device buffer ``staging`` (two slots; copies overlap the GEMM when X is
    pinned).  X must stay unchanged until the stream has run the call."""
    if not isinstance(X, torch.Tensor) or X.is_cuda or X.dtype != torch.bfloat16:
        raise TypeError("X must be a host bf16 tensor")
    _cuda(H, "H", torch.float32)
    _cuda(staging, "staging")
    _same_device(H, "H", (staging, "staging", None), (dev_status, "dev_status", torch.int32))
    n, d = X.shape
    ldx = _row_major(X, "X")
    _check(_lib.gptq_hessian_accumulate_host(_ptr(X), n, d, ldx, _ptr(H), _row_major(H, "H"),
                                             _ptr(dev_status), _ptr(staging),
                                             staging.numel() * staging.element_size(),
                                             _stream(stream)), "gptq_hessian_accumulate_host")


def gptq_hessian_staging_size(d: int, chunk_tokens: int) -> int:
    """Bytes of staging gptq_hessian_accumulate_host needs for chunk_tokens-token chunks."""
    return int(_lib.gptq_hessian_staging_size(int(d), int(chunk_tokens)))


def gptq_prepare_hinv(H: torch.Tensor, cfg: GPTQConfig, U: torch.Tensor, perm: torch.Tensor,
                      dead: torch.Tensor, dev_status: torch.Tensor | None, ws: torch.Tensor,
                      stream=None) -> None:
    """Consumes H (lower triangle); writes U (d x d upper, quantization
    order), perm (int32) and dead (uint8)."""
    _cuda(H, "H", torch.float32)
    _cuda(U, "U", torch.float32)
    _cuda(perm, "perm", torch.int32)
    _cuda(dead, "dead", torch.uint8)
    if ws is None:
        raise ValueError("gptq_prepare_hinv needs a workspace (gptq_workspace_size bytes)")
    _same_device(H, "H", (U, "U", torch.float32), (perm, "perm", torch.int32),
                 (dead, "dead", torch.uint8), (dev_status, "dev_status", torch.int32),
                 (ws, "ws", None))
    d = H.shape[0]
    if not U.is_contiguous() or tuple(U.shape) != (d, d):
        raise ValueError("U must be a contiguous d x d tensor")
    _check(_lib.gptq_prepare_hinv(_ptr(H), d, _row_major(H, "H"), ctypes.byref(cfg), _ptr(U),
                                  _ptr(perm), _ptr(dead), _ptr(dev_status), _ptr(ws),
                                  ws.numel() * ws.element_size(), _stream(stream)),
           "gptq_prepare_hinv")


def gptq_quantize_layer(W: torch.Tensor, U: torch.Tensor, perm: torch.Tensor, dead: torch.Tensor,
                        cfg: GPTQConfig, codes: torch.Tensor, scales: torch.Tensor,
                        zeros: torch.Tensor, dev_status: torch.Tensor | None, ws: torch.Tensor,
                        stream=None) -> None:
    """W (d_row x d_col fp32, original order; overwritten) -> codes (uint8,
    quantization order), scales (fp32 [groups][d_row]), zeros (int32)."""
    _cuda(W, "W", torch.float32)
    _cuda(codes, "codes", torch.uint8)
    _cuda(scales, "scales", torch.float32)
    _cuda(zeros, "zeros", torch.int32)
    if ws is None:
        raise ValueError("gptq_quantize_layer needs a workspace (gptq_workspace_size bytes)")
    _same_device(W, "W", (U, "U", torch.float32), (perm, "perm", torch.int32),
                 (dead, "dead", torch.uint8), (codes, "codes", None), (scales, "scales", None),
                 (zeros, "zeros", None), (dev_status, "dev_status", torch.int32), (ws, "ws", None))
    d_row, d_col = W.shape
    for t, name in ((codes, "codes"), (scales, "scales"), (zeros, "zeros"), (U, "U")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    _check(_lib.gptq_quantize_layer(_ptr(W), d_row, d_col, _row_major(W, "W"), _ptr(U), _ptr(perm),
                                    _ptr(dead), ctypes.byref(cfg), _ptr(codes), _ptr(scales),
                                    _ptr(zeros), _ptr(dev_status), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream)),
           "gptq_quantize_layer")


def gptq_quantize_layer_noalloc(W: torch.Tensor, U: torch.Tensor, perm: torch.Tensor,
                                dead: torch.Tensor, cfg: GPTQConfig, codes: torch.Tensor,
                                scales: torch.Tensor, zeros: torch.Tensor,
                                dev_status: torch.Tensor | None, stream=None) -> None:
    """gptq_quantize_layer without a workspace, for callers that cannot
    allocate device memory (an enqueue call that may not allocate, a memory
    pool that already holds nearly all of HBM, a path that cannot afford the
    device synchronization of cudaMalloc / cudaFree).  The scratch is a fixed
    array inside the library (gptq_noalloc_scratch_bytes() per device), shared
    by every call: calls that overlap on the GPU race on it."""
    _cuda(W, "W", torch.float32)
    _cuda(codes, "codes", torch.uint8)
    _cuda(scales, "scales", torch.float32)
    _cuda(zeros, "zeros", torch.int32)
    d_row, d_col = W.shape
    for t, name in ((codes, "codes"), (scales, "scales"), (zeros, "zeros"), (U, "U")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    # the scratch array used is the current device's: every buffer must be on
    # W's device, and the call runs with that device current
    for t, name in ((U, "U"), (perm, "perm"), (dead, "dead"), (codes, "codes"),
                    (scales, "scales"), (zeros, "zeros"), (dev_status, "dev_status")):
        if t is not None and (not t.is_cuda or t.device != W.device):
            raise ValueError(f"{name} must be on {W.device}, like W")
    for t, name, dtype in ((U, "U", torch.float32), (perm, "perm", torch.int32),
                           (dead, "dead", torch.uint8), (dev_status, "dev_status", torch.int32)):
        if t is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    with torch.cuda.device(W.device):
        _check(_lib.gptq_quantize_layer_noalloc(_ptr(W), d_row, d_col, _row_major(W, "W"),
                                                _ptr(U), _ptr(perm), _ptr(dead),
                                                ctypes.byref(cfg), _ptr(codes), _ptr(scales),
                                                _ptr(zeros), _ptr(dev_status), _stream(stream)),
               "gptq_quantize_layer_noalloc")


def gptq_noalloc_scratch_bytes() -> int:
    return int(_lib.gptq_noalloc_scratch_bytes())


def gptq_pack(codes: torch.Tensor, bits: int, packed: torch.Tensor, stream=None) -> None:
    """codes (d_row x d_col uint8) -> packed (d_row x ceil(d_col*bits/32) int32 view of uint32)."""
    _cuda(codes, "codes", torch.uint8)
    _cuda(packed, "packed")
    _same_device(codes, "codes", (packed, "packed", None))
    if not codes.is_contiguous() or not packed.is_contiguous():
        raise ValueError("codes and packed must be contiguous")
    d_row, d_col = codes.shape
    _check(_lib.gptq_pack(_ptr(codes), d_row, d_col, int(bits), _ptr(packed), _stream(stream)),
           "gptq_pack")


def gptq_dequant_matmul(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                        zeros: torch.Tensor, perm: torch.Tensor | None, bits: int,
                        group_size: int, Y: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """Y = X W_hat^T for a quantized layer (decode form): X (tokens x d_col bf16,
    original column order), packed / scales / zeros / perm as the quantizer
    wrote them, Y (tokens x d_row fp32) overwritten, ws a device workspace of
    gptq_dequant_matmul_workspace_size(tokens, d_col) bytes."""
    _cuda(X, "X", torch.bfloat16)
    _cuda(packed, "packed")
    _cuda(scales, "scales", torch.float32)
    _cuda(zeros, "zeros", torch.int32)
    _cuda(Y, "Y", torch.float32)
    _cuda(ws, "ws")
    if perm is not None:
        _cuda(perm, "perm", torch.int32)
    _same_device(X, "X", (packed, "packed", None), (scales, "scales", None),
                 (zeros, "zeros", None), (perm, "perm", None), (Y, "Y", None), (ws, "ws", None))
    for t, name in ((packed, "packed"), (scales, "scales"), (zeros, "zeros")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    n_tok, d_col = X.shape
    d_row = packed.shape[0]
    _check(_lib.gptq_dequant_matmul(_ptr(X), n_tok, d_col, _row_major(X, "X"), _ptr(packed),
                                    _ptr(scales), _ptr(zeros), _ptr(perm), d_row, int(bits),
                                    int(group_size), _ptr(Y), _row_major(Y, "Y"), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream)),
           "gptq_dequant_matmul")


def gptq_dequant_matmul_workspace_size(n_tok: int, d_col: int) -> int:
    return int(_lib.gptq_dequant_matmul_workspace_size(int(n_tok), int(d_col)))


def gptq_dequant_gemm(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                      zeros: torch.Tensor, perm: torch.Tensor | None, bits: int, group_size: int,
                      Y: torch.Tensor, ws: torch.Tensor | None = None,
                      dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Y = X W_hat^T for a quantized layer, many-token form on the tensor
    cores (W_hat dequantized to bf16 per stage): X (tokens x d_col bf16,
    original column order), packed / scales / zeros / perm as the quantizer
    wrote them, Y (tokens x d_row fp32) overwritten; ws (bytes of
    gptq_dequant_gemm_workspace_size) is needed with a permutation."""
    _cuda(X, "X", torch.bfloat16)
    _cuda(packed, "packed")
    _cuda(scales, "scales", torch.float32)
    _cuda(zeros, "zeros", torch.int32)
    _cuda(Y, "Y", torch.float32)
    if perm is not None:
        _cuda(perm, "perm", torch.int32)
    _same_device(X, "X", (packed, "packed", None), (scales, "scales", None),
                 (zeros, "zeros", None), (perm, "perm", None), (Y, "Y", None), (ws, "ws", None),
                 (dev_status, "dev_status", torch.int32))
    for t, name in ((packed, "packed"), (scales, "scales"), (zeros, "zeros")):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    n_tok, d_col = X.shape
    d_row = packed.shape[0]
    _check(_lib.gptq_dequant_gemm(_ptr(X), n_tok, d_col, _row_major(X, "X"), _ptr(packed),
                                  _ptr(scales), _ptr(zeros), _ptr(perm), d_row, int(bits),
                                  int(group_size), _ptr(Y), _row_major(Y, "Y"), _ptr(dev_status),
                                  _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                  _stream(stream)), "gptq_dequant_gemm")


def gptq_dequant_gemm_workspace_size(n_tok: int, d_col: int) -> int:
    return int(_lib.gptq_dequant_gemm_workspace_size(int(n_tok), int(d_col)))


def _activation(name) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {name!r}")
    return ACTIVATIONS[name]


# The products with an epilogue check their operands through the helpers below:
# few attribute reads per tensor (a decode step's kernel runs a few
# microseconds, and the checks are on its critical path).
_Tensor = torch.Tensor
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _refuse(t, name: str, dtype, dev: int) -> None:
    """Raises for an operand that is not a `dtype` tensor on cuda:dev."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be on cuda:{dev} like the first operand, not on {t.device}")


def _first(t, name: str) -> int:
    """The device index of a call's first operand (2-D, bf16), which has to be
    the current device: the library launches there."""
    if not isinstance(t, _Tensor) or t.dtype is not _BF16 or not t.is_cuda:
        _refuse(t, name, _BF16, 0)
    dev = t.get_device()
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev} but cuda:{torch.cuda.current_device()} is current: "
                         "make its device current (torch.cuda.device(...))")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    return dev


def _launch_stream(stream, dev: int):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(dev)
        stream = torch.cuda.current_stream()
    return getattr(stream, "cuda_stream", stream)


def _pitch(t: torch.Tensor, name: str) -> int:
    """Leading dimension of a 2-D tensor with contiguous, separate rows."""
    n, c = t.shape
    ld, step = t.stride()
    if (step != 1 and c > 1) or (n > 1 and ld < c):
        raise ValueError(f"{name} must have contiguous rows that do not overlap (strides {t.stride()})")
    return ld if ld > c else c


def _rows(t, name: str, n: int, cols: int, dev: int) -> int:
    """Leading dimension of an n x cols bf16 operand (0 for None)."""
    if t is None:
        return 0
    if not isinstance(t, _Tensor) or t.dtype is not _BF16 or t.get_device() != dev:
        _refuse(t, name, _BF16, dev)
    if t.shape != (n, cols):
        raise ValueError(f"{name} must be {n} x {cols}, got {tuple(t.shape)}")
    return _pitch(t, name)


def _whole(t, name: str, dtype, shape: tuple, dev: int):
    """Address of a contiguous operand of this shape (None for None)."""
    if t is None:
        return None
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, name, dtype, dev)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, {' x '.join(map(str, shape))}; got {tuple(t.shape)}")
    return t.data_ptr()


def _buffer(t, name: str, dev: int):
    """(address, bytes) of a workspace."""
    if t is None:
        return None, 0
    if not isinstance(t, _Tensor) or t.get_device() != dev:
        _refuse(t, name, None, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def _status(t, dev: int):
    if t is None:
        return None
    if not isinstance(t, _Tensor) or t.dtype is not _I32 or t.get_device() != dev:
        _refuse(t, "dev_status", _I32, dev)
    return t.data_ptr()


def _layer(packed, scales, zeros, bits: int, group_size: int, d_col: int, dev: int, suffix: str = ""):
    """Addresses of a packed layer of input width d_col, and its d_row."""
    for t, name, dtype in ((packed, "packed", _I32), (scales, "scales", _F32), (zeros, "zeros", _I32)):
        if not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != dev:
            _refuse(t, name + suffix, dtype, dev)
        if not t.is_contiguous():
            raise ValueError(f"{name}{suffix} must be contiguous")
    if packed.dim() != 2 or packed.shape[1] != -(-(d_col * bits) // 32):
        raise ValueError(f"packed{suffix} must be d_row x {-(-(d_col * bits) // 32)} words, "
                         f"got {tuple(packed.shape)}")
    d_row = packed.shape[0]
    if group_size > 0 or group_size == -1:   # (the library refuses the others)
        g = d_col if group_size == -1 or group_size > d_col else group_size
        shape = (-(-d_col // g), d_row)
        if scales.shape != shape or zeros.shape != shape:
            raise ValueError(f"scales{suffix} and zeros{suffix} must be {shape[0]} x {d_row}, "
                             f"got {tuple(scales.shape)} and {tuple(zeros.shape)}")
    return packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(), d_row


def gptq_dequant_matmul_linear(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                               zeros: torch.Tensor, perm: torch.Tensor | None, bits: int,
                               group_size: int, Y: torch.Tensor, ws: torch.Tensor | None = None,
                               bias: torch.Tensor | None = None, activation: str = "none",
                               residual: torch.Tensor | None = None,
                               dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Y = act(X W_hat^T + bias) + residual for a few tokens (decode form): X
    (tokens x d_col bf16, original column order), packed / scales / zeros /
    perm as the quantizer wrote them, bias fp32, residual and Y tokens x d_row
    bf16 (residual may be Y itself); ws (bytes of
    gptq_dequant_matmul_linear_workspace_size) is needed with a permutation
    or when X's rows are not 16-byte aligned."""
    dev = _first(X, "X")
    n_tok, d_col = X.shape
    bits, group_size = int(bits), int(group_size)
    p, s, z, d_row = _layer(packed, scales, zeros, bits, group_size, d_col, dev)
    wsp, wsb = _buffer(ws, "ws", dev)
    _check(_lib.gptq_dequant_matmul_linear(
        X.data_ptr(), n_tok, d_col, _pitch(X, "X"), p, s, z, _whole(perm, "perm", _I32, (d_col,), dev),
        d_row, bits, group_size, _whole(bias, "bias", _F32, (d_row,), dev), _activation(activation),
        _ptr(residual), _rows(residual, "residual", n_tok, d_row, dev), _ptr(Y),
        _rows(Y, "Y", n_tok, d_row, dev), _status(dev_status, dev), wsp, wsb,
        _launch_stream(stream, dev)), "gptq_dequant_matmul_linear")


def gptq_dequant_matmul_linear_workspace_size(n_tok: int, d_col: int) -> int:
    return int(_lib.gptq_dequant_matmul_linear_workspace_size(int(n_tok), int(d_col)))


def gptq_dequant_matmul_gated(X: torch.Tensor, packed_gate: torch.Tensor, scales_gate: torch.Tensor,
                              zeros_gate: torch.Tensor, packed_up: torch.Tensor,
                              scales_up: torch.Tensor, zeros_up: torch.Tensor,
                              perm: torch.Tensor | None, bits: int, group_size: int,
                              activation: str, Y: torch.Tensor, ws: torch.Tensor | None = None,
                              dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Y = act(X Wg_hat^T) * (X Wu_hat^T) for a few tokens (decode form): two
    packed layers that share X, perm, bits and group_size; Y tokens x d_row
    bf16; ws as gptq_dequant_matmul_linear."""
    dev = _first(X, "X")
    n_tok, d_col = X.shape
    bits, group_size = int(bits), int(group_size)
    p, s, z, d_row = _layer(packed_gate, scales_gate, zeros_gate, bits, group_size, d_col, dev, "_gate")
    p2, s2, z2, d_up = _layer(packed_up, scales_up, zeros_up, bits, group_size, d_col, dev, "_up")
    if d_up != d_row:
        raise ValueError("packed_gate and packed_up must have the same number of rows")
    wsp, wsb = _buffer(ws, "ws", dev)
    _check(_lib.gptq_dequant_matmul_gated(
        X.data_ptr(), n_tok, d_col, _pitch(X, "X"), p, s, z, p2, s2, z2,
        _whole(perm, "perm", _I32, (d_col,), dev), d_row, bits, group_size, _activation(activation),
        _ptr(Y), _rows(Y, "Y", n_tok, d_row, dev), _status(dev_status, dev), wsp, wsb,
        _launch_stream(stream, dev)), "gptq_dequant_matmul_gated")


def gptq_dequant_matmul_gated_workspace_size(n_tok: int, d_col: int) -> int:
    return int(_lib.gptq_dequant_matmul_gated_workspace_size(int(n_tok), int(d_col)))


def gptq_dequant_gemm_linear(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                             zeros: torch.Tensor, perm: torch.Tensor | None, bits: int,
                             group_size: int, Y: torch.Tensor, ws: torch.Tensor | None = None,
                             bias: torch.Tensor | None = None, activation: str = "none",
                             residual: torch.Tensor | None = None, pre: torch.Tensor | None = None,
                             dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Y = act(X W_hat^T + bias) + residual for many tokens on the tensor cores
    (W_hat as 16-bit weights): operands as gptq_dequant_matmul_linear; pre
    (tokens x d_row bf16), if given, receives the sums before the activation
    for the backward pass; ws of gptq_dequant_gemm_linear_workspace_size bytes."""
    dev = _first(X, "X")
    n_tok, d_col = X.shape
    bits, group_size = int(bits), int(group_size)
    p, s, z, d_row = _layer(packed, scales, zeros, bits, group_size, d_col, dev)
    wsp, wsb = _buffer(ws, "ws", dev)
    _check(_lib.gptq_dequant_gemm_linear(
        X.data_ptr(), n_tok, d_col, _pitch(X, "X"), p, s, z, _whole(perm, "perm", _I32, (d_col,), dev),
        d_row, bits, group_size, _whole(bias, "bias", _F32, (d_row,), dev), _activation(activation),
        _ptr(residual), _rows(residual, "residual", n_tok, d_row, dev), _ptr(pre),
        _rows(pre, "pre", n_tok, d_row, dev), _ptr(Y), _rows(Y, "Y", n_tok, d_row, dev),
        _status(dev_status, dev), wsp, wsb, _launch_stream(stream, dev)), "gptq_dequant_gemm_linear")


def gptq_dequant_gemm_linear_workspace_size(n_tok: int, d_col: int, d_row: int) -> int:
    return int(_lib.gptq_dequant_gemm_linear_workspace_size(int(n_tok), int(d_col), int(d_row)))


def gptq_dequant_gemm_gated(X: torch.Tensor, packed_gate: torch.Tensor, scales_gate: torch.Tensor,
                            zeros_gate: torch.Tensor, packed_up: torch.Tensor,
                            scales_up: torch.Tensor, zeros_up: torch.Tensor,
                            perm: torch.Tensor | None, bits: int, group_size: int, activation: str,
                            Y: torch.Tensor, ws: torch.Tensor | None = None,
                            gate: torch.Tensor | None = None, up: torch.Tensor | None = None,
                            dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Y = act(X Wg_hat^T) * (X Wu_hat^T) for many tokens on the tensor cores,
    both products, the activation and their product in one kernel; gate and
    up (tokens x d_row bf16), if given, receive the two products for the
    backward pass; ws of gptq_dequant_gemm_gated_workspace_size bytes."""
    dev = _first(X, "X")
    n_tok, d_col = X.shape
    bits, group_size = int(bits), int(group_size)
    p, s, z, d_row = _layer(packed_gate, scales_gate, zeros_gate, bits, group_size, d_col, dev, "_gate")
    p2, s2, z2, d_up = _layer(packed_up, scales_up, zeros_up, bits, group_size, d_col, dev, "_up")
    if d_up != d_row:
        raise ValueError("packed_gate and packed_up must have the same number of rows")
    wsp, wsb = _buffer(ws, "ws", dev)
    _check(_lib.gptq_dequant_gemm_gated(
        X.data_ptr(), n_tok, d_col, _pitch(X, "X"), p, s, z, p2, s2, z2,
        _whole(perm, "perm", _I32, (d_col,), dev), d_row, bits, group_size, _activation(activation),
        _ptr(gate), _rows(gate, "gate", n_tok, d_row, dev), _ptr(up), _rows(up, "up", n_tok, d_row, dev),
        _ptr(Y), _rows(Y, "Y", n_tok, d_row, dev), _status(dev_status, dev), wsp, wsb,
        _launch_stream(stream, dev)), "gptq_dequant_gemm_gated")


def gptq_dequant_gemm_gated_workspace_size(n_tok: int, d_col: int, d_row: int) -> int:
    return int(_lib.gptq_dequant_gemm_gated_workspace_size(int(n_tok), int(d_col), int(d_row)))


def gptq_dequant_gemm_linear_backward(dY: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                                      zeros: torch.Tensor, perm: torch.Tensor | None, bits: int,
                                      group_size: int, dX: torch.Tensor,
                                      ws: torch.Tensor | None = None, activation: str = "none",
                                      pre: torch.Tensor | None = None,
                                      dPre: torch.Tensor | None = None,
                                      dbias: torch.Tensor | None = None,
                                      dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Gradients of gptq_dequant_gemm_linear for its output gradient dY (tokens
    x d_row bf16) and the saved pre: dPre = dY act'(pre) (bf16, 16-byte aligned
    rows; may be None without an activation), dbias = its column sums (fp32,
    optional), dX = dPre W_hat (tokens x d_col bf16, original column order); ws
    of gptq_dequant_gemm_linear_backward_workspace_size bytes."""
    dev = _first(dY, "dY")
    n_tok, d_row = dY.shape
    if not isinstance(dX, _Tensor):
        _refuse(dX, "dX", _BF16, dev)
    d_col = dX.shape[-1]
    bits, group_size = int(bits), int(group_size)
    p, s, z, rows = _layer(packed, scales, zeros, bits, group_size, d_col, dev)
    if rows != d_row:
        raise ValueError(f"packed must have dY's {d_row} columns as rows, got {rows}")
    wsp, wsb = _buffer(ws, "ws", dev)
    _check(_lib.gptq_dequant_gemm_linear_backward(
        dY.data_ptr(), n_tok, d_row, _pitch(dY, "dY"), p, s, z, _whole(perm, "perm", _I32, (d_col,), dev),
        d_col, bits, group_size, _activation(activation), _ptr(pre),
        _rows(pre, "pre", n_tok, d_row, dev), _ptr(dPre), _rows(dPre, "dPre", n_tok, d_row, dev),
        _whole(dbias, "dbias", _F32, (d_row,), dev), _ptr(dX), _rows(dX, "dX", n_tok, d_col, dev),
        _status(dev_status, dev), wsp, wsb, _launch_stream(stream, dev)),
        "gptq_dequant_gemm_linear_backward")


def gptq_dequant_gemm_linear_backward_workspace_size(n_tok: int, d_col: int, d_row: int) -> int:
    return int(_lib.gptq_dequant_gemm_linear_backward_workspace_size(int(n_tok), int(d_col),
                                                                     int(d_row)))


def gptq_dequant_gemm_gated_backward(dY: torch.Tensor, gate: torch.Tensor, up: torch.Tensor,
                                     packed_gate: torch.Tensor, scales_gate: torch.Tensor,
                                     zeros_gate: torch.Tensor, packed_up: torch.Tensor,
                                     scales_up: torch.Tensor, zeros_up: torch.Tensor,
                                     perm: torch.Tensor | None, bits: int, group_size: int,
                                     activation: str, dGate: torch.Tensor, dUp: torch.Tensor,
                                     dX: torch.Tensor, ws: torch.Tensor | None = None,
                                     dev_status: torch.Tensor | None = None, stream=None) -> None:
    """Gradients of gptq_dequant_gemm_gated for its output gradient dY and the
    saved gate and up products: dGate = dY up act'(gate), dUp = dY act(gate)
    (bf16, 16-byte aligned rows), dX = dGate Wg_hat + dUp Wu_hat (tokens x d_col
    bf16, original column order); ws of
    gptq_dequant_gemm_gated_backward_workspace_size bytes."""
    dev = _first(dY, "dY")
    n_tok, d_row = dY.shape
    if not isinstance(dX, _Tensor):
        _refuse(dX, "dX", _BF16, dev)
    d_col = dX.shape[-1]
    bits, group_size = int(bits), int(group_size)
    p, s, z, rows = _layer(packed_gate, scales_gate, zeros_gate, bits, group_size, d_col, dev, "_gate")
    p2, s2, z2, rows2 = _layer(packed_up, scales_up, zeros_up, bits, group_size, d_col, dev, "_up")
    if rows != d_row or rows2 != d_row:
        raise ValueError(f"packed_gate and packed_up must have dY's {d_row} columns as rows, "
                         f"got {rows} and {rows2}")
    wsp, wsb = _buffer(ws, "ws", dev)
    _check(_lib.gptq_dequant_gemm_gated_backward(
        dY.data_ptr(), n_tok, d_row, _pitch(dY, "dY"), _ptr(gate),
        _rows(gate, "gate", n_tok, d_row, dev), _ptr(up), _rows(up, "up", n_tok, d_row, dev),
        p, s, z, p2, s2, z2, _whole(perm, "perm", _I32, (d_col,), dev), d_col, bits, group_size,
        _activation(activation), _ptr(dGate), _rows(dGate, "dGate", n_tok, d_row, dev), _ptr(dUp),
        _rows(dUp, "dUp", n_tok, d_row, dev), _ptr(dX), _rows(dX, "dX", n_tok, d_col, dev),
        _status(dev_status, dev), wsp, wsb, _launch_stream(stream, dev)),
        "gptq_dequant_gemm_gated_backward")


def gptq_dequant_gemm_gated_backward_workspace_size(n_tok: int, d_col: int, d_row: int) -> int:
    return int(_lib.gptq_dequant_gemm_gated_backward_workspace_size(int(n_tok), int(d_col),
                                                                    int(d_row)))


def gptq_debug_arm_wait_probe(kernel: int, limit_ns: int) -> None:
    """Test hook: the next launch of kernel kind 1 (Hessian), 2 (the next
    fp32-accurate tensor-core GEMM) or 4, 5, 6 (the products with an epilogue:
    decode form, up to 256 tokens, beyond) waits once, bounded by limit_ns, on a
    barrier nothing completes, and reports GPTQ_ERR_TIMEOUT."""
    _check(_lib.gptq_debug_arm_wait_probe(int(kernel), int(limit_ns)),
           "gptq_debug_arm_wait_probe")


def gptq_sync_status(dev_status: torch.Tensor, stream=None) -> int:
    """Wait for the stream and return the device status word."""
    out = ctypes.c_int32(0)
    _check(_lib.gptq_sync_status(_stream(stream), _ptr(dev_status), ctypes.byref(out)),
           "gptq_sync_status")
    return int(out.value)
