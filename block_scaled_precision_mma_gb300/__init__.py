"""Python binding of libbsmma, the sm_103a block-scaled GEMM library.

Argument marshalling only: every entry point forwards device pointers, int64
sizes and the current CUDA stream to the C ABI declared in ``include/bsmma.h``;
all arithmetic runs in the library's CUDA kernels.  There is no fallback: if the
shared library is missing or fails to load, every call raises.

Functions mirror the C names:

* :func:`mx_gemm`, :func:`mx_gemm_tiled` -- dense MXFP8 / MXFP4 GEMM, BF16 out, optionally
  with a fused per-column bias and activation.
* :func:`grouped_fp8_gemm` -- grouped groupwise FP8 GEMM, BF16 out.
* :func:`mx_scale_relayout`, :func:`mx_scale_tiled_bytes` -- scale-factor relayout.
* :func:`mx_quantize`, :func:`fp8_group_quantize`, :func:`fp8_block_quantize` -- the
  quantisers that make the GEMMs' operands from BF16 / FP32 tensors.
* :func:`moe_route`, :func:`moe_route_backward`, :func:`moe_plan`, :func:`moe_combine`,
  :func:`moe_combine_backward` -- the expert layer around the grouped GEMMs; :func:`moe_step` --
  its experts and their weighted sum for a few tokens.
* :func:`int8_quantize`, :func:`int8_gemm`, :func:`grouped_int8_gemm` -- INT8 products with
  scales for each token and channel.
* :func:`branch_enter`, :func:`branch_leave`, :func:`branch_enter_backward`,
  :func:`branch_leave_backward`, :func:`dropout` -- a residual branch's norms, gate, dropout and
  residual, with the next product's operand made on the way.
* :func:`device_status`, :func:`reserve_workspace`, :func:`set_wait_limit_ns`,
  :func:`launch_count`, :func:`probe_wait_timeout`, :func:`status_string`.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from .build import LIB_PATH, build

__all__ = ["mx_gemm", "mx_gemm_tiled", "mx_gemm_noalloc", "grouped_fp8_gemm", "grouped_fp8_pack_weights",
           "grouped_bf16_gemm",
           "moe_route", "moe_route_backward", "moe_plan", "moe_plan_workspace_bytes",
           "moe_combine", "moe_combine_backward", "moe_step", "moe_step_workspace_bytes",
           "int8_quantize", "int8_gemm", "grouped_int8_gemm",
           "branch_enter", "branch_enter_backward", "branch_leave", "branch_leave_backward",
           "branch_backward_workspace_bytes", "dropout",
           "mx_scale_relayout",
           "mx_quantize", "fp8_group_quantize", "fp8_block_quantize", "autotune_configure",
           "autotune_lookup",
           "mx_scale_tiled_bytes", "device_status", "reserve_workspace", "set_wait_limit_ns",
           "set_dense_variant", "set_grouped_tile_width", "set_grouped_variant", "set_int8_variant",
           "launch_count", "probe_wait_timeout", "status_string", "BsmmaError", "load",
           "LAYOUTS", "FORMATS", "ROLES", "build", "LIB_PATH"]

LAYOUTS = {"NT": 0, "NN": 1, "TN": 2}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
ROLES = {"A": 0, "B": 1}      # scales of op(A) rows / of op(B) rows
FORMATS = {"e4m3": 0, "e5m2": 1, "e2m1": 2}
STATUS = ["BSMMA_OK", "BSMMA_ERR_INVALID_ARG", "BSMMA_ERR_UNSUPPORTED", "BSMMA_ERR_MISALIGNED",
          "BSMMA_ERR_WORKSPACE", "BSMMA_ERR_CUDA", "BSMMA_DEV_TIMEOUT", "BSMMA_DEV_BAD_MSIZES",
          "BSMMA_ERR_SCRATCH_LIMIT"]

_lib = None
_lock = threading.Lock()


class BsmmaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        name = STATUS[code] if 0 <= code < len(STATUS) else f"status {code}"
        super().__init__(f"{where}: {name}")


def load(path: str | None = None):
    """Loads libbsmma.so (built in-tree by ``build()``) and declares its ABI."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(f"libbsmma.so not built ({path}); run __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        lib.mx_gemm.argtypes = [p, p, p, p, p, i64, i64, i64, i32, i32, i32, p]
        lib.mx_gemm_tiled.argtypes = [p, p, p, p, p, i64, i64, i64, i32, i32, i32, p]
        lib.mx_gemm_noalloc.argtypes = [p, p, p, p, p, i64, i64, i64, i32, i32, i32, p]
        lib.grouped_fp8_gemm.argtypes = [p, p, p, p, p, p, i64, i32, i64, i64, p]
        lib.grouped_fp8_gemm_packed.argtypes = [p, p, p, p, p, p, i64, i32, i64, i64, p]
        lib.grouped_fp8_pack_weights.argtypes = [p, i64, i64, i64, p, p]
        lib.grouped_bf16_gemm.argtypes = [p, p, p, p, i64, i32, i64, i64, p]
        lib.mx_scale_relayout.argtypes = [p, i64, i64, i32, p, p]
        lib.mx_scale_tiled_bytes.argtypes = [i64, i64, i32]
        lib.mx_scale_tiled_bytes.restype = i64
        lib.bsmma_reserve_workspace.argtypes = [i64, p]
        lib.bsmma_device_status.argtypes = [p]
        lib.bsmma_set_wait_limit_ns.argtypes = [i64]
        lib.bsmma_set_dense_variant.argtypes = [i32]
        lib.bsmma_set_grouped_tile_width.argtypes = [i32]
        lib.bsmma_set_grouped_variant.argtypes = [i32]
        lib.bsmma_set_int8_variant.argtypes = [i32, i32]
        lib.bsmma_set_int8_variant.restype = i32
        lib.bsmma_status_string.argtypes = [i32]
        lib.bsmma_status_string.restype = ctypes.c_char_p
        lib.bsmma_launch_count.argtypes = []
        lib.bsmma_launch_count.restype = i64
        lib.bsmma_probe_wait_timeout.argtypes = [i64, p]
        lib.mx_quantize.argtypes = [p, i32, i64, i64, i32, i32, p, p, p]
        lib.mx_gemm_bias_act.argtypes = [p, p, p, p, p, i32, p, i64, i64, i64, i32, i32, i32, p]
        lib.bsmma_autotune_configure.argtypes = [i32, ctypes.c_char_p]
        lib.bsmma_autotune_lookup.argtypes = [ctypes.c_char_p]
        lib.bsmma_autotune_lookup.restype = i32
        lib.mx_gemm_tiled_bias_act.argtypes = [p, p, p, p, p, i32, p, i64, i64, i64, i32, i32, i32, p]
        lib.fp8_group_quantize.argtypes = [p, i32, i64, i64, p, i32, p, p, p]
        lib.fp8_block_quantize.argtypes = [p, i32, i64, i64, i64, p, p, p]
        f32 = ctypes.c_float
        lib.moe_route.argtypes = [p, i32, i64, i32, i32, i32, p, i32, i32, i32, i32, f32, p, p, p]
        lib.moe_route_backward.argtypes = [p, i32, i64, i32, i32, i32, i32, f32, p, p, p, p]
        lib.moe_plan.argtypes = [p, i64, i32, i32, p, p, p, p]
        lib.moe_plan_workspace_bytes.argtypes = [i64, i32, i32]
        lib.moe_plan_workspace_bytes.restype = i64
        lib.moe_combine.argtypes = [p, i32, i64, i64, p, p, i64, i32, p, p]
        lib.moe_combine_backward.argtypes = [p, i32, i64, p, p, p, p, i64, i32, p, p, p]
        lib.int8_quantize.argtypes = [p, i32, i64, i64, p, i32, i64, p, p, p]
        lib.int8_gemm.argtypes = [p, p, p, p, p, p, i32, i64, i64, i64, p]
        lib.grouped_int8_gemm.argtypes = [p, p, p, p, p, i32, p, i64, i32, i64, i64, p]
        lib.moe_step.argtypes = [p, i64, i64, p, p, i32, i32, i64, i32, p, p, p, p, i32, p, p]
        lib.moe_step_workspace_bytes.argtypes = [i64, i32, i64, i64]
        lib.moe_step_workspace_bytes.restype = i64
        lib.branch_enter.argtypes = [p, i32, i64, i64, i32, f32, p, p, i32, p, p, p]
        lib.branch_leave.argtypes = [p, i32, p, i32, i64, i64, i32, f32, p, p, p, i64, f32, f32, f32,
                                     p, p, i32, f32, p, p, i32, p, p, p]
        lib.branch_enter_backward.argtypes = [p, i32, p, i32, i64, i64, i32, f32, p, p, p, p, p, p]
        lib.branch_leave_backward.argtypes = [p, i32, p, i32, i64, i64, i32, f32, p, p, p, i64, f32,
                                              f32, f32, p, p, p, p, p, p, p]
        lib.branch_backward_workspace_bytes.argtypes = [i64, i64]
        lib.branch_backward_workspace_bytes.restype = i64
        lib.dropout.argtypes = [p, i32, i64, f32, p, p, p]
        for name in ("mx_gemm", "mx_gemm_tiled", "mx_gemm_noalloc", "grouped_fp8_gemm",
                     "grouped_fp8_gemm_packed", "grouped_fp8_pack_weights",
                     "mx_scale_relayout",
                     "bsmma_reserve_workspace", "bsmma_device_status", "bsmma_set_wait_limit_ns",
                     "bsmma_set_dense_variant", "bsmma_set_grouped_tile_width",
                     "grouped_bf16_gemm", "bsmma_set_grouped_variant",
                     "bsmma_probe_wait_timeout", "mx_quantize", "fp8_group_quantize",
                     "fp8_block_quantize", "mx_gemm_bias_act", "mx_gemm_tiled_bias_act",
                     "bsmma_autotune_configure", "moe_route", "moe_route_backward", "moe_plan",
                     "moe_combine", "moe_combine_backward", "int8_quantize", "int8_gemm",
                     "grouped_int8_gemm", "moe_step", "branch_enter", "branch_leave", "branch_enter_backward",
                     "branch_leave_backward", "dropout"):
            getattr(lib, name).restype = i32
        _lib = lib
        return lib


def _stream(stream=None) -> int:
    if stream is None:
        # the handle of torch.cuda.current_stream() without building the Stream object,
        # which costs as much host time as a kernel launch
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _check(code: int, where: str):
    if code != 0:
        raise BsmmaError(code, where)


def mx_gemm(A, sA, B, sB, layout="NT", a_fmt="e4m3", b_fmt="e4m3", out=None, M=None, N=None,
            K=None, stream=None, tiled=False, bias=None, act="none"):
    """D = op(A) . op(B)^T in BF16 for MX operands (see ``mx_gemm`` in bsmma.h); with a
    BF16 ``bias`` [N] and/or ``act`` ('relu', 'gelu', 'silu') the output stage computes
    act(acc + bias) before rounding (``mx_gemm_bias_act``).

    A, B: 1-byte tensors in the storage layout of `layout` (FP4 packed, NT only);
    sA [M, K/32], sB [N, K/32] uint8 E8M0 codes (or tiled buffers when
    ``tiled=True``).  Sizes are taken from the shapes unless given.
    """
    fp4 = a_fmt == "e2m1"
    if M is None or N is None or K is None:
        if layout == "NT":
            M, kk = A.shape
            N = B.shape[0]
        elif layout == "NN":
            M, kk = A.shape
            N = B.shape[1]
        else:
            kk, M = A.shape
            N = B.shape[1]
        K = kk * 2 if fp4 else kk
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    if bias is not None or act != "none":
        fn = load().mx_gemm_tiled_bias_act if tiled else load().mx_gemm_bias_act
        if bias is not None and (bias.dtype != torch.bfloat16 or bias.numel() != N):
            raise ValueError("bias must be a BF16 vector of N values")
        _check(fn(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(bias), ACTIVATIONS[act], _ptr(out),
                  M, N, K, LAYOUTS[layout], FORMATS[a_fmt], FORMATS[b_fmt], _stream(stream)),
               "mx_gemm_bias_act")
        return out
    fn = load().mx_gemm_tiled if tiled else load().mx_gemm
    _check(fn(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(out), M, N, K, LAYOUTS[layout],
              FORMATS[a_fmt], FORMATS[b_fmt], _stream(stream)),
           "mx_gemm_tiled" if tiled else "mx_gemm")
    return out


def mx_gemm_noalloc(A, sA, B, sB, layout="NT", a_fmt="e4m3", b_fmt="e4m3", out=None, M=None,
                    N=None, K=None, stream=None):
    """``mx_gemm`` without any device allocation (scales go to the library's fixed
    16 MiB array; see ``mx_gemm_noalloc`` in bsmma.h).  ``out`` must be given."""
    if out is None:
        raise ValueError("mx_gemm_noalloc allocates nothing: pass out=")
    if M is None or N is None or K is None:
        raise ValueError("mx_gemm_noalloc: pass M, N and K")
    _check(load().mx_gemm_noalloc(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(out), M, N, K,
                                  LAYOUTS[layout], FORMATS[a_fmt], FORMATS[b_fmt],
                                  _stream(stream)), "mx_gemm_noalloc")
    return out


def mx_gemm_tiled(A, sA_tiled, B, sB_tiled, layout="NT", a_fmt="e4m3", b_fmt="e4m3", out=None,
                  M=None, N=None, K=None, stream=None, bias=None, act="none"):
    """``mx_gemm`` with scales already relayouted by :func:`mx_scale_relayout`."""
    return mx_gemm(A, sA_tiled, B, sB_tiled, layout, a_fmt, b_fmt, out, M, N, K, stream,
                   tiled=True, bias=bias, act=act)


def grouped_fp8_pack_weights(W, out=None, stream=None):
    """W [G, N, K] E4M3 codes -> the packed layout of ``grouped_fp8_gemm(..., packed=True)``
    (same shape and size; see ``grouped_fp8_pack_weights`` in bsmma.h)."""
    G, N, K = W.shape
    if out is None:
        out = torch.empty_like(W)
    _check(load().grouped_fp8_pack_weights(_ptr(W), G, N, K, _ptr(out), _stream(stream)),
           "grouped_fp8_pack_weights")
    return out


def grouped_fp8_gemm(X, sX, W, sW, m_sizes, out=None, stream=None, packed=False):
    """Grouped groupwise FP8 GEMM (see ``grouped_fp8_gemm`` in bsmma.h).

    X [total_M, K] E4M3 codes, sX float32 per-group block layout, W [G, N, K] E4M3 (or,
    with ``packed=True``, the output of grouped_fp8_pack_weights), sW float32
    [G, N/128, K/128], m_sizes int64 [G] on the device.
    """
    total_M, K = X.shape
    G, N, _ = W.shape
    if m_sizes.dtype != torch.int64 or m_sizes.numel() != G or m_sizes.dim() != 1:
        raise ValueError("m_sizes must be a 1-D int64 tensor of length G")
    if out is None:
        out = torch.empty((total_M, N), dtype=torch.bfloat16, device=W.device)
    fn = load().grouped_fp8_gemm_packed if packed else load().grouped_fp8_gemm
    _check(fn(_ptr(X) if total_M else None, _ptr(sX) if total_M else None,
              _ptr(W), _ptr(sW), _ptr(out) if total_M else None,
              _ptr(m_sizes), total_M, G, N, K, _stream(stream)),
           "grouped_fp8_gemm_packed" if packed else "grouped_fp8_gemm")
    return out


def grouped_bf16_gemm(X, W, m_sizes, out=None, stream=None):
    """Grouped BF16 GEMM (see ``grouped_bf16_gemm`` in bsmma.h): D[r] = X[r] . W[g(r)]^T.

    X [total_M, K] and W [G, N, K] BF16 tensors (or int16/uint16 holding BF16 bit
    patterns), m_sizes int64 [G] on the device; returns D [total_M, N] BF16.
    """
    total_M, K = X.shape
    G, N, _ = W.shape
    if m_sizes.dtype != torch.int64 or m_sizes.numel() != G or m_sizes.dim() != 1:
        raise ValueError("m_sizes must be a 1-D int64 tensor of length G")
    if X.element_size() != 2 or W.element_size() != 2:
        raise ValueError("X and W must hold 16-bit BF16 values")
    if out is None:
        out = torch.empty((total_M, N), dtype=torch.bfloat16, device=W.device)
    _check(load().grouped_bf16_gemm(_ptr(X) if total_M else None, _ptr(W),
                                    _ptr(out) if total_M else None, _ptr(m_sizes), total_M, G,
                                    N, K, _stream(stream)), "grouped_bf16_gemm")
    return out


def mx_scale_tiled_bytes(rows: int, kblocks: int, role="A") -> int:
    return int(load().mx_scale_tiled_bytes(rows, kblocks, ROLES[role]))


def mx_scale_relayout(s_plain, role="A", out=None, stream=None):
    """Plain E8M0 scales [rows, kblocks] -> the tiled layout of `role` ('A': scales
    of op(A) rows, 'B': scales of op(B) rows), as a flat uint8 tensor."""
    rows, kblocks = s_plain.shape
    if out is None:
        out = torch.empty(mx_scale_tiled_bytes(rows, kblocks, role), dtype=torch.uint8,
                          device=s_plain.device)
    _check(load().mx_scale_relayout(_ptr(s_plain), rows, kblocks, ROLES[role], _ptr(out),
                                    _stream(stream)), "mx_scale_relayout")
    return out


def reserve_workspace(nbytes: int, stream=None):
    _check(load().bsmma_reserve_workspace(nbytes, _stream(stream)), "bsmma_reserve_workspace")


def device_status(stream=None) -> int:
    """Synchronises the stream; returns and clears the latched device status code."""
    return int(load().bsmma_device_status(_stream(stream)))


def set_wait_limit_ns(ns: int):
    _check(load().bsmma_set_wait_limit_ns(int(ns)), "bsmma_set_wait_limit_ns")


def set_dense_variant(variant: int):
    """0 automatic (SM-pair MMAs), 1 single-CTA tiles, 3 SM-pair MMAs."""
    _check(load().bsmma_set_dense_variant(int(variant)), "bsmma_set_dense_variant")


def set_grouped_tile_width(width: int):
    """0 automatic, 128 or 256 columns per grouped tile."""
    _check(load().bsmma_set_grouped_tile_width(int(width)), "bsmma_set_grouped_tile_width")


def set_grouped_variant(variant: int):
    """Grouped BF16 tiles: 0 automatic, 1 one CTA per tile, 3 SM-pair 256 x 256 tiles."""
    _check(load().bsmma_set_grouped_variant(int(variant)), "bsmma_set_grouped_variant")


def set_int8_variant(tile: int, fp16_tokens: bool = False):
    """INT8 products: 0 automatic, 1 few-row kernel, or SM-pair tiles of 32, 64, 128 or 256
    rows, or of 192 or 256 rows widened to FP16 beforehand (``fp16_tokens``)."""
    _check(load().bsmma_set_int8_variant(int(tile), int(bool(fp16_tokens))), "bsmma_set_int8_variant")


def launch_count() -> int:
    return int(load().bsmma_launch_count())


def status_string(code: int) -> str:
    return load().bsmma_status_string(int(code)).decode()


def probe_wait_timeout(limit_ns: int, stream=None) -> int:
    return int(load().bsmma_probe_wait_timeout(int(limit_ns), _stream(stream)))


DTYPES = {torch.bfloat16: 0, torch.float32: 1}


def _dtype_code(t) -> int:
    if t.dtype not in DTYPES:
        raise ValueError("quantiser inputs are bfloat16 or float32")
    return DTYPES[t.dtype]


def mx_quantize(x, fmt="e4m3", colwise=False, codes=None, scales=None, stream=None):
    """MX quantisation of x[rows, cols] (BF16 or FP32) -> (codes, scales); see
    ``mx_quantize`` in bsmma.h.  Rowwise: codes [rows, cols] ([rows, cols/2] for e2m1),
    scales [rows, cols/32].  Columnwise: codes [rows, cols], scales [cols, rows/32]."""
    rows, cols = x.shape
    if codes is None:
        codes = torch.empty((rows, cols // 2 if fmt == "e2m1" else cols), dtype=torch.uint8,
                            device=x.device)
    if scales is None:
        shape = (cols, rows // 32) if colwise else (rows, cols // 32)
        scales = torch.empty(shape, dtype=torch.uint8, device=x.device)
    _check(load().mx_quantize(_ptr(x), _dtype_code(x), rows, cols, FORMATS[fmt], int(bool(colwise)),
                              _ptr(codes), _ptr(scales), _stream(stream)), "mx_quantize")
    return codes, scales


def fp8_group_quantize(x, m_sizes, codes=None, scales=None, stream=None):
    """Groupwise E4M3 quantisation of activations x[total_M, K] over 1x128 blocks ->
    (codes [total_M, K], scales float32 [total_M * K/128] in the per-group block layout);
    m_sizes: int64 [G] on the device.  See ``fp8_group_quantize`` in bsmma.h."""
    total_M, K = x.shape
    if codes is None:
        codes = torch.empty((total_M, K), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(total_M * (K // 128), dtype=torch.float32, device=x.device)
    _check(load().fp8_group_quantize(_ptr(x) if total_M else None, _dtype_code(x), total_M, K,
                                     _ptr(m_sizes), m_sizes.numel(),
                                     _ptr(codes) if total_M else None,
                                     _ptr(scales) if total_M else None, _stream(stream)),
           "fp8_group_quantize")
    return codes, scales


def fp8_block_quantize(w, codes=None, scales=None, stream=None):
    """Blockwise E4M3 quantisation of weights w[G, N, K] over 128x128 blocks ->
    (codes [G, N, K], scales float32 [G, N/128, K/128]).  See ``fp8_block_quantize``."""
    G, N, K = w.shape
    if codes is None:
        codes = torch.empty((G, N, K), dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty((G, N // 128, K // 128), dtype=torch.float32, device=w.device)
    _check(load().fp8_block_quantize(_ptr(w), _dtype_code(w), G, N, K, _ptr(codes), _ptr(scales),
                                     _stream(stream)), "fp8_block_quantize")
    return codes, scales


SCORES = {"softmax": 0, "sigmoid": 1}


def _dtype_of(t, what: str) -> int:
    if t.dtype not in DTYPES:
        raise ValueError(f"{what} must be bfloat16 or float32")
    return DTYPES[t.dtype]


def _expect(t, dtype, shape, what: str):
    """`t` (None passes) has this dtype and shape (a tuple)."""
    if t is not None and (t.dtype != dtype or t.shape != shape):
        raise ValueError(f"{what} must be {dtype} of shape {shape}, "
                         f"not {t.dtype} of {tuple(t.shape)}")


def _output(t, dtype, shape, like, what: str):
    """The output to write: `t` if it has this dtype and shape (a tuple), or a new one."""
    if t is None:
        # empty_like takes half the host time of an empty with its shape and device spelt out
        if like.shape == shape:
            return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)
        return torch.empty(shape, dtype=dtype, device=like.device)
    _expect(t, dtype, shape, what)
    return t


def moe_route(logits, k, score="softmax", bias=None, groups=1, topk_groups=1, group_top=1,
              renormalize=True, scale=1.0, ids=None, weights=None, stream=None):
    """Chooses k experts a token from logits [T, E] (BF16 or FP32) -> (ids int32 [T, k],
    weights float32 [T, k]); see ``moe_route`` in bsmma.h.  ``score``: 'softmax' or
    'sigmoid'; ``bias``: float32 [E], added to the scores for the choice alone."""
    T, E = logits.shape
    _expect(bias, torch.float32, (E,), "bias")
    ids = _output(ids, torch.int32, (T, k), logits, "ids")
    weights = _output(weights, torch.float32, (T, k), logits, "weights")
    _check(load().moe_route(_ptr(logits), _dtype_of(logits, "logits"), T, E, k, SCORES[score],
                            _ptr(bias), groups, topk_groups, group_top, int(bool(renormalize)),
                            scale, _ptr(ids), _ptr(weights), _stream(stream)), "moe_route")
    return ids, weights


def moe_route_backward(logits, ids, dweights, score="softmax", renormalize=True, scale=1.0,
                       dlogits=None, stream=None):
    """The gradient of :func:`moe_route`'s weights in its logits, the choice held fixed ->
    dlogits [T, E] of the logits' dtype."""
    T, E = logits.shape
    k = ids.shape[1]
    _expect(ids, torch.int32, (T, k), "ids")
    _expect(dweights, torch.float32, (T, k), "dweights")
    dlogits = _output(dlogits, logits.dtype, (T, E), logits, "dlogits")
    _check(load().moe_route_backward(_ptr(logits), _dtype_of(logits, "logits"), T, E, k,
                                     SCORES[score], int(bool(renormalize)), scale, _ptr(ids),
                                     _ptr(dweights), _ptr(dlogits), _stream(stream)),
           "moe_route_backward")
    return dlogits


def moe_plan_workspace_bytes(T: int, k: int, E: int) -> int:
    """Workspace of :func:`moe_plan` (reserve it before a capture)."""
    return int(load().moe_plan_workspace_bytes(T, k, E))


def moe_plan(ids, experts, m_sizes=None, src=None, pos=None, stream=None):
    """The expert order of the slots ids int32 [T, k] -> (m_sizes int64 [experts], src int32
    [T * k], pos int32 [T, k]); see ``moe_plan`` in bsmma.h."""
    T, k = ids.shape
    _expect(ids, torch.int32, (T, k), "ids")
    m_sizes = _output(m_sizes, torch.int64, (experts,), ids, "m_sizes")
    src = _output(src, torch.int32, (T * k,), ids, "src")
    pos = _output(pos, torch.int32, (T, k), ids, "pos")
    _check(load().moe_plan(_ptr(ids), T, k, experts, _ptr(m_sizes), _ptr(src), _ptr(pos),
                           _stream(stream)), "moe_plan")
    return m_sizes, src, pos


def moe_combine(Y, pos, weights=None, out=None, stream=None):
    """out[t] = sum_j weights[t, j] * Y[pos[t, j]] -> [T, H] of Y's dtype (BF16 or FP32);
    without weights, the plain sum.  See ``moe_combine`` in bsmma.h."""
    R, H = Y.shape
    T, k = pos.shape
    _expect(pos, torch.int32, (T, k), "pos")
    _expect(weights, torch.float32, (T, k), "weights")
    out = _output(out, Y.dtype, (T, H), Y, "out")
    _check(load().moe_combine(_ptr(Y), _dtype_of(Y, "Y"), R, H, _ptr(pos), _ptr(weights), T, k,
                              _ptr(out), _stream(stream)), "moe_combine")
    return out


def moe_combine_backward(dout, Y, src, pos, weights=None, dY=None, dweights=None, stream=None):
    """The gradients of :func:`moe_combine` -> (dY [T * k, H], dweights float32 [T, k]);
    without weights only dY (dweights None), and Y may be None."""
    T, H = dout.shape
    k = pos.shape[1]
    _expect(pos, torch.int32, (T, k), "pos")
    _expect(src, torch.int32, (T * k,), "src")
    _expect(weights, torch.float32, (T, k), "weights")
    _expect(Y, dout.dtype, (T * k, H), "Y")
    if (weights is not None or dweights is not None) and Y is None:
        raise ValueError("Y is needed for the gradient of the weights")
    dY = _output(dY, dout.dtype, (T * k, H), dout, "dY")
    if weights is not None or dweights is not None:
        dweights = _output(dweights, torch.float32, (T, k), dout, "dweights")
    _check(load().moe_combine_backward(_ptr(dout), _dtype_of(dout, "dout"), H, _ptr(Y), _ptr(src),
                                       _ptr(pos), _ptr(weights), T, k, _ptr(dY), _ptr(dweights),
                                       _stream(stream)), "moe_combine_backward")
    return dY, dweights


def int8_quantize(x, src=None, k=1, codes=None, scales=None, stream=None):
    """Symmetric INT8 quantisation by row of x [rows, K] (BF16 or FP32) -> (codes int8,
    scales float32).  With ``src`` (moe_plan's, int32) output row r is row src[r] // k of x,
    or zeros where src[r] < 0.  See ``int8_quantize`` in bsmma.h."""
    x_rows, K = x.shape
    rows = x_rows if src is None else src.numel()
    _expect(src, torch.int32, (rows,), "src")
    codes = _output(codes, torch.int8, (rows, K), x, "codes")
    scales = _output(scales, torch.float32, (rows,), x, "scales")
    _check(load().int8_quantize(_ptr(x), _dtype_of(x, "x"), x_rows, K, _ptr(src), k, rows,
                                _ptr(codes), _ptr(scales), _stream(stream)), "int8_quantize")
    return codes, scales


def int8_gemm(A, sA, B, sB, bias=None, out=None, dtype=torch.bfloat16, stream=None):
    """D[m, n] = sA[m] * sB[n] * (A . B^T)[m, n] (+ bias[n]) for A int8 [M, K], B int8 [N, K],
    in ``dtype`` (BF16 or FP32).  See ``int8_gemm`` in bsmma.h."""
    M, K = A.shape
    N = B.shape[0]
    _expect(A, torch.int8, (M, K), "A")
    _expect(B, torch.int8, (N, K), "B")
    _expect(sA, torch.float32, (M,), "sA")
    _expect(sB, torch.float32, (N,), "sB")
    _expect(bias, torch.bfloat16, (N,), "bias")
    out = _output(out, dtype if out is None else out.dtype, (M, N), A, "out")
    _check(load().int8_gemm(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(bias), _ptr(out),
                            _dtype_of(out, "out"), M, N, K, _stream(stream)), "int8_gemm")
    return out


def grouped_int8_gemm(X, sX, W, sW, m_sizes, out=None, dtype=torch.bfloat16, stream=None):
    """:func:`int8_gemm` for each expert's rows: X int8 [total_M, K], sX float32 [total_M],
    W int8 [G, N, K], sW float32 [G, N], m_sizes int64 [G] on the device (it may sum to less
    than total_M; the rows past it are left as they are).  See ``grouped_int8_gemm``."""
    total_M, K = X.shape
    G, N, _ = W.shape
    _expect(X, torch.int8, (total_M, K), "X")
    _expect(W, torch.int8, (G, N, K), "W")
    _expect(sX, torch.float32, (total_M,), "sX")
    _expect(sW, torch.float32, (G, N), "sW")
    _expect(m_sizes, torch.int64, (G,), "m_sizes")
    out = _output(out, dtype if out is None else out.dtype, (total_M, N), W, "out")
    _check(load().grouped_int8_gemm(_ptr(X) if total_M else None, _ptr(sX) if total_M else None,
                                    _ptr(W), _ptr(sW), _ptr(out) if total_M else None,
                                    _dtype_of(out, "out"), _ptr(m_sizes), total_M, G, N, K,
                                    _stream(stream)), "grouped_int8_gemm")
    return out


def _here(*tensors):
    """The addresses of tensors (None: none), all contiguous and on the current device, whose stream and
    kernels a call uses."""
    here, at = None, []
    for t in tensors:
        if t is None:
            at.append(None)
            continue
        device = t.get_device()
        if here is None and device >= 0:
            here = torch._C._cuda_getDevice()
        if device != here:
            raise ValueError("expected a CUDA tensor on the current device")
        if not t.is_contiguous():
            raise ValueError("expected a contiguous tensor")
        at.append(t.data_ptr())
    return at


NORMS = {"none": 0, "rms": 1, "layer": 2}
OPERANDS = {"bf16": 0, "f32": 1, "int8": 2, "e4m3": 3, "e5m2": 4, "e2m1": 5}
_OPERAND_OF = {torch.bfloat16: "bf16", torch.float32: "f32"}


def _operand(fmt, T, H, like, out, scales):
    """Output and scales (None without) of a [T, H] operand, given or new."""
    if fmt in ("bf16", "f32"):
        if scales is not None:
            raise ValueError(f"{fmt} rows have no scales")
        return _output(out, torch.bfloat16 if fmt == "bf16" else torch.float32, (T, H), like, "out"), None
    if fmt == "int8":
        return (_output(out, torch.int8, (T, H), like, "codes"),
                _output(scales, torch.float32, (T,), like, "scales"))
    return (_output(out, torch.uint8, (T, H // 2 if fmt == "e2m1" else H), like, "codes"),
            _output(scales, torch.uint8, (T, H // 32), like, "scales"))


def _rng(rng, p: float):
    _expect(rng, torch.int64, (2,), "rng")
    if rng is None and p > 0:
        raise ValueError("dropout needs rng, an int64 tensor (seed, offset) on the device")


def _gate(gate, gate_rows, y):
    """The rows that share a row of the gate (all of them unless said).  No rows need no gate, but the
    one that all of them would share may be there."""
    T, H = y.shape
    rows = max(T, 1) if gate_rows is None else gate_rows
    if rows < 1:
        raise ValueError("gate_rows must be at least 1")
    _expect(gate, y.dtype, (1 if T == 0 and gate.shape == (1, H) else -(-T // rows), H), "gate")
    return rows


def branch_enter(x, weight=None, bias=None, norm="rms", eps=1e-6, fmt=None, out=None, scales=None,
                 stream=None):
    """The norm before a block: n(x) * weight + bias for x [T, H] (BF16 or FP32; weight and bias
    float32 [H]), ``norm`` 'rms' or 'layer'.  ``fmt`` None (x's dtype), 'bf16' or 'f32' ->
    [T, H]; 'int8' -> (codes, scales) as :func:`int8_quantize`'s, 'e4m3', 'e5m2', 'e2m1' -> as
    :func:`mx_quantize`'s (rowwise).  See ``branch_enter`` in bsmma.h."""
    T, H = x.shape
    dtype = _dtype_of(x, "x")
    fmt = fmt or _OPERAND_OF[x.dtype]
    if weight is not None:
        _expect(weight, torch.float32, (H,), "weight")
    if bias is not None:
        _expect(bias, torch.float32, (H,), "bias")
    out, scales = _operand(fmt, T, H, x, out, scales)
    x_at, w_at, b_at, out_at, scales_at = _here(x, weight, bias, out, scales)
    _check(load().branch_enter(x_at, dtype, T, H, NORMS[norm], eps, w_at, b_at, OPERANDS[fmt], out_at, scales_at,
                               _stream(stream)), "branch_enter")
    return out if scales is None else (out, scales)


def branch_enter_backward(dh, x, weight=None, norm="rms", eps=1e-6, dres=None, bias=False, dx=None,
                          stream=None):
    """The gradients of :func:`branch_enter` for dh [T, H] (x's dtype, or BF16) -> (dx, dweight,
    dbias).  ``dres``: a gradient of x to add to dx (what reached the stream past the branch);
    dweight float32 [H], None without a weight; dbias None unless ``bias``."""
    T, H = x.shape
    h_dtype, x_dtype = _dtype_of(dh, "dh"), _dtype_of(x, "x")
    _expect(dh, dh.dtype, (T, H), "dh")
    if weight is not None:
        _expect(weight, torch.float32, (H,), "weight")
    if dres is not None:
        _expect(dres, x.dtype, (T, H), "dres")
    dx = _output(dx, x.dtype, (T, H), x, "dx")
    dweight = None if weight is None else torch.empty_like(weight)
    dbias = None
    if bias:
        dbias = torch.empty(H, dtype=torch.float32, device=x.device) if weight is None else torch.empty_like(weight)
    dh_at, x_at, w_at, *rest = _here(dh, x, weight, dres, dx, dweight, dbias)
    _check(load().branch_enter_backward(dh_at, h_dtype, x_at, x_dtype, T, H, NORMS[norm], eps, w_at, *rest,
                                        _stream(stream)), "branch_enter_backward")
    return dx, dweight, dbias


def branch_leave(x, y, weight=None, bias=None, norm="none", eps=1e-6, gate=None, gate_rows=None,
                 x_scale=1.0, y_scale=1.0, p=0.0, rng=None, next_norm="none", next_weight=None,
                 next_bias=None, next_eps=1e-6, fmt=None, out=None, next_out=None, next_scales=None,
                 stream=None):
    """The step after a block: out = x_scale * x + y_scale * gate * drop(n(y) * weight + bias),
    [T, H] of x's dtype; y of x's dtype, or BF16 beside an FP32 x.  ``gate`` (y's dtype) has a row for
    each ``gate_rows`` rows (None: one row for all).  ``p``, ``rng``: as :func:`dropout`.  With
    ``next_norm`` also the following block's :func:`branch_enter` of out, in ``fmt`` (None: y's
    dtype) -> (out, h) or (out, codes, scales).  out may be x.  See ``branch_leave`` in bsmma.h."""
    T, H = x.shape
    x_dtype, y_dtype = _dtype_of(x, "x"), _dtype_of(y, "y")
    _expect(y, y.dtype, (T, H), "y")
    if weight is not None:
        _expect(weight, torch.float32, (H,), "weight")
    if bias is not None:
        _expect(bias, torch.float32, (H,), "bias")
    if next_weight is not None:
        _expect(next_weight, torch.float32, (H,), "next_weight")
    if next_bias is not None:
        _expect(next_bias, torch.float32, (H,), "next_bias")
    gate_rows = 1 if gate is None else _gate(gate, gate_rows, y)
    _rng(rng, p)
    out = _output(out, x.dtype, (T, H), x, "out")
    fmt = fmt or _OPERAND_OF[y.dtype]
    if next_norm != "none":
        next_out, next_scales = _operand(fmt, T, H, x, next_out, next_scales)
    x_at, y_at, w_at, b_at, gate_at, rng_at, out_at, nw_at, nb_at, no_at, ns_at = _here(
        x, y, weight, bias, gate, rng, out, next_weight, next_bias, next_out, next_scales)
    _check(load().branch_leave(x_at, x_dtype, y_at, y_dtype, T, H, NORMS[norm], eps, w_at, b_at, gate_at, gate_rows,
                               x_scale, y_scale, p, rng_at, out_at, NORMS[next_norm], next_eps, nw_at, nb_at,
                               OPERANDS[fmt], no_at, ns_at, _stream(stream)), "branch_leave")
    if next_norm == "none":
        return out
    return (out, next_out) if next_scales is None else (out, next_out, next_scales)


def branch_leave_backward(dout, y, weight=None, bias=None, norm="none", eps=1e-6, gate=None,
                          gate_rows=None, x_scale=1.0, y_scale=1.0, p=0.0, rng=None, dy=None, dx=None,
                          stream=None):
    """The gradients of :func:`branch_leave` (without its next norm) for dout [T, H] and the forward
    call's arguments -> (dy, dx, dweight, dbias, dgate): dy of y's dtype; dx = x_scale * dout, dout itself
    where x_scale is 1; the others float32, None for what was not given.  ``rng`` holds what it
    held in the forward call."""
    T, H = y.shape
    x_dtype, y_dtype = _dtype_of(dout, "dout"), _dtype_of(y, "y")
    _expect(dout, dout.dtype, (T, H), "dout")
    if weight is not None:
        _expect(weight, torch.float32, (H,), "weight")
    if bias is not None:
        _expect(bias, torch.float32, (H,), "bias")
    gate_rows = 1 if gate is None else _gate(gate, gate_rows, y)
    _rng(rng, p)
    dy = _output(dy, y.dtype, (T, H), y, "dy")
    if x_scale != 1 or dx is not None:
        dx = _output(dx, dout.dtype, (T, H), y, "dx")
    dweight = None if weight is None else torch.empty_like(weight)
    dbias = None if bias is None else torch.empty_like(bias)
    dgate = None if gate is None else torch.empty_like(gate, dtype=torch.float32)
    if T == 0 and gate is not None:
        dgate.zero_()
    dout_at, y_at, w_at, b_at, gate_at, rng_at, *grads = _here(dout, y, weight, bias, gate, rng, dy, dx, dweight, dbias,
                                                               dgate)
    _check(load().branch_leave_backward(dout_at, x_dtype, y_at, y_dtype, T, H, NORMS[norm], eps, w_at, b_at, gate_at,
                                        gate_rows, x_scale, y_scale, p, rng_at, *grads, _stream(stream)),
           "branch_leave_backward")
    return dy, dout if dx is None else dx, dweight, dbias, dgate


def moe_step_workspace_bytes(T: int, k: int, H: int, F: int) -> int:
    """Workspace of :func:`moe_step` (reserve it before a capture)."""
    return int(load().moe_step_workspace_bytes(T, k, H, F))


def moe_step(x, ids, weights, w_in, w_out, s_in=None, s_out=None, fmt="bf16", act="silu", out=None,
             stream=None):
    """out[t] = sum_j weights[t, j] * W2[e] (act(Wg[e] x[t]) * (Wu[e] x[t])), e = ids[t, j], for a few
    tokens (T <= 32, T * k <= 1024) x [T, H] BF16; ids int32 and weights float32 [T, k] from
    :func:`moe_route`.  w_in [E, 2F, H] has the gate's rows first, w_out is [E, H, F]; ``fmt``:
    'bf16'; 'int8' with float32 scales [E, 2F] and [E, H]; 'e4m3', 'e5m2' or 'e2m1' (uint8 codes, E2M1
    packed) with uint8 E8M0 scales [E, 2F, H/32] and [E, H, F/32].  See ``moe_step`` in bsmma.h."""
    T, H = x.shape
    k = ids.shape[1]
    E, F = w_in.shape[0], w_in.shape[1] // 2
    pack = 2 if fmt == "e2m1" else 1
    dtype = torch.bfloat16 if fmt == "bf16" else torch.int8 if fmt == "int8" else torch.uint8
    _expect(x, torch.bfloat16, (T, H), "x")
    _expect(ids, torch.int32, (T, k), "ids")
    _expect(weights, torch.float32, (T, k), "weights")
    _expect(w_in, dtype, (E, 2 * F, H // pack), "w_in")
    _expect(w_out, dtype, (E, H, F // pack), "w_out")
    if (fmt == "bf16") != (s_in is None) or (fmt == "bf16") != (s_out is None):
        raise ValueError("s_in and s_out go with codes, not with BF16 weights")
    if fmt == "int8":
        _expect(s_in, torch.float32, (E, 2 * F), "s_in")
        _expect(s_out, torch.float32, (E, H), "s_out")
    else:
        _expect(s_in, torch.uint8, (E, 2 * F, H // 32), "s_in")
        _expect(s_out, torch.uint8, (E, H, F // 32), "s_out")
    out = _output(out, torch.bfloat16, (T, H), x, "out")
    x_at, ids_at, weights_at, *experts, out_at = _here(x, ids, weights, w_in, s_in, w_out, s_out, out)
    _check(load().moe_step(x_at, T, H, ids_at, weights_at, k, E, F, OPERANDS[fmt], *experts, ACTIVATIONS[act], out_at,
                           _stream(stream)), "moe_step")
    return out


def branch_backward_workspace_bytes(T: int, H: int) -> int:
    """Workspace of the branch's gradients (reserve it before a capture)."""
    return int(load().branch_backward_workspace_bytes(T, H))


def dropout(x, p, rng, out=None, stream=None):
    """x with each value dropped with probability p (rounded to 2^-16), the others divided by 1 - p;
    ``rng`` int64 (seed, offset) on the device.  Its gradient is the same call on the output's.
    out may be x.  See ``dropout`` in bsmma.h."""
    _rng(rng, p)
    dtype = _dtype_of(x, "x")
    out = _output(out, x.dtype, x.shape, x, "out")
    x_at, rng_at, out_at = _here(x, rng, out)
    _check(load().dropout(x_at, dtype, x.numel(), p, rng_at, out_at, _stream(stream)), "dropout")
    return out


def autotune_configure(enable=-1, cache_path=None):
    """Turns tile autotuning on (1) / off (0) / to the environment's BSMMA_AUTOTUNE (-1)
    and selects its cache file (None: BSMMA_AUTOTUNE_CACHE or the user cache directory);
    see ``bsmma_autotune_configure`` in bsmma.h."""
    path = None if cache_path is None else os.fsencode(cache_path)
    _check(load().bsmma_autotune_configure(int(enable), path), "bsmma_autotune_configure")


def autotune_lookup(key: str) -> int:
    """The stored choice for a shape-class key, or -1."""
    return int(load().bsmma_autotune_lookup(key.encode()))
