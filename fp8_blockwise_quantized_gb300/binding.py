"""Python binding of the C ABI in include/gmm.h (argument marshalling only).

Every function named like a C entry point passes its tensors' device
pointers, the sizes and the stream straight to the library; every step of the
computation runs in the library's CUDA kernels.  The convenience wrappers
below (``quantize_lhs``, ``fp8_fwd``, ...) additionally allocate the outputs
with torch, which here is only the device-memory allocator.  They take a
``stream`` (a torch stream or a raw handle; the current stream by default), on
which they both allocate and launch.

The library must have been built (``fp8_blockwise_quantized_gb300.build``);
without it every call raises: there is no fallback.
"""
from __future__ import annotations

import array
import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgmm_gb300.so")

GMM_OK = 0
GMM_ERR_GROUP_SIZES = 6
GMM_ERR_TIMEOUT = 7
STATUS_NAMES = {0: "GMM_OK", 1: "GMM_ERR_NULL", 2: "GMM_ERR_SHAPE", 3: "GMM_ERR_ALIGN",
                4: "GMM_ERR_UNSUPPORTED", 5: "GMM_ERR_CUDA", 6: "GMM_ERR_GROUP_SIZES",
                7: "GMM_ERR_TIMEOUT", 8: "GMM_ERR_WORKSPACE"}

EXPORTED = ["gmm_status_string", "gmm_last_cuda_error", "gmm_workspace_bytes", "gmm_tiles_offset",
            "gmm_group_metadata", "gmm_quantize_lhs", "gmm_quantize_rhs", "gmm_fp8_fwd",
            "gmm_bf16_fwd", "tgmm_bf16", "gmm_get_device_status", "gmm_fp8_fwd_noalloc",
            "gmm_bf16_dgrad", "gmm_fp8_fwd_swiglu_quant", "gmm_selftest_wait_timeout", "gmm_fp8_fwd_tiled",
            "gmm_fp8_fwd_swiglu_quant_tiled", "gmm_quantize_rhs_w4", "gmm_fp8_w4_fwd",
            "gmm_fp8_w4_fwd_swiglu_quant", "tgmm_bf16_tiled", "gmm_bf16_swiglu_fwd", "gmm_bf16_swiglu_bwd",
            "tgmm_fp8_ckpt", "tgmm_fp8_ckpt_scratch_bytes", "gmm_mx4_quantize_lhs", "gmm_mx4_quantize_rhs", "gmm_mx4_fwd",
            "gmm_mx4_fwd_swiglu_quant", "gmm_route", "gmm_route_bwd", "gmm_sort_rows_scratch_bytes", "gmm_sort_rows",
            "gmm_gather_rows", "gmm_gather_quantize", "gmm_combine_rows", "gmm_combine_rows_bwd", "gmm_norm_join",
            "gmm_norm_join_bwd_scratch_bytes", "gmm_norm_join_bwd", "gmm_clip_grads_scratch_bytes", "gmm_clip_grads"]


class TileConfig(ctypes.Structure):
    """gmm_fp8_tile_config: bn (128 | 256), ctas (1 .. SMs), unit_order
    (1 row-tile major, 2 column-block major), cta_group (1 one CTA per
    128-row tile, 2 CTA pairs on 256-row tiles), stages (operand ring
    slots), tmem_bufs (TMEM partial buffers); 0 keeps a field's default.
    A shorter tuple leaves the remaining fields 0."""
    _fields_ = [("bn", ctypes.c_int), ("ctas", ctypes.c_int), ("unit_order", ctypes.c_int),
                ("cta_group", ctypes.c_int), ("stages", ctypes.c_int), ("tmem_bufs", ctypes.c_int)]

    def astuple(self):
        return (self.bn, self.ctas, self.unit_order, self.cta_group, self.stages, self.tmem_bufs)


class TgmmConfig(ctypes.Structure):
    """gmm_tgmm_tile_config: stages (4..6), claim_ahead (1..12), max_batch
    (1..4); 0 keeps a field's default.  A shorter tuple leaves the rest 0."""
    _fields_ = [("stages", ctypes.c_int), ("claim_ahead", ctypes.c_int), ("max_batch", ctypes.c_int)]

    def astuple(self):
        return (self.stages, self.claim_ahead, self.max_batch)


class GmmError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = load()
        msg = lib.gmm_status_string(status).decode()
        if status == 5:
            msg += f" ({lib.gmm_last_cuda_error().decode()})"
        super().__init__(f"{where}: {msg}")
        self.status = status


_lib = None


def load():
    """Load the shared library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                           "(run fp8_blockwise_quantized_gb300.build.build())")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    lib.gmm_status_string.restype = ctypes.c_char_p
    lib.gmm_status_string.argtypes = [I]
    lib.gmm_last_cuda_error.restype = ctypes.c_char_p
    lib.gmm_last_cuda_error.argtypes = []
    lib.gmm_workspace_bytes.restype = SZ
    lib.gmm_workspace_bytes.argtypes = [I, I64]
    lib.gmm_tiles_offset.restype = SZ
    lib.gmm_tiles_offset.argtypes = [I]
    lib.gmm_group_metadata.restype = I
    lib.gmm_group_metadata.argtypes = [P, I, I64, P, SZ, P]
    lib.gmm_quantize_lhs.restype = I
    lib.gmm_quantize_lhs.argtypes = [P, I64, I64, P, P, P]
    lib.gmm_quantize_rhs.restype = I
    lib.gmm_quantize_rhs.argtypes = [P, I, I64, I64, P, P, P]
    lib.gmm_fp8_fwd.restype = I
    lib.gmm_fp8_fwd.argtypes = [P, P, P, P, P, I, I64, I64, I64, I, P, P, SZ, P]
    lib.gmm_fp8_fwd_tiled.restype = I
    lib.gmm_fp8_fwd_tiled.argtypes = [P, P, P, P, P, I, I64, I64, I64, I, P, P, SZ, P,
                                      ctypes.POINTER(TileConfig)]
    lib.gmm_bf16_fwd.restype = I
    lib.gmm_bf16_fwd.argtypes = [P, P, P, I, I64, I64, I64, I, P, P, SZ, P]
    lib.tgmm_bf16.restype = I
    lib.tgmm_bf16.argtypes = [P, P, P, I, I64, I64, I64, P, P, SZ, P]
    lib.tgmm_bf16_tiled.restype = I
    lib.tgmm_bf16_tiled.argtypes = [P, P, P, I, I64, I64, I64, P, P, SZ, P, ctypes.POINTER(TgmmConfig)]
    lib.gmm_fp8_fwd_swiglu_quant.restype = I
    lib.gmm_fp8_fwd_swiglu_quant.argtypes = [P, P, P, P, P, I, I64, I64, I64, P, P, P, P, SZ, P]
    lib.gmm_fp8_fwd_swiglu_quant_tiled.restype = I
    lib.gmm_fp8_fwd_swiglu_quant_tiled.argtypes = [P, P, P, P, P, I, I64, I64, I64, P, P, P, P, SZ, P,
                                                   ctypes.POINTER(TileConfig)]
    lib.gmm_bf16_dgrad.restype = I
    lib.gmm_bf16_dgrad.argtypes = [P, P, P, I, I64, I64, I64, P, P, SZ, P]
    lib.gmm_get_device_status.restype = I
    lib.gmm_get_device_status.argtypes = [P, P]
    lib.gmm_selftest_wait_timeout.restype = I
    lib.gmm_selftest_wait_timeout.argtypes = [P, SZ, I, P]
    lib.gmm_fp8_fwd_noalloc.restype = I
    lib.gmm_fp8_fwd_noalloc.argtypes = [P, P, P, P, P, I, I64, I64, I64, I, P, P]
    lib.gmm_quantize_rhs_w4.restype = I
    lib.gmm_quantize_rhs_w4.argtypes = [P, I, I64, I64, P, P, P]
    lib.gmm_fp8_w4_fwd.restype = I
    lib.gmm_fp8_w4_fwd.argtypes = [P, P, P, P, P, I, I64, I64, I64, I, P, P, SZ, P, ctypes.POINTER(TileConfig)]
    lib.gmm_fp8_w4_fwd_swiglu_quant.restype = I
    lib.gmm_fp8_w4_fwd_swiglu_quant.argtypes = [P, P, P, P, P, I, I64, I64, I64, P, P, P, P, SZ, P,
                                                ctypes.POINTER(TileConfig)]
    lib.gmm_bf16_swiglu_fwd.restype = I
    lib.gmm_bf16_swiglu_fwd.argtypes = [P, P, P, I, I64, I64, I64, P, P, P, P, P, SZ, P]
    lib.gmm_bf16_swiglu_bwd.restype = I
    lib.gmm_bf16_swiglu_bwd.argtypes = [P, P, P, P, P, P, I, I64, I64, I64, P, P, P, SZ, P]
    lib.tgmm_fp8_ckpt.restype = I
    lib.tgmm_fp8_ckpt.argtypes = [P, P, P, P, I, I64, I64, I64, P, P, SZ, P, SZ, P]
    lib.tgmm_fp8_ckpt_scratch_bytes.restype = SZ
    lib.tgmm_fp8_ckpt_scratch_bytes.argtypes = [I, I64, I64, I64]
    lib.gmm_mx4_quantize_lhs.restype = I
    lib.gmm_mx4_quantize_lhs.argtypes = [P, I64, I64, P, P, P]
    lib.gmm_mx4_quantize_rhs.restype = I
    lib.gmm_mx4_quantize_rhs.argtypes = [P, I, I64, I64, P, P, P]
    lib.gmm_mx4_fwd.restype = I
    lib.gmm_mx4_fwd.argtypes = [P, P, P, P, P, I, I64, I64, I64, I, P, P, SZ, P]
    lib.gmm_mx4_fwd_swiglu_quant.restype = I
    lib.gmm_mx4_fwd_swiglu_quant.argtypes = [P, P, P, P, P, I, I64, I64, I64, P, P, P, P, SZ, P]
    F = ctypes.c_float
    lib.gmm_route.restype = I
    lib.gmm_route.argtypes = [P, I, P, I64, I, I, I, I, F, P, P, P]
    lib.gmm_route_bwd.restype = I
    lib.gmm_route_bwd.argtypes = [P, P, I, P, I64, I, I, I, I, F, P, P]
    lib.gmm_sort_rows_scratch_bytes.restype = SZ
    lib.gmm_sort_rows_scratch_bytes.argtypes = [I64, I]
    lib.gmm_sort_rows.restype = I
    lib.gmm_sort_rows.argtypes = [P, I64, I, P, P, P, SZ, P]
    lib.gmm_gather_rows.restype = I
    lib.gmm_gather_rows.argtypes = [P, P, I64, I, I64, P, P]
    lib.gmm_gather_quantize.restype = I
    lib.gmm_gather_quantize.argtypes = [P, P, I64, I, I64, P, P, P]
    lib.gmm_combine_rows.restype = I
    lib.gmm_combine_rows.argtypes = [P, P, P, I64, I, I64, P, P]
    lib.gmm_combine_rows_bwd.restype = I
    lib.gmm_combine_rows_bwd.argtypes = [P, P, P, P, I64, I, I64, P, P, P]
    lib.gmm_norm_join.restype = I
    lib.gmm_norm_join.argtypes = [P, I, P, P, P, I, P, I64, I64, F, F, F, P, P, P]
    lib.gmm_norm_join_bwd_scratch_bytes.restype = SZ
    lib.gmm_norm_join_bwd_scratch_bytes.argtypes = [I64, I64]
    lib.gmm_norm_join_bwd.restype = I
    lib.gmm_norm_join_bwd.argtypes = [P, P, P, I, P, P, P, I, P, I64, I64, F, F, F, P, P, P, P, P, P, SZ, P]
    lib.gmm_clip_grads_scratch_bytes.restype = SZ
    lib.gmm_clip_grads_scratch_bytes.argtypes = [I]
    lib.gmm_clip_grads.restype = I
    lib.gmm_clip_grads.argtypes = [P, P, P, P, I, F, P, P, SZ, P]
    _lib = lib
    return lib


def _p(t) -> int | None:
    if t is None:
        return None
    try:
        return t.data_ptr() or None  # a tensor without elements has the address 0
    except AttributeError:
        return int(t)


def _s(stream) -> int | None:
    if stream is None:
        # torch.cuda.current_stream().cuda_stream without building a Stream object
        # (0.4 us instead of 3 us of host time a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, where: str):
    if status != GMM_OK:
        raise GmmError(status, where)


# ---------------------------------------------------------------------------
# C entry points, same names and argument order
# ---------------------------------------------------------------------------

def gmm_workspace_bytes(G: int, M: int) -> int:
    return int(load().gmm_workspace_bytes(G, M))


def gmm_tiles_offset(G: int) -> int:
    return int(load().gmm_tiles_offset(G))


def gmm_group_metadata(group_sizes, G, M, workspace, workspace_bytes, stream=None) -> int:
    return load().gmm_group_metadata(_p(group_sizes), G, M, _p(workspace), workspace_bytes, _s(stream))


def gmm_quantize_lhs(x, M, K, xq, xs, stream=None) -> int:
    return load().gmm_quantize_lhs(_p(x), M, K, _p(xq), _p(xs), _s(stream))


def gmm_quantize_rhs(w, G, K, N, wq, ws, stream=None) -> int:
    return load().gmm_quantize_rhs(_p(w), G, K, N, _p(wq), _p(ws), _s(stream))


def gmm_fp8_fwd(xq, xs, wq, ws, group_sizes, G, M, K, N, fuse_silu_mul, out, workspace,
                workspace_bytes, stream=None) -> int:
    return load().gmm_fp8_fwd(_p(xq), _p(xs), _p(wq), _p(ws), _p(group_sizes), G, M, K, N,
                              int(fuse_silu_mul), _p(out), _p(workspace), workspace_bytes, _s(stream))


def gmm_fp8_fwd_tiled(xq, xs, wq, ws, group_sizes, G, M, K, N, fuse_silu_mul, out, workspace,
                      workspace_bytes, stream=None, config=None) -> int:
    """config: a TileConfig, a (bn, ctas, unit_order[, cta_group[, stages[, tmem_bufs]]]) tuple, or None."""
    if config is not None and not isinstance(config, TileConfig):
        config = TileConfig(*config)
    return load().gmm_fp8_fwd_tiled(_p(xq), _p(xs), _p(wq), _p(ws), _p(group_sizes), G, M, K, N,
                                    int(fuse_silu_mul), _p(out), _p(workspace), workspace_bytes, _s(stream),
                                    ctypes.byref(config) if config is not None else None)


def gmm_fp8_fwd_swiglu_quant(xq, xs, wq, ws, group_sizes, G, M, K, N, h, hq, hs, workspace,
                             workspace_bytes, stream=None) -> int:
    return load().gmm_fp8_fwd_swiglu_quant(_p(xq), _p(xs), _p(wq), _p(ws), _p(group_sizes), G, M, K, N, _p(h),
                                           _p(hq), _p(hs), _p(workspace), workspace_bytes, _s(stream))


def gmm_fp8_fwd_swiglu_quant_tiled(xq, xs, wq, ws, group_sizes, G, M, K, N, h, hq, hs, workspace,
                                   workspace_bytes, stream=None, config=None) -> int:
    """config: a TileConfig, a (bn, ctas, unit_order[, cta_group[, stages[, tmem_bufs]]]) tuple, or None."""
    if config is not None and not isinstance(config, TileConfig):
        config = TileConfig(*config)
    return load().gmm_fp8_fwd_swiglu_quant_tiled(_p(xq), _p(xs), _p(wq), _p(ws), _p(group_sizes), G, M, K, N,
                                                 _p(h), _p(hq), _p(hs), _p(workspace), workspace_bytes, _s(stream),
                                                 ctypes.byref(config) if config is not None else None)


def _cfg(config):
    if config is None:
        return None
    if not isinstance(config, TileConfig):
        config = TileConfig(*config)
    return ctypes.byref(config)


def gmm_quantize_rhs_w4(w, G, K, N, wq4, ws, stream=None) -> int:
    return load().gmm_quantize_rhs_w4(_p(w), G, K, N, _p(wq4), _p(ws), _s(stream))


def gmm_fp8_w4_fwd(xq, xs, wq4, ws, group_sizes, G, M, K, N, fuse_silu_mul, out, workspace, workspace_bytes,
                   stream=None, config=None) -> int:
    return load().gmm_fp8_w4_fwd(_p(xq), _p(xs), _p(wq4), _p(ws), _p(group_sizes), G, M, K, N, int(fuse_silu_mul),
                                 _p(out), _p(workspace), workspace_bytes, _s(stream), _cfg(config))


def gmm_fp8_w4_fwd_swiglu_quant(xq, xs, wq4, ws, group_sizes, G, M, K, N, h, hq, hs, workspace, workspace_bytes,
                                stream=None, config=None) -> int:
    return load().gmm_fp8_w4_fwd_swiglu_quant(_p(xq), _p(xs), _p(wq4), _p(ws), _p(group_sizes), G, M, K, N, _p(h),
                                              _p(hq), _p(hs), _p(workspace), workspace_bytes, _s(stream),
                                              _cfg(config))


def gmm_bf16_fwd(x, w, group_sizes, G, M, K, N, fuse_silu_mul, out, workspace, workspace_bytes,
                 stream=None) -> int:
    return load().gmm_bf16_fwd(_p(x), _p(w), _p(group_sizes), G, M, K, N, int(fuse_silu_mul),
                               _p(out), _p(workspace), workspace_bytes, _s(stream))


def gmm_bf16_dgrad(dy, w, group_sizes, G, M, K, N, dx, workspace, workspace_bytes, stream=None) -> int:
    return load().gmm_bf16_dgrad(_p(dy), _p(w), _p(group_sizes), G, M, K, N, _p(dx), _p(workspace),
                                 workspace_bytes, _s(stream))


def tgmm_bf16(x, dy, group_sizes, G, M, K, N, dw, workspace, workspace_bytes, stream=None) -> int:
    return load().tgmm_bf16(_p(x), _p(dy), _p(group_sizes), G, M, K, N, _p(dw), _p(workspace),
                            workspace_bytes, _s(stream))


def tgmm_bf16_tiled(x, dy, group_sizes, G, M, K, N, dw, workspace, workspace_bytes, stream=None,
                    config=None) -> int:
    """config: a TgmmConfig, a (stages, claim_ahead, max_batch) tuple, or None (defaults)."""
    if config is not None and not isinstance(config, TgmmConfig):
        config = TgmmConfig(*config)
    return load().tgmm_bf16_tiled(_p(x), _p(dy), _p(group_sizes), G, M, K, N, _p(dw), _p(workspace),
                                  workspace_bytes, _s(stream), ctypes.byref(config) if config is not None else None)


def gmm_get_device_status(workspace, stream=None) -> int:
    return load().gmm_get_device_status(_p(workspace), _s(stream))


def gmm_selftest_wait_timeout(workspace, workspace_bytes, limit_ms, stream=None) -> int:
    return load().gmm_selftest_wait_timeout(_p(workspace), workspace_bytes, int(limit_ms), _s(stream))


def gmm_fp8_fwd_noalloc(xq, xs, wq, ws, group_sizes, G, M, K, N, fuse_silu_mul, out,
                        stream=None) -> int:
    """gmm_fp8_fwd for callers that cannot allocate: no workspace argument;
    the metadata lives in the library's static device array (see gmm.h)."""
    return load().gmm_fp8_fwd_noalloc(_p(xq), _p(xs), _p(wq), _p(ws), _p(group_sizes), G, M, K, N,
                                      int(fuse_silu_mul), _p(out), _s(stream))


def gmm_bf16_swiglu_fwd(x, w, group_sizes, G, M, K, N, h, gu, guq, gus, workspace, workspace_bytes,
                        stream=None) -> int:
    return load().gmm_bf16_swiglu_fwd(_p(x), _p(w), _p(group_sizes), G, M, K, N, _p(h), _p(gu), _p(guq), _p(gus),
                                      _p(workspace), workspace_bytes, _s(stream))


def gmm_bf16_swiglu_bwd(dy, w2, gu, guq, gus, group_sizes, G, M, K, N, dgu, h, workspace, workspace_bytes,
                        stream=None) -> int:
    return load().gmm_bf16_swiglu_bwd(_p(dy), _p(w2), _p(gu), _p(guq), _p(gus), _p(group_sizes), G, M, K, N,
                                      _p(dgu), _p(h), _p(workspace), workspace_bytes, _s(stream))


def tgmm_fp8_ckpt_scratch_bytes(G: int, M: int, K: int, N: int) -> int:
    return int(load().tgmm_fp8_ckpt_scratch_bytes(G, M, K, N))


def tgmm_fp8_ckpt(xq, xs, dy, group_sizes, G, M, K, N, dw, scratch, scratch_bytes, workspace, workspace_bytes,
                  stream=None) -> int:
    return load().tgmm_fp8_ckpt(_p(xq), _p(xs), _p(dy), _p(group_sizes), G, M, K, N, _p(dw), _p(scratch),
                                scratch_bytes, _p(workspace), workspace_bytes, _s(stream))


def gmm_mx4_quantize_lhs(x, M, K, xq, xs, stream=None) -> int:
    return load().gmm_mx4_quantize_lhs(_p(x), M, K, _p(xq), _p(xs), _s(stream))


def gmm_mx4_quantize_rhs(w, G, K, N, wq, ws, stream=None) -> int:
    return load().gmm_mx4_quantize_rhs(_p(w), G, K, N, _p(wq), _p(ws), _s(stream))


def gmm_mx4_fwd(xq, xs, wq, ws, group_sizes, G, M, K, N, fuse_silu_mul, out, workspace, workspace_bytes,
                stream=None) -> int:
    return load().gmm_mx4_fwd(_p(xq), _p(xs), _p(wq), _p(ws), _p(group_sizes), G, M, K, N, int(fuse_silu_mul),
                              _p(out), _p(workspace), workspace_bytes, _s(stream))


def gmm_mx4_fwd_swiglu_quant(xq, xs, wq, ws, group_sizes, G, M, K, N, h, hq, hs, workspace, workspace_bytes,
                             stream=None) -> int:
    return load().gmm_mx4_fwd_swiglu_quant(_p(xq), _p(xs), _p(wq), _p(ws), _p(group_sizes), G, M, K, N, _p(h),
                                           _p(hq), _p(hs), _p(workspace), workspace_bytes, _s(stream))


def gmm_route(logits, logits_type, bias, T, E, k, score, renorm, scale, ids, weights, stream=None) -> int:
    return load().gmm_route(_p(logits), logits_type, _p(bias), T, E, k, score, int(renorm), scale, _p(ids),
                            _p(weights), _s(stream))


def gmm_route_bwd(dweights, logits, logits_type, ids, T, E, k, score, renorm, scale, dlogits, stream=None) -> int:
    return load().gmm_route_bwd(_p(dweights), _p(logits), logits_type, _p(ids), T, E, k, score, int(renorm), scale,
                                _p(dlogits), _s(stream))


def gmm_sort_rows_scratch_bytes(N: int, G: int) -> int:
    return int(load().gmm_sort_rows_scratch_bytes(N, G))


def gmm_sort_rows(ids, N, G, rows, group_sizes, scratch, scratch_bytes, stream=None) -> int:
    return load().gmm_sort_rows(_p(ids), N, G, _p(rows), _p(group_sizes), _p(scratch), scratch_bytes, _s(stream))


def gmm_gather_rows(x, rows, T, k, K, out, stream=None) -> int:
    return load().gmm_gather_rows(_p(x), _p(rows), T, k, K, _p(out), _s(stream))


def gmm_gather_quantize(x, rows, T, k, K, xq, xs, stream=None) -> int:
    return load().gmm_gather_quantize(_p(x), _p(rows), T, k, K, _p(xq), _p(xs), _s(stream))


def gmm_combine_rows(y, rows, weights, T, k, K, out, stream=None) -> int:
    return load().gmm_combine_rows(_p(y), _p(rows), _p(weights), T, k, K, _p(out), _s(stream))


def gmm_combine_rows_bwd(dout, y, rows, weights, T, k, K, dy, dweights, stream=None) -> int:
    return load().gmm_combine_rows_bwd(_p(dout), _p(y), _p(rows), _p(weights), T, k, K, _p(dy), _p(dweights),
                                       _s(stream))


def gmm_norm_join(x, stream_type, b, w_post, gate, gate_rows, w_next, T, K, residual_scale, block_scale, eps, out, n,
                  stream=None) -> int:
    return load().gmm_norm_join(_p(x), stream_type, _p(b), _p(w_post), _p(gate), int(gate_rows), _p(w_next), T, K,
                                residual_scale, block_scale, eps, _p(out), _p(n), _s(stream))


def gmm_norm_join_bwd_scratch_bytes(T: int, K: int) -> int:
    return int(load().gmm_norm_join_bwd_scratch_bytes(T, K))


def gmm_norm_join_bwd(dout, dn, out, stream_type, b, w_post, gate, gate_rows, w_next, T, K, residual_scale,
                      block_scale, eps, dx, db, dw_post, dgate, dw_next, scratch, scratch_bytes, stream=None) -> int:
    return load().gmm_norm_join_bwd(_p(dout), _p(dn), _p(out), stream_type, _p(b), _p(w_post), _p(gate),
                                    int(gate_rows), _p(w_next), T, K, residual_scale, block_scale, eps, _p(dx),
                                    _p(db), _p(dw_post), _p(dgate), _p(dw_next), _p(scratch), scratch_bytes,
                                    _s(stream))


def gmm_clip_grads_scratch_bytes(n: int) -> int:
    return int(load().gmm_clip_grads_scratch_bytes(n))


def gmm_clip_grads(grads, out, counts, types, n, max_norm, norm, scratch, scratch_bytes, stream=None) -> int:
    """grads, out, counts, types: addresses of the HOST arrays (out may be None)."""
    return load().gmm_clip_grads(grads, out, counts, types, n, max_norm, _p(norm), _p(scratch), scratch_bytes,
                                 _s(stream))


# ---------------------------------------------------------------------------
# convenience wrappers: allocate outputs with torch, call the C entry points
# ---------------------------------------------------------------------------

def _stream_of(handle, device):
    """torch's stream of a raw handle.  0 and 1 (cudaStreamLegacy) are the default
    stream, for which torch makes no external stream: of 0 it makes a new one."""
    if handle in (0, 1):
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(handle, device=device)


def _other(stream):
    """The context that makes `stream` current, or None where it is already.

    A wrapper that is given a stream starts over inside it: its own allocations
    (outputs, scratch, a temporary workspace and its zero fill) then come from
    that stream's memory.  Memory taken from another stream's pool would be
    ordered by nothing: its zero fill could come after the kernel, and once
    released it could serve that other stream while the kernel still runs.  The
    outputs belong to `stream`, as those of any torch operation on it."""
    current = torch.cuda.current_stream()
    if not isinstance(stream, torch.cuda.Stream):
        stream = _stream_of(int(stream), current.device)
    if stream.cuda_stream == current.cuda_stream and stream.device == current.device:
        return None
    return torch.cuda.stream(stream)


class Workspace:
    """A zero-initialised device workspace sized for (G, M); the zero fill runs
    on the current stream, so another stream that uses it waits for that one."""

    def __init__(self, G: int, M: int, device="cuda"):
        self.G, self.M = G, M
        self.nbytes = gmm_workspace_bytes(G, M)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device)

    def fits(self, G: int, M: int) -> bool:
        return (G == self.G and M == self.M) or gmm_workspace_bytes(G, M) <= self.nbytes

    def status(self, stream=None) -> int:
        return gmm_get_device_status(self.buf, stream)

    def header(self) -> list[int]:
        return self.buf[:16].view(torch.int32).tolist()

    def offsets(self) -> list[int]:
        return self.buf[32:32 + 4 * (self.G + 1)].view(torch.int32).tolist()

    def tiles(self) -> torch.Tensor:
        n = self.header()[3]
        off = gmm_tiles_offset(self.G)
        return self.buf[off:off + 16 * n].view(torch.int32).view(n, 4)[:, :3]

    def _order_offset(self) -> int:
        return gmm_tiles_offset(self.G) + 16 * ((self.M + 127) // 128 + self.G)

    def order(self) -> list[int]:
        """The group ids sorted by size, largest first (ties by id)."""
        off = self._order_offset()
        return self.buf[off:off + 4 * self.G].view(torch.int32).tolist()

    def pair_tiles(self) -> torch.Tensor:
        """The 256-row tiles {g, row0, row1} (the CTA-pair FP8 kernel's)."""
        n = self.buf[24:28].view(torch.int32).item()
        off = self._order_offset() + 16 * ((self.G + 3) // 4)
        return self.buf[off:off + 16 * n].view(torch.int32).view(n, 4)[:, :3]


def _ws(ws, G, M, device):
    if ws is None or not ws.fits(G, M):
        ws = Workspace(G, M, device)
    return ws


def _ws_for(group_sizes, ws, G, M, device):
    """Workspace of a grouped call.  group_sizes=None reuses the metadata that
    an earlier call (or group_metadata) left in `ws`, so `ws` must be given."""
    if group_sizes is None:
        if ws is None or not ws.fits(G, M):
            raise ValueError("group_sizes=None reuses the metadata in `workspace`: pass that workspace")
        return ws
    return _ws(ws, G, M, device)


def quantize_lhs(x: torch.Tensor, stream=None):
    """x bf16 [M, K] -> (xq uint8 [M, K] e4m3 codes, xs float32 [K/128, M])."""
    if stream is not None and (other := _other(stream)):
        with other:
            return quantize_lhs(x, stream)
    M, K = x.shape
    xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    xs = torch.empty((K // 128, M), dtype=torch.float32, device=x.device)
    _check(gmm_quantize_lhs(x, M, K, xq, xs, stream), "gmm_quantize_lhs")
    return xq, xs


def quantize_rhs(w: torch.Tensor, stream=None):
    """w bf16 [G, K, N] -> (wq uint8 [G, N, K] e4m3 codes, ws float32 [G, K/128, N/128])."""
    if stream is not None and (other := _other(stream)):
        with other:
            return quantize_rhs(w, stream)
    G, K, N = w.shape
    wq = torch.empty((G, N, K), dtype=torch.uint8, device=w.device)
    ws = torch.empty((G, K // 128, N // 128), dtype=torch.float32, device=w.device)
    _check(gmm_quantize_rhs(w, G, K, N, wq, ws, stream), "gmm_quantize_rhs")
    return wq, ws


def quantize_rhs_w4(w: torch.Tensor, stream=None):
    """w bf16 [G, K, N] -> (wq4 uint8 [G, N, K/2] packed E2M1 codes, ws float32 [G, K/128, N/128])."""
    if stream is not None and (other := _other(stream)):
        with other:
            return quantize_rhs_w4(w, stream)
    G, K, N = w.shape
    wq4 = torch.empty((G, N, K // 2), dtype=torch.uint8, device=w.device)
    ws = torch.empty((G, K // 128, N // 128), dtype=torch.float32, device=w.device)
    _check(gmm_quantize_rhs_w4(w, G, K, N, wq4, ws, stream), "gmm_quantize_rhs_w4")
    return wq4, ws


def fp8_w4_fwd(xq, xs, wq4, ws, group_sizes, fuse=False, out=None, workspace=None, stream=None, config=None):
    """The FP8 forward with 4-bit weights (wq4 [G, Nw, K/2] from quantize_rhs_w4)."""
    if stream is not None and (other := _other(stream)):
        with other:
            return fp8_w4_fwd(xq, xs, wq4, ws, group_sizes, fuse, out, workspace, stream, config)
    M, K = xq.shape
    G, Nw, K2 = wq4.shape
    assert 2 * K2 == K
    N = Nw // 2 if fuse else Nw
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    ws_ = _ws_for(group_sizes, workspace, G, M, xq.device)
    _check(gmm_fp8_w4_fwd(xq, xs, wq4, ws, group_sizes, G, M, K, N, fuse, out, ws_.buf, ws_.nbytes, stream, config),
           "gmm_fp8_w4_fwd")
    return out


def fp8_w4_fwd_swiglu_quant(xq, xs, wq4, ws, group_sizes, with_h=True, workspace=None, stream=None, config=None,
                            out=None):
    """Fused wi with 4-bit weights: returns (h or None, hq, hs) as fp8_fwd_swiglu_quant."""
    if stream is not None and (other := _other(stream)):
        with other:
            return fp8_w4_fwd_swiglu_quant(xq, xs, wq4, ws, group_sizes, with_h, workspace, stream, config, out)
    M, K = xq.shape
    G, Nw, K2 = wq4.shape
    assert 2 * K2 == K
    N = Nw // 2
    if out is not None:
        h, hq, hs = out
    else:
        h = torch.empty((M, N), dtype=torch.bfloat16, device=xq.device) if with_h else None
        hq = torch.empty((M, N), dtype=torch.uint8, device=xq.device)
        hs = torch.empty((N // 128, M), dtype=torch.float32, device=xq.device)
    ws_ = _ws_for(group_sizes, workspace, G, M, xq.device)
    _check(gmm_fp8_w4_fwd_swiglu_quant(xq, xs, wq4, ws, group_sizes, G, M, K, N, h, hq, hs, ws_.buf, ws_.nbytes,
                                       stream, config), "gmm_fp8_w4_fwd_swiglu_quant")
    return h, hq, hs


def fp8_fwd(xq, xs, wq, ws, group_sizes, fuse=False, out=None, workspace=None, stream=None, config=None):
    """config: a tile configuration (see TileConfig), or None for the defaults."""
    if stream is not None and (other := _other(stream)):
        with other:
            return fp8_fwd(xq, xs, wq, ws, group_sizes, fuse, out, workspace, stream, config)
    M, K = xq.shape
    G, Nw, K2 = wq.shape
    assert K2 == K
    N = Nw // 2 if fuse else Nw
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    ws_ = _ws_for(group_sizes, workspace, G, M, xq.device)
    if config is None:
        _check(gmm_fp8_fwd(xq, xs, wq, ws, group_sizes, G, M, K, N, fuse, out, ws_.buf, ws_.nbytes,
                           stream), "gmm_fp8_fwd")
    else:
        _check(gmm_fp8_fwd_tiled(xq, xs, wq, ws, group_sizes, G, M, K, N, fuse, out, ws_.buf, ws_.nbytes,
                                 stream, config), "gmm_fp8_fwd_tiled")
    return out


def fp8_fwd_swiglu_quant(xq, xs, wq, ws, group_sizes, with_h=True, workspace=None, stream=None, config=None,
                         out=None):
    """Fused wi: returns (h or None, hq [M, N] e4m3 codes, hs [N/128, M]).
    config: a tile configuration (see TileConfig), or None for the defaults;
    out: an (h, hq, hs) triple to write into instead of new tensors."""
    if stream is not None and (other := _other(stream)):
        with other:
            return fp8_fwd_swiglu_quant(xq, xs, wq, ws, group_sizes, with_h, workspace, stream, config, out)
    M, K = xq.shape
    G, Nw, K2 = wq.shape
    assert K2 == K
    N = Nw // 2
    if out is not None:
        h, hq, hs = out
    else:
        h = torch.empty((M, N), dtype=torch.bfloat16, device=xq.device) if with_h else None
        hq = torch.empty((M, N), dtype=torch.uint8, device=xq.device)
        hs = torch.empty((N // 128, M), dtype=torch.float32, device=xq.device)
    ws_ = _ws_for(group_sizes, workspace, G, M, xq.device)
    if config is None:
        _check(gmm_fp8_fwd_swiglu_quant(xq, xs, wq, ws, group_sizes, G, M, K, N, h, hq, hs, ws_.buf, ws_.nbytes,
                                        stream), "gmm_fp8_fwd_swiglu_quant")
    else:
        _check(gmm_fp8_fwd_swiglu_quant_tiled(xq, xs, wq, ws, group_sizes, G, M, K, N, h, hq, hs, ws_.buf,
                                              ws_.nbytes, stream, config), "gmm_fp8_fwd_swiglu_quant_tiled")
    return h, hq, hs


def bf16_fwd(x, w, group_sizes, fuse=False, out=None, workspace=None, stream=None):
    if stream is not None and (other := _other(stream)):
        with other:
            return bf16_fwd(x, w, group_sizes, fuse, out, workspace, stream)
    M, K = x.shape
    G, K2, Nw = w.shape
    assert K2 == K
    N = Nw // 2 if fuse else Nw
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    ws_ = _ws_for(group_sizes, workspace, G, M, x.device)
    _check(gmm_bf16_fwd(x, w, group_sizes, G, M, K, N, fuse, out, ws_.buf, ws_.nbytes, stream),
           "gmm_bf16_fwd")
    return out


def dgrad(dy, w, group_sizes, dx=None, workspace=None, stream=None):
    """dx [M, K] = dy [M, N] . w[g]^T per group, w [G, K, N]."""
    if stream is not None and (other := _other(stream)):
        with other:
            return dgrad(dy, w, group_sizes, dx, workspace, stream)
    M, N = dy.shape
    G, K, N2 = w.shape
    assert N2 == N
    if dx is None:
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=dy.device)
    ws_ = _ws_for(group_sizes, workspace, G, M, dy.device)
    _check(gmm_bf16_dgrad(dy, w, group_sizes, G, M, K, N, dx, ws_.buf, ws_.nbytes, stream), "gmm_bf16_dgrad")
    return dx


def tgmm(x, dy, group_sizes, dw=None, workspace=None, stream=None, config=None):
    if stream is not None and (other := _other(stream)):
        with other:
            return tgmm(x, dy, group_sizes, dw, workspace, stream, config)
    M, K = x.shape
    M2, N = dy.shape
    assert M2 == M
    if group_sizes is not None:
        G = group_sizes.numel()
    elif dw is not None:
        G = dw.shape[0]
    elif workspace is not None:
        G = workspace.G
    else:
        raise ValueError("group_sizes=None reuses the metadata in `workspace`: pass that workspace")
    if dw is None:
        dw = torch.empty((G, K, N), dtype=torch.bfloat16, device=x.device)
    ws_ = _ws_for(group_sizes, workspace, G, M, x.device)
    if config is None:
        _check(tgmm_bf16(x, dy, group_sizes, G, M, K, N, dw, ws_.buf, ws_.nbytes, stream), "tgmm_bf16")
    else:
        _check(tgmm_bf16_tiled(x, dy, group_sizes, G, M, K, N, dw, ws_.buf, ws_.nbytes, stream, config),
               "tgmm_bf16_tiled")
    return dw


def group_metadata(group_sizes, M, workspace=None, stream=None) -> Workspace:
    if stream is not None and (other := _other(stream)):
        with other:
            return group_metadata(group_sizes, M, workspace, stream)
    G = group_sizes.numel()
    ws_ = _ws(workspace, G, M, group_sizes.device)
    _check(gmm_group_metadata(group_sizes, G, M, ws_.buf, ws_.nbytes, stream), "gmm_group_metadata")
    return ws_


def _need(what, t, on, dtype, *shape, flat=False):
    """Refuses what the kernels would read or write wrongly: they take dense
    buffers of their own device (`on`: the index of the call's first tensor,
    which _here compares with the current device) and know neither strides nor
    types.  One number: that many elements, in any shape; flat: or as many in
    one dimension."""
    if len(shape) == 1:
        same = t.numel() == shape[0]
    else:
        same = t.shape == shape or (flat and t.dim() == 1 and t.numel() == math.prod(shape))
    if t.dtype is not dtype or not same or not t.is_contiguous() or t.get_device() != on or on < 0:
        where = "" if on < 0 else f" on cuda:{on}"
        raise ValueError(f"{what}: expected a contiguous CUDA tensor of {'x'.join(map(str, shape))} {dtype} elements"
                         f"{where}, got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _here(on):
    """Refuses tensors of a device that is not current: the kernels run on that one."""
    dev = torch.cuda.current_device()
    if dev != on:
        raise ValueError(f"the tensors are on cuda:{on}, the current device is cuda:{dev}")


def _need_sizes(group_sizes, on, G):
    if group_sizes is not None:
        _need("group_sizes", group_sizes, on, torch.int32, G)


def _ws_on(on, group_sizes, ws, G, M, device):
    """_ws_for, with a workspace given checked for its device."""
    if ws is not None:
        if ws.buf.get_device() != on:
            raise ValueError(f"workspace: expected one on cuda:{on}, got one on {ws.buf.device}")
        if ws.fits(G, M):
            return ws
    return _ws_for(group_sizes, ws, G, M, device)


def _new2(a, b, dtype, device):
    """torch.empty((a, b)) by way of empty_strided, which takes half the host time."""
    return torch.empty_strided((a, b), (b, 1), dtype=dtype, device=device)


def _new3(a, b, c, dtype, device):
    return torch.empty_strided((a, b, c), (b * c, c, 1), dtype=dtype, device=device)


def _need_kept(kept, M, N, keep=None, on=-1):
    """Checks kept gate | up values (of the form `keep`, if given); returns (gu, guq, gus)."""
    if isinstance(kept, (tuple, list)) and keep != "bf16":
        guq, gus = kept
        _need("kept codes", guq, on, torch.uint8, M, 2 * N)
        _need("kept scales", gus, on, torch.float32, 2 * N // 128, M)
        return None, guq, gus
    if keep == "e4m3" or not isinstance(kept, torch.Tensor):
        raise ValueError("kept: expected the gate | up values in bf16, or their (codes, scales)")
    _need("kept", kept, on, torch.bfloat16, M, 2 * N)
    return kept, None, None


def swiglu_fwd(x, w, group_sizes, keep="bf16", workspace=None, stream=None, out=None):
    """The gated block's forward: x bf16 [M, K], w bf16 [G, K, 2N] (gate | up)
    -> (h bf16 [M, N], kept), kept being what swiglu_bwd takes: the gate | up
    values in bf16 [M, 2N] (keep="bf16"), or their 8-bit checkpoint (codes
    uint8 [M, 2N], scales float32 [2N/128, M]) (keep="e4m3").
    out: an (h, kept) pair to write into instead of new tensors."""
    if stream is not None and (other := _other(stream)):
        with other:
            return swiglu_fwd(x, w, group_sizes, keep, workspace, stream, out)
    if keep not in ("bf16", "e4m3"):
        raise ValueError(f"keep must be 'bf16' or 'e4m3', got {keep!r}")
    M, K = x.shape
    G, K2, Nw = w.shape
    assert K2 == K and Nw % 2 == 0
    N = Nw // 2
    on = x.get_device()
    _need("x", x, on, torch.bfloat16, M, K)
    _here(on)
    _need("w", w, on, torch.bfloat16, G, K, Nw)
    _need_sizes(group_sizes, on, G)
    if out is not None:
        h, kept = out
        _need("out h", h, on, torch.bfloat16, M, N)
        _need_kept(kept, M, N, keep, on)
    else:
        h = _new2(M, N, torch.bfloat16, x.device)
        if keep == "bf16":
            kept = _new2(M, Nw, torch.bfloat16, x.device)
        else:
            kept = (_new2(M, Nw, torch.uint8, x.device), _new2(Nw // 128, M, torch.float32, x.device))
    gu, (guq, gus) = (kept, (None, None)) if keep == "bf16" else (None, kept)
    ws_ = _ws_on(on, group_sizes, workspace, G, M, x.device)
    _check(gmm_bf16_swiglu_fwd(x, w, group_sizes, G, M, K, N, h, gu, guq, gus, ws_.buf, ws_.nbytes, stream),
           "gmm_bf16_swiglu_fwd")
    return h, kept


def swiglu_bwd(dy, w2, kept, group_sizes, with_h=True, workspace=None, stream=None, out=None):
    """Its backward pass: dy bf16 [M, K] (the gradient of y = h W2), w2 bf16
    [G, N, K], kept as swiglu_fwd returned it -> (dgu bf16 [M, 2N], the gradient
    of gate | up; h bf16 [M, N], recomputed, or None).
    out: a (dgu, h) pair to write into instead of new tensors."""
    if stream is not None and (other := _other(stream)):
        with other:
            return swiglu_bwd(dy, w2, kept, group_sizes, with_h, workspace, stream, out)
    M, K = dy.shape
    G, N, K2 = w2.shape
    assert K2 == K
    on = dy.get_device()
    _need("dy", dy, on, torch.bfloat16, M, K)
    _here(on)
    _need("w2", w2, on, torch.bfloat16, G, N, K)
    _need_sizes(group_sizes, on, G)
    gu, guq, gus = _need_kept(kept, M, N, on=on)
    if out is not None:
        dgu, h = out
        _need("out dgu", dgu, on, torch.bfloat16, M, 2 * N)
        if h is not None:
            _need("out h", h, on, torch.bfloat16, M, N)
    else:
        dgu = _new2(M, 2 * N, torch.bfloat16, dy.device)
        h = _new2(M, N, torch.bfloat16, dy.device) if with_h else None
    ws_ = _ws_on(on, group_sizes, workspace, G, M, dy.device)
    _check(gmm_bf16_swiglu_bwd(dy, w2, gu, guq, gus, group_sizes, G, M, K, N, dgu, h, ws_.buf, ws_.nbytes, stream),
           "gmm_bf16_swiglu_bwd")
    return dgu, h


def tgmm_ckpt(xq, xs, dy, group_sizes, dw=None, workspace=None, stream=None):
    """tgmm from the 8-bit checkpoint of x: xq uint8 [M, K] e4m3 codes, xs
    float32 [K/128, M] (quantize_lhs), dy bf16 [M, N] -> dw bf16 [G, K, N].
    The scratch that few tiles with many rows need is allocated with torch."""
    if stream is not None and (other := _other(stream)):
        with other:
            return tgmm_ckpt(xq, xs, dy, group_sizes, dw, workspace, stream)
    M, K = xq.shape
    M2, N = dy.shape
    assert M2 == M
    on = xq.get_device()
    _need("xq", xq, on, torch.uint8, M, K)
    _here(on)
    _need("xs", xs, on, torch.float32, K // 128, M)
    _need("dy", dy, on, torch.bfloat16, M, N)
    if group_sizes is not None:
        G = group_sizes.numel()
    elif dw is not None:
        G = dw.shape[0]
    elif workspace is not None:
        G = workspace.G
    else:
        raise ValueError("group_sizes=None reuses the metadata in `workspace`: pass that workspace")
    _need_sizes(group_sizes, on, G)
    if dw is not None:
        _need("dw", dw, on, torch.bfloat16, G, K, N)
    else:
        dw = _new3(G, K, N, torch.bfloat16, dy.device)
    ws_ = _ws_on(on, group_sizes, workspace, G, M, dy.device)
    nbytes = tgmm_fp8_ckpt_scratch_bytes(G, M, K, N)
    scratch = None
    if nbytes:
        scratch = torch.empty(nbytes, dtype=torch.uint8, device=dy.device)
    _check(tgmm_fp8_ckpt(xq, xs, dy, group_sizes, G, M, K, N, dw, scratch, nbytes, ws_.buf, ws_.nbytes, stream),
           "tgmm_fp8_ckpt")
    return dw


def mx4_quantize_lhs(x: torch.Tensor, stream=None, out=None):
    """x bf16 [M, K] -> (xq uint8 [M, K/2] packed E2M1 codes, xs uint8 [K/128, M, 4] E8M0 scales)."""
    if stream is not None and (other := _other(stream)):
        with other:
            return mx4_quantize_lhs(x, stream, out)
    M, K = x.shape
    on = x.get_device()
    _need("x", x, on, torch.bfloat16, M, K)
    _here(on)
    if out is not None:
        xq, xs = out
        _need("out codes", xq, on, torch.uint8, M, K // 2)
        _need("out scales", xs, on, torch.uint8, K // 128, M, 4, flat=True)
    else:
        xq = _new2(M, K // 2, torch.uint8, x.device)
        xs = _new3(K // 128, M, 4, torch.uint8, x.device)
    _check(gmm_mx4_quantize_lhs(x, M, K, xq, xs, stream), "gmm_mx4_quantize_lhs")
    return xq, xs


def mx4_quantize_rhs(w: torch.Tensor, stream=None):
    """w bf16 [G, K, N] -> (wq uint8 [G, N, K/2] packed E2M1 codes, ws uint8 [G, N/128, K/128, 512] E8M0 scales)."""
    if stream is not None and (other := _other(stream)):
        with other:
            return mx4_quantize_rhs(w, stream)
    G, K, N = w.shape
    on = w.get_device()
    _need("w", w, on, torch.bfloat16, G, K, N)
    _here(on)
    wq = _new3(G, N, K // 2, torch.uint8, w.device)
    ws = torch.empty((G, N // 128, K // 128, 512), dtype=torch.uint8, device=w.device)
    _check(gmm_mx4_quantize_rhs(w, G, K, N, wq, ws, stream), "gmm_mx4_quantize_rhs")
    return wq, ws


def _need_mx4(on, xq, xs, wq, ws, group_sizes, M, K2, G, Nw):
    _need("xq", xq, on, torch.uint8, M, K2)
    _here(on)
    _need("xs", xs, on, torch.uint8, K2 // 64, M, 4, flat=True)
    _need("wq", wq, on, torch.uint8, G, Nw, K2)
    _need("ws", ws, on, torch.uint8, G, Nw // 128, K2 // 64, 512, flat=True)
    _need_sizes(group_sizes, on, G)


def mx4_fwd(xq, xs, wq, ws, group_sizes, fuse=False, out=None, workspace=None, stream=None):
    """MXFP4 x MXFP4 grouped product -> bf16 [M, N] (fuse: silu(gate) * up, wq holding gate | up)."""
    if stream is not None and (other := _other(stream)):
        with other:
            return mx4_fwd(xq, xs, wq, ws, group_sizes, fuse, out, workspace, stream)
    M, K2 = xq.shape
    G, Nw, K3 = wq.shape
    assert K3 == K2
    N = Nw // 2 if fuse else Nw
    on = xq.get_device()
    _need_mx4(on, xq, xs, wq, ws, group_sizes, M, K2, G, Nw)
    if out is not None:
        _need("out", out, on, torch.bfloat16, M, N)
    else:
        out = _new2(M, N, torch.bfloat16, xq.device)
    ws_ = _ws_on(on, group_sizes, workspace, G, M, xq.device)
    _check(gmm_mx4_fwd(xq, xs, wq, ws, group_sizes, G, M, 2 * K2, N, fuse, out, ws_.buf, ws_.nbytes, stream),
           "gmm_mx4_fwd")
    return out


def mx4_fwd_swiglu_quant(xq, xs, wq, ws, group_sizes, with_h=True, workspace=None, stream=None, out=None):
    """Fused gate/up product: (h bf16 [M, N] or None, hq, hs), hq and hs being h in MXFP4.
    out: an (h, hq, hs) triple to write into instead of new tensors."""
    if stream is not None and (other := _other(stream)):
        with other:
            return mx4_fwd_swiglu_quant(xq, xs, wq, ws, group_sizes, with_h, workspace, stream, out)
    M, K2 = xq.shape
    G, Nw, K3 = wq.shape
    assert K3 == K2
    N = Nw // 2
    on = xq.get_device()
    _need_mx4(on, xq, xs, wq, ws, group_sizes, M, K2, G, Nw)
    if out is not None:
        h, hq, hs = out
        if h is not None:
            _need("out h", h, on, torch.bfloat16, M, N)
        _need("out hq", hq, on, torch.uint8, M, N // 2)
        _need("out hs", hs, on, torch.uint8, N // 128, M, 4, flat=True)
    else:
        h = _new2(M, N, torch.bfloat16, xq.device) if with_h else None
        hq = _new2(M, N // 2, torch.uint8, xq.device)
        hs = _new3(N // 128, M, 4, torch.uint8, xq.device)
    ws_ = _ws_on(on, group_sizes, workspace, G, M, xq.device)
    _check(gmm_mx4_fwd_swiglu_quant(xq, xs, wq, ws, group_sizes, G, M, 2 * K2, N, h, hq, hs, ws_.buf, ws_.nbytes,
                                    stream), "gmm_mx4_fwd_swiglu_quant")
    return h, hq, hs


# ---------------------------------------------------------------------------
# around the experts: router, sorted rows, norms, clipping
# ---------------------------------------------------------------------------

_SCORES = {"softmax": 0, "sigmoid": 1}


def _type_of(what, t):
    """gmm_type of a tensor that may be bf16 or fp32."""
    if t.dtype is torch.bfloat16:
        return 0
    if t.dtype is torch.float32:
        return 1
    raise ValueError(f"{what}: expected bfloat16 or float32 elements, got {t.dtype}")


def _score_of(score):
    if score not in _SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return _SCORES[score]


def _new1(a, dtype, device):
    return torch.empty_strided((a,), (1,), dtype=dtype, device=device)


def route(logits, top_k, bias=None, score="softmax", renorm=False, scale=1.0, stream=None, out=None):
    """The top_k experts of each token and their weights: logits bf16 or float32
    [T, E] -> (ids int32 [T, top_k], weights float32 [T, top_k]), largest logit +
    bias (float32 [E]) first, ties to the lower id; -1 and 0 where fewer than top_k
    are above -inf.  The weights are the softmax or sigmoid of the logits without
    the bias (renorm: divided by the chosen ones' sum) times scale.
    out: an (ids, weights) pair to write into instead of new tensors."""
    if stream is not None and (other := _other(stream)):
        with other:
            return route(logits, top_k, bias, score, renorm, scale, stream, out)
    T, E = logits.shape
    kind, how, on = _type_of("logits", logits), _score_of(score), logits.get_device()
    _need("logits", logits, on, logits.dtype, T, E)
    _here(on)
    if bias is not None:
        _need("bias", bias, on, torch.float32, E)
    if out is not None:
        ids, weights = out
        _need("out ids", ids, on, torch.int32, T, top_k)
        _need("out weights", weights, on, torch.float32, T, top_k)
    else:
        ids = _new2(T, top_k, torch.int32, logits.device)
        weights = _new2(T, top_k, torch.float32, logits.device)
    _check(gmm_route(logits, kind, bias, T, E, top_k, how, renorm, scale, ids, weights, stream), "gmm_route")
    return ids, weights


def route_bwd(dweights, logits, ids, score="softmax", renorm=False, scale=1.0, stream=None, out=None):
    """Its gradient, the choice held fixed: dweights float32 [T, k], logits and ids
    as in the forward -> dlogits [T, E], of the logits' type.  out: a tensor for it."""
    if stream is not None and (other := _other(stream)):
        with other:
            return route_bwd(dweights, logits, ids, score, renorm, scale, stream, out)
    T, E = logits.shape
    T2, k = ids.shape
    assert T2 == T
    kind, how, on = _type_of("logits", logits), _score_of(score), logits.get_device()
    _need("logits", logits, on, logits.dtype, T, E)
    _here(on)
    _need("ids", ids, on, torch.int32, T, k)
    _need("dweights", dweights, on, torch.float32, T, k)
    if out is not None:
        _need("out", out, on, logits.dtype, T, E)
    else:
        out = _new2(T, E, logits.dtype, logits.device)
    _check(gmm_route_bwd(dweights, logits, kind, ids, T, E, k, how, renorm, scale, out, stream), "gmm_route_bwd")
    return out


def sort_rows(ids, G, stream=None, out=None):
    """Places of the choices among the rows sorted by expert: ids int32 [T, k] (or
    [N]) -> (rows int32 of ids' shape, group_sizes int32 [G]).  Group g holds the
    choices of expert g in their order; an id outside 0..G-1 belongs to no group: its
    row r lies behind them, and rows holds -1 - r.
    out: a (rows, group_sizes) pair to write into instead of new tensors."""
    if stream is not None and (other := _other(stream)):
        with other:
            return sort_rows(ids, G, stream, out)
    N, on = ids.numel(), ids.get_device()
    _need("ids", ids, on, torch.int32, N)
    _here(on)
    if out is not None:
        rows, sizes = out
        _need("out rows", rows, on, torch.int32, *ids.shape)
        _need("out group_sizes", sizes, on, torch.int32, G)
    else:
        rows = torch.empty_strided(ids.shape, ids.stride(), dtype=torch.int32, device=ids.device)
        sizes = _new1(G, torch.int32, ids.device)
    nbytes = gmm_sort_rows_scratch_bytes(N, G)
    scratch = _new1(nbytes, torch.uint8, ids.device) if nbytes else None
    _check(gmm_sort_rows(ids, N, G, rows, sizes, scratch, nbytes, stream), "gmm_sort_rows")
    return rows, sizes


def _need_rows(rows, on):
    T, k = rows.shape
    _need("rows", rows, on, torch.int32, T, k)
    return T, k


def gather_rows(x, rows, stream=None, out=None):
    """x bf16 [T, K] by token, rows int32 [T, k] (sort_rows) -> bf16 [T k, K]: each
    token's row at the places of its choices, zeros behind the groups."""
    if stream is not None and (other := _other(stream)):
        with other:
            return gather_rows(x, rows, stream, out)
    on = x.get_device()
    T, k = _need_rows(rows, on)
    T2, K = x.shape
    assert T2 == T
    _need("x", x, on, torch.bfloat16, T, K)
    _here(on)
    if out is not None:
        _need("out", out, on, torch.bfloat16, T * k, K)
    else:
        out = _new2(T * k, K, torch.bfloat16, x.device)
    _check(gmm_gather_rows(x, rows, T, k, K, out, stream), "gmm_gather_rows")
    return out


def gather_quantize(x, rows, stream=None, out=None):
    """quantize_lhs(gather_rows(x, rows)) in one pass: (xq uint8 [T k, K] e4m3 codes,
    xs float32 [K/128, T k]).  out: an (xq, xs) pair to write into."""
    if stream is not None and (other := _other(stream)):
        with other:
            return gather_quantize(x, rows, stream, out)
    on = x.get_device()
    T, k = _need_rows(rows, on)
    T2, K = x.shape
    assert T2 == T
    _need("x", x, on, torch.bfloat16, T, K)
    _here(on)
    if out is not None:
        xq, xs = out
        _need("out codes", xq, on, torch.uint8, T * k, K)
        _need("out scales", xs, on, torch.float32, K // 128, T * k)
    else:
        xq = _new2(T * k, K, torch.uint8, x.device)
        xs = _new2(K // 128, T * k, torch.float32, x.device)
    _check(gmm_gather_quantize(x, rows, T, k, K, xq, xs, stream), "gmm_gather_quantize")
    return xq, xs


def combine_rows(y, rows, weights=None, stream=None, out=None):
    """The sorted rows joined by token: y bf16 [T k, K], rows int32 [T, k], weights
    float32 [T, k] (None: 1 each, the gradient of gather_rows) -> bf16 [T, K]."""
    if stream is not None and (other := _other(stream)):
        with other:
            return combine_rows(y, rows, weights, stream, out)
    on = y.get_device()
    T, k = _need_rows(rows, on)
    K = y.shape[1]
    _need("y", y, on, torch.bfloat16, T * k, K)
    _here(on)
    if weights is not None:
        _need("weights", weights, on, torch.float32, T, k)
    if out is not None:
        _need("out", out, on, torch.bfloat16, T, K)
    else:
        out = _new2(T, K, torch.bfloat16, y.device)
    _check(gmm_combine_rows(y, rows, weights, T, k, K, out, stream), "gmm_combine_rows")
    return out


def combine_rows_bwd(dout, y, rows, weights, stream=None, out=None):
    """Its gradient: dout bf16 [T, K], the forward's y, rows and weights -> (dy bf16
    [T k, K], dweights float32 [T, k]).  out: a (dy, dweights) pair to write into."""
    if stream is not None and (other := _other(stream)):
        with other:
            return combine_rows_bwd(dout, y, rows, weights, stream, out)
    on = dout.get_device()
    T, k = _need_rows(rows, on)
    T2, K = dout.shape
    assert T2 == T
    _need("dout", dout, on, torch.bfloat16, T, K)
    _here(on)
    _need("y", y, on, torch.bfloat16, T * k, K)
    _need("weights", weights, on, torch.float32, T, k)
    if out is not None:
        dy, dweights = out
        _need("out dy", dy, on, torch.bfloat16, T * k, K)
        _need("out dweights", dweights, on, torch.float32, T, k)
    else:
        dy = _new2(T * k, K, torch.bfloat16, dout.device)
        dweights = _new2(T, k, torch.float32, dout.device)
    _check(gmm_combine_rows_bwd(dout, y, rows, weights, T, k, K, dy, dweights, stream), "gmm_combine_rows_bwd")
    return dy, dweights


def _need_join(on, T, K, b, w_post, gate, w_next):
    """Checks what the norms' two directions share; whether the gate has a row per token."""
    if b is not None:
        _need("b", b, on, torch.bfloat16, T, K)
    elif w_post is not None or gate is not None:
        raise ValueError("w_post and gate apply to the block's output: pass b")
    if w_post is not None:
        _need("w_post", w_post, on, torch.float32, K)
    if w_next is not None:
        _need("w_next", w_next, on, torch.float32, K)
    if gate is None:
        return False
    if gate.dim() == 2:
        _need("gate", gate, on, torch.bfloat16, T, K)
        return True
    _need("gate", gate, on, torch.float32, K)
    return False


def norm_join(x, b=None, w_post=None, gate=None, w_next=None, residual_scale=1.0, block_scale=1.0, eps=1e-6,
              stream=None, out=None):
    """The norms before and after a block, its gate and the residual stream:
        out = residual_scale * x + block_scale * gate * (norm(b) * w_post),
        n = norm(out) * w_next,  norm(v) = v / sqrt(mean(v^2) + eps)
    x bf16 or float32 [T, K]; b bf16 [T, K]; w_post, w_next float32 [K]; gate
    float32 [K] or bf16 [T, K] -> (out, of x's type; n bf16).  Without w_post b is
    not normed, without gate it is 1, without w_next n is None; without b, out is x
    and n the norm in front of a first block.
    out: an (out, n) pair to write into instead of new tensors (out may be x, n b)."""
    if stream is not None and (other := _other(stream)):
        with other:
            return norm_join(x, b, w_post, gate, w_next, residual_scale, block_scale, eps, stream, out)
    T, K = x.shape
    kind, on = _type_of("x", x), x.get_device()
    _need("x", x, on, x.dtype, T, K)
    _here(on)
    full = _need_join(on, T, K, b, w_post, gate, w_next)
    if b is None and w_next is None:
        raise ValueError("without b and w_next there is nothing to compute")
    if out is not None:
        o, n = out
        if b is not None:
            _need("out", o, on, x.dtype, T, K)
        if w_next is not None:
            _need("out n", n, on, torch.bfloat16, T, K)
    else:
        o = x if b is None else _new2(T, K, x.dtype, x.device)
        n = None if w_next is None else _new2(T, K, torch.bfloat16, x.device)
    _check(gmm_norm_join(x, kind, b, w_post, gate, full, w_next, T, K, residual_scale, block_scale, eps,
                         None if b is None else o, n, stream), "gmm_norm_join")
    return (x if b is None else o), n


def norm_join_bwd(dout, dn, out, b=None, w_post=None, gate=None, w_next=None, residual_scale=1.0, block_scale=1.0,
                  eps=1e-6, stream=None, into=None):
    """Its gradient: dout (of out, and of its type) and dn (of n, bf16), one of which
    may be None (zero); out as the forward gave it; the other arguments as in the
    forward -> (dx of out's type, db bf16, dw_post float32 [K], dgate of the gate's
    shape and type, dw_next float32 [K]), None for what the forward was not given.
    into: a (dx, db) pair to write into instead of new tensors (dx may be dout, db dn or b)."""
    if stream is not None and (other := _other(stream)):
        with other:
            return norm_join_bwd(dout, dn, out, b, w_post, gate, w_next, residual_scale, block_scale, eps, stream,
                                 into)
    T, K = out.shape
    kind, on = _type_of("out", out), out.get_device()
    _need("out", out, on, out.dtype, T, K)
    _here(on)
    if dout is None and dn is None:
        raise ValueError("one of dout and dn must be given")
    if dout is not None:
        _need("dout", dout, on, out.dtype, T, K)
    if dn is not None:
        _need("dn", dn, on, torch.bfloat16, T, K)
        if w_next is None:
            raise ValueError("dn is the gradient of n: pass w_next")
    full = _need_join(on, T, K, b, w_post, gate, w_next)
    dx = db = dw_post = dgate = dw_next = None
    if into is not None:
        dx, db = into
        _need("into dx", dx, on, out.dtype, T, K)
        if b is not None:
            _need("into db", db, on, torch.bfloat16, T, K)
    else:
        dx = _new2(T, K, out.dtype, out.device)
        db = None if b is None else _new2(T, K, torch.bfloat16, out.device)
    if w_post is not None:
        dw_post = _new1(K, torch.float32, out.device)
    if gate is not None:
        dgate = _new2(T, K, torch.bfloat16, out.device) if full else _new1(K, torch.float32, out.device)
    if w_next is not None:
        dw_next = _new1(K, torch.float32, out.device)
    nbytes = gmm_norm_join_bwd_scratch_bytes(T, K)
    scratch = _new1(nbytes, torch.uint8, out.device) if nbytes else None
    _check(gmm_norm_join_bwd(dout, dn, out, kind, b, w_post, gate, full, w_next, T, K, residual_scale, block_scale,
                             eps, dx, None if b is None else db, dw_post, dgate, dw_next, scratch, nbytes, stream),
           "gmm_norm_join_bwd")
    return dx, (None if b is None else db), dw_post, dgate, dw_next


def clip_grads(grads, max_norm, out=None, stream=None):
    """Gradients scaled by min(1, max_norm / norm), norm being the root of the sum of
    all their squares, in place or into the tensors of `out` -> norm, float32 [1].
    grads: contiguous bf16 or float32 tensors of any shapes.  A norm that is not
    finite scales nothing; max_norm = math.inf computes the norm only."""
    if stream is not None and (other := _other(stream)):
        with other:
            return clip_grads(grads, max_norm, out, stream)
    grads = list(grads)
    n = len(grads)
    if out is not None and len(out) != n:
        raise ValueError(f"out: expected {n} tensors, got {len(out)}")
    device = grads[0].device if n else torch.device("cuda", torch.cuda.current_device())
    on = grads[0].get_device() if n else device.index
    types, counts = array.array("i"), array.array("q")
    for i, g in enumerate(grads):
        types.append(_type_of(f"grads[{i}]", g))
        counts.append(g.numel())
        if not g.is_contiguous() or g.get_device() != on or on < 0:
            _need(f"grads[{i}]", g, on, g.dtype, *g.shape)
        if out is not None and (out[i].dtype is not g.dtype or out[i].shape != g.shape or
                                not out[i].is_contiguous() or out[i].get_device() != on):
            _need(f"out[{i}]", out[i], on, g.dtype, *g.shape)
    _here(on)
    src = array.array("Q", [g.data_ptr() for g in grads])
    dst = None if out is None else array.array("Q", [o.data_ptr() for o in out])
    norm = _new1(1, torch.float32, device)
    nbytes = gmm_clip_grads_scratch_bytes(n)
    scratch = _new1(nbytes, torch.uint8, device) if nbytes else None
    _check(gmm_clip_grads(src.buffer_info()[0], dst.buffer_info()[0] if dst else None, counts.buffer_info()[0],
                          types.buffer_info()[0], n, max_norm, norm, scratch, nbytes, stream), "gmm_clip_grads")
    return norm
