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
            "tgmm_fp8_ckpt", "tgmm_fp8_ckpt_scratch_bytes", "gmm_mx4_quantize_lhs", "gmm_mx4_quantize_rhs",
            "gmm_mx4_fwd", "gmm_mx4_fwd_swiglu_quant", "gmm_route", "gmm_route_bwd", "gmm_sort_rows_scratch_bytes",
            "gmm_sort_rows", "gmm_gather_rows", "gmm_gather_quantize", "gmm_gather_mx4_quantize", "gmm_combine_rows",
            "gmm_combine_rows_bwd", "gmm_norm_join", "gmm_norm_join_bwd_scratch_bytes", "gmm_norm_join_bwd",
            "gmm_clip_grads_scratch_bytes", "gmm_clip_grads"]


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
    lib.gmm_gather_mx4_quantize.restype = I
    lib.gmm_gather_mx4_quantize.argtypes = [P, P, I64, I, I64, P, P, P]
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
    lib.gmm_clip_grads_scratch_bytes.argtypes = [I, I64]
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


def gmm_gather_mx4_quantize(x, rows, T, k, K, xq, xs, stream=None) -> int:
    return load().gmm_gather_mx4_quantize(_p(x), _p(rows), T, k, K, _p(xq), _p(xs), _s(stream))


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


def gmm_clip_grads_scratch_bytes(n: int, total: int) -> int:
    return int(load().gmm_clip_grads_scratch_bytes(n, total))


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

# These calls are short (a few microseconds of device time for a decoding step), so
# their wrappers look at each operand once and hand the library plain numbers.

_SCORES = {"softmax": 0, "sigmoid": 1}
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_empty, _like = torch.empty_strided, torch.empty_like  # _like takes a little less time
_current_device = torch._C._cuda_getDevice
_data_ptr, _is_contiguous, _get_device = torch.Tensor.data_ptr, torch.Tensor.is_contiguous, torch.Tensor.get_device


def _type_of(what, t):
    """gmm_type of a tensor that may be bf16 or fp32."""
    dtype = t.dtype
    if dtype is _BF16:
        return 0
    if dtype is _F32:
        return 1
    raise ValueError(f"{what}: expected bfloat16 or float32 elements, got {dtype}")


def _score_of(score):
    how = _SCORES.get(score)
    if how is None:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return how


def _want(what, t, on, dtype, shape):
    """_need for one exact shape (a tuple)."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != on:
        _refuse(what, t, on, dtype, shape)


def _refuse(what, t, on, dtype, shape):
    where = "" if on < 0 else f" on cuda:{on}"
    raise ValueError(f"{what}: expected a contiguous CUDA tensor of {'x'.join(map(str, shape))} {dtype} elements"
                     f"{where}, got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _first(what, t, dtype):
    """Checks a call's first tensor, whose shape and device the others have to fit; returns its device."""
    on = t.get_device()
    if on < 0 or t.dtype is not dtype or not t.is_contiguous():
        _refuse(what, t, on, dtype, t.shape)
    return on


def _handle(on, stream):
    """The raw stream of a launch on device `on`, which has to be the current one."""
    dev = _current_device()
    if dev != on:
        raise ValueError(f"the tensors are on cuda:{on}, the current device is cuda:{dev}")
    return torch._C._cuda_getCurrentRawStream(on) if stream is None else _s(stream)


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
    kind, how = _type_of("logits", logits), _score_of(score)
    on = _first("logits", logits, logits.dtype)
    if bias is not None:
        _want("bias", bias, on, _F32, (E,))
    handle = _handle(on, stream)
    if out is None:
        if top_k < 1:
            raise ValueError(f"top_k must be at least 1, got {top_k}")
        device = logits.device
        ids = _empty((T, top_k), (top_k, 1), dtype=_I32, device=device)
        weights = _empty((T, top_k), (top_k, 1), dtype=_F32, device=device)
    else:
        ids, weights = out
        _want("out ids", ids, on, _I32, (T, top_k))
        _want("out weights", weights, on, _F32, (T, top_k))
    status = (_lib or load()).gmm_route(logits.data_ptr(), kind, None if bias is None else bias.data_ptr(), T, E, top_k,
                                        how, bool(renorm), scale, ids.data_ptr(), weights.data_ptr(), handle)
    if status:
        raise GmmError(status, "gmm_route")
    return ids, weights


def route_bwd(dweights, logits, ids, score="softmax", renorm=False, scale=1.0, stream=None, out=None):
    """Its gradient, the choice held fixed: dweights float32 [T, k], logits and ids
    as in the forward -> dlogits [T, E], of the logits' type.  out: a tensor for it."""
    if stream is not None and (other := _other(stream)):
        with other:
            return route_bwd(dweights, logits, ids, score, renorm, scale, stream, out)
    T, E = logits.shape
    k = ids.shape[-1]
    dtype = logits.dtype
    kind, how = _type_of("logits", logits), _score_of(score)
    on = _first("logits", logits, dtype)
    _want("ids", ids, on, _I32, (T, k))
    _want("dweights", dweights, on, _F32, (T, k))
    handle = _handle(on, stream)
    if out is None:
        out = _like(logits)
    else:
        _want("out", out, on, dtype, (T, E))
    status = (_lib or load()).gmm_route_bwd(dweights.data_ptr(), logits.data_ptr(), kind, ids.data_ptr(), T, E, k, how,
                                            bool(renorm), scale, out.data_ptr(), handle)
    if status:
        raise GmmError(status, "gmm_route_bwd")
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
    on, shape, N = _first("ids", ids, _I32), ids.shape, ids.numel()
    handle = _handle(on, stream)
    if out is None:
        if G < 1:
            raise ValueError(f"G must be at least 1, got {G}")
        rows = _like(ids)
        sizes = _empty((G,), (1,), dtype=_I32, device=ids.device)
    else:
        rows, sizes = out
        _want("out rows", rows, on, _I32, shape)
        _want("out group_sizes", sizes, on, _I32, (G,))
    lib = _lib or load()
    nbytes = lib.gmm_sort_rows_scratch_bytes(N, G)
    scratch = _empty((nbytes,), (1,), dtype=torch.uint8, device=ids.device) if nbytes else None
    status = lib.gmm_sort_rows(ids.data_ptr(), N, G, rows.data_ptr(), sizes.data_ptr(),
                               None if scratch is None else scratch.data_ptr(), nbytes, handle)
    if status:
        raise GmmError(status, "gmm_sort_rows")
    return rows, sizes


def gather_rows(x, rows, stream=None, out=None):
    """x bf16 [T, K] by token, rows int32 [T, k] (sort_rows) -> bf16 [T k, K]: each
    token's row at the places of its choices, zeros behind the groups."""
    if stream is not None and (other := _other(stream)):
        with other:
            return gather_rows(x, rows, stream, out)
    T, K = x.shape
    k = rows.shape[-1]
    on = _first("x", x, _BF16)
    _want("rows", rows, on, _I32, (T, k))
    handle = _handle(on, stream)
    if out is None:
        out = _empty((T * k, K), (K, 1), dtype=_BF16, device=x.device)
    else:
        _want("out", out, on, _BF16, (T * k, K))
    status = (_lib or load()).gmm_gather_rows(x.data_ptr(), rows.data_ptr(), T, k, K, out.data_ptr(), handle)
    if status:
        raise GmmError(status, "gmm_gather_rows")
    return out


def gather_quantize(x, rows, stream=None, out=None):
    """quantize_lhs(gather_rows(x, rows)) in one pass: (xq uint8 [T k, K] e4m3 codes,
    xs float32 [K/128, T k]).  out: an (xq, xs) pair to write into."""
    if stream is not None and (other := _other(stream)):
        with other:
            return gather_quantize(x, rows, stream, out)
    T, K = x.shape
    k = rows.shape[-1]
    on, M = _first("x", x, _BF16), T * k
    _want("rows", rows, on, _I32, (T, k))
    handle = _handle(on, stream)
    if out is None:
        device = x.device
        xq = _empty((M, K), (K, 1), dtype=torch.uint8, device=device)
        xs = _empty((K // 128, M), (M, 1), dtype=_F32, device=device)
    else:
        xq, xs = out
        _want("out codes", xq, on, torch.uint8, (M, K))
        _want("out scales", xs, on, _F32, (K // 128, M))
    status = (_lib or load()).gmm_gather_quantize(x.data_ptr(), rows.data_ptr(), T, k, K, xq.data_ptr(), xs.data_ptr(),
                                                  handle)
    if status:
        raise GmmError(status, "gmm_gather_quantize")
    return xq, xs


def gather_mx4_quantize(x, rows, stream=None, out=None):
    """mx4_quantize_lhs(gather_rows(x, rows)) in one pass: (xq uint8 [T k, K/2] packed
    E2M1 codes, xs uint8 [K/128, T k, 4] E8M0 scales).  out: an (xq, xs) pair to write into."""
    if stream is not None and (other := _other(stream)):
        with other:
            return gather_mx4_quantize(x, rows, stream, out)
    T, K = x.shape
    k = rows.shape[-1]
    on, M, KB = _first("x", x, _BF16), T * k, K // 128
    _want("rows", rows, on, _I32, (T, k))
    handle = _handle(on, stream)
    if out is None:
        device = x.device
        xq = _empty((M, K // 2), (K // 2, 1), dtype=torch.uint8, device=device)
        xs = _empty((KB, M, 4), (4 * M, 4, 1), dtype=torch.uint8, device=device)
    else:
        xq, xs = out
        _want("out codes", xq, on, torch.uint8, (M, K // 2))
        _want("out scales", xs, on, torch.uint8, (KB, M, 4))
    status = (_lib or load()).gmm_gather_mx4_quantize(x.data_ptr(), rows.data_ptr(), T, k, K, xq.data_ptr(),
                                                      xs.data_ptr(), handle)
    if status:
        raise GmmError(status, "gmm_gather_mx4_quantize")
    return xq, xs


def combine_rows(y, rows, weights=None, stream=None, out=None):
    """The sorted rows joined by token: y bf16 [T k, K], rows int32 [T, k], weights
    float32 [T, k] (None: 1 each, the gradient of gather_rows) -> bf16 [T, K]."""
    if stream is not None and (other := _other(stream)):
        with other:
            return combine_rows(y, rows, weights, stream, out)
    T, k = rows.shape
    K = y.shape[-1]
    on = _first("rows", rows, _I32)
    _want("y", y, on, _BF16, (T * k, K))
    if weights is not None:
        _want("weights", weights, on, _F32, (T, k))
    handle = _handle(on, stream)
    if out is None:
        out = _empty((T, K), (K, 1), dtype=_BF16, device=y.device)
    else:
        _want("out", out, on, _BF16, (T, K))
    status = (_lib or load()).gmm_combine_rows(y.data_ptr(), rows.data_ptr(),
                                               None if weights is None else weights.data_ptr(), T, k, K, out.data_ptr(),
                                               handle)
    if status:
        raise GmmError(status, "gmm_combine_rows")
    return out


def combine_rows_bwd(dout, y, rows, weights, stream=None, out=None):
    """Its gradient: dout bf16 [T, K], the forward's y, rows and weights -> (dy bf16
    [T k, K], dweights float32 [T, k]).  out: a (dy, dweights) pair to write into."""
    if stream is not None and (other := _other(stream)):
        with other:
            return combine_rows_bwd(dout, y, rows, weights, stream, out)
    T, K = dout.shape
    k = rows.shape[-1]
    on, M = _first("dout", dout, _BF16), T * k
    _want("y", y, on, _BF16, (M, K))
    _want("rows", rows, on, _I32, (T, k))
    _want("weights", weights, on, _F32, (T, k))
    handle = _handle(on, stream)
    if out is None:
        dy = _like(y)
        dweights = _like(weights)
    else:
        dy, dweights = out
        _want("out dy", dy, on, _BF16, (M, K))
        _want("out dweights", dweights, on, _F32, (T, k))
    status = (_lib or load()).gmm_combine_rows_bwd(dout.data_ptr(), y.data_ptr(), rows.data_ptr(), weights.data_ptr(),
                                                   T, k, K, dy.data_ptr(), dweights.data_ptr(), handle)
    if status:
        raise GmmError(status, "gmm_combine_rows_bwd")
    return dy, dweights


def _need_join(on, T, K, b, w_post, gate, w_next):
    """Checks what the norms' two directions share; whether the gate has a row per token."""
    if b is not None:
        _want("b", b, on, _BF16, (T, K))
    elif w_post is not None or gate is not None:
        raise ValueError("w_post and gate apply to the block's output: pass b")
    if w_post is not None:
        _want("w_post", w_post, on, _F32, (K,))
    if w_next is not None:
        _want("w_next", w_next, on, _F32, (K,))
    if gate is None:
        return False
    if gate.dim() == 2:
        _want("gate", gate, on, _BF16, (T, K))
        return True
    _want("gate", gate, on, _F32, (K,))
    return False


def _at(t):
    return None if t is None else t.data_ptr()


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
    dtype = x.dtype
    kind, on = _type_of("x", x), _first("x", x, dtype)
    full = _need_join(on, T, K, b, w_post, gate, w_next)
    if b is None and w_next is None:
        raise ValueError("without b and w_next there is nothing to compute")
    handle = _handle(on, stream)
    if out is None:
        o = x if b is None else _like(x)
        n = None
        if w_next is not None:
            n = _like(b) if b is not None else _empty((T, K), (K, 1), dtype=_BF16, device=x.device)
    else:
        o, n = out
        if b is None:
            o = x
        else:
            _want("out", o, on, dtype, (T, K))
        if w_next is None:
            n = None  # nothing is written to it
        else:
            _want("out n", n, on, _BF16, (T, K))
    status = (_lib or load()).gmm_norm_join(x.data_ptr(), kind, _at(b), _at(w_post), _at(gate), full, _at(w_next), T, K,
                                            residual_scale, block_scale, eps, None if b is None else o.data_ptr(),
                                            _at(n), handle)
    if status:
        raise GmmError(status, "gmm_norm_join")
    return o, n


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
    dtype = out.dtype
    kind, on = _type_of("out", out), _first("out", out, dtype)
    if dout is not None:
        _want("dout", dout, on, dtype, (T, K))
    elif dn is None:
        raise ValueError("one of dout and dn must be given")
    if dn is not None:
        _want("dn", dn, on, _BF16, (T, K))
        if w_next is None:
            raise ValueError("dn is the gradient of n: pass w_next")
    full = _need_join(on, T, K, b, w_post, gate, w_next)
    handle = _handle(on, stream)
    if into is None:
        dx = _like(out)
        db = None if b is None else _like(b)
    else:
        dx, db = into
        _want("into dx", dx, on, dtype, (T, K))
        if b is None:
            db = None
        else:
            _want("into db", db, on, _BF16, (T, K))
    dw_post = None if w_post is None else _like(w_post)
    dw_next = None if w_next is None else _like(w_next)
    dgate = None if gate is None else _like(gate)
    lib = _lib or load()
    nbytes = lib.gmm_norm_join_bwd_scratch_bytes(T, K)
    scratch = _empty((nbytes,), (1,), dtype=torch.uint8, device=out.device) if nbytes else None
    status = lib.gmm_norm_join_bwd(_at(dout), _at(dn), out.data_ptr(), kind, _at(b), _at(w_post), _at(gate), full,
                                   _at(w_next), T, K, residual_scale, block_scale, eps, dx.data_ptr(), _at(db),
                                   _at(dw_post), _at(dgate), _at(dw_next), _at(scratch), nbytes, handle)
    if status:
        raise GmmError(status, "gmm_norm_join_bwd")
    return dx, db, dw_post, dgate, dw_next


def clip_grads(grads, max_norm, out=None, stream=None):
    """Gradients scaled by min(1, max_norm / norm), norm being the root of the sum of
    all their squares, in place or into the tensors of `out` (of the same types and
    numbers of elements) -> norm, float32 [1].  grads: contiguous bf16 or float32
    tensors of any shapes.  A norm that is not finite scales nothing; max_norm =
    math.inf computes the norm only."""
    if stream is not None and (other := _other(stream)):
        with other:
            return clip_grads(grads, max_norm, out, stream)
    grads = list(grads)
    n = len(grads)
    if out is not None and len(out) != n:
        raise ValueError(f"out: expected {n} tensors, got {len(out)}")
    on = grads[0].get_device() if n else _current_device()
    dtypes, counts = _flat_tensors("grads", grads, on)
    if out is not None:
        if _flat_tensors("out", out, on) != (dtypes, counts):
            raise ValueError("out: expected tensors of the gradients' types and numbers of elements")
        dst = array.array("Q", list(map(_data_ptr, out)))
    handle = _handle(on, stream)
    src = array.array("Q", list(map(_data_ptr, grads)))
    types = array.array("i", [d is _F32 for d in dtypes])
    counts = array.array("q", counts)
    device = grads[0].device if n else torch.device("cuda", on)
    lib = _lib or load()
    norm = _empty((1,), (1,), dtype=_F32, device=device)
    nbytes = lib.gmm_clip_grads_scratch_bytes(n, sum(counts))
    scratch = _empty((nbytes,), (1,), dtype=torch.uint8, device=device) if nbytes else None
    status = lib.gmm_clip_grads(src.buffer_info()[0], None if out is None else dst.buffer_info()[0],
                                counts.buffer_info()[0], types.buffer_info()[0], n, max_norm, norm.data_ptr(),
                                _at(scratch), nbytes, handle)
    if status:
        raise GmmError(status, "gmm_clip_grads")
    return norm


def _flat_tensors(what, tensors, on):
    """Types and numbers of elements of contiguous bf16 or fp32 tensors on device `on`."""
    dtypes = [t.dtype for t in tensors]
    if not (all(map(_is_contiguous, tensors)) and set(map(_get_device, tensors)) <= {on} and on >= 0
            and dtypes.count(_BF16) + dtypes.count(_F32) == len(dtypes)):
        for i, t in enumerate(tensors):
            _type_of(f"{what}[{i}]", t)
            _want(f"{what}[{i}]", t, on, t.dtype, t.shape)
            if on < 0:
                _refuse(f"{what}[{i}]", t, on, t.dtype, t.shape)
    return dtypes, [t.numel() for t in tensors]
