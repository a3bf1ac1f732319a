"""Python binding of libminite.so (include/minite.h) through ctypes.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. PyTorch provides device memory and streams. The functions named
``minite_*`` mirror the C entry points one to one and take torch tensors;
the helpers below them only allocate outputs with torch and call those.
Nothing here falls back to a CPU implementation: without the built library
every call raises ``MiniteError``.
"""
from __future__ import annotations

import ctypes
import math
import os
from array import array
from itertools import chain

import numpy as np
import torch

from . import build as _build

SCALE_PER_ROW, SCALE_PER_GROUP = 0, 1
ALONG_COLS, ALONG_ROWS = 0, 1
OUT_BF16, OUT_FP32 = 0, 1
OP_QUANTIZE, OP_PERMUTE_QUANT, OP_COMBINE_BACKWARD_QUANT, OP_QUANTIZE_TOKENS = 0, 1, 2, 3
OP_GATE_UP_SWIGLU, OP_PERMUTE_ROWS, OP_GRAD_NORM, OP_VERIFY_DRAFTS = 4, 5, 6, 7
NORM_2, NORM_MAX = 0, 1
W_NK, W_KN = 0, 1
ERR_TIMEOUT, ERR_BAD_ROUTING, ERR_BAD_TOKEN = 4, 5, 7

EXPORTS = [
    "minite_quantize_nvfp4", "minite_moe_permute_quant", "minite_grouped_gemm_nvfp4",
    "minite_swiglu_weighted_quant", "minite_swiglu_backward_quant", "minite_moe_combine",
    "minite_workspace_bytes",
    "minite_status_string", "minite_version", "minite_test_convert",
    "minite_set_wait_budget_ns", "minite_moe_permute_quant_noalloc", "minite_set_gemm_variant",
    "minite_test_div6_exhaustive", "minite_test_convert_digest", "minite_quantize_nvfp4_dual",
    "minite_moe_combine_backward_quant", "minite_quantize_tokens_nvfp4",
    "minite_swiglu_weighted_quant_keep_h", "minite_grouped_gemm_wgrad_nvfp4",
    "minite_swiglu_backward_quant_keep", "minite_gate_up_swiglu_quant_nvfp4",
    "minite_grouped_gemm_bf16", "minite_grouped_wgrad_bf16", "minite_token_logprobs",
    "minite_token_logprobs_backward", "minite_adamw_step", "minite_test_adamw_math",
    "minite_moe_permute_rows", "minite_moe_spread_rows", "minite_moe_combine_rows",
    "minite_moe_combine_rows_backward", "minite_grad_norm", "minite_clip_grads",
    "minite_verify_drafts",
]


class MiniteError(RuntimeError):
    pass


_LIB = None
_vp, _i64, _i32, _int, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_size_t


def load(path: str | None = None):
    """Load libminite.so (built in-tree by ``build.build()``)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = path or _build.LIB
    if not os.path.exists(path):
        raise MiniteError(f"{path} is not built; run nvfp4_w4a4_moe_permute_gb300.build.build()")
    lib = ctypes.CDLL(path)
    sig = {
        "minite_quantize_nvfp4": [_vp, _i64, _i64, _i64, _int, _int, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp],
        "minite_quantize_nvfp4_dual": [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp,
                                       _vp],
        "minite_moe_permute_quant": [_vp, _vp, _vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                                     _vp, _vp, _vp, _vp, _sz, _vp, _vp],
        "minite_moe_permute_quant_noalloc": [_vp, _vp, _vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp,
                                             _vp, _vp, _vp, _vp, _vp, _vp, _vp],
        "minite_moe_combine_backward_quant": [_vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                                              _vp, _vp, _vp, _sz, _vp, _vp],
        "minite_quantize_tokens_nvfp4": [_vp, _i64, _vp, _vp, _i64, _i64, _i32, _vp, _i64, _vp, _vp,
                                         _vp, _vp, _vp, _sz, _vp, _vp],
        "minite_grouped_gemm_wgrad_nvfp4": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64,
                                            _vp, _int, _vp, _vp],
        "minite_grouped_gemm_nvfp4": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32,
                                      _vp, _int, _vp, _vp],
        "minite_gate_up_swiglu_quant_nvfp4": [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                                              _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp,
                                              _vp],
        "minite_swiglu_weighted_quant": [_vp, _vp, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
        "minite_swiglu_weighted_quant_keep_h": [_vp, _vp, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp,
                                                _vp, _vp, _vp, _vp],
        "minite_swiglu_backward_quant": [_vp, _vp, _vp, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                         _vp],
        "minite_swiglu_backward_quant_keep": [_vp, _vp, _vp, _i64, _i64, _i32, _vp, _vp, _vp, _vp,
                                              _vp, _vp, _vp, _vp, _vp],
        "minite_moe_combine": [_vp, _vp, _i64, _i64, _i64, _i32, _vp, _vp, _vp],
        "minite_grouped_gemm_bf16": [_vp, _i64, _vp, _int, _vp, _i64, _i64, _i64, _i32, _vp, _i64,
                                     _int, _vp, _vp],
        "minite_grouped_wgrad_bf16": [_vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i32, _vp, _int,
                                      _int, _vp, _vp],
        "minite_token_logprobs": [_vp, _int, _i64, _i64, _i64, _vp, _int, ctypes.c_float, _vp, _vp,
                                  _vp, _i32, _vp, _vp, _vp, _vp],
        "minite_token_logprobs_backward": [_vp, _int, _i64, _i64, _i64, _vp, _int, ctypes.c_float,
                                           _vp, _vp, _vp, _vp, _vp, _i64, _vp, _vp],
        "minite_adamw_step": [_vp, _i64, _int, _int, _int] + [ctypes.c_double] * 5 +
                             [_i64, _vp, _vp],
        "minite_moe_permute_rows": [_vp, _int, _i64, _vp, _i64, _i64, _i32, _i32, _vp, _i64, _vp, _vp, _vp,
                                    _vp, _sz, _vp, _vp],
        "minite_moe_spread_rows": [_vp, _int, _i64, _vp, _i64, _i64, _i64, _i32, _vp, _i64, _vp, _vp],
        "minite_moe_combine_rows": [_vp, _int, _i64, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _i64, _vp,
                                    _vp],
        "minite_moe_combine_rows_backward": [_vp, _int, _i64, _vp, _i64, _vp, _vp, _i64, _i64, _i64,
                                             _i32, _vp, _i64, _vp, _vp, _vp],
        "minite_grad_norm": [_vp, _i64, _int, ctypes.c_double, _vp, _vp, _vp, _sz, _vp],
        "minite_clip_grads": [_vp, _i64, _vp, _vp],
        "minite_verify_drafts": [_vp, _int, _i64, _vp, _int, _i64, _vp, _vp, _vp, _i64, _i64, _i32, _i64,
                                 ctypes.c_float, _vp, _vp, _vp, _vp, _sz, _vp, _vp],
        "minite_test_convert": [_vp, _i64, _vp, _vp, _vp, _vp],
        "minite_test_div6_exhaustive": [_vp, _vp],
        "minite_test_adamw_math": [_vp, _vp],
        "minite_test_convert_digest": [ctypes.c_ulonglong, ctypes.c_ulonglong, _vp, _vp],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = _int
    lib.minite_workspace_bytes.argtypes = [_int, _i64, _i64, _i32, _i32]
    lib.minite_workspace_bytes.restype = _sz
    lib.minite_status_string.argtypes = [_int]
    lib.minite_status_string.restype = ctypes.c_char_p
    lib.minite_version.argtypes = []
    lib.minite_version.restype = ctypes.c_char_p
    lib.minite_set_wait_budget_ns.argtypes = [ctypes.c_uint64]
    lib.minite_set_wait_budget_ns.restype = None
    lib.minite_set_gemm_variant.argtypes = [_int]
    lib.minite_set_gemm_variant.restype = None
    _LIB = lib
    return lib


def _current_device():
    """Index of the device that kernels are launched on."""
    return torch._C._cuda_getDevice()


def _elsewhere(what, index, dev):
    return MiniteError(f"expected a CUDA {what} on cuda:{dev}, the current device, got one on "
                       f"{'the CPU' if index < 0 else f'cuda:{index}'}")


def _p(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise MiniteError("expected a CUDA tensor")
    if t.get_device() != _current_device():
        raise _elsewhere("tensor", t.get_device(), _current_device())
    return ctypes.c_void_p(t.data_ptr())


def _s(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    elif stream.device_index != _current_device():
        raise _elsewhere("stream", stream.device_index, _current_device())
    return ctypes.c_void_p(stream.cuda_stream)


def _check(rc: int, name: str):
    if rc != 0:
        raise MiniteError(f"{name}: {minite_status_string(rc)} (status {rc})")


def minite_status_string(rc: int) -> str:
    return load().minite_status_string(rc).decode()


def minite_version() -> str:
    return load().minite_version().decode()


def minite_workspace_bytes(op: int, a: int, b: int = 0, E: int = 0, k: int = 0) -> int:
    return int(load().minite_workspace_bytes(op, a, b, E, k))


def minite_set_wait_budget_ns(ns: int):
    load().minite_set_wait_budget_ns(int(ns))


def minite_set_gemm_variant(variant: int):
    """0 automatic, 1 single-CTA grouped-GEMM kernel, 2 CTA-pair kernel."""
    load().minite_set_gemm_variant(int(variant))


def minite_quantize_nvfp4(x, scale_mode, orientation, codes, sf, gscale_out, gscale_in=None,
                          workspace=None, status=None, stream=None):
    """x: bf16 [groups, rows, cols] (or [rows, cols] = one group)."""
    g, r, c = (1,) + tuple(x.shape) if x.dim() == 2 else tuple(x.shape)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().minite_quantize_nvfp4(_p(x), g, r, c, scale_mode, orientation, _p(gscale_in),
                                      _p(codes), _p(sf), _p(gscale_out), _p(workspace), ws_bytes,
                                      _p(status), _s(stream))
    _check(rc, "minite_quantize_nvfp4")


def minite_quantize_nvfp4_dual(x, codes_k, sf_k, codes_n, sf_n, gscale_out, workspace,
                               status=None, stream=None):
    """x: bf16 [groups, rows, cols] (or [rows, cols] = one group); per-group scales."""
    g, r, c = (1,) + tuple(x.shape) if x.dim() == 2 else tuple(x.shape)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().minite_quantize_nvfp4_dual(_p(x), g, r, c, _p(codes_k), _p(sf_k), _p(codes_n),
                                           _p(sf_n), _p(gscale_out), _p(workspace), ws_bytes,
                                           _p(status), _s(stream))
    _check(rc, "minite_quantize_nvfp4_dual")


def quantize_dual(x, stream=None):
    """Weight x ([rows, cols] or [groups, rows, cols]) quantized per group in both
    orientations; returns (forward dict, transposed dict) like quantize()."""
    dev = x.device
    g3 = x if x.dim() == 3 else x.unsqueeze(0)
    G, R, C = g3.shape
    fk = dict(codes=torch.empty((G, R, C // 2), dtype=torch.uint8, device=dev),
              sf=torch.empty((G, sf_bytes((R + 127) // 128 * 128, C)), dtype=torch.uint8, device=dev))
    fn = dict(codes=torch.empty((G, C, R // 2), dtype=torch.uint8, device=dev),
              sf=torch.empty((G, sf_bytes((C + 127) // 128 * 128, R)), dtype=torch.uint8, device=dev))
    g = torch.empty((G,), dtype=torch.float32, device=dev)
    ws = torch.empty(minite_workspace_bytes(OP_QUANTIZE, G), dtype=torch.uint8, device=dev)
    minite_quantize_nvfp4_dual(g3, fk["codes"], fk["sf"], fn["codes"], fn["sf"], g, ws, stream=stream)
    fk["g"] = g
    fn["g"] = g
    if x.dim() == 2:
        for d in (fk, fn):
            d["codes"], d["sf"] = d["codes"][0], d["sf"][0]
    return fk, fn


def minite_moe_permute_quant(x, topk_ids, topk_w, E, codes, sf, row_g, expert_offsets,
                             sf_row_offsets, perm_src, dest_row, perm_w, workspace, status=None,
                             stream=None):
    T, H = x.shape
    k = topk_ids.shape[1]
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().minite_moe_permute_quant(_p(x), _p(topk_ids), _p(topk_w), T, H, E, k, _p(codes),
                                         _p(sf), _p(row_g), _p(expert_offsets),
                                         _p(sf_row_offsets), _p(perm_src), _p(dest_row),
                                         _p(perm_w), _p(workspace), ws_bytes, _p(status),
                                         _s(stream))
    _check(rc, "minite_moe_permute_quant")


def minite_moe_permute_quant_noalloc(x, topk_ids, topk_w, E, codes, sf, row_g, expert_offsets,
                                     sf_row_offsets, perm_src, dest_row, perm_w, status=None,
                                     stream=None):
    """As minite_moe_permute_quant, with the library's built-in scratch array
    instead of a caller workspace (for callers that cannot allocate)."""
    T, H = x.shape
    k = topk_ids.shape[1]
    rc = load().minite_moe_permute_quant_noalloc(_p(x), _p(topk_ids), _p(topk_w), T, H, E, k,
                                                 _p(codes), _p(sf), _p(row_g), _p(expert_offsets),
                                                 _p(sf_row_offsets), _p(perm_src), _p(dest_row),
                                                 _p(perm_w), _p(status), _s(stream))
    _check(rc, "minite_moe_permute_quant_noalloc")


def minite_grouped_gemm_nvfp4(a_codes, a_sf, a_g, b_codes, b_sf, b_g, expert_offsets,
                              sf_row_offsets, out, status=None, stream=None):
    M, K2 = a_codes.shape
    E, N, _ = b_codes.shape
    out_dtype = OUT_FP32 if out.dtype == torch.float32 else OUT_BF16
    rc = load().minite_grouped_gemm_nvfp4(_p(a_codes), _p(a_sf), _p(a_g), _p(b_codes), _p(b_sf),
                                          _p(b_g), _p(expert_offsets), _p(sf_row_offsets), M, N,
                                          2 * K2, E, _p(out), out_dtype, _p(status), _s(stream))
    _check(rc, "minite_grouped_gemm_nvfp4")


def minite_gate_up_swiglu_quant_nvfp4(a_codes, a_sf, a_g, b_codes, b_sf, b_g, expert_offsets,
                                      sf_row_offsets, perm_w, h_codes, h_sf, h_g, workspace,
                                      gate_up=None, status=None, stream=None):
    """b_codes [E, 2I, K/2]; h_codes [M, I/2]; workspace uint8 of at least
    minite_workspace_bytes(OP_GATE_UP_SWIGLU, M, I, 0, 0) bytes."""
    M, K2 = a_codes.shape
    E, N, _ = b_codes.shape
    rc = load().minite_gate_up_swiglu_quant_nvfp4(
        _p(a_codes), _p(a_sf), _p(a_g), _p(b_codes), _p(b_sf), _p(b_g), _p(expert_offsets),
        _p(sf_row_offsets), M, N // 2, 2 * K2, E, _p(perm_w), _p(gate_up), _p(h_codes), _p(h_sf),
        _p(h_g), _p(workspace), workspace.numel() * workspace.element_size(), _p(status),
        _s(stream))
    _check(rc, "minite_gate_up_swiglu_quant_nvfp4")


def minite_swiglu_weighted_quant(gate_up, perm_w, E, expert_offsets, sf_row_offsets, codes, sf,
                                 row_g, status=None, stream=None):
    M, I2 = gate_up.shape
    rc = load().minite_swiglu_weighted_quant(_p(gate_up), _p(perm_w), M, I2 // 2, E,
                                             _p(expert_offsets), _p(sf_row_offsets), _p(codes),
                                             _p(sf), _p(row_g), _p(status), _s(stream))
    _check(rc, "minite_swiglu_weighted_quant")


def minite_swiglu_weighted_quant_keep_h(gate_up, perm_w, E, expert_offsets, sf_row_offsets, codes,
                                        sf, row_g, h_out, status=None, stream=None, h_amax=None):
    M, I2 = gate_up.shape
    rc = load().minite_swiglu_weighted_quant_keep_h(_p(gate_up), _p(perm_w), M, I2 // 2, E,
                                                    _p(expert_offsets), _p(sf_row_offsets),
                                                    _p(codes), _p(sf), _p(row_g), _p(h_out),
                                                    _p(h_amax), _p(status), _s(stream))
    _check(rc, "minite_swiglu_weighted_quant_keep_h")


def minite_swiglu_backward_quant(gate_up, dh, perm_w, E, expert_offsets, sf_row_offsets, codes,
                                 sf, row_g, status=None, stream=None):
    M, I2 = gate_up.shape
    rc = load().minite_swiglu_backward_quant(_p(gate_up), _p(dh), _p(perm_w), M, I2 // 2, E,
                                             _p(expert_offsets), _p(sf_row_offsets), _p(codes),
                                             _p(sf), _p(row_g), _p(status), _s(stream))
    _check(rc, "minite_swiglu_backward_quant")


def minite_swiglu_backward_quant_keep(gate_up, dh, perm_w, E, expert_offsets, sf_row_offsets,
                                      codes, sf, row_g, dgu_out, status=None, stream=None,
                                      dgu_amax=None):
    M, I2 = gate_up.shape
    rc = load().minite_swiglu_backward_quant_keep(_p(gate_up), _p(dh), _p(perm_w), M, I2 // 2, E,
                                                  _p(expert_offsets), _p(sf_row_offsets),
                                                  _p(codes), _p(sf), _p(row_g), _p(dgu_out),
                                                  _p(dgu_amax), _p(status), _s(stream))
    _check(rc, "minite_swiglu_backward_quant_keep")


def minite_moe_combine_backward_quant(dy, E, dest_row, expert_offsets, sf_row_offsets, perm_src,
                                      codes, sf, row_g, workspace, status=None, stream=None):
    T, H = dy.shape
    k = dest_row.shape[1]
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().minite_moe_combine_backward_quant(_p(dy), T, H, E, k, _p(dest_row),
                                                  _p(expert_offsets), _p(sf_row_offsets),
                                                  _p(perm_src), _p(codes), _p(sf), _p(row_g),
                                                  _p(workspace), ws_bytes, _p(status), _s(stream))
    _check(rc, "minite_moe_combine_backward_quant")


def minite_quantize_tokens_nvfp4(x, row_src, m_cap, E, expert_offsets, k_cap, codes, sf, g, kofs,
                                 workspace, status=None, stream=None, row_amax=None):
    x_rows, C = x.shape
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().minite_quantize_tokens_nvfp4(_p(x), x_rows, _p(row_src), _p(row_amax), m_cap, C, E,
                                             _p(expert_offsets), k_cap, _p(codes), _p(sf), _p(g),
                                             _p(kofs), _p(workspace), ws_bytes, _p(status),
                                             _s(stream))
    _check(rc, "minite_quantize_tokens_nvfp4")


def minite_grouped_gemm_wgrad_nvfp4(a, b, out, status=None, stream=None):
    """a, b: ``quantize_tokens`` results over the same routing; out [E, Ma, Nb]."""
    E, M, N = out.shape
    if a["k_cap"] != b["k_cap"]:
        raise MiniteError("minite_grouped_gemm_wgrad_nvfp4: operands with different token capacity")
    out_dtype = OUT_FP32 if out.dtype == torch.float32 else OUT_BF16
    rc = load().minite_grouped_gemm_wgrad_nvfp4(_p(a["codes"]), _p(a["sf"]), _p(a["g"]),
                                                _p(b["codes"]), _p(b["sf"]), _p(b["g"]),
                                                _p(a["kofs"]), E, M, N, a["k_cap"], _p(out),
                                                out_dtype, _p(status), _s(stream))
    _check(rc, "minite_grouped_gemm_wgrad_nvfp4")


def quantize_tokens(x, expert_offsets, E, row_src=None, m_cap=None, stream=None, row_amax=None):
    """Weight-gradient operand of x's permuted rows (x[row_src[m]] or x[m]):
    dict(codes [C, k_cap/2], sf, g [E], kofs [E+1], k_cap) with
    k_cap = m_cap + 256 E rounded up to 256. ``row_amax`` [x_rows]: each row's
    |x| maximum when the producer wrote it (x is then read once)."""
    dev = x.device
    x_rows, C = x.shape
    m_cap = (row_src.numel() if row_src is not None else x_rows) if m_cap is None else m_cap
    k_cap = (m_cap + 256 * E + 255) // 256 * 256
    out = dict(codes=torch.empty((C, k_cap // 2), dtype=torch.uint8, device=dev),
               sf=torch.empty(((C + 127) // 128 * 128) * (k_cap // 16), dtype=torch.uint8, device=dev),
               g=torch.empty(E, dtype=torch.float32, device=dev),
               kofs=torch.empty(E + 1, dtype=torch.int32, device=dev), k_cap=k_cap)
    gathered = row_src is not None and row_amax is None
    ws = torch.empty(max(4, minite_workspace_bytes(OP_QUANTIZE_TOKENS, E, x_rows if gathered else 0)),
                     dtype=torch.uint8, device=dev)
    minite_quantize_tokens_nvfp4(x, row_src, m_cap, E, expert_offsets, k_cap, out["codes"],
                                 out["sf"], out["g"], out["kofs"], ws, stream=stream,
                                 row_amax=row_amax)
    return out


def minite_moe_combine(expert_out, dest_row, y, status=None, stream=None):
    M, N = expert_out.shape
    T, k = dest_row.shape
    rc = load().minite_moe_combine(_p(expert_out), _p(dest_row), T, M, N, k, _p(y), _p(status),
                                   _s(stream))
    _check(rc, "minite_moe_combine")


# The BF16 learner operators are called for as little as one token, so their
# checks below build no text and no ctypes object unless something is wrong.
_DTYPES = {torch.bfloat16: OUT_BF16, torch.float32: OUT_FP32}


def _dtype(t, name):
    """OUT_BF16 or OUT_FP32 of a tensor."""
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise MiniteError(f"{name}: expected bfloat16 or float32, got {t.dtype}")
    return d


def _device(t):
    """Index of the device of a call's first operand: it has to be the current one,
    where the kernel is launched, and every other operand has to be there too."""
    d = t.get_device()
    if d < 0:
        raise MiniteError("expected a CUDA tensor")
    if d != _current_device():
        raise _elsewhere("tensor", d, _current_device())
    return d


def _ptr(t, dev):
    """Address of a tensor on this device, None for None."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise _elsewhere("tensor", t.get_device(), dev)
    return t.data_ptr()


def _raw(stream, dev):
    """The stream's handle: the device's current stream when none is given."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise _elsewhere("stream", stream.device_index, dev)
    return stream.cuda_stream


def _shape(t, dims, name, what):
    """A tensor's sizes, of which there have to be so many."""
    if len(t.shape) != dims:
        raise MiniteError(f"{name}: expected {what} with {dims} dimensions, got {list(t.shape)}")
    return t.shape


def _status(t, name, dev):
    """Address of the word that device errors are OR-ed into, None for None."""
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.numel() < 1:
        raise MiniteError(f"{name}: status is int32, one element")
    return _ptr(t, dev)


def _rows(t, name):
    """Row stride of a 2-D tensor whose rows are contiguous and do not overlap."""
    n, c = _shape(t, 2, name, "a matrix")
    rs, cs = t.stride()
    if (c > 1 and cs != 1) or (n > 1 and rs < c):
        raise MiniteError(f"{name}: expected 2-D with contiguous rows that do not overlap")
    return rs if n > 1 else (c + 7) // 8 * 8


def _offsets(t, E, name, dev):
    if t.dtype is not torch.int32 or t.shape != (E + 1,) or not t.is_contiguous():
        raise MiniteError(f"{name}: expert_offsets is int32 [E + 1], contiguous")
    return _ptr(t, dev)


def minite_grouped_gemm_bf16(a, w, expert_offsets, out, w_layout=W_NK, status=None, stream=None):
    """a bf16 [M, K]; w bf16 [E, N, K] (W_NK) or [E, K, N] (W_KN); out [M, N] bf16 or fp32."""
    name = "minite_grouped_gemm_bf16"
    if a.dtype is not torch.bfloat16 or w.dtype is not torch.bfloat16 or not w.is_contiguous():
        raise MiniteError(f"{name}: a and w are bfloat16, w contiguous")
    E, N, K = _shape(w, 3, name, "w")
    if w_layout == W_KN:
        N, K = K, N
    M, Ka = _shape(a, 2, name, "a")
    if Ka != K or out.shape != (M, N):
        raise MiniteError(f"{name}: shapes of a, w and out do not match")
    d = _device(a)
    rc = load().minite_grouped_gemm_bf16(a.data_ptr(), _rows(a, name), _ptr(w, d), w_layout,
                                         _offsets(expert_offsets, E, name, d), M, N, K, E,
                                         _ptr(out, d), _rows(out, name), _dtype(out, name),
                                         _status(status, name, d), _raw(stream, d))
    if rc:
        _check(rc, name)


def minite_grouped_wgrad_bf16(a, b, expert_offsets, out, accumulate=False, status=None, stream=None):
    """a bf16 [M, Na], b bf16 [M, Nb] in expert order; out [E, Na, Nb] bf16 or fp32."""
    name = "minite_grouped_wgrad_bf16"
    if a.dtype is not torch.bfloat16 or b.dtype is not torch.bfloat16 or not out.is_contiguous():
        raise MiniteError(f"{name}: a and b are bfloat16, out contiguous")
    E, Na, Nb = _shape(out, 3, name, "out")
    M = _shape(a, 2, name, "a")[0]
    if a.shape != (M, Na) or b.shape != (M, Nb):
        raise MiniteError(f"{name}: shapes of a, b and out do not match")
    d = _device(a)
    rc = load().minite_grouped_wgrad_bf16(a.data_ptr(), _rows(a, name), _ptr(b, d), _rows(b, name),
                                          _offsets(expert_offsets, E, name, d), M, Na, Nb, E,
                                          _ptr(out, d), _dtype(out, name), 1 if accumulate else 0,
                                          _status(status, name, d), _raw(stream, d))
    if rc:
        _check(rc, name)


def _targets(targets, N, name):
    if targets is None:
        return 0
    if targets.dtype not in (torch.int32, torch.int64) or targets.shape != (N,) or \
            not targets.is_contiguous():
        raise MiniteError(f"{name}: targets is int32 or int64 [N], contiguous")
    return 1 if targets.dtype is torch.int64 else 0


def _f32(t, shape, name, what, dev):
    """Address of an FP32 tensor of this shape on this device, None for None."""
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.shape != shape or not t.is_contiguous():
        raise MiniteError(f"{name}: {what} is float32 {list(shape)}, contiguous")
    return _ptr(t, dev)


def minite_token_logprobs(logits, targets, logprob, entropy=None, stats=None, temperature=1.0,
                          alt_ids=None, alt_logprobs=None, status=None, stream=None):
    """logits [N, V] bf16 or fp32; logprob, entropy fp32 [N]; stats fp32 [N, 2];
    alt_ids int32 and alt_logprobs fp32 [N, k]."""
    name = "minite_token_logprobs"
    ld = _rows(logits, name)
    N, V = logits.shape
    k = 0
    if alt_ids is not None:
        k = _shape(alt_ids, 2, name, "alt_ids")[1]
        if alt_ids.dtype is not torch.int32 or alt_ids.shape[0] != N or not alt_ids.is_contiguous():
            raise MiniteError(f"{name}: alt_ids is int32 [N, k], contiguous")
    d = _device(logits)
    rc = load().minite_token_logprobs(logits.data_ptr(), _dtype(logits, name), N, V, ld,
                                      _ptr(targets, d), _targets(targets, N, name), temperature,
                                      _f32(logprob, (N,), name, "logprob", d),
                                      _f32(entropy, (N,), name, "entropy", d),
                                      _f32(stats, (N, 2), name, "stats", d), k, _ptr(alt_ids, d),
                                      _f32(alt_logprobs, (N, k), name, "alt_logprobs", d),
                                      _status(status, name, d), _raw(stream, d))
    if rc:
        _check(rc, name)


def minite_token_logprobs_backward(logits, targets, stats, entropy, grad_logprob, grad_entropy,
                                   dlogits, temperature=1.0, status=None, stream=None):
    """dlogits: the type and shape of logits (may be logits itself)."""
    name = "minite_token_logprobs_backward"
    ld = _rows(logits, name)
    N, V = logits.shape
    if dlogits.dtype is not logits.dtype or dlogits.shape != logits.shape or stats is None:
        raise MiniteError(f"{name}: needs the forward's stats, and dlogits of the type and shape of logits")
    d = _device(logits)
    rc = load().minite_token_logprobs_backward(
        logits.data_ptr(), _dtype(logits, name), N, V, ld, _ptr(targets, d), _targets(targets, N, name),
        temperature, _f32(stats, (N, 2), name, "stats", d), _f32(entropy, (N,), name, "entropy", d),
        _f32(grad_logprob, (N,), name, "grad_logprob", d),
        _f32(grad_entropy, (N,), name, "grad_entropy", d),
        _ptr(dlogits, d), _rows(dlogits, name), _status(status, name, d), _raw(stream, d))
    if rc:
        _check(rc, name)


def _int32(t, shape, name, what, dev):
    """Address of an int32 tensor of this shape on this device."""
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous():
        raise MiniteError(f"{name}: {what} is int32 {list(shape)}, contiguous")
    return _ptr(t, dev)


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _same_type(a, b, name):
    if a.dtype is not b.dtype:
        raise MiniteError(f"{name}: the matrices have one type")


def minite_moe_permute_rows(x, topk_ids, E, rows, expert_offsets, perm_src, dest_row, workspace,
                            status=None, stream=None):
    """x [T, H] and rows [T*k, H] bf16 or fp32; topk_ids, dest_row int32 [T, k]; perm_src int32 [T*k]."""
    name = "minite_moe_permute_rows"
    T, H = _shape(x, 2, name, "x")
    k = _shape(topk_ids, 2, name, "topk_ids")[1]
    _same_type(x, rows, name)
    if rows.shape != (T * k, H):
        raise MiniteError(f"{name}: rows is [T * k, H]")
    d = _device(x)
    rc = load().minite_moe_permute_rows(
        x.data_ptr(), _dtype(x, name), _rows(x, name), _int32(topk_ids, (T, k), name, "topk_ids", d), T, H, E, k,
        _ptr(rows, d), _rows(rows, name), _offsets(expert_offsets, E, name, d),
        _int32(perm_src, (T * k,), name, "perm_src", d), _int32(dest_row, (T, k), name, "dest_row", d),
        _ptr(workspace, d), _bytes(workspace), _status(status, name, d), _raw(stream, d))
    if rc:
        _check(rc, name)


def minite_moe_spread_rows(x, dest_row, rows, status=None, stream=None):
    """x [T, H] and rows [M, H] bf16 or fp32; dest_row int32 [T, k]."""
    name = "minite_moe_spread_rows"
    T, H = _shape(x, 2, name, "x")
    k = _shape(dest_row, 2, name, "dest_row")[1]
    _same_type(x, rows, name)
    M, Hr = _shape(rows, 2, name, "rows")
    if Hr != H:
        raise MiniteError(f"{name}: shapes of x and rows do not match")
    d = _device(x)
    rc = load().minite_moe_spread_rows(
        x.data_ptr(), _dtype(x, name), _rows(x, name), _int32(dest_row, (T, k), name, "dest_row", d), T, M, H, k,
        _ptr(rows, d), _rows(rows, name), _status(status, name, d), _raw(stream, d))
    if rc:
        _check(rc, name)


def minite_moe_combine_rows(rows, dest_row, weights, y, status=None, stream=None):
    """rows [M, H] and y [T, H] bf16 or fp32; dest_row int32, weights fp32 (or None) [T, k]."""
    name = "minite_moe_combine_rows"
    M, H = _shape(rows, 2, name, "rows")
    T, k = _shape(dest_row, 2, name, "dest_row")
    _same_type(rows, y, name)
    if y.shape != (T, H):
        raise MiniteError(f"{name}: y is [T, H]")
    d = _device(rows)
    rc = load().minite_moe_combine_rows(
        rows.data_ptr(), _dtype(rows, name), _rows(rows, name), _int32(dest_row, (T, k), name, "dest_row", d),
        _f32(weights, (T, k), name, "weights", d), T, M, H, k, _ptr(y, d), _rows(y, name),
        _status(status, name, d), _raw(stream, d))
    if rc:
        _check(rc, name)


def minite_moe_combine_rows_backward(dy, rows, dest_row, weights, drows, dweights, status=None, stream=None):
    """dy [T, H], rows (or None, with dweights None) and drows [M, H] bf16 or fp32; dest_row int32,
    weights and dweights fp32 [T, k]."""
    name = "minite_moe_combine_rows_backward"
    T, H = _shape(dy, 2, name, "dy")
    k = _shape(dest_row, 2, name, "dest_row")[1]
    _same_type(dy, drows, name)
    if rows is not None:
        _same_type(dy, rows, name)
    M, Hr = _shape(drows, 2, name, "drows")
    if Hr != H or (rows is not None and rows.shape != (M, H)):
        raise MiniteError(f"{name}: shapes of dy, rows and drows do not match")
    d = _device(dy)
    rc = load().minite_moe_combine_rows_backward(
        dy.data_ptr(), _dtype(dy, name), _rows(dy, name), _ptr(rows, d), 0 if rows is None else _rows(rows, name),
        _int32(dest_row, (T, k), name, "dest_row", d), _f32(weights, (T, k), name, "weights", d), T, M, H, k,
        _ptr(drows, d), _rows(drows, name), _f32(dweights, (T, k), name, "dweights", d), _status(status, name, d),
        _raw(stream, d))
    if rc:
        _check(rc, name)


def _grad_table(grads, outs, name):
    """struct minite_grad_tensor of every gradient and its destination (outs may be
    grads, None: they are only read), the device, and the number of elements."""
    if len(grads) == 0:
        raise MiniteError(f"{name}: needs gradients")
    d = _device(grads[0])
    sizes = [g.numel() for g in grads]
    at = [g.data_ptr() for g in grads]
    kinds = [_DTYPES.get(g.dtype) for g in grads]
    tensors = grads
    out_at, out_kinds = at, kinds
    if outs is not None and outs is not grads:
        if [o.numel() for o in outs] != sizes:
            raise MiniteError(f"{name}: one destination a gradient, of its size")
        out_at = [o.data_ptr() for o in outs]
        out_kinds = [_DTYPES.get(o.dtype) for o in outs]
        tensors = [*grads, *outs]
    if not all([t.is_contiguous() for t in tensors]):
        raise MiniteError(f"{name}: gradients and destinations are contiguous")
    if None in kinds or None in out_kinds:
        raise MiniteError(f"{name}: expected bfloat16 or float32")
    places = [t.get_device() for t in tensors]
    if places.count(d) != len(places):
        raise _elsewhere("tensor", next(i for i in places if i != d), d)
    if outs is not None and len(set(out_at)) != len(out_at):
        # a tensor that is written twice would be scaled twice, or once and a half
        used = [a for a, n in zip(out_at, sizes) if n]
        if len(set(used)) != len(used):
            raise MiniteError(f"{name}: a destination appears twice")
    both = [a | b << 32 for a, b in zip(kinds, out_kinds)]
    return array("q", chain.from_iterable(zip(at, out_at, sizes, both))), d, sum(sizes)


def minite_grad_norm(grads, order, max_norm, norm, factor, workspace, stream=None):
    """grads: contiguous bf16 or fp32 tensors; norm and factor fp32 [1], one of them may be None."""
    name = "minite_grad_norm"
    table, d, _ = _grad_table(grads, None, name)
    rc = load().minite_grad_norm(table.buffer_info()[0], len(grads), order, max_norm,
                                 _f32(norm, (1,), name, "norm", d), _f32(factor, (1,), name, "factor", d),
                                 _ptr(workspace, d), _bytes(workspace), _raw(stream, d))
    if rc:
        _check(rc, name)


def minite_clip_grads(grads, outs, factor, stream=None, table=None):
    """outs[i] = grads[i] * factor; outs[i] may be grads[i]; factor fp32 [1]."""
    name = "minite_clip_grads"
    table, d, _ = _grad_table(grads, outs, name) if table is None else table
    rc = load().minite_clip_grads(table.buffer_info()[0], len(grads), _f32(factor, (1,), name, "factor", d),
                                  _raw(stream, d))
    if rc:
        _check(rc, name)


def _sequence_rows(t, name, what):
    """Row stride of [B, R, V] whose B * R rows are contiguous and evenly spaced."""
    B, R, V = _shape(t, 3, name, what)
    s0, s1, s2 = t.stride()
    ld = s1 if R > 1 else s0 if B > 1 else V
    if (V > 1 and s2 != 1) or ld < V or (R > 1 and B > 1 and s0 != R * s1):
        raise MiniteError(f"{name}: {what} has contiguous rows that are evenly spaced")
    return ld


def _verify(target, draft, draft_tokens, uniforms, noise, temperature, tokens, accepted, logprobs, workspace,
            ws_bytes, status, stream, d, name):
    """The inputs' checks and the call; outputs are addresses."""
    B, S1, V = target.shape
    S = _shape(draft_tokens, 2, name, "draft_tokens")[1]
    if S1 != S + 1 or (draft is not None and draft.shape != (B, S, V)):
        raise MiniteError(f"{name}: the target's logits are [B, S + 1, V], the draft's [B, S, V], draft_tokens [B, S]")
    if noise.dtype is not torch.float32 or noise.shape != (B, V):
        raise MiniteError(f"{name}: noise is float32 [B, V]")
    draft_at, draft_dtype, draft_ld = None, OUT_BF16, V
    if draft is not None and S:
        draft_at, draft_dtype, draft_ld = _ptr(draft, d), _dtype(draft, name), _sequence_rows(draft, name, "draft")
    rc = load().minite_verify_drafts(
        target.data_ptr(), _dtype(target, name), _sequence_rows(target, name, "target"), draft_at, draft_dtype,
        draft_ld, _int32(draft_tokens, (B, S), name, "draft_tokens", d),
        _f32(uniforms, (B, S), name, "uniforms", d), _ptr(noise, d), _rows(noise, name), B, S, V, temperature,
        tokens, accepted, logprobs, workspace, ws_bytes, _status(status, name, d), _raw(stream, d))
    if rc:
        _check(rc, "minite_verify_drafts")


def minite_verify_drafts(target, draft, draft_tokens, uniforms, noise, temperature, tokens, accepted, logprobs,
                         workspace, status=None, stream=None):
    """target [B, S + 1, V], draft [B, S, V] (or None) bf16 or fp32; draft_tokens int32 and uniforms
    fp32 [B, S]; noise fp32 [B, V]; tokens int32 and logprobs (or None) fp32 [B, S + 1]; accepted int32 [B]."""
    name = "minite_verify_drafts"
    B, S1, _ = _shape(target, 3, name, "target")
    d = _device(target)
    _verify(target, draft, draft_tokens, uniforms, noise, temperature, _int32(tokens, (B, S1), name, "tokens", d),
            _int32(accepted, (B,), name, "accepted", d), _f32(logprobs, (B, S1), name, "logprobs", d),
            _ptr(workspace, d), _bytes(workspace), status, stream, d, name)


# struct minite_adamw_tensor
ADAMW_TENSOR = np.dtype([("param", "u8"), ("grad", "u8"), ("exp_avg", "u8"), ("exp_avg_sq", "u8"),
                         ("exp_avg_scale", "u8"), ("exp_avg_sq_scale", "u8"), ("param_bf16", "u8"),
                         ("n", "i8")])


def minite_adamw_step(tensors, param_dtype, grad_dtype, state_bits, lr, beta1, beta2, eps,
                      weight_decay, step, grad_scale=None, stream=None):
    """tensors: numpy array of ADAMW_TENSOR on the host, one descriptor a tensor, with
    addresses on the current device."""
    if tensors.dtype != ADAMW_TENSOR or not tensors.flags.c_contiguous:
        raise MiniteError("minite_adamw_step: tensors is a contiguous array of ADAMW_TENSOR")
    rc = load().minite_adamw_step(tensors.ctypes.data, len(tensors), param_dtype, grad_dtype,
                                  state_bits, lr, beta1, beta2, eps, weight_decay, step,
                                  _p(grad_scale), _s(stream))
    _check(rc, "minite_adamw_step")


def minite_test_convert(x, out_e2m1=None, out_e4m3=None, out_exp=None, stream=None):
    rc = load().minite_test_convert(_p(x), x.numel(), _p(out_e2m1), _p(out_e4m3), _p(out_exp),
                                    _s(stream))
    _check(rc, "minite_test_convert")


def minite_test_convert_digest(first_chunk, n_chunks, digests, stream=None):
    """Adds the device converters' digests of chunks [first_chunk, first_chunk
    + n_chunks) of 2^20 float32 bit patterns into digests (int64 [n_chunks, 3])."""
    rc = load().minite_test_convert_digest(first_chunk, n_chunks, _p(digests), _s(stream))
    _check(rc, "minite_test_convert_digest")


def minite_test_div6_exhaustive(counter, stream=None):
    rc = load().minite_test_div6_exhaustive(_p(counter), _s(stream))
    _check(rc, "minite_test_div6_exhaustive")


def minite_test_adamw_math(counters, stream=None):
    """counters: int64 [2], zeroed by the caller."""
    _check(load().minite_test_adamw_math(_p(counters), _s(stream)), "minite_test_adamw_math")


# ---------------------------------------------------------------- allocation helpers


def _kc(cols: int) -> int:
    return ((cols // 16) + 3) // 4 * 4


def sf_bytes(rows_padded: int, cols: int) -> int:
    return rows_padded * _kc(cols)


def quantize(x, per_group=False, along_rows=False, g_in=None, stream=None):
    """Quantize bf16 x ([rows, cols] or [groups, rows, cols]); returns dict(codes, sf, g)."""
    dev = x.device
    g3 = x if x.dim() == 3 else x.unsqueeze(0)
    G, R, C = g3.shape
    Rq, Cq = (C, R) if along_rows else (R, C)
    codes = torch.empty((G, Rq, Cq // 2), dtype=torch.uint8, device=dev)
    sf = torch.empty((G, sf_bytes((Rq + 127) // 128 * 128, Cq)), dtype=torch.uint8, device=dev)
    g = torch.empty((G,) if per_group else (G * Rq,), dtype=torch.float32, device=dev)
    ws = None
    if per_group and g_in is None:
        ws = torch.empty(minite_workspace_bytes(OP_QUANTIZE, G), dtype=torch.uint8, device=dev)
    minite_quantize_nvfp4(g3, SCALE_PER_GROUP if per_group else SCALE_PER_ROW,
                          ALONG_ROWS if along_rows else ALONG_COLS, codes, sf, g, g_in, ws,
                          stream=stream)
    if x.dim() == 2:
        codes, sf = codes[0], sf[0]
    return dict(codes=codes, sf=sf, g=g)


def _need(cond, what):
    if not cond:
        raise MiniteError(what)


def _empty(shape, dtype, like, stream):
    """A new tensor that belongs to the stream that the kernel runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def grouped_gemm_bf16(x, w, expert_offsets, w_as_stored=False, out=None, out_dtype=torch.bfloat16,
                      status=None, stream=None):
    """x [M, K] bf16 in expert order times each expert's w: x @ w[e].T for w
    [E, N, K] (the forward), or x @ w[e] for w [E, K, N] with ``w_as_stored``
    (the activation gradient of that forward, x its output's gradient).
    Returns [M, N]."""
    if out is None:
        name = "grouped_gemm_bf16"
        rows, cols = _shape(x, 2, name, "x")[0], _shape(w, 3, name, "w")[2 if w_as_stored else 1]
        out = _empty((rows, cols), out_dtype, x, stream)
    minite_grouped_gemm_bf16(x, w, expert_offsets, out, W_KN if w_as_stored else W_NK, status, stream)
    return out


def grouped_wgrad_bf16(dy, x, expert_offsets, out=None, out_dtype=torch.float32, accumulate=False,
                       status=None, stream=None):
    """dw[e] = dy_e.T @ x_e over each expert's rows, [E, Na, Nb]; added to
    ``out`` (fp32) with ``accumulate``."""
    if out is None:
        if accumulate:
            raise MiniteError("grouped_wgrad_bf16: accumulate needs out")
        name = "grouped_wgrad_bf16"
        if expert_offsets.numel() < 2:
            raise MiniteError(f"{name}: expert_offsets is int32 [E + 1], contiguous")
        out = _empty((expert_offsets.numel() - 1, _shape(dy, 2, name, "dy")[1], _shape(x, 2, name, "x")[1]),
                     out_dtype, x, stream)
    minite_grouped_wgrad_bf16(dy, x, expert_offsets, out, accumulate, status, stream)
    return out


def token_logprobs(logits, targets=None, temperature=1.0, alternatives=0, status=None, stream=None):
    """Log probability of each row's target token under softmax(logits /
    temperature), with the row's entropy and its ``alternatives`` most likely
    tokens. Returns dict(logprob (None without targets), entropy, stats,
    alt_ids, alt_logprobs); a negative target marks a row that is skipped."""
    name = "token_logprobs"
    ld = _rows(logits, name)
    if alternatives < 0:
        raise MiniteError(f"{name}: alternatives is {alternatives}")
    N, V = logits.shape
    d = _device(logits)
    f32 = torch.float32
    entropy, stats = _empty((N,), f32, logits, stream), _empty((N, 2), f32, logits, stream)
    logprob = alt_ids = alt_logprobs = None
    if targets is not None:
        logprob = _empty((N,), f32, logits, stream)
    if alternatives:
        alt_ids = _empty((N, alternatives), torch.int32, logits, stream)
        alt_logprobs = _empty((N, alternatives), f32, logits, stream)
    rc = load().minite_token_logprobs(
        logits.data_ptr(), _dtype(logits, name), N, V, ld, _ptr(targets, d), _targets(targets, N, name),
        temperature, None if logprob is None else logprob.data_ptr(),
        entropy.data_ptr(), stats.data_ptr(), alternatives,
        alt_ids.data_ptr() if alternatives else None,
        alt_logprobs.data_ptr() if alternatives else None, _status(status, name, d), _raw(stream, d))
    if rc:
        _check(rc, "minite_token_logprobs")
    return {"logprob": logprob, "entropy": entropy, "stats": stats, "alt_ids": alt_ids,
            "alt_logprobs": alt_logprobs}


def token_logprobs_backward(logits, targets, forward, grad_logprob=None, grad_entropy=None,
                            temperature=1.0, out=None, status=None, stream=None):
    """Gradient of token_logprobs' logprob and entropy with respect to the
    logits; ``forward`` is its result for the same logits, targets and
    temperature. ``out`` may be the logits themselves."""
    if out is None:
        out = _empty(logits.shape, logits.dtype, logits, stream)
    minite_token_logprobs_backward(logits, targets, forward["stats"], forward["entropy"],
                                   grad_logprob, grad_entropy, out, temperature, status, stream)
    return out


def _workspace(op, like, stream, a, b=0, E=0, k=0):
    n = load().minite_workspace_bytes(op, a, b, E, k)
    return _empty((n,), torch.uint8, like, stream) if n else None


def permute_rows(x, topk_ids, E, into=None, status=None, stream=None):
    """Rows of x [T, H] (bf16 or fp32) sorted by expert: rows[dest_row[t, j]] = x[t]
    for every slot with an id in [0, E) (a negative one is not used). Returns
    dict(rows [T*k, H], offsets [E + 1], perm_src [T*k], dest_row [T, k]); ``into``
    is such a dict whose tensors are written again. Rows from offsets[E] on are
    left as they were, their perm_src is -1."""
    T, H = _shape(x, 2, "permute_rows", "x")
    k = _shape(topk_ids, 2, "permute_rows", "topk_ids")[1]
    if into is None:
        into = dict(rows=_empty((T * k, H), x.dtype, x, stream), offsets=_empty((E + 1,), torch.int32, x, stream),
                    perm_src=_empty((T * k,), torch.int32, x, stream),
                    dest_row=_empty((T, k), torch.int32, x, stream))
    minite_moe_permute_rows(x, topk_ids, E, into["rows"], into["offsets"], into["perm_src"], into["dest_row"],
                            _workspace(OP_PERMUTE_ROWS, x, stream, T, 0, E, k), status, stream)
    return into


def permute_rows_backward(drows, dest_row, out=None, status=None, stream=None):
    """The gradient of permute_rows' x: dx[t] = sum over slots of drows[dest_row[t, j]]."""
    return combine_rows(drows, dest_row, None, out, status, stream)


def spread_rows(x, dest_row, rows, status=None, stream=None):
    """rows[dest_row[t, j]] = x[t] by a routing that is already there; returns ``rows``
    (those that no slot names are left as they were)."""
    minite_moe_spread_rows(x, dest_row, rows, status, stream)
    return rows


def combine_rows(rows, dest_row, weights=None, out=None, status=None, stream=None):
    """y[t] = sum over slots of weights[t, j] * rows[dest_row[t, j]] (weights fp32
    [T, k], None for 1), summed in FP32 in slot order. Returns [T, H]."""
    if out is None:
        H = _shape(rows, 2, "combine_rows", "rows")[1]
        out = _empty((_shape(dest_row, 2, "combine_rows", "dest_row")[0], H), rows.dtype, rows, stream)
    minite_moe_combine_rows(rows, dest_row, weights, out, status, stream)
    return out


def combine_rows_backward(dy, rows, dest_row, weights, out=None, status=None, stream=None):
    """The gradients of combine_rows: (drows, dweights). ``out`` receives drows (it may be
    ``rows``); its rows that no slot names are not written. With rows None (and
    ``out`` given) the weights' gradient is left out: (drows, None)."""
    if out is None:
        if rows is None:
            raise MiniteError("combine_rows_backward: needs rows or out")
        out = _empty(tuple(rows.shape), rows.dtype, rows, stream)
    dweights = None if rows is None else _empty(tuple(dest_row.shape), torch.float32, dy, stream)
    minite_moe_combine_rows_backward(dy, rows, dest_row, weights, out, dweights, status, stream)
    return out, dweights


def _norm_of(grads, max_norm, order, stream, table, name):
    if order not in (2, math.inf):
        raise MiniteError(f"{name}: order is 2 or inf, not {order}")
    table, d, elements = table
    like = grads[0]
    norm, scale = _empty((1,), torch.float32, like, stream), _empty((1,), torch.float32, like, stream)
    lib = load()
    n = lib.minite_workspace_bytes(OP_GRAD_NORM, len(grads), elements, 0, 0)
    ws = _empty((n,), torch.uint8, like, stream) if n else None
    rc = lib.minite_grad_norm(table.buffer_info()[0], len(grads), NORM_2 if order == 2 else NORM_MAX, max_norm,
                              norm.data_ptr(), scale.data_ptr(), ws.data_ptr() if n else None, n, _raw(stream, d))
    if rc:
        _check(rc, "minite_grad_norm")
    return {"norm": norm, "scale": scale}


def grad_norm(grads, max_norm=math.inf, order=2.0, stream=None):
    """The global norm of a list of gradients (bf16 and fp32 may be mixed), and the
    factor min(1, max_norm / (norm + 1e-6)) for ``AdamW.step(grad_scale=)``:
    dict(norm [1], scale [1]), on the device. order: 2 or math.inf (the largest |g|)."""
    return _norm_of(grads, max_norm, order, stream, _grad_table(grads, None, "grad_norm"), "grad_norm")


def clip_grads(grads, max_norm, order=2.0, out=None, stream=None):
    """Gradients times grad_norm's factor, in place or into the tensors ``out``
    (of either type). Returns grad_norm's dict."""
    out = grads if out is None else out
    table = _grad_table(grads, out, "clip_grads")
    r = _norm_of(grads, max_norm, order, stream, table, "clip_grads")
    minite_clip_grads(grads, out, r["scale"], stream, table)
    return r


def verify_drafts(logits, draft_tokens, uniforms, noise, draft_logits=None, temperature=1.0, status=None,
                  stream=None):
    """Drafted tokens [B, S] int32 (negative: no more drafts) verified against the
    target's logits [B, S + 1, V] with ``uniforms`` [B, S] in [0, 1) and exponential
    variates ``noise`` [B, V]; ``draft_logits`` [B, S, V] is what the drafts were
    sampled from at the same temperature, None where they were looked up. Returns
    dict(tokens [B, S + 1], accepted [B], logprobs [B, S + 1]): the drafts that stand,
    the token that follows them, -1."""
    B, S1, V = _shape(logits, 3, "verify_drafts", "logits")
    d = _device(logits)
    tokens, accepted = _empty((B, S1), torch.int32, logits, stream), _empty((B,), torch.int32, logits, stream)
    logprobs = _empty((B, S1), torch.float32, logits, stream)
    n = load().minite_workspace_bytes(OP_VERIFY_DRAFTS, B, V, S1 - 1, 0)
    ws = _empty((n,), torch.uint8, logits, stream)
    _verify(logits, draft_logits, draft_tokens, uniforms, noise, temperature, tokens.data_ptr(), accepted.data_ptr(),
            logprobs.data_ptr(), ws.data_ptr(), n, status, stream, d, "verify_drafts")
    return {"tokens": tokens, "accepted": accepted, "logprobs": logprobs}


class AdamW:
    """AdamW over a list of contiguous tensors of one type (bf16 or fp32), one
    launch a step, with FP32 states or 8-bit ones (E4M3 codes and one scale per
    256 elements). ``copies``: bf16 tensors that receive the rounded parameters
    (for fp32 parameters). The states are flat buffers in which each tensor
    starts at a multiple of 256 elements (``starts``); ``state`` takes buffers
    of this layout and a step count to continue from. A step uses ``params``,
    ``copies`` and the states as they are then: their storage may be replaced
    between steps, by some of the same type and size.

    One learning rate and one weight decay for all tensors (an optimizer for each
    group that has its own). Step count and rates are host values: a captured
    graph replays one step's bias corrections. Non-finite gradients are not
    skipped."""

    BLOCK = 256

    def __init__(self, params, copies=None, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
                 weight_decay=0.01, state_bits=32, state=None):
        _need(len(params) > 0 and state_bits in (8, 32), "AdamW: needs tensors and state_bits 8 or 32")
        dev = params[0].device
        self._param_dtype = _dtype(params[0], "AdamW")
        self._dtype = params[0].dtype
        self.params, self.copies = list(params), None if copies is None else list(copies)
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.state_bits = state_bits
        self._numel = [p.numel() for p in params]
        sizes = np.array(self._numel, dtype=np.int64)
        blocks = -(-sizes // self.BLOCK)
        first = np.concatenate([[0], np.cumsum(blocks)[:-1]]).astype(np.int64)
        self.starts = (first * self.BLOCK).tolist()
        n_blocks = int(blocks.sum())
        # each state's type, size, and elements in front of every tensor's part
        codes = (torch.float8_e4m3fn if state_bits == 8 else torch.float32, n_blocks * self.BLOCK, first * self.BLOCK)
        self._states = dict(exp_avg=codes, exp_avg_sq=codes)
        if state_bits == 8:
            self._states["exp_avg_scale"] = self._states["exp_avg_sq_scale"] = (torch.float32, n_blocks, first)
        _need(all(p.is_cuda for p in params), "AdamW: parameters are CUDA tensors")
        self.step_count = 0 if state is None else int(state["step"])
        for name, (dtype, n, _) in self._states.items():
            setattr(self, name, torch.zeros(n, dtype=dtype, device=dev) if state is None else state[name])
        d = self._tensors = np.zeros(len(params), dtype=ADAMW_TENSOR)
        self._address, self._grads = d.ctypes.data, d["grad"]
        d["n"] = sizes
        self._bind(self._kept())

    def _kept(self):
        """What a step works on besides gradients, as it lies now."""
        t = [*self.params, self.exp_avg, self.exp_avg_sq]
        if self.state_bits == 8:
            t += (self.exp_avg_scale, self.exp_avg_sq_scale)
        if self.copies is not None:
            t += self.copies
        return [(x.data_ptr(), x.numel(), x.dtype, x.is_contiguous()) for x in t]

    def _bind(self, kept):
        """Checks all of that, then writes its addresses into the descriptors."""
        dev, places = self.exp_avg.device, {}
        _need(len(self.params) == len(self._numel), "AdamW: a parameter was added or taken away")
        for i, p in enumerate(self.params):
            _need(p.is_cuda and p.device == dev and p.dtype == self._dtype and p.is_contiguous() and
                  p.numel() == self._numel[i],
                  f"AdamW: parameter {i} is not a contiguous {self._dtype} tensor of {self._numel[i]} elements on {dev}")
        _need(self.copies is None or (len(self.copies) == len(self.params) and all(
            c.dtype == torch.bfloat16 and c.shape == p.shape and c.is_contiguous() and c.device == dev
            for c, p in zip(self.copies, self.params))), "AdamW: copies are bfloat16 tensors like the parameters")
        for name, (dtype, n, first) in self._states.items():
            t = getattr(self, name)
            _need(t.numel() == n and t.dtype == dtype and t.is_contiguous() and t.device == dev,
                  f"AdamW: state {name} is not {dtype} [{n}] on {dev}")
            places[name] = t.data_ptr() + first * t.element_size()
        places["param"] = [p.data_ptr() for p in self.params]
        places["param_bf16"] = 0 if self.copies is None else [c.data_ptr() for c in self.copies]
        for name, address in places.items():
            self._tensors[name] = address
        self._bound = kept

    def step(self, grads, grad_scale=None, lr=None, stream=None):
        """One step with grads[i] (bf16 or fp32, all one type) for tensor i, each
        times the device scalar ``grad_scale``."""
        d = _device(self.exp_avg)
        if [g.numel() for g in grads] != self._numel or len({g.dtype for g in grads}) != 1 or \
                not all([g.is_contiguous() and g.get_device() == d for g in grads]):
            raise MiniteError("AdamW.step: gradients are contiguous tensors of one type on the parameters' "
                              "device, one a parameter and of its size")
        if grad_scale is not None and (grad_scale.dtype is not torch.float32 or grad_scale.numel() != 1):
            raise MiniteError("AdamW.step: grad_scale is one float32")
        kept = self._kept()
        if kept != self._bound:   # storage was replaced
            self._bind(kept)
        self._grads[:] = [g.data_ptr() for g in grads]
        rc = load().minite_adamw_step(
            self._address, len(self.params), self._param_dtype, _dtype(grads[0], "AdamW.step"),
            self.state_bits, self.lr if lr is None else lr, *self.betas, self.eps, self.weight_decay,
            self.step_count + 1, _ptr(grad_scale, d), _raw(stream, d))
        if rc:
            _check(rc, "minite_adamw_step")
        self.step_count += 1


class MoEMLP:
    """Preallocated device buffers for the expert-MLP forward of one shape
    (T tokens, hidden H, intermediate I, E experts, top-k), so that a step
    allocates nothing and can be captured in a CUDA graph."""

    def __init__(self, T, H, I, E, k, device="cuda"):
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        M = T * k
        self.M = M
        d = torch.device(device)
        u8, f32, i32 = torch.uint8, torch.float32, torch.int32
        sf_rows = M + 128 * E
        self.a_codes = torch.empty((M, H // 2), dtype=u8, device=d)
        self.a_sf = torch.empty(sf_bytes(sf_rows, H), dtype=u8, device=d)
        self.a_g = torch.empty(M, dtype=f32, device=d)
        self.offsets = torch.empty(E + 1, dtype=i32, device=d)
        self.sf_offsets = torch.empty(E + 1, dtype=i32, device=d)
        self.perm_src = torch.empty(M, dtype=i32, device=d)
        self.dest_row = torch.empty((T, k), dtype=i32, device=d)
        self.perm_w = torch.empty(M, dtype=f32, device=d)
        self.ws = torch.empty(minite_workspace_bytes(OP_PERMUTE_QUANT, T, H, E, k), dtype=u8, device=d)
        self.gate_up = torch.empty((M, 2 * I), dtype=torch.bfloat16, device=d)
        self.h_codes = torch.empty((M, I // 2), dtype=u8, device=d)
        self.h_sf = torch.empty(sf_bytes(sf_rows, I), dtype=u8, device=d)
        self.h_g = torch.empty(M, dtype=f32, device=d)
        self.down = torch.empty((M, H), dtype=torch.bfloat16, device=d)
        self.y = torch.empty((T, H), dtype=torch.bfloat16, device=d)
        self.status = torch.zeros(1, dtype=i32, device=d)
        # the fused gate_up + SwiGLU kernel takes I % 128 == 0 and E <= 663
        self.fused_ok = I % 128 == 0 and 128 <= I <= 8192 and E <= 663
        self.sw_ws = torch.empty(max(16, minite_workspace_bytes(OP_GATE_UP_SWIGLU, M, I, 0, 0)),
                                 dtype=u8, device=d) if self.fused_ok else None

    def permute_quant(self, x, topk_ids, topk_w, stream=None):
        minite_moe_permute_quant(x, topk_ids, topk_w, self.E, self.a_codes, self.a_sf, self.a_g,
                                 self.offsets, self.sf_offsets, self.perm_src, self.dest_row,
                                 None if topk_w is None else self.perm_w, self.ws, self.status,
                                 stream)

    def gate_up_swiglu(self, wgu, stream=None, fused=True, keep_gate_up=False):
        """h = weighted SwiGLU of the gate_up GEMM, quantized into h_codes /
        h_sf / h_g: one fused launch (the BF16 gate_up stored only with
        keep_gate_up), or the GEMM into gate_up followed by the SwiGLU."""
        if fused:
            if not self.fused_ok:
                raise MiniteError("the fused gate_up + SwiGLU kernel needs I % 128 == 0, E <= 663")
            minite_gate_up_swiglu_quant_nvfp4(
                self.a_codes, self.a_sf, self.a_g, wgu["codes"], wgu["sf"], wgu["g"],
                self.offsets, self.sf_offsets, self.perm_w, self.h_codes, self.h_sf, self.h_g,
                self.sw_ws, gate_up=self.gate_up if keep_gate_up else None, status=self.status,
                stream=stream)
            return
        minite_grouped_gemm_nvfp4(self.a_codes, self.a_sf, self.a_g, wgu["codes"], wgu["sf"],
                                  wgu["g"], self.offsets, self.sf_offsets, self.gate_up,
                                  self.status, stream)
        minite_swiglu_weighted_quant(self.gate_up, self.perm_w, self.E, self.offsets,
                                     self.sf_offsets, self.h_codes, self.h_sf, self.h_g,
                                     self.status, stream)

    def forward(self, x, topk_ids, topk_w, wgu, wd, stream=None, fused=False, keep_gate_up=True):
        """x [T,H] bf16, topk_ids [T,k] int32, topk_w [T,k] f32; wgu / wd are
        ``quantize(..., per_group=True)`` results of [E,2I,H] and [E,H,I].
        fused: gate_up GEMM, SwiGLU and requantization in one launch."""
        self.permute_quant(x, topk_ids, topk_w, stream)
        self.gate_up_swiglu(wgu, stream, fused=fused, keep_gate_up=keep_gate_up)
        minite_grouped_gemm_nvfp4(self.h_codes, self.h_sf, self.h_g, wd["codes"], wd["sf"],
                                  wd["g"], self.offsets, self.sf_offsets, self.down, self.status,
                                  stream)
        minite_moe_combine(self.down, self.dest_row, self.y, self.status, stream)
        return self.y
