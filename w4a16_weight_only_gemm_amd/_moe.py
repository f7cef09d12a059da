"""Binding of include/w4a16_moe.h: routing, experts' products, combine and the
8-bit integer product. Argument marshalling only; the names match the C ABI and
are re-exported by the package."""
from __future__ import annotations

import ctypes

import numpy as np

from . import (W4A16_ERR_INVALID_ARG, W4A16_OK, W4A16Error, _check_sizes, _lib, _ptr, _stream,
               _torch, w4a16_qweight_bytes, w4a16_scales_bytes)

W4A16_ROUTE_MAX_EXPERTS = 1024
W4A16_ROUTE_MAX_TOP_K = 32
W4A16_ROUTE_MAX_GROUPS = 64
W4A16_ROUTE_SOFTMAX = 0
W4A16_ROUTE_SIGMOID = 1
W4A16_LOGITS_F32 = 0
W4A16_LOGITS_BF16 = 1
W4A16_ACT_NONE = 0
W4A16_ACT_SWIGLU = 1


class w4a16_route_config(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_int), ("top_k", ctypes.c_int), ("scoring", ctypes.c_int),
                ("logits_type", ctypes.c_int), ("groups", ctypes.c_int),
                ("groups_kept", ctypes.c_int), ("group_top", ctypes.c_int),
                ("renormalize", ctypes.c_int), ("scale", ctypes.c_float)]


# Every symbol include/w4a16_moe.h declares, with its ctypes signature.
_vp, _int, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
MOE_SIGNATURES = {
    "w4a16_moe_route_workspace_bytes": (_sz, [_int, _int]),
    "w4a16_moe_route": (_int, [_vp, _vp, _vp, _int, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "w4a16_gemm_experts": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _int, _int, _int, _int, _int,
                                  _int, _int, _vp]),
    "w4a16_moe_combine": (_int, [_vp, _vp, _vp, _vp, _vp, _int, _int, _int, _vp]),
    "w8a8_qweight_bytes": (_sz, [_int, _int]),
    "w8a8_pack": (_int, [_vp, _vp, _int, _int]),
    "w8a8_gemm": (_int, [_vp, _vp, _vp, _vp, _vp, _int, _int, _int, _vp]),
}
for _name, (_res, _args) in MOE_SIGNATURES.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def _check_types(**need):
    """name=(tensor or address, torch dtype name): dtype checks for torch tensors."""
    if _torch is None:
        return
    for name, (t, dtype) in need.items():
        if isinstance(t, _torch.Tensor) and t.dtype != getattr(_torch, dtype):
            raise TypeError(f"{name} must be torch.{dtype}")


def w4a16_moe_route_workspace_bytes(T: int, experts: int) -> int:
    return int(_lib.w4a16_moe_route_workspace_bytes(T, experts))


def moe_route_status(logits, bias, config: w4a16_route_config, T, ids, weights, offsets, rows,
                     workspace, workspace_bytes, stream=None) -> int:
    """Raw status of w4a16_moe_route, without raising (for tests of the error paths)."""
    return int(_lib.w4a16_moe_route(
        _ptr(logits), _ptr(bias), ctypes.addressof(config) if config is not None else None, T,
        _ptr(ids), _ptr(weights), _ptr(offsets), _ptr(rows), _ptr(workspace), workspace_bytes,
        _stream(stream)))


def w4a16_moe_route(logits, bias, T: int, E: int, top_k: int, ids, weights, offsets, rows,
                    workspace, *, scoring: int = W4A16_ROUTE_SOFTMAX, groups: int = 1,
                    groups_kept: int = 1, group_top: int = 1, renormalize: bool = True,
                    scale: float = 1.0, logits_type: int | None = None,
                    workspace_bytes: int | None = None, stream=None) -> None:
    """Experts, weights and the experts' row lists of T tokens from their logits [T][E]
    (float32 or bfloat16; `logits_type` is needed for a raw address only). bias and, where
    w4a16_moe_route_workspace_bytes is 0, workspace may be None."""
    if logits_type is None:
        if _torch is None or not isinstance(logits, _torch.Tensor):
            raise TypeError("logits_type is needed for a raw address")
        if logits.dtype not in (_torch.float32, _torch.bfloat16):
            raise TypeError("logits must be torch.float32 or torch.bfloat16")
        logits_type = W4A16_LOGITS_BF16 if logits.dtype == _torch.bfloat16 else W4A16_LOGITS_F32
    elif logits_type in (W4A16_LOGITS_F32, W4A16_LOGITS_BF16):
        _check_types(logits=(logits,
                             "bfloat16" if logits_type == W4A16_LOGITS_BF16 else "float32"))
    _check_types(bias=(bias, "float32"), ids=(ids, "int32"), weights=(weights, "float32"),
                 offsets=(offsets, "int32"), rows=(rows, "int32"))
    size = 2 if logits_type == W4A16_LOGITS_BF16 else 4
    _check_sizes(logits=(logits, size * T * E), bias=(bias, 4 * E), ids=(ids, 4 * T * top_k),
                 weights=(weights, 4 * T * top_k), offsets=(offsets, 4 * (E + 1)),
                 rows=(rows, 4 * T * top_k))
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    config = w4a16_route_config(E, top_k, scoring, logits_type, groups, groups_kept, group_top,
                                int(bool(renormalize)), scale)
    rc = moe_route_status(logits, bias, config, T, ids, weights, offsets, rows, workspace,
                          workspace_bytes, stream)
    if rc != W4A16_OK:
        raise W4A16Error(rc, "w4a16_moe_route")


def gemm_experts_status(x, qweight, scales, y, rows, offsets, slots, experts, x_div, N, K, group,
                        act=W4A16_ACT_NONE, stream=None) -> int:
    """Raw status of w4a16_gemm_experts, without raising (for tests of the error paths)."""
    return int(_lib.w4a16_gemm_experts(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(y), _ptr(rows),
                                       _ptr(offsets), slots, experts, x_div, N, K, group, act,
                                       _stream(stream)))


def w4a16_gemm_experts(x, qweight, scales, y, rows, offsets, slots: int, experts: int, x_div: int,
                       N: int, K: int, group: int, act: int = W4A16_ACT_NONE,
                       stream=None) -> None:
    """Every expert's W4A16 product over the slots listed for it: y[s] = x[s // x_div] .
    dequant(weights of the expert), with W4A16_ACT_SWIGLU silu(gate) * up."""
    _check_types(x=(x, "bfloat16"), y=(y, "bfloat16"), rows=(rows, "int32"),
                 offsets=(offsets, "int32"))
    if group > 0 and K % group == 0 and x_div > 0 and slots >= 0:
        out = N // 2 if act == W4A16_ACT_SWIGLU else N
        _check_sizes(x=(x, 2 * -(-slots // x_div) * K), y=(y, 2 * slots * out),
                     qweight=(qweight, experts * w4a16_qweight_bytes(N, K)),
                     scales=(scales, experts * w4a16_scales_bytes(N, K, group)),
                     rows=(rows, 4 * slots), offsets=(offsets, 4 * (experts + 1)))
    rc = gemm_experts_status(x, qweight, scales, y, rows, offsets, slots, experts, x_div, N, K,
                             group, act, stream)
    if rc != W4A16_OK:
        raise W4A16Error(rc, "w4a16_gemm_experts")


def moe_combine_status(y, ids, weights, base, out, T, top_k, N, stream=None) -> int:
    """Raw status of w4a16_moe_combine, without raising (for tests of the error paths)."""
    return int(_lib.w4a16_moe_combine(_ptr(y), _ptr(ids), _ptr(weights), _ptr(base), _ptr(out), T,
                                      top_k, N, _stream(stream)))


def w4a16_moe_combine(y, ids, weights, base, out, T: int, top_k: int, N: int,
                      stream=None) -> None:
    """out[T][N] = base (None: 0) + weighted sum of each token's top_k rows of y."""
    _check_types(y=(y, "bfloat16"), base=(base, "bfloat16"), out=(out, "bfloat16"),
                 ids=(ids, "int32"), weights=(weights, "float32"))
    _check_sizes(y=(y, 2 * T * top_k * N), base=(base, 2 * T * N), out=(out, 2 * T * N),
                 ids=(ids, 4 * T * top_k), weights=(weights, 4 * T * top_k))
    rc = moe_combine_status(y, ids, weights, base, out, T, top_k, N, stream)
    if rc != W4A16_OK:
        raise W4A16Error(rc, "w4a16_moe_combine")


def w8a8_qweight_bytes(N: int, K: int) -> int:
    return int(_lib.w8a8_qweight_bytes(N, K))


def w8a8_pack_status(q_ptr, out_ptr, N, K) -> int:
    """Raw status of w8a8_pack on raw host addresses (for tests of the error paths)."""
    return int(_lib.w8a8_pack(q_ptr, out_ptr, N, K))


def w8a8_pack(q: np.ndarray) -> np.ndarray:
    """Host packing of int8 weights [N, K] into the device arrangement (flat int8 array)."""
    q = np.ascontiguousarray(q)
    if q.dtype != np.int8 or q.ndim != 2:
        raise TypeError("q must be a 2-D int8 array")
    N, K = q.shape
    if K % 16 != 0:
        raise W4A16Error(W4A16_ERR_INVALID_ARG, "w8a8_pack")
    out = np.empty(w8a8_qweight_bytes(N, K), dtype=np.int8)
    rc = w8a8_pack_status(q.ctypes.data, out.ctypes.data, N, K)
    if rc != W4A16_OK:
        raise W4A16Error(rc, "w8a8_pack")
    return out


def w8a8_gemm_status(xq, sx, qweight, scales, y, M, N, K, stream=None) -> int:
    """Raw status of w8a8_gemm, without raising (for tests of the error paths)."""
    return int(_lib.w8a8_gemm(_ptr(xq), _ptr(sx), _ptr(qweight), _ptr(scales), _ptr(y), M, N, K,
                              _stream(stream)))


def w8a8_gemm(xq, sx, qweight, scales, y, M: int, N: int, K: int, stream=None) -> None:
    """y[M][N] (bf16) = 8-bit integer product of the codes and row scales written by
    w4a8_quantize and the weights written by w8a8_pack, with fp32 scales per column."""
    _check_types(xq=(xq, "int8"), sx=(sx, "float32"), scales=(scales, "float32"),
                 y=(y, "bfloat16"))
    _check_sizes(xq=(xq, M * K), sx=(sx, 4 * M), y=(y, 2 * M * N), scales=(scales, 4 * N),
                 qweight=(qweight, w8a8_qweight_bytes(N, K)))
    rc = w8a8_gemm_status(xq, sx, qweight, scales, y, M, N, K, stream)
    if rc != W4A16_OK:
        raise W4A16Error(rc, "w8a8_gemm")
