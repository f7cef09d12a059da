"""Binding of include/w4a16_moe.h: routing, experts' products, combine and the
8-bit integer product. Argument marshalling only; the names match the C ABI and
are re-exported by the package."""
from __future__ import annotations

import ctypes
import functools

import numpy as np

from . import (W4A16_ERR_INVALID_ARG, W4A16_OK, W4A16Error, _lib, _ptr, _stream, _torch,
               w4a16_qweight_bytes, w4a16_scales_bytes)

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


if _torch is not None:
    _Tensor, _F32, _BF16 = _torch.Tensor, _torch.float32, _torch.bfloat16
    _I32, _I8 = _torch.int32, _torch.int8
    _raw_stream = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
else:  # pragma: no cover - torch is optional for host-only use
    _Tensor, _F32, _BF16, _I32, _I8, _raw_stream = (), None, None, None, None, None


def _device() -> int:
    """The current device's index, or -2 where no device tensor can exist yet."""
    if _torch is None or not _torch.cuda.is_initialized():
        return -2
    return _torch.cuda.current_device()


def _at(name: str, t, dtype, nbytes: int, dev: int):
    """Address of a buffer: a raw address or None as it is, a tensor after its checks
    (any dtype where `dtype` is None). A few hundred nanoseconds each: small calls
    are bound by the host."""
    if isinstance(t, _Tensor):
        if dtype is not None and t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}")
        if t.get_device() != dev:
            raise ValueError(f"{name} must be on the current device")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.nbytes < nbytes:
            raise ValueError(f"{name} holds {t.nbytes} bytes, needs {nbytes}")
        return t.data_ptr()
    if t is None or isinstance(t, int):
        return t
    raise TypeError(f"unsupported buffer type {type(t)} for {name}")


def _on(stream, dev: int):
    """Address of the stream: the given one, else torch's current stream of `dev`."""
    if stream is None and dev >= 0 and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


@functools.lru_cache(maxsize=256)
def _config(*fields) -> w4a16_route_config:
    return w4a16_route_config(*fields)


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
        if not isinstance(logits, _Tensor):
            raise TypeError("logits_type is needed for a raw address")
        if logits.dtype is _F32:
            logits_type = W4A16_LOGITS_F32
        elif logits.dtype is _BF16:
            logits_type = W4A16_LOGITS_BF16
        else:
            raise TypeError("logits must be torch.float32 or torch.bfloat16")
    bf16 = logits_type == W4A16_LOGITS_BF16
    dev = _device()
    places = 4 * T * top_k
    if workspace_bytes is None:
        workspace_bytes = workspace.nbytes if isinstance(workspace, _Tensor) else 0
    rc = _lib.w4a16_moe_route(
        _at("logits", logits, _BF16 if bf16 else _F32, (2 if bf16 else 4) * T * E, dev),
        _at("bias", bias, _F32, 4 * E, dev),
        ctypes.addressof(_config(E, top_k, scoring, logits_type, groups, groups_kept, group_top,
                                 1 if renormalize else 0, scale)),
        T, _at("ids", ids, _I32, places, dev), _at("weights", weights, _F32, places, dev),
        _at("offsets", offsets, _I32, 4 * (E + 1), dev), _at("rows", rows, _I32, places, dev),
        _at("workspace", workspace, None, workspace_bytes, dev), workspace_bytes,
        _on(stream, dev))
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
    dev = _device()
    xb = yb = qb = sb = 0
    if group > 0 and K % group == 0 and x_div > 0:
        xb = 2 * -(-slots // x_div) * K
        yb = 2 * slots * (N // 2 if act == W4A16_ACT_SWIGLU else N)
        qb = experts * w4a16_qweight_bytes(N, K)
        sb = experts * w4a16_scales_bytes(N, K, group)
    rc = _lib.w4a16_gemm_experts(
        _at("x", x, _BF16, xb, dev), _at("qweight", qweight, None, qb, dev),
        _at("scales", scales, None, sb, dev), _at("y", y, _BF16, yb, dev),
        _at("rows", rows, _I32, 4 * slots, dev),
        _at("offsets", offsets, _I32, 4 * (experts + 1), dev), slots, experts, x_div, N, K, group,
        act, _on(stream, dev))
    if rc != W4A16_OK:
        raise W4A16Error(rc, "w4a16_gemm_experts")


def moe_combine_status(y, ids, weights, base, out, T, top_k, N, stream=None) -> int:
    """Raw status of w4a16_moe_combine, without raising (for tests of the error paths)."""
    return int(_lib.w4a16_moe_combine(_ptr(y), _ptr(ids), _ptr(weights), _ptr(base), _ptr(out), T,
                                      top_k, N, _stream(stream)))


def w4a16_moe_combine(y, ids, weights, base, out, T: int, top_k: int, N: int,
                      stream=None) -> None:
    """out[T][N] = base (None: 0) + weighted sum of each token's top_k rows of y."""
    dev = _device()
    row, places = 2 * T * N, 4 * T * top_k
    rc = _lib.w4a16_moe_combine(
        _at("y", y, _BF16, row * top_k, dev), _at("ids", ids, _I32, places, dev),
        _at("weights", weights, _F32, places, dev), _at("base", base, _BF16, row, dev),
        _at("out", out, _BF16, row, dev), T, top_k, N, _on(stream, dev))
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
    dev = _device()
    rc = _lib.w8a8_gemm(
        _at("xq", xq, _I8, M * K, dev), _at("sx", sx, _F32, 4 * M, dev),
        _at("qweight", qweight, None, w8a8_qweight_bytes(N, K), dev),
        _at("scales", scales, _F32, 4 * N, dev), _at("y", y, _BF16, 2 * M * N, dev), M, N, K,
        _on(stream, dev))
    if rc != W4A16_OK:
        raise W4A16Error(rc, "w8a8_gemm")
