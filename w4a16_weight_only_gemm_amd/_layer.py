"""Binding of include/w4a16_layer.h: the product with an epilogue, the norms around a
block and a whole expert layer for a few tokens. Argument marshalling only; the names
match the C ABI and are re-exported by the package."""
from __future__ import annotations

import ctypes
import functools
import struct

from . import W4A16_OK, W4A16Error, _lib, _ptr, _stream, w4a16_qweight_bytes, w4a16_scales_bytes
from ._moe import (_BF16, _F32, _I8, _I32, W4A16_ACT_NONE, W4A16_ACT_SWIGLU, W4A16_LOGITS_BF16,
                   W4A16_LOGITS_F32, W4A16_ROUTE_SOFTMAX, _at, _device, _on, _Tensor,
                   w4a16_route_config)

W4A16_ACT_SILU = 2
W4A16_ACT_GELU = 3
W4A16_ACT_GELU_TANH = 4
W4A16_ACT_RELU = 5
W4A16_ACT_GEGLU = 6
W4A16_NORM_MAX_COLUMNS = 65536
W4A16_NORM_RMS = 0
W4A16_NORM_LAYER = 1
W4A16_RESIDUAL_BF16 = 0
W4A16_RESIDUAL_F32 = 1
W4A16_MOE_LAYER_MAX_TOKENS = 16

_vp, _int, _sz, _f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float


class w4a16_epilogue(ctypes.Structure):
    _fields_ = [("bias", _vp), ("residual", _vp), ("scale", _f32), ("act", _int)]


class w4a16_norm_args(ctypes.Structure):
    _fields_ = [("y", _vp), ("post_norm", _int), ("gate_rows", _int), ("post_weight", _vp),
                ("post_bias", _vp), ("gate", _vp), ("scale", _f32), ("residual_type", _int),
                ("residual", _vp), ("residual_out", _vp), ("weight", _vp), ("bias", _vp),
                ("x", _vp), ("xq", _vp), ("sx", _vp), ("kind", _int), ("unit_offset", _int),
                ("eps", _f32)]


class w4a16_moe_layer_args(ctypes.Structure):
    _fields_ = [("route", w4a16_route_config), ("router_type", _int), ("hidden", _int),
                ("width", _int), ("group", _int), ("router", _vp), ("route_bias", _vp),
                ("gate_up", _vp), ("gate_up_scales", _vp), ("down", _vp), ("down_scales", _vp)]


# Every symbol include/w4a16_layer.h declares, with its ctypes signature.
LAYER_SIGNATURES = {
    "w4a16_gemm_epilogue": (_int, [_vp, _vp, _vp, _vp, _vp, _int, _int, _int, _int, _vp]),
    "w4a16_norm": (_int, [_vp, _int, _int, _vp]),
    "w4a16_moe_layer_workspace_bytes": (_sz, [_int, _int, _int, _int, _int]),
    "w4a16_moe_layer": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _int, _vp, _sz, _vp]),
}
for _name, (_res, _args) in LAYER_SIGNATURES.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


# The same structures as bytes: a call's own, made in a fraction of the time ctypes takes
# (small calls are bound by the host).
_PACK_EPILOGUE = struct.Struct("@PPfi0P").pack
_PACK_MOE_LAYER = struct.Struct("@8if4iPPPPPP").pack
_PACK_NORM = struct.Struct("@PiiPPPfiPPPPPPPiif0P").pack


def _address(args):
    return ctypes.addressof(args) if args is not None else None


def _or_0(name: str, t, dtype, nbytes: int, dev: int) -> int:
    """_at for a field of a packed structure, where an absent buffer is 0."""
    return 0 if t is None else _at(name, t, dtype, nbytes, dev) or 0


def gemm_epilogue_status(x, qweight, scales, epilogue: w4a16_epilogue | None, y, M, N, K, group,
                         stream=None) -> int:
    """Raw status of w4a16_gemm_epilogue, without raising (for tests of the error paths)."""
    return int(_lib.w4a16_gemm_epilogue(_ptr(x), _ptr(qweight), _ptr(scales), _address(epilogue),
                                        _ptr(y), M, N, K, group, _stream(stream)))


@functools.lru_cache(maxsize=1024)
def _packed_bytes(N: int, K: int, group: int):
    return w4a16_qweight_bytes(N, K), w4a16_scales_bytes(N, K, group)


def w4a16_gemm_epilogue(x, qweight, scales, y, M: int, N: int, K: int, group: int, *, bias=None,
                        residual=None, act: int = W4A16_ACT_NONE, scale: float = 1.0,
                        stream=None) -> None:
    """y = residual + scale * act(x . dequant(weights) + bias), in fp32 and rounded once; the
    gated activations (W4A16_ACT_SWIGLU, W4A16_ACT_GEGLU) write N / 2 columns. residual may be
    y itself."""
    dev = _device()
    out = N // 2 if act in (W4A16_ACT_SWIGLU, W4A16_ACT_GEGLU) else N
    qb = sb = 0
    if N >= 0 and K >= 0 and group > 0 and group % 32 == 0 and K % group == 0:
        qb, sb = _packed_bytes(N, K, group)
    ep = _PACK_EPILOGUE(_or_0("bias", bias, _BF16, 2 * N, dev),
                        _or_0("residual", residual, _BF16, 2 * M * out, dev), scale, act)
    rc = _lib.w4a16_gemm_epilogue(
        _at("x", x, _BF16, 2 * M * K, dev), _at("qweight", qweight, None, qb, dev),
        _at("scales", scales, None, sb, dev), ep,
        _at("y", y, _BF16, 2 * M * out, dev), M, N, K, group, _on(stream, dev))
    if rc != W4A16_OK:
        raise W4A16Error(rc, "w4a16_gemm_epilogue")


def norm_status(args: w4a16_norm_args | None, T, N, stream=None) -> int:
    """Raw status of w4a16_norm, without raising (for tests of the error paths)."""
    return int(_lib.w4a16_norm(_address(args), T, N, _stream(stream)))


def w4a16_norm(T: int, N: int, *, y=None, residual=None, residual_out=None, post_norm: bool = False,
               post_weight=None, post_bias=None, gate=None, gate_rows: int = 1, scale: float = 1.0,
               weight=None, bias=None, x=None, xq=None, sx=None, kind: int = W4A16_NORM_RMS,
               eps: float = 1e-6, unit_offset: bool = False, residual_type: int | None = None,
               stream=None) -> None:
    """r = residual + scale * gate * (norm of) y and the norm of r for the next block, T rows of
    N: r into residual_out (which may be residual), its norm into x (bfloat16) or into xq and sx
    (the codes and scales of w4a8_quantize). residual is bfloat16 or float32; residual_type is
    needed only where both it and residual_out are raw addresses."""
    dev = _device()
    if residual_type is None:
        one = residual if isinstance(residual, _Tensor) else residual_out
        residual_type = (W4A16_RESIDUAL_F32 if isinstance(one, _Tensor) and one.dtype is _F32
                         else W4A16_RESIDUAL_BF16)
    wide = residual_type == W4A16_RESIDUAL_F32
    stored, row, vec = _F32 if wide else _BF16, 2 * T * N, 2 * N
    full = 2 * row if wide else row
    gates = -(-T // gate_rows) if gate_rows > 0 else 0
    args = _PACK_NORM(
        _or_0("y", y, _BF16, row, dev), 1 if post_norm else 0, gate_rows,
        _or_0("post_weight", post_weight, _BF16, vec, dev),
        _or_0("post_bias", post_bias, _BF16, vec, dev), _or_0("gate", gate, _BF16, gates * vec, dev),
        scale, residual_type, _or_0("residual", residual, stored, full, dev),
        _or_0("residual_out", residual_out, stored, full, dev),
        _or_0("weight", weight, _BF16, vec, dev), _or_0("bias", bias, _BF16, vec, dev),
        _or_0("x", x, _BF16, row, dev), _or_0("xq", xq, _I8, T * N, dev),
        _or_0("sx", sx, _F32, 4 * T, dev), kind, 1 if unit_offset else 0, eps)
    rc = _lib.w4a16_norm(args, T, N, _on(stream, dev))
    if rc != W4A16_OK:
        raise W4A16Error(rc, "w4a16_norm")


def w4a16_moe_layer_workspace_bytes(T: int, experts: int, top_k: int, hidden: int,
                                    width: int) -> int:
    return int(_lib.w4a16_moe_layer_workspace_bytes(T, experts, top_k, hidden, width))


def moe_layer_status(layer: w4a16_moe_layer_args | None, x, live, base, out, ids, weights, T,
                     workspace, workspace_bytes, stream=None) -> int:
    """Raw status of w4a16_moe_layer, without raising (for tests of the error paths)."""
    return int(_lib.w4a16_moe_layer(_address(layer), _ptr(x), _ptr(live), _ptr(base), _ptr(out),
                                    _ptr(ids), _ptr(weights), T, _ptr(workspace), workspace_bytes,
                                    _stream(stream)))


def w4a16_moe_layer(x, router, gate_up, gate_up_scales, down, down_scales, out, ids, weights,
                    T: int, E: int, top_k: int, hidden: int, width: int, group: int, workspace, *,
                    route_bias=None, base=None, live=None, scoring: int = W4A16_ROUTE_SOFTMAX,
                    groups: int = 1, groups_kept: int = 1, group_top: int = 1,
                    renormalize: bool = True, scale: float = 1.0, router_type: int | None = None,
                    workspace_bytes: int | None = None, stream=None) -> None:
    """A whole mixture-of-experts layer for up to W4A16_MOE_LAYER_MAX_TOKENS tokens: out = base
    + the weighted outputs of each token's top_k experts, chosen by the router's logits
    (router [E][hidden], float32 or bfloat16; `router_type` is needed for a raw address only).
    live: int32 [T], 0 for a padding token."""
    if router_type is None:
        if not isinstance(router, _Tensor):
            raise TypeError("router_type is needed for a raw address")
        if router.dtype is _F32:
            router_type = W4A16_LOGITS_F32
        elif router.dtype is _BF16:
            router_type = W4A16_LOGITS_BF16
        else:
            raise TypeError("router must be torch.float32 or torch.bfloat16")
    half = router_type == W4A16_LOGITS_BF16
    dev = _device()
    gb = gs = db = ds = 0
    if hidden > 0 and width > 0 and group > 0 and group % 32 == 0 and hidden % group == 0 and width % group == 0:
        gb, gs = _packed_bytes(2 * width, hidden, group)
        db, ds = _packed_bytes(hidden, width, group)
    if workspace_bytes is None:
        workspace_bytes = workspace.nbytes if isinstance(workspace, _Tensor) else 0
    row, places = 2 * T * hidden, 4 * T * top_k
    args = _PACK_MOE_LAYER(
        E, top_k, scoring, router_type, groups, groups_kept, group_top, 1 if renormalize else 0,
        scale, router_type, hidden, width, group,
        _or_0("router", router, _BF16 if half else _F32, (2 if half else 4) * E * hidden, dev),
        _or_0("route_bias", route_bias, _F32, 4 * E, dev),
        _or_0("gate_up", gate_up, None, E * gb, dev),
        _or_0("gate_up_scales", gate_up_scales, None, E * gs, dev),
        _or_0("down", down, None, E * db, dev), _or_0("down_scales", down_scales, None, E * ds, dev))
    rc = _lib.w4a16_moe_layer(
        args, _at("x", x, _BF16, row, dev), _at("live", live, _I32, 4 * T, dev),
        _at("base", base, _BF16, row, dev), _at("out", out, _BF16, row, dev),
        _at("ids", ids, _I32, places, dev), _at("weights", weights, _F32, places, dev), T,
        _at("workspace", workspace, None, workspace_bytes, dev), workspace_bytes, _on(stream, dev))
    if rc != W4A16_OK:
        raise W4A16Error(rc, "w4a16_moe_layer")
