"""Host-only tests of include/w4a16_layer.h: exported symbols and bindings,
structures of the C ABI's size, workspace sizes, and every refusal (each returns
before any launch; the addresses are never used)."""
import ctypes
import os
import re
import subprocess

import pytest

import w4a16_weight_only_gemm_amd as w4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B = 1 << 20, (1 << 20) + 8  # aligned and misaligned addresses, never dereferenced
ODD = (1 << 20) + 1
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
INF, NAN = float("inf"), float("nan")


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "w4a16_layer.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(w4a16_\w+)\s*\(", text)))
    assert names == sorted(w4.LAYER_SIGNATURES)
    lib = ctypes.CDLL(w4.LIB_PATH)
    for name in names:
        assert hasattr(lib, name) and hasattr(w4, name), name


def test_structures_match_the_header(tmp_path):
    """Sizes and field offsets of the ctypes structures against the C compiler's."""
    structs = {"w4a16_epilogue": w4.w4a16_epilogue, "w4a16_norm_args": w4.w4a16_norm_args,
               "w4a16_moe_layer_args": w4.w4a16_moe_layer_args}
    lines = []
    for name, st in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in st._fields_]
    src = tmp_path / "s.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "w4a16_layer.h"\n'
                   "int main(void) {" + "\n".join(lines) + "return 0;}")
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for st in structs.values():
        want += [ctypes.sizeof(st)] + [getattr(st, f).offset for f, _ in st._fields_]
    assert got == want


def test_packed_structures_are_the_same():
    """The bytes the calls pass, against the ctypes structures of the same values."""
    from w4a16_weight_only_gemm_amd import _layer
    assert _layer._PACK_EPILOGUE(1, 2, 0.5, 3) == bytes(w4.w4a16_epilogue(1, 2, 0.5, 3))
    v = [11, 1, 2, 12, 13, 14, 0.25, 1, 15, 16, 17, 18, 19, 20, 21, 1, 1, 0.125]
    assert _layer._PACK_NORM(*v) == bytes(w4.w4a16_norm_args(*v))
    r = [8, 2, 1, 1, 4, 2, 2, 1, 1.5]
    tail = [1, 256, 128, 32, 31, 32, 33, 34, 35, 36]
    assert (_layer._PACK_MOE_LAYER(*r, *tail)
            == bytes(w4.w4a16_moe_layer_args(w4.w4a16_route_config(*r), *tail)))


def ep(bias=None, residual=None, scale=1.0, act=0):
    return w4.w4a16_epilogue(bias, residual, scale, act)


def test_epilogue_refusals():
    st = w4.gemm_epilogue_status
    ok = lambda e, M=4, N=64, K=256, g=128, x=A, q=A, s=A, y=A: st(x, q, s, e, y, M, N, K, g)  # noqa: E731
    assert ok(ep(), M=0) == OK
    assert ok(None) == INVALID
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(x=None), dict(q=None), dict(s=None), dict(y=None)):
        assert ok(ep(), **bad) == INVALID, bad
    for bad in (ep(act=-1), ep(act=7), ep(scale=INF), ep(scale=NAN), ep(scale=-INF)):
        assert ok(bad) == INVALID
        assert ok(bad, M=0) == INVALID
    for bad in (dict(N=0), dict(K=0), dict(g=48), dict(g=512, K=1024), dict(K=200), dict(g=0)):
        assert ok(ep(), **bad) == UNSUPPORTED, bad
    for act in (w4.W4A16_ACT_SWIGLU, w4.W4A16_ACT_GEGLU):
        for N in (16, 33, 48, 100):
            assert ok(ep(act=act), N=N) == UNSUPPORTED, (act, N)
    for bad in (dict(x=B), dict(q=B), dict(s=B), dict(y=B)):
        assert ok(ep(), **bad) == MISALIGNED, bad
    assert ok(ep(residual=B)) == MISALIGNED and ok(ep(bias=ODD)) == MISALIGNED
    # grids past 2^32 threads, and rows past what a group-256 product holds
    assert ok(ep(), M=65535 * 16, N=2**31 - 16, K=256, g=256) == UNSUPPORTED
    assert ok(ep(), M=65535 * 16 + 1, N=16, K=256, g=256) == UNSUPPORTED


def norm(**kw):
    a = dict(y=A, post_norm=0, gate_rows=1, post_weight=None, post_bias=None, gate=None, scale=1.0,
             residual_type=0, residual=A, residual_out=A, weight=A, bias=None, x=A, xq=None,
             sx=None, kind=0, unit_offset=0, eps=1e-6)
    a.update(kw)
    return w4.w4a16_norm_args(**a)


def test_norm_refusals():
    st = w4.norm_status
    assert st(norm(), 0, 64) == OK and st(None, 1, 64) == INVALID
    assert st(norm(), -1, 64) == INVALID and st(norm(), 1, -1) == INVALID
    for bad in (dict(kind=2), dict(kind=-1), dict(residual_type=2), dict(residual_type=-1), dict(eps=-1e-9),
                dict(eps=NAN), dict(eps=INF), dict(scale=INF), dict(scale=NAN), dict(gate_rows=0),
                dict(gate_rows=-3), dict(xq=A, x=None), dict(sx=A), dict(xq=A, sx=A),
                dict(y=None, residual=None), dict(residual_out=None, x=None)):
        assert st(norm(**bad), 1, 64) == INVALID, bad
        assert st(norm(**bad), 0, 64) == INVALID, bad
    # without a block its fields count for nothing
    assert st(norm(y=None, scale=NAN, gate_rows=0), 0, 64) == OK
    for N in (0, w4.W4A16_NORM_MAX_COLUMNS + 1):
        assert st(norm(), 1, N) == UNSUPPORTED, N
    assert st(norm(x=None, xq=A, sx=A), 1, 72) == UNSUPPORTED
    for bad in ("y", "gate", "residual", "residual_out", "x"):
        assert st(norm(**{bad: B}), 1, 64) == MISALIGNED, bad
    assert st(norm(x=None, xq=B, sx=A), 1, 64) == MISALIGNED
    assert st(norm(x=None, xq=A, sx=A + 2), 1, 64) == MISALIGNED
    for bad in ("weight", "bias", "post_weight", "post_bias"):
        assert st(norm(**{bad: ODD}), 1, 64) == MISALIGNED, bad
    assert st(norm(), 2**31 - 1, 65536) == UNSUPPORTED  # a grid past 2^32 threads


def layer(**kw):
    r = dict(experts=16, top_k=4, scoring=0, logits_type=0, groups=1, groups_kept=1, group_top=1,
             renormalize=1, scale=1.0)
    a = dict(router_type=0, hidden=256, width=128, group=128, router=A, route_bias=None, gate_up=A,
             gate_up_scales=A, down=A, down_scales=A)
    for k, v in kw.items():
        (r if k in r else a)[k] = v
    return w4.w4a16_moe_layer_args(route=w4.w4a16_route_config(*r.values()), **a)


def test_moe_layer_refusals():
    def st(l, T=4, x=A, live=None, base=None, out=A, ids=A, w=A, ws=A, n=1 << 40):
        return w4.moe_layer_status(l, x, live, base, out, ids, w, T, ws, n)
    assert st(layer(), T=0) == OK and st(None) == INVALID and st(layer(), T=-1) == INVALID
    for bad in (dict(experts=0), dict(experts=1025), dict(top_k=0), dict(top_k=17), dict(top_k=33, experts=64),
                dict(scoring=2), dict(groups=0), dict(groups=3), dict(groups=65, experts=130), dict(groups_kept=0),
                dict(groups_kept=2), dict(group_top=0), dict(group_top=3), dict(scale=INF), dict(scale=NAN),
                dict(router_type=2), dict(router_type=-1), dict(hidden=-1), dict(width=-1)):
        assert st(layer(**bad)) == INVALID, bad
        assert st(layer(**bad), T=0) == INVALID, bad
    assert st(layer(logits_type=77), T=0) == OK
    for bad in (dict(x=None), dict(out=None), dict(ids=None), dict(w=None), dict(ws=None)):
        assert st(layer(), **bad) == INVALID, bad
    for bad in ("router", "gate_up", "gate_up_scales", "down", "down_scales"):
        assert st(layer(**{bad: None})) == INVALID, bad
        assert st(layer(**{bad: B})) == MISALIGNED, bad
    assert st(layer(), T=17) == UNSUPPORTED
    for bad in (dict(hidden=0), dict(width=0), dict(group=0), dict(group=96), dict(hidden=192), dict(width=64),
                dict(hidden=1 << 17, width=1 << 17), dict(width=2**30, hidden=128),
                dict(hidden=32, width=1 << 27, group=32)):  # inner rows past 4 GB
        assert st(layer(**bad)) == UNSUPPORTED, bad
    need = w4.w4a16_moe_layer_workspace_bytes(4, 16, 4, 256, 128)
    assert need > 0 and st(layer(), n=need - 1) == INVALID
    assert st(layer(), ws=A + 128) == MISALIGNED
    for bad in (dict(x=B), dict(base=B), dict(out=B), dict(ids=A + 2), dict(w=A + 2), dict(live=A + 2)):
        assert st(layer(), **bad) == MISALIGNED, bad
    assert st(layer(route_bias=A + 2)) == MISALIGNED


def test_moe_layer_workspace_bytes():
    n = w4.w4a16_moe_layer_workspace_bytes
    for bad in ((-1, 8, 2, 128, 128), (17, 8, 2, 128, 128), (1, 0, 1, 128, 128), (1, 1025, 2, 128, 128),
                (1, 8, 0, 128, 128), (1, 8, 9, 128, 128), (1, 64, 33, 128, 128), (1, 8, 2, 0, 128), (1, 8, 2, 128, 0)):
        assert n(*bad) == 0, bad
    sizes = [n(T, 128, 8, 5120, 1024) for T in range(1, 17)]
    assert sizes == sorted(sizes) and sizes[0] > 0  # enough for fewer tokens
    # the logits, the experts' inner rows and a counter per 16 columns fit
    assert n(16, 1024, 32, 8192, 2048) >= 16 * 1024 * 8 + 16 * 32 * 2048 * 2 + 8192 // 16 * 4


@pytest.mark.parametrize("name", ["w4a16_gemm_epilogue", "w4a16_norm", "w4a16_moe_layer"])
def test_binding_raises_what_the_library_refuses(name):
    with pytest.raises(w4.W4A16Error):
        if name == "w4a16_gemm_epilogue":
            w4.w4a16_gemm_epilogue(A, A, A, A, 1, 64, 200, 128, stream=1)
        elif name == "w4a16_norm":
            w4.w4a16_norm(1, 64, y=A, stream=1)
        else:
            w4.w4a16_moe_layer(A, A, A, A, A, A, A, A, A, 17, 16, 4, 256, 128, 128, A,
                               router_type=0, workspace_bytes=1 << 40, stream=1)


def test_binding_checks_buffers():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current device"):
        w4.w4a16_norm(4, 64, y=x, x=A, stream=1)
    with pytest.raises(TypeError, match="router_type"):
        w4.w4a16_moe_layer(A, A, A, A, A, A, A, A, A, 1, 16, 4, 256, 128, 128, A)
    with pytest.raises(TypeError, match="bfloat16"):
        w4.w4a16_norm(4, 64, y=x.float(), x=A, stream=1)
