"""Host-only tests of include/w4a16_moe.h: exported symbols and bindings, the
W8A8 packing against an entry-by-entry definition, sizes, and every refusal
(each returns before any launch; the addresses are never used)."""
import ctypes
import os
import re

import numpy as np
import pytest

import moe_ref
import w4a16_weight_only_gemm_amd as w4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B = 1 << 20, (1 << 20) + 8  # aligned and misaligned addresses, never dereferenced
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "w4a16_moe.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(w(?:4a16|8a8)_\w+)\s*\(", text)))
    assert names == sorted(w4.MOE_SIGNATURES)
    lib = ctypes.CDLL(w4.LIB_PATH)
    for name in names:
        assert hasattr(lib, name) and hasattr(w4, name), name


@pytest.mark.parametrize("N,K", [(1, 16), (16, 64), (17, 48), (33, 80), (20, 128), (5, 208)])
def test_w8a8_pack(N, K):
    q = np.random.default_rng(N * K).integers(-128, 128, (N, K)).astype(np.int8)
    packed = w4.w8a8_pack(q)
    assert packed.size == w4.w8a8_qweight_bytes(N, K)
    assert np.array_equal(packed, moe_ref.w8a8_pack(q))


def test_w8a8_pack_hand_position():
    q = np.zeros((18, 144), np.int8)
    q[17, 64 + 16 + 5] = 77  # block 1, step 1, lane 16 + 1, offset 5 in byte 3
    at = np.flatnonzero(w4.w8a8_pack(q))
    assert at.tolist() == [((1 * 3 + 1) * 64 + 17) * 16 + 3]


def test_w8a8_sizes_and_pack_refusals():
    assert w4.w8a8_qweight_bytes(7168, 5120) == 7168 * 5120
    assert w4.w8a8_qweight_bytes(17, 16) == 2 * 1024
    assert w4.w8a8_qweight_bytes(0, 64) == 0 and w4.w8a8_qweight_bytes(4, 0) == 0
    assert w4.w8a8_qweight_bytes(-1, 16) == 0 and w4.w8a8_qweight_bytes(4, 24) == 0
    assert w4.w8a8_pack_status(None, None, 0, 64) == OK
    assert w4.w8a8_pack_status(None, None, 4, 64) == INVALID
    assert w4.w8a8_pack_status(A, A, -1, 64) == INVALID
    assert w4.w8a8_pack_status(A, A, 4, 72) == INVALID
    with pytest.raises(TypeError):
        w4.w8a8_pack(np.zeros((4, 16), np.int16))


def test_w8a8_gemm_refusals():
    st = w4.w8a8_gemm_status
    assert st(A, A, A, A, A, 0, 64, 64) == OK
    assert st(A, A, A, A, A, -1, 64, 64) == INVALID
    for i in range(5):
        p = [A] * 5
        p[i] = None
        assert st(*p, 1, 64, 64) == INVALID
    for M, N, K in [(1, 0, 64), (1, 64, 0), (1, 64, 24), (1, 64, 131072 + 16), (1, 1 << 20, 8192)]:
        assert st(A, A, A, A, A, M, N, K) == UNSUPPORTED, (M, N, K)
    for i in (0, 2, 4):
        p = [A] * 5
        p[i] = B
        assert st(*p, 1, 64, 64) == MISALIGNED
    assert st(A, A + 2, A, A, A, 1, 64, 64) == MISALIGNED


def _cfg(**kw):
    d = dict(experts=64, top_k=4, scoring=0, logits_type=0, groups=1, groups_kept=1, group_top=1,
             renormalize=1, scale=1.0)
    d.update(kw)
    return w4.w4a16_route_config(*(d[n] for n, _ in w4.w4a16_route_config._fields_))


def _route(cfg, T=4, logits=A, bias=None, ids=A, weights=A, offsets=A, rows=A, ws=None, nws=0):
    return w4.moe_route_status(logits, bias, cfg, T, ids, weights, offsets, rows, ws, nws)


@pytest.mark.parametrize("bad", [
    dict(experts=0), dict(experts=1025), dict(top_k=0), dict(top_k=33), dict(experts=8, top_k=9),
    dict(scoring=2), dict(logits_type=2), dict(groups=0), dict(groups=65, experts=130),
    dict(groups=3), dict(groups=4, groups_kept=0), dict(groups=4, groups_kept=5),
    dict(group_top=0), dict(group_top=3), dict(scale=float("nan")), dict(scale=float("inf"))],
    ids=str)
def test_route_bad_config(bad):
    assert _route(_cfg(**bad)) == INVALID


def test_route_refusals():
    assert _route(None) == INVALID
    assert _route(_cfg(), T=-1) == INVALID
    for name in ("logits", "ids", "weights", "offsets", "rows"):
        assert _route(_cfg(), **{name: None}) == INVALID, name
    assert _route(_cfg(), logits=B) == MISALIGNED
    for name in ("bias", "ids", "weights", "offsets", "rows"):
        assert _route(_cfg(), **{name: A + 2}) == MISALIGNED, name
    need = w4.w4a16_moe_route_workspace_bytes(1000, 64)
    assert need > 0 and w4.w4a16_moe_route_workspace_bytes(1, 64) == 0
    assert _route(_cfg(), T=1000) == INVALID
    assert _route(_cfg(), T=1000, ws=A, nws=need - 1) == INVALID
    assert _route(_cfg(), T=1000, ws=B, nws=need) == MISALIGNED
    assert _route(_cfg(), T=1 << 29, ws=A, nws=1 << 40) == UNSUPPORTED
    assert w4.w4a16_moe_route_workspace_bytes(-1, 64) == 0
    assert w4.w4a16_moe_route_workspace_bytes(1000, 0) == 0
    assert w4.w4a16_moe_route_workspace_bytes(1000, 1025) == 0
    for E in (1, 8, 200, 256, 257, 1024):  # a workspace for the most tokens serves fewer
        sizes = [w4.w4a16_moe_route_workspace_bytes(T, E)
                 for T in (*range(0, 40), 1000, 1024, 1025, 4096, 4097, 8192, 8193, 100000)]
        assert sizes == sorted(sizes), E
    for T in (0, 17, 1025, 9000):
        sizes = [w4.w4a16_moe_route_workspace_bytes(T, E) for E in range(1, 1025)]
        assert sizes == sorted(sizes), T


def test_experts_refusals():
    def st(x=A, qw=A, sp=A, y=A, rows=A, offsets=A, slots=8, E=4, div=2, N=64, K=128, g=128, act=0):
        return w4.gemm_experts_status(x, qw, sp, y, rows, offsets, slots, E, div, N, K, g, act)
    assert st(slots=0) == OK
    for kw in (dict(slots=-1), dict(E=0), dict(E=1025), dict(div=0), dict(N=-1), dict(K=-1),
               dict(act=2), dict(x=None), dict(qw=None), dict(sp=None), dict(y=None),
               dict(rows=None), dict(offsets=None)):
        assert st(**kw) == INVALID, kw
    for kw in (dict(g=48), dict(K=192), dict(N=0), dict(K=0), dict(act=1, N=48),
               dict(slots=(1 << 30) + 1), dict(slots=1 << 25, div=1),  # x of 8 GB
               dict(N=1 << 20, K=8192)):                                # one expert's 4 GB
        assert st(**kw) == UNSUPPORTED, kw
    for kw in (dict(x=B), dict(qw=B), dict(sp=B), dict(y=B), dict(rows=A + 2), dict(offsets=A + 2)):
        assert st(**kw) == MISALIGNED, kw


def test_combine_refusals():
    def st(y=A, ids=A, w=A, base=None, out=A, T=2, k=2, N=64):
        return w4.moe_combine_status(y, ids, w, base, out, T, k, N)
    assert st(T=0) == OK
    for kw in (dict(T=-1), dict(N=-1), dict(k=0), dict(k=33), dict(y=None), dict(ids=None),
               dict(w=None), dict(out=None)):
        assert st(**kw) == INVALID, kw
    assert st(N=0) == UNSUPPORTED and st(T=1 << 30, k=2) == UNSUPPORTED
    for kw in (dict(y=B), dict(base=B), dict(out=B), dict(ids=A + 2), dict(w=A + 1)):
        assert st(**kw) == MISALIGNED, kw


def test_reference_routing_by_hand():
    z = np.array([[1.0, 3.0, 3.0, 2.0], [-np.inf, 0.0, np.nan, -np.inf], [-np.inf] * 4])
    ids, w, off, rows = moe_ref.route(z, None, 2)
    assert ids.tolist() == [[1, 2], [1, -1], [-1, -1]]
    assert np.allclose(w, [[0.5, 0.5], [1, 0], [0, 0]])
    assert off.tolist() == [0, 0, 2, 3, 3] and rows.tolist() == [0, 2, 1, -1, -1, -1]
    # two groups of two, the better by the sum of both, then the best two of it
    z = np.log(np.array([[0.45, 0.05, 0.3, 0.2]]))
    ids, _, _, _ = moe_ref.route(z, None, 2, groups=2, groups_kept=1, group_top=2)
    assert ids.tolist() == [[0, 1]] or ids.tolist() == [[2, 3]]
    ids, _, _, _ = moe_ref.route(z, np.array([0, 0, 0.1, 0.1]), 2, groups=2, groups_kept=1, group_top=2)
    assert ids.tolist() == [[2, 3]]
