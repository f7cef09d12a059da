"""w4a16_gemm_experts on the GPU against a 64-bit product per expert (moe_ref),
over both kernels' row ranges, every group size, ragged sizes, empty experts,
lists with holes, and SwiGLU."""
import sys

import numpy as np
import pytest

import moe_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible to torch")
    import w4a16_weight_only_gemm_amd  # noqa: F401  (fails loudly if the library is missing)
    yield


def log(*a):
    print(*a, file=sys.stderr, flush=True)


def dev_bf16(bits):
    import torch
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def host_bits(t):
    import torch
    torch.cuda.synchronize()
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


class Experts:
    """Random weights of E experts, packed one after another."""

    def __init__(self, E, N, K, group, seed):
        import torch

        import w4a16_weight_only_gemm_amd as w4
        rng = np.random.default_rng(seed)
        self.E, self.N, self.K, self.group = E, N, K, group
        self.q = rng.integers(-8, 8, (E, N, K)).astype(np.int8)
        s16 = ((rng.random((E, N, K // group)) + 0.5) / (4 * np.sqrt(K))).astype(np.float16)
        self.s = s16.astype(np.float64)
        packs = [w4.w4a16_pack(self.q[e], s16[e], group) for e in range(E)]
        self.qw = torch.from_numpy(np.concatenate([p[0] for p in packs]).view(np.int32)).cuda()
        self.sp = torch.from_numpy(np.concatenate([p[1] for p in packs]).view(np.int16)).cuda()


def lists(ids, E):
    """offsets and rows of slots' experts (-1: nowhere)."""
    parts = [np.flatnonzero(ids == e) for e in range(E)]
    off = np.concatenate([[0], np.cumsum([p.size for p in parts])]).astype(np.int32)
    rows = np.full(ids.size, -1, np.int32)
    flat = np.concatenate(parts)
    rows[:flat.size] = flat
    return off, rows


def run(w, x_bits, off, rows, x_div, swiglu, stream=None):
    import torch

    import w4a16_weight_only_gemm_amd as w4
    out = w.N // 2 if swiglu else w.N
    y = torch.full((rows.size, out), -3.0, dtype=torch.bfloat16, device="cuda")
    w4.w4a16_gemm_experts(dev_bf16(x_bits), w.qw, w.sp, y, torch.from_numpy(rows).cuda(),
                          torch.from_numpy(off).cuda(), rows.size, w.E, x_div, w.N, w.K, w.group,
                          act=w4.W4A16_ACT_SWIGLU if swiglu else w4.W4A16_ACT_NONE, stream=stream)
    return host_bits(y)


def check(E, N, K, group, ids, x_div, swiglu, seed=0):
    log(f"experts E={E} N={N} K={K} g={group} slots={ids.size} div={x_div} swiglu={swiglu}")
    rng = np.random.default_rng(seed + 1)
    w = Experts(E, N, K, group, seed)
    off, rows = lists(ids, E)
    x_bits = moe_ref.bf16_bits(rng.standard_normal((-(-ids.size // x_div), K)).astype(np.float32))
    got = run(w, x_bits, off, rows, x_div, swiglu)
    ref, tol = moe_ref.experts(moe_ref.bf16_value(x_bits), w.q, w.s, rows, off, x_div, group, swiglu)
    named = ids >= 0
    moe_ref.check(got[named], ref[named], tol[named])
    assert np.all(got[~named] == 0xC040)  # rows in no list: as they were (-3)


def spread(rng, slots, E, holes=0.0, weights=None):
    ids = rng.choice(E, size=slots, p=weights)
    return np.where(rng.random(slots) < holes, -1, ids)


@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("slots", [1, 7, 40, 200, 700, 1500])
def test_groups_and_rows(group, swiglu, slots):
    """8 experts, so 0 to 187 rows each on average: every kernel form."""
    rng = np.random.default_rng(slots + group)
    check(8, 96 if swiglu else 100, 768, group, spread(rng, slots, 8), 1, swiglu, seed=slots)


@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (5, 96, 32), (16, 128, 128), (17, 128, 64),
                                       (260, 384, 128), (40, 2176, 128), (33, 160, 32), (513, 256, 256)])
@pytest.mark.parametrize("slots", [3, 130, 420])
def test_odd_sizes(N, K, group, slots):
    rng = np.random.default_rng(N + slots)
    check(3, N, K, group, spread(rng, slots, 3, holes=0.1), 1, False, seed=N)


@pytest.mark.parametrize("N", [32, 64, 96, 544])
@pytest.mark.parametrize("slots", [6, 330])
def test_swiglu_widths(N, slots):
    rng = np.random.default_rng(N)
    check(3, N, 256, 128, spread(rng, slots, 3), 1, True, seed=N)


@pytest.mark.parametrize("T,k,E", [(1, 8, 128), (9, 3, 65), (50, 4, 6), (200, 8, 10)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_shared_rows(T, k, E, swiglu):
    """x_div = top_k: the slots of a token read its one row; distinct experts per token."""
    rng = np.random.default_rng(T)
    ids = np.concatenate([rng.permutation(E)[:k] for _ in range(T)])
    check(E, 64, 256, 128, ids, k, swiglu, seed=T)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("swiglu,N", [(False, 5000), (False, 5003), (True, 9952)])
def test_tall_tiles(group, swiglu, N):
    """Enough rows and columns for 128-row tiles, with experts of every tail: one
    row, up to 32, 64 and 128 rows past whole tiles, none."""
    rng = np.random.default_rng(group)
    count = [1, 0, 128, 129, 257 + 31, 384 + 33, 512 + 64, 512 + 65, 512 + 127, 640, 30, 3]
    ids = np.concatenate([np.full(c, e) for e, c in enumerate(count)] + [np.full(800, 4)])
    check(len(count), N, 256 + group, group, rng.permutation(ids), 1, swiglu, seed=group)


@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("T,N", [(1, 2048), (8, 4096), (40, 2048)])
def test_deep_products_of_few_rows(group, swiglu, T, N):
    """The K-splitting form at both widths, tiles of at most 4 rows, up to 16 and past 16."""
    rng = np.random.default_rng(T)
    ids = np.concatenate([rng.permutation(10)[:8] for _ in range(T)])
    ids[rng.random(ids.size) < 0.3] = 1  # one expert past 16 rows at 40 tokens
    check(10, N, 2560, group, ids, 8, swiglu, seed=T)


@pytest.mark.parametrize("E,slots", [(300, 5), (300, 900), (1024, 40), (1024, 6000)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_many_experts(E, slots, swiglu):
    """More experts than a lane holds offsets of in registers; most of them empty or small."""
    rng = np.random.default_rng(E + slots)
    ids = np.minimum((rng.random(slots) ** 2 * E).astype(int), E - 1)
    check(E, 32, 64, 32, np.where(rng.random(slots) < 0.1, -1, ids), 1, swiglu, seed=slots)


def test_one_expert_takes_all_and_others_none():
    for slots in (5, 100, 900):
        check(4, 64, 256, 128, np.full(slots, 2), 1, False)
        check(1, 64, 256, 128, np.zeros(slots, int), 1, True)


def test_uneven_load():
    """Means that pick the few-rows form while one expert holds most rows, and
    means that pick the tile engine while some hold one row."""
    rng = np.random.default_rng(2)
    p = np.array([0.9] + [0.1 / 31] * 31)
    check(32, 64, 256, 128, spread(rng, 300, 32, weights=p), 1, False)
    check(32, 64, 256, 128, spread(rng, 6000, 32, weights=p), 1, True)


def test_nothing_routed():
    check(4, 64, 256, 128, np.full(9, -1), 1, False)


def test_unused_rows_may_hold_anything():
    """NaN rows of x that no list names do not reach any result."""
    rng = np.random.default_rng(4)
    for slots, E in ((20, 4), (800, 4)):
        w = Experts(E, 64, 256, 128, 9)
        ids = spread(rng, slots, E, holes=0.3)
        off, rows = lists(ids, E)
        x = moe_ref.bf16_bits(rng.standard_normal((slots, 256)).astype(np.float32))
        x[ids < 0] = 0x7FC0
        got = run(w, x, off, rows, 1, False)
        x[ids < 0] = 0
        assert np.array_equal(got, run(w, x, off, rows, 1, False))


def test_a_row_with_nan_stays_its_own():
    rng = np.random.default_rng(6)
    for slots, E in ((20, 4), (800, 4)):
        w = Experts(E, 64, 256, 128, 9)
        ids = spread(rng, slots, E)
        off, rows = lists(ids, E)
        x = moe_ref.bf16_bits(rng.standard_normal((slots, 256)).astype(np.float32))
        clean = run(w, x, off, rows, 1, False)
        x[3] = 0x7FC0
        got = run(w, x, off, rows, 1, False)
        keep = np.arange(slots) != 3
        assert np.array_equal(got[keep], clean[keep])
        assert np.isnan(moe_ref.bf16_value(got[3])).all()


def test_bad_list_entries_are_ignored():
    """Entries outside the slots, and offsets outside them, are not followed."""
    rng = np.random.default_rng(7)
    w = Experts(3, 64, 256, 128, 1)
    for slots in (12, 600):
        ids = spread(rng, slots, 3)
        off, rows = lists(ids, 3)
        x = moe_ref.bf16_bits(rng.standard_normal((slots, 256)).astype(np.float32))
        good = run(w, x, off, rows, 1, False)
        bad = rows.copy()
        hit = [0, slots // 2, slots - 1]
        lost = rows[hit]
        bad[hit] = [-5, slots, 2**31 - 1]
        got = run(w, x, off, bad, 1, False)
        keep = np.ones(slots, bool)
        keep[lost] = False
        assert np.array_equal(got[keep], good[keep])
        assert np.all(got[lost] == 0xC040)
        wild = off.copy()
        wild[0], wild[-1] = -9, 2**30
        assert np.array_equal(run(w, x, wild, rows, 1, False), good)


def test_same_bits_every_call_and_on_another_stream():
    import torch
    rng = np.random.default_rng(3)
    w = Experts(8, 128, 512, 128, 2)
    for slots in (30, 1000):
        off, rows = lists(spread(rng, slots, 8), 8)
        x = moe_ref.bf16_bits(rng.standard_normal((slots, 512)).astype(np.float32))
        first = run(w, x, off, rows, 1, True)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = run(w, x, off, rows, 1, True)
        assert np.array_equal(first, again)


def test_first_expert_equals_the_dense_product():
    """With one expert and every row, the sums are those of w4a16_gemm up to rounding."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    rng = np.random.default_rng(3)
    w = Experts(1, 256, 1024, 128, 2)
    x = moe_ref.bf16_bits(rng.standard_normal((9, 1024)).astype(np.float32))
    off, rows = lists(np.zeros(9, int), 1)
    a = moe_ref.bf16_value(run(w, x, off, rows, 1, False))
    y = torch.empty((9, 256), dtype=torch.bfloat16, device="cuda")
    w4.w4a16_gemm(dev_bf16(x), w.qw, w.sp, y, 9, 256, 1024, 128)
    b = moe_ref.bf16_value(host_bits(y))
    assert np.linalg.norm(a - b) <= 2 * moe_ref.BF16 * np.linalg.norm(b)
