"""w4a16_moe_route and w4a16_moe_combine on the GPU against 64-bit definitions
(moe_ref): choices, offsets and lists equal, weights within two roundings of
fp32 (the 64-bit score chain adds far less), sums within their bound."""
import math
import sys

import numpy as np
import pytest

import moe_ref

pytestmark = pytest.mark.gpu
SENTINEL = -77


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible to torch")
    import w4a16_weight_only_gemm_amd  # noqa: F401  (fails loudly if the library is missing)
    yield


def log(*a):
    print(*a, file=sys.stderr, flush=True)


def run_route(logits, bias, top_k, bf16=False, **kw):
    """One call; `logits` fp32 values (already bf16-representable with bf16)."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    T, E = logits.shape
    dl = torch.from_numpy(np.ascontiguousarray(logits, np.float32)).cuda()
    if bf16:
        dl = dl.to(torch.bfloat16)
    db = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    ids = torch.full((T, top_k), SENTINEL, dtype=torch.int32, device="cuda")
    w = torch.full((T, top_k), float("nan"), device="cuda")
    off = torch.full((E + 1,), SENTINEL, dtype=torch.int32, device="cuda")
    rows = torch.full((T * top_k,), SENTINEL, dtype=torch.int32, device="cuda")
    n = w4.w4a16_moe_route_workspace_bytes(T, E)
    ws = torch.full((max(n // 4, 1),), SENTINEL, dtype=torch.int32, device="cuda")
    kw = dict(kw)
    kw["scoring"] = (w4.W4A16_ROUTE_SIGMOID if kw.get("scoring") == "sigmoid"
                     else w4.W4A16_ROUTE_SOFTMAX)
    w4.w4a16_moe_route(dl, db, T, E, top_k, ids, w, off, rows, ws, **kw)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy(), off.cpu().numpy(), rows.cpu().numpy()


def check_route(logits, bias, top_k, bf16=False, **kw):
    if bf16:
        logits = moe_ref.bf16_value(moe_ref.bf16_bits(logits)).astype(np.float32)
    log("route", logits.shape, top_k, kw)
    got = run_route(logits, bias, top_k, bf16, **kw)
    ref = moe_ref.route(logits, None if bias is None else np.float32(bias), top_k, **kw)
    assert np.array_equal(got[0], ref[0])
    assert np.array_equal(got[2], ref[2])
    assert np.array_equal(got[3], ref[3])
    assert np.all(np.abs(got[1] - ref[1]) <= 2 * moe_ref.F32 * np.abs(ref[1]) + 1e-45)


@pytest.mark.parametrize("E,top_k", [(1, 1), (3, 2), (8, 2), (60, 4), (64, 6), (65, 8), (128, 8),
                                     (257, 8), (384, 8), (512, 32), (1000, 10), (1024, 32)])
@pytest.mark.parametrize("T", [1, 5])
def test_experts_and_top_k(T, E, top_k):
    rng = np.random.default_rng(E * 100 + T)
    z = rng.standard_normal((T, E)).astype(np.float32) * 2
    check_route(z, None, top_k)
    check_route(z, rng.standard_normal(E) * 0.1, top_k, scoring="sigmoid", renormalize=False,
                scale=2.5, bf16=True)


@pytest.mark.parametrize("T", [16, 17, 32, 33, 64, 100, 1000])
def test_tokens(T):
    rng = np.random.default_rng(T)
    z = rng.standard_normal((T, 40)).astype(np.float32)
    check_route(z, None, 3)
    check_route(z, rng.standard_normal(40) * 0.1, 3, scoring="sigmoid", groups=4, groups_kept=2,
                group_top=2)


def test_more_chunks_than_one_pass_sums():
    rng = np.random.default_rng(3)
    T = 32 * 256 + 33  # one chunk of 32 tokens past 256, and a ragged one
    check_route(rng.standard_normal((T, 20)).astype(np.float32), None, 2)
    check_route(rng.standard_normal((T - 33, 20)).astype(np.float32), None, 2)


@pytest.mark.parametrize("groups,kept,E", [(2, 1, 6), (8, 4, 256), (3, 2, 39), (64, 5, 64),
                                           (33, 7, 66), (4, 4, 128), (5, 1, 1020)])
@pytest.mark.parametrize("scoring,group_top,bias", [("softmax", 1, False), ("sigmoid", 2, True),
                                                    ("softmax", 2, True)])
def test_groups(groups, kept, E, scoring, group_top, bias):
    rng = np.random.default_rng(groups * 10 + kept)
    z = rng.standard_normal((9, E)).astype(np.float32) * 1.5
    b = rng.standard_normal(E) * 0.05 if bias else None
    check_route(z, b, min(8, E // groups * kept), scoring=scoring, groups=groups,
                groups_kept=kept, group_top=group_top)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_equal_values_go_to_the_lowest_index(scoring, bias):
    rng = np.random.default_rng(8)
    z = rng.integers(-2, 3, (40, 200)).astype(np.float32)  # five values over 200 experts
    z[0] = 0.0
    z[1] = np.where(rng.random(200) < 0.5, 0.0, -0.0)
    check_route(z, np.zeros(200) if bias else None, 8, scoring=scoring)
    check_route(z, np.zeros(200) if bias else None, 8, scoring=scoring, groups=8, groups_kept=3)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("T", [12, 50])
def test_masked_and_extreme_logits(scoring, bias, renormalize, T):
    """-inf and NaN are never chosen, rows that leave nothing go nowhere, +inf and
    the type's extremes are ordinary large values."""
    rng = np.random.default_rng(5)
    E = 70
    low = float(np.finfo(np.float32).min)
    z = rng.standard_normal((T, E)).astype(np.float32)
    z[0] = -np.inf
    z[1] = np.nan
    z[2, 3:] = -np.inf
    z[3, ::2] = np.nan
    z[4] = low
    z[5, 10:] = low
    z[6, 7] = np.inf
    z[7] = -low
    z[8, 68:] = -np.inf
    z[9] = -np.inf
    z[9, 69] = low
    b = rng.standard_normal(E) * 0.1 if bias else None
    kw = dict(scoring=scoring, renormalize=renormalize)
    check_route(z, b, 5, **kw)
    check_route(z, b, 5, groups=7, groups_kept=2, group_top=2, **kw)


def test_every_token_to_one_expert():
    z = np.zeros((300, 128), np.float32)
    z[:, 77] = 5.0
    check_route(z, None, 1)


@pytest.mark.parametrize("E", [8, 256, 257, 1024])
def test_no_tokens(E):
    import torch

    import w4a16_weight_only_gemm_amd as w4
    off = torch.full((E + 1,), SENTINEL, dtype=torch.int32, device="cuda")
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    f = torch.empty(0, device="cuda")
    n = w4.w4a16_moe_route_workspace_bytes(0, E)
    ws = torch.zeros(n // 4, dtype=torch.int32, device="cuda") if n else None
    w4.w4a16_moe_route(torch.empty(0, E, device="cuda"), None, 0, E, 2, e, f, off, e, ws)
    torch.cuda.synchronize()
    assert off.tolist() == [0] * (E + 1)


@pytest.mark.parametrize("E,T", [(300, 40), (700, 7), (1024, 1500), (257, 9000)])
def test_many_experts(E, T):
    """More experts than one launch and four per lane hold, with few and many tokens."""
    rng = np.random.default_rng(E)
    z = rng.standard_normal((T, E)).astype(np.float32)
    check_route(z, None, 4)
    if T < 2000:
        check_route(z, rng.standard_normal(E) * 0.1, 8, scoring="sigmoid", groups=E // 10 if E == 300 else 4
                    if E % 4 == 0 else 1, groups_kept=2 if E % 4 == 0 else 1, group_top=2)


def test_repeated_calls_give_the_same_bits():
    z = np.random.default_rng(1).standard_normal((500, 96)).astype(np.float32)
    first = run_route(z, np.linspace(-.1, .1, 96), 6, scoring="sigmoid")
    for _ in range(3):
        again = run_route(z, np.linspace(-.1, .1, 96), 6, scoring="sigmoid")
        assert all(np.array_equal(a, b) for a, b in zip(first, again))


# ------------------------------------------------------------------ combine

@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 8, 5120), (3, 2, 7), (33, 4, 264), (5, 32, 100),
                                   (7, 3, 2049), (257, 8, 512)])
@pytest.mark.parametrize("base", [False, True])
def test_combine(T, k, N, base):
    import torch

    import w4a16_weight_only_gemm_amd as w4
    log("combine", T, k, N, base)
    rng = np.random.default_rng(T * N + k)
    yb = moe_ref.bf16_bits(rng.standard_normal((T * k, N)).astype(np.float32))
    bb = moe_ref.bf16_bits(rng.standard_normal((T, N)).astype(np.float32))
    ids = rng.integers(-1, 5, (T, k)).astype(np.int32)  # about a sixth left out
    w = rng.random((T, k)).astype(np.float32)
    yb.reshape(T, k, N)[ids < 0] = 0x7FC0               # rows left out are not read
    ref, tol = moe_ref.combine(moe_ref.bf16_value(yb), ids, w.astype(np.float64),
                               moe_ref.bf16_value(bb) if base else None)
    dev = lambda a: torch.from_numpy(a.view(np.int16)).cuda().view(torch.bfloat16)  # noqa: E731
    y, b = dev(yb), dev(bb)
    out = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    di, dw = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    w4.w4a16_moe_combine(y, di, dw, b if base else None, out, T, k, N)
    torch.cuda.synchronize()
    got = out.view(torch.int16).cpu().numpy().view(np.uint16)
    moe_ref.check(got, ref, tol)
    if base:  # in place
        w4.w4a16_moe_combine(y, di, dw, b, b, T, k, N)
        torch.cuda.synchronize()
        assert np.array_equal(b.view(torch.int16).cpu().numpy().view(np.uint16), got)


def test_binding_refuses_wrong_tensors():
    import torch

    import w4a16_weight_only_gemm_amd as w4
    z = torch.zeros(4, 16, device="cuda")
    i = torch.zeros(8, dtype=torch.int32, device="cuda")
    f = torch.zeros(8, device="cuda")
    off = torch.zeros(17, dtype=torch.int32, device="cuda")
    good = dict(logits=z, bias=None, ids=i, weights=f, offsets=off, rows=i.clone())

    def call(**kw):
        d = {**good, **kw}
        w4.w4a16_moe_route(d["logits"], d["bias"], 4, 16, 2, d["ids"], d["weights"], d["offsets"],
                           d["rows"], None)
    call()
    for kw in (dict(logits=z.half()), dict(ids=f), dict(weights=i), dict(offsets=off.long()),
               dict(bias=z.half()[0])):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(logits=z[:3]), dict(ids=i[:7]), dict(offsets=off[:16]), dict(rows=i[:7]),
               dict(logits=torch.zeros(16, 4, device="cuda").t()), dict(weights=f.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    assert math.isfinite(float(f.sum()))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("gap", [0.0, 1e-9, 3e-8, 1e-6, 1e-4])
def test_values_next_to_each_other(scoring, gap):
    """Choice values nearer than fp32 resolves (and some that it does): a logit's
    last bits and a bias that nearly makes up for them decide as in 64 bits."""
    rng = np.random.default_rng(2)
    T, E = 300, 96
    z = np.round(rng.standard_normal((T, E)) * 4).astype(np.float32) / 4
    z = np.nextafter(z, np.where(rng.random((T, E)) < 0.5, np.inf, -np.inf).astype(np.float32))
    b = np.where(rng.random(E) < 0.5, gap, 0.0)
    for kw in (dict(), dict(groups=8, groups_kept=3, group_top=2)):
        check_route(z, b, 8, scoring=scoring, **kw)


@pytest.mark.parametrize("bias", [1e30, -1e30, 1000.0])
def test_large_biases(bias):
    rng = np.random.default_rng(4)
    b = np.where(rng.random(64) < 0.4, bias, 0.1)
    check_route(rng.standard_normal((50, 64)).astype(np.float32), b, 6, scoring="sigmoid")
    check_route(rng.standard_normal((50, 64)).astype(np.float32) * 60, b, 6, groups=4, groups_kept=2)


@pytest.mark.parametrize("E", [40, 128, 256, 500, 1000])
@pytest.mark.parametrize("bf16", [False, True])
def test_logits_next_to_each_other(E, bf16):
    """Neighbouring logits, in every order within and across lanes: 0 to 15 steps
    of fp32 apart (bf16: of bf16), some of them equal."""
    rng = np.random.default_rng(E)
    base = np.float32([3.0, -3.0, 1e-3, 0.0, 100.0] * 12)[:, None]
    steps = rng.integers(0, 16, (60, E)).astype(np.int64)
    bits = np.repeat(base, E, 1).view(np.int32).astype(np.int64) + steps * (65536 if bf16 else 1)
    z = bits.astype(np.int32).view(np.float32)
    z[1::2, 5:] -= 50.0  # few of them alone at the top
    check_route(z, None, 8, bf16=bf16)
    check_route(z, None, 5, bf16=bf16, renormalize=False)
    check_route(z, None, 3, bf16=bf16, scoring="sigmoid", groups=4, groups_kept=2, group_top=2)


@pytest.mark.parametrize("E,groups", [(72, 8), (256, 8), (1024, 16)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_many_equal_values(E, groups, scoring):
    """More equal values than a wave has lanes, beside distinct ones."""
    rng = np.random.default_rng(E)
    z = np.where(rng.random((40, E)) < 0.9, 0.5, rng.standard_normal((40, E)) * 2).astype(np.float32)
    z[0] = 0.5
    for b in (None, np.full(E, 0.25)):
        check_route(z, b, 8, scoring=scoring)
        check_route(z, b, 8, scoring=scoring, groups=groups, groups_kept=3, group_top=2)


@pytest.mark.parametrize("T", [5, 40, 3000])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_bias_out_of_range_keeps_lists_whole(T, bad):
    """A bias outside the interface's range: any choice, but distinct experts and
    lists that agree with them."""
    rng = np.random.default_rng(T)
    E, k = 96, 8
    z = rng.standard_normal((T, E)).astype(np.float32)
    b = np.where(rng.random(E) < 0.3, bad, 0.1)
    for kw in (dict(scoring="sigmoid"), dict(groups=8, groups_kept=4, group_top=2), dict(groups=3, groups_kept=2)):
        ids, _, off, rows = run_route(z, b, k, **kw)
        assert ids.min() >= -1 and ids.max() < E
        for row in ids:
            chosen = row[row >= 0]
            assert len(set(chosen.tolist())) == len(chosen)
        flat = ids.reshape(-1)
        assert off[0] == 0 and off[E] == (flat >= 0).sum()
        for e in range(E):
            assert np.array_equal(rows[off[e]:off[e + 1]], np.flatnonzero(flat == e))
        assert np.all(rows[off[E]:] == -1)


@pytest.mark.parametrize("T,k,N", [(1, 2, 8), (3, 1, 9), (40, 3, 15), (700, 3, 1209), (90, 8, 4588)])
def test_combine_rows_at_any_address(T, k, N):
    """Rows that start between 16-byte borders; nothing is written behind the last."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    log("combine", T, k, N)
    g = torch.Generator().manual_seed(N)
    y = torch.randn(T * k, N, generator=g).to(torch.bfloat16)
    b = torch.randn(T, N, generator=g).to(torch.bfloat16)
    w = torch.rand(T, k, generator=g)
    ids = torch.randint(-1, 5, (T, k), generator=g, dtype=torch.int32)
    ref, tol = moe_ref.combine(y.double().numpy(), ids.numpy(), w.double().numpy(), b.double().numpy())
    buf = torch.full((T * N + 64,), -5.0, dtype=torch.bfloat16, device="cuda")
    buf[:T * N] = b.cuda().reshape(-1)
    out = buf[:T * N].view(T, N)  # in place
    w4.w4a16_moe_combine(y.cuda(), ids.cuda(), w.cuda(), out, out, T, k, N)
    torch.cuda.synchronize()
    moe_ref.check(out.view(torch.int16).cpu().numpy().view(np.uint16), ref, tol)
    assert bool((buf[T * N:] == -5.0).all())
