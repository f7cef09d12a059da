"""w4a16_moe_layer on the GPU against a whole layer in 64 bits (layer_ref): token
counts, experts, groups, group sizes and widths at every kernel form, ties, padding
tokens, dirty workspaces, the same bits on every run."""
import sys

import numpy as np
import pytest

import layer_ref
import moe_ref
from test_gpu_experts import dev_bf16, gpu, host_bits  # noqa: F401  (gpu: the fixture)

pytestmark = pytest.mark.gpu


def log(*a):
    print(*a, file=sys.stderr, flush=True)


class Whole:
    """Random weights of a layer."""

    def __init__(self, E, H, I, group, seed=0, half=True, bias=False):
        import torch

        import w4a16_weight_only_gemm_amd as w4
        rng = np.random.default_rng(seed)
        self.E, self.H, self.I, self.group, self.half = E, H, I, group, half

        def pack(N, K):
            q = rng.integers(-8, 8, (E, N, K)).astype(np.int8)
            s = ((rng.random((E, N, K // group)) + 0.5) / (4 * np.sqrt(K))).astype(np.float16)
            p = [w4.w4a16_pack(q[e], s[e], group) for e in range(E)]
            return (q, s.astype(np.float64),
                    torch.from_numpy(np.concatenate([a for a, _ in p]).view(np.int32)).cuda(),
                    torch.from_numpy(np.concatenate([b for _, b in p]).view(np.int16)).cuda())
        self.up, self.down = pack(2 * I, H), pack(H, I)
        r = (rng.standard_normal((E, H)) * 1.5 / np.sqrt(H)).astype(np.float32)
        self.set_router(r)
        self.bias = (rng.standard_normal(E) * 0.05).astype(np.float32) if bias else None
        self.dbias = torch.from_numpy(self.bias).cuda() if bias else None

    def set_router(self, r):
        import torch
        if self.half:
            bits = moe_ref.bf16_bits(r)
            self.router, self.drouter = moe_ref.bf16_value(bits), dev_bf16(bits)
        else:
            self.router, self.drouter = r.astype(np.float64), torch.from_numpy(np.ascontiguousarray(r)).cuda()

    def buffers(self, T, k, fill=0xFF):
        import torch

        import w4a16_weight_only_gemm_amd as w4
        n = w4.w4a16_moe_layer_workspace_bytes(T, self.E, k, self.H, self.I)
        return dict(T=T, k=k, x=torch.zeros((T, self.H), dtype=torch.bfloat16, device="cuda"),
                    base=torch.zeros((T, self.H), dtype=torch.bfloat16, device="cuda"),
                    live=torch.ones(T, dtype=torch.int32, device="cuda"),
                    out=torch.full((T + 1, self.H), -3.0, dtype=torch.bfloat16, device="cuda"),
                    ids=torch.full((T, k), -77, dtype=torch.int32, device="cuda"),
                    w=torch.full((T, k), -77.0, device="cuda"),
                    ws=torch.full((n,), fill, dtype=torch.uint8, device="cuda"))

    def fill(self, b, seed, pad=0):
        import torch
        rng = np.random.default_rng(seed)
        x = moe_ref.bf16_bits(rng.standard_normal((b["T"], self.H)).astype(np.float32))
        base = moe_ref.bf16_bits(rng.standard_normal((b["T"], self.H)).astype(np.float32))
        live = np.ones(b["T"], np.int32)
        if pad:
            gone = rng.permutation(b["T"])[:pad]
            live[gone] = 0
            x[gone] = 0x7FC0  # rows of padding tokens may hold anything
        b["x"].view(torch.int16).copy_(torch.from_numpy(x.view(np.int16)))
        b["base"].view(torch.int16).copy_(torch.from_numpy(base.view(np.int16)))
        b["live"].copy_(torch.from_numpy(live))
        return x, base, live

    def call(self, b, use_base=True, use_live=True, out=None, stream=None, **route):
        import w4a16_weight_only_gemm_amd as w4
        kw = dict(route)
        kw["scoring"] = w4.W4A16_ROUTE_SIGMOID if kw.get("scoring") == "sigmoid" else w4.W4A16_ROUTE_SOFTMAX
        w4.w4a16_moe_layer(b["x"], self.drouter, self.up[2], self.up[3], self.down[2], self.down[3],
                           b["out"][:b["T"]] if out is None else out, b["ids"], b["w"], b["T"], self.E, b["k"],
                           self.H, self.I, self.group, b["ws"], route_bias=self.dbias,
                           base=b["base"] if use_base else None, live=b["live"] if use_live else None,
                           stream=stream, **kw)

    def logits(self, x_bits):
        with np.errstate(invalid="ignore"):
            return moe_ref.bf16_value(x_bits) @ self.router.T

    def reference(self, x, base, live, k, **route):
        xv = np.where(np.asarray(live)[:, None] != 0, moe_ref.bf16_value(np.where(x == 0x7FC0, 0, x)), 0.0)
        return layer_ref.moe_layer(xv, self.logits(np.where(x == 0x7FC0, 0, x)), self.up[0], self.up[1], self.down[0],
                                   self.down[1], self.group, k, None if base is None else moe_ref.bf16_value(base),
                                   live, self.bias, **route)

    def check(self, T, k, seed=1, pad=0, base=True, **route):
        log(f"moe E={self.E} H={self.H} I={self.I} g={self.group} T={T} k={k} pad={pad} {route}")
        b = self.buffers(T, k)
        x, bs, live = self.fill(b, seed, pad)
        self.call(b, use_base=base, use_live=pad > 0, **route)
        ids, w, out, tol = self.reference(x, bs if base else None, live, k, **route)
        got = host_bits(b["out"])
        assert np.all(got[T] == 0xC040)
        assert np.array_equal(b["ids"].cpu().numpy(), ids)
        gw = b["w"].double().cpu().numpy()
        # the weight in 64 bits (a few thousand roundings at most), rounded to fp32
        assert np.all(np.abs(gw - w) <= moe_ref.F32 * np.abs(w) + 1e-12 * (1 + np.abs(w)))
        gv = moe_ref.bf16_value(got[:T])
        assert np.all(np.abs(gv - out) <= tol), float(np.max(np.abs(gv - out) - tol))
        # the rounding of out, and of nothing else to bf16
        assert np.linalg.norm(gv - out) <= moe_ref.BF16 * max(np.linalg.norm(out), 1e-30)


@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("T", [1, 2, 5, 8, 15, 16])
def test_groups_and_tokens(group, T):
    Whole(12, 512, 256, group, T).check(T, 3, pad=T // 5)


@pytest.mark.parametrize("H,I,group", [(32, 32, 32), (96, 32, 32), (160, 96, 32), (64, 64, 64), (320, 192, 64), (128, 128, 128),
                                       (256, 256, 256), (384, 128, 128), (2304, 128, 128), (1056, 2080, 32),
                                       (2560, 256, 256), (3328, 128, 128), (4096, 128, 64), (5120, 128, 128),
                                       (5376, 256, 256), (6144, 128, 128), (6272, 128, 128), (7168, 128, 128),
                                       (8192, 64, 64), (8448, 256, 256), (9344, 128, 128), (128, 3328, 128)])
def test_sizes(H, I, group):
    w = Whole(4, H, I, group, H)
    w.check(1, 2)
    w.check(7, 3, pad=1)


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (5, 3), (63, 8), (64, 8), (65, 7), (128, 8), (129, 32), (200, 1),
                                 (256, 8), (257, 16), (512, 8), (513, 4), (1024, 32)])
def test_experts(E, k):
    w = Whole(E, 64, 32, 32, E, half=E % 2 == 0)
    w.check(16, k)
    w.check(3, k, pad=1, scoring="sigmoid", renormalize=False, scale=2.0)


@pytest.mark.parametrize("E,groups,kept,top", [(16, 4, 2, 2), (16, 4, 1, 1), (256, 8, 4, 2), (64, 64, 5, 2), (120, 8, 8, 1),
                                               (1024, 32, 3, 2), (33, 3, 2, 2), (40, 1, 1, 2)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_groups_of_experts(E, groups, kept, top, scoring, bias):
    w = Whole(E, 64, 32, 32, E, half=False, bias=bias)
    # as many choices as the groups that are kept hold, and one more
    for k in sorted({1, 4, min(32, E // groups * kept + 1, E)}):
        w.check(6, k, scoring=scoring, groups=groups, groups_kept=kept, group_top=top, scale=1.25)


@pytest.mark.parametrize("T,E", [(1, 4), (1, 65), (1, 132), (1, 256), (1, 260), (2, 64), (2, 128), (2, 132), (2, 256),
                                 (8, 64), (9, 64), (16, 8)])
def test_where_the_choice_is_made(T, E):
    """Tokens and experts on both sides of where the choice gets a launch of its own,
    by the logit and by values within groups."""
    w = Whole(E, 64, 32, 32, 7 * E + T, bias=True)
    w.check(T, min(E, 8), renormalize=False)
    w.check(T, min(E, 8), scoring="sigmoid", pad=T // 4)
    if E % 4 == 0:
        w.check(T, min(E // 2, 32), groups=4, groups_kept=2, group_top=2, scale=2.5)
    Whole(E, 64, 32, 32, 7 * E + T, half=True).check(T, min(E, 32))


def test_equal_logits():
    """Experts with the same router row: the lowest index wins; with groups, the lowest
    group."""
    w = Whole(48, 96, 32, 32, 3)
    r = np.random.default_rng(0).standard_normal((6, 96)).astype(np.float32) * 0.1
    w.set_router(np.tile(r, (8, 1)))
    b = w.buffers(5, 9)
    x, base, live = w.fill(b, 1)
    w.call(b)
    z = w.logits(x)[:, :6]
    want = []
    for t in range(5):
        order = np.argsort(-z[t], kind="stable")
        want.append([order[0] + 6 * i for i in range(8)] + [order[1]])
    assert np.array_equal(b["ids"].cpu().numpy(), np.array(want))
    w.set_router(np.zeros((48, 96), np.float32))
    w.call(b, groups=8, groups_kept=2, group_top=2)
    assert np.array_equal(b["ids"].cpu().numpy()[:, :], np.tile(np.arange(9), (5, 1)))
    assert np.allclose(b["w"].cpu().numpy(), 1 / 9)


def test_near_logits():
    """Two experts whose logits differ by less than fp32 holds: 64 bits tell them apart."""
    w = Whole(8, 256, 32, 32, 4, half=False)
    r = np.zeros((8, 256), np.float32)
    r[:, 0] = [1, 1, 1, 1, 1, 1, 1, 1]
    r[5, 1] = 2.0 ** -30
    r[6, 1] = 2.0 ** -29
    w.set_router(r)
    b = w.buffers(2, 3)
    b["x"].fill_(1.0)
    w.call(b)
    assert b["ids"].cpu().tolist() == [[6, 5, 0], [6, 5, 0]]


@pytest.mark.parametrize("T", [1, 6, 16])
def test_no_live_token(T):
    import torch
    w = Whole(10, 256, 128, 128, 5)
    b = w.buffers(T, 4)
    x, base, live = w.fill(b, 2, pad=T)
    w.call(b)
    assert np.array_equal(host_bits(b["out"])[:T], base)
    assert bool((b["ids"] == -1).all()) and bool((b["w"] == 0).all())
    w.call(b, use_base=False)
    torch.cuda.synchronize()
    assert bool((b["out"][:T] == 0).all()) and bool((b["out"][T] == -3.0).all())


def test_weights_that_vanish():
    """renormalised sums of 0 (scores underflow) and scale 0: out is base."""
    w = Whole(6, 64, 32, 32, 6)
    b = w.buffers(3, 2)
    x, base, live = w.fill(b, 3)
    w.call(b, scale=0.0)
    assert np.array_equal(host_bits(b["out"])[:3], base) and bool((b["w"] == 0).all())


@pytest.mark.parametrize("T,E,k", [(1, 16, 4), (4, 16, 4), (16, 40, 8)])
def test_same_bits(T, E, k):
    """Whatever the workspace held, whatever its neighbours' timing, in place on base."""
    import torch
    w = Whole(E, 1280, 384, 128, 7)
    want = None
    for fill in (0x00, 0xFF, 0x5A, 0x7F, 0x01):
        b = w.buffers(T, k, fill)
        w.fill(b, 9)
        for _ in range(4):
            w.call(b)
            got = (host_bits(b["out"]).copy(), b["ids"].cpu().numpy(), b["w"].cpu().numpy())
            if want is None:
                want = got
            assert all(np.array_equal(p, q) for p, q in zip(got, want))
    w.call(b, out=b["base"])
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(b["base"]), want[0][:T])


def test_tokens_do_not_meet():
    """A token's row is the same alone and among others, whatever the others hold."""
    w = Whole(16, 512, 256, 128, 8)
    b = w.buffers(6, 4)
    x, base, live = w.fill(b, 4)
    w.call(b, use_live=False)
    whole = host_bits(b["out"]).copy()
    b["x"][2] = float("nan")
    w.call(b, use_live=False)  # a NaN row chooses nothing
    got = host_bits(b["out"])
    keep = [0, 1, 3, 4, 5]
    ids = b["ids"].cpu().numpy()
    assert np.all(ids[2] == -1) and np.array_equal(got[2], base[2])
    a, c = moe_ref.bf16_value(whole[keep]), moe_ref.bf16_value(got[keep])
    # the order of a row's additions may differ: as far as two results in their bounds
    _, _, _, tol = w.reference(x, base, live, 4)
    assert np.all(np.abs(a - c) <= 2 * tol[keep])


def test_scales_that_are_not_finite():
    """An expert with infinite scales reaches only the tokens that chose it."""
    import torch
    w = Whole(8, 256, 128, 128, 9)
    b = w.buffers(8, 2)
    x, base, live = w.fill(b, 5)
    w.call(b)
    clean, ids = host_bits(b["out"]).copy(), b["ids"].cpu().numpy()
    e = ids[0, 0]
    for packed in (w.up[3], w.down[3]):
        per = packed.numel() // 8
        keep = packed[e * per:(e + 1) * per].clone()
        packed[e * per:(e + 1) * per] = 0x7C00
        w.call(b)
        got = host_bits(b["out"])
        chose = (ids == e).any(1)
        assert np.array_equal(got[:8][~chose], clean[:8][~chose]) and chose.any()
        assert not np.isfinite(moe_ref.bf16_value(got[:8][chose])).all()
        packed[e * per:(e + 1) * per] = keep
    torch.cuda.synchronize()


def test_far_weights():
    """Packed experts past 2^31 bytes and 2^32 bytes."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    E, H, I, group, T, k = 600, 2048, 4096, 128, 4, 3
    log("moe far weights")
    g = torch.Generator(device="cuda").manual_seed(1)
    per_up, per_down = w4.w4a16_qweight_bytes(2 * I, H), w4.w4a16_qweight_bytes(H, I)
    assert E * per_up > 1 << 32 and E * per_down > 1 << 31

    def words(n):
        return torch.randint(-2**31, 2**31, (E, n // 4), generator=g, device="cuda", dtype=torch.int32)

    def scales(N, K):
        s = torch.rand((E, N // 16, K // group, 16), generator=g, device="cuda") + 0.5
        return (s / (4 * K ** 0.5)).to(torch.float16)
    up, down, su, sd = words(per_up), words(per_down), scales(2 * I, H), scales(H, I)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    router = torch.randn((E, H), generator=g, device="cuda") / H ** 0.5
    router[[0, 299, 599]] = x[:3].float() * 0.02  # the ends and the middle are chosen
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    wt = torch.empty((T, k), device="cuda")
    ws = torch.empty(w4.w4a16_moe_layer_workspace_bytes(T, E, k, H, I), dtype=torch.uint8, device="cuda")
    w4.w4a16_moe_layer(x, router, up, su, down, sd, out, ids, wt, T, E, k, H, I, group, ws)
    got = ids.cpu().numpy()
    assert got[0, 0] == 0 and got[1, 0] == 299 and got[2, 0] == 599

    def matrix(q, s, e, N, K):
        """codes [N][K] and scales [N][G] of expert e, from the arrangement of w4a16_pack."""
        w = q[e].cpu().numpy().view(np.uint32).reshape(N // 16, K // group, 4, 16, group // 32)
        c = np.stack([(w >> np.uint32(4 * n)) & 15 for n in (0, 4, 1, 5, 2, 6, 3, 7)], -1).astype(np.int64)
        c = ((c ^ 8) - 8).transpose(0, 3, 1, 2, 4, 5).reshape(N, K)
        return c.astype(np.int8), s[e].double().cpu().numpy().transpose(0, 2, 1).reshape(N, K // group)
    used = sorted(set(got.reshape(-1).tolist()))
    ups = [matrix(up, su, e, 2 * I, H) for e in used]
    downs = [matrix(down, sd, e, H, I) for e in used]
    z = x.double().cpu().numpy() @ router[used].double().cpu().numpy().T
    full = x.double().cpu().numpy() @ router.double().cpu().numpy().T
    assert np.array_equal(np.argsort(-full, axis=1)[:, :k], got)
    _, _, ref, tol = layer_ref.moe_layer(x.double().cpu().numpy(), z, np.stack([a for a, _ in ups]),
                                         np.stack([a for _, a in ups]), np.stack([a for a, _ in downs]),
                                         np.stack([a for _, a in downs]), group, k)
    gv = moe_ref.bf16_value(host_bits(out))
    assert np.all(np.abs(gv - ref) <= tol)
