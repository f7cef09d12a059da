"""The operators of include/w4a16_moe.h on buffers whose element index passes
2^31 or whose bytes pass 2^32: rows at both ends and at the borders, against
the 64-bit definitions."""
import sys

import numpy as np
import pytest

import moe_ref
from test_gpu_experts import Experts, gpu, host_bits, lists  # noqa: F401  (gpu: the fixture)

pytestmark = pytest.mark.gpu


def log(*a):
    print(*a, file=sys.stderr, flush=True)


def normal(rows, cols, seed):
    """bf16 [rows][cols] on the device."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    for r in range(0, rows, 1 << 15):
        n = min(1 << 15, rows - r)
        out[r:r + n] = torch.randn((n, cols), generator=g, device="cuda")
    return out


def sample(rows, per_row, seed):
    """Row numbers: both ends, where elements pass 2^31 and bytes (of 2) 2^32, some between."""
    rng = np.random.default_rng(seed)
    border = (1 << 31) // per_row
    r = np.r_[0, 1, rows - 2, rows - 1, rng.integers(0, rows, 20), np.arange(border - 2, border + 3)]
    return np.unique(r[(r >= 0) & (r < rows)])


def values(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("T,k,N", [(66000, 8, 5120), (262200, 1, 8200)])
def test_combine(T, k, N):
    import torch

    import w4a16_weight_only_gemm_amd as w4
    log("combine", T, k, N)
    assert T * k * N > 1 << 31
    y, base = normal(T * k, N, 1), normal(T, N, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.rand((T, k), generator=g, device="cuda")
    ids = torch.randint(-1, 9, (T, k), generator=g, device="cuda", dtype=torch.int32)
    out = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.w4a16_moe_combine(y, ids, w, base, out, T, k, N)
    torch.cuda.synchronize()
    at = torch.from_numpy(sample(T, k * N, T)).cuda()
    ref, tol = moe_ref.combine(values(y.view(T, k, N)[at]).reshape(-1, N), ids[at].cpu().numpy(),
                               values(w[at]), values(base[at]))
    moe_ref.check(host_bits(out[at]), ref, tol)
    assert not bool(torch.isnan(out).any())


def routed(rng, slots, E):
    import torch
    ids = rng.integers(0, E, slots)
    order = np.argsort(ids, kind="stable").astype(np.int32)
    off = np.r_[0, np.cumsum(np.bincount(ids, minlength=E))].astype(np.int32)
    return ids, torch.from_numpy(order).cuda(), torch.from_numpy(off).cuda()


@pytest.mark.parametrize("slots,N,K", [((1 << 20) + 3, 2064, 128), (500_000, 40, 4096)])
@pytest.mark.parametrize("group", [32, 128])
def test_experts_rows(slots, N, K, group):
    """y past 2^31 elements; x of 4.1 of the 4.29 GB that it may have."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    log("experts", slots, N, K, group)
    rng = np.random.default_rng(slots)
    E = 4
    w = Experts(E, N, K, group, 5)
    ids, rows, off = routed(rng, slots, E)
    x = normal(slots, K, 6)
    y = torch.full((slots, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.w4a16_gemm_experts(x, w.qw, w.sp, y, rows, off, slots, E, 1, N, K, group)
    torch.cuda.synchronize()
    at = np.unique(np.r_[sample(slots, N, 7), sample(slots, K, 8)])
    sub_off, sub_rows = lists(ids[at], E)
    dev = torch.from_numpy(at).cuda()
    ref, tol = moe_ref.experts(values(x[dev]), w.q, w.s, sub_rows, sub_off, 1, group)
    moe_ref.check(host_bits(y[dev]), ref, tol)
    assert not bool(torch.isnan(y).any())


@pytest.mark.parametrize("group", [64, 256])
@pytest.mark.parametrize("slots", [40, 3000])
def test_experts_weights(group, slots):
    """Weights of 5.4 GB. All codes 1, a scale per expert, so that a row of
    another expert is another multiple of the activations' sum."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    log("experts' weights", group, slots)
    rng = np.random.default_rng(slots)
    E, N, K = 512, 4096, 5120
    G = K // group
    qw = torch.full((E * N * K // 8,), 0x11111111, dtype=torch.int32, device="cuda")
    assert qw.numel() * 4 > 1 << 32
    scale = (torch.arange(E, device="cuda") + 1).to(torch.float16) / 512
    sp = scale.view(E, 1).expand(E, N * G).contiguous()
    ids, rows, off = routed(rng, slots, E)
    x = torch.ones((slots, K), dtype=torch.bfloat16, device="cuda")
    y = torch.full((slots, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.w4a16_gemm_experts(x, qw, sp, y, rows, off, slots, E, 1, N, K, group)
    torch.cuda.synchronize()
    want = torch.from_numpy(K * (ids + 1) / 512).cuda().view(-1, 1)  # exact in fp32, then one rounding
    assert bool((y == want.float().to(torch.bfloat16)).all())


@pytest.mark.parametrize("M,N,K", [
    (131200, 16400, 64),                        # y
    (40000, 40, 131072),                        # activations of 5.2 GB
    (4, 25000, 131072), (130, 25000, 131072)])  # weights of 3.3 GB
def test_w8a8(M, N, K):
    import torch

    import w4a16_weight_only_gemm_amd as w4
    log("w8a8", M, N, K)
    g = torch.Generator(device="cuda").manual_seed(M)
    blocks, steps = (N + 15) // 16, K // 64
    xq = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    qw = torch.randint(-127, 128, (blocks, steps, 64, 16), generator=g, device="cuda", dtype=torch.int8)
    sx = (torch.rand(M, generator=g, device="cuda") + 0.5) / 100
    sw = (torch.rand(N, generator=g, device="cuda") + 0.5) / 100
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.w8a8_gemm(xq, sx, qw, sw, y, M, N, K)
    torch.cuda.synchronize()
    back = [moe_ref.ORDER.index(i) for i in range(16)]
    m = torch.from_numpy(sample(M, N, 1) if M > 200 else np.arange(M)[:40]).cuda()
    n = np.arange(N) if K == 64 else sample(N, K, 2)
    tiles = qw[torch.from_numpy(n // 16).cuda()].view(n.size, steps, 4, 16, 16)
    rows = tiles[torch.arange(n.size), :, :, torch.from_numpy(n % 16).cuda()]  # [n][steps][4][16]
    codes = rows.reshape(n.size, K // 16, 16)[:, :, back].reshape(n.size, K).cpu().numpy()
    xs = xq[m].view(-1, K // 16, 16)[:, :, back].reshape(-1, K).cpu().numpy()
    ref, tol = moe_ref.w8a8(xs, sx[m].cpu().numpy(), codes, sw.cpu().numpy()[n])
    moe_ref.check(host_bits(y[m][:, torch.from_numpy(n).cuda()].contiguous()), ref, tol)
    assert not bool(torch.isnan(y).any())


@pytest.mark.parametrize("bias", [False, True])
def test_route(bias):
    """Logits of 8.6 GB: sampled tokens' choices, and the lists of all."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    T, E, k = 1 << 21, 1024, 2
    log("route", T, E, bias)
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn((T, E), generator=g, device="cuda")
    b = torch.randn(E, generator=g, device="cuda") * 0.01 if bias else None
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    rows = torch.empty(T * k, dtype=torch.int32, device="cuda")
    ws = torch.empty(w4.w4a16_moe_route_workspace_bytes(T, E), dtype=torch.int8, device="cuda")
    w4.w4a16_moe_route(z, b, T, E, k, ids, w, off, rows, ws)
    torch.cuda.synchronize()
    at = torch.from_numpy(sample(T, E, 4)).cuda()
    ref = moe_ref.route(values(z[at]), None if b is None else b.cpu().numpy(), k)
    assert np.array_equal(ids[at].cpu().numpy(), ref[0])
    assert np.all(np.abs(values(w[at]) - ref[1]) <= 2 * moe_ref.F32 * ref[1])
    flat = ids.view(-1).long()
    assert int(flat.min()) >= 0
    assert torch.equal(rows.long(), torch.sort(flat, stable=True).indices)
    count = torch.bincount(flat, minlength=E)
    assert torch.equal(off.long(), torch.cat([count.new_zeros(1), torch.cumsum(count, 0)]))
