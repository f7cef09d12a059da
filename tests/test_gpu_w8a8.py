"""w8a8_gemm on the GPU against exact integer sums (moe_ref), from one row to
the tile engine, ragged columns and k, extreme codes, and after w4a8_quantize."""
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


def run(xq, sx, q, sw, guard=16):
    """One call; the output has guard rows behind it that must keep their value."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    M, K = xq.shape
    N = q.shape[0]
    y = torch.full((M + guard, N), -3.0, dtype=torch.bfloat16, device="cuda")
    w4.w8a8_gemm(torch.from_numpy(moe_ref.arrange_codes(xq)).cuda(), torch.from_numpy(sx).cuda(),
                 torch.from_numpy(w4.w8a8_pack(q)).cuda(), torch.from_numpy(sw).cuda(), y, M, N, K)
    torch.cuda.synchronize()
    bits = y.view(torch.int16).cpu().numpy().view(np.uint16)
    assert np.all(bits[M:] == 0xC040)
    return bits[:M]


def check(M, N, K, seed=0, low=-127, high=128):
    log(f"w8a8 M={M} N={N} K={K}")
    rng = np.random.default_rng(seed)
    xq = rng.integers(low, high, (M, K)).astype(np.int8)
    q = rng.integers(-128, 128, (N, K)).astype(np.int8)
    sx = (rng.random(M) + 0.5).astype(np.float32) / 100
    sw = (rng.random(N) + 0.5).astype(np.float32) / 100
    ref, tol = moe_ref.w8a8(xq, sx, q, sw)
    moe_ref.check(run(xq, sx, q, sw), ref, tol, (M, N, K))


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 129, 200, 256, 257, 300, 513])
@pytest.mark.parametrize("N,K", [(96, 512), (100, 208)])
def test_rows(M, N, K):
    check(M, N, K, seed=M)


@pytest.mark.parametrize("M", [1, 40, 150, 530])
@pytest.mark.parametrize("N", [1, 15, 17, 255, 258, 1030])
def test_columns(M, N):
    check(M, N, 272, seed=N)


@pytest.mark.parametrize("M", [3, 70, 140, 600])
@pytest.mark.parametrize("K", [16, 32, 48, 64, 80, 112, 128, 144, 192, 240, 1040, 2064])
def test_depths(M, K):
    check(M, 40, K, seed=K)


@pytest.mark.parametrize("M,N,K", [
    (1, 200, 1040), (5, 5000, 656), (12, 5000, 656),          # one row block by one and two
    (120, 800, 1040), (30, 7000, 656), (60, 3500, 1040),      # also several row tiles; two by two
    (60, 7000, 656), (60, 5000, 1040), (90, 5000, 1040),      # two by four and three
    (120, 5000, 656), (101, 5010, 656), (64, 11000, 400),     # tiles of 64 x 64
    (190, 5000, 784), (437, 1811, 784), (64, 9000, 2064),
    (520, 1000, 272), (1100, 2950, 144), (1090, 2957, 208),   # 64 x 64 and 128 x 128
    (4000, 2950, 144), (3970, 2941, 272), (4090, 2944, 64)])  # 256 x 192
def test_every_form(M, N, K):
    check(M, N, K, seed=M + N)


@pytest.mark.parametrize("K", [48, 144, 272, 400, 544, 656, 784, 1040])
@pytest.mark.parametrize("M,N", [(553, 217), (66, 8555), (135, 11790), (389, 12643), (261, 12069),
                                 (775, 12447), (654, 11010)])
def test_k_tiles(M, N, K):
    """The tiles (64 x 64, 64 x 128, 128 x 128 and 128 x 192 with many and with two
    buffers, 256 x 192) over fewer k-tiles of 128 than they hold buffers, as many,
    and more; the last one partial."""
    check(M, N, K, seed=K)


@pytest.mark.parametrize("M", [1, 130])
def test_deepest_sum(M):
    """Every product 127 * 127 or -128 * 127 at the largest K: the sums are the
    largest there are, and exact."""
    K = 131072
    sx, sw = np.full(M, 1.0, np.float32), np.full(2, 1.0, np.float32)
    q = np.stack([np.full(K, 127, np.int8), np.full(K, -128, np.int8)])
    xq = np.full((M, K), 127, np.int8)
    ref, tol = moe_ref.w8a8(xq, sx, q, sw)
    moe_ref.check(run(xq, sx, q, sw), ref, tol)


def test_zero_scales_and_codes():
    rng = np.random.default_rng(0)
    for M in (4, 260):
        xq = rng.integers(-127, 128, (M, 128)).astype(np.int8)
        q = rng.integers(-128, 128, (20, 128)).astype(np.int8)
        sx, sw = np.ones(M, np.float32), np.ones(20, np.float32)
        sx[1], sw[3], xq[2], q[5] = 0, 0, 0, 0
        got = moe_ref.bf16_value(run(xq, sx, q, sw))
        assert np.all(got[1] == 0) and np.all(got[:, 3] == 0)
        assert np.all(got[2] == 0) and np.all(got[:, 5] == 0)


@pytest.mark.parametrize("M", [1, 5, 64, 300])
def test_after_quantize(M):
    """bf16 rows through w4a8_quantize: the product of the codes it wrote."""
    import torch

    import oracle
    import w4a16_weight_only_gemm_amd as w4
    rng = np.random.default_rng(M)
    K, N = 640, 72
    x = moe_ref.bf16_bits(rng.standard_normal((M, K)).astype(np.float32))
    q = rng.integers(-128, 128, (N, K)).astype(np.int8)
    sw = (rng.random(N) + 0.5).astype(np.float32) / 100
    dx = torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)
    xq = torch.empty((M, K), dtype=torch.int8, device="cuda")
    sx = torch.empty(M, device="cuda")
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    w4.w4a8_quantize(dx, xq, sx, M, K)
    w4.w8a8_gemm(xq, sx, torch.from_numpy(w4.w8a8_pack(q)).cuda(), torch.from_numpy(sw).cuda(), y,
                 M, N, K)
    torch.cuda.synchronize()
    codes, scale = oracle.quantize_rows(x)
    assert np.array_equal(moe_ref.arrange_codes(codes), xq.cpu().numpy())
    ref, tol = moe_ref.w8a8(codes, scale, q, sw)
    moe_ref.check(y.view(torch.int16).cpu().numpy().view(np.uint16), ref, tol)


def test_no_rows():
    import torch

    import w4a16_weight_only_gemm_amd as w4
    t = torch.zeros(64 * 64, dtype=torch.int8, device="cuda")
    f = torch.zeros(64, device="cuda")
    w4.w8a8_gemm(t, f, t, f, torch.zeros(64, dtype=torch.bfloat16, device="cuda"), 0, 64, 64)
