"""One matrix of 2 to 4 GiB of packed weights through every kernel that reads it by a
buffer of 32-bit size: w4a16_gemm's tiles, its epilogue, its grouped schedule, the
experts' products and w4a8_gemm. N x K is 2^32 and more here, so a size formed from it
before it is halved would not fit. Columns repeat every PART, so one small matrix in 64
bits stands for all of them."""
import sys

import numpy as np
import pytest

import layer_ref
import moe_ref
from moe_ref import BF16, F32
from test_gpu_epilogue import Case
from test_gpu_experts import gpu, host_bits  # noqa: F401  (gpu: the fixture)

pytestmark = pytest.mark.gpu

K, PART, GROUP = 16384, 1024, 128
# N x K = 2^32, 3/2 of it, and the last repetition below 4 GiB of weights
WIDTHS = [262144, 393216, 523264]


def log(*a):
    print(*a, file=sys.stderr, flush=True)


def weights(c, N):
    import w4a16_weight_only_gemm_amd as w4
    assert N % PART == 0 and N * K >= 1 << 32 and w4.w4a16_qweight_bytes(N, K) < 1 << 32
    return c.qw.repeat(N // PART), c.sp.repeat(N // PART)


def check(y, ref, tol, what):
    """The first repetition against 64 bits, and each other by the first's bits."""
    import torch
    first = y[:, :PART].contiguous()
    moe_ref.check(host_bits(first), ref, tol, what)
    for i in range(1, y.shape[1] // PART):
        assert torch.equal(y[:, i * PART:(i + 1) * PART], first), (what, i)


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("M", [17, 33, 200])
def test_products(M, N):
    import torch

    import w4a16_weight_only_gemm_amd as w4
    log(f"tile weights M={M} N={N}")
    c = Case(M, PART, K, GROUP, M)
    qw, sp = weights(c, N)
    x = moe_ref.bf16_value(c.x)
    y = torch.full((M, N), -3.0, dtype=torch.bfloat16, device="cuda")
    w4.w4a16_gemm_ex(c.dx, qw, sp, y, M, N, K, GROUP, w4.W4A16_PATH_LARGE)
    check(y, *layer_ref.epilogue(x, c.q, c.s, GROUP), "tiles")
    y.fill_(-3.0)
    w4.w4a16_gemm(c.dx, qw, sp, y, M, N, K, GROUP)
    check(y, *layer_ref.epilogue(x, c.q, c.s, GROUP), "gemm")
    y.fill_(-3.0)
    w4.w4a16_gemm_epilogue(c.dx, qw, sp, y, M, N, K, GROUP, act=w4.W4A16_ACT_SILU)
    check(y, *layer_ref.epilogue(x, c.q, c.s, GROUP, "silu"), "epilogue")
    half = torch.full((M, N // 2), -3.0, dtype=torch.bfloat16, device="cuda")
    w4.w4a16_gemm_epilogue(c.dx, qw, sp, half, M, N, K, GROUP, act=w4.W4A16_ACT_SWIGLU)
    up = (np.arange(PART) + N // 2) % PART
    check(half[:, :half.shape[1] // PART * PART],
          *layer_ref.epilogue(x, np.concatenate([c.q, c.q[up]]), np.concatenate([c.s, c.s[up]]), GROUP, "swiglu"),
          "gated")


def test_grouped():
    """The schedule over several problems adds a tile's parts in another order where a
    cut lies, so every repetition is held to the bound."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    M, N = 64, 393216
    log("tile weights grouped")
    c = Case(M, PART, K, GROUP, 1)
    qw, sp = weights(c, N)
    ys = [torch.full((M, N), -3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = torch.zeros(w4.w4a16_workspace_bytes(M, 2 * N) // 4 + 1, dtype=torch.int32, device="cuda")
    w4.w4a16_gemm_grouped([(c.dx, qw, sp, y, N, K) for y in ys], M, GROUP, ws)
    ref, _ = layer_ref.product(moe_ref.bf16_value(c.x), c.q, c.s, GROUP)
    # the bound of a whole sum, and of the parts': at most K / GROUP more additions
    mag = np.abs(moe_ref.bf16_value(c.x)) @ ((np.abs(24.0 + c.q) + 24.0) * np.repeat(c.s, GROUP, axis=1)).T
    d = (GROUP + 2 * (K // GROUP) + 20) * F32 * mag
    tol = d + BF16 * (np.abs(ref) + d)
    want, tol = torch.from_numpy(ref).cuda(), torch.from_numpy(tol).cuda()
    for y in ys:
        off = (y.view(M, -1, PART).double() - want[:, None]).abs() - tol[:, None]
        assert float(off.max()) <= 0.0


@pytest.mark.parametrize("slots", [20, 200])
def test_experts(slots):
    import torch

    import w4a16_weight_only_gemm_amd as w4
    N = 393216
    log(f"tile weights experts {slots}")
    c = Case(slots, PART, K, GROUP, 2)
    qw, sp = weights(c, N)
    rows = torch.arange(slots, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, slots], dtype=torch.int32, device="cuda")
    y = torch.full((slots, N), -3.0, dtype=torch.bfloat16, device="cuda")
    w4.w4a16_gemm_experts(c.dx, qw, sp, y, rows, off, slots, 1, 1, N, K, GROUP, act=w4.W4A16_ACT_NONE)
    ref, tol = moe_ref.experts(moe_ref.bf16_value(c.x), c.q[None], c.s[None], np.arange(slots), np.array([0, slots]), 1,
                               GROUP)
    check(y, ref, tol, "experts")


@pytest.mark.parametrize("M", [40, 300])
@pytest.mark.parametrize("N", WIDTHS[1:])
def test_w4a8(M, N):
    import torch

    import w4a16_weight_only_gemm_amd as w4
    log(f"tile weights w4a8 M={M} N={N}")
    c = Case(M, PART, K, GROUP, 3)
    qw, sp = weights(c, N)
    xq = torch.empty((M, K), dtype=torch.int8, device="cuda")
    sx = torch.empty(M, dtype=torch.float32, device="cuda")
    w4.w4a8_quantize(c.dx, xq, sx, M, K)
    y = torch.full((M, N), -3.0, dtype=torch.bfloat16, device="cuda")
    w4.w4a8_gemm(xq, sx, qw, sp, y, M, N, K, GROUP)
    codes = layer_ref.natural(xq.cpu().numpy()).astype(np.float64)
    scale = sx.double().cpu().numpy()[:, None]
    ref = codes @ (c.q * np.repeat(c.s, GROUP, axis=1)).T * scale
    # integer sums of a group are exact; each is converted, scaled and added in fp32
    mag = np.abs(codes) @ (np.abs(c.q) * np.repeat(c.s, GROUP, axis=1)).T * scale
    d = (K // GROUP + 4) * F32 * mag
    check(y, ref, d + BF16 * (np.abs(ref) + d), "w4a8")
