"""w4a16_norm where a row's sums are what decides: constant and nearly constant rows of
any value, and finite rows whose sum or sum of squares is past fp32 while their mean is
not, or both are."""
import sys

import numpy as np
import pytest

import layer_ref
import moe_ref
from moe_ref import BF16
from test_gpu_experts import dev_bf16, gpu, host_bits  # noqa: F401  (gpu: the fixture)

pytestmark = pytest.mark.gpu

# both sides of every kernel's range
LENGTHS = [2, 5, 7, 8, 100, 128, 250, 512, 640, 2741, 5120, 8200, 16384, 20000, 30001, 65535, 65536]
FLT_MAX = float(np.finfo(np.float32).max)


def log(*a):
    print(*a, file=sys.stderr, flush=True)


def run(rows, kind, bias=None, code=False, post=False, eps=1e-6):
    """rows fp32 [T][N] as the residual, or bf16 bits as a block's output with post norm:
    x in fp64, or codes in natural order and scales."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    T, N = rows.shape
    kw = dict(kind=w4.W4A16_NORM_LAYER if kind == "layer" else w4.W4A16_NORM_RMS, eps=eps)
    b = None if bias is None else dev_bf16(bias)
    if post:
        out = torch.full((T, N), -3.0, dtype=torch.float32, device="cuda")
        w4.w4a16_norm(T, N, y=dev_bf16(rows), residual_out=out, post_norm=True, post_bias=b, **kw)
        return out.double().cpu().numpy()
    res = torch.from_numpy(np.ascontiguousarray(rows)).cuda()
    if code:
        xq = torch.full((T, N), 99, dtype=torch.int8, device="cuda")
        sx = torch.full((T,), -3.0, dtype=torch.float32, device="cuda")
        w4.w4a16_norm(T, N, residual=res, bias=b, xq=xq, sx=sx, **kw)
        return layer_ref.natural(xq.cpu().numpy()).astype(np.float64), sx.double().cpu().numpy()
    x = torch.full((T, N), -3.0, dtype=torch.bfloat16, device="cuda")
    w4.w4a16_norm(T, N, residual=res, bias=b, x=x, **kw)
    return moe_ref.bf16_value(host_bits(x))


def constant_rows(values, N):
    rng = np.random.default_rng(N)
    rows = np.repeat(np.asarray(values, np.float32)[:, None], N, axis=1)
    assert np.all(run(rows, "layer") == 0.0)
    b = moe_ref.bf16_bits(rng.standard_normal(N).astype(np.float32))
    assert np.all(run(rows, "layer", bias=b) == moe_ref.bf16_value(b))
    if N % 16 == 0:
        q, s = run(rows, "layer", code=True)
        assert np.all(q == 0) and np.all(s == 0)


@pytest.mark.parametrize("N", LENGTHS)
def test_constant_rows(N):
    """A layer norm's deviations of equal values are 0, whatever the value."""
    log("norm constant", N)
    constant_rows([1910.2607, 0.1, -3.3e-5, 1 / 3, 7.7e8, *np.random.default_rng(N).uniform(1000, 2000, 12)], N)


@pytest.mark.parametrize("N", [n for n in LENGTHS if n > 2])
def test_nearly_constant_rows(N):
    """Values a few steps of fp32 from 1500, without eps. Steps are exact in 64 bits, and the
    bound is layer_ref's for the steps alone: the deviations of v are those of the steps, which
    have no mean to speak of, so nothing of the size of 1500 x 2^-24 is in it."""
    log("norm nearly constant", N)
    rng = np.random.default_rng(N)
    ulp = 2.0 ** -13  # of numbers in 1024 .. 2048
    for most in (1, 3, 40):
        steps = rng.integers(-most, most + 1, (4, N)).astype(np.float64)
        steps[:, 0], steps[:, 1] = most, -most  # not constant
        rows = (1500.0 + steps * ulp).astype(np.float32)
        assert np.array_equal(rows.astype(np.float64), 1500.0 + steps * ulp)
        _, (v, d) = layer_ref.norm(residual=steps * ulp, kind="layer", eps=0.0)
        got = run(rows, "layer", eps=0.0)
        assert np.all(np.abs(got - v) <= d + BF16 * (np.abs(v) + d)), most


@pytest.mark.parametrize("N", LENGTHS)
def test_far_constant_rows(N):
    """Values whose sum, or whose sum's rounding squared, is past fp32."""
    log("norm far constant", N)
    constant_rows([1.3e25, 2.0 ** 86 / 3, -1.7e31, 1e35 / 3, 2.9e38, -FLT_MAX], N)


@pytest.mark.parametrize("N", LENGTHS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_squares_whose_sum_overflows(N, kind):
    """Mean squares inside fp32 (below 2^127), sums of squares past it for most rows."""
    log("norm squares", N, kind)
    rng = np.random.default_rng(N)
    size = np.array([2.0 ** 57, 2.0 ** 59, 2.0 ** 61, 2.0 ** 62])[:, None]
    rows = (np.clip(rng.standard_normal((4, N)), -2.5, 2.5) * size).astype(np.float32)
    wide = rows.astype(np.float64)
    assert ((wide ** 2).mean(1) < 2.0 ** 127).all()
    b = moe_ref.bf16_bits(rng.standard_normal(N).astype(np.float32))
    _, (v, d) = layer_ref.norm(residual=wide, kind=kind, bias=moe_ref.bf16_value(b))
    got = run(rows, kind, bias=b)
    assert np.all(np.abs(got - v) <= d + BF16 * (np.abs(v) + d))
    if N % 16 == 0:
        q, s = run(rows, kind, bias=b, code=True)
        assert layer_ref.codes(q, s, v, d)
    # the same as a post norm, of bf16 rows
    y = moe_ref.bf16_bits(rows)
    (r, dr), _ = layer_ref.norm(y=moe_ref.bf16_value(y), kind=kind, post=True, post_bias=moe_ref.bf16_value(b))
    assert np.all(np.abs(run(y, kind, bias=b, post=True) - r) <= dr)


@pytest.mark.parametrize("N", [2, 7, 8, 100, 128, 512, 2741, 5120, 16384, 30001, 65536])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_mean_squares_past_fp32(N, kind):
    """The mean square is infinite, of a layer norm often the plain sum, the mean on the way to
    it or a deviation too: the row is zeros and biases."""
    log("norm past fp32", N, kind)
    rng = np.random.default_rng(N)
    alternate = np.where(np.arange(N) % 2 == 0, 1.0, -1.0)
    rows = np.stack([rng.standard_normal(N) * 1e30, alternate * 3.3e38, np.where(np.arange(N) < N // 2, 1.0, -1.0) * 3.3e38,
                     np.where(np.arange(N) == N // 2, -1.0, 1.0) * FLT_MAX, rng.uniform(1e35, 3e38, N),
                     np.where(np.arange(N) == 0, FLT_MAX, 1.0)]).astype(np.float32)
    wide = rows.astype(np.float64)
    dev = wide - wide.mean(1, keepdims=True) if kind == "layer" else wide
    assert ((dev ** 2).mean(1) > 2.0 ** 128).all()
    assert np.all(run(rows, kind) == 0.0)
    b = moe_ref.bf16_bits(rng.standard_normal(N).astype(np.float32))
    bv = moe_ref.bf16_value(b)
    assert np.all(run(rows, kind, bias=b) == bv)
    if N % 16 == 0:
        q, s = run(rows, kind, code=True)
        assert np.all(q == 0) and np.all(s == 0)
        q, s = run(rows, kind, bias=b, code=True)
        assert layer_ref.codes(q, s, np.repeat(bv[None], 6, axis=0), np.zeros((6, N)))
    # the same as a post norm, of bf16 rows (FLT_MAX and 3.3e38 to values that bf16 holds)
    y = moe_ref.bf16_bits(np.clip(rows, -3.3e38, 3.3e38))
    assert np.all(run(y, kind, bias=b, post=True) == bv)


@pytest.mark.parametrize("N", [7, 100, 512, 2741, 5120, 16384])
def test_not_finite_stays_in_its_row(N):
    """Infinities and NaN among rows that need the sums' other ways: a layer norm's row is NaN,
    an RMS norm's row of an infinity is NaN there and 0 elsewhere, and the others are as they
    are without."""
    rng = np.random.default_rng(N)
    rows = np.concatenate([rng.standard_normal((3, N)), np.full((2, N), 1910.2607), rng.standard_normal((2, N)) * 2.0 ** 61,
                           np.full((2, N), 2.9e38)]).astype(np.float32)
    bad = rows.copy()
    for t, v in ((1, np.inf), (3, np.nan), (5, -np.inf), (7, np.inf)):
        bad[t, N - 1] = v
    keep = [0, 2, 4, 6, 8]
    for kind in ("rms", "layer"):
        want, got = run(rows, kind), run(bad, kind)
        assert np.array_equal(want[keep], got[keep]) and np.isfinite(want).all()
        assert np.isnan(got[[1, 3, 5, 7], N - 1]).all() and np.isnan(got[3]).all()
        if kind == "layer":
            assert np.isnan(got[[1, 3, 5, 7]]).all()
        else:
            assert np.all(got[[1, 5, 7], :N - 1] == 0.0)
