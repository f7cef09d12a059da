"""w4a16_norm where a row's sums are what decides: constant and nearly constant rows of any
value."""
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
