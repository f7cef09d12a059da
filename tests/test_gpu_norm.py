"""w4a16_norm on the GPU against 64 bits (layer_ref): every row length range, both
kinds, every combination of post norm, gate, residual type and output."""
import itertools
import sys

import numpy as np
import pytest

import layer_ref
import moe_ref
from moe_ref import BF16, F32
from test_gpu_experts import dev_bf16, gpu, host_bits  # noqa: F401  (gpu: the fixture)

pytestmark = pytest.mark.gpu


def log(*a):
    print(*a, file=sys.stderr, flush=True)


def run(T, N, seed, kind="rms", post=False, gate=0, wide=False, code=False, scale=1.0, unit=False,
        weights=True, bias=False, block=True, has_residual=True, in_place=False, size=1.0, eps=1e-6,
        stream=None):
    """One call on random rows: outputs and their references."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    rng = np.random.default_rng(seed)

    def bits(*shape, size=1.0, mean=0.0):
        return moe_ref.bf16_bits((rng.standard_normal(shape) * size + mean).astype(np.float32))

    mean = 0.0 if unit else 1.0
    host, dev = {}, {}

    def vector(name, on, mean=0.0):
        host[name] = bits(N, size=0.3, mean=mean) if on else None
        dev[name] = None if host[name] is None else dev_bf16(host[name])
        return None if host[name] is None else moe_ref.bf16_value(host[name])

    y = bits(T, N, size=size) if block else None
    w = vector("weight", weights, mean)
    b = vector("bias", bias)
    pw = vector("post_weight", post and weights, mean)
    pb = vector("post_bias", post and bias)
    g = bits(-(-T // gate), N) if gate else None
    if wide:
        res32 = (rng.standard_normal((T, N)) * 2 * size).astype(np.float32)
        res, dres = res32.astype(np.float64), torch.from_numpy(res32).cuda()
    else:
        r = bits(T, N, size=2 * size)
        res, dres = moe_ref.bf16_value(r), dev_bf16(r)
    if not has_residual:
        res = dres = None
    stored = torch.float32 if wide else torch.bfloat16
    # guards behind the last row
    rout = torch.full(((T + 1) * N,), -3.0, dtype=stored, device="cuda")
    if in_place:
        rout[:T * N] = dres.reshape(-1)
        dres = rout[:T * N]
    x = torch.full(((T + 1) * N,), -3.0, dtype=torch.bfloat16, device="cuda") if not code else None
    xq = torch.full(((T + 1) * N,), 99, dtype=torch.int8, device="cuda") if code else None
    sx = torch.full((T + 1,), -3.0, dtype=torch.float32, device="cuda") if code else None
    w4.w4a16_norm(T, N, y=None if y is None else dev_bf16(y), residual=dres, residual_out=rout,
                  post_norm=post, gate=None if g is None else dev_bf16(g), gate_rows=max(gate, 1),
                  scale=scale, x=x, xq=xq, sx=sx, eps=eps, unit_offset=unit,
                  kind=w4.W4A16_NORM_LAYER if kind == "layer" else w4.W4A16_NORM_RMS,
                  residual_type=w4.W4A16_RESIDUAL_F32 if wide else w4.W4A16_RESIDUAL_BF16,
                  stream=stream, **dev)
    torch.cuda.synchronize()
    refs = layer_ref.norm(None if y is None else moe_ref.bf16_value(y), res, kind, eps, post, pw, pb,
                          None if g is None else moe_ref.bf16_value(g), max(gate, 1), scale, w, b, unit)
    return rout, x, xq, sx, refs


def verify(T, N, seed, **kw):
    log("norm", T, N, kw)
    rout, x, xq, sx, ((r, dr), (v, dv)) = run(T, N, seed, **kw)
    assert bool((rout[T * N:] == -3.0).all())
    if kw.get("wide"):
        got = rout[:T * N].view(T, N).double().cpu().numpy()
        assert np.all(np.abs(got - r) <= dr)  # its rounding is in dr: r is held in fp32
    else:
        moe_ref.check(host_bits(rout[:T * N]).reshape(T, N), r, dr + BF16 * (np.abs(r) + dr), "residual")
    if x is not None:
        assert bool((x[T * N:] == -3.0).all())
        moe_ref.check(host_bits(x[:T * N]).reshape(T, N), v, dv + BF16 * (np.abs(v) + dv), "x")
    else:
        assert bool((xq[T * N:] == 99).all()) and float(sx[T]) == -3.0
        q = layer_ref.natural(xq[:T * N].view(T, N).cpu().numpy()).astype(np.float64)
        assert layer_ref.codes(q, sx[:T].double().cpu().numpy(), v, dv)


# row lengths at both sides of every kernel's range, and odd ones
LENGTHS = [1, 2, 7, 8, 9, 100, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1000, 2741, 5120, 8191, 8192, 8193,
           16384, 16385, 20000]


@pytest.mark.parametrize("N", LENGTHS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_lengths(N, kind):
    # one column's deviation from its mean is 0: eps decides
    verify(5, N, N, kind=kind, post=True, bias=kind == "layer", eps=1e-5)
    verify(3, N, N + 1, kind=kind, wide=True, gate=2, scale=0.5)


@pytest.mark.parametrize("N", [32768, 40001, 65535, 65536])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_long_rows(N, kind):
    verify(3, N, N, kind=kind, post=True, bias=True, gate=3)


@pytest.mark.parametrize("kind,post,gate,wide,code,unit", itertools.product(
    ["rms", "layer"], [False, True], [0, 3], [False, True], [False, True], [False, True]))
def test_combinations(kind, post, gate, wide, code, unit):
    verify(7, 272, 11, kind=kind, post=post, gate=gate, wide=wide, code=code, unit=unit, bias=True, scale=0.7)


@pytest.mark.parametrize("N", [16, 112, 128, 144, 256, 512, 528, 1024, 5120, 8192, 8208, 17408, 65536])
def test_codes(N):
    verify(4, N, N, code=True, post=True)
    verify(2, N, N, code=True, block=False, wide=True)


@pytest.mark.parametrize("T", [1, 2, 3, 15, 16, 17, 1000, 5000])
@pytest.mark.parametrize("N", [64, 250, 500, 1030])
def test_rows(T, N):
    verify(T, N, T, post=True, gate=T)
    verify(T, N, T, block=False)


@pytest.mark.parametrize("kw", [dict(weights=False), dict(weights=False, post=True, kind="layer"),
                                dict(has_residual=False), dict(has_residual=False, post=True, gate=1, wide=True),
                                dict(block=False, bias=True), dict(scale=0.0), dict(scale=-3.0, post=True),
                                dict(eps=0.0), dict(eps=0.5, post=True), dict(size=1e-12), dict(size=1e15),
                                dict(size=1e-4, kind="layer", post=True)])
def test_parts_left_out(kw):
    verify(6, 600, 3, **kw)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("N", [250, 5120])
def test_residual_in_place(wide, N):
    a = run(9, N, 4, post=True, wide=wide)
    b = run(9, N, 4, post=True, wide=wide, in_place=True)
    import torch
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_only_one_output():
    import torch

    import w4a16_weight_only_gemm_amd as w4
    y = torch.randn(5, 640, device="cuda").to(torch.bfloat16)
    r = torch.randn(5, 640, device="cuda").to(torch.bfloat16)
    x1, x2, ro1, ro2 = (torch.full((5, 640), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    w4.w4a16_norm(5, 640, y=y, residual=r, residual_out=ro1, x=x1)
    w4.w4a16_norm(5, 640, y=y, residual=r, x=x2)
    w4.w4a16_norm(5, 640, y=y, residual=r, residual_out=ro2)
    assert torch.equal(x1, x2) and torch.equal(ro1, ro2)
    assert torch.equal(ro1, (y.float() + r.float()).to(torch.bfloat16))


def test_mean_far_from_zero():
    """Layer norms of rows whose mean is 1000 of their deviations: two passes."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    rng = np.random.default_rng(1)
    for N in (100, 700, 5120):
        res = (rng.standard_normal((4, N)) + 1000).astype(np.float32)
        x = torch.empty((4, N), dtype=torch.bfloat16, device="cuda")
        w4.w4a16_norm(4, N, residual=torch.from_numpy(res).cuda(), x=x, kind=w4.W4A16_NORM_LAYER)
        _, (v, dv) = layer_ref.norm(residual=res.astype(np.float64), kind="layer")
        moe_ref.check(host_bits(x), v, dv + BF16 * (np.abs(v) + dv))


def test_rows_of_zeros():
    import torch

    import w4a16_weight_only_gemm_amd as w4
    for N in (64, 400, 2048):
        y = torch.zeros((3, N), dtype=torch.bfloat16, device="cuda")
        y[1] = 1.0
        for kind in (w4.W4A16_NORM_RMS, w4.W4A16_NORM_LAYER):
            x = torch.empty_like(y)
            w4.w4a16_norm(3, N, y=y, x=x, kind=kind)
            want = 0.0 if kind == w4.W4A16_NORM_LAYER else 1.0
            assert bool((x[0] == 0).all()) and bool((x[2] == 0).all()) and bool((x[1] == want).all())
            xq = torch.full((3, N), 5, dtype=torch.int8, device="cuda")
            sx = torch.full((3,), 5.0, device="cuda")
            w4.w4a16_norm(3, N, y=y, xq=xq, sx=sx, kind=kind)
            assert bool((xq[0] == 0).all()) and float(sx[0]) == 0.0 and float(sx[2]) == 0.0
            assert bool((xq[1] == (0 if want == 0 else 127)).all())


def test_not_finite_stays_in_its_row():
    import torch

    import w4a16_weight_only_gemm_amd as w4
    for N in (64, 300, 1500):
        y = torch.randn(9, N, device="cuda").to(torch.bfloat16)
        r = torch.randn(9, N, device="cuda").to(torch.bfloat16)
        x0, x1 = torch.empty_like(y), torch.empty_like(y)
        w4.w4a16_norm(9, N, y=y, residual=r, x=x0, post_norm=True)
        y[4, N - 1], r[7, 0] = float("nan"), float("inf")
        w4.w4a16_norm(9, N, y=y, residual=r, x=x1, post_norm=True)
        keep = [i for i in range(9) if i not in (4, 7)]
        assert torch.equal(x0[keep], x1[keep])
        assert bool(torch.isnan(x1[4]).all()) and bool(torch.isnan(x1[7, 0]))


def test_overflowing_squares():
    import torch

    import w4a16_weight_only_gemm_amd as w4
    y = torch.full((2, 256), 3e38, dtype=torch.bfloat16, device="cuda")
    x = torch.empty_like(y)
    w4.w4a16_norm(2, 256, y=y, x=x)
    assert bool((x == 0).all())


@pytest.mark.parametrize("N", [1000, 5120])
def test_codes_near_those_of_two_calls(N):
    """The codes of the norm's own rounding to bf16 first differ by at most one where the
    bf16 row is off by half a step (127 / a times it is below one unit)."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    N = N // 16 * 16
    y = torch.randn(6, N, device="cuda").to(torch.bfloat16)
    x = torch.empty_like(y)
    w4.w4a16_norm(6, N, y=y, x=x)
    q1, q2 = (torch.empty((6, N), dtype=torch.int8, device="cuda") for _ in range(2))
    s1, s2 = (torch.empty(6, dtype=torch.float32, device="cuda") for _ in range(2))
    w4.w4a16_norm(6, N, y=y, xq=q1, sx=s1)
    w4.w4a8_quantize(x, q2, s2, 6, N)
    assert int((q1.int() - q2.int()).abs().max()) <= 1
    assert bool(((s1 - s2).abs() <= (BF16 + 4 * F32) * s1).all())


def test_far_rows():
    """Elements past 2^31: border rows and the ends, in place."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    for T, N in ((1050000, 2056), (8500000, 256)):
        log("norm far rows", T, N)
        assert T * N > 1 << 31
        g = torch.Generator(device="cuda").manual_seed(1)
        r = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        for t in range(0, T, 1 << 18):
            n = min(1 << 18, T - t)
            r[t:t + n] = torch.randn((n, N), generator=g, device="cuda")
        border = (1 << 31) // N
        at = torch.tensor([0, 1, border - 1, border, border + 1, T - 2, T - 1], device="cuda")
        before = r[at].double().cpu().numpy()
        x, y = torch.empty_like(r), r.clone()
        w4.w4a16_norm(T, N, y=y, residual=r, residual_out=r, x=x, scale=0.5)
        (a, da), (v, dv) = layer_ref.norm(before, before, scale=0.5)
        moe_ref.check(host_bits(r[at]), a, da + BF16 * (np.abs(a) + da))
        moe_ref.check(host_bits(x[at]), v, dv + BF16 * (np.abs(v) + dv))
        del r, x, y


def test_codes_of_tiny_rows():
    """Rows whose 127 / max is past fp32: codes still follow the values. A value is off by
    a few half steps of fp32 and by half a step of the smallest number, 2^-150, which is
    2^-150 * 127 / max < 2^-16 of a code here."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    rng = np.random.default_rng(5)
    T, N = 3, 64
    y = moe_ref.bf16_bits(rng.standard_normal((T, N)).astype(np.float32))
    w = np.full(N, 2.0 ** -126, np.float32)
    xq = torch.full((T, N), 99, dtype=torch.int8, device="cuda")
    sx = torch.full((T,), -3.0, dtype=torch.float32, device="cuda")
    w4.w4a16_norm(T, N, y=dev_bf16(y), weight=dev_bf16(moe_ref.bf16_bits(w)), xq=xq, sx=sx)
    torch.cuda.synchronize()
    yv = moe_ref.bf16_value(y)
    v = yv / np.sqrt((yv * yv).mean(1, keepdims=True) + float(np.float32(1e-6))) * 2.0 ** -126
    a = np.abs(v).max(1, keepdims=True)
    assert np.all(a < 127.0 / 2.0 ** 128)
    q = layer_ref.natural(xq.cpu().numpy()).astype(np.float64)
    assert np.all(np.abs(q - v * 127.0 / a) <= 0.5 + 2.0 ** -10)
    assert np.all(np.abs(sx.double().cpu().numpy() - a[:, 0] / 127.0) <= 2.0 ** -148)
