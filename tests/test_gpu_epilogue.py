"""w4a16_gemm_epilogue on the GPU against a 64-bit product and epilogue (layer_ref):
every activation, both kernels' row ranges, every group size, ragged sizes, in-place
residuals, and w4a16_gemm's bits where nothing follows the product."""
import sys

import numpy as np
import pytest

import layer_ref
import moe_ref
from test_gpu_experts import dev_bf16, gpu, host_bits  # noqa: F401  (gpu: the fixture)

pytestmark = pytest.mark.gpu

ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu", "swiglu", "geglu"]
GATED = ("swiglu", "geglu")


def log(*a):
    print(*a, file=sys.stderr, flush=True)


class Case:
    def __init__(self, M, N, K, group, seed, x_scale=1.0):
        import torch

        import w4a16_weight_only_gemm_amd as w4
        rng = np.random.default_rng(seed)
        self.M, self.N, self.K, self.group, self.rng = M, N, K, group, rng
        self.q = rng.integers(-8, 8, (N, K)).astype(np.int8)
        s16 = ((rng.random((N, K // group)) + 0.5) / (4 * np.sqrt(K))).astype(np.float16)
        self.s = s16.astype(np.float64)
        qw, sp = w4.w4a16_pack(self.q, s16, group)
        self.qw = torch.from_numpy(qw.view(np.int32)).cuda()
        self.sp = torch.from_numpy(sp.view(np.int16)).cuda()
        self.x = self.bits(M, K, size=x_scale)
        self.dx = dev_bf16(self.x)

    def bits(self, *shape, size=1.0):
        return moe_ref.bf16_bits((self.rng.standard_normal(shape) * size).astype(np.float32))

    def run(self, act="none", bias=None, residual=None, scale=1.0, in_place=False, stream=None):
        import torch

        import w4a16_weight_only_gemm_amd as w4
        out = self.N // 2 if act in GATED else self.N
        # a guard row behind y: what follows the last row stays as it is
        y = torch.full((self.M + 1, out), -3.0, dtype=torch.bfloat16, device="cuda")
        res = None if residual is None else dev_bf16(residual)
        if in_place:
            y[:self.M] = res
            res = y[:self.M]
        w4.w4a16_gemm_epilogue(self.dx, self.qw, self.sp, y[:self.M], self.M, self.N, self.K, self.group,
                               bias=None if bias is None else dev_bf16(bias), residual=res, scale=scale,
                               act=getattr(w4, "W4A16_ACT_" + act.upper()), stream=stream)
        got = host_bits(y)
        assert np.all(got[self.M] == 0xC040)
        return got[:self.M]

    def check(self, act="none", bias=False, residual=False, scale=1.0, in_place=False):
        log(f"epilogue M={self.M} N={self.N} K={self.K} g={self.group} {act} bias={bias} residual={residual}")
        out = self.N // 2 if act in GATED else self.N
        b = self.bits(self.N) if bias else None
        r = self.bits(self.M, out) if residual else None
        got = self.run(act, b, r, scale, in_place)
        ref, tol = layer_ref.epilogue(moe_ref.bf16_value(self.x), self.q, self.s, self.group, act,
                                      None if b is None else moe_ref.bf16_value(b),
                                      None if r is None else moe_ref.bf16_value(r), scale)
        moe_ref.check(got, ref, tol, (act, self.M, self.N))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("M", [1, 7, 16, 40, 200])
def test_activations(act, group, M):
    Case(M, 160, 768, group, M).check(act, bias=True, residual=True, scale=0.75)


@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (5, 96, 32), (16, 128, 128), (17, 128, 64), (260, 384, 128),
                                       (40, 2176, 128), (33, 160, 32), (513, 256, 256), (8200, 128, 128)])
@pytest.mark.parametrize("M", [1, 3, 33, 130])
def test_odd_sizes(N, K, group, M):
    c = Case(M, N, K, group, N)
    c.check("silu", bias=True, residual=True)
    c.check("none", residual=True, scale=-0.5)


@pytest.mark.parametrize("N,K,group", [(32, 128, 128), (96, 96, 32), (544, 256, 64), (16896, 128, 128), (1088, 1536, 128),
                                       (320, 512, 256), (6240, 2176, 128)])
@pytest.mark.parametrize("M", [1, 2, 4, 8, 12, 16, 17, 31, 64, 65, 129])
def test_gated_forms(N, K, group, M):
    Case(M, N, K, group, N + M).check("swiglu", bias=M % 2 == 0)


@pytest.mark.parametrize("N,K,M", [(2080, 6144, 1), (2080, 12800, 2), (2048, 5120, 8), (2048, 1024, 16),
                                   (16448, 640, 3), (16448, 640, 14), (16448, 640, 28), (4128, 640, 300),
                                   (4128, 1280, 700)])
@pytest.mark.parametrize("act", ["none", "geglu"])
def test_every_form(N, K, M, act):
    """The shapes at which w4a16_gemm changes its form, few and many rows."""
    Case(M, N, K, 128, M).check(act, residual=True, scale=2.0)


@pytest.mark.parametrize("M,N,K,group", [(1, 100, 256, 128), (5, 4096, 1024, 128), (16, 16400, 256, 128),
                                         (33, 600, 512, 64), (300, 1000, 640, 128), (70, 300, 512, 256)])
def test_bits_of_the_plain_product(M, N, K, group):
    import torch

    import w4a16_weight_only_gemm_amd as w4
    c = Case(M, N, K, group, 3)
    y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    w4.w4a16_gemm(c.dx, c.qw, c.sp, y, M, N, K, group)
    assert np.array_equal(host_bits(y), c.run())


@pytest.mark.parametrize("M,act", [(1, "none"), (16, "swiglu"), (50, "gelu"), (300, "swiglu"), (300, "none")])
def test_residual_in_place(M, act):
    c = Case(M, 1056, 384, 128, M)
    r = c.bits(M, 528 if act in GATED else 1056)
    assert np.array_equal(c.run(act, None, r, 0.5), c.run(act, None, r, 0.5, in_place=True))
    c.check(act, residual=True, scale=0.5, in_place=True)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu", "swiglu", "geglu"])
@pytest.mark.parametrize("M", [4, 130])
def test_far_values(act, M):
    """Sums of -40 to 40: the activations' flat ends."""
    Case(M, 64, 256, 64, 5, x_scale=8.0).check(act, residual=True)


def test_values_past_the_exponential():
    """Sums of a few thousand: silu and gelu are 0 or the value itself, no NaN."""
    for act in ACTS:
        for M in (3, 140):
            c = Case(M, 64, 256, 128, 6, x_scale=3000.0)
            got = moe_ref.bf16_value(c.run(act))
            assert np.isfinite(got).all(), act
            p, _ = layer_ref.product(moe_ref.bf16_value(c.x), c.q, c.s, 128)
            far = np.abs(p) > 200
            if act not in GATED:
                want = np.where(p > 0, p, 0.0) if act != "none" else p
                assert np.all(np.abs(got - want)[far] <= 0.01 * np.abs(want)[far]), act


@pytest.mark.parametrize("M", [2, 200])
def test_not_finite(M):
    """A NaN or an infinity stays in its row; a NaN in bias or residual in its column."""
    c = Case(M, 64, 256, 128, 7)
    clean = c.run("silu")
    bits = c.x.copy()
    bits[1, 3] = 0x7FC0
    c.dx = dev_bf16(bits)
    got = c.run("silu")
    assert np.isnan(moe_ref.bf16_value(got)[1]).all()
    assert np.array_equal(np.delete(got, 1, 0), np.delete(clean, 1, 0))
    c.dx = dev_bf16(c.x)
    b = c.bits(64)
    b[5] = 0x7FC0
    got = moe_ref.bf16_value(c.run("relu", bias=b))
    assert np.isnan(got[:, 5]).all() and np.isfinite(np.delete(got, 5, 1)).all()


def test_no_residual_keeps_the_sign_of_zero():
    c = Case(2, 32, 128, 128, 8)
    c.dx.zero_()
    r = np.full((2, 32), 0x8000, np.uint16)
    assert np.all(c.run("none", scale=-1.0) == 0x8000)
    assert np.all(c.run("none", residual=r, scale=1.0) == 0x0000)  # 0 + -0


def test_bias_at_an_odd_address():
    import torch

    import w4a16_weight_only_gemm_amd as w4
    for M in (3, 200):
        c = Case(M, 100, 256, 128, 9)
        b = c.bits(101)
        d = dev_bf16(b)
        y = torch.empty((M, 100), dtype=torch.bfloat16, device="cuda")
        w4.w4a16_gemm_epilogue(c.dx, c.qw, c.sp, y, M, 100, 256, 128, bias=d[1:])
        assert np.array_equal(host_bits(y), c.run(bias=b[1:].copy()))


def test_far_rows():
    """Elements of x and y past 2^31: the first, last and border rows."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    N, K, M = 4128, 256, 1050000
    log("epilogue far rows")
    c = Case(1, N, K, 128, 10)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    y = torch.full((M, N // 2), 0.5, dtype=torch.bfloat16, device="cuda")
    assert y.numel() > 1 << 31
    w4.w4a16_gemm_epilogue(x, c.qw, c.sp, y, M, N, K, 128, residual=y, act=w4.W4A16_ACT_SWIGLU)
    border = (1 << 31) // (N // 2)
    at = torch.tensor([0, 1, border - 1, border, border + 1, M - 2, M - 1], device="cuda")
    ref, tol = layer_ref.epilogue(x[at].double().cpu().numpy(), c.q, c.s, 128, "swiglu",
                                  residual=np.full((7, N // 2), 0.5))
    moe_ref.check(host_bits(y[at]), ref, tol)


@pytest.mark.parametrize("M", [1, 16, 17, 32, 40])
def test_gated_weights_past_4_gb(M):
    """More weights than the tiles' 32-bit offsets reach, at the row counts whose form
    comes in no pairs and beside them. Columns repeat every 1024, and the up half begins
    in the middle of a repetition."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    K, part, group = 1024, 1024, 128
    N = (2 ** 33 // K // (2 * part) + 2) * 2 * part + part
    assert w4.w4a16_qweight_bytes(N, K) > 2 ** 32 and (N // 2) % part == part // 2
    c = Case(M, part, K, group, M)
    times = N // part
    qw, sp = c.qw.repeat(times), c.sp.repeat(times)
    y = torch.full((M + 1, N // 2), -3.0, dtype=torch.bfloat16, device="cuda")
    w4.w4a16_gemm_epilogue(c.dx, qw, sp, y[:M], M, N, K, group, act=w4.W4A16_ACT_SWIGLU)
    assert bool((y[M] == -3.0).all())
    up = (np.arange(part) + N // 2) % part
    ref, tol = layer_ref.epilogue(moe_ref.bf16_value(c.x), np.concatenate([c.q, c.q[up]]),
                                  np.concatenate([c.s, c.s[up]]), group, "swiglu")
    first = y[:M, :part].contiguous()
    moe_ref.check(host_bits(first), ref, tol, M)
    for i in range(1, N // 2 // part):  # every repetition has the first's bits
        assert torch.equal(y[:M, i * part:(i + 1) * part], first), i
