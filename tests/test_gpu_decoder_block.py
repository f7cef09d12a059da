"""The operators of include/w4a16_layer.h run together as a decode step uses them: a
norm into a dense block (product with bias, product with SwiGLU, product onto the
residual stream), a norm with a post norm into a whole expert layer, and a last norm as
codes into w8a8_gemm; eager, captured into graphs that are replayed between eager
calls, and on two streams at once."""
import sys

import numpy as np
import pytest

import layer_ref
import moe_ref
from test_gpu_epilogue import Case
from test_gpu_experts import gpu, host_bits  # noqa: F401  (gpu: the fixture)
from test_gpu_moe_whole import Whole

pytestmark = pytest.mark.gpu


def log(*a):
    print(*a, file=sys.stderr, flush=True)


class Block:
    H, F, G = 256, 384, 128
    E, K, I = 12, 3, 128

    def __init__(self, seed=0):
        import torch

        import w4a16_weight_only_gemm_amd as w4
        rng = np.random.default_rng(seed)
        self.qkv = Case(1, self.H, self.H, self.G, seed + 1)
        self.up = Case(1, 2 * self.F, self.H, self.G, seed + 2)
        self.down = Case(1, self.H, self.F, self.G, seed + 3)
        self.moe = Whole(self.E, self.H, self.I, self.G, seed + 4, half=False)
        self.bits = {n: moe_ref.bf16_bits((rng.standard_normal(self.H) * 0.2 + 1).astype(np.float32))
                     for n in ("n1", "n2", "p2", "n3")}
        self.bits["bias"] = moe_ref.bf16_bits((rng.standard_normal(self.H) * 0.3).astype(np.float32))
        dev = lambda b: torch.from_numpy(b.view(np.int16)).cuda().view(torch.bfloat16)  # noqa: E731
        self.dev = {n: dev(b) for n, b in self.bits.items()}
        self.q8 = rng.integers(-127, 128, (self.H, self.H)).astype(np.int8)
        self.s8 = ((rng.random(self.H) + 0.5) / (70 * np.sqrt(self.H))).astype(np.float32)
        self.d8 = (torch.from_numpy(w4.w8a8_pack(self.q8)).cuda(), torch.from_numpy(self.s8).cuda())

    def buffers(self, T):
        import torch
        bf = lambda n: torch.empty((T, n), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        b = self.moe.buffers(T, self.K)
        b.update(res=torch.empty((T, self.H), device="cuda"), res2=torch.empty((T, self.H), device="cuda"),
                 a=bf(self.H), v=bf(self.H), h=bf(self.F), y=bf(self.H), y8=bf(self.H),
                 xq=torch.empty((T, self.H), dtype=torch.int8, device="cuda"), sx=torch.empty(T, device="cuda"))
        return b

    def fill(self, b, seed):
        import torch
        r = np.random.default_rng(seed).standard_normal((b["T"], self.H)).astype(np.float32)
        b["res"].copy_(torch.from_numpy(r))
        b["ws"].fill_(seed % 256)
        return r

    def step(self, b):
        import w4a16_weight_only_gemm_amd as w4
        T, H, F, G, d = b["T"], self.H, self.F, self.G, self.dev
        w4.w4a16_norm(T, H, residual=b["res"], weight=d["n1"], x=b["a"])
        w4.w4a16_gemm_epilogue(b["a"], self.qkv.qw, self.qkv.sp, b["v"], T, H, H, G, bias=d["bias"],
                               act=w4.W4A16_ACT_GELU_TANH)
        w4.w4a16_gemm_epilogue(b["v"], self.up.qw, self.up.sp, b["h"], T, 2 * F, H, G,
                               act=w4.W4A16_ACT_SWIGLU)
        w4.w4a16_gemm_epilogue(b["h"], self.down.qw, self.down.sp, b["y"], T, H, F, G,
                               residual=b["a"], scale=0.5)
        w4.w4a16_norm(T, H, y=b["y"], post_norm=True, post_weight=d["p2"], residual=b["res"],
                      residual_out=b["res2"], weight=d["n2"], x=b["x"])
        self.moe.call(b, use_base=False, use_live=False)
        w4.w4a16_norm(T, H, y=b["out"][:T], residual=b["res2"], residual_out=b["res2"], weight=d["n3"],
                      xq=b["xq"], sx=b["sx"], scale=0.5)
        w4.w8a8_gemm(b["xq"], b["sx"], self.d8[0], self.d8[1], b["y8"], T, H, H)

    def outputs(self, b):
        return [host_bits(b[n]).copy() for n in ("a", "v", "h", "y", "x")] + \
               [host_bits(b["out"])[:b["T"]].copy(), b["ids"].cpu().numpy(), b["w"].cpu().numpy(),
                b["res2"].cpu().numpy(), b["xq"].cpu().numpy(), b["sx"].cpu().numpy(), host_bits(b["y8"]).copy()]


def test_against_64_bits():
    """Every stage in 64 bits from the stage before as the device holds it."""
    for T in (1, 5, 16):
        log("block", T)
        blk = Block()
        b = blk.buffers(T)
        r = blk.fill(b, T).astype(np.float64)
        blk.step(b)
        a, v, h, y, x, out, ids, w, res2, xq, sx, y8 = blk.outputs(b)
        val = moe_ref.bf16_value
        one = moe_ref.BF16

        def near(got, pair):
            ref, d = pair
            moe_ref.check(got, ref, d + one * (np.abs(ref) + d))
        near(a, layer_ref.norm(residual=r, weight=val(blk.bits["n1"]))[1])
        c = blk.qkv
        moe_ref.check(v, *layer_ref.epilogue(val(a), c.q, c.s, 128, "gelu_tanh", val(blk.bits["bias"])))
        moe_ref.check(h, *layer_ref.epilogue(val(v), blk.up.q, blk.up.s, 128, "swiglu"))
        moe_ref.check(y, *layer_ref.epilogue(val(h), blk.down.q, blk.down.s, 128, residual=val(a), scale=0.5))
        (r2, dr2), nx = layer_ref.norm(val(y), r, post=True, post_weight=val(blk.bits["p2"]),
                                       weight=val(blk.bits["n2"]))
        near(x, nx)
        live = np.ones(T, np.int32)
        rid, rw, ro, ro_tol = blk.moe.reference(x, None, live, blk.K)
        assert np.array_equal(ids, rid)
        assert np.all(np.abs(val(out) - ro) <= ro_tol)
        # res2 was written twice; dr2 is its first rounding, once more carried through the sum
        r3 = r2 + 0.5 * val(out)
        d3 = dr2 + 3 * moe_ref.F32 * (np.abs(r3) + np.abs(0.5 * val(out)) + dr2)
        assert np.all(np.abs(res2 - r3) <= d3)
        nv, dnv = layer_ref._normalise(r3, d3, "rms", 1e-6, val(blk.bits["n3"]), None, False)
        q = layer_ref.natural(xq)
        assert layer_ref.codes(q.astype(np.float64), sx.astype(np.float64), nv, dnv)
        moe_ref.check(y8, *moe_ref.w8a8(q, sx, blk.q8, blk.s8))


@pytest.mark.parametrize("T", [1, 7, 16])
def test_captured(T):
    """Two graphs that share one set of weights, and one workspace, replayed in turn
    between eager steps on other inputs: every replay gives the eager bits."""
    import torch
    blk = Block(1)
    bufs = [blk.buffers(T) for _ in range(2)]
    bufs[1]["ws"] = bufs[0]["ws"]  # one after the other on one stream
    eager = blk.buffers(T)
    graphs = []
    for b in bufs:
        blk.fill(b, 1)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            blk.step(b)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            blk.step(b)
        graphs.append(g)
    for turn in range(4):
        for i, (b, g) in enumerate(zip(bufs, graphs)):
            seed = 10 + 2 * turn + i
            blk.fill(eager, seed)
            blk.step(eager)
            want = blk.outputs(eager)
            blk.fill(b, seed)
            b["out"].fill_(float("nan"))
            b["ids"].fill_(-9)
            g.replay()
            assert all(np.array_equal(p, q) for p, q in zip(blk.outputs(b), want)), (turn, i)


def test_two_streams_at_once():
    import torch
    blk = Block(2)
    bufs = [blk.buffers(16) for _ in range(2)]
    want = []
    for i, b in enumerate(bufs):
        blk.fill(b, 50 + i)
        blk.step(b)
        want.append(blk.outputs(b))
        b["out"].fill_(float("nan"))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, s in zip(bufs, streams):
            with torch.cuda.stream(s):
                blk.step(b)
    torch.cuda.synchronize()
    for b, w in zip(bufs, want):
        assert all(np.array_equal(p, q) for p, q in zip(blk.outputs(b), w))
