"""The operators of a quantized mixture-of-experts layer run together, as a
decode or prefill step uses them: routing, the experts' gate and up products
with SwiGLU, their down products, a shared expert through w4a8_quantize and
w8a8_gemm, and the combine; eager, on a side stream, and captured into graphs
that are replayed between eager calls."""
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


class Layer:
    E, K, H, I, G = 12, 3, 256, 128, 64   # experts, per token, hidden, expert width, group
    GROUPS, KEPT, SCALE = 4, 2, 1.5

    def __init__(self, seed=0):
        import torch

        import w4a16_weight_only_gemm_amd as w4
        rng = np.random.default_rng(seed)
        E, H, I, G = self.E, self.H, self.I, self.G

        def pack(N, K):
            q = rng.integers(-8, 8, (E, N, K)).astype(np.int8)
            s = ((rng.random((E, N, K // G)) + 0.5) / (4 * np.sqrt(K))).astype(np.float16)
            p = [w4.w4a16_pack(q[e], s[e], G) for e in range(E)]
            return (q, s.astype(np.float64),
                    torch.from_numpy(np.concatenate([a for a, _ in p]).view(np.int32)).cuda(),
                    torch.from_numpy(np.concatenate([b for _, b in p]).view(np.int16)).cuda())
        self.up = pack(2 * I, H)
        self.down = pack(H, I)
        self.q8 = rng.integers(-127, 128, (H, H)).astype(np.int8)
        self.s8 = ((rng.random(H) + 0.5) / (70 * np.sqrt(H))).astype(np.float32)
        self.d8 = (torch.from_numpy(w4.w8a8_pack(self.q8)).cuda(), torch.from_numpy(self.s8).cuda())
        self.bias = (rng.standard_normal(E) * 0.05).astype(np.float32)
        self.dbias = torch.from_numpy(self.bias).cuda()

    def buffers(self, T):
        import torch

        import w4a16_weight_only_gemm_amd as w4
        bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")     # noqa: E731
        R = T * self.K
        return dict(T=T, x=bf(T, self.H), logits=torch.empty(T, self.E, device="cuda"), ids=i32(R),
                    w=torch.empty(R, device="cuda"), off=i32(self.E + 1), rows=i32(R),
                    ws=i32(max(1, w4.w4a16_moe_route_workspace_bytes(T, self.E) // 4)),
                    h=bf(R, self.I), y=bf(R, self.H), shared=bf(T, self.H), out=bf(T, self.H),
                    xq=torch.empty(T, self.H, dtype=torch.int8, device="cuda"),
                    sx=torch.empty(T, device="cuda"))

    def fill(self, b, seed):
        import torch
        rng = np.random.default_rng(seed)
        x = moe_ref.bf16_bits(rng.standard_normal((b["T"], self.H)).astype(np.float32))
        z = rng.standard_normal((b["T"], self.E)).astype(np.float32)
        if b["T"] > 4:
            z[-2:] = -np.inf  # padding tokens
        b["x"].view(torch.int16).copy_(torch.from_numpy(x.view(np.int16)))
        b["logits"].copy_(torch.from_numpy(z))
        b["h"].zero_()
        b["y"].zero_()
        return x, z

    def step(self, b):
        import w4a16_weight_only_gemm_amd as w4
        T, E, k, H, I, G = b["T"], self.E, self.K, self.H, self.I, self.G
        w4.w4a16_moe_route(b["logits"], self.dbias, T, E, k, b["ids"], b["w"], b["off"], b["rows"],
                           b["ws"], scoring=w4.W4A16_ROUTE_SIGMOID, groups=self.GROUPS,
                           groups_kept=self.KEPT, group_top=2, scale=self.SCALE)
        w4.w4a16_gemm_experts(b["x"], self.up[2], self.up[3], b["h"], b["rows"], b["off"], T * k, E,
                              k, 2 * I, H, G, act=w4.W4A16_ACT_SWIGLU)
        w4.w4a16_gemm_experts(b["h"], self.down[2], self.down[3], b["y"], b["rows"], b["off"],
                              T * k, E, 1, H, I, G)
        w4.w4a8_quantize(b["x"], b["xq"], b["sx"], T, H)
        w4.w8a8_gemm(b["xq"], b["sx"], self.d8[0], self.d8[1], b["shared"], T, H, H)
        w4.w4a16_moe_combine(b["y"], b["ids"], b["w"], b["shared"], b["out"], T, k, H)

    def reference(self, x, z):
        """Each stage in 64 bits with the bf16 roundings the stages hand on; returns
        (out, bound): the stages' bounds carried through the following ones."""
        import oracle
        ids, w, off, rows = moe_ref.route(z, self.bias, self.K, "sigmoid", self.GROUPS, self.KEPT,
                                          2, True, self.SCALE)
        xv = moe_ref.bf16_value(x)
        h, dh = moe_ref.experts(xv, self.up[0], self.up[1], rows, off, self.K, self.G, True)
        h, dh = np.nan_to_num(h), np.nan_to_num(dh)
        y, dy = moe_ref.experts(h, self.down[0], self.down[1], rows, off, 1, self.G)
        for e in range(self.E):  # the error of h through the down weights
            mine = rows[off[e]:off[e + 1]]
            wd = np.abs(self.down[0][e] * np.repeat(self.down[1][e], self.G, axis=1))
            dy[mine] += (dh[mine] @ wd.T) * (1 + moe_ref.BF16)
        y, dy = np.nan_to_num(y), np.nan_to_num(dy)
        codes, sx = oracle.quantize_rows(x)
        sh, dsh = moe_ref.w8a8(codes, sx, self.q8, self.s8)
        out, d = moe_ref.combine(y, ids, w, sh)
        T = ids.shape[0]
        d += (dsh + (np.abs(w)[:, :, None] * dy.reshape(T, self.K, -1)).sum(1)) * (1 + moe_ref.BF16)
        return out, d


def bits(t):
    import torch
    torch.cuda.synchronize()
    return t.view(torch.int16).cpu().numpy().view(np.uint16).copy()


@pytest.mark.parametrize("T", [1, 2, 31, 70, 900])
def test_layer(T):
    log("layer", T)
    layer = Layer()
    b = layer.buffers(T)
    x, z = layer.fill(b, T)
    layer.step(b)
    got = moe_ref.bf16_value(bits(b["out"]))
    ref, tol = layer.reference(x, z)
    assert np.all(np.abs(got - ref) <= tol)
    # four bf16 roundings in a row at most reach any result (h, y or shared, out)
    assert np.linalg.norm(got - ref) <= 3 * moe_ref.BF16 * np.linalg.norm(ref)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_captured_layers(T):
    """Two graphs of the layer, one workspace each, replayed in turn between eager
    steps on other inputs: every replay gives the eager bits of its inputs."""
    import torch
    layer = Layer(1)
    bufs = [layer.buffers(T) for _ in range(2)]
    eager = layer.buffers(T)
    graphs = []
    for b in bufs:
        layer.fill(b, 1)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer.step(b)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.step(b)
        graphs.append(g)
    for turn in range(3):
        for i, (b, g) in enumerate(zip(bufs, graphs)):
            seed = 10 + 2 * turn + i
            layer.fill(eager, seed)
            layer.step(eager)
            want = bits(eager["out"])
            layer.fill(b, seed)
            b["out"].fill_(float("nan"))
            g.replay()
            assert np.array_equal(bits(b["out"]), want), (turn, i)


def test_two_streams_at_once():
    import torch
    layer = Layer(2)
    bufs = [layer.buffers(100) for _ in range(2)]
    want = []
    for i, b in enumerate(bufs):
        layer.fill(b, 50 + i)
        layer.step(b)
        want.append(bits(b["out"]))
        b["out"].fill_(float("nan"))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s in zip(bufs, streams):
            with torch.cuda.stream(s):
                layer.step(b)
    torch.cuda.synchronize()
    for b, w in zip(bufs, want):
        assert np.array_equal(bits(b["out"]), w)
