"""Calls of the layer operators beside those of their own files: x of more than 4 GB,
scores that vanish, the same bits whatever runs beside."""
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


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_epilogue_activations_over_4gb(act):
    """The tiles in two launches, the first of 65,408 rows, onto a residual in place."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    M, part, times, K, group = 65600, 512, 8, 32768, 128
    N = part * times
    assert 2 * M * K > 1 << 32 and w4.w4a16_select_form(M, N, K, group)[0] == w4.W4A16_PATH_LARGE
    log("epilogue x over 4 GB", act)
    c = Case(1, part, K, group, 12)
    qw, sp = c.qw.repeat(times), c.sp.repeat(times)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    for r in range(0, M, 1 << 14):
        n = min(1 << 14, M - r)
        x[r:r + n] = torch.randn((n, K), generator=g, device="cuda")
    out = N // 2 if act == "swiglu" else N  # a gate and its up are equal columns
    y = torch.randn((M + 1, out), generator=g, device="cuda").to(torch.bfloat16)
    rows = torch.tensor([0, 1, 65407, 65408, 65409, M - 1], device="cuda")
    before, guard = y[rows].double().cpu().numpy(), y[M].clone()
    w4.w4a16_gemm_epilogue(x, qw, sp, y[:M], M, N, K, group, residual=y[:M], scale=0.5,
                           act=getattr(w4, "W4A16_ACT_" + act.upper()))
    assert torch.equal(y[M], guard)
    many = 2 if act == "swiglu" else 1
    for i in range(0, out, part):
        ref, tol = layer_ref.epilogue(x[rows].double().cpu().numpy(), np.concatenate([c.q] * many),
                                      np.concatenate([c.s] * many), group, act, None, before[:, i:i + part], 0.5)
        moe_ref.check(host_bits(y[rows][:, i:i + part]), ref, tol, (act, i))


@pytest.mark.parametrize("E", [8, 72, 136, 300])
@pytest.mark.parametrize("T", [1, 2, 5, 16])
def test_sums_of_scores_that_vanish(T, E):
    """Chosen scores of 0 (sigmoids of logits below -750; a softmax whose choice, by bias and
    group, lies 800 below the largest logit): weights 0 with and without renormalising, out
    is base."""
    log("moe vanishing scores", T, E)
    w = Whole(E, 64, 32, 32, E, half=False)
    b = w.buffers(T, 3)
    _, base, _ = w.fill(b, 3)
    b["x"].fill_(1.0)
    low = np.zeros((E, 64), np.float32)
    low[:, 0] = -800.0 - np.arange(E)
    w.set_router(low)
    for renormalize in (True, False):
        b["ids"].fill_(-77)
        w.call(b, scoring="sigmoid", renormalize=renormalize)
        assert np.array_equal(host_bits(b["out"])[:T], base)
        assert b["ids"].cpu().tolist() == [[0, 1, 2]] * T and bool((b["w"] == 0).all())
    import torch
    half = E // 2
    low[:] = 0.0
    low[half:, 0] = -800.0
    w.set_router(low)
    w.bias = np.where(np.arange(E) >= half, 10.0, 0.0).astype(np.float32)
    w.dbias = torch.from_numpy(w.bias).cuda()
    for renormalize in (True, False):
        b["ids"].fill_(-77)
        w.call(b, groups=2, groups_kept=1, group_top=2, renormalize=renormalize)
        assert np.array_equal(host_bits(b["out"])[:T], base)
        assert b["ids"].cpu().tolist() == [[half, half + 1, half + 2]] * T and bool((b["w"] == 0).all())


def test_same_bits_beside_other_work():
    """Each operator's bits while another stream keeps the card busy, against those alone."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    w = Whole(16, 1280, 384, 128, 7)
    bufs = [w.buffers(T, 4) for T in (1, 7, 16)]
    for i, b in enumerate(bufs):
        w.fill(b, i)
    products = []
    for M, act in ((1, "none"), (16, "swiglu"), (50, "gelu"), (300, "swiglu")):
        c = Case(M, 1056, 768, 128, M)
        out = torch.empty((M, 528 if act == "swiglu" else 1056), dtype=torch.bfloat16, device="cuda")
        products.append((c, getattr(w4, "W4A16_ACT_" + act.upper()), out))
    y, r = (torch.randn(500, 2741, device="cuda").to(torch.bfloat16) for _ in range(2))
    x, ro = torch.empty_like(y), torch.empty_like(y)

    def outputs():
        out = []
        for b in bufs:
            w.call(b)
            out.append(b["out"].clone())
        for c, act, to in products:
            w4.w4a16_gemm_epilogue(c.dx, c.qw, c.sp, to, c.M, c.N, c.K, c.group, act=act)
            out.append(to.clone())
        w4.w4a16_norm(500, 2741, y=y, residual=r, residual_out=ro, x=x, post_norm=True, kind=w4.W4A16_NORM_LAYER)
        return out + [ro.clone(), x.clone()]
    want = outputs()
    a = torch.randn(4096, 4096, device="cuda").to(torch.bfloat16)
    busy, mine = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        with torch.cuda.stream(busy):
            for _ in range(30):
                torch.mm(a, a)
        with torch.cuda.stream(mine):
            got = [outputs() for _ in range(5)]
        torch.cuda.synchronize()
        for outs in got:
            for p, q in zip(outs, want):
                assert torch.equal(p.view(torch.int16), q.view(torch.int16))
