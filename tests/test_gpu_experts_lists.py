"""w4a16_gemm_experts on the GPU with offsets that do not ascend, so that the
lists overlap: every value of y is one of its experts' results or left as it was,
and nothing outside is touched. Results are told apart by the experts' scales:
all codes and activations are 1, so expert e gives K * scale[e]."""
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible to torch")
    import w4a16_weight_only_gemm_amd  # noqa: F401  (fails loudly if the library is missing)
    yield


def run(off, rows, slots, E, N, K, x_div):
    """Ones throughout; scale of expert e: e % 7 + 1. Returns y with 64 values behind it."""
    import torch

    import w4a16_weight_only_gemm_amd as w4
    blocks = (N + 15) // 16
    qw = torch.full((E, blocks, K // 32, 64), 0x11111111, dtype=torch.int32, device="cuda")
    sc = (torch.arange(E, device="cuda") % 7 + 1).to(torch.float16)
    sc = sc.view(E, 1, 1).expand(E, blocks, K // 32 * 16).contiguous()
    x = torch.ones((-(-slots // x_div), K), dtype=torch.bfloat16, device="cuda")
    y = torch.full((slots * N + 64,), -3.0, dtype=torch.bfloat16, device="cuda")
    w4.w4a16_gemm_experts(x, qw, sc, y, rows, torch.tensor(off, dtype=torch.int32).cuda(), slots, E,
                          x_div, N, K, 32)
    torch.cuda.synchronize()
    assert bool((y[slots * N:] == -3).all())
    return y[:slots * N].view(slots, N)


@pytest.mark.parametrize("slots", [5, 90, 700, 3000])
@pytest.mark.parametrize("E", [6, 130, 700])
def test_overlapping_lists(slots, E):
    import torch
    print("overlapping lists", slots, E, file=sys.stderr, flush=True)
    K = 64
    rng = np.random.default_rng(slots + E)
    rows = torch.arange(slots, dtype=torch.int32).cuda()
    zigzag = [slots if e % 2 else 0 for e in range(E + 1)]
    anyhow = rng.integers(-3, slots + 4, E + 1).tolist()
    falling = np.linspace(slots, 0, E + 1).astype(int).tolist()
    for off in (zigzag, anyhow, falling):
        y = run(off, rows, slots, E, 40, K, 1).float().cpu().numpy()
        edge = np.clip(off, 0, slots)
        may = np.zeros((slots, 8), bool)
        for e in range(E):
            may[edge[e]:edge[e + 1], e % 7 + 1] = True
        left = y == -3
        which = np.where(left, 0, y / K).astype(int)
        assert np.all(left | (which * K == y))
        assert np.all(left | np.take_along_axis(may, which, 1))
        if off is falling:
            assert left.all()


def test_more_listed_rows_than_an_int_counts():
    """512 experts that each list all of 2^27 slots: 2^31 row tiles of 32."""
    import torch
    slots, E, K = 1 << 27, 1024, 32
    rows = torch.arange(slots, dtype=torch.int32, device="cuda")
    y = run([slots if e % 2 else 0 for e in range(E + 1)], rows, slots, E, 1, K, 1 << 20)
    which = y.float() / K
    assert bool(((y == -3) | ((which >= 1) & (which <= 7) & (which == which.round()))).all())
