"""w4a16_moe_route on the GPU where a group's two largest values nearly cancel:
each is rounded at its own size, so a sum says nothing about how far off it is.
Groups are made a little apart in 64 bits and have to be kept as there."""
import sys

import numpy as np
import pytest

import moe_ref
from test_gpu_moe_route import gpu, run_route  # noqa: F401  (gpu: the fixture)

pytestmark = pytest.mark.gpu


def check(z, bias, top_k, **kw):
    """Choices and lists as in 64 bits (bias: fp32 values)."""
    print("route", z.shape, top_k, kw, file=sys.stderr, flush=True)
    got = run_route(z, bias, top_k, **kw)
    ref = moe_ref.route(z, bias, top_k, **kw)
    assert np.array_equal(got[0], ref[0])
    assert np.array_equal(got[2], ref[2])
    assert np.array_equal(got[3], ref[3])
    assert np.all(np.abs(got[1] - ref[1]) <= 2 * moe_ref.F32 * np.abs(ref[1]) + 1e-45)


def test_two_groups_by_hand():
    """The sums are 0.94345218 and 0.94345937; rounded to fp32 at the size of 1000
    they are 0.94348145 and 0.94342040."""
    z = np.float32([[-1.0498050451, 0.7730932236, 1.4346925020, -1.8503828049]])
    b = np.float32([1000, -1000, 1000, -1000])
    s = 1.0 / (1.0 + np.exp(-z[0].astype(np.float64))) + b
    assert s[2] + s[3] > s[0] + s[1]
    got = run_route(z, b, 2, scoring="sigmoid", groups=2, groups_kept=1, group_top=2)
    assert got[0].tolist() == [[2, 3]]


def near_sums(rng, T, groups, per, scoring, apart):
    """Logits whose two first scores of every group sum to nearly the same
    (apart: the largest difference), the group's others small."""
    a = rng.uniform(0.2, 0.8, (T, groups))
    c = 1.0 + rng.uniform(-apart, apart, (T, groups)) / 2 - a
    s = np.full((T, groups, per), 0.05)
    s[:, :, 0], s[:, :, 1] = a, c
    z = np.log(s / (1 - s)) if scoring == "sigmoid" else np.log(s)
    return z.reshape(T, groups * per).astype(np.float32)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [30, 50, 100, 1000, 1e4, 1e5])
@pytest.mark.parametrize("groups,per", [(2, 2), (8, 2), (5, 3), (32, 2), (64, 4), (16, 64)])
def test_cancelling_biases(groups, per, size, scoring):
    """Biases of +size and -size in every group, the others below both; group
    sums as far apart as two such roundings to fp32."""
    rng = np.random.default_rng(groups * per + int(size))
    z = near_sums(rng, 60, groups, per, scoring, size * 4 * moe_ref.F32)
    b = np.full((groups, per), -3.0 * size)
    b[:, 0], b[:, 1] = size, -size
    kept = max(1, groups // 3)
    check(z, np.float32(b.reshape(-1)), min(8, 2 * kept), scoring=scoring, groups=groups,
          groups_kept=kept, group_top=2)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,per", [(6, 2), (5, 3), (16, 16)])
def test_groups_of_different_size(groups, per, scoring):
    """The same with another size in every group: the one whose sum is far off may
    be any, not only the last one kept or the first one dropped."""
    rng = np.random.default_rng(groups)
    z = near_sums(rng, 300, groups, per, scoring, 2e-3)
    size = 2.0 ** rng.integers(0, 15, groups)  # sums of +size and -size cancel exactly
    b = np.full((groups, per), -1e5)
    b[:, 0], b[:, 1] = size, -size
    for kept in (1, groups // 2, groups - 1):
        check(z, np.float32(b.reshape(-1)), 2, scoring=scoring, groups=groups, groups_kept=kept,
              group_top=2)
