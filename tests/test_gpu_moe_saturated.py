"""w4a16_moe_route on the GPU where different logits have one score in 64 bits:
told apart by the logits without bias and groups, equal values (the lowest index
first) with either."""
import numpy as np
import pytest

import moe_ref
from test_gpu_moe_route import gpu, run_route  # noqa: F401  (gpu: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scoring,logits,by_logit,by_score", [
    ("sigmoid", [40, 41, 36, 60, 0, 38], [3, 1, 0, 5], [0, 1, 3, 5]),
    ("sigmoid", [-1, -746, -745.5, -800, -747, -900], [0, 2, 1, 4], [0, 1, 2, 3]),
    ("softmax", [-800, 0, -790, -1000, -795, -1], [1, 5, 2, 4], [1, 5, 0, 2])])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T", [1, 40])
def test_saturated_scores(scoring, logits, by_logit, by_score, bf16, T):
    z = np.float32([logits] * T)
    if bf16:
        z = moe_ref.bf16_value(moe_ref.bf16_bits(z)).astype(np.float32)
    for bias, groups, want in ((None, 1, by_logit), (np.zeros(6), 1, by_score), (None, 2, by_score)):
        got = run_route(z, bias, 4, bf16, scoring=scoring, groups=groups, groups_kept=groups)
        ref = moe_ref.route(z, bias, 4, scoring, groups, groups)
        assert np.array_equal(got[0], ref[0])
        if not bf16:
            assert got[0].tolist() == [want] * T
        assert np.all(np.abs(got[1] - ref[1]) <= 2 * moe_ref.F32 * np.abs(ref[1]) + 1e-45)
