"""Host-only tests of include/w4a16_layer.h, fields whose value does not matter or is past
the C type: each call returns before any launch."""
import pytest

import w4a16_weight_only_gemm_amd as w4
from test_layer_host import A, B, INVALID, MISALIGNED, ODD, UNSUPPORTED, norm

NONE = dict(y=None, gate=B, post_weight=ODD, post_bias=ODD, gate_rows=0, post_norm=1, scale=float("nan"))
FAR = (2**31 - 1, 65536)  # a grid past 2^32 threads: refused behind the checks of addresses


def test_a_block_that_is_not_there_counts_for_nothing():
    assert w4.norm_status(norm(**NONE), *FAR) == UNSUPPORTED
    for name in ("gate", "post_weight", "post_bias"):
        assert w4.norm_status(norm(y=None, **{name: NONE[name]}), *FAR) == UNSUPPORTED, name
        assert w4.norm_status(norm(**{name: NONE[name]}), *FAR) == MISALIGNED, name


# the first double that is rounded to infinity, and doubles far past it
@pytest.mark.parametrize("v", [2.0**128 - 2.0**103, 1e39, 1e308])
def test_numbers_past_fp32_are_refused_by_the_library(v):
    calls = [lambda s: w4.w4a16_gemm_epilogue(A, A, A, A, 1, 64, 256, 128, scale=s, stream=1),
             lambda s: w4.w4a16_norm(1, 64, y=A, x=A, scale=s, stream=1),
             lambda s: w4.w4a16_norm(1, 64, y=A, x=A, eps=s, stream=1),
             lambda s: w4.w4a16_moe_layer(A, A, A, A, A, A, A, A, A, 1, 16, 4, 256, 128, 128, A, scale=s,
                                          router_type=0, workspace_bytes=1 << 40, stream=1)]
    for call in calls:
        for s in (v, -v):
            with pytest.raises(w4.W4A16Error) as e:
                call(s)
            assert e.value.status == INVALID
