"""Sizes at the ends of what include/w4a16_moe.h supports: refused before any
launch (the addresses are never used)."""
import w4a16_weight_only_gemm_amd as w4

A = 1 << 20
UNSUPPORTED = 2


def test_w8a8_grid_of_few_rows_form():
    """The few-rows form of many columns: more than 2^32 threads."""
    N, K = 40_000_000, 16
    assert w4.w8a8_qweight_bytes(N, K) < 1 << 32
    assert w4.w8a8_gemm_status(A, A, A, A, A, 512, N, K) == UNSUPPORTED


def test_combine_columns():
    """8 columns a thread: the last few below 2^31 have no whole piece in an int."""
    for N in range((1 << 31) - 7, 1 << 31):
        assert w4.moe_combine_status(A, A, A, None, A, 1, 1, N) == UNSUPPORTED, N
