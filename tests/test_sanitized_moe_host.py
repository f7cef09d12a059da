"""Host code of the mixture-of-experts and W8A8 operators under AddressSanitizer
and UndefinedBehaviorSanitizer (CPU only): sizes, packing into buffers of the
exact size, and argument checks at the ends of their ranges, each returning
before any launch. Device code is built as usual."""
import os
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a16_weight_only_gemm_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
SOURCES = ["w4a16_moe_host.cpp", "w4a16_moe.hip", "w4a16_experts.hip", "w8a8.hip"]

DRIVER = textwrap.dedent(r'''
    import ctypes, sys
    import numpy as np
    sys.path.insert(0, ROOT)
    import w4a16_weight_only_gemm_amd as w4
    ref = ctypes.CDLL(w4.LIB_PATH, ctypes.RTLD_GLOBAL)   # the sizes of the packed 4-bit weights
    san = ctypes.CDLL(LIB)
    for name, (res, args) in w4.MOE_SIGNATURES.items():
        fn = getattr(san, name)
        fn.restype, fn.argtypes = res, args
    rng = np.random.default_rng(0)
    for (N, K) in [(1, 16), (15, 48), (16, 64), (17, 80), (33, 144), (40, 1040)]:
        q = rng.integers(-128, 128, (N, K)).astype(np.int8)
        nb = san.w8a8_qweight_bytes(N, K)
        out = np.zeros(nb, np.int8)
        assert san.w8a8_pack(q.ctypes.data, out.ctypes.data, N, K) == 0
        assert np.array_equal(out, w4.w8a8_pack(q))
    for N, K in [(-1, 16), (2**31 - 1, 2**31 - 16), (2**31 - 1, 24), (0, 0)]:
        assert san.w8a8_qweight_bytes(N, K) == w4.w8a8_qweight_bytes(N, K)
    for T in (0, 1, 8, 9, 1024, 1025, 4096, 4097, 8192, 8193, 1 << 26, 2**31 - 1, -1):
        for E in (0, 1, 256, 257, 1024, 1025):
            assert (san.w4a16_moe_route_workspace_bytes(T, E)
                    == w4.w4a16_moe_route_workspace_bytes(T, E))
    A, B, BIG = 1 << 20, (1 << 20) + 8, 2**31 - 1
    c = w4.w4a16_route_config(64, 4, 0, 0, 1, 1, 1, 1, 1.0)
    route = lambda T, ws, n: san.w4a16_moe_route(A, None, ctypes.addressof(c), T, A, A, A, A, ws, n, None)
    assert route(BIG, A, 1 << 50) == 2 and route(1 << 25, A, 1 << 50) == 2
    assert route(1000, None, 0) == 1 and route(1000, B, 1 << 50) == 3 and route(-1, A, 0) == 1
    ex = lambda slots, E, div, N, K, g, act: san.w4a16_gemm_experts(A, A, A, A, A, A, slots, E, div, N, K, g, act, None)
    for args in [(BIG, 1, 1, BIG, BIG - 127, 128, 0), (BIG, 1024, BIG, BIG, 128, 128, 0),
                 (1 << 30, 1024, BIG, 1 << 20, 128, 128, 0), (1 << 30, 1024, BIG, 1 << 20, 256, 256, 0)]:
        assert ex(*args) == 2, args     # too large for 32-bit buffers or one grid
    assert ex(1, 1, 0, 1, 32, 32, 0) == 1 and ex(0, 1, 1, 1, 32, 32, 0) == 0
    assert san.w4a16_moe_combine(A, A, A, None, A, BIG, 32, BIG, None) == 2
    assert san.w4a16_moe_combine(A, A, A, B, A, 1, 1, 1, None) == 3
    for M, N, K in [(BIG, BIG, 131072), (BIG, 1 << 20, 64), (1, BIG, 16), (1, 1, BIG - 15)]:
        assert san.w8a8_gemm(A, A, A, A, A, M, N, K, None) == 2, (M, N, K)
    print("SANITIZED_MOE_HOST_OK")
''')


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
def test_moe_host_under_sanitizers(tmp_path):
    lib = str(tmp_path / "libw4a16_moe_san.so")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC", "-shared",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-I", os.path.join(ROOT, "include"), *[os.path.join(CSRC, s) for s in SOURCES],
           "-Wl,-rpath,/opt/rocm/lib", "-o", lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    runtime = subprocess.run([HIPCC, "-print-file-name=libclang_rt.asan-x86_64.so"],
                             capture_output=True, text=True).stdout.strip()
    assert os.path.exists(runtime), runtime
    env = dict(os.environ, LD_PRELOAD=runtime,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    code = f"ROOT = {ROOT!r}\nLIB = {lib!r}\n" + DRIVER
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, timeout=600)
    assert r.returncode == 0 and "SANITIZED_MOE_HOST_OK" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
