"""Host code of include/w4a16_layer.h under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): workspace sizes and argument checks at the
ends of their ranges, each returning before any launch. Device code is built as
usual."""
import os
import subprocess
import sys
import textwrap
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a16_weight_only_gemm_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
SOURCES = ["w4a16_host.cpp", "w4a16_plain.hip", "w4a16_skinny.hip", "w4a16_large.hip", "w4a8.hip", "w4a16_probe.hip",
           "w4a16_layer_host.cpp", "w4a16_epilogue.hip", "w4a16_norm.hip", "w4a16_moe_layer.hip"]

DRIVER = textwrap.dedent(r'''
    import ctypes, itertools, sys
    sys.path.insert(0, ROOT)
    import w4a16_weight_only_gemm_amd as w4
    san = ctypes.CDLL(LIB)
    for name, (res, args) in w4.LAYER_SIGNATURES.items():
        fn = getattr(san, name)
        fn.restype, fn.argtypes = res, args
    A, B, BIG = 1 << 20, (1 << 20) + 8, 2**31 - 1
    for args in itertools.product((-1, 0, 1, 16, 17, BIG), (0, 1, 1024, 1025, BIG), (0, 1, 32, 33), (0, 1, BIG),
                                  (0, 1, BIG)):
        assert san.w4a16_moe_layer_workspace_bytes(*args) == w4.w4a16_moe_layer_workspace_bytes(*args), args
    e = w4.w4a16_epilogue(None, None, 1.0, 0)
    gemm = lambda M, N, K, g: san.w4a16_gemm_epilogue(A, A, A, ctypes.addressof(e), A, M, N, K, g, None)
    for act in range(7):
        e.act = act
        for M, N, K, g in [(65535 * 16, BIG - 31, 256, 256), (65535 * 16 + 1, 32, 256, 256), (BIG, BIG - 31, 128, 128),
                           (BIG, 64, BIG - 127, 128), (1, BIG - 31, BIG - 255, 256)]:
            assert gemm(M, N, K, g) in (2, 3), (act, M, N, K, g)
        assert gemm(0, BIG, BIG, 77) == 0 and gemm(1, BIG, BIG, 128) == 2 and gemm(-1, 1, 1, 1) == 1
    n = w4.w4a16_norm_args(y=A, gate_rows=1, scale=1.0, residual=A, residual_out=A, x=A, eps=0.0)
    norm = lambda T, N: san.w4a16_norm(ctypes.addressof(n), T, N, None)
    assert norm(BIG, 65536) == 2 and norm(BIG, 16384) == 2 and norm(1, 65537) == 2 and norm(0, BIG) == 0
    n.gate_rows = 0
    assert norm(1, 64) == 1
    r = w4.w4a16_route_config(1024, 32, 0, 0, 1, 1, 1, 1, 1.0)
    l = w4.w4a16_moe_layer_args(route=r, hidden=128, width=128, group=128, router=A, gate_up=A, gate_up_scales=A,
                                down=A, down_scales=A)
    layer = lambda T, ws, n: san.w4a16_moe_layer(ctypes.addressof(l), A, None, None, A, A, A, T, ws, n, None)
    assert layer(16, A, 0) == 1 and layer(BIG, A, 1 << 50) == 2 and layer(16, A + 64, 1 << 50) == 3
    for H, I in [(BIG - 127, 128), (128, BIG - 127), (BIG - 127, BIG - 127), (1 << 20, 1 << 20), (1 << 16, 1 << 16)]:
        l.hidden, l.width = H, I
        assert layer(16, B, 0) in (1, 2), (H, I)
    print("SANITIZED_LAYER_HOST_OK")
''')


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
def test_layer_host_under_sanitizers(tmp_path):
    lib = str(tmp_path / "libw4a16_layer_san.so")
    flags = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
             "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=undefined",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", os.path.join(ROOT, "include")]

    def compile_one(source):
        obj = str(tmp_path / (source + ".o"))
        r = subprocess.run([HIPCC, *flags, "-c", os.path.join(CSRC, source), "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        return obj
    with ThreadPoolExecutor(4) as pool:
        objects = list(pool.map(compile_one, SOURCES))
    r = subprocess.run([HIPCC, *flags, "-shared", *objects, "-Wl,-rpath,/opt/rocm/lib", "-o", lib],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    runtime = subprocess.run([HIPCC, "-print-file-name=libclang_rt.asan-x86_64.so"],
                             capture_output=True, text=True).stdout.strip()
    assert os.path.exists(runtime), runtime
    env = dict(os.environ, LD_PRELOAD=runtime,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    code = f"ROOT = {ROOT!r}\nLIB = {lib!r}\n" + DRIVER
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, timeout=600)
    assert r.returncode == 0 and "SANITIZED_LAYER_HOST_OK" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
