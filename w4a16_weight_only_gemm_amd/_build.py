"""In-tree build of the HIP library libw4a16.so for gfx950 (hipcc, no JIT)."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libw4a16.so")
SOURCES = ["w4a16_host.cpp", "w4a16_plain.hip", "w4a16_skinny.hip", "w4a16_large.hip", "w4a8.hip",
           "w4a16_probe.hip", "w4a16_noalloc.hip", "w4a16_moe_host.cpp", "w4a16_moe.hip",
           "w4a16_experts.hip", "w8a8.hip", "w4a16_layer_host.cpp", "w4a16_epilogue.hip",
           "w4a16_norm.hip", "w4a16_moe_layer.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall", "-Werror=return-type",
         # no packed-fp32 VALU forms anywhere in the device code
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(ROOT, "include")]


def _run(cmd: list[str]) -> None:
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + proc.stdout + proc.stderr)


def build() -> str:
    """Compile every source (side by side) and link the library."""
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as d:
        objects = [os.path.join(d, s + ".o") for s in SOURCES]
        with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(lambda so: _run([HIPCC, *FLAGS, "-c", os.path.join(CSRC, so[0]), "-o", so[1]]),
                          zip(SOURCES, objects)))
        _run([HIPCC, "--offload-arch=gfx950", "-shared", *objects, "-Wl,-rpath,/opt/rocm/lib", "-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build())
