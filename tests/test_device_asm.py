"""Inline assembly of the device sources (read as text, no GPU): every register
that a block names as written is in its clobber list, as the compiler knows of
no other."""
import glob
import os
import re

import w4a16_weight_only_gemm_amd as w4

CSRC = os.path.join(os.path.dirname(os.path.abspath(w4.__file__)), "csrc")


def blocks():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.h"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
            depth, end = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[end], 0)
                end += 1
            yield os.path.basename(path), text[m.end():end - 1]


def test_written_registers_are_clobbers():
    seen = 0
    for name, body in blocks():
        code, _, _, clobbers = body.split(":")  # template, outputs, inputs, clobbers
        written = set(re.findall(r"\bs_\w+ (m0|vcc|exec|s\d+)\b", code))
        seen += len(written)
        assert written <= set(re.findall(r'"([^"]+)"', clobbers)), (name, body)
    assert seen  # the copy to LDS sets m0
