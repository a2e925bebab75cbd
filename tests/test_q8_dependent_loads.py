"""Loads of the 8-bit kernels that are launched as programmatic dependents (no GPU).

Such a kernel may be resident before the one that writes its inputs has ended. The non-coherent path
(__ldg, ld.global.nc, pointers marked const __restrict__) is for memory that is read-only for the
whole life of a kernel, so none of them may use it.
"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "qwen3_vl_decoder_b200", "csrc")
# launched in plain stream order: starts after everything before it has ended
PLAIN = {"q8_rows.cu": ("quantize_weight_kernel",)}


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_dependent_kernels_load_coherently():
    for name in ("attn_q8.cu", "linear_q8.cu", "q8_rows.cu", "q8.cuh"):
        text = _code(name)
        assert not re.search(r"__ldg\s*\(|ld\.global(\.\w+)*\.nc|__ldcs\s*\(", text), name
        for kernel in PLAIN.get(name, ()):
            assert re.search(kernel + r"<<<", text), kernel
            text = re.sub(kernel + r"\([^)]*\)", "", text)
        assert "__restrict__" not in text, name
