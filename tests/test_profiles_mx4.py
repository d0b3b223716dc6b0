"""The captures of the 4-bit and distillation kernels are of the present sources: profiles/mx4_distill_kernels.md states
the hash of their code, without its comments and line breaks."""
import hashlib
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = ("zr_mx4_quant.cu", "zr_mx4_gemm.cu", "zr_distill.cu", "zr_mx4.cuh", "zr_tensor.cuh", "zr_device.cuh", "zr_launch.h")


def code_hash():
    h = hashlib.sha256()
    for name in SOURCES:
        text = open(os.path.join(ROOT, "zero_gradient_reduction_gb300", "csrc", name)).read()
        text = re.sub(r"/\*.*?\*/", " ", re.sub(r"//[^\n]*", "", text), flags=re.S)
        h.update(" ".join(text.split()).encode())
    return h.hexdigest()[:16]


def test_captures_are_of_the_present_code():
    text = open(os.path.join(ROOT, "profiles", "mx4_distill_kernels.md")).read()
    assert re.findall(r"code_sha256_16: `([0-9a-f]+)`", text) == [code_hash()], "retake the captures"
