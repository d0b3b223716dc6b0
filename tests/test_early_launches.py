"""Kernels that begin while the launch before them runs read what it writes, once they have waited for its end, by the
coherent path: the read-only one (ld.global.nc, __ldg) is defined only for memory that nothing writes between a launch's
beginning and its end, and the helpers that take it are not held behind the wait."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "zero_gradient_reduction_gb300", "csrc")
READ_ONLY = re.compile(r"\b(ld_once|ld_once_f4|load8|load16|__ldg)\b|ld\.global\.nc")


def kernels(text):
    """(name, body) of each __global__ function."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__", text):
        name = re.search(r"\b(\w+_kernel)\s*\(", text[m.end():])
        at = text.index("{", m.end() + name.end())
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        yield name.group(1), text[at:end]


def test_what_waits_reads_by_the_coherent_path():
    waiting = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "zr_*.cu"))):
        for name, body in kernels(open(path).read()):
            if "wait_for_previous" in body:
                waiting[name] = body
    # (few_kernel takes in tokens by that path in the form that does not begin early)
    assert {"column_kernel", "dequant_kernel", "gemm_kernel", "few_kernel", "logprob_kernel", "policy_kernel", "score_kernel", "pair_kernel",
            "gradient_kernel"} == set(waiting)
    assert not [name for name, body in waiting.items() if READ_ONLY.search(body)]
