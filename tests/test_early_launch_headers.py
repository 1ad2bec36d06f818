"""As test_early_launch_loads, for kernels whose early launch stands in a header that they
include: every source that launches early or waits by such a helper, and every header
that has one, reads through the coherent path alone."""
import glob
import os
import re

import pytest

from mixture_experts_layer_11_gb300 import build as mbuild
from test_early_launch_loads import code_of

FORMS = (r"ld\.global\.nc", r"\b__ldg\s*\(", r"\b__restrict__\b")
SOURCES = sorted(glob.glob(os.path.join(mbuild.CSRC, "*.cu")) + glob.glob(os.path.join(mbuild.CSRC, "*.h"))
                 + glob.glob(os.path.join(mbuild.CSRC, "*.cuh")))
EARLY = re.compile(r"griddepcontrol|\bwait_front\s*\(|\blaunch_early\s*\(|ProgrammaticStreamSerialization")


def included(path, seen=()):
    """path and what it includes of the same folder, at any depth."""
    if path in seen:
        return set(seen)
    seen = set(seen) | {path}
    for name in re.findall(r'#include\s+"([^"]+)"', open(path).read()):
        near = os.path.join(os.path.dirname(path), name)
        if os.path.exists(near):
            seen |= included(near, tuple(seen))
    return seen


# sources that have or include an early launch (a header's helpers, unused, do no harm)
FILES = [p for p in SOURCES if EARLY.search(code_of(p))]


def test_the_files_that_launch_early_are_known():
    names = {os.path.basename(p) for p in FILES}
    assert {"few.cu", "grads.cu", "head.h", "head.cu", "head_simt.cu", "head_tc.cu"} <= names


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_early_kernels_and_their_headers_read_coherently(path):
    for part in included(path):
        for form in FORMS:
            assert re.search(form, code_of(part)) is None, (part, form)


def test_every_early_kernel_waits():
    # a kernel of these files that is launched early calls the wait (or has it inline)
    seen = set()
    for path in FILES:
        text = code_of(path)
        launched = set(re.findall(r"launch_early\(\s*(?:\w+ \? )?(\w+_kernel)\b", text))
        for kernel in launched:
            at = re.search(r"__global__[^;{]*?\b%s\s*\([^{]*\)\s*\{" % kernel, text, flags=re.S)
            if at is None:
                continue   # of another file
            seen.add(kernel)
            body = text[at.end():]
            depth, i = 1, 0
            while depth and i < len(body):
                depth += {"{": 1, "}": -1}.get(body[i], 0)
                i += 1
            assert "wait_front()" in body[:i] or "griddepcontrol.wait" in body[:i], kernel
    assert {"head_scan_kernel", "head_gather_kernel", "head_loss_kernel", "head_gradient_kernel", "head_entries_kernel",
            "head_round_kernel", "head_simt_z_kernel", "head_simt_grad_kernel", "head_simt_cluster_kernel",
            "head_simt_join_kernel", "head_tc_kernel", "head_join_kernel"} <= seen
