"""Kernels that are launched early (their blocks may begin before the kernel in
front of them in the stream has ended) must not read through the non-coherent
path: its data may not change while a kernel runs, and that kernel may still
write it.  Shown on the source: such files use neither ld.global.nc nor __ldg
nor pointers that allow the compiler to choose that path."""
import glob
import os
import re

import pytest

from mixture_experts_layer_11_gb300 import build as mbuild

FILES = sorted(p for p in glob.glob(os.path.join(mbuild.CSRC, "*.cu"))
               if "griddepcontrol" in open(p).read())


def code_of(path):
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    return re.sub(r"//[^\n]*", " ", text)


def test_some_files_launch_early():
    assert {"few.cu", "grads.cu"} <= {os.path.basename(p) for p in FILES}


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
@pytest.mark.parametrize("form", [r"ld\.global\.nc", r"\b__ldg\s*\(", r"\b__restrict__\b"])
def test_early_kernels_read_coherently(path, form):
    assert re.search(form, code_of(path)) is None
