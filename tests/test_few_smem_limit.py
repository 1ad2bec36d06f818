"""The shared-memory limit of few_experts_kernel is a setting of each device: the
first launch on a device sets it there, later ones do not, and a failure is not
remembered.  The function is taken from few.cu as it stands and compiled for the
host with a stand-in for the runtime."""
import os
import re
import shutil
import subprocess

import pytest

from mixture_experts_layer_11_gb300 import build as mbuild

HARNESS = r"""
#include <cstdio>
#include <mutex>
enum cudaError_t { cudaSuccess, cudaErrorInvalidDevice, cudaErrorOther };
enum { cudaFuncAttributeMaxDynamicSharedMemorySize };
struct cudaFuncAttributes { size_t sharedSizeBytes; };
int current, set_on[3], fail;
template <typename T> void few_experts_kernel() {}
cudaError_t cudaGetDevice(int* d) { *d = current; return cudaSuccess; }
template <typename F> cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, F) {
    a->sharedSizeBytes = 16384;
    return cudaSuccess;
}
template <typename F> cudaError_t cudaFuncSetAttribute(F, int, int) {
    if (fail) return cudaErrorOther;
    ++set_on[current];
    return cudaSuccess;
}
constexpr int kFewSmem = 227 * 1024;
%s
int main() {
    int n = 0, bad = 0;
    fail = 1;
    bad += few_smem_limit<float>(&n) == cudaSuccess;
    fail = 0;
    for (int turn = 0; turn < 2; ++turn)
        for (current = 0; current < 3; ++current)
            bad += few_smem_limit<float>(&n) != cudaSuccess || n != kFewSmem - 16384 || set_on[current] != 1;
    return bad;
}
"""


def test_limit_is_set_on_every_device(tmp_path):
    with open(os.path.join(mbuild.CSRC, "few.cu")) as fh:
        body = re.search(r"^template <typename T> cudaError_t few_smem_limit\(.*?^\}", fh.read(),
                         re.M | re.S).group(0)
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "limit.cc", str(tmp_path / "limit")
    src.write_text(HARNESS % body)
    r = subprocess.run([cxx, "-std=c++17", "-w", str(src), "-o", exe, "-pthread"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[:3000]
    assert subprocess.run([exe], timeout=60).returncode == 0
