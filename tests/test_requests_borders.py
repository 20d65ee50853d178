"""Adapters, probabilities and verification where one path ends and the next begins: what needs no GPU."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import requests_oracle_np as orc


@pytest.mark.parametrize("u,taken", [(1.0, True), (2.0, True), (np.inf, True), (0.5, True), (np.nan, True), (-1.0, True)])
def test_oracle_holds_random_numbers_below_one(u, taken):
    """A token as likely in the target as in the draft is accepted whatever the number is: below 1 they all are."""
    p = np.float32([[0.25, 0.75], [0, 1]])
    tokens, accepted = orc.verify(p, p[:1], np.int32([0]), np.int32([0, 1]), np.float32([u]), np.float32([u]))
    assert accepted[0] == taken and list(tokens) == [0, 1]


CLUSTERS_HELD = r"""
#include <cuda_runtime.h>
#include <stdio.h>
static cudaError_t answer = cudaSuccess, last = cudaSuccess;  // the runtime's last error, which a machine without a GPU never clears
template <typename... Args>
static cudaError_t fake_occupancy(int* n, Args...) {
  *n = 19;
  return last = answer;
}
static cudaError_t fake_last_error() {
  const cudaError_t e = last;
  last = cudaSuccess;
  return e;
}
#define cudaOccupancyMaxActiveClusters fake_occupancy
#define cudaGetLastError fake_last_error
#include "mnb_internal.h"
__global__ void kernel() {}
int main() {
  static std::atomic<int> known[64];
  mnb::LaunchCtx ctx = {};
  answer = cudaErrorInvalidValue;
  int n = mnb::clusters_held(ctx, kernel, 8, 128, 0, known);
  printf("%d %d ", n, (int)last);
  answer = cudaSuccess;
  n = mnb::clusters_held(ctx, kernel, 8, 128, 0, known);
  answer = cudaErrorInvalidValue;  // not asked any more
  printf("%d %d\n", n, mnb::clusters_held(ctx, kernel, 8, 128, 0, known));
  return 0;
}
"""


def test_unknown_occupancy_leaves_no_error(tmp_path):
    """A GPU that can't say how many clusters it holds: 0, no error for the launch that follows, and asked again."""
    import os
    import subprocess

    from gemm_mnb_gemv_gb300 import _build
    try:
        nvcc = _build._nvcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    src, exe = tmp_path / "held.cu", tmp_path / "held"
    src.write_text(CLUSTERS_HELD)
    made = subprocess.run([nvcc, *_build.ARCH, "-std=c++17", "-I", os.path.join(_build.ROOT, "include"), "-I", _build.CSRC, str(src), "-o",
                           str(exe), "-cudart", "static"], capture_output=True, text=True)
    assert made.returncode == 0, made.stderr
    ran = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert ran.stdout.split() == ["0", "0", "19", "19"], ran.stdout + ran.stderr


def test_arguments_that_are_no_tensors_are_named():
    import torch

    import gemm_mnb_gemv_gb300 as mnb
    for pool in ((1, 2), None, torch.zeros(1)):
        with pytest.raises(TypeError, match="pool must be an MnbLoraPool"):
            mnb.mnb_lora(None, pool, None)
    for wrong in ([0, 1], (0.5,), 3, "x", None, np.zeros(2, np.float32), torch.zeros(2)):
        with pytest.raises(TypeError, match="temperature must be a CUDA tensor"):
            mnb._vector("temperature", wrong, torch.float32, (2,), None)
        with pytest.raises(TypeError, match="base must be a CUDA tensor"):
            mnb._matrix("base", wrong, (2, 1), torch.float32, None)
