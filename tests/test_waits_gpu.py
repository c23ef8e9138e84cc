"""The bounded waits of the kernels: one that nothing ends runs out, and the others then do not wait."""
import ctypes
import os
import subprocess

import pytest
import torch

from host_offload_serving_gb300 import _build

pytestmark = pytest.mark.gpu

# Three barriers of one arrival each; only the third gets it.  Two warps wait on the first and the
# second.  out: 1 where a wait returned that its phase came, and the microseconds it took.
SOURCE = r"""
#include "waits.cuh"
__global__ void wait_kernel(int *out) {
  __shared__ uint64_t bars[3];
  __shared__ int fail;
  const uint32_t bar = smem_u32(bars);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 3; ++i) bar_init(bar + 8 * i, 1);
    fail = 0;
  }
  __syncthreads();
  if (threadIdx.x == 0) bar_arrive(bar + 16);
  const int warp = threadIdx.x >> 5;
  bool came[3];
  long long at[4] = {clock64()};
  came[0] = bar_wait(bar + 16, 0, &fail);
  at[1] = clock64();
  came[1] = bar_wait(bar + 8 * warp, 0, &fail);
  at[2] = clock64();
  came[2] = bar_wait(bar + 8 * (1 - warp), 0, &fail);
  at[3] = clock64();
  if ((threadIdx.x & 31) == 0)
    for (int i = 0; i < 3; ++i) {
      out[warp * 6 + 2 * i] = came[i];
      out[warp * 6 + 2 * i + 1] = static_cast<int>((at[i + 1] - at[i]) >> 10);
    }
  __syncthreads();
  if (threadIdx.x == 0) out[12] = fail;
}
extern "C" int run(int *out, void *stream) {
  wait_kernel<<<1, 64, 0, static_cast<cudaStream_t>(stream)>>>(out);
  return cudaGetLastError();
}
"""


def test_a_wait_that_nothing_ends_runs_out(tmp_path):
    src, lib = tmp_path / "wait.cu", tmp_path / "wait.so"
    src.write_text(SOURCE)
    subprocess.check_call([_build.nvcc(), *_build.ARCH, "-std=c++17", "-O3", "-shared", "-Xcompiler", "-fPIC", "-I",
                           _build.CSRC, "-I", os.path.join(_build.ROOT, "include"), "-o", str(lib), str(src)])
    out = torch.full((13,), -1, dtype=torch.int32, device="cuda")
    run = ctypes.CDLL(str(lib)).run
    run.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    assert run(out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    got = out.tolist()
    assert got[12] == 1                                   # the flag, once for all
    for w in (0, 1):
        came, took = got[6 * w:6 * w + 6:2], got[6 * w + 1:6 * w + 6:2]
        assert came == [1, 0, 0]
        assert took[0] < 2 ** 10                          # (in 1024 cycles) at once
        assert took[1] < 2 ** 21                          # at the limit of 2^30 cycles, within twice
        assert took[2] < 2 ** 10                          # and no second time
    assert max(got[3], got[9]) >= 2 ** 20
