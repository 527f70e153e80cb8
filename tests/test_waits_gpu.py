"""GPU: the kernels' bounded waits give up after about a second, and say so."""
import ctypes
import os
import subprocess

import pytest
import torch

import compressed_sparse_long_gb300 as v4a
from compressed_sparse_long_gb300 import build

SOURCE = r"""
#include <cuda_runtime.h>
#include "tc.cuh"
using namespace v4a;

// Thread 0 waits for a barrier on which nobody arrives; the others look on.
template <int kWhich>
__global__ void waits(int32_t* err, unsigned long long* ns, int* gave_up) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    tc::mbar_init(&bar, 1);
    tc::fence_mbar_init();
    abort_flag = 0;
    const uint64_t t = tc::globaltimer();
    bool ok;
    if constexpr (kWhich == 0) ok = tc::mbar_wait(&bar, 0, &abort_flag, err);
    else if constexpr (kWhich == 1) ok = tc::mbar_wait_few(&bar, 0, &abort_flag, err);
    else ok = tc::mbar_wait_drain(&bar, 0);
    *ns = tc::globaltimer() - t;
    // and what the abort flag does for a wait that has not begun
    bool later = true;
    if constexpr (kWhich == 0) later = tc::mbar_wait(&bar, 0, &abort_flag, err);
    else if constexpr (kWhich == 1) later = tc::mbar_wait_few(&bar, 0, &abort_flag, err);
    *gave_up = (ok ? 0 : 1) | (later ? 0 : 2) | (abort_flag ? 4 : 0);
  }
}

extern "C" int run(int which, int32_t* err, unsigned long long* ns, int* gave_up) {
  if (which == 0) waits<0><<<1, 32>>>(err, ns, gave_up);
  else if (which == 1) waits<1><<<1, 32>>>(err, ns, gave_up);
  else waits<2><<<1, 32>>>(err, ns, gave_up);
  return (int)cudaDeviceSynchronize();
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("waits")
    (d / "waits.cu").write_text(SOURCE)
    out = d / "libwaits.so"
    subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-shared", "-cudart", "shared", "-I", build.CSRC,
                    "-I", os.path.join(os.path.dirname(build.PKG), "include"), str(d / "waits.cu"), "-o", str(out)],
                   check=True, capture_output=True)
    return out


def test_the_waits_compile(lib):
    assert os.path.exists(lib)


@pytest.mark.gpu
@pytest.mark.parametrize("which,status,bits", [(0, 7, 16), (1, 7, 16), (2, 1, 0)], ids=["wait", "few", "drain"])
def test_a_wait_gives_up_after_a_second(lib, which, status, bits):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ns = torch.zeros(1, dtype=torch.int64, device="cuda")
    gave_up = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    so = ctypes.CDLL(str(lib))
    assert so.run(which, ctypes.c_void_p(err.data_ptr()), ctypes.c_void_p(ns.data_ptr()),
                  ctypes.c_void_p(gave_up.data_ptr())) == 0
    # the limit, and up to 64 tries until the clock is looked at: those are some microseconds each
    assert 1.0e9 <= ns.item() <= 1.5e9, ns.item()
    assert gave_up.item() == status and v4a.v4a_get_error(err) == bits
