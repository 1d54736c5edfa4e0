"""The bounded wait of the expert products and the few-token layer: every lane of
a warp gets the same answer, also when the barrier completes while another warp
gives up, and a wait that nothing ends returns after a second."""
import ctypes
import subprocess
import time

import pytest
import torch

from combine_ep_layout_02_gb300 import build as cuda_build

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

SOURCE = r"""
#include "ep_tcgen05.cuh"
// One round per block.  Warp 0 waits; warp 1 (mode 0), once the waiting warp also
// looks at the others' flag, gives up and arrives, in either order and up to a
// few polls apart, or (mode 1) does neither.
__global__ void rounds(uint32_t* answers, int* left, int mode) {
    __shared__ alignas(8) uint64_t bar;
    __shared__ int gave_up;
    if (threadIdx.x == 0) {
        ep::mbar_init(ep::smem_addr(&bar), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        gave_up = 0;
    }
    __syncthreads();
    volatile int* flag = &gave_up;
    if (threadIdx.x < 32) {
        answers[blockIdx.x * 32 + threadIdx.x] = ep::mbar_wait(ep::smem_addr(&bar), 0, flag);
    } else if (threadIdx.x == 32 && mode == 0) {
        const uint64_t start = ep::global_ns();
        while (ep::global_ns() - start < 400000) {
        }
        const long long first = clock64();
        while (clock64() - first < (blockIdx.x / 2 % 64) * 128) {
        }
        if (blockIdx.x & 1) ep::mbar_arrive(ep::smem_addr(&bar));
        *flag = 1;
        const long long second = clock64();
        while (clock64() - second < (blockIdx.x / 128 % 64) * 128) {
        }
        if (!(blockIdx.x & 1)) ep::mbar_arrive(ep::smem_addr(&bar));
    }
    __syncthreads();
    if (threadIdx.x == 0) left[blockIdx.x] = gave_up;
}
extern "C" EP_API int run(uint32_t* answers, int* left, int blocks, int mode) {
    rounds<<<blocks, 64>>>(answers, left, mode);
    return (int)cudaDeviceSynchronize();
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("waits")
    src, so = str(d / "waits.cu"), str(d / "waits.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([cuda_build._nvcc()] + cuda_build.NVCC_FLAGS + ["-shared", src, "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.run.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int]
    return lib


def run(lib, blocks, mode):
    answers = torch.full((blocks, 32), 7, dtype=torch.int32, device=DEV)
    left = torch.zeros(blocks, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    start = time.monotonic()
    assert lib.run(answers.data_ptr(), left.data_ptr(), blocks, mode) == 0
    return answers.cpu(), left.cpu(), time.monotonic() - start


def test_lanes_agree_while_another_warp_gives_up(lib):
    answers, left, _ = run(lib, 65536, 0)
    assert ((answers == 0) | (answers == 1)).all()
    assert (answers == answers[:, :1]).all()
    assert (left == 1).all()
    assert 0 < answers[:, 0].sum() < len(answers)  # both happened


def test_a_wait_that_nothing_ends_returns_after_a_second(lib):
    answers, left, took = run(lib, 4, 1)
    assert (answers == 0).all() and (left == 1).all()
    assert 0.9 < took < 10.0
    assert torch.ones(8, device=DEV).sum().item() == 8  # the context is usable
