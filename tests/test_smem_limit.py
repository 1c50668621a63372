"""How often the library raises a kernel's shared-memory limit: counted against fakes of the two CUDA calls, on the host."""
import os
import subprocess

from compressed_sparse_attention_13_b200 import build

HARNESS = r"""
#include <cuda_runtime_api.h>
#include <cstdio>
#include <cstdint>

namespace csa { cudaError_t ensure_smem_impl(const void* kernel, size_t bytes); }

static int device = 0, sets = 0;
static cudaError_t answer = cudaSuccess;
extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { ++sets; return answer; }

static int round_of(int kernels, int devices, size_t bytes) {
    sets = 0;
    for (device = 0; device < devices; ++device)
        for (int k = 0; k < kernels; ++k)
            if (csa::ensure_smem_impl((const void*)(uintptr_t(0x10000) + 16 * k), bytes) != answer) return -1;
    return sets;
}

int main() {
    printf("%d\n", round_of(110, 16, 1000));  // once each
    printf("%d\n", round_of(110, 16, 1000));  // known
    printf("%d\n", round_of(110, 16, 900));   // known to be more
    printf("%d\n", round_of(110, 16, 2000));  // more is asked for
    printf("%d\n", round_of(110, 16, 2000));
    answer = cudaErrorInvalidValue;
    printf("%d\n", round_of(110, 1, 3000));   // refused: an error each time, the old limit stays known
    answer = cudaSuccess;
    printf("%d\n", round_of(110, 1, 2000));
    sets = round_of(3000, 1, 1);              // more than there is room for: set again, never lost
    printf("%d\n", round_of(3000, 1, 1) < 3000);
    return 0;
}
"""


def test_a_limit_is_set_once_per_kernel_and_device(tmp_path):
    src, exe = str(tmp_path / "harness.cpp"), str(tmp_path / "harness")
    with open(src, "w") as f:
        f.write(HARNESS)
    inc = os.path.join(os.path.dirname(os.path.dirname(build.NVCC)), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{inc}", src, "-x", "c++", os.path.join(build.CSRC, "smem_limit.cu"), "-o", exe,
                    "-lpthread"], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=60).stdout.split()
    n = 110 * 16
    assert out == [str(n), "0", "0", str(n), "0", "110", "0", "1"]
