// Raising a kernel's limit of dynamic shared memory: once per kernel and device.
#include <cuda_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>

namespace csa {

// The limits set so far, by (kernel, device): about 110 kernels of the library on
// up to 16 devices.  A fixed table, since callers may be unable to allocate.  A pair
// that finds no place is set again at each launch.
constexpr unsigned kPlaces = 4096;  // a power of two

cudaError_t ensure_smem_impl(const void* kernel, size_t bytes) {
    struct Entry { const void* k; int dev; size_t bytes; };
    static Entry table[kPlaces];
    static unsigned used = 0;
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    unsigned i = unsigned(((reinterpret_cast<uintptr_t>(kernel) + unsigned(dev)) * 0x9E3779B97F4A7C15ull) >> 52);
    while (table[i].k && (table[i].k != kernel || table[i].dev != dev)) i = (i + 1) % kPlaces;
    if (table[i].k && table[i].bytes >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
    if (e != cudaSuccess) return e;
    if (table[i].k) table[i].bytes = bytes;
    else if (used < kPlaces / 2) { table[i] = Entry{kernel, dev, bytes}; ++used; }  // (half: searches stay short and end)
    return e;
}

}  // namespace csa
