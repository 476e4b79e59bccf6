// kernel_setup.cuh -- what a launcher asks of the runtime once per kernel and
// device instead of at every call: the opt-in to large dynamic shared memory
// (about 1 us a time), the number of resident blocks (about 5 us).
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace ssm {

constexpr int kSetupDevices = 64;  // beyond these the runtime is asked every time

// Lets KERNEL use up to SMEM bytes (the most that its launcher asks for) of
// dynamic shared memory on the current device.
template <auto KERNEL, int SMEM>
cudaError_t allow_smem() {
    static std::atomic<bool> allowed[kSetupDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kSetupDevices;
    if (known && allowed[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e == cudaSuccess && known) allowed[dev].store(true, std::memory_order_release);
    return e;
}

// Blocks of KERNEL (THREADS threads, SMEM bytes of dynamic shared memory) that
// an SM holds at once; allows that shared memory too.
template <auto KERNEL, int THREADS, int SMEM>
cudaError_t resident_blocks(int *per_sm) {
    static std::atomic<int> held[kSetupDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kSetupDevices;
    if (known && (*per_sm = held[dev].load(std::memory_order_acquire)) > 0) return cudaSuccess;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(per_sm, KERNEL, THREADS, SMEM);
    if (e != cudaSuccess) return e;
    if (*per_sm < 1) *per_sm = 1;
    if (known) held[dev].store(*per_sm, std::memory_order_release);
    return cudaSuccess;
}

}  // namespace ssm
