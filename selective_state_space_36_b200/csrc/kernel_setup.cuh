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

// A kernel that follows another one of the same call may be launched before that
// has ended (programmatic dependent launch): its launch and set-up, 2 to 3 us,
// then lie under the other's end.  The first calls next_may_start() as soon as
// it likes; the second calls previous_done() in every thread before it reads
// what the first wrote or writes what the first reads.  (For kernels whose blocks
// fill an SM it gains nothing: the early blocks of the gated delta rule's chain
// cost 1 to 5 %.)
__device__ __forceinline__ void previous_done() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), int64_t blocks, unsigned threads, size_t smem, cudaStream_t st,
                             const A &...args) {
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    c.gridDim = dim3((unsigned)blocks);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = attr;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

}  // namespace ssm
