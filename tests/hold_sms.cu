// Test helper: `blocks` blocks that each take an SM's shared memory and return after
// `ns` nanoseconds (or a fixed number of looks at the clock, whichever comes first).
#include <cuda_runtime.h>

__global__ void hold_kernel(unsigned long long ns) {
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
    for (int i = 0; i < 20000000; ++i) {
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
        if (t - t0 >= ns) break;
        __nanosleep(200);
    }
}

extern "C" int hold_sms(int blocks, unsigned long long ns, void* stream) {
    const int smem = 200 * 1024;
    if (ns > 3000000000ull) return -1;
    if (cudaFuncSetAttribute(hold_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return -2;
    hold_kernel<<<blocks, 32, smem, static_cast<cudaStream_t>(stream)>>>(ns);
    return cudaGetLastError() == cudaSuccess ? 0 : -3;
}
