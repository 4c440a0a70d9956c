// A stand-in for another library's kernel that lets the stream's next kernel
// begin before it has written its results: every block triggers the dependents,
// waits delay_ns (capped at 200 us), then copies n bytes.
#include <cuda_runtime.h>
#include <stdint.h>

__device__ __forceinline__ uint64_t now() {
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

__global__ void __launch_bounds__(256) early_producer(uint8_t* dst, const uint8_t* src, int64_t n, uint64_t delay_ns) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint64_t t0 = now(), limit = delay_ns < 200000 ? delay_ns : 200000;
    for (int i = 0; i < (1 << 20) && now() - t0 < limit; ++i) {
    }
    for (int64_t i = threadIdx.x; i < n; i += 256) dst[i] = src[i];
}

extern "C" __attribute__((visibility("default"))) int early_producer_launch(void* dst, const void* src, int64_t n,
                                                                            int64_t delay_ns, void* stream) {
    early_producer<<<1, 256, 0, (cudaStream_t)stream>>>(static_cast<uint8_t*>(dst), static_cast<const uint8_t*>(src), n,
                                                        (uint64_t)delay_ns);
    return (int)cudaGetLastError();
}
