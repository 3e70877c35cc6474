// late_writer.cu -- a producer for the tests of early launches: it lets the kernels behind it start at once, and writes
// their inputs some time later.
#include <cuda_runtime.h>

struct Jobs {
    int n;
    unsigned char* dst[16];
    const unsigned char* src[16];
    size_t bytes[16];
};

__global__ void __launch_bounds__(256) late_kernel(const __grid_constant__ Jobs jobs, unsigned ns) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    unsigned long long start, now;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(start));
    for (int i = 0; i < 100000; ++i) {  // bounded, also where the clock stands still
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        if (now - start >= ns) break;
        __nanosleep(200);
    }
    for (int j = 0; j < jobs.n; ++j)
        for (size_t i = blockIdx.x * blockDim.x + threadIdx.x; i < jobs.bytes[j]; i += static_cast<size_t>(gridDim.x) * blockDim.x)
            jobs.dst[j][i] = jobs.src[j][i];
}

extern "C" int late_writes(int n, void* const* dst, void* const* src, const size_t* bytes, unsigned ns, void* stream) {
    if (n < 0 || n > 16) return -1;
    Jobs jobs{};
    jobs.n = n;
    for (int i = 0; i < n; ++i) {
        jobs.dst[i] = static_cast<unsigned char*>(dst[i]);
        jobs.src[i] = static_cast<const unsigned char*>(src[i]);
        jobs.bytes[i] = bytes[i];
    }
    late_kernel<<<16, 256, 0, static_cast<cudaStream_t>(stream)>>>(jobs, ns);
    return static_cast<int>(cudaGetLastError());
}
