// A kernel that lets the launch behind it start at once, writes its output only
// after a while and then ends: what a sampling kernel or an optimiser step that
// uses programmatic dependent launch may do.
#include <cuda_runtime.h>

__global__ void early_copy(unsigned *dst, const unsigned *src, long long n, unsigned long long ns)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    do {
        __nanosleep(1000);
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    } while (t - t0 < ns);
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x)
        dst[i] = src[i];
}

extern "C" int early_copy_launch(unsigned *dst, const unsigned *src, long long n, unsigned long long ns, void *stream)
{
    early_copy<<<4, 256, 0, static_cast<cudaStream_t>(stream)>>>(dst, src, n, ns);
    return static_cast<int>(cudaGetLastError());
}
