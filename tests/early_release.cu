// A kernel that lets its stream's next one start at once and writes afterwards: what a
// kernel launched with programmatic overlap must wait for before it reads.
#include <cstdint>
#include <cuda_runtime.h>

__global__ void early_release_kernel(const uint4* from, uint4* to, long long n, int naps) {
    asm volatile("griddepcontrol.launch_dependents;");
    for (int i = 0; i < naps; ++i) __nanosleep(1000);
    const long long step = (long long)gridDim.x * blockDim.x;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) to[i] = from[i];
}

// Copies n 16-byte words on `stream`, some `naps` microseconds after the kernel's start.
extern "C" int early_release_copy(const void* from, void* to, long long n, int naps, void* stream) {
    early_release_kernel<<<64, 128, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<const uint4*>(from),
                                                                            static_cast<uint4*>(to), n, naps);
    return (int)cudaGetLastError();
}
