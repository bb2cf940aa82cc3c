// A stand-in for the CUDA runtime under the library's host code: one device, whose memory is host
// memory; a cudaMemset is done when its stream is waited for, not when it returns; an error stays
// until it is asked for.
#include <cstdlib>
#include <cstring>
#include <vector>

#include <cuda_runtime_api.h>

struct Fill {
    void* p;
    int value;
    size_t n;
};
static std::vector<Fill>& fills()
{
    static std::vector<Fill> f;
    return f;
}
static cudaError_t finish()
{
    for (const Fill& f : fills()) std::memset(f.p, f.value, f.n);
    fills().clear();
    return cudaSuccess;
}
static cudaError_t last = cudaSuccess;
int unfinished_fills() { return static_cast<int>(fills().size()); }

extern "C" {
cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaSetDevice(int d) { return d == 0 ? cudaSuccess : (last = cudaErrorInvalidDevice); }
cudaError_t cudaGetLastError()
{
    const cudaError_t e = last;
    last = cudaSuccess;
    return e;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { return *v = 152, cudaSuccess; }
cudaError_t cudaMalloc(void** p, size_t n)
{
    *p = std::malloc(n);
    if (!*p) return cudaErrorMemoryAllocation;
    std::memset(*p, 0xa5, n);   // what was there before
    return cudaSuccess;
}
cudaError_t cudaFree(void* p) { return finish(), std::free(p), cudaSuccess; }
cudaError_t cudaMemset(void* p, int value, size_t n) { return fills().push_back({p, value, n}), cudaSuccess; }
cudaError_t cudaMemcpy(void* to, const void* from, size_t n, cudaMemcpyKind) { return finish(), std::memcpy(to, from, n), cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return finish(); }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return finish(); }
// what a compiled .cu file registers when it is loaded
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, void*, void*, void*, void*, int*) {}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
}
