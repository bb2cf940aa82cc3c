// The vocabulary operators' handle: a workspace of the caller's size, an error word
// and the counters.
#include <new>

#include "vocab_common.cuh"

using namespace lmloss;

extern "C" {

lmloss_status lmloss_vocab_create(lmloss_vocab_handle* handle, int device, size_t workspace_bytes)
{
    if (!handle) return LMLOSS_ERR_INVALID_ARG;
    *handle = nullptr;
    VocabDeviceGuard g(device);
    if (!g.ok) return LMLOSS_ERR_CUDA;
    if (workspace_bytes > SIZE_MAX / 2) return LMLOSS_ERR_INVALID_ARG;
    lmloss_vocab_ctx* h = new (std::nothrow) lmloss_vocab_ctx();
    if (!h) return LMLOSS_ERR_CUDA;
    h->device = device;
    h->ws_bytes = vocab_align(workspace_bytes);
    constexpr size_t kHead = 256 + kVocabCounters * sizeof(unsigned);
    unsigned char* mem = nullptr;
    if (cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess ||
        cudaMalloc(&mem, kHead + h->ws_bytes) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return LMLOSS_ERR_CUDA;
    }
    // A memset may return before it is done, and a stream that is not ordered after the legacy one
    // would count blocks from what the memory held.
    if (cudaMemset(mem, 0, kHead + h->ws_bytes) != cudaSuccess || cudaStreamSynchronize(nullptr) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(mem);
        delete h;
        return LMLOSS_ERR_CUDA;
    }
    h->mem = mem;
    h->err = reinterpret_cast<int*>(mem);
    h->counters = reinterpret_cast<unsigned*>(mem + 256);
    h->ws = mem + kHead;
    *handle = h;
    return LMLOSS_OK;
}

lmloss_status lmloss_vocab_reserve(lmloss_vocab_handle h, size_t workspace_bytes)
{
    if (!h || workspace_bytes > SIZE_MAX / 2) return LMLOSS_ERR_INVALID_ARG;
    if (workspace_bytes <= h->ws_bytes) return LMLOSS_OK;
    VocabDeviceGuard g(h->device);
    if (!g.ok) return LMLOSS_ERR_CUDA;
    const size_t bytes = vocab_align(workspace_bytes);
    // a capture forbids allocations unless the thread says that it knows about them
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) {
        cudaGetLastError();
        return LMLOSS_ERR_CUDA;
    }
    unsigned char* ws = nullptr;
    const bool there = cudaMalloc(&ws, bytes) == cudaSuccess;
    if (!there) cudaGetLastError();
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (!there) return LMLOSS_ERR_CUDA;
    try {
        h->more.push_back(ws);
    } catch (...) {
        cudaFree(ws);
        return LMLOSS_ERR_CUDA;
    }
    // (what a workspace holds when a call begins is of no matter: the counters lie apart from it)
    h->ws = ws;
    h->ws_bytes = bytes;
    return LMLOSS_OK;
}

lmloss_status lmloss_vocab_destroy(lmloss_vocab_handle h)
{
    if (!h) return LMLOSS_ERR_INVALID_ARG;
    VocabDeviceGuard g(h->device);
    cudaDeviceSynchronize();
    bool freed = cudaFree(h->mem) == cudaSuccess;
    for (unsigned char* ws : h->more) freed &= cudaFree(ws) == cudaSuccess;
    delete h;
    return freed ? LMLOSS_OK : LMLOSS_ERR_CUDA;
}

lmloss_status lmloss_vocab_get_device_error(lmloss_vocab_handle h)
{
    if (!h) return LMLOSS_ERR_INVALID_ARG;
    VocabDeviceGuard g(h->device);
    if (!g.ok || cudaDeviceSynchronize() != cudaSuccess) return LMLOSS_ERR_CUDA;
    int code = 0;
    if (cudaMemcpy(&code, h->err, sizeof code, cudaMemcpyDeviceToHost) != cudaSuccess) return LMLOSS_ERR_CUDA;
    // done before it returns: it must not clear what the next call reports
    if (cudaMemset(h->err, 0, sizeof code) != cudaSuccess || cudaStreamSynchronize(nullptr) != cudaSuccess)
        return LMLOSS_ERR_CUDA;
    return static_cast<lmloss_status>(code);
}

}  // extern "C"
