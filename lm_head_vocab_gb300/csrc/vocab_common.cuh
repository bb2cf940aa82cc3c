// What the vocabulary operators share: their handle, the error word, and 16-byte
// vectors of the three floating types widened to fp32.
#pragma once

#include <cstdint>
#include <vector>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/lmloss.h"
#include "kernels.cuh"

// Counters of blocks that have finished, apart from the workspace: all zero
// between calls, each returned to zero by the block that finds it full.
constexpr int kVocabCounters = 1 << 16;

struct lmloss_vocab_ctx {
    int device = 0;
    int num_sms = 0;
    unsigned char* mem = nullptr;    // what was allocated: the error word, the counters, the workspace
    int* err = nullptr;
    unsigned* counters = nullptr;    // [kVocabCounters]
    unsigned char* ws = nullptr;     // [ws_bytes]
    size_t ws_bytes = 0;
    std::vector<unsigned char*> more;   // workspaces of lmloss_vocab_reserve
    uint32_t limits_raised = 0;      // sorting kernels whose launch limits were raised
};

namespace lmloss {

enum : int { kErrBadParent = 8 };

struct VocabDeviceGuard {
    int prev = -1;
    bool ok = true, moved = false;
    explicit VocabDeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) { ok = false; return; }
        if (prev == dev) return;
        moved = cudaSetDevice(dev) == cudaSuccess;
        if (!moved) {
            cudaGetLastError();   // not left for the next launch's check
            ok = false;
        }
    }
    ~VocabDeviceGuard()
    {
        if (moved) cudaSetDevice(prev);
    }
};

inline lmloss_status vocab_launch_err()
{
    return cudaGetLastError() == cudaSuccess ? LMLOSS_OK : LMLOSS_ERR_CUDA;
}

inline size_t vocab_align(size_t x) { return (x + 255) / 256 * 256; }

inline int float_bytes(int32_t dtype) { return dtype == LMLOSS_FP32 ? 4 : 2; }

inline bool float_dtype(int32_t dtype) { return dtype == LMLOSS_BF16 || dtype == LMLOSS_FP32 || dtype == LMLOSS_FP16; }

// ------------------------------------------------------------- float types
struct Bf16 {
    static constexpr int kIndex = 0;
    using raw = uint16_t;
    static constexpr int kBytes = 2;
    __device__ static __forceinline__ float widen(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
    __device__ static __forceinline__ uint16_t round(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
    __device__ static __forceinline__ uint32_t round2(float lo, float hi)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
struct Fp16 {
    static constexpr int kIndex = 1;
    using raw = uint16_t;
    static constexpr int kBytes = 2;
    __device__ static __forceinline__ float widen(uint16_t b) { return __half2float(__ushort_as_half(b)); }
    __device__ static __forceinline__ uint16_t round(float x) { return __half_as_ushort(__float2half_rn(x)); }
    __device__ static __forceinline__ uint32_t round2(float lo, float hi)
    {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
struct Fp32 {
    static constexpr int kIndex = 2;
    using raw = uint32_t;
    static constexpr int kBytes = 4;
    __device__ static __forceinline__ float widen(uint32_t b) { return __uint_as_float(b); }
    __device__ static __forceinline__ uint32_t round(float x) { return __float_as_uint(x); }
};

// N consecutive elements of type T in registers: whole 16-byte vectors (8-byte
// where N elements are only that long), or one element.
template <class T, int N>
struct Pack {
    static constexpr int kBytes = N * T::kBytes;
    static constexpr int kWords = kBytes / 4 > 0 ? kBytes / 4 : 1;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const void* p)
    {
        if constexpr (kBytes % 16 == 0) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) {
                const uint4 q = __ldg(static_cast<const uint4*>(p) + i);
                w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
            }
        } else {
            static_assert(N == 1, "whole vectors or one element");
            w[0] = *static_cast<const typename T::raw*>(p);
        }
    }
    // for memory that the same kernel also writes: no read-only path
    __device__ __forceinline__ void load_rw(const void* p)
    {
        if constexpr (kBytes % 16 == 0) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) {
                const uint4 q = *(static_cast<const uint4*>(p) + i);
                w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
            }
        } else {
            w[0] = *static_cast<const typename T::raw*>(p);
        }
    }
    __device__ __forceinline__ void store(void* p) const
    {
        if constexpr (kBytes % 16 == 0) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i)
                static_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else {
            *static_cast<typename T::raw*>(p) = static_cast<typename T::raw>(w[0]);
        }
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (T::kBytes == 4) return __uint_as_float(w[i]);
        else return T::widen(static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1))));
    }
    __device__ __forceinline__ void set(int i, float x)
    {
        if constexpr (T::kBytes == 4) {
            w[i] = __float_as_uint(x);
        } else {
            const uint32_t b = T::round(x);
            if (i & 1) w[i / 2] = (w[i / 2] & 0xffffu) | (b << 16);
            else w[i / 2] = (N > 1 ? (w[i / 2] & 0xffff0000u) : 0u) | b;
        }
    }
    // all N elements, rounded in pairs
    __device__ __forceinline__ void set_all(const float (&x)[N])
    {
        static_assert(N % 2 == 0, "pairs");
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            if constexpr (T::kBytes == 4) {
                w[i] = __float_as_uint(x[i]);
                w[i + 1] = __float_as_uint(x[i + 1]);
            } else {
                w[i / 2] = T::round2(x[i], x[i + 1]);
            }
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
};

// N elements from an address aligned to one element only: the aligned 16-byte
// blocks around it, shifted into place in registers.  Every block must lie inside
// memory that may be read, [lo, hi); `inside_blocks` says so.
template <class T, int N>
__device__ __forceinline__ bool inside_blocks(const unsigned char* p, const unsigned char* lo, const unsigned char* hi)
{
    const unsigned char* a = reinterpret_cast<const unsigned char*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15));
    return a >= lo && a + N * T::kBytes + 16 <= hi;
}
// The N elements that begin `addr` % 16 bytes into the blocks v.
template <class T, int N, int VECS>
__device__ __forceinline__ void shift_blocks(Pack<T, N>& q, const uint4 (&v)[VECS], uint32_t addr)
{
    static_assert(VECS == N * T::kBytes / 16 + 1, "one block more than the elements fill");
    uint32_t w[4 * VECS];
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        w[4 * i] = v[i].x; w[4 * i + 1] = v[i].y; w[4 * i + 2] = v[i].z; w[4 * i + 3] = v[i].w;
    }
    if (addr & 8u) {
#pragma unroll
        for (int i = 0; i + 2 < 4 * VECS; ++i) w[i] = w[i + 2];
    }
    if (addr & 4u) {
#pragma unroll
        for (int i = 0; i + 1 < 4 * VECS; ++i) w[i] = w[i + 1];
    }
    if constexpr (T::kBytes == 2) {
        const uint32_t sh = (addr & 2u) * 8u;   // 0 or 16 bits
#pragma unroll
        for (int i = 0; i < Pack<T, N>::kWords; ++i) q.w[i] = __funnelshift_r(w[i], w[i + 1], sh);
    } else {
#pragma unroll
        for (int i = 0; i < Pack<T, N>::kWords; ++i) q.w[i] = w[i];
    }
}

// Counts this block's arrival; what the block wrote before a barrier that this
// thread has passed is visible to whoever sees the count, and what others wrote
// before theirs to this one.
__device__ __forceinline__ unsigned count_done(unsigned* counter)
{
    unsigned old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
    return old;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace lmloss
