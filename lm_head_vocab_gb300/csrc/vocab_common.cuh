// What the vocabulary operators share: their handle, the error word, and 16-byte
// vectors of the three floating types widened to fp32.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/lmloss.h"
#include "kernels.cuh"

struct lmloss_vocab_ctx {
    int device = 0;
    int num_sms = 0;
    int smem_optin = 0;
    unsigned char* ws = nullptr;   // [ws_bytes], after the error word's 256 bytes
    size_t ws_bytes = 0;
    int* err = nullptr;
};

namespace lmloss {

enum : int { kErrBadParent = 8 };

struct VocabDeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit VocabDeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) { ok = false; return; }
        if (prev != dev && cudaSetDevice(dev) != cudaSuccess) ok = false;
    }
    ~VocabDeviceGuard()
    {
        if (prev >= 0) cudaSetDevice(prev);
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
    using raw = uint16_t;
    static constexpr int kBytes = 2;
    __device__ static __forceinline__ float widen(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
    __device__ static __forceinline__ uint16_t round(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
};
struct Fp16 {
    using raw = uint16_t;
    static constexpr int kBytes = 2;
    __device__ static __forceinline__ float widen(uint16_t b) { return __half2float(__ushort_as_half(b)); }
    __device__ static __forceinline__ uint16_t round(float x) { return __half_as_ushort(__float2half_rn(x)); }
};
struct Fp32 {
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
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace lmloss
