// What the kernels that stream rows of logits and keep the largest share: the order of a row's
// logits as keys, thresholds by groups of threads, and vectors of logits at any alignment.
#pragma once

#include <type_traits>

#include "vocab_common.cuh"

namespace lmloss {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Order of the candidates of a row as one 64-bit number, larger is better: the
// logit, then the lower column.  0 stands for no candidate (-inf and NaN).
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o)
{
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, int col)
{
    // -0 and +0 are equal logits
    if (x == 0.f) x = 0.f;
    return (static_cast<uint64_t>(ordered(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(col));
}
__device__ __forceinline__ float key_logit(uint64_t k) { return unordered(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ int key_col(uint64_t k) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)); }

// The M-th largest of n > M different keys in shared memory, found eight bits at a time:
// counts of the next eight bits among the keys that share what was found so far.
// (Bit by bit, with a barrier for each, it took 25 us of a block.)
__device__ __noinline__ uint64_t mth_largest(const uint64_t* keys, int n, int M, uint32_t* counts)
{
    const int tid = threadIdx.x, lane = tid & 31;
    uint64_t found = 0;
    int want = M;
#pragma unroll 1
    for (int shift = 56; shift >= 0; shift -= 8) {
        counts[tid] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t k = keys[i];
            if (shift == 56 || (k ^ found) >> (shift + 8) == 0) atomicAdd(&counts[static_cast<uint32_t>(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        // every warp for itself: lane l's eight counts from 8 (31 - l) on, so that lower lanes have the larger bits
        uint32_t sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += counts[8 * (31 - lane) + j];
        uint32_t inc = sum;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        const uint32_t has = __ballot_sync(0xffffffffu, inc >= static_cast<uint32_t>(want));
        const int in = __ffs(has) - 1;   // the first lane by which there are enough: n > M
        uint32_t above = __shfl_sync(0xffffffffu, inc - sum, in);
        int digit = 8 * (31 - in) + 7;
        while (above + counts[digit] < static_cast<uint32_t>(want)) above += counts[digit--];
        found |= static_cast<uint64_t>(digit) << shift;
        want -= static_cast<int>(above);
        __syncthreads();
    }
    return found;
}

__device__ __forceinline__ float warp_max(float x)
{
    return unordered(__reduce_max_sync(0xffffffffu, ordered(x)));
}

// The threshold of a set of values spread over the block's threads: the M-th largest
// of the maxima of groups of neighbouring threads, 0 where fewer than M groups have
// one.  At least M values reach it, and few more do: G groups leave about
// -G ln(1 - M / G) of them, so with 32 groups for M <= 16, 64 for M <= 32 and 128
// above, at most 1.4 M.
//
// v: the thread's largest value, ordered, 0 = none.  *thr has to be 0, or an earlier
// threshold, before the barrier in here, and holds the threshold after the next one.
__device__ __forceinline__ void rank_groups(uint32_t v, int M, uint32_t* group, uint32_t* thr)
{
    const int tid = threadIdx.x;
    const int groups = M <= 16 ? 32 : (M <= 32 ? 64 : 128), gt = kThreads / groups;
    v = max(v, __shfl_xor_sync(0xffffffffu, v, 1));
    if (gt >= 4) v = max(v, __shfl_xor_sync(0xffffffffu, v, 2));
    if (gt >= 8) v = max(v, __shfl_xor_sync(0xffffffffu, v, 4));
    if ((tid & (gt - 1)) == 0) group[tid / gt] = v;
    __syncthreads();
    if (tid >= groups) return;
    const uint32_t mine = group[tid];
    int above = 0;
#pragma unroll 4
    for (int i = 0; i < groups; i += 4) {
        const uint4 o = *reinterpret_cast<const uint4*>(group + i);
        const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) above += (w[k] > mine || (w[k] == mine && i + k < tid)) ? 1 : 0;
    }
    if (above == M - 1 && mine) *thr = mine;
}

template <class T>
struct Logits {
    static constexpr int E = 16 / T::kBytes;
    // Largest of a vector's logits; a NaN is passed over here and shows up in the sum.
    __device__ static __forceinline__ float largest(const Pack<T, E>& q)
    {
        if constexpr (T::kBytes == 4) {
            return fmaxf(fmaxf(q.get(0), q.get(1)), fmaxf(q.get(2), q.get(3)));
        } else {
            using H2 = typename std::conditional<std::is_same<T, Bf16>::value, __nv_bfloat162, __half2>::type;
            const H2* h = reinterpret_cast<const H2*>(q.w);
            const H2 r = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
            const uint32_t w = *reinterpret_cast<const uint32_t*>(&r);
            return fmaxf(T::widen(static_cast<uint16_t>(w & 0xffffu)), T::widen(static_cast<uint16_t>(w >> 16)));
        }
    }
    // The same of those whose bit is set.
    __device__ static __forceinline__ float largest_allowed(Pack<T, E> q, uint32_t allow)
    {
        constexpr uint32_t kNone = T::kBytes == 4 ? 0xff800000u : (std::is_same<T, Bf16>::value ? 0xff80ff80u : 0xfc00fc00u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t keep;
            if constexpr (T::kBytes == 4) keep = 0u - (allow >> i & 1u);
            else keep = ((0u - (allow >> (2 * i) & 1u)) & 0xffffu) | ((0u - (allow >> (2 * i + 1) & 1u)) << 16);
            q.w[i] = (q.w[i] & keep) | (kNone & ~keep);
        }
        return largest(q);
    }
};

// What is read of one row.  Vectors from column lo to hi are read as they lie in
// memory (around an unaligned one the aligned words, all inside the call's logits);
// the few at the ends of a row, or of the logits, one by one.
template <class T>
struct RowLogits {
    const typename T::raw* z;
    int V, lo, hi;
};

template <class T>
__device__ __noinline__ uint4 load_ends(const RowLogits<T>& r, int c)
{
    constexpr int E = Logits<T>::E;
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const uint32_t x = c + i < r.V ? static_cast<uint32_t>(r.z[c + i]) : static_cast<uint32_t>(T::round(-INFINITY));
        if constexpr (T::kBytes == 4) w[i] = x;
        else w[i / 2] |= x << (16 * (i & 1));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// E logits from column c on, in flight; c between lo and hi.
template <class T, bool ALIGNED>
struct InFlight {
    static constexpr int E = Logits<T>::E;
    uint4 v;
    uint32_t w[5];   // unaligned: the words around them.  They need one shift each and five registers;
                     // two aligned blocks of 16 bytes need eight and a choice of words first (387
                     // rows of 218302 bf16: 57 us by blocks, 52 by three times 8 bytes, 47 by words)

    __device__ __forceinline__ void load(const RowLogits<T>& r, int c)
    {
        if constexpr (ALIGNED) {
            v = __ldg(reinterpret_cast<const uint4*>(r.z + c));
        } else {
            const uint32_t* a = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(r.z + c) & ~uintptr_t(3));
#pragma unroll
            for (int i = 0; i < (T::kBytes == 4 ? 4 : 5); ++i) w[i] = __ldg(a + i);
        }
    }
    __device__ __forceinline__ void unpack(Pack<T, E>& q, const RowLogits<T>& r, int c) const
    {
        if constexpr (ALIGNED) {
            q.w[0] = v.x; q.w[1] = v.y; q.w[2] = v.z; q.w[3] = v.w;
        } else {
            const uint32_t addr = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(r.z + c));
#pragma unroll
            for (int i = 0; i < 4; ++i) q.w[i] = T::kBytes == 4 ? w[i] : __funnelshift_r(w[i], w[i + 1], (addr & 2u) * 8u);
        }
    }
};

// E logits from any column on, those past V as -inf.
template <class T, bool ALIGNED>
__device__ __forceinline__ void load_logits(Pack<T, Logits<T>::E>& q, const RowLogits<T>& r, int c)
{
    if (c >= r.lo && c <= r.hi) {
        InFlight<T, ALIGNED> f;
        f.load(r, c);
        f.unpack(q, r, c);
    } else {
        const uint4 x = load_ends(r, c);
        q.w[0] = x.x; q.w[1] = x.y; q.w[2] = x.z; q.w[3] = x.w;
    }
}

}  // namespace
}  // namespace lmloss
