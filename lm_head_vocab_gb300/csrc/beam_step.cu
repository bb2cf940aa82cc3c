// Beam search's step: the M best continuations of each sequence's K beams over the
// whole vocabulary.
//
//   score(k, v) = scores[k] + z[k][v] - lse_k,   lse_k = ln sum_v e^z[k][v]
//
// The logits are read once.  Within a row the order of the candidates is the
// order of the logits, whatever the row's normaliser, so one pass over a slice of
// a row can keep both its softmax partials and its M largest logits; a
// second, small kernel joins the slices of a row, turns logits into scores in fp64
// and picks the M best of the sequence's rows.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "vocab_common.cuh"

namespace lmloss {
namespace {

constexpr int kMaxM = LMLOSS_MAX_BEAMS;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCap = 2048;                   // candidate keys of a slice held at once
constexpr int kSmall = 256;                  // few enough to be ranked by counting
constexpr int kFinal = 768;                  // candidates of a sequence held at once
constexpr int kDepths = 8;                   // lists a thread: rows * slices <= 8 * kThreads
constexpr int kMaxLists = kDepths * kThreads;

struct BeamParams {
    const void* logits;
    int64_t ld;
    int B, K, M, V;
    int slices;                  // of a row
    float alpha;
    int64_t eos;
    const float* scores;
    const uint8_t* finished;
    const int32_t* lengths;
    const int32_t* mask;
    int64_t mask_stride;
    float* scores_out;
    int32_t* parents_out;
    int64_t* tokens_out;
    float* lse_out;
    uint8_t* finished_out;
    int32_t* lengths_out;
    uint64_t* keys;              // [rows][M][slices]: each slice's candidates, best first, 0 = none
    float2* stats;               // [rows][slices] (m, s): the slice's sum of e^z is s e^m
    unsigned* done;              // [B] slices finished; 0 between calls
};

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
__device__ __forceinline__ uint64_t ordered64(double x)
{
    if (x == 0.0) x = 0.0;
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x));
    return (b >> 63) ? ~b : (b | (uint64_t(1) << 63));
}

// the M-th largest of n > M different keys in shared memory, found bit by bit
__device__ __noinline__ uint64_t mth_largest(const uint64_t* keys, int n, int M)
{
    uint64_t t = 0;
    for (int bit = 63; bit >= 0; --bit) {
        const uint64_t cand = t | (uint64_t(1) << bit);
        int c = 0;
        for (int i0 = 0; i0 < n; i0 += kThreads) {
            const int i = i0 + threadIdx.x;
            c += __syncthreads_count(i < n && keys[i] >= cand);
        }
        if (c >= M) t = cand;
    }
    return t;
}

// Groups of neighbouring threads whose maxima give the threshold: 32 of eight
// threads for M <= 16, 64 of four for more.  At least M candidates reach the M-th
// largest of at least 2 M (or 64) maxima, and few more do: with random order about
// ln 2 of a candidate a group lies above the middle one.
__device__ __forceinline__ int group_threads(int M) { return M <= 16 ? 8 : 4; }

// The group maxima of `v` (0 = none) into group[], by every thread of the block.
__device__ __forceinline__ void group_maxima(uint32_t v, int gt, uint32_t* group)
{
    v = max(v, __shfl_xor_sync(0xffffffffu, v, 1));
    v = max(v, __shfl_xor_sync(0xffffffffu, v, 2));
    if (gt == 8) v = max(v, __shfl_xor_sync(0xffffffffu, v, 4));
    if ((threadIdx.x & (gt - 1)) == 0) group[threadIdx.x / gt] = v;
}

// The M-th largest of the group maxima, 0 where there are fewer; one warp, after
// a barrier.
__device__ __forceinline__ uint32_t group_threshold(const uint32_t* group, int gt, int M)
{
    const int lane = threadIdx.x & 31;
    const int groups = kThreads / gt;
    uint32_t found = 0;
    for (int g0 = 0; g0 < groups; g0 += 32) {
        const uint32_t v = group[g0 + lane];
        int above = 0;
        for (int i = 0; i < groups; i += 4) {
            const uint4 o = *reinterpret_cast<const uint4*>(group + i);
            const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) above += (w[k] > v || (w[k] == v && i + k < g0 + lane)) ? 1 : 0;
        }
        if (above == M - 1) found = v;
    }
    return __reduce_max_sync(0xffffffffu, found);
}

struct __align__(16) Shared {
    uint64_t buf[kCap];                      // a slice's candidates; a sequence's finalists
    uint32_t group[64];
    float red[kWarps];
    uint32_t thr;
    int count;
    int last;
    // of a sequence's rows
    double base[kMaxM], norm[kMaxM];
    float m[kMaxM], hi[kMaxM], lo[kMaxM], base_f[kMaxM], inv_f[kMaxM];
    uint8_t done[kMaxM];
    // the slow way of picking
    uint64_t wbest[kWarps], wplace[kWarps];
    int wlist[kWarps];
    int lead;
};

// A candidate's score and rank key in fp64; false where it is none.
__device__ __forceinline__ bool exact_score(const BeamParams& p, const Shared& sm, int k, float z, uint64_t& rank)
{
    const double score = sm.done[k] ? sm.base[k] : sm.base[k] + static_cast<double>(z);
    if (!isfinite(score)) return false;
    rank = ordered64(p.lengths ? score / sm.norm[k] : score);
    return true;
}

__device__ __forceinline__ uint64_t list_key(const BeamParams& p, const Shared& sm, int64_t r0, int list, int d)
{
    const int k = list / p.slices, s = list - k * p.slices;
    if (sm.done[k]) return s == 0 && d == 0 ? 1 : 0;
    return __ldcg(p.keys + ((r0 + k) * p.M + d) * p.slices + s);
}

__device__ __forceinline__ void write_pick(const BeamParams& p, const Shared& sm, int b, int out, int k, float z, int token)
{
    const int64_t o = static_cast<int64_t>(b) * p.M + out, r = static_cast<int64_t>(b) * p.K + k;
    const bool done = sm.done[k];
    const int64_t t = done ? p.eos : token;
    p.scores_out[o] = static_cast<float>(done ? sm.base[k] : sm.base[k] + static_cast<double>(z));
    p.parents_out[o] = k;
    p.tokens_out[o] = t;
    if (p.finished_out) p.finished_out[o] = done || t == p.eos ? 1 : 0;
    if (p.lengths_out) p.lengths_out[o] = p.lengths[r] + (done ? 0 : 1);
}

__device__ __forceinline__ void write_empty(const BeamParams& p, int b, int out)
{
    const int64_t o = static_cast<int64_t>(b) * p.M + out;
    const int k = out % p.K;
    p.scores_out[o] = -INFINITY;
    p.parents_out[o] = k;
    p.tokens_out[o] = LMLOSS_IGNORE_INDEX;
    if (p.finished_out) p.finished_out[o] = 0;
    if (p.lengths_out) p.lengths_out[o] = p.lengths[static_cast<int64_t>(b) * p.K + k];
}

// M rounds of taking the best head of the sorted lists (one a row and slice): for
// sequences with more equal or nearly equal candidates than kFinal.
__device__ __noinline__ void pick_by_rounds(const BeamParams& p, Shared& sm, const int b)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t r0 = static_cast<int64_t>(b) * p.K;
    const int lists = p.K * p.slices;
    uint64_t depth = 0;          // a byte for each of the thread's lists
    uint64_t rank = 0, place = 0;
    int list = -1;
    bool stale = true;
    for (int out = 0; out < p.M; ++out) {
        if (stale) {
            rank = 0;
            place = ~uint64_t(0);
            list = -1;
            for (int j = 0; j < kDepths; ++j) {
                const int i = tid + j * kThreads, d = static_cast<int>(depth >> (8 * j)) & 255;
                if (i >= lists || d >= p.M) continue;
                const uint64_t key = list_key(p, sm, r0, i, d);
                const int k = i / p.slices;
                uint64_t cr;
                if (key == 0 || !exact_score(p, sm, k, key_logit(key), cr)) continue;
                const uint64_t cp = (static_cast<uint64_t>(k) << 32) | static_cast<uint32_t>(sm.done[k] ? 0 : key_col(key));
                if (cr > rank || (cr == rank && cp < place)) {
                    rank = cr;
                    place = cp;
                    list = i;
                }
            }
            stale = false;
        }
        uint64_t br = rank, bp = place;
        int bl = list;
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t r2 = __shfl_xor_sync(0xffffffffu, br, o), p2 = __shfl_xor_sync(0xffffffffu, bp, o);
            const int l2 = __shfl_xor_sync(0xffffffffu, bl, o);
            if (r2 > br || (r2 == br && p2 < bp)) {
                br = r2;
                bp = p2;
                bl = l2;
            }
        }
        if (lane == 0) {
            sm.wbest[warp] = br;
            sm.wplace[warp] = bp;
            sm.wlist[warp] = bl;
        }
        __syncthreads();
        if (tid == 0) {
            int w = 0;
            for (int x = 1; x < kWarps; ++x)
                if (sm.wbest[x] > sm.wbest[w] || (sm.wbest[x] == sm.wbest[w] && sm.wplace[x] < sm.wplace[w])) w = x;
            sm.lead = sm.wbest[w] ? sm.wlist[w] : -1;
        }
        __syncthreads();
        const int won = sm.lead;
        if (won < 0) {
            if (tid == 0) write_empty(p, b, out);
        } else if (won % kThreads == tid) {
            const int j = won / kThreads, d = static_cast<int>(depth >> (8 * j)) & 255;
            depth += uint64_t(1) << (8 * j);
            const uint64_t key = list_key(p, sm, r0, won, d);
            write_pick(p, sm, b, out, won / p.slices, key_logit(key), key_col(key));
            stale = true;
        }
    }
}

// The block that finishes a sequence's last slice picks its M best.
__device__ __noinline__ void pick(const BeamParams& p, Shared& sm, const int b)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = p.K, M = p.M, S = p.slices;
    const int64_t r0 = static_cast<int64_t>(b) * K;

    // ---- the rows' normalisers: the slices' sums are added as pairs of fp32 (an
    // error-free sum and what it leaves), since fp64 is slow on this GPU; only the
    // logarithm is taken in fp64, one lane a row
    for (int k = warp; k < K; k += kWarps) {
        const int64_t r = r0 + k;
        const bool done = p.finished && p.finished[r];
        float m = -INFINITY, hi = 0.f, lo = 0.f;
        if (!done) {
            for (int s = lane; s < S; s += 32) m = fmaxf(m, __ldcg(&p.stats[r * S + s]).x);
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            auto add = [&](float x, float e) {
                const float t = hi + x, v = t - hi;
                lo += ((hi - (t - v)) + (x - v)) + e;
                hi = t;
            };
            for (int s = lane; s < S; s += 32) {
                const float2 q = __ldcg(&p.stats[r * S + s]);
                // an empty slice (-inf, 0) adds nothing; NaN stays
                add(q.x == m ? q.y : q.y * exp2f((q.x - m) * kLog2e), 0.f);
            }
            for (int o = 16; o > 0; o >>= 1) {
                const float x = __shfl_xor_sync(0xffffffffu, hi, o), e = __shfl_xor_sync(0xffffffffu, lo, o);
                add(x, e);
            }
        }
        if (lane == 0) {
            sm.m[k] = m;
            sm.hi[k] = hi;
            sm.lo[k] = lo;
            sm.done[k] = done ? 1 : 0;
        }
    }
    __syncthreads();
    if (tid < K) {
        const int64_t r = r0 + tid;
        const bool done = sm.done[tid];
        const double score = static_cast<double>(p.scores[r]);
        double lse = 0.0;
        if (!done) {
            const double sum = static_cast<double>(sm.hi[tid]) + static_cast<double>(sm.lo[tid]);
            lse = sm.m[tid] == -INFINITY && sum == 0.0 ? -INFINITY : static_cast<double>(sm.m[tid]) + log(sum);
        }
        if (p.lse_out) p.lse_out[r] = static_cast<float>(lse);
        double d = 1.0;
        if (p.lengths) {
            const int64_t len = static_cast<int64_t>(p.lengths[r]) + (done ? 0 : 1);
            d = pow(static_cast<double>(len < 1 ? 1 : len), static_cast<double>(p.alpha));
        }
        sm.base[tid] = score - lse;
        sm.norm[tid] = d;
        sm.base_f[tid] = static_cast<float>(score - lse);
        sm.inv_f[tid] = static_cast<float>(1.0 / d);
    }
    if (tid == 0) sm.count = 0;
    __syncthreads();

    // ---- a threshold in fp32.  Each candidate's rank key lies within `err` of its
    // fp32 value: four roundings of at most 2^-24 of the terms.
    const int lists = K * S;
    auto bounds = [&](int k, uint64_t key, float& low, float& high) {
        const float z = sm.done[k] ? 0.f : key_logit(key);
        const float x = (sm.base_f[k] + z) * sm.inv_f[k];
        const float err = (fabsf(sm.base_f[k]) + fabsf(z)) * sm.inv_f[k] * 4.8e-7f + 1e-37f;
        low = x - err;
        high = x + err;
        if (!(fabsf(x) < INFINITY && err < INFINITY)) {
            low = -INFINITY;
            high = INFINITY;
        }
        if (!isfinite(sm.base[k])) high = low = -INFINITY;   // the row is out
    };
    const int gt = group_threads(M);
    {
        // heads first, and deeper where there are few lists
        const int depths = lists >= kThreads ? 1 : min(M, (kThreads + lists - 1) / lists);
        float best = -INFINITY;
        for (int e = tid; e < lists * depths; e += kThreads) {
            const int d = e / lists, i = e - d * lists;
            const uint64_t key = list_key(p, sm, r0, i, d);
            if (key == 0) continue;
            float low, high;
            bounds(i / S, key, low, high);
            best = fmaxf(best, low);
        }
        group_maxima(best > -INFINITY ? ordered(best) : 0u, gt, sm.group);
        __syncthreads();
        if (warp == 0) {
            const uint32_t t = group_threshold(sm.group, gt, M);
            if (lane == 0) sm.thr = t;
        }
        __syncthreads();
    }
    const float thr = sm.thr ? unordered(sm.thr) : -INFINITY;

    // ---- the candidates that may reach it, ranked by counting in fp64
    uint64_t* rank_of = sm.buf;
    uint64_t* place_of = sm.buf + kFinal;
    float* z_of = reinterpret_cast<float*>(sm.buf + 2 * kFinal);
    static_assert(2 * kFinal + kFinal / 2 <= kCap, "finalists fit");
    for (int i = tid; i < lists; i += kThreads) {
        const int k = i / S;
        for (int d = 0; d < M; ++d) {
            const uint64_t key = list_key(p, sm, r0, i, d);
            if (key == 0) break;
            float low, high;
            bounds(k, key, low, high);
            // the list goes down: nothing after this one either
            if (high < thr || high == -INFINITY) break;
            uint64_t rank;
            const float z = sm.done[k] ? 0.f : key_logit(key);
            if (!exact_score(p, sm, k, z, rank)) continue;
            const int to = atomicAdd(&sm.count, 1);
            if (to < kFinal) {
                rank_of[to] = rank;
                place_of[to] = (static_cast<uint64_t>(k) << 32) | static_cast<uint32_t>(sm.done[k] ? 0 : key_col(key));
                z_of[to] = z;
            }
        }
    }
    __syncthreads();
    const int n = sm.count;
    if (n > kFinal) {
        pick_by_rounds(p, sm, b);
        return;
    }
    for (int i = tid; i < n; i += kThreads) {
        const uint64_t rank = rank_of[i], place = place_of[i];
        int above = 0;
        for (int o = 0; o < n; ++o) above += (rank_of[o] > rank || (rank_of[o] == rank && place_of[o] < place)) ? 1 : 0;
        if (above < M)
            write_pick(p, sm, b, above, static_cast<int>(place >> 32), z_of[i], static_cast<int>(place & 0xffffffffu));
    }
    for (int i = n + tid; i < M; i += kThreads) write_empty(p, b, i);
}

// ------------------------------------------------------------- one slice
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
};

// E logits from column c on, those past V as -inf.
template <class T, bool ALIGNED>
__device__ __forceinline__ void load_logits(Pack<T, Logits<T>::E>& q, const typename T::raw* z, int64_t c, int V,
                                            const unsigned char* lo, const unsigned char* hi)
{
    constexpr int E = Logits<T>::E;
    if (ALIGNED && c + E <= V) {
        q.load(z + c);
    } else if (!ALIGNED && c + E <= V && inside_blocks<T, E>(reinterpret_cast<const unsigned char*>(z + c), lo, hi)) {
        load_shifted<T, E>(q, reinterpret_cast<const unsigned char*>(z + c));
    } else {
        q.zero();
#pragma unroll
        for (int i = 0; i < E; ++i) q.set(i, c + i < V ? T::widen(z[c + i]) : -INFINITY);
    }
}

// Slice s of row r: kThreads * VPT vectors of E columns, vector j of a thread at
// column ((s * VPT + j) * kThreads + thread) * E.  Columns, not addresses, fix
// which thread adds what, so equal rows give equal bits wherever they start.
//
// The whole slice is in registers at once, so its maximum is known before the
// first exponential and nothing is rescaled.  Only vectors whose largest logit
// reaches the threshold are looked at a second time.
template <class T, int VPT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 4) beam_step_kernel(const __grid_constant__ BeamParams p)
{
    constexpr int E = Logits<T>::E;
    __shared__ Shared sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / p.slices, slice = blockIdx.x - row * p.slices;
    const int b = row / p.K;
    if (!(p.finished && p.finished[row])) {
        const typename T::raw* z = static_cast<const typename T::raw*>(p.logits) + static_cast<int64_t>(row) * p.ld;
        const unsigned char* lo = static_cast<const unsigned char*>(p.logits);
        const unsigned char* hi = lo + ((static_cast<int64_t>(p.B) * p.K - 1) * p.ld + p.V) * T::kBytes;
        const int32_t* mask = p.mask ? p.mask + row * p.mask_stride : nullptr;
        // V is at most kMaxLists slices long, far below 2^31
        const int first = slice * (VPT * kThreads * E) + tid * E;

        Pack<T, E> q[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) load_logits<T, ALIGNED>(q[j], z, first + j * (kThreads * E), p.V, lo, hi);

        // ---- maxima: of all logits (for the sum) and of the allowed ones (for the order)
        float m = -INFINITY, vmax[VPT], best = -INFINITY;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            vmax[j] = Logits<T>::largest(q[j]);
            m = fmaxf(m, vmax[j]);
        }
        if (mask) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = first + j * (kThreads * E);
                const uint32_t allow = c < p.V ? static_cast<uint32_t>(mask[c >> 5]) >> (c & 31) : 0u;
                float x = -INFINITY;
#pragma unroll
                for (int i = 0; i < E; ++i)
                    if (allow >> i & 1u) x = fmaxf(x, q[j].get(i));
                vmax[j] = x;
            }
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) best = fmaxf(best, vmax[j]);
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int gt = group_threads(p.M);
        group_maxima(best > -INFINITY ? ordered(best == 0.f ? 0.f : best) : 0u, gt, sm.group);
        if (lane == 0) sm.red[warp] = m;
        if (tid == 0) sm.count = 0;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.red[w]);
        if (warp == 0) {
            const uint32_t t = group_threshold(sm.group, gt, p.M);
            if (lane == 0) sm.thr = t;
        }

        // ---- sum of exponentials.  The maximum is taken off before the change to
        // base 2: z log2 e alone would overflow at the type's lowest values.
        const float shift = m == -INFINITY ? 0.f : m;
        const uint64_t off2 = f2_pack(-shift, -shift), l2 = f2_pack(kLog2e, kLog2e);
        uint64_t s2 = f2_pack(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            uint64_t part = f2_pack(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                float a, c;
                f2_unpack(f2_mul(f2_add(f2_pack(q[j].get(i), q[j].get(i + 1)), off2), l2), a, c);
                part = f2_add(part, f2_pack(ex2(a), ex2(c)));
            }
            s2 = f2_add(s2, part);
        }
        float s, s1;
        f2_unpack(s2, s, s1);
        s += s1;
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        __syncthreads();   // thr written, red read
        if (lane == 0) sm.red[warp] = s;

        // ---- collect the candidates from the threshold up, raising it while they
        // are more than the buffer holds (many equal logits, or the best ones side
        // by side in one group)
        uint64_t thr = static_cast<uint64_t>(sm.thr) << 32;
        if (thr == 0) thr = 1;   // fewer than M groups have one: all of them
        int n;
        while (true) {
            const float least = thr > 1 ? key_logit(thr) : -INFINITY;
            uint32_t hits = 0;
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (vmax[j] >= least && vmax[j] > -INFINITY) hits |= 1u << j;
            while (hits) {
                const int j = __ffs(hits) - 1;
                hits &= hits - 1;
                const int c = first + j * (kThreads * E);
                Pack<T, E> v;
                load_logits<T, ALIGNED>(v, z, c, p.V, lo, hi);
                const uint32_t allow = mask ? static_cast<uint32_t>(mask[c >> 5]) >> (c & 31) : 0xffffffffu;
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float x = v.get(i);
                    if (x >= least && x > -INFINITY && (allow >> i & 1u)) {
                        const uint64_t k = key_of(x, c + i);
                        if (k >= thr) {
                            const int to = atomicAdd(&sm.count, 1);
                            if (to < kCap) sm.buf[to] = k;
                        }
                    }
                }
            }
            __syncthreads();
            n = sm.count;
            if (n <= kCap) break;
            thr = mth_largest(sm.buf, kCap, p.M);
            __syncthreads();
            if (tid == 0) sm.count = 0;
            __syncthreads();
        }
        if (tid == 0) {
            float total = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) total += sm.red[w];
            p.stats[blockIdx.x] = make_float2(m, total);
        }
        uint64_t* out = p.keys + static_cast<int64_t>(row) * p.M * p.slices + slice;
        const uint64_t cut = n > kSmall ? mth_largest(sm.buf, n, p.M) : 0;
        // rank by counting: exact, and the keys are all different
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t k = sm.buf[i];
            if (k < cut) continue;
            int above = 0;
            for (int o = 0; o < n; ++o) above += sm.buf[o] > k ? 1 : 0;
            if (above < p.M) out[static_cast<int64_t>(above) * p.slices] = k;
        }
        for (int i = n + tid; i < p.M; i += kThreads) out[static_cast<int64_t>(i) * p.slices] = 0;
    }

    // ---- the sequence's last block goes on to pick
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        const unsigned all = static_cast<unsigned>(p.K) * static_cast<unsigned>(p.slices);
        const bool last = atomicAdd(&p.done[b], 1u) == all - 1;
        if (last) p.done[b] = 0;
        sm.last = last;
        __threadfence();
    }
    __syncthreads();
    if (sm.last) pick(p, sm, b);
}

// ------------------------------------------------------------------- host
lmloss_status check_beam(const lmloss_beam_args* a, bool pointers)
{
    if (!a) return LMLOSS_ERR_INVALID_ARG;
    if (a->B < 0 || a->V < 1 || a->ld < a->V) return LMLOSS_ERR_INVALID_ARG;
    if (a->K < 1 || a->K > LMLOSS_MAX_BEAMS || a->M < 1 || a->M > LMLOSS_MAX_BEAMS) return LMLOSS_ERR_INVALID_ARG;
    if (!float_dtype(a->dtype)) return LMLOSS_ERR_INVALID_ARG;
    if (!(a->length_penalty >= 0.f) || !std::isfinite(a->length_penalty)) return LMLOSS_ERR_INVALID_ARG;
    if (a->eos_token < -1 || a->eos_token >= a->V || a->mask_stride < 0) return LMLOSS_ERR_INVALID_ARG;
    if (a->V >= (int64_t(1) << 31) - 1 || a->B > (int64_t(1) << 24)) return LMLOSS_ERR_UNSUPPORTED;
    if (a->B > 0 && a->ld > INT64_MAX / 16 / (a->B * a->K)) return LMLOSS_ERR_INVALID_ARG;
    if (!pointers) return LMLOSS_OK;
    if (a->length_penalty > 0.f && !a->lengths) return LMLOSS_ERR_INVALID_ARG;
    if (a->lengths_out && !a->lengths) return LMLOSS_ERR_INVALID_ARG;
    if (a->finished && a->eos_token < 0) return LMLOSS_ERR_INVALID_ARG;
    if (a->token_mask && a->mask_stride != 0 && a->mask_stride < (a->V + 31) / 32) return LMLOSS_ERR_INVALID_ARG;
    if (a->B > 0) {
        if (!a->logits || !a->scores || !a->scores_out || !a->parents_out || !a->tokens_out)
            return LMLOSS_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(a->logits) % float_bytes(a->dtype)) return LMLOSS_ERR_INVALID_ARG;
    }
    return LMLOSS_OK;
}

constexpr int kMaxVpt = 8;

struct BeamPlan {
    int vpt, slices;
    size_t keys, stats, total;
};

// The slice length: 8 vectors a thread, or fewer while that leaves the GPU's
// SMs without two blocks each.
lmloss_status plan_beam(const lmloss_beam_args* a, int num_sms, BeamPlan& P)
{
    const int64_t rows = a->B * a->K, E = 16 / float_bytes(a->dtype);
    int vpt = kMaxVpt;
    int64_t slices = 0;
    for (;; vpt /= 2) {
        const int64_t len = static_cast<int64_t>(vpt) * kThreads * E;
        slices = (a->V + len - 1) / len;
        if (vpt == 1 || rows * slices >= 2 * num_sms) break;
    }
    while (slices * a->K > kMaxLists && vpt < kMaxVpt) {
        vpt *= 2;
        const int64_t len = static_cast<int64_t>(vpt) * kThreads * E;
        slices = (a->V + len - 1) / len;
    }
    if (slices * a->K > kMaxLists) return LMLOSS_ERR_UNSUPPORTED;
    if (rows * slices >= (int64_t(1) << 31)) return LMLOSS_ERR_UNSUPPORTED;
    P.vpt = vpt;
    P.slices = static_cast<int>(slices);
    P.keys = 0;
    P.stats = vocab_align(sizeof(uint64_t) * static_cast<size_t>(rows * slices * a->M));
    P.total = P.stats + vocab_align(sizeof(float2) * static_cast<size_t>(rows * slices));
    return LMLOSS_OK;
}

template <class T, int VPT>
lmloss_status launch_slices(const BeamParams& p, bool aligned, cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.K * p.slices);
    if (aligned) beam_step_kernel<T, VPT, true><<<grid, kThreads, 0, stream>>>(p);
    else beam_step_kernel<T, VPT, false><<<grid, kThreads, 0, stream>>>(p);
    return vocab_launch_err();
}

template <class T>
lmloss_status launch_slices(const BeamParams& p, int vpt, bool aligned, cudaStream_t stream)
{
    switch (vpt) {
    case 1: return launch_slices<T, 1>(p, aligned, stream);
    case 2: return launch_slices<T, 2>(p, aligned, stream);
    case 4: return launch_slices<T, 4>(p, aligned, stream);
    default: return launch_slices<T, 8>(p, aligned, stream);
    }
}

}  // namespace
}  // namespace lmloss

using namespace lmloss;

extern "C" {

lmloss_status lmloss_beam_check_args(const lmloss_beam_args* a) { return check_beam(a, true); }

lmloss_status lmloss_beam_workspace(const lmloss_beam_args* a, size_t* bytes)
{
    if (!bytes) return LMLOSS_ERR_INVALID_ARG;
    lmloss_status st = check_beam(a, false);
    if (st != LMLOSS_OK) return st;
    // the shortest slices that any GPU's plan takes: enough for every plan
    BeamPlan P{};
    if ((st = plan_beam(a, 1 << 20, P)) != LMLOSS_OK) return st;
    *bytes = P.total;
    return LMLOSS_OK;
}

lmloss_status lmloss_beam_step(lmloss_vocab_handle h, const lmloss_beam_args* a, cudaStream_t stream)
{
    if (!h) return LMLOSS_ERR_INVALID_ARG;
    lmloss_status st = check_beam(a, true);
    if (st != LMLOSS_OK) return st;
    BeamPlan P{};
    if ((st = plan_beam(a, h->num_sms, P)) != LMLOSS_OK) return st;
    if (P.total > h->ws_bytes) return LMLOSS_ERR_INVALID_ARG;
    if (a->B == 0) return LMLOSS_OK;
    VocabDeviceGuard g(h->device);
    if (!g.ok) return LMLOSS_ERR_CUDA;
    const bool aligned = aligned16(a->logits) && a->ld * float_bytes(a->dtype) % 16 == 0;
    // as many sequences a launch as there are counters
    for (int64_t b0 = 0; b0 < a->B; b0 += kVocabCounters) {
        const int64_t r0 = b0 * a->K, o0 = b0 * a->M;
        BeamParams p{};
        p.logits = static_cast<const unsigned char*>(a->logits) + r0 * a->ld * float_bytes(a->dtype);
        p.ld = a->ld;
        p.B = static_cast<int>(std::min<int64_t>(a->B - b0, kVocabCounters));
        p.K = a->K;
        p.M = a->M;
        p.V = static_cast<int>(a->V);
        p.slices = P.slices;
        p.alpha = a->length_penalty;
        p.eos = a->eos_token;
        p.scores = a->scores + r0;
        p.finished = a->finished ? a->finished + r0 : nullptr;
        p.lengths = a->lengths ? a->lengths + r0 : nullptr;
        p.mask = a->token_mask ? a->token_mask + r0 * a->mask_stride : nullptr;
        p.mask_stride = a->mask_stride;
        p.scores_out = a->scores_out + o0;
        p.parents_out = a->parents_out + o0;
        p.tokens_out = a->tokens_out + o0;
        p.lse_out = a->lse_out ? a->lse_out + r0 : nullptr;
        p.finished_out = a->finished_out ? a->finished_out + o0 : nullptr;
        p.lengths_out = a->lengths_out ? a->lengths_out + o0 : nullptr;
        p.keys = reinterpret_cast<uint64_t*>(h->ws + P.keys);
        p.stats = reinterpret_cast<float2*>(h->ws + P.stats);
        p.done = h->counters;
        switch (a->dtype) {
        case LMLOSS_BF16: st = launch_slices<Bf16>(p, P.vpt, aligned, stream); break;
        case LMLOSS_FP16: st = launch_slices<Fp16>(p, P.vpt, aligned, stream); break;
        default: st = launch_slices<Fp32>(p, P.vpt, aligned, stream); break;
        }
        if (st != LMLOSS_OK) return st;
    }
    return LMLOSS_OK;
}

}  // extern "C"
