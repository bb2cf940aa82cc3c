// Log-probabilities of given tokens over rows of logits, with the rows' entropies and
// their largest alternatives, and the gradient of the logits.
//
// With y = z / tau over the allowed columns, u = (z - m) log2(e) / tau and m the row's maximum:
//
//   s = sum 2^u,   e = sum u 2^u
//   lse = m / tau + ln s,   H = ln s - ln2 e / s,   logp_j = z[t_j] / tau - lse
//
// so one pass with a running maximum gives all of it: a part of a row keeps (m, s, e), and
// when m rises by d (in u's units) s becomes s 2^-d and e becomes (e - d s) 2^-d.  In place of m log2(e) / tau
// stands its fp32 value R, so that u is one fused operation; what R is off by goes into lse.  (Maxima for which R is off
// by more than 2 are taken off before the product.)
// Alternatives are kept as in a beam step: a threshold from group maxima, vectors noted against it.
//
// The gradient is one more pass, from m, ln s and H alone: p = e^((z - m) / tau - ln s), or, given only lse, e^(y - lse).
//
// 4096 x 128256 bf16: forward 172 us without alternatives (0.91 of the copy's rate), 183 with 5, 245 with 64, 429 where
// every row is summed again; the gradient with entropies 312 us (1.01).  One row of 128256 with 20 alternatives: 11 us, the latency of two dependent
// steps (a part's threshold and ranking, the join).  The forward is bound by memory and instructions together (64%
// of the issue slots: unpacking, maximum, ex2, two sums); alternatives add the work at a part's end, when few
// loads are on their way.  Rows at odd elements: 2048 x 128251, 118 us (0.66), by their shifts.
#include <algorithm>
#include <cmath>

#include "beam_math.cuh"
#include "beam_plan.cuh"
#include "row_stream.cuh"

namespace lmloss {
namespace {

constexpr int kMaxTop = LMLOSS_MAX_ALTERNATIVES;
constexpr int kCap = 1024;                   // candidate keys held at once
constexpr int kHits = 1024;                  // vectors of a part that reach its first threshold
constexpr int kSmall = 256;                  // few enough to be ranked by counting
constexpr int kMaxParts = 4096;              // parts of all rows, where rows are cut
constexpr float kLeast = -1000.f;            // an exponent whose power is 0: 0 * -inf would be NaN
constexpr double kLn2 = 0.693147180559945309417;

struct LogprobsParams {
    const void* logits;
    int64_t ld;
    int T, V;
    int64_t n;
    int M;
    int slices, tiles;           // parts of a row, tiles of a part
    float mul;                   // log2(e) / tau
    float near, counted;         // 2^26 and 2^27 over mul: see usual and counts
    double inv_tau;
    const void* tokens;
    int ids32;
    const int32_t* mask;
    int64_t mask_stride;
    float* logp_out;
    float* lse_out;
    float* entropy_out;
    float* top_logp_out;
    int64_t* top_tokens_out;
    float* row_max_out;
    float* log_sum_out;
    uint64_t* keys;              // [T][slices][M] where rows are cut: each part's best, 0 = none
    float4* stats;               // [T][slices] (m, s, e, -)
    unsigned* done;              // [T] parts finished; 0 between calls
    int* err;
};

__device__ __forceinline__ int64_t load_token(const void* tokens, int ids32, int64_t i)
{
    return ids32 ? static_cast<int64_t>(static_cast<const int32_t*>(tokens)[i]) : static_cast<const int64_t*>(tokens)[i];
}

__device__ __forceinline__ bool allowed(const int32_t* mask, int c)
{
    return !mask || (static_cast<uint32_t>(mask[c >> 5]) >> (c & 31) & 1u);
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A running sum of 2^u and u 2^u about r, the fp32 value of the maximum in base 2.
struct Sums {
    float r = -INFINITY, s = 0.f, e = 0.f;
    __device__ __forceinline__ void raise(float top)
    {
        if (top > r) {
            // (from -inf: s and e are 0)
            const float d = fmaxf(r - top, kLeast), f = ex2(d);
            e = fmaf(s, d, e) * f;
            s *= f;
            r = top;
        }
    }
};

// Whether a part's sums may go about R = fl(m mul).  What R is off, half of its last place at most, stands in every
// exponent: from m mul = 2^30 on 2^(m mul - R) leaves fp32's range, and well before the entropy loses its last places, as
// ln s and e / s both hold it.  Up to 2^26 (logits of 46 at a temperature of 1e-6) it is 2 at most.  Parts of larger maxima
// are summed again, by sum_slowly.
__device__ __forceinline__ bool usual(const LogprobsParams& p, float m) { return fabsf(m) < p.near; }
// Whether a thread's or a warp's logits count yet.  Those of a lower maximum than -2^27 / mul are left out: they lie 2^26 below
// any maximum that is usual, and the others' parts are summed again.
__device__ __forceinline__ bool counts(const LogprobsParams& p, float m) { return fabsf(m) < p.counted; }

// Of bf16 -2^100 stands in the place of -inf (and of what lies below) in the sum of u 2^u: nothing beside a maximum that
// counts.
template <class T>
__device__ __forceinline__ uint32_t floor_pair(uint32_t w)
{
    if constexpr (T::kIndex == Bf16::kIndex) {
        const uint32_t least = 0xf180f180u;
        const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&least));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    return w;
}

// Largest of several vectors' logits; NaN are passed over here and show up in the sum.
template <class T, int VPT>
__device__ __forceinline__ float largest_of(const Pack<T, Logits<T>::E> (&q)[VPT])
{
    if constexpr (T::kBytes == 4) {
        float r = Logits<T>::largest(q[0]);
#pragma unroll
        for (int j = 1; j < VPT; ++j) r = fmaxf(r, Logits<T>::largest(q[j]));
        return r;
    } else {
        using H2 = typename std::conditional<std::is_same<T, Bf16>::value, __nv_bfloat162, __half2>::type;
        H2 r = *reinterpret_cast<const H2*>(&q[0].w[0]);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) r = __hmax2(r, *reinterpret_cast<const H2*>(&q[j].w[i]));
        const uint32_t w = *reinterpret_cast<const uint32_t*>(&r);
        return fmaxf(T::widen(static_cast<uint16_t>(w & 0xffffu)), T::widen(static_cast<uint16_t>(w >> 16)));
    }
}

// For each of 8 (fp32: 4) bits all ones or zeros over its element, as words.
template <int BYTES>
__device__ __forceinline__ void spread_bits(uint32_t allow, uint32_t (&keep)[4])
{
    // bit k of four to the top of byte k, then the byte's top bit over whole bytes
    auto prmt = [](uint32_t x, uint32_t sel) {
        uint32_t r;
        asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(x), "r"(sel));
        return r;
    };
    const uint32_t low = (allow & 15u) * 0x10204080u;
    if (BYTES == 4) {
        keep[0] = prmt(low, 0x8888u);
        keep[1] = prmt(low, 0x9999u);
        keep[2] = prmt(low, 0xaaaau);
        keep[3] = prmt(low, 0xbbbbu);
    } else {
        const uint32_t high = (allow >> 4 & 15u) * 0x10204080u;
        keep[0] = prmt(low, 0x9988u);
        keep[1] = prmt(low, 0xbbaau);
        keep[2] = prmt(high, 0x9988u);
        keep[3] = prmt(high, 0xbbaau);
    }
}

// rank_groups for this kernel: the same groups, but a group's number stands in its maximum's low bits, which makes
// them all different at the price of a threshold that much lower, and two or four threads share the counting of
// one of 64 or 128 groups.  (Of 128 groups counted by a thread each the ranking took 1.6 us.)
__device__ __forceinline__ void rank_keys(uint32_t v, int M, uint32_t* group, uint32_t* thr)
{
    const int tid = threadIdx.x;
    const int groups = M <= 16 ? 32 : (M <= 32 ? 64 : 128), gt = kThreads / groups;
    v = max(v, __shfl_xor_sync(0xffffffffu, v, 1));
    if (gt >= 4) v = max(v, __shfl_xor_sync(0xffffffffu, v, 2));
    if (gt >= 8) v = max(v, __shfl_xor_sync(0xffffffffu, v, 4));
    const uint32_t mine = (v & ~127u) | static_cast<uint32_t>(127 - tid / gt);
    if ((tid & (gt - 1)) == 0) group[tid / gt] = mine;
    __syncthreads();
    // a group's gt threads (8, 4 or 2) count a part of the others each
    const int part = groups / gt, from = (tid & (gt - 1)) * part;
    int above = 0;
#pragma unroll 4
    for (int i = 0; i < part; i += 4) {
        const uint4 o = *reinterpret_cast<const uint4*>(group + from + i);
        above += (o.x > mine ? 1 : 0) + (o.y > mine ? 1 : 0) + (o.z > mine ? 1 : 0) + (o.w > mine ? 1 : 0);
    }
    above += __shfl_xor_sync(0xffffffffu, above, 1);
    if (gt >= 4) above += __shfl_xor_sync(0xffffffffu, above, 2);
    if (gt >= 8) above += __shfl_xor_sync(0xffffffffu, above, 4);
    if (above == M - 1 && (tid & (gt - 1)) == 0 && mine > 127u) *thr = mine & ~127u;
}

struct __align__(16) LogprobsShared {
    uint64_t buf[kCap];                      // candidates
    uint4 data[kHits];                       // noted vectors
    int32_t col[kHits];
    uint64_t best[kMaxTop];                  // the part's or row's best, in order
    uint32_t group[kThreads / 2], counts[kThreads];
    uint32_t thr, thr_end;
    float red_m[kWarps], red_s[kWarps], red_e[kWarps];
    int count, hit_count, few, last;
    uint64_t cut;
    double lse;
};

// The M best of n candidates (all different) into sm.best, best first, 0 where there are none.  `few` has
// room for M of them.
__device__ __noinline__ void rank_best(LogprobsShared& sm, const uint64_t* set, uint64_t* few, int n, int M)
{
    const int tid = threadIdx.x;
    const uint64_t cut = n > kSmall ? mth_largest(set, n, M, sm.counts) : 0;
    if (cut) {
        for (int i = tid; i < n; i += kThreads)
            if (set[i] >= cut) few[atomicAdd(&sm.few, 1)] = set[i];
        __syncthreads();
        n = M;
        set = few;
    }
    for (int i = tid; i < n; i += kThreads) {
        const uint64_t k = set[i];
        int above = 0;
#pragma unroll 8
        for (int o = 0; o < n; ++o) above += set[o] > k ? 1 : 0;
        if (above < M) sm.best[above] = k;
    }
    for (int i = n + tid; i < M; i += kThreads) sm.best[i] = 0;
    __syncthreads();
}

// What R = fl(m mul) is off from m mul, which the sums of a part about R hold: exact.  0 for sums about m itself.
__device__ __forceinline__ float off_by(const LogprobsParams& p, float m)
{
    return usual(p, m) ? fmaf(-m, p.mul, __fmul_rn(m, p.mul)) : 0.f;
}

// A row's statistics from its maximum and sums, by one thread.
__device__ __forceinline__ void write_sums(const LogprobsParams& p, LogprobsShared& sm, int row, float m, float hi, float lo, float e)
{
    const bool none = m == -INFINITY && hi == 0.f;
    const double log_s = none ? -INFINITY : (m == INFINITY ? NAN : log_of_sum(hi, lo));
    const double log_sum = log_s + kLn2 * static_cast<double>(off_by(p, m));
    const double lse = static_cast<double>(m) * p.inv_tau + log_sum;
    sm.lse = lse;
    if (p.lse_out) p.lse_out[row] = static_cast<float>(lse);
    if (p.entropy_out) p.entropy_out[row] = none ? 0.f : static_cast<float>(log_s - kLn2 * static_cast<double>(e / hi));
    if (p.row_max_out) p.row_max_out[row] = m;
    if (p.log_sum_out) p.log_sum_out[row] = static_cast<float>(log_sum);
}

// Given token j of a row: what stands for its log-probability until lse is known.
struct Given {
    float z;
    int kind;                    // 0 a logit, 1 none, 2 not in the vocabulary
};
template <class T>
__device__ __forceinline__ Given load_given(const LogprobsParams& p, int row, int64_t j)
{
    const int64_t t = load_token(p.tokens, p.ids32, static_cast<int64_t>(row) * p.n + j);
    Given g{0.f, t == LMLOSS_IGNORE_INDEX ? 1 : (t < 0 || t >= p.V ? 2 : 0)};
    if (g.kind == 0) {
        const typename T::raw* z = static_cast<const typename T::raw*>(p.logits) + static_cast<int64_t>(row) * p.ld;
        const int32_t* mask = p.mask ? p.mask + row * p.mask_stride : nullptr;
        g.z = allowed(mask, static_cast<int>(t)) ? T::widen(z[t]) : -INFINITY;
    }
    return g;
}

// What follows a row's statistics: its given tokens (each thread's first one is there already) and, from sm.best,
// alternatives.  After a barrier that follows write_sums and rank_best.
template <class T>
__device__ __forceinline__ void write_row(const LogprobsParams& p, LogprobsShared& sm, int row, Given first)
{
    const int tid = threadIdx.x;
    const double lse = sm.lse;
    for (int64_t j = tid; j < p.n; j += kThreads) {
        const Given g = j == tid ? first : load_given<T>(p, row, j);
        float out = lse == -INFINITY ? -INFINITY : static_cast<float>(static_cast<double>(g.z) * p.inv_tau - lse);
        if (g.kind == 1) out = 0.f;
        if (g.kind == 2) {
            set_error(p.err, kErrBadTarget);
            out = NAN;
        }
        p.logp_out[static_cast<int64_t>(row) * p.n + j] = out;
    }
    for (int i = tid; i < p.M; i += kThreads) {
        const uint64_t k = sm.best[i];
        const int64_t o = static_cast<int64_t>(row) * p.M + i;
        // a row with NaN or +inf has an lse of NaN
        const bool some = k != 0 && lse == lse && key_logit(k) < INFINITY;
        p.top_logp_out[o] = some ? static_cast<float>(static_cast<double>(key_logit(k)) * p.inv_tau - lse) : -INFINITY;
        p.top_tokens_out[o] = some ? key_col(k) : LMLOSS_IGNORE_INDEX;
    }
}

// The block that finishes a row's last part joins the parts.
template <class T>
__device__ __noinline__ void join_row(const LogprobsParams& p, LogprobsShared& sm, int row, Given first)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = p.slices, M = p.M;
    // the candidates on their way beside the sums
    const uint64_t* const keys = p.keys + static_cast<int64_t>(row) * S * M;
    uint64_t head = 0, mine[8];
    if (M > 0 && tid < S) head = __ldcg(keys + static_cast<int64_t>(tid) * M);
#pragma unroll
    for (int i = 0; i < 8; ++i) mine[i] = tid + i * kThreads < S * M ? __ldcg(keys + tid + i * kThreads) : 0;
    // sums: error-free pairs of fp32
    float m = -INFINITY, hi = 0.f, lo = 0.f, e = 0.f;
    if (warp == 0) {
        const float4* st = p.stats + static_cast<int64_t>(row) * S;
        for (int s = lane; s < S; s += 32) m = fmaxf(m, __ldcg(&st[s]).x);
        m = warp_max(m);
        auto add = [&](float x, float err) {
            const float t = hi + x, v = t - hi;
            lo += ((hi - (t - v)) + (x - v)) + err;
            hi = t;
        };
        for (int s = lane; s < S; s += 32) {
            const float4 q = __ldcg(&st[s]);
            // (of two values of R the difference is exact where it matters; next to where sums go about m itself what R is off counts)
            const float apart = usual(p, q.x) && usual(p, m) ? __fmul_rn(q.x, p.mul) - __fmul_rn(m, p.mul)
                                                             : (q.x - m) * p.mul + (off_by(p, q.x) - off_by(p, m));
            const float d = q.x == m ? 0.f : fmaxf(apart, kLeast), f = exp2f(d);
            add(q.y * f, 0.f);
            e += fmaf(q.y, d, q.z) * f;
        }
        for (int o = 16; o > 0; o >>= 1) {
            const float x = __shfl_xor_sync(0xffffffffu, hi, o), y = __shfl_xor_sync(0xffffffffu, lo, o);
            add(x, y);
            e += __shfl_xor_sync(0xffffffffu, e, o);
        }
    }
    if (tid == 0) write_sums(p, sm, row, m, hi, lo, e);
    if (M > 0) {
        const int all = S * M;
        uint64_t* const held = reinterpret_cast<uint64_t*>(sm.data);
        if (tid == 0) sm.count = sm.few = 0;
        // candidates: below the M-th largest of the parts' best there are none
        constexpr int kMine = 8;
        uint64_t thr = 1;
        bool done = false;
        if (all <= kMine * kThreads && S <= kThreads) {
            if (tid < S) sm.buf[tid] = head;
            if (tid == 0) sm.cut = 1;
            __syncthreads();
            if (S > M && tid < S) {
                int above = 0;
#pragma unroll 4
                for (int o = 0; o < S; ++o) above += sm.buf[o] > head ? 1 : 0;
                if (above == M - 1 && head) sm.cut = head;   // (equal ones are parts without a candidate)
            }
            __syncthreads();
            thr = sm.cut;
#pragma unroll
            for (int i = 0; i < kMine; ++i)
                if (mine[i] >= thr) {
                    const int to = atomicAdd(&sm.count, 1);
                    if (to < kCap) held[to] = mine[i];
                }
            __syncthreads();
            done = sm.count <= kCap;
        }
        const uint64_t* set = held;
        if (!done) {
            set = sm.buf;
            while (true) {
                __syncthreads();
                if (tid == 0) sm.count = 0;
                __syncthreads();
                for (int i = tid; i < all; i += kThreads) {
                    const uint64_t k = __ldcg(keys + i);
                    if (k >= thr) {
                        const int to = atomicAdd(&sm.count, 1);
                        if (to < kCap) sm.buf[to] = k;
                    }
                }
                __syncthreads();
                if (sm.count <= kCap) break;
                thr = mth_largest(sm.buf, kCap, M, sm.counts);
            }
        }
        rank_best(sm, set, set == held ? sm.buf : held, sm.count, M);
    } else {
        __syncthreads();
    }
    write_row<T>(p, sm, row, first);
}

// A part whose maximum is finite and not usual: 2^u about the maximum itself, taken off before the product.  Each warp's
// sums into its place.
template <class T, bool ALIGNED>
__device__ __noinline__ void sum_slowly(const LogprobsParams& p, LogprobsShared& sm, const RowLogits<T> r, const int32_t* mask, int begin, int end,
                                        float top)
{
    constexpr int E = Logits<T>::E;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float s = 0.f, e = 0.f;
#pragma unroll 2
    for (int c = begin + tid * E; c < end; c += kThreads * E) {
        Pack<T, E> q;
        load_logits<T, ALIGNED>(q, r, c);
        const uint32_t allow = mask ? static_cast<uint32_t>(mask[c >> 5]) >> (c & 31) : 0xffffffffu;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float z = allow >> i & 1u ? q.get(i) : -INFINITY, u = max_nan((z - top) * p.mul, kLeast), w = ex2(u);
            s += w;
            e = fmaf(w, u, e);
        }
    }
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        e += __shfl_xor_sync(0xffffffffu, e, o);
    }
    __syncthreads();   // everyone has read the maxima
    if (lane == 0) {
        sm.red_m[warp] = top;
        sm.red_s[warp] = s;
        sm.red_e[warp] = e;
    }
    __syncthreads();
}

// A block takes `tiles` tiles of one row, one after the other, with the next tile's loads in
// flight; columns, not addresses, fix which thread adds what.
template <class T, int VPT, bool ALIGNED, bool ENT>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const __grid_constant__ LogprobsParams p)
{
    constexpr int E = Logits<T>::E;
    constexpr int kTileCols = VPT * kThreads * E;
    constexpr uint32_t kNone = T::kBytes == 4 ? 0xff800000u : (std::is_same<T, Bf16>::value ? 0xff80ff80u : 0xfc00fc00u);
    __shared__ LogprobsShared sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / p.slices, part = blockIdx.x - row * p.slices;
    RowLogits<T> r;
    r.z = static_cast<const typename T::raw*>(p.logits) + static_cast<int64_t>(row) * p.ld;
    r.V = p.V;
    r.lo = 0;
    r.hi = p.V - E;
    if (!ALIGNED) {
        // at the first and last row: nothing before or after the logits is read
        const int64_t after = (static_cast<int64_t>(p.T) - 1 - row) * p.ld;
        if (row == 0) r.lo = E;
        if (after < E) r.hi = p.V - 2 * E;
    }
    const int32_t* mask = p.mask ? p.mask + row * p.mask_stride : nullptr;
    const int begin = part * p.tiles * kTileCols, end = part_end(begin, p.tiles, kTileCols, p.V);
    if (tid == 0) {
        sm.count = 0;
        sm.hit_count = 0;
        sm.few = 0;
        sm.thr = 0;
        sm.thr_end = 0;
    }
    const Given first = tid < p.n ? load_given<T>(p, row, tid) : Given{0.f, 1};   // under the way of the row
    Sums sum;
    float m = -INFINITY, least = 0.f;   // m: the thread's largest allowed logit
    int tile = 0;
    auto use_tile = [&](Pack<T, E> (&q)[VPT], int c0) {
        if (mask) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = c0 + j * (kThreads * E);
                uint32_t keep[4];
                spread_bits<T::kBytes>(c < p.V ? static_cast<uint32_t>(mask[c >> 5]) >> (c & 31) : 0u, keep);
#pragma unroll
                for (int i = 0; i < 4; ++i) q[j].w[i] = (q[j].w[i] & keep[i]) | (kNone & ~keep[i]);
            }
        }
        const float tmax = largest_of<T, VPT>(q);
        m = fmaxf(m, tmax);
        bool raise = false;
        if (p.M > 0) {
            // tiles 0, 1, 3, 7, ... raise the threshold; where ranking takes longer, 0, 3, 15, ...
            raise = (tile & (tile + 1)) == 0 && (p.M <= 16 || !(tile & 1) || (0x55555555 & (tile + 1)) != 0);
            ++tile;
            if (raise) rank_keys(m > -INFINITY ? ordered(m == 0.f ? 0.f : m) : 0u, p.M, sm.group, &sm.thr);
        }
        sum.raise(counts(p, m) ? __fmul_rn(m, p.mul) : -INFINITY);
        const float less = sum.r == -INFINITY ? 0.f : -sum.r;
        const uint64_t less2 = f2_pack(less, less), mul2 = f2_pack(p.mul, p.mul);
        uint64_t s2 = f2_pack(0.f, 0.f), e2 = f2_pack(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            Pack<T, E> y = q[j];
            if (ENT) {
#pragma unroll
                for (int i = 0; i < 4; ++i) y.w[i] = floor_pair<T>(y.w[i]);
            }
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const uint64_t u2 = f2_fma(f2_pack(y.get(i), y.get(i + 1)), mul2, less2);
                float a, c;
                f2_unpack(u2, a, c);
                const uint64_t w2 = f2_pack(ex2(a), ex2(c));
                s2 = f2_add(s2, w2);
                if (ENT) e2 = f2_fma(w2, T::kIndex == Bf16::kIndex ? u2 : f2_pack(max_nan(a, kLeast), max_nan(c, kLeast)), e2);
            }
        }
        float a, c;
        f2_unpack(s2, a, c);
        sum.s += a + c;
        if (ENT) {
            f2_unpack(e2, a, c);
            sum.e += a + c;
        }
        if (p.M > 0) {
            if (raise) {
                __syncthreads();   // the threshold; without one every logit but -inf
                least = sm.thr ? unordered(sm.thr) : __uint_as_float(0xff7fffffu);
            }
            if (tmax >= least) {
#pragma unroll
                for (int j = 0; j < VPT; ++j)
                    if (Logits<T>::largest(q[j]) >= least) {
                        const int to = atomicAdd(&sm.hit_count, 1);
                        if (to < kHits) {
                            sm.data[to] = make_uint4(q[j].w[0], q[j].w[1], q[j].w[2], q[j].w[3]);
                            sm.col[to] = c0 + j * (kThreads * E);
                        }
                    }
            }
        }
    };
    int t0 = begin;
    auto whole_tiles = [&] {
        InFlight<T, ALIGNED> next[VPT];
        auto issue = [&](int c) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) next[j].load(r, c + (j * kThreads + tid) * E);
        };
        const int last = min(end, r.hi + E) - kTileCols;   // the last whole tile begins here or before
        if (t0 <= last) issue(t0);
        for (; t0 <= last; t0 += kTileCols) {
            Pack<T, E> q[VPT];
#pragma unroll
            for (int j = 0; j < VPT; ++j) next[j].unpack(q[j], r, t0 + (j * kThreads + tid) * E);
            if (t0 + kTileCols <= last) issue(t0 + kTileCols);
            use_tile(q, t0 + tid * E);
        }
    };
    __syncthreads();
    for (bool before = true;; before = false) {
        const int to = before ? min(r.lo, end) : end;
        for (; t0 < to; t0 += kTileCols) {
            Pack<T, E> q[VPT];
#pragma unroll
            for (int j = 0; j < VPT; ++j) load_logits<T, ALIGNED>(q[j], r, t0 + (j * kThreads + tid) * E);
            use_tile(q, t0 + tid * E);
        }
        if (!before) break;
        whole_tiles();
    }

    // ---- the part's sums
    {
        const float top = warp_max(m);
        sum.raise(counts(p, top) ? __fmul_rn(top, p.mul) : -INFINITY);
        for (int o = 16; o > 0; o >>= 1) {
            sum.s += __shfl_xor_sync(0xffffffffu, sum.s, o);
            if (ENT) sum.e += __shfl_xor_sync(0xffffffffu, sum.e, o);
        }
        if (lane == 0) {
            sm.red_m[warp] = top;
            sm.red_s[warp] = sum.s;
            sm.red_e[warp] = sum.e;
        }
    }
    if (p.M > 0) rank_keys(m > -INFINITY ? ordered(m == 0.f ? 0.f : m) : 0u, p.M, sm.group, &sm.thr_end);
    __syncthreads();
    float top = sm.red_m[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm.red_m[w]);
    if (!usual(p, top) && fabsf(top) < INFINITY) sum_slowly<T, ALIGNED>(p, sm, r, mask, begin, end, top);
    if (warp == 0) {
        Sums w;
        const float mw = lane < kWarps ? sm.red_m[lane] : -INFINITY;
        w.r = usual(p, top) ? __fmul_rn(mw, p.mul) : mw;
        w.s = lane < kWarps ? sm.red_s[lane] : 0.f;
        w.e = lane < kWarps ? sm.red_e[lane] : 0.f;
        w.raise(usual(p, top) ? __fmul_rn(top, p.mul) : top);
        for (int o = 4; o > 0; o >>= 1) {
            w.s += __shfl_xor_sync(0xffffffffu, w.s, o);
            w.e += __shfl_xor_sync(0xffffffffu, w.e, o);
        }
        if (lane == 0) {
            if (p.slices > 1) p.stats[blockIdx.x] = make_float4(top, w.s, w.e, 0.f);
            else write_sums(p, sm, row, top, w.s, 0.f, w.e);
        }
    }

    if (p.M > 0) {
        // ---- candidates: the logits of the noted vectors that reach the threshold.  With more
        // vectors noted than are kept all are looked at; with more candidates than are kept the
        // threshold rises to the M-th largest of those held.
        uint64_t thr = sm.thr_end ? static_cast<uint64_t>(sm.thr_end) << 32 : 1;
        int n;
        while (true) {
            const int noted = sm.hit_count;
            const bool all = noted > kHits;
            const int elements = all ? end - begin : noted * E;
#pragma unroll 1
            for (int i = tid; i < elements; i += kThreads) {
                const int c = all ? begin + i : sm.col[i / E] + i % E;
                const float z = T::widen(all ? r.z[c] : reinterpret_cast<const typename T::raw*>(&sm.data[i / E])[i % E]);
                // past V: -inf
                if (z > -INFINITY && allowed(mask, c)) {
                    const uint64_t k = key_of(z, c);
                    if (k >= thr) {
                        const int to = atomicAdd(&sm.count, 1);
                        if (to < kCap) sm.buf[to] = k;
                    }
                }
            }
            __syncthreads();
            n = sm.count;
            if (n <= kCap) break;
            thr = mth_largest(sm.buf, kCap, p.M, sm.counts);
            __syncthreads();
            if (tid == 0) sm.count = 0;
            __syncthreads();
        }
        rank_best(sm, sm.buf, reinterpret_cast<uint64_t*>(sm.data), n, p.M);
        if (p.slices > 1) {
            uint64_t* out = p.keys + static_cast<int64_t>(blockIdx.x) * p.M;
            for (int i = tid; i < p.M; i += kThreads) out[i] = sm.best[i];
        }
    }
    if (p.slices == 1) {
        if (p.M == 0) __syncthreads();
        write_row<T>(p, sm, row, first);
        return;
    }
    __syncthreads();
    if (tid == 0) {
        sm.last = count_done(&p.done[row]) == static_cast<unsigned>(p.slices) - 1;
        if (sm.last) p.done[row] = 0;
    }
    __syncthreads();
    if (sm.last) join_row<T>(p, sm, row, first);
}

// ---------------------------------------------------------------- gradient
struct GradParams {
    const void* logits;
    int64_t ld;
    int T, V;
    int n;
    int parts, loops;            // parts of a row; a part is loops * kGradVecs * kThreads vectors
    float tau_inv, tau_inv_lo;   // 1 / tau as an fp32 pair
    const void* tokens;
    int ids32;
    const int32_t* mask;
    int64_t mask_stride;
    const float* row_max;        // with log_sum; NULL: 0, with lse
    const float* less;           // log_sum, or lse
    const float* entropy;
    const float* grad_logp;
    const float* grad_entropy;
    void* grad;
    int64_t ld_grad;
    int* err;
};

constexpr int kGradVecs = 4;     // vectors a thread, on their way together

struct __align__(16) GradShared {
    int32_t token[LMLOSS_MAX_GIVEN];         // -1 = none
    float g[LMLOSS_MAX_GIVEN], z[LMLOSS_MAX_GIVEN];
    float red[kWarps];
};

// -p (sum g + gH (ln p + H)) / tau for the columns without a given token's own part, p = e^d, d = (z - m) / tau - less: m the
// row's maximum and less its ln s, or 0 and lse.  lse alone has 2^-24 of itself for all that p is to be known by:
// nothing at temperatures near 1e-6.  The difference is taken in two fused operations, 1 / tau as a pair, before the
// change to base 2: of rows at the type's lowest values it is all that is left.
template <bool ENT>
struct GradColumn {
    float tau_inv, tau_inv_lo, max, less, base, ge;
    __device__ __forceinline__ GradColumn(const GradParams& p, float m, float less, float sum, float h, float gh)
        : tau_inv(p.tau_inv), tau_inv_lo(p.tau_inv_lo), max(-m), less(-less), base(-(ENT ? fmaf(gh, h, sum) : sum) * p.tau_inv), ge(-gh * p.tau_inv)
    {
    }
    __device__ __forceinline__ void two(float& a, float& c) const
    {
        f2_unpack(f2_add(f2_pack(a, c), f2_pack(max, max)), a, c);
        // (-inf takes no second product, and 0 * -inf would be NaN)
        const uint64_t d2 = f2_fma(f2_pack(max_nan(a, -3.402823466e38f), max_nan(c, -3.402823466e38f)), f2_pack(tau_inv_lo, tau_inv_lo),
                                   f2_fma(f2_pack(a, c), f2_pack(tau_inv, tau_inv), f2_pack(less, less)));
        float da, dc, ua, uc;
        f2_unpack(d2, da, dc);
        if (ENT) {
            da = max_nan(da, kLeast);
            dc = max_nan(dc, kLeast);
        }
        f2_unpack(f2_mul(f2_pack(da, dc), f2_pack(kLog2e, kLog2e)), ua, uc);
        const uint64_t by2 = ENT ? f2_fma(f2_pack(ge, ge), f2_pack(da, dc), f2_pack(base, base)) : f2_pack(base, base);
        f2_unpack(f2_mul(f2_pack(ex2(ua), ex2(uc)), by2), a, c);
    }
    __device__ __forceinline__ float one(float a) const
    {
        float c = a;
        two(a, c);
        return a;
    }
};

// Columns [c, c + E) of a row that reach past its ends, or past what may be read: one by one.
template <class T, bool ENT>
__device__ __noinline__ void grad_ends(const GradColumn<ENT>& f, const typename T::raw* z, typename T::raw* g, const int32_t* mask, int64_t c, int V,
                                       bool none)
{
    for (int i = 0; i < Logits<T>::E; ++i)
        if (c + i >= 0 && c + i < V) {
            const bool in = !none && allowed(mask, static_cast<int>(c) + i);
            g[c + i] = static_cast<typename T::raw>(T::round(in ? f.one(T::widen(z[c + i])) : 0.f));
        }
}

// A thread's vectors start on 16-byte boundaries of the row that it writes; SAME: the logits' do too.  Given tokens'
// columns are written again at the end, from logits looked at before anything is written (it may be in place).
template <class T, bool ENT, bool SAME>
__global__ void __launch_bounds__(kThreads) logprobs_grad_kernel(const __grid_constant__ GradParams p)
{
    constexpr int E = Logits<T>::E;
    using raw = typename T::raw;
    __shared__ GradShared sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / p.parts, part = blockIdx.x - row * p.parts;
    const raw* z = static_cast<const raw*>(p.logits) + static_cast<int64_t>(row) * p.ld;
    raw* g = static_cast<raw*>(p.grad) + static_cast<int64_t>(row) * p.ld_grad;
    const int32_t* mask = p.mask ? p.mask + row * p.mask_stride : nullptr;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(g) & 15u) / T::kBytes);   // columns of the first vector before the row
    const int per = p.loops * kGradVecs * kThreads;
    const int64_t c0 = static_cast<int64_t>(part) * per * E - off, c_end = min(c0 + static_cast<int64_t>(per) * E, static_cast<int64_t>(p.V));
    const float less = p.less[row], row_max = p.row_max ? p.row_max[row] : 0.f;
    const bool none = less == -INFINITY;

    // ---- the first vectors on their way, then the given tokens: the sum of their gradients
    uint4 x[kGradVecs];
    uint32_t w5[SAME ? 1 : kGradVecs];   // what unaligned logits need beside
    // (unaligned: the words around the columns, inside the call's logits)
    const int64_t safe_lo = SAME || row > 0 ? 0 : 2, safe_hi = SAME || row < p.T - 1 ? p.V : p.V - 2;
    auto whole = [&](int64_t c) { return c >= safe_lo && c + E <= safe_hi; };
    auto load = [&](int64_t first) {
#pragma unroll
        for (int k = 0; k < kGradVecs; ++k) {
            const int64_t c = first + static_cast<int64_t>(k * kThreads + tid) * E;
            if (!whole(c)) continue;
            if constexpr (SAME) {
                x[k] = *reinterpret_cast<const uint4*>(z + c);
            } else {
                const uint32_t* a = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(z + c) & ~uintptr_t(3));
                x[k] = make_uint4(a[0], a[1], a[2], a[3]);
                w5[k] = T::kBytes == 4 ? 0u : a[4];
            }
        }
    };
    load(c0);
    float sum = 0.f;
    for (int j = tid; j < p.n; j += kThreads) {
        const int64_t o = static_cast<int64_t>(row) * p.n + j, t = load_token(p.tokens, p.ids32, o);
        const bool in = t >= 0 && t < p.V;
        if (!in && t != LMLOSS_IGNORE_INDEX) set_error(p.err, kErrBadTarget);
        const float y = in ? p.grad_logp[o] : 0.f;
        const bool here = in && t >= c0 && t < c_end;
        sm.token[j] = here ? static_cast<int>(t) : -1;
        sm.g[j] = y;
        sm.z[j] = here ? T::widen(z[t]) : 0.f;
        sum += y;
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sm.red[warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sm.red[w];
    const GradColumn<ENT> f(p, row_max, less, sum, ENT ? p.entropy[row] : 0.f, ENT ? p.grad_entropy[row] : 0.f);

    for (int64_t first = c0; first < c_end; first += kGradVecs * kThreads * E) {
        if (first != c0) load(first);
#pragma unroll
        for (int k = 0; k < kGradVecs; ++k) {
            const int64_t c = first + static_cast<int64_t>(k * kThreads + tid) * E;
            if (c >= p.V) break;
            if (!whole(c)) {
                grad_ends<T, ENT>(f, z, g, mask, c, p.V, none);
                continue;
            }
            Pack<T, E> q;
            q.w[0] = x[k].x; q.w[1] = x[k].y; q.w[2] = x[k].z; q.w[3] = x[k].w;
            if constexpr (!SAME && T::kBytes == 2) {
                const uint32_t sh = (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(z + c)) & 2u) * 8u;
                q.w[0] = __funnelshift_r(x[k].x, x[k].y, sh);
                q.w[1] = __funnelshift_r(x[k].y, x[k].z, sh);
                q.w[2] = __funnelshift_r(x[k].z, x[k].w, sh);
                q.w[3] = __funnelshift_r(x[k].w, w5[k], sh);
            }
            float out[E];
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                out[i] = q.get(i);
                out[i + 1] = q.get(i + 1);
                f.two(out[i], out[i + 1]);
            }
            if (none) {
#pragma unroll
                for (int i = 0; i < E; ++i) out[i] = 0.f;
            }
            q.set_all(out);
            if (mask) {
                // (rows begin inside a vector: its columns may lie in two words)
                const int b = static_cast<int>(c);
                const uint32_t m0 = static_cast<uint32_t>(mask[b >> 5]), m1 = ((b + E - 1) >> 5) != (b >> 5) ? static_cast<uint32_t>(mask[(b >> 5) + 1]) : 0u;
                uint32_t keep[4];
                spread_bits<T::kBytes>(__funnelshift_r(m0, m1, b & 31), keep);
#pragma unroll
                for (int i = 0; i < 4; ++i) q.w[i] &= keep[i];
            }
            q.store(g + c);
        }
    }
    if (none || p.n == 0) return;
    __syncthreads();
    for (int j = tid; j < p.n; j += kThreads) {
        const int t = sm.token[j];
        if (t < 0 || !allowed(mask, t)) continue;
        // the first of equal tokens adds them all
        bool before = false;
        for (int i = 0; i < j; ++i) before = before || sm.token[i] == t;
        if (before) continue;
        float own = sm.g[j];
        for (int i = j + 1; i < p.n; ++i)
            if (sm.token[i] == t) own += sm.g[i];
        g[t] = static_cast<raw>(T::round(fmaf(own, p.tau_inv, f.one(sm.z[j]))));
    }
}

// ------------------------------------------------------------------- host
constexpr int kMaxRowsALaunch = kVocabCounters;
constexpr int64_t kMaxCols = (int64_t(1) << 31) - (1 << 16);   // a block's columns run a little past V in 32 bits

bool good_temperature(float t) { return t >= 0x1p-20f && t <= 0x1p20f; }

lmloss_status check_logprobs(const lmloss_logprobs_args* a, bool pointers)
{
    if (!a) return LMLOSS_ERR_INVALID_ARG;
    if (a->T < 0 || a->V < 1 || a->ld < a->V || a->n < 0) return LMLOSS_ERR_INVALID_ARG;
    if (a->M < 0 || a->M > kMaxTop || !float_dtype(a->dtype)) return LMLOSS_ERR_INVALID_ARG;
    if (a->ids_dtype != LMLOSS_INT64 && a->ids_dtype != LMLOSS_INT32) return LMLOSS_ERR_INVALID_ARG;
    if (!good_temperature(a->temperature) || a->mask_stride < 0) return LMLOSS_ERR_INVALID_ARG;
    if (a->V > kMaxCols || a->T >= (int64_t(1) << 30) || a->n > (int64_t(1) << 20)) return LMLOSS_ERR_UNSUPPORTED;
    if (a->T > 0 && a->ld > INT64_MAX / 16 / a->T) return LMLOSS_ERR_INVALID_ARG;
    if (!pointers) return LMLOSS_OK;
    if (a->token_mask && a->mask_stride != 0 && a->mask_stride < (a->V + 31) / 32) return LMLOSS_ERR_INVALID_ARG;
    if (a->T > 0) {
        const int id_bytes = a->ids_dtype == LMLOSS_INT64 ? 8 : 4;
        if (!a->logits || reinterpret_cast<uintptr_t>(a->logits) % float_bytes(a->dtype)) return LMLOSS_ERR_INVALID_ARG;
        if (a->n > 0 && (!a->tokens || !a->logp_out || reinterpret_cast<uintptr_t>(a->tokens) % id_bytes))
            return LMLOSS_ERR_INVALID_ARG;
        if (a->M > 0 && (!a->top_logp_out || !a->top_tokens_out)) return LMLOSS_ERR_INVALID_ARG;
    }
    return LMLOSS_OK;
}

struct LogprobsPlan {
    int vpt, tiles, slices;
    size_t keys, stats, total;
};

// As a beam step's: tiles of four vectors a thread, or of one where those would not give
// every SM a block; a block costs its tiles and the fixed part.  Cut rows leave at most kMaxParts
// parts in all.
LogprobsPlan plan_logprobs(const lmloss_logprobs_args* a, int num_sms)
{
    LogprobsPlan P{};
    const int64_t rows = std::min<int64_t>(std::max<int64_t>(a->T, 1), kMaxRowsALaunch), E = 16 / float_bytes(a->dtype);
    auto tiles_of = [&](int vpt) { return (a->V + vpt * kThreads * E - 1) / (vpt * kThreads * E); };
    P.vpt = rows * tiles_of(4) >= num_sms ? 4 : 1;
    const int64_t all = tiles_of(P.vpt), fixed = P.vpt == 4 ? 8 : 32;
    const int64_t most = std::min<int64_t>(std::max<int64_t>(kMaxParts / rows, 1), kMaxLists);
    const int64_t least = (all + most - 1) / most;
    int64_t tiles = all, best = INT64_MAX;
    for (int64_t t = least; t <= all && t <= least + 63; ++t) {
        const int64_t blocks = rows * ((all + t - 1) / t);
        const int64_t cost = std::max<int64_t>((blocks + num_sms - 1) / num_sms, 3) * (t + fixed);
        if (cost < best) {
            best = cost;
            tiles = t;
        }
    }
    P.tiles = static_cast<int>(tiles);
    P.slices = static_cast<int>((all + tiles - 1) / tiles);
    const size_t parts = P.slices > 1 ? static_cast<size_t>(rows) * P.slices : 0;
    P.stats = vocab_align(sizeof(uint64_t) * parts * a->M);
    P.total = P.stats + vocab_align(sizeof(float4) * parts);
    return P;
}

template <class T, int VPT, bool ALIGNED>
void launch_rows(const LogprobsParams& p, cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>(p.T) * static_cast<unsigned>(p.slices);
    if (p.entropy_out) logprobs_kernel<T, VPT, ALIGNED, true><<<grid, kThreads, 0, stream>>>(p);
    else logprobs_kernel<T, VPT, ALIGNED, false><<<grid, kThreads, 0, stream>>>(p);
}
template <class T>
void launch_rows(const LogprobsParams& p, int vpt, bool aligned, cudaStream_t stream)
{
    if (vpt == 4) aligned ? launch_rows<T, 4, true>(p, stream) : launch_rows<T, 4, false>(p, stream);
    else aligned ? launch_rows<T, 1, true>(p, stream) : launch_rows<T, 1, false>(p, stream);
}

lmloss_status check_grad(const lmloss_logprobs_grad_args* a)
{
    if (!a) return LMLOSS_ERR_INVALID_ARG;
    if (a->T < 0 || a->V < 1 || a->ld < a->V || a->ld_grad < a->V || a->n < 0) return LMLOSS_ERR_INVALID_ARG;
    if (!float_dtype(a->dtype) || (a->ids_dtype != LMLOSS_INT64 && a->ids_dtype != LMLOSS_INT32)) return LMLOSS_ERR_INVALID_ARG;
    if (!good_temperature(a->temperature) || a->mask_stride < 0) return LMLOSS_ERR_INVALID_ARG;
    if (a->V > kMaxCols || a->T >= (int64_t(1) << 30) || a->n > LMLOSS_MAX_GIVEN) return LMLOSS_ERR_UNSUPPORTED;
    if (a->T > 0 && (a->ld > INT64_MAX / 16 / a->T || a->ld_grad > INT64_MAX / 16 / a->T)) return LMLOSS_ERR_INVALID_ARG;
    if (a->token_mask && a->mask_stride != 0 && a->mask_stride < (a->V + 31) / 32) return LMLOSS_ERR_INVALID_ARG;
    if (a->T > 0) {
        const uintptr_t z = reinterpret_cast<uintptr_t>(a->logits), g = reinterpret_cast<uintptr_t>(a->grad_out);
        const int es = float_bytes(a->dtype), id_bytes = a->ids_dtype == LMLOSS_INT64 ? 8 : 4;
        if (!z || !g || z % es || g % es || (!a->lse && !a->log_sum)) return LMLOSS_ERR_INVALID_ARG;
        if ((a->row_max == nullptr) != (a->log_sum == nullptr)) return LMLOSS_ERR_INVALID_ARG;
        if (a->n > 0 && (!a->tokens || !a->grad_logp || reinterpret_cast<uintptr_t>(a->tokens) % id_bytes))
            return LMLOSS_ERR_INVALID_ARG;
        if (a->grad_entropy && !a->entropy) return LMLOSS_ERR_INVALID_ARG;
        if (z == g) {
            if (a->ld != a->ld_grad && a->T > 1) return LMLOSS_ERR_INVALID_ARG;
        } else {
            const uintptr_t z_end = z + static_cast<uintptr_t>(((a->T - 1) * a->ld + a->V) * es);
            const uintptr_t g_end = g + static_cast<uintptr_t>(((a->T - 1) * a->ld_grad + a->V) * es);
            // (side by side in the rows of one tensor they do not meet either)
            const uintptr_t row = static_cast<uintptr_t>(a->ld) * es, cols = static_cast<uintptr_t>(a->V) * es;
            const uintptr_t apart = z < g ? (g - z) % row : (row - (z - g) % row) % row;
            const bool beside = a->ld == a->ld_grad && apart >= cols && row - apart >= cols;
            if (z < g_end && g < z_end && !beside) return LMLOSS_ERR_INVALID_ARG;
        }
    }
    return LMLOSS_OK;
}

template <class T, bool SAME>
void launch_grad(const GradParams& p, cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>(p.T) * static_cast<unsigned>(p.parts);
    if (p.grad_entropy) logprobs_grad_kernel<T, true, SAME><<<grid, kThreads, 0, stream>>>(p);
    else logprobs_grad_kernel<T, false, SAME><<<grid, kThreads, 0, stream>>>(p);
}
template <class T>
void launch_grad(const GradParams& p, bool same, cudaStream_t stream)
{
    if (same) launch_grad<T, true>(p, stream);
    else launch_grad<T, false>(p, stream);
}

}  // namespace
}  // namespace lmloss

using namespace lmloss;

extern "C" {

lmloss_status lmloss_logprobs_check_args(const lmloss_logprobs_args* a) { return check_logprobs(a, true); }

lmloss_status lmloss_logprobs_check_grad_args(const lmloss_logprobs_grad_args* a) { return check_grad(a); }

lmloss_status lmloss_logprobs_workspace(const lmloss_logprobs_args* a, size_t* bytes)
{
    if (!bytes) return LMLOSS_ERR_INVALID_ARG;
    const lmloss_status st = check_logprobs(a, false);
    if (st != LMLOSS_OK) return st;
    // enough for any plan of no more rows
    const size_t parts = a->T > 0 ? kMaxParts : 0;
    *bytes = vocab_align(sizeof(uint64_t) * parts * a->M) + vocab_align(sizeof(float4) * parts);
    return LMLOSS_OK;
}

lmloss_status lmloss_logprobs_forward(lmloss_vocab_handle h, const lmloss_logprobs_args* a, cudaStream_t stream)
{
    if (!h) return LMLOSS_ERR_INVALID_ARG;
    const lmloss_status st = check_logprobs(a, true);
    if (st != LMLOSS_OK) return st;
    if (a->T == 0) return LMLOSS_OK;
    VocabDeviceGuard g(h->device);
    if (!g.ok) return LMLOSS_ERR_CUDA;
    const int es = float_bytes(a->dtype), id_bytes = a->ids_dtype == LMLOSS_INT64 ? 8 : 4;
    const bool aligned = aligned16(a->logits) && a->ld * es % 16 == 0;
    // as many rows a launch as there are counters: whole rows, which need no workspace, but for the last launch's, which
    // are looked at before the first
    lmloss_logprobs_args part = *a;
    if (a->T > kMaxRowsALaunch) {
        part.T = (a->T - 1) % kMaxRowsALaunch + 1;
        if (plan_logprobs(&part, h->num_sms).total > h->ws_bytes) return LMLOSS_ERR_INVALID_ARG;
    }
    for (int64_t r0 = 0; r0 < a->T; r0 += kMaxRowsALaunch) {
        part.T = std::min<int64_t>(a->T - r0, kMaxRowsALaunch);
        const LogprobsPlan P = plan_logprobs(&part, h->num_sms);
        if (P.total > h->ws_bytes) return LMLOSS_ERR_INVALID_ARG;
        LogprobsParams p{};
        p.logits = static_cast<const unsigned char*>(a->logits) + r0 * a->ld * es;
        p.ld = a->ld;
        p.T = static_cast<int>(part.T);
        p.V = static_cast<int>(a->V);
        p.n = a->n;
        p.M = a->M;
        p.slices = P.slices;
        p.tiles = P.tiles;
        p.mul = static_cast<float>(1.4426950408889634074 / static_cast<double>(a->temperature));
        p.near = 0x1p26f / p.mul;
        p.counted = 0x1p27f / p.mul;
        p.inv_tau = 1.0 / static_cast<double>(a->temperature);
        p.tokens = a->n ? static_cast<const unsigned char*>(a->tokens) + r0 * a->n * id_bytes : nullptr;
        p.ids32 = a->ids_dtype == LMLOSS_INT32;
        p.mask = a->token_mask ? a->token_mask + r0 * a->mask_stride : nullptr;
        p.mask_stride = a->mask_stride;
        p.logp_out = a->n ? a->logp_out + r0 * a->n : nullptr;
        p.lse_out = a->lse_out ? a->lse_out + r0 : nullptr;
        p.entropy_out = a->entropy_out ? a->entropy_out + r0 : nullptr;
        p.top_logp_out = a->M ? a->top_logp_out + r0 * a->M : nullptr;
        p.top_tokens_out = a->M ? a->top_tokens_out + r0 * a->M : nullptr;
        p.row_max_out = a->row_max_out ? a->row_max_out + r0 : nullptr;
        p.log_sum_out = a->log_sum_out ? a->log_sum_out + r0 : nullptr;
        p.keys = reinterpret_cast<uint64_t*>(h->ws);
        p.stats = reinterpret_cast<float4*>(h->ws + P.stats);
        p.done = h->counters;
        p.err = h->err;
        switch (a->dtype) {
        case LMLOSS_BF16: launch_rows<Bf16>(p, P.vpt, aligned, stream); break;
        case LMLOSS_FP16: launch_rows<Fp16>(p, P.vpt, aligned, stream); break;
        default: launch_rows<Fp32>(p, P.vpt, aligned, stream); break;
        }
        const lmloss_status launched = vocab_launch_err();
        if (launched != LMLOSS_OK) return launched;
    }
    return LMLOSS_OK;
}

lmloss_status lmloss_logprobs_backward(lmloss_vocab_handle h, const lmloss_logprobs_grad_args* a, cudaStream_t stream)
{
    if (!h) return LMLOSS_ERR_INVALID_ARG;
    const lmloss_status st = check_grad(a);
    if (st != LMLOSS_OK) return st;
    if (a->T == 0) return LMLOSS_OK;
    VocabDeviceGuard g(h->device);
    if (!g.ok) return LMLOSS_ERR_CUDA;
    const int es = float_bytes(a->dtype), id_bytes = a->ids_dtype == LMLOSS_INT64 ? 8 : 4;
    const int64_t E = 16 / es, vecs = (a->V + E - 1 + E - 1) / E;   // a vector more where rows start inside one
    // a part's given tokens and its barriers cost about as much as a loop: four loops where that leaves
    // every SM its blocks (four of each) all the same
    int64_t loops = 1;
    while (loops < 4 && a->T * ((vecs + 2 * loops * kGradVecs * kThreads - 1) / (2 * loops * kGradVecs * kThreads)) >= 8 * h->num_sms) loops *= 2;
    const int64_t per = loops * kGradVecs * kThreads, parts = (vecs + per - 1) / per;
    const bool same = ((reinterpret_cast<uintptr_t>(a->logits) ^ reinterpret_cast<uintptr_t>(a->grad_out)) & 15u) == 0 &&
                      (a->T == 1 || (a->ld - a->ld_grad) * es % 16 == 0);
    const int64_t most = std::max<int64_t>(((int64_t(1) << 31) - 1) / parts, 1);
    for (int64_t r0 = 0; r0 < a->T; r0 += most) {
        GradParams p{};
        p.logits = static_cast<const unsigned char*>(a->logits) + r0 * a->ld * es;
        p.ld = a->ld;
        p.T = static_cast<int>(std::min<int64_t>(a->T - r0, most));
        p.V = static_cast<int>(a->V);
        p.n = static_cast<int>(a->n);
        p.parts = static_cast<int>(parts);
        p.loops = static_cast<int>(loops);
        const double inv = 1.0 / static_cast<double>(a->temperature);
        p.tau_inv = static_cast<float>(inv);
        p.tau_inv_lo = static_cast<float>(inv - static_cast<double>(p.tau_inv));
        p.tokens = a->n ? static_cast<const unsigned char*>(a->tokens) + r0 * a->n * id_bytes : nullptr;
        p.ids32 = a->ids_dtype == LMLOSS_INT32;
        p.mask = a->token_mask ? a->token_mask + r0 * a->mask_stride : nullptr;
        p.mask_stride = a->mask_stride;
        p.row_max = a->row_max ? a->row_max + r0 : nullptr;
        p.less = (a->log_sum ? a->log_sum : a->lse) + r0;
        p.entropy = a->grad_entropy ? a->entropy + r0 : nullptr;
        p.grad_logp = a->n ? a->grad_logp + r0 * a->n : nullptr;
        p.grad_entropy = a->grad_entropy ? a->grad_entropy + r0 : nullptr;
        p.grad = static_cast<unsigned char*>(a->grad_out) + r0 * a->ld_grad * es;
        p.ld_grad = a->ld_grad;
        p.err = h->err;
        switch (a->dtype) {
        case LMLOSS_BF16: launch_grad<Bf16>(p, same, stream); break;
        case LMLOSS_FP16: launch_grad<Fp16>(p, same, stream); break;
        default: launch_grad<Fp32>(p, same, stream); break;
        }
        const lmloss_status launched = vocab_launch_err();
        if (launched != LMLOSS_OK) return launched;
    }
    return LMLOSS_OK;
}

}  // extern "C"
