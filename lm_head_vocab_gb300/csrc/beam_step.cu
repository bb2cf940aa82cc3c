// Beam search's step: the M best continuations of each sequence's K beams over the
// whole vocabulary.
//
//   score(k, v) = scores[k] + z[k][v] - lse_k,   lse_k = ln sum_v e^z[k][v]
//
// The logits are read once.  Within a row the order of the candidates is the
// order of the logits, whatever the row's normaliser, so one pass over a part of
// a row can keep both its softmax partials and its M largest logits; the block that
// finishes a sequence's last part joins the parts of its rows, turns logits into
// scores in fp64 and picks the M best.
//
// Measured (GB300, copy bandwidth 6.69 TB/s): 512 rows of 262144 bf16, M = 16, 51 us = 5.3
// TB/s of logits (79% of the copy's rate).  Bound by the issue of instructions and by
// what the memory leaves waiting (0.57 instructions a cycle and scheduler, 7.4 for each
// logit: the unpacking, the maximum, ex2 and the sum; long-scoreboard stalls the most),
// with 512 blocks over 152 SMs, four on some and three on the others.  One sequence
// of four beams at 128256: 10 to 11 us, latency from end to end: 1 us of loads, 2.5 us to
// the part's candidates, 1 us to count the block, 5 us to pick.  512 rows of 262143, which start
// at no vector boundary: 67.5 us, each vector from five words; rows of 262144 with one mask 60 us,
// with a mask each 63.5.
#include <algorithm>
#include <cmath>

#include "beam_math.cuh"
#include "beam_plan.cuh"
#include "row_stream.cuh"

namespace lmloss {
namespace {

constexpr int kMaxM = LMLOSS_MAX_BEAMS;
constexpr int kCap = 1024;                   // candidate keys of a part held at once
constexpr int kHits = 1024;                  // vectors of a part that reach its first threshold
constexpr int kSmall = 256;                  // few enough to be ranked by counting
constexpr int kFinal = 512;                  // candidates of a sequence held at once

struct BeamParams {
    const void* logits;
    int64_t ld;
    int B, K, M, V;
    int slices;                  // parts of a row
    int tiles;                   // tiles of a part
    double alpha;
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
    uint64_t* keys;              // [rows][slices][M]: each part's candidates, best first, 0 = none
    float2* stats;               // [rows][slices] (m, s): the part's sum of e^z is s e^m
    unsigned* done;              // [B] parts finished; 0 between calls
};

__device__ __forceinline__ uint64_t ordered64(double x)
{
    if (x == 0.0) x = 0.0;
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x));
    return (b >> 63) ? ~b : (b | (uint64_t(1) << 63));
}

// of a row: has candidates, goes on as it is, has none
enum : uint8_t { kAlive = 0, kFinished = 1, kOut = 2 };

struct __align__(16) Shared {
    uint64_t buf[kCap];                      // a part's candidates
    union {
        struct {
            uint4 data[kHits];               // a part's noted vectors
            int32_t col[kHits];
        } hit;
        struct {
            uint64_t rank[kFinal], place[kFinal];   // a sequence's finalists
            float z[kFinal];
            uint16_t lists[kMaxLists];       // its lists that reach the first threshold
        } pick;
    };
    uint32_t group[kThreads / 2], counts[kThreads];
    uint32_t thr, thr_end;                   // of the first tile, of all
    float red_m[kWarps], red_s[kWarps];
    int count, hit_count, few;
    int last;
    // of a sequence's rows
    double base[kMaxM], norm[kMaxM];
    float base_f[kMaxM], inv_f[kMaxM];
    float row_m[kMaxM], row_hi[kMaxM], row_lo[kMaxM];
    uint8_t state[kMaxM];
    // the slow way of picking
    uint64_t wbest[kWarps], wplace[kWarps];
    int wlist[kWarps];
    int lead;
};

// A candidate's score and rank key in fp64; false where it is none.
__device__ __forceinline__ bool exact_score(const BeamParams& p, const Shared& sm, int k, float z, uint64_t& rank)
{
    const double score = sm.state[k] == kFinished ? sm.base[k] : sm.base[k] + static_cast<double>(z);
    if (!isfinite(score)) return false;
    rank = ordered64(p.alpha != 0.0 ? score / sm.norm[k] : score);
    return true;
}

// Candidate d of a sequence's list (list / slices: its row); a finished row has one, any
// non-zero key.
__device__ __forceinline__ uint64_t list_key(const BeamParams& p, const Shared& sm, int64_t r0, int list, int d, int& k)
{
    k = list / p.slices;
    if (sm.state[k] == kFinished) return list == k * p.slices && d == 0 ? 1 : 0;
    return __ldcg(p.keys + (r0 * p.slices + list) * p.M + d);
}

__device__ __forceinline__ void write_pick(const BeamParams& p, const Shared& sm, int b, int out, int k, float z, int token)
{
    const int64_t o = static_cast<int64_t>(b) * p.M + out, r = static_cast<int64_t>(b) * p.K + k;
    const bool done = sm.state[k] == kFinished;
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

// M rounds of taking the best head of the sorted lists (one a row and part): for
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
                int k;
                const uint64_t key = list_key(p, sm, r0, i, d, k);
                uint64_t cr;
                if (key == 0 || !exact_score(p, sm, k, key_logit(key), cr)) continue;
                const uint64_t cp = (static_cast<uint64_t>(k) << 32) | static_cast<uint32_t>(sm.state[k] == kFinished ? 0 : key_col(key));
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
            int k;
            const uint64_t key = list_key(p, sm, r0, won, d, k);
            write_pick(p, sm, b, out, k, key_logit(key), key_col(key));
            stale = true;
        }
    }
}

// The block that finishes a sequence's last part picks its M best.
__device__ __noinline__ void pick(const BeamParams& p, Shared& sm, const int b)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = p.K, M = p.M, S = p.slices;
    const int64_t r0 = static_cast<int64_t>(b) * K;
    const int lists = K * S;   // one a row and part, best first

    // The first candidates of the lists, as many of each as give every thread one, are
    // read under the way of the rows' sums.
    const int depths = lists < kThreads ? min(M, kThreads / lists) : 1;
    const int list0 = tid / depths, depth0 = tid - list0 * depths;
    auto key_at = [&](int list, int d) { return __ldcg(p.keys + (r0 * S + list) * M + d); };
    uint64_t key0 = list0 < lists ? key_at(list0, depth0) : 0;

    // ---- the rows' normalisers: the parts' sums are added as pairs of fp32, an
    // error-free sum and what it leaves; then one thread a row goes on (fp64 is slow on
    // this GPU, and slower when several warps want it)
#pragma unroll 1
    for (int k = warp; k < K; k += kWarps) {
        const int64_t r = r0 + k;
        const float2 q0 = lane < S ? __ldcg(&p.stats[r * S + lane]) : make_float2(-INFINITY, 0.f);
        float m = q0.x, hi = 0.f, lo = 0.f;
        for (int s = lane + 32; s < S; s += 32) m = fmaxf(m, __ldcg(&p.stats[r * S + s]).x);
        m = warp_max(m);
        auto add = [&](float x, float e) {
            const float t = hi + x, v = t - hi;
            lo += ((hi - (t - v)) + (x - v)) + e;
            hi = t;
        };
        // an empty part (-inf, 0) adds nothing; NaN stays
        auto part = [&](float2 q) { return q.x == m ? q.y : q.y * exp2f((q.x - m) * kLog2e); };
        add(part(q0), 0.f);
        for (int s = lane + 32; s < S; s += 32) add(part(__ldcg(&p.stats[r * S + s])), 0.f);
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1) {
            const float x = __shfl_xor_sync(0xffffffffu, hi, o), e = __shfl_xor_sync(0xffffffffu, lo, o);
            add(x, e);
        }
        if (lane == 0) {
            sm.row_m[k] = m;
            sm.row_hi[k] = hi;
            sm.row_lo[k] = lo;
        }
    }
    if (tid == 0) {
        sm.count = 0;
        sm.hit_count = 0;
        sm.thr = 0;
        sm.thr_end = 0;
    }
    const int own = min(tid, K - 1);
    const bool own_done = p.finished && p.finished[r0 + own];
    const float own_score = p.scores[r0 + own];
    const int own_len = p.lengths ? p.lengths[r0 + own] : 0;
    __syncthreads();
    if (tid < K) {
        double lse = 0.0;
        if (!own_done) {
            const float m = sm.row_m[tid], hi = sm.row_hi[tid];
            lse = m == -INFINITY && hi == 0.f ? -INFINITY : static_cast<double>(m) + log_of_sum(hi, sm.row_lo[tid]);
        }
        if (p.lse_out) p.lse_out[r0 + tid] = static_cast<float>(lse);
        const double base = static_cast<double>(own_score) - lse;
        double d = 1.0;
        float inv = 1.f;
        if (p.alpha != 0.0) {
            const int64_t len = static_cast<int64_t>(own_len) + (own_done ? 0 : 1);
            d = power(static_cast<int>(min(max(len, int64_t(1)), int64_t(0x7fffffff))), p.alpha);
            inv = 1.f / static_cast<float>(d);
        }
        sm.base[tid] = base;
        sm.norm[tid] = d;
        sm.base_f[tid] = static_cast<float>(base);
        sm.inv_f[tid] = inv;
        sm.state[tid] = own_done ? kFinished : (isfinite(base) ? kAlive : kOut);
    }
    __syncthreads();

    // ---- a threshold in fp32, from bounds on the candidates' rank keys
    auto bounds = [&](int k, uint64_t key, float& low, float& high) {
        low = high = -INFINITY;
        if (key == 0 || sm.state[k] == kOut) return;
        rank_bounds(sm.base_f[k], sm.state[k] == kFinished ? 0.f : key_logit(key), sm.inv_f[k], low, high);
    };
    // a finished row has one candidate
    auto own_key = [&](int list, int d, uint64_t key) {
        const int k = list / S;
        return sm.state[k] == kFinished ? (list == k * S && d == 0 ? uint64_t(1) : uint64_t(0)) : key;
    };
    auto lower = [&](int list, uint64_t key) {
        float low, high;
        bounds(list / S, key, low, high);
        return low;
    };
    auto reaches = [&](int list, uint64_t key, float thr) {
        float low, high;
        bounds(list / S, key, low, high);
        return high >= thr && high > -INFINITY;
    };
    auto offer = [&](int list, uint64_t key, float thr) {
        if (!reaches(list, key, thr)) return;
        const int k = list / S;
        uint64_t rank;
        const float z = sm.state[k] == kFinished ? 0.f : key_logit(key);
        if (!exact_score(p, sm, k, z, rank)) return;
        const int to = atomicAdd(&sm.count, 1);
        if (to < kFinal) {
            sm.pick.rank[to] = rank;
            sm.pick.place[to] = (static_cast<uint64_t>(k) << 32) | static_cast<uint32_t>(sm.state[k] == kFinished ? 0 : key_col(key));
            sm.pick.z[to] = z;
        }
    };
    auto threshold = [&](float best, uint32_t* to) {
        rank_groups(best > -INFINITY ? ordered(best) : 0u, M, sm.group, to);
        __syncthreads();
        return *to ? unordered(*to) : -INFINITY;
    };
    float best = -INFINITY;
#pragma unroll 1
    for (int i = list0; i < lists; i += kThreads) {
        if (i != list0) key0 = key_at(i, 0);
        best = fmaxf(best, lower(i, own_key(i, depth0, key0)));
    }
    float thr = threshold(best, &sm.thr);
    // a list whose last of these stays below the threshold has nothing more
    if (depths < M && depth0 == depths - 1) {
#pragma unroll 1
        for (int i = list0; i < lists; i += kThreads) {
            if (lists > kThreads) key0 = key_at(i, 0);
            if (reaches(i, own_key(i, depth0, key0), thr)) sm.pick.lists[atomicAdd(&sm.hit_count, 1)] = static_cast<uint16_t>(i);
        }
    }
    __syncthreads();
    const int more = M - depths, entries = sm.hit_count * more;
    auto each_entry = [&](auto&& use) {
        constexpr int kAhead = 4;   // on their way
#pragma unroll 1
        for (int e0 = tid; e0 < entries; e0 += kAhead * kThreads) {
            uint64_t key[kAhead];
            int list[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int e = e0 + j * kThreads, x = min(e, entries - 1) / more;
                list[j] = sm.pick.lists[x];
                key[j] = e < entries ? own_key(list[j], 1, key_at(list[j], depths + e - x * more)) : 0;
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (key[j]) use(list[j], key[j]);
        }
    };
    if (entries > kThreads / 2) {
        // many: a threshold from all of them as well.  (Ranking by counting costs the square
        // of what is left: 768 candidates took 100 us.)
        each_entry([&](int list, uint64_t key) { best = fmaxf(best, lower(list, key)); });
        thr = fmaxf(thr, threshold(best, &sm.thr_end));
    }
#pragma unroll 1
    for (int i = list0; i < lists; i += kThreads) {
        if (lists > kThreads) key0 = key_at(i, 0);
        offer(i, own_key(i, depth0, key0), thr);
    }
    each_entry([&](int list, uint64_t key) { offer(list, key, thr); });

    // ---- what is left, ranked by counting in fp64
    __syncthreads();
    const int n = sm.count;
    if (n > kFinal) {
        pick_by_rounds(p, sm, b);
        return;
    }
    for (int i = tid; i < n; i += kThreads) {
        const uint64_t rank = sm.pick.rank[i], place = sm.pick.place[i];
        int above = 0;
#pragma unroll 8
        for (int o = 0; o < n; ++o) {
            const uint64_t x = sm.pick.rank[o], y = sm.pick.place[o];
            above += static_cast<int>(x > rank) | (static_cast<int>(x == rank) & static_cast<int>(y < place));
        }
        if (above < M)
            write_pick(p, sm, b, above, static_cast<int>(place >> 32), sm.pick.z[i], static_cast<int>(place & 0xffffffffu));
    }
    for (int i = n + tid; i < M; i += kThreads) write_empty(p, b, i);
}

// ------------------------------------------------------------- one part
// A block takes `tiles` tiles of one row, one after the other, with the next tile's
// loads in flight.  A tile is kThreads * VPT vectors of E columns, vector j of a
// thread at column (tile * VPT + j) * kThreads * E + thread * E: columns, not
// addresses, fix which thread adds what, so equal rows give equal bits wherever
// they start.
//
// Each thread keeps its own running maximum and sum.  The threads' running maxima
// give a threshold after the first tile, and a higher one after the second, fourth
// and so on; vectors that reach it are noted, and the other tiles pass without a
// barrier.  (A warp raising it on its own, from whatever maxima it saw, took as long
// at M = 16 and half as long again at M = 64.)
// At the end the noted vectors are looked through once for logits that reach the
// threshold of the whole part.
template <class T, int VPT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 4) beam_step_kernel(const __grid_constant__ BeamParams p)
{
    constexpr int E = Logits<T>::E;
    constexpr int kTileCols = VPT * kThreads * E;
    __shared__ Shared sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / p.slices, part = blockIdx.x - row * p.slices;
    const int b = row / p.K;
    if (!(p.finished && p.finished[row])) {
        RowLogits<T> r;
        r.z = static_cast<const typename T::raw*>(p.logits) + static_cast<int64_t>(row) * p.ld;
        r.V = p.V;
        r.lo = 0;
        r.hi = p.V - E;
        if (!ALIGNED) {
            // at the first and last row: nothing before or after the logits is read
            const int64_t after = (static_cast<int64_t>(p.B) * p.K - 1 - row) * p.ld;
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
        float m = -INFINITY, s = 0.f, best = -INFINITY, least = 0.f;
        int tile = 0;
        auto use_tile = [&](const Pack<T, E> (&q)[VPT], int c0) {
            // ---- maxima: of all logits (for the sum) and of the allowed ones (for the order)
            float vmax[VPT], tmax;
#pragma unroll
            for (int j = 0; j < VPT; ++j) vmax[j] = Logits<T>::largest(q[j]);
            tmax = vmax[0];
#pragma unroll
            for (int j = 1; j < VPT; ++j) tmax = fmaxf(tmax, vmax[j]);
            const float top = fmaxf(m, tmax);
            // tiles 0, 1, 3, 7, ... raise the threshold
            const bool raise = (tile & (tile + 1)) == 0;
            ++tile;
            // The mask is looked at where a logit reaches the threshold: what lies below it, allowed
            // or not, is no candidate and raises no threshold.  (387 rows of 218304 bf16 with a mask
            // each: 58 us when every vector's mask was looked at, 50 so, 39 without a mask.)
            if (mask && !raise && !(tmax >= least)) tmax = -INFINITY;
            else if (mask) {
                tmax = -INFINITY;
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int c = c0 + j * (kThreads * E);
                    const uint32_t allow = c < p.V ? static_cast<uint32_t>(mask[c >> 5]) >> (c & 31) : 0u;
                    vmax[j] = Logits<T>::largest_allowed(q[j], allow);
                    tmax = fmaxf(tmax, vmax[j]);
                }
            }
            best = fmaxf(best, tmax);
            const uint32_t now = best > -INFINITY ? ordered(best == 0.f ? 0.f : best) : 0u;
            if (raise) rank_groups(now, p.M, sm.group, &sm.thr);
            // ---- sum of exponentials.  The maximum is taken off before the change to
            // base 2: z log2 e alone would overflow at the type's lowest values.  In fp32, by
            // ex2.approx (within 2^-22): fp64 would take sixty-four times as long, and a row's
            // logsumexp comes out within one fp32 step of the exact one (1000 to 262144
            // columns, logits spread by 0.1 to 8).
            if (top > m) {
                s *= ex2((m - top) * kLog2e);
                m = top;
            }
            const float shift = m == -INFINITY ? 0.f : m;
            const uint64_t off2 = f2_pack(-shift, -shift), l2 = f2_pack(kLog2e, kLog2e);
            uint64_t s2 = f2_pack(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
#pragma unroll
                for (int i = 0; i < E; i += 2) {
                    float a, c;
                    f2_unpack(f2_mul(f2_add(f2_pack(q[j].get(i), q[j].get(i + 1)), off2), l2), a, c);
                    s2 = f2_add(s2, f2_pack(ex2(a), ex2(c)));
                }
            }
            float sa, sb;
            f2_unpack(s2, sa, sb);
            s += sa + sb;
            if (raise) {
                __syncthreads();   // the threshold; without one (fewer than M groups) every logit but -inf
                least = sm.thr ? unordered(sm.thr) : __uint_as_float(0xff7fffffu);
            }
            if (tmax >= least) {
#pragma unroll
                for (int j = 0; j < VPT; ++j)
                    if (vmax[j] >= least) {
                        const int to = atomicAdd(&sm.hit_count, 1);
                        if (to < kHits) {
                            sm.hit.data[to] = make_uint4(q[j].w[0], q[j].w[1], q[j].w[2], q[j].w[3]);
                            sm.hit.col[to] = c0 + j * (kThreads * E);
                        }
                    }
            }
        };
        // whole tiles, the next one in flight; then what is left
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
        for (bool before = true;; before = false) {
            // before the whole tiles only the first tile of the logits' first row, if that is
            // not whole; after them what is left
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

        // ---- the part's sum, and the threshold of all of it
        const float top = warp_max(m);
        if (m < top) s *= ex2((m - top) * kLog2e);
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) {
            sm.red_m[warp] = top;
            sm.red_s[warp] = s;
        }
        rank_groups(best > -INFINITY ? ordered(best == 0.f ? 0.f : best) : 0u, p.M, sm.group, &sm.thr_end);
        __syncthreads();
        if (warp == kWarps - 1) {
            const float mw = lane < kWarps ? sm.red_m[lane] : -INFINITY;
            float all = mw;
            for (int o = 4; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
            float total = lane < kWarps ? (mw == all ? sm.red_s[lane] : sm.red_s[lane] * ex2((mw - all) * kLog2e)) : 0.f;
            for (int o = 4; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
            if (lane == 0) p.stats[blockIdx.x] = make_float2(all, total);
        }

        // ---- candidates: the logits of the noted vectors that reach the threshold.
        // With more vectors noted than are kept (the largest logits late in the part)
        // all are looked at; with more candidates than are kept (many equal logits) the
        // threshold rises to the M-th largest of those held.
        uint64_t thr = sm.thr_end ? static_cast<uint64_t>(sm.thr_end) << 32 : 1;
        int n;
        while (true) {
            // a thread an element: little code, which is fetched once a block
            const int noted = sm.hit_count;
            const bool all = noted > kHits;
            const int elements = all ? end - begin : noted * E;
#pragma unroll 1
            for (int i = tid; i < elements; i += kThreads) {
                const int c = all ? begin + i : sm.hit.col[i / E] + i % E;
                const float z = T::widen(all ? r.z[c] : reinterpret_cast<const typename T::raw*>(&sm.hit.data[i / E])[i % E]);
                // past V: -inf
                if (z > -INFINITY && (!mask || (static_cast<uint32_t>(mask[c >> 5]) >> (c & 31) & 1u))) {
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

        // ---- the M best of them, best first: ranked by counting (exact: the keys are
        // all different)
        uint64_t* out = p.keys + static_cast<int64_t>(blockIdx.x) * p.M;
        const uint64_t cut = n > kSmall ? mth_largest(sm.buf, n, p.M, sm.counts) : 0;
        const uint64_t* set = sm.buf;
        if (cut) {
            // exactly M are left: a row's short end, where few groups have a logit, or equal ones
            uint64_t* few = reinterpret_cast<uint64_t*>(sm.hit.data);
            for (int i = tid; i < n; i += kThreads)
                if (sm.buf[i] >= cut) few[atomicAdd(&sm.few, 1)] = sm.buf[i];
            __syncthreads();
            n = p.M;
            set = few;
        }
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t k = set[i];
            int above = 0;
#pragma unroll 8
            for (int o = 0; o < n; ++o) above += set[o] > k ? 1 : 0;
            if (above < p.M) out[above] = k;
        }
        for (int i = n + tid; i < p.M; i += kThreads) out[i] = 0;
    }

    // ---- the sequence's last block goes on to pick
    __syncthreads();
    if (tid == 0) {
        const unsigned all = static_cast<unsigned>(p.K) * static_cast<unsigned>(p.slices);
        sm.last = count_done(&p.done[b]) == all - 1;
        if (sm.last) p.done[b] = 0;
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
    if (!(a->length_penalty >= 0.0) || !std::isfinite(a->length_penalty)) return LMLOSS_ERR_INVALID_ARG;
    if (a->eos_token < -1 || a->eos_token >= a->V || a->mask_stride < 0) return LMLOSS_ERR_INVALID_ARG;
    // a block's columns run a little past V in 32 bits
    if (a->V > (int64_t(1) << 31) - (1 << 16) || a->B > (int64_t(1) << 24)) return LMLOSS_ERR_UNSUPPORTED;
    if (a->B > 0 && a->ld > INT64_MAX / 16 / (a->B * a->K)) return LMLOSS_ERR_INVALID_ARG;
    if (!pointers) return LMLOSS_OK;
    if (a->length_penalty > 0.0 && !a->lengths) return LMLOSS_ERR_INVALID_ARG;
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

template <class T, int VPT>
lmloss_status launch_parts(const BeamParams& p, bool aligned, cudaStream_t stream)
{
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(p.B) * p.K * p.slices);
    if (aligned) beam_step_kernel<T, VPT, true><<<grid, kThreads, 0, stream>>>(p);
    else beam_step_kernel<T, VPT, false><<<grid, kThreads, 0, stream>>>(p);
    return vocab_launch_err();
}

template <class T>
lmloss_status launch_parts(const BeamParams& p, int vpt, bool aligned, cudaStream_t stream)
{
    return vpt == 4 ? launch_parts<T, 4>(p, aligned, stream) : launch_parts<T, 1>(p, aligned, stream);
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
    BeamPlan P{};
    if ((st = plan_beam(a, 1, P)) != LMLOSS_OK) return st;
    // enough for any plan: tiles of one, as many parts as a sequence's rows may have
    const int64_t rows = a->B * a->K, cols = kThreads * (16 / float_bytes(a->dtype));
    const size_t parts = static_cast<size_t>(std::min<int64_t>((a->V + cols - 1) / cols, kMaxLists / a->K));
    P.total = vocab_align(sizeof(uint64_t) * rows * parts * a->M) + vocab_align(sizeof(float2) * rows * parts);
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
        p.tiles = P.tiles;
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
        case LMLOSS_BF16: st = launch_parts<Bf16>(p, P.vpt, aligned, stream); break;
        case LMLOSS_FP16: st = launch_parts<Fp16>(p, P.vpt, aligned, stream); break;
        default: st = launch_parts<Fp32>(p, P.vpt, aligned, stream); break;
        }
        if (st != LMLOSS_OK) return st;
    }
    return LMLOSS_OK;
}

}  // extern "C"
