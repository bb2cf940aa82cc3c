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
#include <cmath>

#include "vocab_common.cuh"

namespace lmloss {
namespace {

constexpr int kMaxM = LMLOSS_MAX_BEAMS;
constexpr int kThreads = 256;
constexpr int kGroups = 64;                  // groups of four neighbouring threads
constexpr int kCap = 2048;                   // candidate keys held at once
constexpr int kSmall = 256;                  // few enough to be ranked by counting

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
    uint64_t* keys;              // [rows][slices][M], best first, 0 = none
    float2* stats;               // [rows][slices] (m, s): the slice's sum of e^z is s e^m
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

// the M-th largest of n > M different keys in shared memory, found bit by bit
__device__ uint64_t mth_largest(const uint64_t* keys, int n, int M)
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

// One vector's 16 bytes of logits as E floats.
template <class T>
struct Logits {
    static constexpr int E = 16 / T::kBytes;
};

// Slice s of row r: kThreads * VPT vectors of E columns, vector j of a thread at
// column ((s * VPT + j) * kThreads + thread) * E.  Columns, not addresses, fix
// which thread adds what, so equal rows give equal bits wherever they start.
template <class T, int VPT, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) beam_slice_kernel(const BeamParams p)
{
    constexpr int E = Logits<T>::E;
    __shared__ uint64_t buf[kCap];
    __shared__ uint32_t gmax[kGroups];
    __shared__ float red[kThreads / 32];
    __shared__ uint32_t thr_sh;
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / p.slices, slice = blockIdx.x - row * p.slices;
    if (p.finished && p.finished[row]) return;
    const int64_t base = static_cast<int64_t>(row) * p.ld;
    const typename T::raw* z = static_cast<const typename T::raw*>(p.logits) + base;
    const int32_t* mask = p.mask ? p.mask + row * p.mask_stride : nullptr;
    const int first = slice * (VPT * kThreads * E) + tid * E;   // < 2^31: V < 2^31 - 1 and the slice starts below V

    // ---- load; columns past V read as -inf
    Pack<T, E> q[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int64_t c = static_cast<int64_t>(first) + static_cast<int64_t>(j) * (kThreads * E);
        if (ALIGNED && c + E <= p.V) {
            q[j].load(z + c);
        } else {
            q[j].zero();
#pragma unroll
            for (int i = 0; i < E; ++i) q[j].set(i, c + i < p.V ? T::widen(z[c + i]) : -INFINITY);
        }
    }
    // ---- maxima: of all logits (for the sum) and of the allowed ones (for the order)
    float m = -INFINITY, vmax[VPT], best = -INFINITY;
    uint32_t allow[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int64_t c = static_cast<int64_t>(first) + static_cast<int64_t>(j) * (kThreads * E);
        allow[j] = (1u << E) - 1u;
        if (mask && c < p.V) allow[j] = (static_cast<uint32_t>(mask[c >> 5]) >> (c & 31)) & ((1u << E) - 1u);
        vmax[j] = -INFINITY;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float x = q[j].get(i);
            m = fmaxf(m, x);
            if (allow[j] >> i & 1u) vmax[j] = fmaxf(vmax[j], x);
        }
        best = fmaxf(best, vmax[j]);
    }
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float g = best;
    g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 1));
    g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
    if (lane == 0) red[warp] = m;
    if ((tid & 3) == 0) gmax[tid >> 2] = g > -INFINITY ? ordered(g == 0.f ? 0.f : g) : 0u;
    if (tid == 0) {
        thr_sh = 0;
        count = 0;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, red[w]);

    // ---- threshold: the M-th largest of the groups' maxima.  At least M
    // candidates reach it, and few more do.
    {
        const int own = tid >> 2, part = (tid & 3) * (kGroups / 4);
        const uint32_t v = gmax[own];
        int above = 0;
#pragma unroll
        for (int i = 0; i < kGroups / 4; ++i) {
            const uint32_t o = gmax[part + i];
            above += (o > v || (o == v && part + i < own)) ? 1 : 0;
        }
        above += __shfl_xor_sync(0xffffffffu, above, 1);
        above += __shfl_xor_sync(0xffffffffu, above, 2);
        if ((tid & 3) == 0 && above == p.M - 1) thr_sh = v;
    }
    // ---- sum of exponentials.  The maximum is taken off before the change to
    // base 2: z log2 e alone would overflow at the type's lowest values.
    float s = 0.f;
    const float shift = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) part += ex2((q[j].get(i) - shift) * kLog2e);
        s += part;
    }
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();   // thr_sh written, red read
    if (lane == 0) red[warp] = s;

    // ---- collect the candidates from the threshold up, raising it while they
    // are more than the buffer holds (many equal logits, or the best ones side
    // by side in one thread)
    uint64_t thr = static_cast<uint64_t>(thr_sh) << 32;
    if (thr == 0) thr = 1;   // fewer than M groups have one: all of them
    int n;
    while (true) {
        const float least = key_logit(thr);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (thr > 1 ? vmax[j] >= least : vmax[j] > -INFINITY) {
                const int c = first + j * (kThreads * E);
                for (int i = 0; i < E; ++i) {
                    const float x = q[j].get(i);
                    if ((allow[j] >> i & 1u) && x > -INFINITY) {
                        const uint64_t k = key_of(x, c + i);
                        if (k >= thr) {
                            const int to = atomicAdd(&count, 1);
                            if (to < kCap) buf[to] = k;
                        }
                    }
                }
            }
        }
        __syncthreads();
        n = count;
        if (n <= kCap) break;
        const uint64_t t = mth_largest(buf, kCap, p.M);
        __syncthreads();
        if (tid == 0) count = 0;
        thr = t;
        __syncthreads();
    }
    if (tid == 0) {
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) total += red[w];
        p.stats[blockIdx.x] = make_float2(m, total);
    }
    uint64_t* out = p.keys + static_cast<int64_t>(blockIdx.x) * p.M;
    const uint64_t cut = n > kSmall ? mth_largest(buf, n, p.M) : 0;
    // rank by counting: exact, and the keys are all different
    for (int i = tid; i < n; i += kThreads) {
        const uint64_t k = buf[i];
        if (k < cut) continue;
        int above = 0;
        for (int o = 0; o < n; ++o) above += buf[o] > k ? 1 : 0;
        if (above < p.M) out[above] = k;
    }
    for (int i = n + tid; i < p.M; i += kThreads) out[i] = 0;
}

__device__ __forceinline__ uint64_t ordered64(double x)
{
    if (x == 0.0) x = 0.0;
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x));
    return (b >> 63) ? ~b : (b | (uint64_t(1) << 63));
}

// One block a sequence: the rows' normalisers, then M rounds of taking the best
// head of the rows' sorted lists (one a slice).
__global__ void __launch_bounds__(kThreads) beam_pick_kernel(const BeamParams p)
{
    __shared__ double base[kMaxM], norm[kMaxM], row_score[kMaxM];
    __shared__ uint64_t wbest[kThreads / 32], wplace[kThreads / 32];
    __shared__ int wlist[kThreads / 32];
    __shared__ int lead;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x, K = p.K, M = p.M, S = p.slices;

    for (int k = warp; k < K; k += kThreads / 32) {
        const int64_t r = static_cast<int64_t>(b) * K + k;
        const bool done = p.finished && p.finished[r];
        const double score = static_cast<double>(p.scores[r]);
        double lse = 0.0;
        if (!done) {
            float m = -INFINITY;
            for (int s = lane; s < S; s += 32) m = fmaxf(m, p.stats[r * S + s].x);
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            double sum = 0.0;
            for (int s = lane; s < S; s += 32) {
                const float2 q = p.stats[r * S + s];
                // an empty slice (-inf, 0) adds nothing; NaN stays
                sum += q.x == m ? static_cast<double>(q.y) : static_cast<double>(q.y * exp2f((q.x - m) * kLog2e));
            }
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            lse = m == -INFINITY && sum == 0.0 ? -INFINITY : static_cast<double>(m) + log(sum);
        }
        if (lane == 0) {
            if (p.lse_out) p.lse_out[r] = static_cast<float>(lse);
            base[k] = score - lse;
            row_score[k] = score;
            double d = 1.0;
            if (p.lengths) {
                const int64_t len = static_cast<int64_t>(p.lengths[r]) + (done ? 0 : 1);
                d = pow(static_cast<double>(len < 1 ? 1 : len), static_cast<double>(p.alpha));
            }
            norm[k] = d;
        }
    }
    __syncthreads();

    // list i: row i / S, slice i % S; a thread takes lists tid, tid + 256, ...
    const int lists = K * S;
    // rank and score of list i's candidate at depth d; false when there is none
    auto candidate = [&](int i, int d, uint64_t& rank, uint64_t& place, double& score, int64_t& token) -> bool {
        const int k = i / S, s = i - k * S;
        const int64_t r = static_cast<int64_t>(b) * K + k;
        if (p.finished && p.finished[r]) {
            if (s != 0 || d != 0) return false;
            score = row_score[k];
            token = p.eos;
        } else {
            if (d >= M) return false;
            const uint64_t key = p.keys[(r * S + s) * M + d];
            if (key == 0) return false;
            score = base[k] + static_cast<double>(key_logit(key));
            token = key_col(key);
        }
        if (!isfinite(score)) return false;
        rank = ordered64(p.lengths ? score / norm[k] : score);
        place = static_cast<uint64_t>(k) * static_cast<uint64_t>(p.V) + static_cast<uint64_t>(token);
        return true;
    };
    // the thread's best head; its lists' depths are few enough to keep as a count
    // of what was taken from each (the winner's list alone moves on)
    constexpr int kPer = 8;   // lists a thread: K * S <= 2048
    uint8_t depth[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) depth[j] = 0;
    uint64_t rank = 0, place = 0;
    int list = -1;
    bool stale = true;
    for (int out = 0; out < M; ++out) {
        if (stale) {
            rank = 0;
            place = ~uint64_t(0);
            list = -1;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int i = tid + j * kThreads;
                uint64_t cr, cp;
                double cs;
                int64_t ct;
                if (i < lists && candidate(i, depth[j], cr, cp, cs, ct) && (cr > rank || (cr == rank && cp < place))) {
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
            wbest[warp] = br;
            wplace[warp] = bp;
            wlist[warp] = bl;
        }
        __syncthreads();
        if (tid == 0) {
            int w = 0;
            for (int x = 1; x < kThreads / 32; ++x)
                if (wbest[x] > wbest[w] || (wbest[x] == wbest[w] && wplace[x] < wplace[w])) w = x;
            lead = wbest[w] ? wlist[w] : -1;
        }
        __syncthreads();
        const int won = lead;
        const int64_t o = static_cast<int64_t>(b) * M + out;
        if (won < 0) {
            // fewer than M candidates: the rest is empty
            if (tid == 0) {
                const int k = out % K;
                p.scores_out[o] = -INFINITY;
                p.parents_out[o] = k;
                p.tokens_out[o] = LMLOSS_IGNORE_INDEX;
                if (p.finished_out) p.finished_out[o] = 0;
                if (p.lengths_out) p.lengths_out[o] = p.lengths[static_cast<int64_t>(b) * K + k];
            }
        } else if (won % kThreads == tid) {
            const int j = won / kThreads, k = won / S;
            const int64_t r = static_cast<int64_t>(b) * K + k;
            int d = 0;
#pragma unroll
            for (int x = 0; x < kPer; ++x)
                if (x == j) d = depth[x]++;
            uint64_t cr, cp;
            double score = 0.0;
            int64_t token = 0;
            candidate(won, d, cr, cp, score, token);
            const bool done = p.finished && p.finished[r];
            p.scores_out[o] = static_cast<float>(score);
            p.parents_out[o] = k;
            p.tokens_out[o] = token;
            if (p.finished_out) p.finished_out[o] = done || token == p.eos ? 1 : 0;
            if (p.lengths_out) p.lengths_out[o] = p.lengths[r] + (done ? 0 : 1);
            stale = true;
        }
    }
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

constexpr int kMaxLists = 2048;   // K * slices: eight lists a thread of the second kernel
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
    if (aligned) beam_slice_kernel<T, VPT, true><<<grid, kThreads, 0, stream>>>(p);
    else beam_slice_kernel<T, VPT, false><<<grid, kThreads, 0, stream>>>(p);
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
    BeamParams p{};
    p.logits = a->logits;
    p.ld = a->ld;
    p.B = static_cast<int>(a->B);
    p.K = a->K;
    p.M = a->M;
    p.V = static_cast<int>(a->V);
    p.slices = P.slices;
    p.alpha = a->length_penalty;
    p.eos = a->eos_token;
    p.scores = a->scores;
    p.finished = a->finished;
    p.lengths = a->lengths;
    p.mask = a->token_mask;
    p.mask_stride = a->mask_stride;
    p.scores_out = a->scores_out;
    p.parents_out = a->parents_out;
    p.tokens_out = a->tokens_out;
    p.lse_out = a->lse_out;
    p.finished_out = a->finished_out;
    p.lengths_out = a->lengths_out;
    p.keys = reinterpret_cast<uint64_t*>(h->ws + P.keys);
    p.stats = reinterpret_cast<float2*>(h->ws + P.stats);
    const bool aligned = aligned16(a->logits) && a->ld * float_bytes(a->dtype) % 16 == 0;
    switch (a->dtype) {
    case LMLOSS_BF16: st = launch_slices<Bf16>(p, P.vpt, aligned, stream); break;
    case LMLOSS_FP16: st = launch_slices<Fp16>(p, P.vpt, aligned, stream); break;
    default: st = launch_slices<Fp32>(p, P.vpt, aligned, stream); break;
    }
    if (st != LMLOSS_OK) return st;
    beam_pick_kernel<<<static_cast<unsigned>(p.B), kThreads, 0, stream>>>(p);
    return vocab_launch_err();
}

}  // extern "C"
