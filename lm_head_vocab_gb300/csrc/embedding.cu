// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward    rows[t]   = scale * table[ids[t]]
//   backward   table[v] (+)= scale * sum_{t : ids[t] = v} rows[t]
//
// Both are bound by memory: the lookup reads each row that occurs and writes
// [T, D]; the gradient reads [T, D] and writes [V, D] (or reads and writes the
// rows that occur).  The gradient's sums run over the positions sorted by token,
// so each table row is written once, by one block, in an order that the ids alone
// fix: no float atomics.
#include <cmath>
#include <new>

#include "vocab_common.cuh"

namespace lmloss {
namespace {

constexpr int kIgnore = LMLOSS_IGNORE_INDEX;

struct EmbParams {
    const void* ids;
    int ids32;
    int T;
    int V;
    int64_t D;
    void* table;
    int64_t ld_table;
    void* rows;
    int64_t ld_rows;
    float scale;
    int accumulate;
    int* err;
};

__device__ __forceinline__ int64_t load_id(const EmbParams& p, int64_t t)
{
    return p.ids32 ? static_cast<int64_t>(static_cast<const int32_t*>(p.ids)[t]) : static_cast<const int64_t*>(p.ids)[t];
}

template <class T>
__device__ __forceinline__ const unsigned char* at(const void* base, int64_t row, int64_t ld, int64_t c)
{
    return static_cast<const unsigned char*>(base) + (row * ld + c) * T::kBytes;
}
template <class T>
__device__ __forceinline__ unsigned char* at(void* base, int64_t row, int64_t ld, int64_t c)
{
    return static_cast<unsigned char*>(base) + (row * ld + c) * T::kBytes;
}

// Columns [c, c + N) of a row, those past D as zeros / not stored.
// RW: memory that this kernel also writes.
template <class T, int N, bool RW = false>
__device__ __forceinline__ void load_cols(Pack<T, N>& q, const void* base, int64_t row, int64_t ld, int64_t c, int64_t D)
{
    if (c + N <= D) {
        if constexpr (RW) q.load_rw(at<T>(base, row, ld, c));
        else q.load(at<T>(base, row, ld, c));
    } else {
        q.zero();
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c + i < D) {
                Pack<T, 1> e;
                e.load_rw(at<T>(base, row, ld, c + i));
                q.set(i, e.get(0));
            }
    }
}
template <class T, int N>
__device__ __forceinline__ void store_cols(const Pack<T, N>& q, void* base, int64_t row, int64_t ld, int64_t c, int64_t D)
{
    if (c + N <= D) {
        q.store(at<T>(base, row, ld, c));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c + i < D) {
                Pack<T, 1> e;
                e.zero();
                e.set(0, q.get(i));
                e.store(at<T>(base, row, ld, c + i));
            }
    }
}

// ------------------------------------------------------------------ lookup
// `tpr` threads a row (a power of two), each with four vectors in flight.
constexpr int kFwdThreads = 128;
constexpr int kFwdUnroll = 4;

template <class TW, class TO, int N>
__global__ void __launch_bounds__(kFwdThreads) embedding_forward_kernel(const EmbParams p, const int tpr)
{
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kFwdThreads / tpr) + threadIdx.x / tpr;
    if (t >= p.T) return;
    const int lane = threadIdx.x & (tpr - 1);
    const int64_t id = load_id(p, t);
    const bool valid = id >= 0 && id < p.V;
    if (!valid && id != kIgnore && lane == 0) set_error(p.err, kErrBadTarget);
    const int64_t step = static_cast<int64_t>(tpr) * N;
    if (!valid) {
        const float fill = id == kIgnore ? 0.f : __int_as_float(0x7fc00000);
        Pack<TO, N> o;
        o.zero();
#pragma unroll
        for (int i = 0; i < N; ++i) o.set(i, fill);
        for (int64_t c = lane * N; c < p.D; c += step) store_cols<TO, N>(o, p.rows, t, p.ld_rows, c, p.D);
        return;
    }
    for (int64_t c0 = lane * N; c0 < p.D; c0 += step * kFwdUnroll) {
        Pack<TW, N> w[kFwdUnroll];
#pragma unroll
        for (int u = 0; u < kFwdUnroll; ++u)
            if (c0 + u * step < p.D) load_cols<TW, N>(w[u], p.table, id, p.ld_table, c0 + u * step, p.D);
#pragma unroll
        for (int u = 0; u < kFwdUnroll; ++u)
            if (c0 + u * step < p.D) {
                Pack<TO, N> o;
                o.zero();
#pragma unroll
                for (int i = 0; i < N; ++i) o.set(i, w[u].get(i) * p.scale);
                store_cols<TO, N>(o, p.rows, t, p.ld_rows, c0 + u * step, p.D);
            }
    }
}

// -------------------------------------------------------- sort by token
// Least-significant-digit radix sort of (token, position), stable, so that the
// positions of a token stay in their order.  A position without a valid token gets
// the key V and ends up last.  Per pass: each tile counts its digits, one block
// turns the counts into offsets, each tile places its keys.
constexpr int kDigitBits = 8;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kSortThreads = 256;
constexpr int kSortRounds = 8;                            // keys a thread
constexpr int kTile = kSortThreads * kSortRounds;

__device__ __forceinline__ uint32_t first_key(const EmbParams& p, int64_t t)
{
    const int64_t id = load_id(p, t);
    if (id >= 0 && id < p.V) return static_cast<uint32_t>(id);
    if (id != kIgnore) set_error(p.err, kErrBadTarget);
    return static_cast<uint32_t>(p.V);
}

__global__ void __launch_bounds__(kSortThreads)
sort_count_kernel(const EmbParams p, const uint32_t* keys, const int shift, const int tiles, uint32_t* counts)
{
    __shared__ uint32_t bin[kDigits];
    bin[threadIdx.x] = 0;
    __syncthreads();
    for (int i = 0; i < kSortRounds; ++i) {
        const int64_t t = static_cast<int64_t>(blockIdx.x) * kTile + i * kSortThreads + threadIdx.x;
        if (t < p.T) {
            const uint32_t k = keys ? keys[t] : first_key(p, t);
            atomicAdd(&bin[(k >> shift) & (kDigits - 1)], 1u);
        }
    }
    __syncthreads();
    counts[static_cast<int64_t>(threadIdx.x) * tiles + blockIdx.x] = bin[threadIdx.x];
}

// exclusive prefix sums of counts[n], in place, by one block
__global__ void __launch_bounds__(1024) sort_offsets_kernel(uint32_t* counts, const int n)
{
    __shared__ uint32_t part[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (n + 1023) / 1024;
    const int lo = min(n, tid * per), hi = min(n, lo + per);
    uint32_t sum = 0;
    for (int i = lo; i < hi; ++i) sum += counts[i];
    uint32_t inc = sum;
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const uint32_t own = part[lane];
        uint32_t w = own;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += v;
        }
        part[lane] = w - own;
    }
    __syncthreads();
    uint32_t base = part[warp] + inc - sum;
    for (int i = lo; i < hi; ++i) {
        const uint32_t v = counts[i];
        counts[i] = base;
        base += v;
    }
}

__global__ void __launch_bounds__(kSortThreads)
sort_place_kernel(const EmbParams p, const uint32_t* keys, const uint32_t* pos, const int shift, const int tiles,
                  const uint32_t* offsets, uint32_t* keys_out, uint32_t* pos_out)
{
    constexpr int kWarps = kSortThreads / 32;
    __shared__ uint32_t bin[kWarps][kDigits];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kWarps * kDigits; i += kSortThreads) (&bin[0][0])[i] = 0;
    __syncthreads();
    // a warp's keys are consecutive, so ranks count up in position order
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTile + warp * (32 * kSortRounds) + lane;
    uint32_t key[kSortRounds], rank[kSortRounds];
#pragma unroll
    for (int i = 0; i < kSortRounds; ++i) {
        const int64_t t = t0 + i * 32;
        const bool in = t < p.T;
        key[i] = in ? (keys ? keys[t] : first_key(p, t)) : 0u;
        const uint32_t d = in ? (key[i] >> shift) & (kDigits - 1) : kDigits;
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        if (in) rank[i] = bin[warp][d] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (in && lane == __ffs(same) - 1) bin[warp][d] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // digit `tid`: offsets of the tile's warps
    uint32_t base = offsets[static_cast<int64_t>(tid) * tiles + blockIdx.x];
    for (int w = 0; w < kWarps; ++w) {
        const uint32_t n = bin[w][tid];
        bin[w][tid] = base;
        base += n;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortRounds; ++i) {
        const int64_t t = t0 + i * 32;
        if (t < p.T) {
            const uint32_t to = bin[warp][(key[i] >> shift) & (kDigits - 1)] + rank[i];
            keys_out[to] = key[i];
            pos_out[to] = pos ? pos[t] : static_cast<uint32_t>(t);
        }
    }
}

// ------------------------------------------------------- sums by token
// A block takes a window of kWindow sorted positions and a range of columns.  A
// token whose positions all lie in the window is summed and written.  One that
// crosses a window's border leaves the window's part of its sum, in fp32: in slot 1
// where it begins in this window, in slot 0 where it came from the window before;
// the join adds a token's parts in window order.
constexpr int kWindow = 32;
constexpr int kSumThreads = 128;
constexpr int kRowsAhead = 8;

struct SumParams {
    EmbParams e;
    const uint32_t* keys;   // sorted
    const uint32_t* pos;
    float* parts;           // [windows][2][ld_parts]
    int64_t ld_parts;
    int windows;
};

// acc: NP packs of N columns, pack j at column c + j * kSumThreads * N
template <class TO, int N, int NP>
__device__ __forceinline__ void write_sum(const EmbParams& e, uint32_t v, int64_t c, const float (&acc)[NP * N])
{
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        const int64_t cj = c + static_cast<int64_t>(j) * kSumThreads * N;
        if (cj >= e.D) break;
        Pack<TO, N> o;
        o.zero();
        if (e.accumulate) {
            Pack<TO, N> old;
            load_cols<TO, N, true>(old, e.table, v, e.ld_table, cj, e.D);
#pragma unroll
            for (int i = 0; i < N; ++i) o.set(i, fmaf(acc[j * N + i], e.scale, old.get(i)));
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) o.set(i, acc[j * N + i] * e.scale);
        }
        store_cols<TO, N>(o, e.table, v, e.ld_table, cj, e.D);
    }
}

template <class TG, class TO, int N, int NP>
__global__ void __launch_bounds__(kSumThreads) token_sum_kernel(const SumParams p)
{
    __shared__ uint32_t key[kWindow], row[kWindow];
    __shared__ uint32_t before, after;
    const EmbParams& e = p.e;
    const uint32_t none = static_cast<uint32_t>(e.V);
    const int tid = threadIdx.x;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kWindow;
    const int n = static_cast<int>(min(static_cast<int64_t>(kWindow), e.T - i0));
    if (tid < n) {
        key[tid] = p.keys[i0 + tid];
        row[tid] = p.pos[i0 + tid];
    }
    if (tid == 32) before = i0 > 0 ? p.keys[i0 - 1] : none;
    if (tid == 33) after = i0 + n < e.T ? p.keys[i0 + n] : none;
    __syncthreads();
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * kSumThreads * NP + tid) * N;
    if (c >= e.D) return;

    float acc[NP * N];
#pragma unroll
    for (int i = 0; i < NP * N; ++i) acc[i] = 0.f;
    int first = 0;   // where the current token's run begins in the window
    for (int b = 0; b < n; b += kRowsAhead) {
        if (key[b] == none) break;
        Pack<TG, N> g[kRowsAhead][NP];
#pragma unroll
        for (int r = 0; r < kRowsAhead; ++r)
            if (b + r < n && key[b + r] != none) {
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    const int64_t cj = c + static_cast<int64_t>(j) * kSumThreads * N;
                    if (cj < e.D) load_cols<TG, N>(g[r][j], e.rows, row[b + r], e.ld_rows, cj, e.D);
                    else g[r][j].zero();
                }
            }
#pragma unroll
        for (int r = 0; r < kRowsAhead; ++r) {
            const int i = b + r;
            if (i >= n || key[i] == none) break;
#pragma unroll
            for (int j = 0; j < NP; ++j)
#pragma unroll
                for (int k = 0; k < N; ++k) acc[j * N + k] += g[r][j].get(k);
            const uint32_t next = i + 1 < n ? key[i + 1] : after;
            if (i + 1 < n && next == key[i]) continue;
            // the run ends here, or goes on in the next window
            const bool from = first == 0 && before == key[i];
            const bool on = i + 1 == n && next == key[i];
            if (!from && !on) {
                write_sum<TO, N, NP>(e, key[i], c, acc);
            } else {
                float* part = p.parts + (2 * static_cast<int64_t>(blockIdx.x) + (from ? 0 : 1)) * p.ld_parts;
#pragma unroll
                for (int j = 0; j < NP; ++j)
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        const int64_t ck = c + static_cast<int64_t>(j) * kSumThreads * N + k;
                        if (ck < e.D) part[ck] = acc[j * N + k];
                    }
            }
#pragma unroll
            for (int k = 0; k < NP * N; ++k) acc[k] = 0.f;
            first = i + 1;
        }
    }
}

// The block of the window in which a crossing token begins adds its parts.
template <class TO, int N, int NP>
__global__ void __launch_bounds__(kSumThreads) token_join_kernel(const SumParams p)
{
    const EmbParams& e = p.e;
    const uint32_t none = static_cast<uint32_t>(e.V);
    const int64_t w = blockIdx.x;
    const int64_t end = (w + 1) * kWindow;   // the next window's first position
    if (end >= e.T) return;
    const uint32_t v = p.keys[end];
    if (v == none || p.keys[end - 1] != v) return;
    // it began before this window
    if (w > 0 && p.keys[w * kWindow - 1] == v) return;
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * kSumThreads * NP + threadIdx.x) * N;
    if (c >= e.D) return;
    float acc[NP * N];
    auto add = [&](int64_t slot, bool first) {
        const float* part = p.parts + slot * p.ld_parts;
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int64_t ck = c + static_cast<int64_t>(j) * kSumThreads * N + k;
                const float x = ck < e.D ? part[ck] : 0.f;
                acc[j * N + k] = first ? x : acc[j * N + k] + x;
            }
    };
    add(2 * w + 1, true);
    for (int64_t x = w + 1;; ++x) {
        add(2 * x, false);
        const int64_t next = (x + 1) * kWindow;
        if (next >= e.T || p.keys[next] != v) break;
    }
    write_sum<TO, N, NP>(e, v, c, acc);
}

// zeros in the first D columns of every row
template <class TO, int N>
__global__ void __launch_bounds__(256) zero_rows_kernel(const EmbParams p)
{
    const int64_t per = (p.D + N - 1) / N, total = per * p.V;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    Pack<TO, N> z;
    z.zero();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += step) {
        const int64_t r = i / per;
        store_cols<TO, N>(z, p.table, r, p.ld_table, (i - r * per) * N, p.D);
    }
}

// ------------------------------------------------------------------- host
lmloss_status check_embedding(const lmloss_embedding_args* a, bool pointers)
{
    if (!a) return LMLOSS_ERR_INVALID_ARG;
    if (a->T < 0 || a->V < 1 || a->D < 1) return LMLOSS_ERR_INVALID_ARG;
    if (a->ld_table < a->D || a->ld_rows < a->D) return LMLOSS_ERR_INVALID_ARG;
    if (!float_dtype(a->table_dtype) || !float_dtype(a->rows_dtype)) return LMLOSS_ERR_INVALID_ARG;
    if (a->ids_dtype != LMLOSS_INT64 && a->ids_dtype != LMLOSS_INT32) return LMLOSS_ERR_INVALID_ARG;
    if (!std::isfinite(a->scale)) return LMLOSS_ERR_INVALID_ARG;
    if (a->accumulate != 0 && a->accumulate != 1) return LMLOSS_ERR_INVALID_ARG;
    // 32-bit positions and tokens in the kernels; byte offsets fit in 64 bits
    if (a->T >= (int64_t(1) << 30) || a->V >= (int64_t(1) << 31) - 1) return LMLOSS_ERR_UNSUPPORTED;
    if (a->ld_table > INT64_MAX / 16 / a->V || (a->T > 0 && a->ld_rows > INT64_MAX / 16 / a->T))
        return LMLOSS_ERR_INVALID_ARG;
    if (!pointers) return LMLOSS_OK;
    if (!a->table || (a->T > 0 && (!a->ids || !a->rows))) return LMLOSS_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a->table) % float_bytes(a->table_dtype)) return LMLOSS_ERR_INVALID_ARG;
    if (a->T > 0 && (reinterpret_cast<uintptr_t>(a->rows) % float_bytes(a->rows_dtype) ||
                     reinterpret_cast<uintptr_t>(a->ids) % (a->ids_dtype == LMLOSS_INT64 ? 8 : 4)))
        return LMLOSS_ERR_INVALID_ARG;
    return LMLOSS_OK;
}

// every row of both matrices starts on a 16-byte boundary: vectors of 8 columns
bool vector_rows(const lmloss_embedding_args* a)
{
    return aligned16(a->table) && aligned16(a->rows) && a->ld_table * float_bytes(a->table_dtype) % 16 == 0 &&
           a->ld_rows * float_bytes(a->rows_dtype) % 16 == 0;
}

EmbParams params(const lmloss_vocab_ctx* h, const lmloss_embedding_args* a)
{
    EmbParams p{};
    p.ids = a->ids;
    p.ids32 = a->ids_dtype == LMLOSS_INT32;
    p.T = static_cast<int>(a->T);
    p.V = static_cast<int>(a->V);
    p.D = a->D;
    p.table = a->table;
    p.ld_table = a->ld_table;
    p.rows = a->rows;
    p.ld_rows = a->ld_rows;
    p.scale = a->scale;
    p.accumulate = a->accumulate;
    p.err = h->err;
    return p;
}

struct SortSpace {
    size_t keys[2], pos[2], counts, parts, total;
    int tiles, windows;
    int64_t ld_parts;
};

SortSpace sort_space(const lmloss_embedding_args* a)
{
    SortSpace s{};
    const size_t T = static_cast<size_t>(a->T);
    s.tiles = static_cast<int>((a->T + kTile - 1) / kTile);
    s.windows = static_cast<int>((a->T + kWindow - 1) / kWindow);
    s.ld_parts = (a->D + 7) / 8 * 8;
    size_t off = 0;
    auto take = [&](size_t bytes) { size_t o = off; off = vocab_align(off + bytes); return o; };
    for (int i = 0; i < 2; ++i) {
        s.keys[i] = take(4 * T);
        s.pos[i] = take(4 * T);
    }
    s.counts = take(sizeof(uint32_t) * kDigits * static_cast<size_t>(s.tiles));
    s.parts = take(sizeof(float) * 2 * static_cast<size_t>(s.windows) * static_cast<size_t>(s.ld_parts));
    s.total = off;
    return s;
}

template <class F>
lmloss_status by_type(int32_t dtype, F&& f)
{
    switch (dtype) {
    case LMLOSS_BF16: return f(Bf16{});
    case LMLOSS_FP16: return f(Fp16{});
    default: return f(Fp32{});
    }
}

template <class TW, class TO, int N>
lmloss_status launch_forward(const EmbParams& p, cudaStream_t stream)
{
    const int64_t vecs = (p.D + N - 1) / N;
    int tpr = 8;
    while (tpr < kFwdThreads && tpr < vecs) tpr *= 2;
    const int rows = kFwdThreads / tpr;
    embedding_forward_kernel<TW, TO, N><<<(p.T + rows - 1) / rows, kFwdThreads, 0, stream>>>(p, tpr);
    return vocab_launch_err();
}

template <class TG, class TO, int N, int NP>
lmloss_status launch_sums(const SumParams& p, cudaStream_t stream)
{
    const int64_t cols = static_cast<int64_t>(kSumThreads) * N * NP;
    const dim3 grid(static_cast<unsigned>(p.windows), static_cast<unsigned>((p.e.D + cols - 1) / cols));
    token_sum_kernel<TG, TO, N, NP><<<grid, kSumThreads, 0, stream>>>(p);
    lmloss_status st = vocab_launch_err();
    if (st != LMLOSS_OK) return st;
    token_join_kernel<TO, N, NP><<<grid, kSumThreads, 0, stream>>>(p);
    return vocab_launch_err();
}

template <class TO, int N>
lmloss_status launch_zero(const lmloss_vocab_ctx* h, const EmbParams& p, cudaStream_t stream)
{
    zero_rows_kernel<TO, N><<<8 * h->num_sms, 256, 0, stream>>>(p);
    return vocab_launch_err();
}

lmloss_status sort_tokens(const lmloss_vocab_ctx* h, const EmbParams& p, const SortSpace& s, SumParams& q,
                          cudaStream_t stream)
{
    int bits = 1;
    while ((static_cast<int64_t>(p.V) >> bits) != 0) ++bits;   // the keys are 0 .. V
    uint32_t* counts = reinterpret_cast<uint32_t*>(h->ws + s.counts);
    const uint32_t *keys = nullptr, *pos = nullptr;
    int to = 0;
    for (int shift = 0; shift < bits; shift += kDigitBits) {
        uint32_t* keys_out = reinterpret_cast<uint32_t*>(h->ws + s.keys[to]);
        uint32_t* pos_out = reinterpret_cast<uint32_t*>(h->ws + s.pos[to]);
        sort_count_kernel<<<s.tiles, kSortThreads, 0, stream>>>(p, keys, shift, s.tiles, counts);
        sort_offsets_kernel<<<1, 1024, 0, stream>>>(counts, kDigits * s.tiles);
        sort_place_kernel<<<s.tiles, kSortThreads, 0, stream>>>(p, keys, pos, shift, s.tiles, counts, keys_out, pos_out);
        lmloss_status st = vocab_launch_err();
        if (st != LMLOSS_OK) return st;
        keys = keys_out;
        pos = pos_out;
        to ^= 1;
    }
    q.keys = keys;
    q.pos = pos;
    return LMLOSS_OK;
}

}  // namespace
}  // namespace lmloss

using namespace lmloss;

extern "C" {

lmloss_status lmloss_embedding_check_args(const lmloss_embedding_args* a) { return check_embedding(a, true); }

lmloss_status lmloss_embedding_workspace(const lmloss_embedding_args* a, size_t* bytes)
{
    if (!bytes) return LMLOSS_ERR_INVALID_ARG;
    const lmloss_status st = check_embedding(a, false);
    if (st != LMLOSS_OK) return st;
    *bytes = sort_space(a).total;
    return LMLOSS_OK;
}

lmloss_status lmloss_embedding_forward(lmloss_vocab_handle h, const lmloss_embedding_args* a, cudaStream_t stream)
{
    if (!h) return LMLOSS_ERR_INVALID_ARG;
    const lmloss_status st = check_embedding(a, true);
    if (st != LMLOSS_OK) return st;
    if (a->T == 0) return LMLOSS_OK;
    VocabDeviceGuard g(h->device);
    if (!g.ok) return LMLOSS_ERR_CUDA;
    const EmbParams p = params(h, a);
    const bool vec = vector_rows(a);
    return by_type(a->table_dtype, [&](auto tw) {
        return by_type(a->rows_dtype, [&](auto to) {
            using TW = decltype(tw);
            using TO = decltype(to);
            return vec ? launch_forward<TW, TO, 8>(p, stream) : launch_forward<TW, TO, 1>(p, stream);
        });
    });
}

lmloss_status lmloss_embedding_backward(lmloss_vocab_handle h, const lmloss_embedding_args* a, cudaStream_t stream)
{
    if (!h) return LMLOSS_ERR_INVALID_ARG;
    lmloss_status st = check_embedding(a, true);
    if (st != LMLOSS_OK) return st;
    const SortSpace s = sort_space(a);
    if (s.total > h->ws_bytes) return LMLOSS_ERR_INVALID_ARG;
    // blocks are numbered by windows and column ranges
    if (a->D > 65535LL * kSumThreads * 4) return LMLOSS_ERR_UNSUPPORTED;
    VocabDeviceGuard g(h->device);
    if (!g.ok) return LMLOSS_ERR_CUDA;
    SumParams q{};
    q.e = params(h, a);
    const bool vec = vector_rows(a);
    if (!a->accumulate) {
        st = by_type(a->table_dtype, [&](auto to) {
            using TO = decltype(to);
            return vec ? launch_zero<TO, 8>(h, q.e, stream) : launch_zero<TO, 1>(h, q.e, stream);
        });
        if (st != LMLOSS_OK) return st;
    }
    if (a->T == 0) return LMLOSS_OK;
    if ((st = sort_tokens(h, q.e, s, q, stream)) != LMLOSS_OK) return st;
    q.parts = reinterpret_cast<float*>(h->ws + s.parts);
    q.ld_parts = s.ld_parts;
    q.windows = s.windows;
    return by_type(a->rows_dtype, [&](auto tg) {
        return by_type(a->table_dtype, [&](auto to) {
            using TG = decltype(tg);
            using TO = decltype(to);
            return vec ? launch_sums<TG, TO, 8, 1>(q, stream) : launch_sums<TG, TO, 1, 4>(q, stream);
        });
    });
}

}  // extern "C"
