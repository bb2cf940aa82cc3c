// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward    rows[t]   = scale * table[ids[t]]
//   backward   table[v] (+)= scale * sum_{t : ids[t] = v} rows[t]
//
// Both are bound by memory: the lookup reads each row that occurs and writes
// [T, D]; the gradient reads [T, D] and writes [V, D] (or reads and writes the
// rows that occur).  The gradient's sums run over the positions sorted by token,
// so each table row is written once, by one block, in an order that the ids alone
// fix: no element is added to twice by different blocks.
//
// Measured (GB300, copy bandwidth 6.69 TB/s; ids as frequent as words are):
//   lookup    32767 of 151936 x 2048, fp32 to bf16: 39.5 us = 5.9 TB/s of what it must move;
//             8 of 128256 x 4096 bf16: 2.2 us
//   gradient  65536 bf16 rows into bf16 262144 x 2048, whole: 232 us = 5.8 TB/s, of which the
//             sort (beside 125 MB of zeros) 35, sums and zeros 180 (82% of the DRAM's time),
//             join 17;
//             16384 bf16 rows added to fp32 128256 x 4096: 76 us = 4.7 TB/s: sort 14 us, which
//             nothing but a prefetch runs beside, sums 55 (72% of the DRAM's time), join 12;
//             4097 of bf16 32003 x 1001 (no row on a vector boundary), whole: 25 us = 2.9 TB/s,
//             three kernels of 6 to 10 us, each a chain of latencies
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

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
    // all memory that may be read as `rows` and as `table`
    const unsigned char *rows_end, *table_end;
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


// ------------------------------------------------------- unaligned rows
// A thread works on N columns that start on a 16-byte boundary of the row it WRITES;
// where rows do not (odd widths), the first vector of a row begins before its first
// column, and what it reads is put together from aligned blocks.  Vectors at a row's
// ends go element by element, out of line.
template <class T>
constexpr int kGranule = 16 / T::kBytes;

template <class T>
__device__ __noinline__ uint4 gather_ends(const unsigned char* row, int64_t c, int64_t D)
{
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kGranule<T>; ++i)
        if (c + i >= 0 && c + i < D) {
            const uint32_t x = reinterpret_cast<const typename T::raw*>(row)[c + i];
            if constexpr (T::kBytes == 4) w[i] = x;
            else w[i / 2] |= x << (16 * (i & 1));
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <class T>
__device__ __noinline__ void scatter_ends(unsigned char* row, int64_t c, int64_t D, uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < kGranule<T>; ++i)
        if (c + i >= 0 && c + i < D) {
            if constexpr (T::kBytes == 4) reinterpret_cast<uint32_t*>(row)[c + i] = w[i];
            else reinterpret_cast<uint16_t*>(row)[c + i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
        }
}

template <class T, int N>
__device__ __forceinline__ void load_ends(Pack<T, N>& q, const unsigned char* row, int64_t c, int64_t D)
{
#pragma unroll
    for (int g = 0; g < N / kGranule<T>; ++g) {
        const uint4 x = gather_ends<T>(row, c + g * kGranule<T>, D);
        q.w[4 * g] = x.x; q.w[4 * g + 1] = x.y; q.w[4 * g + 2] = x.z; q.w[4 * g + 3] = x.w;
    }
}

// Columns [c, c + N) of a row of an input, whatever its alignment; what lies outside
// [0, D) has no meaning.  lo, hi: the memory that may be read.  A vector at a row's end
// reads on into its neighbour; only at the ends of that memory columns go one by one.
template <class T, int N, bool ALIGNED>
__device__ __forceinline__ void load_row(Pack<T, N>& q, const unsigned char* row, int64_t c, int64_t D,
                                         const unsigned char* lo, const unsigned char* hi)
{
    const unsigned char* p = row + c * T::kBytes;
    if (ALIGNED ? p + N * T::kBytes <= hi : inside_blocks<T, N>(p, lo, hi)) {
        if constexpr (ALIGNED) {
            q.load(p);
        } else {
            constexpr int kVecs = N * T::kBytes / 16 + 1;
            const uint4* a = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15));
            uint4 v[kVecs];
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i] = __ldg(a + i);
            shift_blocks<T, N>(q, v, static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)));
        }
    } else {
        load_ends(q, row, c, D);
    }
}
// The same columns of a row that is being written: row + c is on a 16-byte boundary.
// (At a row's ends the vector holds columns of a neighbouring row, which another block
// may be writing: those are not used.)
template <class T, int N>
__device__ __forceinline__ void load_own(Pack<T, N>& q, const unsigned char* row, int64_t c, int64_t D,
                                         const unsigned char* lo, const unsigned char* hi)
{
    const unsigned char* p = row + c * T::kBytes;
    if (p >= lo && p + N * T::kBytes <= hi) q.load_rw(p);
    else load_ends(q, row, c, D);
}
template <class T, int N>
__device__ __forceinline__ void store_row(const Pack<T, N>& q, unsigned char* row, int64_t c, int64_t D)
{
    if (c >= 0 && c + N <= D) {
        q.store(row + c * T::kBytes);
    } else {
#pragma unroll
        for (int g = 0; g < N / kGranule<T>; ++g)
            scatter_ends<T>(row, c + g * kGranule<T>, D,
                            make_uint4(q.w[4 * g], q.w[4 * g + 1], q.w[4 * g + 2], q.w[4 * g + 3]));
    }
}
// elements from the 16-byte boundary at or before the row to its first column
template <class T, bool ALIGNED>
__device__ __forceinline__ int row_offset(const unsigned char* row)
{
    return ALIGNED ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u) / T::kBytes;
}

// Eight fp32 columns of a thread are a 32-byte sector, written by two instructions of 16
// bytes: each would touch every sector of its warp's columns, by halves.  (Measured where
// a table is added to: 84 us with halves, 75 with whole sectors.)  So neighbouring threads
// exchange halves first.  `put` gets the addresses and four columns at a time; pairs: all
// threads of the warp have whole vectors of one row, next to one another.
template <class F>
__device__ __forceinline__ void put_columns(float* f, const float (&x)[8], bool pairs, F&& put)
{
    if (!pairs) {
        put(f, x[0], x[1], x[2], x[3]);
        put(f + 4, x[4], x[5], x[6], x[7]);
        return;
    }
    const bool odd = threadIdx.x & 1;
    float y[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float theirs = __shfl_xor_sync(0xffffffffu, odd ? x[j] : x[j + 4], 1);
        y[j] = odd ? theirs : x[j];
        y[j + 4] = odd ? x[j + 4] : theirs;
    }
    // even: its own first half and its neighbour's; odd: its neighbour's second half and its own
    float* even = f - (odd ? 8 : 0);
    put(even + (odd ? 4 : 0), y[0], y[1], y[2], y[3]);
    put(even + (odd ? 12 : 8), y[4], y[5], y[6], y[7]);
}
__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d)
{
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}

// ------------------------------------------------------------------ lookup
// `tpr` threads a row (a power of two), each with four vectors in flight.
constexpr int kVec = 8;                      // columns of a vector
constexpr int kFwdThreads = 128;
constexpr int kFwdUnroll = 4;

template <class TW, class TO, bool ALIGNED>
__global__ void __launch_bounds__(kFwdThreads) embedding_forward_kernel(const EmbParams p, const int tpr)
{
    constexpr int N = kVec;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kFwdThreads / tpr) + threadIdx.x / tpr;
    if (t >= p.T) return;
    const int lane = threadIdx.x & (tpr - 1);
    const int64_t id = load_id(p, t);
    const bool valid = id >= 0 && id < p.V;
    if (!valid && id != kIgnore && lane == 0) set_error(p.err, kErrBadTarget);
    unsigned char* out = at<TO>(p.rows, t, p.ld_rows, 0);
    const int off = row_offset<TO, ALIGNED>(out), D = static_cast<int>(p.D);
    const int step = tpr * N;
    if (!valid) {
        const float fill = id == kIgnore ? 0.f : __int_as_float(0x7fc00000);
        const float all[N] = {fill, fill, fill, fill, fill, fill, fill, fill};
        Pack<TO, N> o;
        o.set_all(all);
        for (int c = lane * N - off; c < D; c += step) store_row<TO, N>(o, out, c, D);
        return;
    }
    const unsigned char* w = at<TW>(const_cast<const void*>(p.table), id, p.ld_table, 0);
    const unsigned char* lo = static_cast<const unsigned char*>(p.table);
    // aligned rows: a row's last vector reads on into the next row, which the last one lacks
    const int whole = id + 1 < p.V ? D : D - N + 1;
    const bool warp_row = ALIGNED && tpr >= 32;
    for (int c0 = lane * N - off; c0 < D; c0 += step * kFwdUnroll) {
        Pack<TW, N> x[kFwdUnroll];
#pragma unroll
        for (int u = 0; u < kFwdUnroll; ++u) {
            const int c = c0 + u * step;
            if (c >= D) continue;
            if constexpr (ALIGNED) {
                if (c < whole) x[u].load(w + static_cast<int64_t>(c) * TW::kBytes);
                else load_ends(x[u], w, c, D);
            } else {
                load_row<TW, N, false>(x[u], w, c, D, lo, p.table_end);
            }
        }
#pragma unroll
        for (int u = 0; u < kFwdUnroll; ++u) {
            const int c = c0 + u * step;
            if (c >= D) continue;
            float y[N];
#pragma unroll
            for (int i = 0; i < N; ++i) y[i] = x[u].get(i) * p.scale;
            if (TO::kBytes == 4 && warp_row && c - (lane & 31) * N + 32 * N <= D) {
                put_columns(reinterpret_cast<float*>(out) + c, y, true, store4);
                continue;
            }
            Pack<TO, N> o;
            o.set_all(y);
            store_row<TO, N>(o, out, c, D);
        }
    }
}

// One table row's columns [c, c + N) from their sum.
template <class TO>
__device__ __forceinline__ void write_sum(const EmbParams& p, unsigned char* row, int64_t c, const float (&acc)[kVec])
{
    float y[kVec];
    if (p.accumulate) {
        Pack<TO, kVec> old;
        load_own<TO, kVec>(old, row, c, p.D, static_cast<const unsigned char*>(p.table), p.table_end);
#pragma unroll
        for (int i = 0; i < kVec; ++i) y[i] = fmaf(acc[i], p.scale, old.get(i));
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) y[i] = acc[i] * p.scale;
    }
    Pack<TO, kVec> o;
    o.set_all(y);
    store_row<TO, kVec>(o, row, c, p.D);
}

// ------------------------------------------- gradient of a few positions
// Zeros in this block's share of the rows [v0, v0 + rows) that are not `held`: the
// grid's second dimension divides the columns, all threads of the block one row.
template <class TO, bool ALIGNED, int THREADS>
__device__ __forceinline__ void zero_rows_not_held(const EmbParams& p, int64_t v0, int rows, const uint8_t* held)
{
    constexpr int kCols = kGranule<TO>;
    Pack<TO, kCols> z;
    z.zero();
    const int step = THREADS * gridDim.y;
    // Rows one after another: each run of them is one piece of memory, so that narrow rows
    // give every thread work too.  A row at a time, 74296 x 64 fp16 took 16 us, as runs 6; the
    // bf16 gradient of 262144 x 2048 takes 232 to 235 us either way.
    if (p.ld_table == p.D) {
        for (int r = 0; r < rows;) {
            if (held[r]) {
                ++r;
                continue;
            }
            int r1 = r + 1;
            while (r1 < rows && !held[r1]) ++r1;
            unsigned char* out = at<TO>(p.table, v0 + r, p.ld_table, 0);
            const int64_t n = (r1 - r) * p.D, off = row_offset<TO, ALIGNED>(out);
            for (int64_t c = static_cast<int64_t>(blockIdx.y * THREADS + threadIdx.x) * kCols - off; c < n; c += static_cast<int64_t>(step) * kCols)
                store_row<TO, kCols>(z, out, c, n);
            r = r1;
        }
        return;
    }
    const int per = static_cast<int>((p.D + (ALIGNED ? 0 : kGranule<TO> - 1) + kCols - 1) / kCols);
    for (int r = 0; r < rows; ++r) {
        if (held[r]) continue;
        unsigned char* out = at<TO>(p.table, v0 + r, p.ld_table, 0);
        const int off = row_offset<TO, ALIGNED>(out);
        for (int x = blockIdx.y * THREADS + threadIdx.x; x < per; x += step) {
            const int64_t c = static_cast<int64_t>(x) * kCols - off;
            if (c < p.D) store_row<TO, kCols>(z, out, c, p.D);
        }
    }
}

// One launch and no workspace.  A block takes one position and a range of columns: it
// looks through all ids for its own token, leaves if the token has an earlier position,
// and otherwise adds up all of them in order.  The blocks after these write zeros in
// the rows that no id names.  Every block reads all ids, so this is for few of them
// (measured, bf16 added to an fp32 table of 128256 x 4096: 192 positions 4.5 us here and
// 12.8 us sorted, 1024 positions 14.8 and 17.1).
constexpr int kFewThreads = 128;
constexpr int kFewSpan = 64;                 // table rows of a block that writes zeros, at most
constexpr int kFewPositions = 1024;
constexpr int kRowsAhead = 8;
static_assert(kFewPositions <= 32 * 32, "a warp holds the words of matches");

template <class TG, class TO, bool ALIGNED>
__global__ void __launch_bounds__(kFewThreads) few_positions_kernel(const EmbParams p, const int span)
{
    __shared__ uint32_t match[32];
    __shared__ uint16_t list[kFewPositions];
    __shared__ uint8_t held[kFewSpan];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // positions' blocks spread evenly among the others: they wait for memory, the others fill it
    const int64_t before = static_cast<int64_t>(blockIdx.x) * p.T / gridDim.x;
    if (before == (static_cast<int64_t>(blockIdx.x) + 1) * p.T / gridDim.x) {
        const int64_t v0 = (blockIdx.x - before) * span;
        if (tid < kFewSpan) held[tid] = 0;
        __syncthreads();
        for (int i = tid; i < p.T; i += kFewThreads) {
            const int64_t d = load_id(p, i) - v0;
            if (d >= 0 && d < span) held[d] = 1;
        }
        __syncthreads();
        zero_rows_not_held<TO, ALIGNED, kFewThreads>(p, v0, static_cast<int>(min(static_cast<int64_t>(span), p.V - v0)), held);
        return;
    }
    const int t = static_cast<int>(before);
    const int64_t id = load_id(p, t);
    if (tid < 32) match[tid] = 0;
    __syncthreads();
    bool earlier = false;
    for (int b = 0; b < p.T; b += kFewThreads) {
        const int i = b + tid;
        const bool same = i < p.T && load_id(p, i) == id;
        earlier = earlier || (same && i < t);
        const uint32_t word = __ballot_sync(0xffffffffu, same);
        if (lane == 0 && b / 32 + warp < 32) match[b / 32 + warp] = word;
    }
    if (id < 0 || id >= p.V) {
        if (id != kIgnore && tid == 0 && blockIdx.y == 0) set_error(p.err, kErrBadTarget);
        return;
    }
    if (__syncthreads_or(earlier)) return;
    if (warp == 0) {
        uint32_t word = match[lane];
        int inc = __popc(word);
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        for (int to = inc - __popc(word); word; word &= word - 1) list[to++] = static_cast<uint16_t>(lane * 32 + __ffs(word) - 1);
        if (lane == 31) count = inc;
    }
    __syncthreads();
    unsigned char* row = at<TO>(p.table, id, p.ld_table, 0);
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * kFewThreads + tid) * kVec - row_offset<TO, ALIGNED>(row);
    if (c >= p.D) return;
    const unsigned char* lo = static_cast<const unsigned char*>(p.rows);
    const int n = count;
    float acc[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) acc[k] = 0.f;
    for (int i = 0; i < n; i += kRowsAhead) {
        Pack<TG, kVec> g[kRowsAhead];
#pragma unroll
        for (int a = 0; a < kRowsAhead; ++a)
            if (i + a < n) load_row<TG, kVec, ALIGNED>(g[a], at<TG>(const_cast<const void*>(p.rows), list[i + a], p.ld_rows, 0), c, p.D, lo, p.rows_end);
#pragma unroll
        for (int a = 0; a < kRowsAhead; ++a)
            if (i + a < n) {
#pragma unroll
                for (int k = 0; k < kVec; ++k) acc[k] += g[a].get(k);
            }
    }
    write_sum<TO>(p, row, c, acc);
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

// The same by one thread-block cluster, for as many positions as its shared
// memory holds: each block keeps an equal share, and a pass moves keys between the
// blocks' shared memories.  (The passes above are nine launches of a few microseconds
// each, whose latency is most of a gradient's time at 10^4 positions.)  The launch's
// other clusters write zeros into the first table rows meanwhile, or, where the table is
// added to, bring the gradient's first rows into L2, from where the sums then read them
// (16384 x 4096 bf16 into fp32: 87.8 -> 84.1 us).
constexpr int kClusterBits = 9;
constexpr int kClusterDigits = 1 << kClusterBits;
constexpr int kClusterThreads = 1024;
constexpr int kClusterWarps = kClusterThreads / 32;
constexpr int kClusterMax = 16;              // blocks
constexpr int kClusterRounds = 8;            // keys a thread
constexpr int kClusterPositions = kClusterMax * kClusterRounds * kClusterThreads;

// Memory into L2, by the 16 bytes: a hint.
__device__ __forceinline__ void prefetch_l2(uintptr_t addr, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(addr), "r"(bytes) : "memory");
}

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t a)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(a) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t a, uint32_t b)
{
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// zeros in columns [0, D) of rows [r0, r1), by threads `me` of `all`
template <class TO, bool ALIGNED>
__device__ void zero_rows(const EmbParams& p, int64_t r0, int64_t r1, int64_t me, int64_t all)
{
    constexpr int kCols = kGranule<TO>;
    Pack<TO, kCols> z;
    z.zero();
    if (p.ld_table == p.D) {
        // one run of memory
        unsigned char* base = at<TO>(p.table, r0, p.ld_table, 0);
        const int64_t n = (r1 - r0) * p.D, off = row_offset<TO, ALIGNED>(base);
        for (int64_t c = me * kCols - off; c < n; c += all * kCols) store_row<TO, kCols>(z, base, c, n);
        return;
    }
    const int64_t per = (p.D + (ALIGNED ? 0 : kCols - 1) + kCols - 1) / kCols, n = per * (r1 - r0);
    for (int64_t i = me; i < n; i += all) {
        const int64_t r = i / per;
        unsigned char* row = at<TO>(p.table, r0 + r, p.ld_table, 0);
        const int64_t c = (i - r * per) * kCols - row_offset<TO, ALIGNED>(row);
        if (c < p.D) store_row<TO, kCols>(z, row, c, p.D);
    }
}

// What the SMs that do not sort do meanwhile, by threads `me` of `all`: zeros in the first
// `blind` rows of the table, the first `ahead` bytes of the gradient's rows into L2.
template <class TO, bool ALIGNED>
__device__ __forceinline__ void fill_or_fetch(const EmbParams& p, int64_t blind, int64_t ahead, int64_t me, int64_t all)
{
    zero_rows<TO, ALIGNED>(p, 0, blind, me, all);
    constexpr int kPiece = 2048;
    const uintptr_t from = (reinterpret_cast<uintptr_t>(p.rows) + 15) & ~uintptr_t(15);
    for (int64_t b = me * kPiece; b + kPiece <= ahead; b += all * kPiece) prefetch_l2(from + b, kPiece);
}

struct ClusterSort {
    int blocks, share;           // of the cluster; keys of a block
    int fill;                    // blocks that write zeros
    int bits, passes;            // of a digit
    int64_t blind, ahead;
    uint32_t *keys, *pos;        // [T] out
};

// dynamic shared memory: [2][share] (key, position), [warps][digits] 16-bit counts,
// [blocks][digits] 16-bit totals, [4][digits / 2] sums of a quarter of the warps, [digits] bases
__host__ __device__ constexpr size_t cluster_smem(int share)
{
    return sizeof(uint2) * 2 * static_cast<size_t>(share) +
           sizeof(uint16_t) * (kClusterWarps + kClusterMax) * kClusterDigits + 3 * sizeof(uint32_t) * kClusterDigits;
}

template <class TO, bool ALIGNED>
__global__ void __launch_bounds__(kClusterThreads) cluster_sort_kernel(const EmbParams p, const ClusterSort q)
{
    extern __shared__ __align__(16) unsigned char mem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dep_launch();
    if (blockIdx.x >= static_cast<unsigned>(q.blocks)) {
        fill_or_fetch<TO, ALIGNED>(p, q.blind, q.ahead, static_cast<int64_t>(blockIdx.x - q.blocks) * kClusterThreads + tid,
                                   static_cast<int64_t>(gridDim.x - q.blocks) * kClusterThreads);
        return;
    }
    // No block writes to another's shared memory before that one has started: the wait is
    // before the first such write, after the first pass's counting.
    cluster_arrive_relaxed();
    uint2* buf = reinterpret_cast<uint2*>(mem);
    uint16_t* bin = reinterpret_cast<uint16_t*>(buf + 2 * q.share);
    uint32_t* totals = reinterpret_cast<uint32_t*>(bin + kClusterWarps * kClusterDigits);
    uint32_t* quarters = totals + kClusterMax * kClusterDigits / 2;
    uint32_t* base = quarters + 2 * kClusterDigits;
    __shared__ uint32_t part[kClusterDigits / 32];
    uint32_t valid = 0;
    const int me = static_cast<int>(cluster_rank());
    const uint32_t magic = static_cast<uint32_t>(((uint64_t(1) << 32) + q.share - 1) / q.share);
    int held = max(0, min(q.share, p.T - me * q.share));
    // a warp's keys are consecutive, so ranks count up in position order
    const int per = (q.share + kClusterWarps - 1) / kClusterWarps;
    const int i0 = warp * per;

    for (int pass = 0; pass < q.passes; ++pass) {
        const int shift = pass * q.bits, digits = 1 << q.bits;
        const uint2* in = buf + (pass & 1) * q.share;
        uint4* z = reinterpret_cast<uint4*>(bin);
        for (int i = tid; i < kClusterWarps * kClusterDigits / 8; i += kClusterThreads) z[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        uint2 kp[kClusterRounds];
        uint32_t rank[kClusterRounds];
#pragma unroll
        for (int r = 0; r < kClusterRounds; ++r) {
            const int i = i0 + r * 32 + lane;
            const bool have = r * 32 + lane < per && i < held;
            if (have) {
                if (pass == 0) {
                    const int64_t t = static_cast<int64_t>(me) * q.share + i;
                    const uint32_t k = first_key(p, t);
                    kp[r] = make_uint2(k, k < static_cast<uint32_t>(p.V) ? static_cast<uint32_t>(t) : 0xffffffffu);
                } else {
                    kp[r] = in[i];
                }
            } else {
                kp[r] = make_uint2(0, 0xffffffffu);
            }
        }
#pragma unroll
        for (int r = 0; r < kClusterRounds; ++r) {
            if (r * 32 >= per) break;
            const bool have = kp[r].y != 0xffffffffu;
            const uint32_t d = have ? (kp[r].x >> shift) & (digits - 1) : kClusterDigits;
            const uint32_t same = __match_any_sync(0xffffffffu, d);
            uint16_t* c = bin + warp * kClusterDigits + d;
            uint32_t before = 0;
            if (have) before = *c;
            __syncwarp();
            if (have && lane == __ffs(same) - 1) *c = static_cast<uint16_t>(before + __popc(same));
            __syncwarp();
            rank[r] = before + __popc(same & ((1u << lane) - 1u));
        }
        __syncthreads();
        // digits 2 d and 2 d + 1 together, in the halves of a word: the warps' offsets by
        // quarters, and the block's totals, sent to every block of the cluster
        {
            constexpr int kPairs = kClusterDigits / 2, kQuarter = kClusterWarps / 4;
            const int d = tid & (kPairs - 1), quarter = tid / kPairs;
            uint32_t* word = reinterpret_cast<uint32_t*>(bin) + quarter * kQuarter * kPairs + d;
            uint32_t n[kQuarter], sum = 0;
#pragma unroll
            for (int w = 0; w < kQuarter; ++w) {
                n[w] = word[w * kPairs];
                sum += n[w];
            }
            quarters[quarter * kPairs + d] = sum;
            __syncthreads();
            uint32_t run = 0, total = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t y = quarters[x * kPairs + d];
                run += x < quarter ? y : 0;
                total += y;
            }
#pragma unroll
            for (int w = 0; w < kQuarter; ++w) {
                word[w * kPairs] = run;
                run += n[w];
            }
            const uint32_t mine = smem_addr(totals + me * kPairs + d);
            if (pass == 0) cluster_wait();
            for (int b = quarter; b < q.blocks; b += 4) st_cluster(dsmem_map(mine, b), total);
        }
        cluster_sync_all();
        // where the digit begins: after all smaller digits, and after the same digit of
        // the blocks before this one
        uint32_t all = 0, before_me = 0;
        if (tid < kClusterDigits) {
            const uint16_t* t = reinterpret_cast<const uint16_t*>(totals) + tid;
#pragma unroll 8
            for (int b = 0; b < q.blocks; ++b) {
                const uint32_t n = t[b * kClusterDigits];
                all += n;
                before_me += b < me ? n : 0;
            }
        }
        uint32_t inc = all;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31 && warp < kClusterDigits / 32) part[warp] = inc;
        __syncthreads();
        uint32_t smaller = 0;
        valid = 0;
#pragma unroll
        for (int x = 0; x < kClusterDigits / 32; ++x) {
            const uint32_t y = part[x];
            smaller += x < warp ? y : 0;
            valid += y;
        }
        if (tid < kClusterDigits) base[tid] = smaller + inc - all + before_me;
        __syncthreads();
        const bool last = pass + 1 == q.passes;
        const uint32_t out = smem_addr(buf + ((pass + 1) & 1) * q.share);
#pragma unroll
        for (int r = 0; r < kClusterRounds; ++r) {
            if (kp[r].y == 0xffffffffu) continue;
            const uint32_t d = (kp[r].x >> shift) & (digits - 1);
            const uint32_t to = base[d] + bin[warp * kClusterDigits + d] + rank[r];
            if (last) {
                q.keys[to] = kp[r].x;
                q.pos[to] = kp[r].y;
            } else {
                const uint32_t b = q.share == 1 ? to : __umulhi(to, magic);
                st_cluster(dsmem_map(out + static_cast<uint32_t>(sizeof(uint2)) * (to - b * q.share), b), kp[r].x, kp[r].y);
            }
        }
        // positions without a valid token were left out; they are the list's end
        held = max(0, min(q.share, static_cast<int>(valid) - me * q.share));
        if (last)
            for (int i = static_cast<int>(valid) + me * kClusterThreads + tid; i < p.T; i += q.blocks * kClusterThreads)
                q.keys[i] = static_cast<uint32_t>(p.V);
        // the next pass's keys are in place, and no block's totals are read any more
        cluster_sync_all();
    }
}

// A few thousand positions by counting: a position's place is the number of those that
// come before it, with a smaller token or the same one earlier.  A block takes kRanked
// positions, its threads take the others' keys from memory.  Nothing is passed between blocks,
// so T^2 comparisons spread over all SMs take less time than a cluster's passes, for as long
// as there are few of them (measured, whole gradients, bf16 rows of 4096 added to fp32 and of
// 512 to bf16, by counting and by a cluster: 1500 positions 17.6 and 23.6 us, 15.2 and 19.9;
// 4097 positions 28.2 and 32.5, 19.1 and 21.7; 6000 positions 32.6 and 35.7, 20.8 and 22.7;
// 8192 positions 52.3 and 50.5, 25.8 and 23.5).
// The blocks after these do what the cluster sort's other clusters do.
constexpr int kRankThreads = 256;
constexpr int kRankWarps = kRankThreads / 32;
constexpr int kRanked = 16;
constexpr int kRankAhead = 8;
constexpr int kRankPositions = 6144;

struct RankSort {
    int blocks;
    int64_t blind, ahead;
    uint32_t *keys, *pos;        // [T] out
};

template <class TO, bool ALIGNED>
__global__ void __launch_bounds__(kRankThreads) rank_sort_kernel(const EmbParams p, const RankSort q)
{
    __shared__ uint32_t own[kRanked];
    __shared__ uint32_t below[kRankWarps][kRanked];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dep_launch();
    if (blockIdx.x >= static_cast<unsigned>(q.blocks)) {
        fill_or_fetch<TO, ALIGNED>(p, q.blind, q.ahead, static_cast<int64_t>(blockIdx.x - q.blocks) * kRankThreads + tid,
                                   static_cast<int64_t>(gridDim.x - q.blocks) * kRankThreads);
        return;
    }
    const int i0 = static_cast<int>(blockIdx.x) * kRanked;
    if (tid < kRanked) own[tid] = i0 + tid < p.T ? first_key(p, i0 + tid) : 0;
    __syncthreads();
    int key[kRanked];
    uint32_t n[kRanked];
#pragma unroll
    for (int c = 0; c < kRanked; ++c) {
        key[c] = static_cast<int>(own[c]);
        n[c] = 0;
    }
    for (int j0 = tid; j0 < p.T; j0 += kRankAhead * kRankThreads) {
        int other[kRankAhead];
#pragma unroll
        for (int r = 0; r < kRankAhead; ++r) {
            const int j = j0 + r * kRankThreads;
            const int64_t id = j < p.T ? load_id(p, j) : p.V;
            // one less where it comes first among equals; keys are below 2^31
            other[r] = j < p.T ? (id >= 0 && id < p.V ? static_cast<int>(id) : p.V) - (j < i0 ? 1 : 0) : INT_MAX;
        }
#pragma unroll
        for (int r = 0; r < kRankAhead; ++r)
#pragma unroll
            for (int c = 0; c < kRanked; ++c) n[c] += other[r] < key[c] ? 1 : 0;
    }
#pragma unroll
    for (int c = 0; c < kRanked; ++c) {
        const uint32_t sum = __reduce_add_sync(0xffffffffu, n[c]);
        if (lane == 0) below[warp][c] = sum;
    }
    __syncthreads();
    if (tid >= kRanked || i0 + tid >= p.T) return;
    uint32_t to = 0;
#pragma unroll
    for (int w = 0; w < kRankWarps; ++w) to += below[w][tid];
    for (int c = 0; c < tid; ++c) to += own[c] == own[tid] ? 1 : 0;
    q.keys[to] = own[tid];
    q.pos[to] = static_cast<uint32_t>(i0 + tid);
}

// ------------------------------------------------------- sums by token
// A group of `tpr` threads takes a window of sorted positions and a vector of columns
// each.  A token whose positions all lie in the window is summed and written.  One that
// crosses a window's border leaves the window's part of its sum, in fp32: in slot 1
// where it begins in this window, in slot 0 where it came from the window before; the
// join adds a token's parts in an order that the windows fix.
//
// The blocks after these write zeros where no position holds the token: a block
// finds its rows' range in the sorted keys and passes over those that occur.
constexpr int kWindow = 32;                  // positions of a window, at most
constexpr int kSumThreads = 128;
constexpr int kZeroSpan = 64;                // table rows of a block that writes zeros
constexpr int kMaxGroups = 16;               // of a block: tpr >= 8

struct SumParams {
    EmbParams e;
    const uint32_t* keys;   // sorted
    const uint32_t* pos;
    float* parts;           // [windows][2][ld_parts]
    int64_t ld_parts;
    int window;
    int tpr;
    int sum_blocks;
    int64_t blind;          // rows already zero
    uint32_t* crossing;     // [windows] windows in which a crossing token begins
    unsigned* counters;     // [2] how many; blocks of the join finished
};

// the first sorted position whose key is at least v, by a block of kSumThreads
__device__ __forceinline__ int lower_bound(const uint32_t* keys, int n, uint32_t v)
{
    int lo = 0, hi = n;                                       // in [lo, hi]
    while (hi - lo > 0) {
        // each thread one probe; the probes below v come first
        const int step = (hi - lo + kSumThreads) / (kSumThreads + 1);
        const int64_t at = lo + static_cast<int64_t>(threadIdx.x + 1) * step - 1;
        const int below = __syncthreads_count(at < hi && keys[at] < v);
        lo += below * step;
        if (below < kSumThreads) hi = min(hi, lo + step - 1);   // the next probe is at least v
    }
    return lo;
}

template <class TO, bool ALIGNED>
__device__ void zero_absent_rows(const SumParams& p, int64_t v0, uint8_t* held)
{
    const EmbParams& e = p.e;
    const int tid = threadIdx.x;
    const int rows = static_cast<int>(min(static_cast<int64_t>(kZeroSpan), e.V - v0));
    if (tid < kZeroSpan) held[tid] = 0;
    int i = lower_bound(p.keys, e.T, static_cast<uint32_t>(v0)) + tid;
    __syncthreads();
    for (; i < e.T; i += kSumThreads) {
        const uint32_t k = p.keys[i];
        if (k >= v0 + rows) break;
        held[k - v0] = 1;
    }
    __syncthreads();
    zero_rows_not_held<TO, ALIGNED, kSumThreads>(e, v0, rows, held);
}

// Adds to memory without reading it first; every element is added to once, so the
// order of the blocks does not matter.  The price is a rounding (the product's, before the
// sum's) and that subnormals are flushed, the old value's too; a load and a fused product and sum
// would keep both and wait for each row's load (16384 bf16 rows added to 128256 x 4096, all of
// them tokens: 115 us that way, 85 this way; 65536 to 128256 x 2048: 182 and 142).
__device__ __forceinline__ void red_add4(float* p, float a, float b, float c, float d)
{
    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

template <class TG, class TO, bool ALIGNED>
__global__ void __launch_bounds__(kSumThreads, !ALIGNED ? 6 : (TO::kBytes == 4 ? 5 : 8)) token_sum_kernel(const SumParams p)
{
    constexpr int kAhead = TG::kBytes == 4 ? kRowsAhead / 2 : kRowsAhead;   // rows on their way
    __shared__ uint32_t key[kMaxGroups][kWindow + 2], row[kMaxGroups][kWindow];
    __shared__ int8_t shift[kMaxGroups][kWindow];   // from a 16-byte boundary to the table row
    __shared__ uint32_t ends_of[kMaxGroups];
    grid_dep_wait();
    grid_dep_launch();
    const EmbParams& e = p.e;
    const uint32_t none = static_cast<uint32_t>(e.V);
    const int tid = threadIdx.x;
    if (blockIdx.x >= static_cast<unsigned>(p.sum_blocks)) {
        zero_absent_rows<TO, ALIGNED>(p, p.blind + static_cast<int64_t>(blockIdx.x - p.sum_blocks) * kZeroSpan,
                                      reinterpret_cast<uint8_t*>(row));
        return;
    }
    const int groups = kSumThreads / p.tpr, g = tid / p.tpr, lane = tid & (p.tpr - 1);
    const int w = static_cast<int>(blockIdx.x) * groups + g;
    const int64_t i0 = static_cast<int64_t>(w) * p.window;
    if (lane == 0) ends_of[g] = 0;
    // key[.][0] and key[.][window + 1]: the keys before and after the window
    for (int i = lane; i < p.window + 2; i += p.tpr) {
        const int64_t at_ = i0 - 1 + i;
        key[g][i] = at_ >= 0 && at_ < e.T ? p.keys[at_] : none;
        if (i < p.window) row[g][i] = i0 + i < e.T ? p.pos[i0 + i] : 0;
    }
    __syncthreads();
    const uint32_t* k = key[g] + 1;
    for (int i = lane; i < p.window; i += p.tpr) {
        if (k[i] != none && (k[i + 1] != k[i] || i + 1 == p.window)) atomicOr(&ends_of[g], 1u << i);
        if (!ALIGNED)
            shift[g][i] = k[i] == none ? 0 : static_cast<int8_t>(row_offset<TO, ALIGNED>(at<TO>(e.table, k[i], e.ld_table, 0)));
    }
    __syncthreads();
    const uint32_t ends = ends_of[g];       // positions after which a run's sum is due
    if (ends == 0) return;
    const int n = 32 - __clz(ends);         // the last valid position ends a run
    const int64_t vec = static_cast<int64_t>(blockIdx.y) * p.tpr + lane;
    if (vec * kVec - (ALIGNED ? 0 : kGranule<TO> - 1) >= e.D) return;
    const int64_t c0 = vec * kVec;          // the vector's first column, where table rows are aligned
    const unsigned char* lo = static_cast<const unsigned char*>(e.rows);
    const unsigned char* base = lo + c0 * TG::kBytes;
    const int64_t ld_bytes = e.ld_rows * TG::kBytes;
    const uint32_t whole = c0 + kVec <= e.D ? 0xffffffffu : static_cast<uint32_t>(e.T - 1);

    // whole warps of whole vectors, of one window
    const bool pairs = ALIGNED && TO::kBytes == 4 && p.tpr >= 32 && (vec - (lane & 31) + 32) * kVec <= e.D;

    float acc[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) acc[i] = 0.f;
    int first = 0;   // where the current token's run begins in the window
    for (int b = 0; b < n; b += kAhead) {
        Pack<TG, kVec> x[kAhead];
#pragma unroll
        for (int r = 0; r < kAhead; ++r) {
            if (b + r >= n) continue;
            const uint32_t t = row[g][b + r];
            if constexpr (ALIGNED) {
                // a row's last vector reads on into the next row, which the last one lacks
                if (t < whole) x[r].load(base + t * ld_bytes);
                else load_ends(x[r], lo + t * ld_bytes, c0, e.D);
            } else {
                load_row<TG, kVec, false>(x[r], lo + t * ld_bytes, c0 - shift[g][b + r], e.D, lo, e.rows_end);
            }
        }
#pragma unroll
        for (int r = 0; r < kAhead; ++r) {
            const int i = b + r;
            if (i >= n) continue;
#pragma unroll
            for (int j = 0; j < kVec; ++j) acc[j] += x[r].get(j);
            if (!(ends >> i & 1u)) continue;
            // the run ends here, or goes on in the next window
            const uint32_t v = k[i];
            const bool from = first == 0 && k[-1] == v, on = i + 1 == p.window && k[i + 1] == v;
            const int64_t c = c0 - (ALIGNED ? 0 : shift[g][i]);
            if (from || on) {
                float* part = p.parts + (2 * static_cast<int64_t>(w) + (from ? 0 : 1)) * p.ld_parts;
                if (ALIGNED && c + kVec <= e.D) {
                    put_columns(part + c, acc, pairs, store4);
                } else {
#pragma unroll
                    for (int j = 0; j < kVec; ++j)
                        if (c + j >= 0 && c + j < e.D) part[c + j] = acc[j];
                }
                if (on && !from && lane == 0 && blockIdx.y == 0) p.crossing[atomicAdd(&p.counters[0], 1u)] = static_cast<uint32_t>(w);
            } else if (c < e.D) {
                unsigned char* out = at<TO>(e.table, v, e.ld_table, 0);
                if (TO::kBytes == 4 && e.accumulate && c >= 0 && c + kVec <= e.D) {
                    float* f = reinterpret_cast<float*>(out) + c;
                    float y[kVec];
#pragma unroll
                    for (int j = 0; j < kVec; ++j) y[j] = acc[j] * e.scale;
                    put_columns(f, y, pairs, red_add4);
                } else if (TO::kBytes == 4 && pairs) {
                    float y[kVec];
#pragma unroll
                    for (int j = 0; j < kVec; ++j) y[j] = acc[j] * e.scale;
                    put_columns(reinterpret_cast<float*>(out) + c, y, true, store4);
                } else {
                    write_sum<TO>(e, out, c, acc);
                }
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j) acc[j] = 0.f;
            first = i + 1;
        }
    }
}

// Crossing tokens' sums, kJoinCols columns an item.  A warp adds up the few windows of
// most tokens by itself, in window order; a token of more than kJoinAlone windows is left
// to the whole block, whose warps take every eighth window and are added in warp order.
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinCols = 128;
constexpr int kJoinAlone = 7;

template <class TO>
__global__ void __launch_bounds__(kJoinThreads) token_join_kernel(const SumParams p)
{
    __shared__ float4 sum[kJoinWarps][32];
    __shared__ int64_t long_item[kJoinWarps];
    __shared__ int long_more[kJoinWarps];
    const EmbParams& e = p.e;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dep_wait();
    const int64_t ranges = (e.D + kJoinCols - 1) / kJoinCols;
    const int64_t items = static_cast<int64_t>(__ldcg(p.counters)) * ranges;
    // windows first, first + step, ... of the `more` after window w, and w itself (x = 0);
    // eight are on their way at a time
    auto add = [&](int64_t w, int64_t c, int first, int more, int step) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c >= e.D) return acc;
        for (int x0 = first; x0 <= more; x0 += 8 * step) {
            float4 y[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int x = x0 + u * step;
                const int64_t slot = x == 0 ? 2 * w + 1 : 2 * (w + x);
                y[u] = x <= more ? __ldcg(reinterpret_cast<const float4*>(p.parts + slot * p.ld_parts + c))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                acc.x += y[u].x;
                acc.y += y[u].y;
                acc.z += y[u].z;
                acc.w += y[u].w;
            }
        }
        return acc;
    };
    struct Old {
        float x[4];
    };
    auto read_old = [&](uint32_t v, int64_t c) {
        const typename TO::raw* out = reinterpret_cast<const typename TO::raw*>(at<TO>(e.table, v, e.ld_table, 0));
        Old o{{0.f, 0.f, 0.f, 0.f}};
        if (e.accumulate) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < e.D) o.x[j] = TO::widen(out[c + j]);
        }
        return o;
    };
    auto write = [&](uint32_t v, int64_t c, float4 acc, const Old& o) {
        const float total[4] = {acc.x, acc.y, acc.z, acc.w};
        typename TO::raw* out = reinterpret_cast<typename TO::raw*>(at<TO>(e.table, v, e.ld_table, 0));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < e.D) out[c + j] = TO::round(e.accumulate ? fmaf(total[j], e.scale, o.x[j]) : total[j] * e.scale);
    };
    // neighbouring items, likely of one long token, go to different blocks
    for (int64_t item0 = blockIdx.x; item0 < items; item0 += static_cast<int64_t>(gridDim.x) * kJoinWarps) {
        const int64_t item = item0 + static_cast<int64_t>(warp) * gridDim.x;
        if (lane == 0) long_item[warp] = -1;
        if (item < items) {
            const int64_t w = __ldcg(p.crossing + item / ranges), c = (item % ranges) * kJoinCols + lane * 4;
            // the windows after this one that begin with its last token
            int more = 0;
            uint32_t v = 0;
            while (true) {
                const int64_t next = (w + 1 + more + lane) * p.window;
                const uint32_t k = next < e.T ? __ldcg(p.keys + next) : static_cast<uint32_t>(e.V);
                if (more == 0) v = __shfl_sync(0xffffffffu, k, 0);
                const int n = __popc(__ballot_sync(0xffffffffu, k == v));
                more += n;
                if (n < 32) break;
            }
            if (more <= kJoinAlone) {
                const Old o = read_old(v, c);
                write(v, c, add(w, c, 0, more, 1), o);
            } else if (lane == 0) {
                long_item[warp] = item;
                long_more[warp] = more;
            }
        }
        __syncthreads();
        for (int l = 0; l < kJoinWarps; ++l) {
            if (long_item[l] < 0) continue;
            const int64_t w = __ldcg(p.crossing + long_item[l] / ranges), c = (long_item[l] % ranges) * kJoinCols + lane * 4;
            float4 acc = add(w, c, warp, long_more[l], kJoinWarps);
            sum[warp][lane] = acc;
            __syncthreads();
            if (warp == 0) {
                for (int x = 1; x < kJoinWarps; ++x) {
                    const float4 y = sum[x][lane];
                    acc.x += y.x;
                    acc.y += y.y;
                    acc.z += y.z;
                    acc.w += y.w;
                }
                const uint32_t v = __ldcg(p.keys + (w + 1) * p.window);
                write(v, c, acc, read_old(v, c));
            }
            __syncthreads();
        }
        __syncthreads();
    }
    // the last block leaves the counters at zero
    __syncthreads();
    if (tid == 0 && count_done(&p.counters[1]) == gridDim.x - 1) {
        p.counters[0] = 0;
        p.counters[1] = 0;
    }
}

template <class TO, bool ALIGNED>
__global__ void __launch_bounds__(256) zero_table_kernel(const EmbParams p)
{
    zero_rows<TO, ALIGNED>(p, 0, p.V, static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x,
                           static_cast<int64_t>(gridDim.x) * blockDim.x);
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
    if (a->D > (int64_t(1) << 30)) return LMLOSS_ERR_UNSUPPORTED;
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

// every row of both matrices starts on a 16-byte boundary
bool aligned_rows(const lmloss_embedding_args* a)
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
    p.table_end = static_cast<const unsigned char*>(a->table) + ((a->V - 1) * a->ld_table + a->D) * float_bytes(a->table_dtype);
    p.rows_end = static_cast<const unsigned char*>(a->rows) +
                 (a->T > 0 ? ((a->T - 1) * a->ld_rows + a->D) * float_bytes(a->rows_dtype) : 0);
    return p;
}

// vectors of the longest row, its first one possibly begun early
int64_t row_vectors(const lmloss_embedding_args* a, int32_t written, bool aligned)
{
    return (a->D + (aligned ? 0 : 16 / float_bytes(written) - 1) + kVec - 1) / kVec;
}

// threads of a row: a power of two from 8 to `most`, as many as it has vectors
int threads_of_row(int64_t vecs, int most)
{
    int tpr = 8;
    while (tpr < most && tpr < vecs) tpr *= 2;
    return tpr;
}

struct SortSpace {
    size_t keys[2], pos[2], counts, crossing, parts, total;
    int tiles, window, windows;
    int64_t ld_parts;
};

SortSpace sort_space(const lmloss_embedding_args* a)
{
    SortSpace s{};
    const size_t T = static_cast<size_t>(a->T);
    s.tiles = static_cast<int>((a->T + kTile - 1) / kTile);
    // Windows of 32 positions, or fewer where those leave an SM without four windows, or without
    // two blocks; four where the rows are fp32, of which a thread has half as many on their way
    // (fp32 rows, 21064 x 64: 42 blocks 32.0 us, 165 blocks 26.5; 57897 x 137: 452 blocks 48.5, 905
    // blocks 44.1; bf16 rows, 65536 x 128: 512 blocks 39.9, 1024 blocks 45.6).
    const int64_t vecs = (a->D + kVec - 1) / kVec;
    const int tpr = threads_of_row(vecs, kSumThreads);
    const int64_t ranges = (vecs + tpr - 1) / tpr;
    s.window = kWindow;
    while (s.window > 8) {
        const int64_t groups = (a->T + s.window - 1) / s.window * ranges;
        if (groups >= 600 && groups * tpr / kSumThreads >= (a->rows_dtype == LMLOSS_FP32 ? 600 : 300)) break;
        s.window /= 2;
    }
    s.windows = static_cast<int>((a->T + s.window - 1) / s.window);
    s.ld_parts = (a->D + 7) / 8 * 8;
    size_t off = 0;
    auto take = [&](size_t bytes) { size_t o = off; off = vocab_align(off + bytes); return o; };
    for (int i = 0; i < 2; ++i) {
        s.keys[i] = take(4 * T);
        s.pos[i] = take(4 * T);
    }
    s.counts = take(sizeof(uint32_t) * kDigits * static_cast<size_t>(s.tiles));
    s.crossing = take(sizeof(uint32_t) * static_cast<size_t>(s.windows));
    s.parts = take(sizeof(float) * 2 * static_cast<size_t>(s.windows) * static_cast<size_t>(s.ld_parts));
    s.total = off;
    return s;
}

// What any gradient of up to T positions and D columns needs, whatever its rows' type.
// A window is halved, from 2 w to w, only where 2 w leaves fewer than 600 groups or fewer than
// 600 blocks of them: then ceil(T / 2 w) x ranges x tpr < 600 kSumThreads, where ranges x tpr is
// at least the row's vectors and at least 8.  So a call has windows of 32, or at most `most` of
// them and of their vectors; the bound on each grows with T and D, though a call's own need does
// not (4800 positions of 4096 columns: 16 a window; 4096 positions: 8 a window, and more parts).
size_t most_space(int64_t T, int64_t D)
{
    const int64_t vecs = (D + kVec - 1) / kVec, most = 2 * (600 * kSumThreads - 1);
    const int64_t long_ = (T + kWindow - 1) / kWindow, short_ = (T + 7) / 8;
    const int64_t windows = std::max(long_, std::min(short_, most / 8));
    const int64_t parts = std::max(long_ * vecs, std::min(short_ * vecs, most)) * kVec;
    const int64_t tiles = (T + kTile - 1) / kTile;
    return 4 * vocab_align(4 * static_cast<size_t>(T)) + vocab_align(sizeof(uint32_t) * kDigits * static_cast<size_t>(tiles)) +
           vocab_align(sizeof(uint32_t) * static_cast<size_t>(windows)) + vocab_align(sizeof(float) * 2 * static_cast<size_t>(parts));
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
template <class F>
lmloss_status by_types(const lmloss_embedding_args* a, F&& f)
{
    const bool aligned = aligned_rows(a);
    return by_type(a->table_dtype, [&](auto table) {
        return by_type(a->rows_dtype, [&](auto rows) {
            return aligned ? f(table, rows, std::true_type{}) : f(table, rows, std::false_type{});
        });
    });
}

// A kernel that may be launched while the one before it on the stream still runs (it
// waits for that one's writes itself).
template <class K, class P>
lmloss_status launch_after(K* fn, dim3 grid, int threads, cudaStream_t stream, const P& p)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fn, p) != cudaSuccess) {
        cudaGetLastError();
        return LMLOSS_ERR_CUDA;
    }
    return LMLOSS_OK;
}

template <class TO, bool ALIGNED>
lmloss_status launch_cluster_sort(lmloss_vocab_ctx* h, const EmbParams& p, ClusterSort& q, cudaStream_t stream)
{
    auto* fn = cluster_sort_kernel<TO, ALIGNED>;
    const size_t smem = cluster_smem(q.share);
    // the kernel's limits, raised to the most that any call needs, once a handle
    const uint32_t bit = 1u << (2 * TO::kIndex + (ALIGNED ? 1 : 0));
    if (!(h->limits_raised & bit)) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(cluster_smem(kClusterRounds * kClusterThreads))) != cudaSuccess ||
            cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
            cudaGetLastError();
            return LMLOSS_ERR_CUDA;
        }
        h->limits_raised |= bit;
    }
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(q.blocks);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(q.blocks + q.fill));
    cfg.blockDim = dim3(kClusterThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fn, p, q) != cudaSuccess) {
        cudaGetLastError();
        return LMLOSS_ERR_CUDA;
    }
    return LMLOSS_OK;
}

// The table rows to fill blindly, or the bytes to fetch, in the `us` microseconds of a sort:
// about what the other SMs write in that time, at 5 TB/s.
void meanwhile(const lmloss_embedding_args* a, const EmbParams& p, int64_t us, int64_t& blind, int64_t& ahead)
{
    const int64_t row_bytes = a->D * float_bytes(a->table_dtype), bytes = us * 5000000;
    if (a->accumulate) {
        // whole rows' memory less the bytes before its first 16-byte boundary; half of L2
        const int64_t held = static_cast<int64_t>(p.rows_end - static_cast<const unsigned char*>(a->rows));
        ahead = std::min<int64_t>({held - 16, bytes, int64_t(64) << 20});
    } else {
        blind = bytes / row_bytes;
        if (blind > a->V * 3 / 4) blind = a->V;   // little is left to be found out
    }
}

lmloss_status sort_by_rank(const lmloss_vocab_ctx* h, const lmloss_embedding_args* a, const SortSpace& s, SumParams& p,
                           cudaStream_t stream)
{
    RankSort q{};
    q.blocks = (p.e.T + kRanked - 1) / kRanked;
    q.keys = reinterpret_cast<uint32_t*>(h->ws + s.keys[0]);
    q.pos = reinterpret_cast<uint32_t*>(h->ws + s.pos[0]);
    // more than fits beside the counting, which takes 2 to 6 us: zeros written here need no
    // look at the keys (bf16 tables of 32003 x 1001, 128256 x 512 and 100000 x 1024, 2048 positions:
    // 26.2, 34.8 and 49.1 us with 4 us of zeros, 24.6, 30.4 and 44.1 with 13, 24.5, 33.5 and 50 with 30)
    meanwhile(a, p.e, 13, q.blind, q.ahead);
    p.keys = q.keys;
    p.pos = q.pos;
    p.blind = q.blind;
    const bool aligned = aligned_rows(a);
    const unsigned grid = static_cast<unsigned>(q.blocks + 12 * h->num_sms);
    return by_type(a->table_dtype, [&](auto to) {
        using TO = decltype(to);
        if (aligned) rank_sort_kernel<TO, true><<<grid, kRankThreads, 0, stream>>>(p.e, q);
        else rank_sort_kernel<TO, false><<<grid, kRankThreads, 0, stream>>>(p.e, q);
        return vocab_launch_err();
    });
}

lmloss_status sort_in_cluster(lmloss_vocab_ctx* h, const lmloss_embedding_args* a, const SortSpace& s, SumParams& p,
                              cudaStream_t stream)
{
    ClusterSort q{};
    q.blocks = 1;
    while (q.blocks < kClusterMax && q.blocks * kClusterThreads < p.e.T) q.blocks *= 2;
    q.share = (p.e.T + q.blocks - 1) / q.blocks;
    int bits = 1;
    while ((static_cast<int64_t>(p.e.V - 1) >> bits) != 0) ++bits;
    q.passes = (bits + kClusterBits - 1) / kClusterBits;
    q.bits = (bits + q.passes - 1) / q.passes;
    q.keys = reinterpret_cast<uint32_t*>(h->ws + s.keys[0]);
    q.pos = reinterpret_cast<uint32_t*>(h->ws + s.pos[0]);
    // by the SMs that the cluster leaves
    q.fill = (h->num_sms - q.blocks) / q.blocks * q.blocks;
    // measured: 12 us and 1 us more for every 4700 positions
    if (q.fill > 0) meanwhile(a, p.e, 12 + a->T / 4700, q.blind, q.ahead);
    p.keys = q.keys;
    p.pos = q.pos;
    p.blind = q.blind;
    const bool aligned = aligned_rows(a);
    return by_type(a->table_dtype, [&](auto to) {
        using TO = decltype(to);
        return aligned ? launch_cluster_sort<TO, true>(h, p.e, q, stream) : launch_cluster_sort<TO, false>(h, p.e, q, stream);
    });
}

lmloss_status sort_in_passes(const lmloss_vocab_ctx* h, const SortSpace& s, SumParams& q, cudaStream_t stream)
{
    const EmbParams& p = q.e;
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
    q.blind = 0;
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
    *bytes = a->T <= kFewPositions ? 0 : most_space(a->T, a->D);
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
    return by_types(a, [&](auto tw, auto to, auto aligned) {
        const int64_t vecs = row_vectors(a, a->rows_dtype, aligned.value);
        const int tpr = threads_of_row((vecs + kFwdUnroll - 1) / kFwdUnroll, kFwdThreads), rows = kFwdThreads / tpr;
        embedding_forward_kernel<decltype(tw), decltype(to), aligned.value>
            <<<static_cast<unsigned>((p.T + rows - 1) / rows), kFwdThreads, 0, stream>>>(p, tpr);
        return vocab_launch_err();
    });
}

lmloss_status lmloss_embedding_backward(lmloss_vocab_handle h, const lmloss_embedding_args* a, cudaStream_t stream)
{
    if (!h) return LMLOSS_ERR_INVALID_ARG;
    lmloss_status st = check_embedding(a, true);
    if (st != LMLOSS_OK) return st;
    const bool few = a->T <= kFewPositions;   // one launch, no workspace
    const SortSpace s = few ? SortSpace{} : sort_space(a);
    if (s.total > h->ws_bytes) return LMLOSS_ERR_INVALID_ARG;
    // column ranges are numbered by the grid's second dimension
    const bool aligned = aligned_rows(a);
    const int64_t vecs = row_vectors(a, a->table_dtype, aligned);
    if (vecs > 65535LL * kSumThreads) return LMLOSS_ERR_UNSUPPORTED;
    VocabDeviceGuard g(h->device);
    if (!g.ok) return LMLOSS_ERR_CUDA;
    SumParams q{};
    q.e = params(h, a);
    if (a->T == 0) {
        if (a->accumulate) return LMLOSS_OK;
        return by_types(a, [&](auto to, auto, auto al) {
            zero_table_kernel<decltype(to), al.value><<<8 * h->num_sms, 256, 0, stream>>>(q.e);
            return vocab_launch_err();
        });
    }
    if (few) {
        const int64_t ranges = (vecs + kFewThreads - 1) / kFewThreads;
        int span = kFewSpan;   // or fewer rows, where that leaves SMs without four blocks
        while (span > 1 && (a->V + span - 1) / span * ranges < 4 * h->num_sms) span /= 2;
        const int64_t zero_blocks = a->accumulate ? 0 : (a->V + span - 1) / span;
        const dim3 grid(static_cast<unsigned>(a->T + zero_blocks), static_cast<unsigned>(ranges));
        return by_types(a, [&](auto to, auto tg, auto al) {
            few_positions_kernel<decltype(tg), decltype(to), al.value><<<grid, kFewThreads, 0, stream>>>(q.e, span);
            return vocab_launch_err();
        });
    }
    st = a->T <= kRankPositions      ? sort_by_rank(h, a, s, q, stream)
         : a->T <= kClusterPositions ? sort_in_cluster(h, a, s, q, stream)
                                     : sort_in_passes(h, s, q, stream);
    if (st != LMLOSS_OK) return st;
    q.parts = reinterpret_cast<float*>(h->ws + s.parts);
    q.ld_parts = s.ld_parts;
    q.window = s.window;
    q.crossing = reinterpret_cast<uint32_t*>(h->ws + s.crossing);
    q.counters = h->counters;
    q.tpr = threads_of_row(vecs, kSumThreads);
    const int groups = kSumThreads / q.tpr;
    q.sum_blocks = (s.windows + groups - 1) / groups;
    const int64_t zero_blocks = a->accumulate ? 0 : (a->V - q.blind + kZeroSpan - 1) / kZeroSpan;
    const dim3 grid(static_cast<unsigned>(q.sum_blocks + zero_blocks), static_cast<unsigned>((vecs + q.tpr - 1) / q.tpr));
    return by_types(a, [&](auto to, auto tg, auto al) {
        const lmloss_status e =
            launch_after(token_sum_kernel<decltype(tg), decltype(to), al.value>, grid, kSumThreads, stream, q);
        if (e != LMLOSS_OK) return e;
        return launch_after(token_join_kernel<decltype(to)>, dim3(static_cast<unsigned>(5 * h->num_sms)), kJoinThreads, stream, q);
    });
}

}  // extern "C"
