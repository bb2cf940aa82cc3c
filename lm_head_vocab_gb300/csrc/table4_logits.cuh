// What the two kernels of a 4-bit table's logits share: how numbers widen, how hidden rows are laid out,
// what a stage of the table holds.
#pragma once

#include <cuda.h>

#include "table4.cuh"
#include "tcgen05.cuh"

namespace lmloss {

constexpr int kBlockCols = 128;              // columns that hidden rows are laid out by
constexpr int kMaxStages = 8;
constexpr uint32_t kMaxShared = 227 * 1024;
constexpr int kFewRows = 8;                 // operand rows up to which warps multiply on their own

struct LogitsParams {
    const uint8_t* values;
    int64_t ld_values;
    const unsigned char* scales;
    int64_t ld_scales;
    const uint8_t* zeros;
    int64_t ld_zeros;
    int V, D, shift;             // shift: log2 of the group
    int scale_dtype, scale_bytes;
    int groups;                  // of a row
    int kblocks;                 // runs of kBlockCols columns of a row
    int T;                       // hidden rows
    int N;                       // operand rows of a block's product
    int per;                     // hidden rows a block takes: N, or N / 2 as pairs
    int tblocks;                 // runs of `per` hidden rows
    int vtiles;
    int pairs;                   // operand rows 0 .. N / 2 - 1 the upper parts, the others the lower ones times 2^11
    const unsigned char* x;      // [tblocks][kblocks][N * 256 bytes]: the hidden rows as fp16
    const float* inverse;        // [T] by which a row's sums are multiplied; NaN: the row is not finite
    const void* hidden;          // the rows as they came
    int64_t ld_hidden;
    int hidden_dtype;
    void* out;
    int64_t ld_out;
    int out_dtype;
    float scale;
    int qstages, xstages;
    uint32_t stage_bytes;        // of a stage of the table
    int* err;
};

// A word's eight numbers as fp16 pairs in the order 0 4 1 5 2 6 3 7.  The bits of a number in an fp16's low
// bits ARE q 2^-24, a subnormal; four bits further up q 2^-20.  So the odd places' hidden values are laid out
// divided by 16, and five operations widen eight numbers.  (By magic numbers: nine.)
__device__ __forceinline__ void widen_word(uint32_t w, uint32_t* out)
{
    const uint32_t w8 = w >> 8;
    out[0] = w & 0x000f000fu;
    out[1] = w & 0x00f000f0u;
    out[2] = w8 & 0x000f000fu;
    out[3] = w8 & 0x00f000f0u;
}
// (a & b) | c as one operation
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// The same less a zero point, (q - z) 2^-14 and (q - z) 2^-10, exact: under an exponent whose last place is 2^-14, less
// 2^-4 + z 2^-14 or 2^-4 + z 2^-10, exact.  As fp16's normal numbers: of subnormal ones the tensor cores cut sums off at some
// 2^-24 of what their exponent could hold, 2^6 to 2^10 times what they do (logits of bf16 rows 5e-7 off, not 2e-7, and
// far more beside one large column).
__device__ __forceinline__ void widen_word(uint32_t w, __half2 z, __half2 z16, uint32_t* out)
{
    const uint32_t w8 = w >> 8;
    out[0] = and_or(w, 0x000f000fu, 0x2c002c00u);
    out[1] = and_or(w, 0x00f000f0u, 0x2c002c00u);
    out[2] = and_or(w8, 0x000f000fu, 0x2c002c00u);
    out[3] = and_or(w8, 0x00f000f0u, 0x2c002c00u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(out + i), i & 1 ? z16 : z);
        out[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
}

__device__ __forceinline__ float widen_any(const void* base, int dtype, int64_t i)
{
    if (dtype == LMLOSS_BF16) return Bf16::widen(static_cast<const uint16_t*>(base)[i]);
    if (dtype == LMLOSS_FP16) return Fp16::widen(static_cast<const uint16_t*>(base)[i]);
    return static_cast<const float*>(base)[i];
}

__device__ __forceinline__ void store_logit(const LogitsParams& p, int64_t t, int64_t v, float x)
{
    const int64_t at = t * p.ld_out + v;
    if (p.out_dtype == LMLOSS_BF16) static_cast<uint16_t*>(p.out)[at] = Bf16::round(x);
    else if (p.out_dtype == LMLOSS_FP16) static_cast<uint16_t*>(p.out)[at] = Fp16::round(x);
    else static_cast<float*>(p.out)[at] = x;
}

// The power of two that brings a row's largest finite value to between 2^14 and 2^15, at most 2^126.  (A
// subnormal's exponent counts as -127.)
__device__ __forceinline__ float hidden_scale(float top)
{
    const int e = static_cast<int>(__float_as_uint(top) >> 23);
    return top > 0.f ? __uint_as_float(static_cast<uint32_t>(min(14 + 254 - e, 253)) << 23) : 1.f;
}
// Eight columns of a hidden row from c on, 0 past the last.
template <class X>
__device__ __forceinline__ void load_part(const typename X::raw* x, int c, int D, Pack<X, 8>& q)
{
    if (c + 8 <= D && (reinterpret_cast<uintptr_t>(x + c) & 15u) == 0) {
        q.load(x + c);
    } else {
        q.zero();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < D) q.set(i, X::widen(x[c + i]));
    }
}
// They scaled as a 16-byte part: fp16 in the order 0 4 1 5 2 6 3 7, the places 1 5 and 3 7 divided by 16.  The sums are of
// what the parts stand for, in the products' unit of 2^-24.  A scale of 0 is a row that is not finite.
// Of a pair, lo is what hi leaves, times 2^11, and hi a whole number of steps, the same for all columns of a table's
// group, 2^11 of which reach its largest: then a group's sum of products, below 15 * 2^11 * 128 < 2^22 steps, is exact.
// The tensor cores cut their sums off, one way, at some 2^-24 of the largest term: with hi rounded by each value's own
// exponent logits of 1001 columns were up to 2e-6 off, ten times as far as sums in fp32.
// What is left out: lo has 11 bits of a rest below 2^-11 of the power of two at or below the group's largest, 2^-23 of
// that largest, down to half a subnormal's step, 2^-36 (2^-32 in the places divided by 16), or hi's least step's:
// 2^-46 of the row's largest.  A third part would hold the rest, for half as many operand rows again; where one
// column is thousands of times the others only logits that it does not enter (q = z there) show the difference.
template <class X, bool PAIR>
__device__ __forceinline__ void hidden_part(const Pack<X, 8>& v, float scale, float group_top, uint4& hi, uint4& lo, float& sum, float& sum_lo)
{
    uint32_t h[4], l[4] = {0, 0, 0, 0};
    sum = sum_lo = 0.f;
    // x + magic - magic: x in steps of 2^-10 of the power of two at or below the group's largest, or of 2^-20 (fp16's
    // last place, for the places divided by 16)
    const uint32_t e = __float_as_uint(group_top * scale) >> 23;
    const float magic = 1.5f * __uint_as_float((max(e, 117u) + 13u) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float by = i & 1 ? scale * 0.0625f : scale, back = i & 1 ? 0x1p-20f : 0x1p-24f;
        const float a = scale > 0.f ? v.get(i) * by : 0.f, b = scale > 0.f ? v.get(i + 4) * by : 0.f;
        const float m = i & 1 ? magic * 0.0625f : magic;
        const __half2 p = PAIR ? __floats2half2_rn(__fadd_rn(__fadd_rn(a, m), -m), __fadd_rn(__fadd_rn(b, m), -m)) : __floats2half2_rn(a, b);
        h[i] = *reinterpret_cast<const uint32_t*>(&p);
        const float2 f = __half22float2(p);
        sum = fmaf(f.x, back, fmaf(f.y, back, sum));
        if (PAIR) {
            const __half2 r = __floats2half2_rn((a - f.x) * 2048.f, (b - f.y) * 2048.f);
            l[i] = *reinterpret_cast<const uint32_t*>(&r);
            const float2 e = __half22float2(r);
            sum_lo = fmaf(e.x, back, fmaf(e.y, back, sum_lo));
        }
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}
// The largest finite magnitude of eight columns, and whether there are others.
template <class X>
__device__ __forceinline__ float part_top(const Pack<X, 8>& v, bool& odd)
{
    float top = 0.f;
    odd = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = fabsf(v.get(i));
        if (a < INFINITY) top = fmaxf(top, a);
        else odd = true;
    }
    return top;
}
// The largest over the `lanes` (4, 8 or 16) neighbouring threads of a group, 16 threads together.
__device__ __forceinline__ float group_top(int lanes, float top)
{
    const uint32_t together = 0xffffu << (threadIdx.x & 16);
    for (int o = 1; o < lanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(together, top, o));
    return top;
}
// Sums over the `lanes` (4, 8 or 16) neighbouring threads of a group, 16 threads together.
__device__ __forceinline__ void group_sums(int lanes, float& sum, float& sum_lo)
{
    const uint32_t together = 0xffffu << (threadIdx.x & 16);
    for (int o = 1; o < lanes; o <<= 1) {
        sum += __shfl_xor_sync(together, sum, o);
        sum_lo += __shfl_xor_sync(together, sum_lo, o);
    }
}

// One logit of a row with infinities or NaN, from the formula: operands that are all finite and sums taken
// apart do not give what such a row gives.
static __device__ __noinline__ void store_plain(const LogitsParams& p, int64_t t, int64_t v)
{
    float acc = 0.f;
    for (int g = 0; g < p.groups; ++g) {
        const float s = widen_any(p.scales, p.scale_dtype, g * p.ld_scales + v);
        const float z = p.zeros ? static_cast<float>(p.zeros[g * p.ld_zeros + v]) : 8.f;
        const int end = min(p.D, (g + 1) << p.shift);
        float sum = 0.f;
        for (int c = g << p.shift; c < end; ++c) {
            const int q = p.values[v * p.ld_values + (c >> 1)] >> (4 * (c & 1)) & 15;
            sum = fmaf(widen_any(p.hidden, p.hidden_dtype, t * p.ld_hidden + c), static_cast<float>(q) - z, sum);
        }
        acc = fmaf(s, sum, acc);
    }
    store_logit(p, t, v, acc * p.scale);
}

// A ring's position: which slot, and the parity of the round.
struct Ring {
    int slot = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next(int n)
    {
        if (++slot == n) {
            slot = 0;
            parity ^= 1u;
        }
    }
};

// Where a stage's parts begin, and what they hold: values [runs of 256 columns][rows][128 bytes, 16-byte parts at
// (part ^ row % 8)], scales and zeros [groups of the stage][rows].
struct StageLayout {
    uint32_t scales, zeros, copied, bytes;
    __host__ __device__ StageLayout(int rows, int columns, int shift, int scale_bytes, bool has_zeros)
    {
        const int n = columns >> shift;
        scales = rows * (columns / 2);
        zeros = scales + n * rows * scale_bytes;
        copied = zeros + (has_zeros ? n * rows : 0);
        bytes = (copied + 1023) / 1024 * 1024;
    }
};

// A table's parts as tiles: [V, D / 2 bytes] by rows x 128, [G, V] by a stage's groups x rows.  What lies
// outside is 0.
struct TableMaps {
    CUtensorMap values, scales, zeros;
};

// Copies of `runs` runs of 256 columns from 256 `run` on and their groups, for the tile at row v0, by one thread:
// lay.copied bytes less the values of missing runs.  (As bulk copies, one a group, scales took longer than the
// values: 128256 x 4096, no arithmetic, 63 us with them and 46 without.)
__device__ __forceinline__ void copy_table(const LogitsParams& p, const StageLayout& lay, const TableMaps& maps, int rows, int run, int runs, int v0,
                                           uint32_t to, uint32_t bar)
{
    const int g = (run * 256) >> p.shift;
    for (int i = 0; i < runs; ++i) tile_load_2d(to + i * rows * 128, &maps.values, (run + i) * 128, v0, bar);
    tile_load_2d(to + lay.scales, &maps.scales, v0, g, bar);
    if (p.zeros) tile_load_2d(to + lay.zeros, &maps.zeros, v0, g, bar);
}

// Whether the kernel of independent warps takes a call: up to kFewRows operand rows that fit into shared memory
// beside two stages.
bool few_rows_fit(const LogitsParams& p);
// Its tiles, for the maps: rows, and columns of a stage.
constexpr int kFewTile = 64, kFewCols = 1024;
lmloss_status launch_few_rows(LogitsParams& p, const TableMaps& maps, lmloss_vocab_ctx* h, cudaStream_t stream);

}  // namespace lmloss
