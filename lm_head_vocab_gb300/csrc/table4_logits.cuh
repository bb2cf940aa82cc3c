// What the two kernels of a 4-bit table's logits share: how numbers widen, how hidden rows are laid out,
// what a stage of the table holds.
#pragma once

#include <cuda.h>

#include "table4.cuh"
#include "tcgen05.cuh"

namespace lmloss {

constexpr int kTile = 256;                   // rows of the table a block takes at once
constexpr int kStageCols = 256;              // columns of the table a stage holds
constexpr int kBlockCols = 128;              // columns that hidden rows are laid out by
constexpr int kMaxStages = 8;
constexpr uint32_t kMaxShared = 227 * 1024;
constexpr int kFewRows = 32;                 // operand rows up to which warps multiply on their own

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
    int pairs;                   // fp32: operand rows 0 .. N / 2 - 1 the upper parts, the others the lower ones times 2^11
    const unsigned char* x;      // [tblocks][kblocks][N * 256 bytes]: the hidden rows as fp16
    const float* sums;           // [tblocks][groups][N]: sums of their groups, as the products count them
    const float* inverse;        // [T] by which a row's sums are multiplied; NaN: the row is not finite
    const void* hidden;          // the rows as they came
    int64_t ld_hidden;
    int hidden_dtype;
    void* out;
    int64_t ld_out;
    int out_dtype;
    float scale;
    int qstages, xstages;
    uint32_t stage_bytes;        // of a stage of the table: values, scales, zeros, sums (and hidden rows)
    int* err;
};

// A word's eight numbers as fp16 pairs in the order 0 4 1 5 2 6 3 7.  The bits of a number in an fp16's low
// bits ARE q 2^-24, a subnormal; four bits further up q 2^-20.  So the odd places' hidden values are laid out
// divided by 16, and five operations widen eight numbers.  (q - z by magic numbers: nine.)  The zero points
// are taken off the sums: sum (q - z) x = sum q x - z sum x.
__device__ __forceinline__ void widen_word(uint32_t w, uint32_t* out)
{
    const uint32_t w8 = w >> 8;
    out[0] = w & 0x000f000fu;
    out[1] = w & 0x00f000f0u;
    out[2] = w8 & 0x000f000fu;
    out[3] = w8 & 0x00f000f0u;
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

// Where a stage's parts begin, and what they hold: values [256 rows][128 bytes, 16-byte parts at
// (part ^ row % 8)], scales, zeros [groups of the stage][256 rows], sums [groups][N].
struct StageLayout {
    uint32_t scales, zeros, sums, x, bytes;
    __host__ __device__ StageLayout(int shift, int scale_bytes, bool has_zeros, int N, uint32_t x_bytes)
    {
        const int n = kStageCols >> shift;
        scales = kTile * 128;
        zeros = scales + n * kTile * scale_bytes;
        sums = zeros + (has_zeros ? n * kTile : 0);
        x = sums + n * N * 4;
        bytes = (x + x_bytes + 1023) / 1024 * 1024;
    }
};

// Copies of the table's part of stage `st` of the tile at row v0, by a whole warp; the barrier expects
// stage_tx(...) bytes.
__device__ __forceinline__ uint32_t stage_rows(int rows, int bytes)
{
    // to the end of the 16 bytes that hold the last row's
    const int whole = 16 / bytes;
    return static_cast<uint32_t>((min(rows, kTile) + whole - 1) / whole * whole);
}
__device__ __forceinline__ uint32_t stage_tx(const LogitsParams& p, int n, int v0)
{
    return kTile * 128 + n * (stage_rows(p.V - v0, p.scale_bytes) * p.scale_bytes + (p.zeros ? stage_rows(p.V - v0, 1) : 0u) + p.N * 4);
}
__device__ __forceinline__ void copy_table(const LogitsParams& p, const StageLayout& lay, const CUtensorMap& map, int st, int n, int v0,
                                           uint32_t to, uint32_t bar)
{
    const int lane = threadIdx.x & 31;
    if (lane == 0) tile_load_2d(to, &map, st * 128, v0, bar);
    if (lane < n) {
        const int64_t g = static_cast<int64_t>(st) * (kStageCols >> p.shift) + lane;
        bulk_load(to + lay.scales + lane * kTile * p.scale_bytes, p.scales + (g * p.ld_scales + v0) * p.scale_bytes,
                  stage_rows(p.V - v0, p.scale_bytes) * p.scale_bytes, bar);
        if (p.zeros) bulk_load(to + lay.zeros + lane * kTile, p.zeros + g * p.ld_zeros + v0, stage_rows(p.V - v0, 1), bar);
    }
}
__device__ __forceinline__ void copy_sums(const LogitsParams& p, const StageLayout& lay, int st, int n, int tb, uint32_t to, uint32_t bar)
{
    // the groups of a stage lie side by side
    bulk_load(to + lay.sums, p.sums + (static_cast<int64_t>(tb) * p.groups + st * (kStageCols >> p.shift)) * p.N, n * p.N * 4, bar);
}

lmloss_status launch_few_rows(LogitsParams& p, const CUtensorMap& map, lmloss_vocab_ctx* h, cudaStream_t stream);

}  // namespace lmloss
