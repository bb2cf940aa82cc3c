// Logits from hidden rows and a vocabulary table in 4 bits.
//
//   logits[t][v] = scale sum_g s[g][v] sum_{c in g} x[t][c] (q[v][c] - z[g][v])
//
// The whole numbers q - z are exact in fp16, and so is a hidden row in fp16 once a power of two
// brings its largest value to 2^13 (bf16: what underflows is below 2^-38 of that; fp32 as a pair of fp16,
// within 2^-24).  So the tensor cores sum exact products within a group, in fp32, and the group's sum is
// scaled by s in fp32: no weight is rounded.
//
// A block takes 256 rows of the table at a time and up to N hidden rows.  Its parts, each a step of a ring
// ahead of the next:
//   one warp    copies 256 rows x 128 bytes of the table, their scales and zeros    (TMA, HBM)
//   one warp    copies the hidden rows' 128 columns, fp16, laid out for the product  (bulk copies, L2)
//   8 warps     widen 4 bits to fp16, a thread a row, into tensor memory             (operand A)
//   one thread  multiplies: [128 x 128] by [128 x N] for each half, a sum for each group
//   8 warps     read a group's sums from tensor memory, a thread a row, and add them scaled
// A first kernel lays the hidden rows out; the main one begins under its way.
#include <algorithm>
#include <cmath>

#include <cuda.h>

#include "table4.cuh"
#include "tcgen05.cuh"

namespace lmloss {
namespace {

constexpr int kTile = 256;                   // rows of the table a block takes at once
constexpr int kStageCols = 256;              // columns of the table a stage holds
constexpr int kBlockCols = 128;              // columns a product takes
constexpr int kMaxRows = 1024;               // hidden rows a launch
constexpr int kMaxStages = 8;
constexpr int kLoThreads = 19 * 32;          // 8 warps widen, 8 add, then: table, hidden rows, product
constexpr uint32_t kHeader = 1024;           // barriers, before the stages

struct LogitsParams {
    Table4 t;
    int scale_dtype, scale_bytes;
    int groups;                  // of a row
    int kblocks;                 // runs of kBlockCols columns of a row
    int T;                       // hidden rows
    int per;                     // hidden rows a block takes: N, or N / 2 as pairs
    int tblocks;                 // runs of `per` hidden rows
    int vtiles;
    int pairs;                   // fp32: the first N / 2 rows the upper parts, the others the lower ones times 2^11
    const unsigned char* x;      // [tblocks][2 kblocks][N][128 bytes], as mma_desc_128b wants them
    const float* inverse;        // [T] by which a row's sums are multiplied
    void* out;
    int64_t ld_out;
    int out_dtype;
    float scale;
    int qstages, xstages;
    uint32_t stage_bytes;        // of a stage of the table: values, scales, zeros
    int* err;
};

// ------------------------------------------------------------- hidden rows
struct HiddenParams {
    const void* x;
    int64_t ld;
    int D, kblocks;
    int N, per;
    unsigned char* out;
    float* inverse;
};

// A block a row.  Eight columns go to a 16-byte part in the order 0 4 1 5 2 6 3 7, as the table's words widen.
template <class X>
__global__ void __launch_bounds__(256) hidden_kernel(const __grid_constant__ HiddenParams p)
{
    grid_dep_launch();
    __shared__ float red[8];
    const int tid = threadIdx.x, row = blockIdx.x;
    const typename X::raw* x = static_cast<const typename X::raw*>(p.x) + row * p.ld;
    constexpr bool kPair = X::kBytes == 4;
    float scale = 1.f;
    if (!std::is_same<X, Fp16>::value) {
        float top = 0.f;   // of what is finite
        for (int c = tid; c < p.D; c += 256) {
            const float a = fabsf(X::widen(x[c]));
            if (a < INFINITY) top = fmaxf(top, a);
        }
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if ((tid & 31) == 0) red[tid >> 5] = top;
        __syncthreads();
        for (int w = 0; w < 8; ++w) top = fmaxf(top, red[w]);
        // 2^(13 - exponent), at most 2^126; (a subnormal's exponent counts as -127)
        const int e = static_cast<int>(__float_as_uint(top) >> 23);
        scale = top > 0.f ? __uint_as_float(static_cast<uint32_t>(min(13 + 254 - e, 253)) << 23) : 1.f;
    }
    if (tid == 0) p.inverse[row] = 1.f / scale;
    const int block = row / p.per, n = row - block * p.per;
    unsigned char* out = p.out + static_cast<int64_t>(block) * (2 * p.kblocks) * p.N * 128;
    for (int u = tid; u < p.kblocks * 16; u += 256) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[2];
            __half h[2], l[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int c = 8 * u + i + 4 * k;
                v[k] = c < p.D ? X::widen(x[c]) * scale : 0.f;
                h[k] = __float2half_rn(v[k]);
                const float rest = (v[k] - __half2float(h[k])) * 2048.f;
                l[k] = __float2half_rn(fabsf(v[k]) < INFINITY ? rest : 0.f);
            }
            hi[i] = static_cast<uint32_t>(__half_as_ushort(h[0])) | static_cast<uint32_t>(__half_as_ushort(h[1])) << 16;
            lo[i] = static_cast<uint32_t>(__half_as_ushort(l[0])) | static_cast<uint32_t>(__half_as_ushort(l[1])) << 16;
        }
        const int half = u >> 3, part = u & 7;
        auto place = [&](int r) { return out + (static_cast<int64_t>(half) * p.N + r) * 128 + ((part ^ (r & 7)) << 4); };
        *reinterpret_cast<uint4*>(place(n)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (kPair) *reinterpret_cast<uint4*>(place(n + p.N / 2)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

// ------------------------------------------------------------------- main
struct __align__(16) LogitsBarriers {
    uint64_t q_full[kMaxStages], q_empty[kMaxStages], x_full[kMaxStages], x_empty[kMaxStages];
    uint64_t a_full[2][2], a_empty[2][2], d_full[2][4], d_empty[2][4];
    uint32_t tmem;
    int failed;
};

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

// q - z of a word's eight numbers as fp16, in the order 0 4 1 5 2 6 3 7: 0x6400 | q is 1024 + q, and with q four
// bits further up 1024 + 16 q.  low: 1024 + z twice; high: -(64 + z) twice.
__device__ __forceinline__ void widen_word(uint32_t w, __half2 low, __half2 high, uint32_t* out)
{
    const __half2 sixteenth = __floats2half2_rn(0.0625f, 0.0625f);
    const uint32_t w8 = w >> 8;
    uint32_t a[4] = {(w & 0x000f000fu) | 0x64006400u, (w & 0x00f000f0u) | 0x64006400u, (w8 & 0x000f000fu) | 0x64006400u,
                     (w8 & 0x00f000f0u) | 0x64006400u};
    __half2* h = reinterpret_cast<__half2*>(a);
    h[0] = __hsub2(h[0], low);
    h[1] = __hfma2(h[1], sixteenth, high);
    h[2] = __hsub2(h[2], low);
    h[3] = __hfma2(h[3], sixteenth, high);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = a[i];
}

__device__ __forceinline__ void store_logit(const LogitsParams& p, int64_t t, int64_t v, float x)
{
    const int64_t at = t * p.ld_out + v;
    if (p.out_dtype == LMLOSS_BF16) static_cast<uint16_t*>(p.out)[at] = Bf16::round(x);
    else if (p.out_dtype == LMLOSS_FP16) static_cast<uint16_t*>(p.out)[at] = Fp16::round(x);
    else static_cast<float*>(p.out)[at] = x;
}

template <int N>
__global__ void __launch_bounds__(kLoThreads, 1) logits_kernel(const __grid_constant__ LogitsParams p, const __grid_constant__ CUtensorMap map)
{
    // tensor memory: A two buffers of 64 columns for each half, D kSums of N columns for each half
    constexpr int kSums = N == 64 ? 2 : 4;
    constexpr uint32_t kColumns = 256 + 2 * kSums * N <= 512 ? 512 : 0;
    static_assert(kColumns == 512, "tensor memory");
    constexpr uint32_t kIdesc = mma_f16_idesc(N);
    extern __shared__ __align__(1024) unsigned char smem[];
    LogitsBarriers& b = *reinterpret_cast<LogitsBarriers*>(smem);
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned char* const stages = smem + kHeader;
    const uint32_t xbase = base + kHeader + p.qstages * p.stage_bytes;   // stage_bytes: a multiple of 1024
    constexpr uint32_t kXBytes = N * 256;
    const int gs = 1 << p.t.shift, per_block = kBlockCols >> p.t.shift, per_stage = kStageCols >> p.t.shift;
    const int stages_a_tile = (p.kblocks + 1) / 2;
    const int tiles = p.vtiles * p.tblocks;

    if (tid == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(smem_addr(&b.q_full[i]), 1);
            mbar_init(smem_addr(&b.q_empty[i]), 16);
            mbar_init(smem_addr(&b.x_full[i]), 1);
            mbar_init(smem_addr(&b.x_empty[i]), 1);
        }
        for (int h = 0; h < 2; ++h) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_addr(&b.a_full[h][i]), 4);
                mbar_init(smem_addr(&b.a_empty[h][i]), 1);
            }
            for (int i = 0; i < 4; ++i) {
                mbar_init(smem_addr(&b.d_full[h][i]), 1);
                mbar_init(smem_addr(&b.d_empty[h][i]), 4);
            }
        }
        b.failed = 0;
        fence_mbar_init();
    }
    if (warp == 18) tmem_alloc(smem_addr(&b.tmem), kColumns);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = b.tmem;

    // A wait that runs out ends the block: everyone's next wait runs out too.
    auto wait_one = [&](uint64_t& bar, uint32_t parity) {
        if (mbar_wait_bounded(smem_addr(&bar), parity, kWaitLimitCycles)) return true;
        b.failed = 1;
        set_error(p.err, kErrTimeout);
        return false;
    };
    // by a whole warp, together again after it
    auto wait = [&](uint64_t& bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_one(bar, parity)) != 0; };

    if (warp < 8) {
        // ---- widen: a thread a row of its half
        const int half = warp >> 2, quarter = warp & 3, row = tid;   // 0 .. 255
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        Ring q, a;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            for (int st = 0; st < stages_a_tile; ++st) {
                if (!wait(b.q_full[q.slot], q.parity)) goto done;
                const unsigned char* const stage = stages + q.slot * p.stage_bytes;
                const unsigned char* const zeros = stage + kTile * 128 + per_stage * kTile * p.scale_bytes;
                const int blocks = min(2, p.kblocks - 2 * st);
                for (int kb = 0; kb < blocks; ++kb) {
                    if (!wait(b.a_empty[half][a.slot], a.parity ^ 1u)) goto done;
                    tcgen05_after_sync();
                    const uint32_t to = tmem + lanes + half * 128 + a.slot * 64;
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        uint32_t r[32];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int unit = kb * 4 + part * 2 + i;   // 32 columns
                            float z = 8.f;
                            if (p.t.zeros) z = static_cast<float>(zeros[((unit * 32) >> p.t.shift) * kTile + row]);
                            const __half2 low = __float2half2_rn(1024.f + z), high = __float2half2_rn(-64.f - z);
                            const uint4 w = *reinterpret_cast<const uint4*>(stage + row * 128 + ((unit ^ (row & 7)) << 4));
                            widen_word(w.x, low, high, r + 16 * i);
                            widen_word(w.y, low, high, r + 16 * i + 4);
                            widen_word(w.z, low, high, r + 16 * i + 8);
                            widen_word(w.w, low, high, r + 16 * i + 12);
                        }
                        tmem_store32(to + part * 32, r);
                    }
                    tmem_wait_store();
                    tcgen05_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&b.a_full[half][a.slot]));
                    a.next(2);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&b.q_empty[q.slot]));
                q.next(p.qstages);
            }
        }
        for (int i = 0; i < 2; ++i, a.next(2))   // the products have read them
            if (!wait(b.a_empty[half][a.slot], a.parity ^ 1u)) goto done;
    } else if (warp < 16) {
        // ---- add the groups' sums
        const int half = (warp - 8) >> 2, quarter = warp & 3, row = tid - 256;
        const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + 256 + half * (kSums * N);
        Ring q, d;
        bool waited = false;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const int vt = tile / p.tblocks, tb = tile - vt * p.tblocks;
            float acc[N];
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = 0.f;
            for (int st = 0; st < stages_a_tile; ++st) {
                if (!wait(b.q_full[q.slot], q.parity)) goto done;
                const unsigned char* const scales = stages + q.slot * p.stage_bytes + kTile * 128;
                const int n = min(per_stage, p.groups - st * per_stage);
                for (int g = 0; g < n; ++g) {
                    const int at = g * kTile + row;
                    float s;
                    if (p.scale_dtype == LMLOSS_FP16) s = Fp16::widen(reinterpret_cast<const uint16_t*>(scales)[at]);
                    else if (p.scale_dtype == LMLOSS_BF16) s = Bf16::widen(reinterpret_cast<const uint16_t*>(scales)[at]);
                    else s = reinterpret_cast<const float*>(scales)[at];
                    if (!wait(b.d_full[half][d.slot], d.parity)) goto done;
                    tcgen05_after_sync();
#pragma unroll
                    for (int c = 0; c < N; c += 16) {
                        float f[16];
                        tmem_load16(from + d.slot * N + c, f);
                        tmem_wait_load(f);
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[c + i] = fmaf(s, f[i], acc[c + i]);
                    }
                    tcgen05_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&b.d_empty[half][d.slot]));
                    d.next(kSums);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&b.q_empty[q.slot]));
                q.next(p.qstages);
            }
            if (!waited) {
                grid_dep_wait();
                waited = true;
            }
            const int64_t v = static_cast<int64_t>(vt) * kTile + row;
            if (v < p.t.V) {
                const int t0 = tb * p.per;
                if (p.pairs) {
#pragma unroll
                    for (int i = 0; i < N / 2; ++i)
                        if (t0 + i < p.T)
                            store_logit(p, t0 + i, v, fmaf(acc[i + N / 2], 1.f / 2048.f, acc[i]) * p.inverse[t0 + i] * p.scale);
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        if (t0 + i < p.T) store_logit(p, t0 + i, v, acc[i] * p.inverse[t0 + i] * p.scale);
                }
            }
        }
    } else if (warp == 16) {
        // ---- the table
        Ring q;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const int v0 = tile / p.tblocks * kTile;
            // to the end of the 16 bytes that hold the last row's
            const int rows = min(kTile, p.t.V - v0), whole = 16 / p.scale_bytes;
            const uint32_t srows = (rows + whole - 1) / whole * whole, zrows = p.t.zeros ? (rows + 15) / 16 * 16 : 0u;
            for (int st = 0; st < stages_a_tile; ++st) {
                bool ok = true;
                const uint32_t bar = smem_addr(&b.q_full[q.slot]), to = base + kHeader + q.slot * p.stage_bytes;
                const int n = min(per_stage, p.groups - st * per_stage);
                if (lane == 0) {
                    ok = wait_one(b.q_empty[q.slot], q.parity ^ 1u);
                    if (ok) {
                        mbar_arrive_expect_tx(bar, kTile * 128 + n * (srows * p.scale_bytes + zrows));
                        tile_load_2d(to, &map, st * 128, v0, bar);
                    }
                }
                if (!__shfl_sync(0xffffffffu, ok, 0)) goto done;
                if (lane < n) {
                    const int64_t g = static_cast<int64_t>(st) * per_stage + lane;
                    bulk_load(to + kTile * 128 + lane * kTile * p.scale_bytes,
                              static_cast<const unsigned char*>(p.t.scales) + (g * p.t.ld_scales + v0) * p.scale_bytes,
                              srows * p.scale_bytes, bar);
                    if (p.t.zeros)
                        bulk_load(to + kTile * 128 + per_stage * kTile * p.scale_bytes + lane * kTile,
                                  p.t.zeros + g * p.t.ld_zeros + v0, zrows, bar);
                }
                q.next(p.qstages);
            }
        }
    } else if (warp == 17) {
        // ---- the hidden rows
        if (lane == 0) {
            grid_dep_wait();
            Ring x;
            for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
                const unsigned char* from = p.x + static_cast<int64_t>(tile % p.tblocks) * p.kblocks * kXBytes;
                for (int kb = 0; kb < p.kblocks; ++kb) {
                    if (!wait_one(b.x_empty[x.slot], x.parity ^ 1u)) goto done;
                    const uint32_t bar = smem_addr(&b.x_full[x.slot]);
                    mbar_arrive_expect_tx(bar, kXBytes);
                    bulk_load(xbase + x.slot * kXBytes, from + static_cast<int64_t>(kb) * kXBytes, kXBytes, bar);
                    x.next(p.xstages);
                }
            }
            // the products have read them all: nothing arrives at a barrier after the block's end
            for (int i = 0; i < p.xstages; ++i, x.next(p.xstages))
                if (!wait_one(b.x_empty[x.slot], x.parity ^ 1u)) goto done;
        }
    } else if (lane == 0) {
        // ---- the products
        Ring x, a, d;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            for (int kb = 0; kb < p.kblocks; ++kb) {
                if (!wait_one(b.x_full[x.slot], x.parity)) goto done;
                const uint64_t desc = mma_desc_128b(xbase + x.slot * kXBytes);
                const int n = min(per_block, p.groups - kb * per_block);
                Ring d0 = d;
                for (int half = 0; half < 2; ++half) {
                    if (!wait_one(b.a_full[half][a.slot], a.parity)) goto done;
                    tcgen05_after_sync();
                    const uint32_t from = tmem + half * 128 + a.slot * 64;
                    d = d0;
                    for (int g = 0; g < n; ++g) {
                        if (!wait_one(b.d_empty[half][d.slot], d.parity ^ 1u)) goto done;
                        tcgen05_after_sync();
                        const uint32_t to = tmem + 256 + (half * kSums + d.slot) * N;
                        for (int k = 0; k < gs / 16; ++k) {
                            const int step = g * (gs / 16) + k;   // 16 columns; 64 lie in one run of N rows
                            mma_f16_ts(to, from + step * 8, desc + (step >> 2) * (N * 128 / 16) + (step & 3) * 2, kIdesc, k > 0);
                        }
                        mma_commit(smem_addr(&b.d_full[half][d.slot]));
                        d.next(kSums);
                    }
                    mma_commit(smem_addr(&b.a_empty[half][a.slot]));
                }
                mma_commit(smem_addr(&b.x_empty[x.slot]));
                x.next(p.xstages);
                a.next(2);
            }
        }
    }
done:
    __syncwarp();
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (b.failed && tid == 0) {
        // copies may be in flight: no barrier's phase is known any more, so give them their time
        const long long start = clock64();
        while (clock64() - start < 20000000) {
        }
    }
    __syncthreads();
    if (warp == 18) tmem_free(tmem, kColumns);
}

// ------------------------------------------------------------------- host
lmloss_status check_logits(const lmloss_table4_logits_args* a, bool pointers)
{
    if (!a) return LMLOSS_ERR_INVALID_ARG;
    const lmloss_status st = table4_check(a->table, pointers);
    if (st != LMLOSS_OK) return st;
    if (a->T < 0 || !float_dtype(a->hidden_dtype)) return LMLOSS_ERR_INVALID_ARG;
    if (a->T >= (int64_t(1) << 24)) return LMLOSS_ERR_UNSUPPORTED;
    if (!pointers) return LMLOSS_OK;
    if (!float_dtype(a->logits_dtype) || !std::isfinite(a->scale)) return LMLOSS_ERR_INVALID_ARG;
    if (a->ld_hidden < a->table.D || a->ld_logits < a->table.V) return LMLOSS_ERR_INVALID_ARG;
    if (a->T > 0) {
        if (a->ld_hidden > INT64_MAX / 16 / a->T || a->ld_logits > INT64_MAX / 16 / a->T) return LMLOSS_ERR_INVALID_ARG;
        if (!a->hidden || reinterpret_cast<uintptr_t>(a->hidden) % float_bytes(a->hidden_dtype)) return LMLOSS_ERR_INVALID_ARG;
        if (!a->logits || reinterpret_cast<uintptr_t>(a->logits) % float_bytes(a->logits_dtype)) return LMLOSS_ERR_INVALID_ARG;
    }
    return LMLOSS_OK;
}

// Columns of the product for `rows` operand rows (a pair counts twice).
int columns_for(int64_t rows) { return rows <= 16 ? 16 : (rows <= 32 ? 32 : 64); }

int64_t kblocks_of(int64_t D) { return (D + kBlockCols - 1) / kBlockCols; }

// Workspace of the hidden rows of a launch: operand rows, padded to whole blocks, and their factors.
size_t hidden_bytes(int64_t T, int64_t D, bool pairs)
{
    const int64_t rows = std::min<int64_t>(T, kMaxRows) * (pairs ? 2 : 1);
    const int64_t N = columns_for(rows), padded = (rows + N - 1) / N * N;
    return vocab_align(static_cast<size_t>(padded * kblocks_of(D) * kBlockCols * 2));
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

// [V, (D + 1) / 2] bytes, copied 128 bytes by kTile rows at a time.
bool table_map(const lmloss_table4& t, CUtensorMap* map)
{
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>((t.D + 1) / 2), static_cast<cuuint64_t>(t.V)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(t.ld_values)};
    const cuuint32_t box[2] = {128, kTile}, steps[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, t.values, dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr uint32_t kMaxShared = 227 * 1024;

template <int N>
lmloss_status launch_logits(LogitsParams& p, const CUtensorMap& map, lmloss_vocab_ctx* h, cudaStream_t stream)
{
    const int per_stage = kStageCols >> p.t.shift;
    p.stage_bytes = kTile * 128 + per_stage * kTile * (p.scale_bytes + (p.t.zeros ? 1 : 0));   // multiples of 1024
    p.stage_bytes = (p.stage_bytes + 1023) / 1024 * 1024;
    p.xstages = N == 64 ? 4 : 6;
    const uint32_t left = kMaxShared - kHeader - p.xstages * N * 256;
    p.qstages = std::min<int>(kMaxStages, left / p.stage_bytes);
    const uint32_t bytes = kHeader + p.qstages * p.stage_bytes + p.xstages * N * 256;
    // per device, and cheap: the attribute is the function's, whoever set it before
    if (cudaFuncSetAttribute(logits_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared) != cudaSuccess) {
        cudaGetLastError();
        return LMLOSS_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(static_cast<int64_t>(p.vtiles) * p.tblocks, h->num_sms)));
    cfg.blockDim = dim3(kLoThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, logits_kernel<N>, p, map) != cudaSuccess) {
        cudaGetLastError();
        return LMLOSS_ERR_CUDA;
    }
    return LMLOSS_OK;
}

}  // namespace
}  // namespace lmloss

using namespace lmloss;

extern "C" {

lmloss_status lmloss_table4_check_logits_args(const lmloss_table4_logits_args* a) { return check_logits(a, true); }

lmloss_status lmloss_table4_logits_workspace(const lmloss_table4_logits_args* a, size_t* bytes)
{
    if (!bytes) return LMLOSS_ERR_INVALID_ARG;
    const lmloss_status st = check_logits(a, false);
    if (st != LMLOSS_OK) return st;
    *bytes = 0;
    if (a->T == 0) return LMLOSS_OK;
    // pairs take the most
    *bytes = hidden_bytes(a->T, a->table.D, true) + vocab_align(sizeof(float) * std::min<int64_t>(a->T, kMaxRows));
    return LMLOSS_OK;
}

lmloss_status lmloss_table4_logits(lmloss_vocab_handle h, const lmloss_table4_logits_args* a, cudaStream_t stream)
{
    if (!h) return LMLOSS_ERR_INVALID_ARG;
    lmloss_status st = check_logits(a, true);
    if (st != LMLOSS_OK) return st;
    if (a->T == 0) return LMLOSS_OK;
    const bool pairs = a->hidden_dtype == LMLOSS_FP32;
    const size_t x_bytes = hidden_bytes(a->T, a->table.D, pairs);
    if (x_bytes + vocab_align(sizeof(float) * std::min<int64_t>(a->T, kMaxRows)) > h->ws_bytes) return LMLOSS_ERR_INVALID_ARG;
    VocabDeviceGuard g(h->device);
    if (!g.ok) return LMLOSS_ERR_CUDA;
    CUtensorMap map;
    if (!table_map(a->table, &map)) return LMLOSS_ERR_CUDA;
    for (int64_t t0 = 0; t0 < a->T; t0 += kMaxRows) {
        const int T = static_cast<int>(std::min<int64_t>(a->T - t0, kMaxRows));
        const int N = columns_for(static_cast<int64_t>(T) * (pairs ? 2 : 1));
        HiddenParams x{};
        x.x = static_cast<const unsigned char*>(a->hidden) + t0 * a->ld_hidden * float_bytes(a->hidden_dtype);
        x.ld = a->ld_hidden;
        x.D = static_cast<int>(a->table.D);
        x.kblocks = static_cast<int>(kblocks_of(a->table.D));
        x.N = N;
        x.per = pairs ? N / 2 : N;
        x.out = h->ws;
        x.inverse = reinterpret_cast<float*>(h->ws + x_bytes);
        switch (a->hidden_dtype) {
        case LMLOSS_BF16: hidden_kernel<Bf16><<<T, 256, 0, stream>>>(x); break;
        case LMLOSS_FP16: hidden_kernel<Fp16><<<T, 256, 0, stream>>>(x); break;
        default: hidden_kernel<Fp32><<<T, 256, 0, stream>>>(x); break;
        }
        if ((st = vocab_launch_err()) != LMLOSS_OK) return st;
        LogitsParams p{};
        p.t = table4_params(a->table);
        p.scale_dtype = a->table.scale_dtype;
        p.scale_bytes = float_bytes(a->table.scale_dtype);
        p.groups = static_cast<int>((a->table.D + a->table.group - 1) / a->table.group);
        p.kblocks = x.kblocks;
        p.T = T;
        p.per = x.per;
        p.tblocks = (T + x.per - 1) / x.per;
        p.vtiles = static_cast<int>((a->table.V + kTile - 1) / kTile);
        p.pairs = pairs;
        p.x = x.out;
        p.inverse = x.inverse;
        p.out = static_cast<unsigned char*>(a->logits) + t0 * a->ld_logits * float_bytes(a->logits_dtype);
        p.ld_out = a->ld_logits;
        p.out_dtype = a->logits_dtype;
        p.scale = a->scale;
        p.err = h->err;
        st = N == 16 ? launch_logits<16>(p, map, h, stream) : (N == 32 ? launch_logits<32>(p, map, h, stream) : launch_logits<64>(p, map, h, stream));
        if (st != LMLOSS_OK) return st;
    }
    return LMLOSS_OK;
}

}  // extern "C"
