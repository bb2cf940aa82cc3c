// Logits of few hidden rows from a 4-bit table: a decoding step's.
//
// Bound by memory, as long as the instructions that widen 4 bits stay beside it: an SM gets about 46 numbers a
// clock.  So each warp goes on its own, from one barrier a stage to the next: ldmatrix brings a warp's words in
// the order in which mma.sync takes its A operand (a thread's word is eight columns of one row), five
// operations widen a word, and a thread's group sums are scaled where they are.  For so few rows that is less
// than tensor memory costs: there, what widens, multiplies and adds are different warps, and the barriers and
// copies between them took more instructions than the numbers (128256 x 4096, one row: 90 us).
#include <algorithm>

#include "table4_logits.cuh"

namespace lmloss {
namespace {

constexpr int kSumWarps = 16;                // 32 rows of the tile each, and every second run of 128 columns
constexpr int kRowsThreads = (kSumWarps + 1) * 32;
constexpr uint32_t kHead = 1024;             // barriers, before the stages

struct __align__(16) RowsBarriers {
    uint64_t full[kMaxStages], empty[kMaxStages];
    int failed;
};

// Four 8 x 16-byte matrices: lane l's address is row l % 8 of matrix l / 8; of each it gets word l % 4 of row l / 4.
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int NT, class S>
__global__ void __launch_bounds__(kRowsThreads, 1) rows_kernel(const __grid_constant__ LogitsParams p, const __grid_constant__ CUtensorMap map)
{
    constexpr int N = 8 * NT;
    extern __shared__ __align__(1024) unsigned char smem[];
    RowsBarriers& b = *reinterpret_cast<RowsBarriers*>(smem);
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const StageLayout lay(p.shift, S::kBytes, p.zeros != nullptr, N, 2 * N * 256);
    float* const pads = reinterpret_cast<float*>(smem + kHead + p.qstages * p.stage_bytes);   // [8 warps][N][33]
    const int per_stage = kStageCols >> p.shift, stages = (p.kblocks + 1) / 2;
    const int tiles = p.vtiles * p.tblocks;

    if (tid == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(smem_addr(&b.full[i]), 1);
            mbar_init(smem_addr(&b.empty[i]), kSumWarps);
        }
        b.failed = 0;
        fence_mbar_init();
    }
    __syncthreads();
    auto wait = [&](uint64_t& bar, uint32_t parity) {
        if (!mbar_sleep_bounded(smem_addr(&bar), parity, kWaitLimitCycles, &b.failed)) set_error(p.err, kErrTimeout);
        __syncwarp();
    };

    if (warp == kSumWarps) {
        // ---- copies.  The table's first stages go out before the hidden rows are waited for.
        Ring q;
        const int64_t mine = static_cast<int64_t>((tiles - 1 - static_cast<int>(blockIdx.x)) / static_cast<int>(gridDim.x) + 1) * stages;
        const int64_t early = min(mine, static_cast<int64_t>(p.qstages));
        auto copy = [&](int64_t i, int slot, bool table, bool rows) {
            const int tile = static_cast<int>(blockIdx.x + i / stages * gridDim.x), st = static_cast<int>(i % stages);
            const int vt = tile / p.tblocks, tb = tile - vt * p.tblocks;
            const int n = min(per_stage, p.groups - st * per_stage), blocks = min(2, p.kblocks - 2 * st);
            const uint32_t to = base + kHead + slot * p.stage_bytes, bar = smem_addr(&b.full[slot]);
            if (table) {
                if (lane == 0) mbar_arrive_expect_tx(bar, stage_tx(p, n, vt * kTile) + blocks * N * 256);
                __syncwarp();
                copy_table(p, lay, map, st, n, vt * kTile, to, bar);
            }
            if (rows && lane == 0) {
                copy_sums(p, lay, st, n, tb, to, bar);
                bulk_load(to + lay.x, p.x + (static_cast<int64_t>(tb) * p.kblocks + 2 * st) * (N * 256), blocks * N * 256, bar);
            }
        };
        for (int64_t i = 0; i < early; ++i) copy(i, static_cast<int>(i), true, false);
        grid_dep_wait();
        for (int64_t i = 0; i < early; ++i) copy(i, static_cast<int>(i), false, true);
        for (int64_t i = 0; i < mine; ++i, q.next(p.qstages)) {
            if (i < early) continue;
            wait(b.empty[q.slot], q.parity ^ 1u);
            copy(i, q.slot, true, true);
        }
    } else {
        const int half = warp >> 3, pair = warp & 7, g8 = lane >> 2, i4 = lane & 3;
        const int r0 = pair * 32;
        float* const pad = pads + pair * (N * 33);
        // of the matrices that ldmatrix takes: rows 0-7 and 8-15 of one part, then of the next
        const int row_in = r0 + ((lane >> 3) & 1) * 8 + (lane & 7), part_in = lane >> 4;
        Ring q;
        bool waited = false;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const int vt = tile / p.tblocks, tb = tile - vt * p.tblocks;
            float acc[2][NT][4] = {};
            for (int st = 0; st < stages; ++st) {
                wait(b.full[q.slot], q.parity);
                if (2 * st + half < p.kblocks) {
                    const unsigned char* const stage = smem + kHead + q.slot * p.stage_bytes;
                    const uint32_t values = base + kHead + q.slot * p.stage_bytes;
                    float d[2][NT][4] = {};
#pragma unroll
                    for (int u2 = 0; u2 < 2; ++u2) {
                        uint32_t w[2][4];
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
                            ldmatrix4(w[mt], values + (row_in + mt * 16) * 128 + (((half * 4 + u2 * 2 + part_in) ^ (lane & 7)) << 4));
#pragma unroll
                        for (int u1 = 0; u1 < 2; ++u1) {
                            const int unit = u2 * 2 + u1;   // 32 columns
                            uint32_t a[2][2][4];
#pragma unroll
                            for (int mt = 0; mt < 2; ++mt) {
                                widen_word(w[mt][2 * u1], a[mt][0]);
                                widen_word(w[mt][2 * u1 + 1], a[mt][1]);
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint4 x = *reinterpret_cast<const uint4*>(stage + lay.x + (half * N + nt * 8 + g8) * 256 +
                                                                                (((unit * 4 + i4) ^ ((g8 & 1) << 2)) << 4));
#pragma unroll
                                for (int mt = 0; mt < 2; ++mt) {
                                    mma_m16n8k16(d[mt][nt], a[mt][0][0], a[mt][1][0], a[mt][0][1], a[mt][1][1], x.x, x.y);
                                    mma_m16n8k16(d[mt][nt], a[mt][0][2], a[mt][1][2], a[mt][0][3], a[mt][1][3], x.z, x.w);
                                }
                            }
                            // ---- a group's end: its sums, less the zero points', scaled
                            const int columns = (half * 4 + unit + 1) * 32, gl = (columns - 1) >> p.shift;
                            if ((columns & ((1 << p.shift) - 1)) == 0 && st * per_stage + gl < p.groups) {
                                const float* const sums = reinterpret_cast<const float*>(stage + lay.sums) + gl * N;
                                const typename S::raw* const scales = reinterpret_cast<const typename S::raw*>(stage + lay.scales) + gl * kTile + r0 + g8;
                                const unsigned char* const zeros = stage + lay.zeros + gl * kTile + r0 + g8;
                                float s[4], sz[4];   // rows g8, + 8, + 16, + 24
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    s[k] = S::widen(scales[8 * k]);
                                    sz[k] = p.zeros ? -static_cast<float>(zeros[8 * k]) : -8.f;
                                }
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    const float2 x = *reinterpret_cast<const float2*>(sums + nt * 8 + 2 * i4);
#pragma unroll
                                    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
                                        for (int k = 0; k < 4; ++k) {
                                            const int r = 2 * mt + (k >> 1);
                                            acc[mt][nt][k] = fmaf(s[r], fmaf(sz[r], k & 1 ? x.y : x.x, d[mt][nt][k]), acc[mt][nt][k]);
                                            d[mt][nt][k] = 0.f;
                                        }
                                    }
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&b.empty[q.slot]));
                q.next(p.qstages);
            }
            // ---- the two halves of the columns together, and out along the table's rows
            auto at = [&](int mt, int nt, int k) -> float& { return pad[(nt * 8 + 2 * i4 + (k & 1)) * 33 + mt * 16 + (k >> 1) * 8 + g8]; };
            if (half == 1) {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k) at(mt, nt, k) = acc[mt][nt][k];
            }
            asm volatile("bar.sync %0, 64;" ::"r"(pair + 1) : "memory");
            if (half == 0) {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k) at(mt, nt, k) += acc[mt][nt][k];
            }
            asm volatile("bar.sync %0, 64;" ::"r"(pair + 1) : "memory");
            if (!waited) {
                grid_dep_wait();
                waited = true;
            }
            const int64_t v = static_cast<int64_t>(vt) * kTile + r0 + lane;
            if (v < p.V) {
                const int t0 = tb * p.per, rows = min(p.per, p.T - t0);
                for (int n = half; n < rows; n += 2) {
                    const float inverse = p.inverse[t0 + n];
                    float x = pad[n * 33 + lane];
                    if (p.pairs) x = fmaf(pad[(n + N / 2) * 33 + lane], 1.f / 2048.f, x);
                    if (inverse == inverse) store_logit(p, t0 + n, v, x * 0x1p24f * inverse * p.scale);
                    else store_plain(p, t0 + n, v);
                }
            }
            asm volatile("bar.sync %0, 64;" ::"r"(pair + 1) : "memory");   // before the next tile's
        }
    }
    __syncthreads();
    if (b.failed && tid == 0) {
        // copies may be in flight: give them their time
        const long long start = clock64();
        while (clock64() - start < 20000000) {
        }
    }
    __syncthreads();
}

template <int NT, class S>
lmloss_status launch(LogitsParams& p, const CUtensorMap& map, lmloss_vocab_ctx* h, cudaStream_t stream)
{
    constexpr int N = 8 * NT;
    const StageLayout lay(p.shift, p.scale_bytes, p.zeros != nullptr, N, 2 * N * 256);
    const uint32_t pads = 8 * N * 33 * 4;
    p.stage_bytes = lay.bytes;
    p.qstages = std::min<int>(kMaxStages, (kMaxShared - kHead - pads) / lay.bytes);
    auto* fn = rows_kernel<NT, S>;
    const uint32_t bit = 1u << (8 + 3 * (NT == 1 ? 0 : (NT == 2 ? 1 : 2)) + S::kIndex);
    if (!(h->limits_raised & bit)) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared) != cudaSuccess) {
            cudaGetLastError();
            return LMLOSS_ERR_CUDA;
        }
        h->limits_raised |= bit;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(static_cast<int64_t>(p.vtiles) * p.tblocks, h->num_sms)));
    cfg.blockDim = dim3(kRowsThreads);
    cfg.dynamicSmemBytes = kHead + p.qstages * lay.bytes + pads;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fn, p, map) != cudaSuccess) {
        cudaGetLastError();
        return LMLOSS_ERR_CUDA;
    }
    return LMLOSS_OK;
}

template <int NT>
lmloss_status launch(LogitsParams& p, const CUtensorMap& map, lmloss_vocab_ctx* h, cudaStream_t stream)
{
    if (p.scale_dtype == LMLOSS_BF16) return launch<NT, Bf16>(p, map, h, stream);
    if (p.scale_dtype == LMLOSS_FP16) return launch<NT, Fp16>(p, map, h, stream);
    return launch<NT, Fp32>(p, map, h, stream);
}

}  // namespace

lmloss_status launch_few_rows(LogitsParams& p, const CUtensorMap& map, lmloss_vocab_ctx* h, cudaStream_t stream)
{
    if (p.N == 8) return launch<1>(p, map, h, stream);
    if (p.N == 16) return launch<2>(p, map, h, stream);
    return launch<4>(p, map, h, stream);
}

}  // namespace lmloss
