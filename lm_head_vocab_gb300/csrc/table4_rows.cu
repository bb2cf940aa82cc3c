// Logits of few hidden rows from a 4-bit table: a decoding step's.
//
// Bound by memory, as long as the instructions that widen 4 bits stay beside it: an SM gets about 46 numbers a
// clock.  So each warp goes on its own, from one barrier a stage to the next: ldmatrix brings a warp's words in
// the order in which mma.sync takes its A operand (a thread's word is eight columns of one row), five or nine
// operations widen a word, and a thread's group sums are scaled where they are.  For so few rows that is less than tensor memory costs: there, what widens, multiplies and adds are
// different warps, and the barriers and copies between them took more instructions than the numbers (128256 x 4096,
// one row, by the kernel for more rows: 71 us, 51 here).
// Each block lays the hidden rows out in its own shared memory, under the way of its first stages.
//
// Up to 4 rows are pairs of fp16 whatever their type, multiplied by the numbers' own bits, subnormal fp16, and the
// zero points' part z sum x is taken off a group's sums: the upper parts' are exact, and what the tensor cores cut off of the
// lower parts' (relative to what a subnormal's exponent could hold) is past fp32.  5 to 8 rows of 16 bits are
// multiplied as they are, by numbers less their zero points as normal fp16.  (Such rows by subnormal numbers took 59 and
// 66 us for 5 and 8 rows, 67 and 71 so.  But one column 3000 times the others, as models' hidden rows have them, then
// cut off the others' sums: logits that it does not even enter, as q = z there, were 2e-3 of their size off.)
//
// 128256 x 4096 in groups of 128: one row 51 us, 4 rows 56, 8 rows 71 (5.3, 4.9 and 3.9 TB/s; 41 us at the copy's rate),
// one row by 32 with zeros 79.  Half of the issue slots are used (some 240 instructions for 32 rows x 128 columns, the
// smaller the group the more), and the DRAM 68% of the time: neither alone bounds it.
#include <algorithm>
#include <type_traits>

#include "table4_logits.cuh"

namespace lmloss {
namespace {

constexpr int kSumWarps = 16;                // 32 of the tile's 64 rows each, and 128 of a stage's 1024 columns
constexpr int kSumThreads = kSumWarps * 32;
constexpr int kRowsThreads = kSumThreads + 32;
constexpr uint32_t kHead = 1024;             // barriers and what is said of hidden rows, before the stages

struct __align__(16) RowsHead {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint32_t top[kFewRows];                  // bits of a hidden row's largest finite value
    int odd[kFewRows];                       // whether it has others
    int failed;
};
static_assert(sizeof(RowsHead) <= kHead, "head");

// Hidden rows [kblocks][N][256 bytes], 16-byte part i of a row at i ^ 4 (row % 2); sums [groups][N]; what warps
// hand on, of tiles in turn [2][16][hidden rows][33].
struct RowsLayout {
    uint32_t sums, pads, bytes;
    __host__ __device__ RowsLayout(int N, int T, int kblocks, int groups)
    {
        sums = N * kblocks * 256;
        pads = sums + groups * N * 4;
        bytes = pads + 2 * kSumWarps * T * 33 * 4;
    }
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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// What widen_word takes off, twice each: 2^-4 + z 2^-14, whose mantissa z is, and of it 2^-4 + z 2^-10, exact.  (By
// conversions of z a call of 5 rows in groups of 32 took 99 us for 86.)
__device__ __forceinline__ void zero_points(uint32_t z, __half2& z1, __half2& z16)
{
    const uint32_t bits = z * 0x00010001u + 0x2c002c00u;
    z1 = *reinterpret_cast<const __half2*>(&bits);
    z16 = __hfma2(z1, __float2half2_rn(16.f), __float2half2_rn(-0.9375f));
}

// The hidden rows into shared memory, by the first kSumThreads threads: read once, as many rows at a time as their
// registers hold.
template <class X, bool PAIR>
__device__ __noinline__ void lay_out(const LogitsParams& p, RowsHead& head, unsigned char* x, float* sums, int N)
{
    constexpr int kHold = 16 / X::kBytes;
    const int tid = threadIdx.x;
    const uint32_t together = 0xffffu << (tid & 16);   // 16 threads have parts of the same row
    const typename X::raw* hidden = static_cast<const typename X::raw*>(p.hidden);
    const int parts = p.kblocks * 16, lanes = (1 << p.shift) / 8, rows = kHold * kSumThreads / parts;   // few_rows_fit: at least one
    for (int r0 = 0; r0 < p.T; r0 += rows) {
        const int n = min(rows, p.T - r0) * parts;
        Pack<X, 8> v[kHold];
        int r[kHold];
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int at = tid + i * kSumThreads;
            r[i] = at < n ? r0 + at / parts : -1;
            if (r[i] >= 0) load_part<X>(hidden + r[i] * p.ld_hidden, (at - (r[i] - r0) * parts) * 8, p.D, v[i]);
        }
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            if (r[i] < 0) continue;
            bool odd;
            const uint32_t top = __reduce_max_sync(together, __float_as_uint(part_top<X>(v[i], odd)));
            odd = __any_sync(together, odd);
            if ((tid & 15) == 0) {
                atomicMax(&head.top[r[i]], top);
                if (odd) head.odd[r[i]] = 1;
            }
        }
        asm volatile("bar.sync 9, %0;" ::"n"(kSumThreads) : "memory");
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            if (r[i] < 0) continue;
            const int u = tid + i * kSumThreads - (r[i] - r0) * parts;
            uint4 hi, lo;
            float sum, sum_lo;
            bool odd;
            const float largest = PAIR ? group_top(lanes, part_top<X>(v[i], odd)) : 0.f;
            hidden_part<X, PAIR>(v[i], head.odd[r[i]] ? 0.f : hidden_scale(__uint_as_float(head.top[r[i]])), largest, hi, lo, sum, sum_lo);
            auto place = [&](int k) { return reinterpret_cast<uint4*>(x + ((u >> 4) * N + k) * 256 + (((u & 15) ^ ((k & 1) << 2)) << 4)); };
            *place(r[i]) = hi;
            if (PAIR) *place(r[i] + N / 2) = lo;
            if (!PAIR) continue;
            group_sums(lanes, sum, sum_lo);
            const int g = (8 * u) >> p.shift;
            if ((u & (lanes - 1)) == 0 && g < p.groups) {
                sums[g * N + r[i]] = sum;
                sums[g * N + r[i] + N / 2] = sum_lo;
            }
        }
    }
    asm volatile("bar.sync 9, %0;" ::"n"(kSumThreads) : "memory");
}

template <int GROUP, bool PAIRS>
__global__ void __launch_bounds__(kRowsThreads, 1) rows_kernel(const __grid_constant__ LogitsParams p, const __grid_constant__ TableMaps maps)
{
    constexpr int N = kFewRows;
    static_assert(N == 8, "columns of one mma.sync");
    constexpr int kPerStage = kFewCols / GROUP, kUnits = GROUP / 32;   // groups of a stage; runs of 32 columns of a group
    extern __shared__ __align__(1024) unsigned char smem[];
    RowsHead& b = *reinterpret_cast<RowsHead*>(smem);
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const StageLayout lay(kFewTile, kFewCols, p.shift, p.scale_bytes, p.zeros != nullptr);
    const RowsLayout rl(N, p.T, p.kblocks, p.groups);
    unsigned char* const rows = smem + kHead + p.qstages * p.stage_bytes;
    const int stages = (p.kblocks + 7) / 8;

    if (tid == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(smem_addr(&b.full[i]), 1);
            mbar_init(smem_addr(&b.empty[i]), kSumWarps);
        }
        b.failed = 0;
        fence_mbar_init();
    }
    if (tid < kFewRows) {
        b.top[tid] = 0;
        b.odd[tid] = 0;
    }
    __syncthreads();
    auto wait_one = [&](uint64_t& bar, uint32_t parity) {
        if (!mbar_sleep_bounded(smem_addr(&bar), parity, kWaitLimitCycles, &b.failed)) set_error(p.err, kErrTimeout);
    };

    if (warp == kSumWarps) {
        // ---- copies
        if (lane == 0) {
            Ring q;
            for (int tile = blockIdx.x; tile < p.vtiles; tile += gridDim.x)
                for (int st = 0; st < stages; ++st) {
                    wait_one(b.empty[q.slot], q.parity ^ 1u);
                    const uint32_t bar = smem_addr(&b.full[q.slot]);
                    const int runs = min(4, (p.kblocks - st * 8 + 1) / 2);
                    mbar_arrive_expect_tx(bar, lay.copied - (4 - runs) * (kFewTile * 128));
                    copy_table(p, lay, maps, kFewTile, st * 4, runs, tile * kFewTile, base + kHead + q.slot * p.stage_bytes, bar);
                    q.next(p.qstages);
                }
        }
        __syncwarp();
    } else {
        float* const all_sums = reinterpret_cast<float*>(rows + rl.sums);
        if (p.hidden_dtype == LMLOSS_BF16) lay_out<Bf16, PAIRS>(p, b, rows, all_sums, N);
        else if (p.hidden_dtype == LMLOSS_FP16) lay_out<Fp16, PAIRS>(p, b, rows, all_sums, N);
        else if constexpr (PAIRS) lay_out<Fp32, true>(p, b, rows, all_sums, N);
        const int half = warp & 1, block = warp & 7, team = warp >> 3, g8 = lane >> 2, i4 = lane & 3;   // block: of 128 columns of a stage
        const int r0 = team * 32;
        float* pads = reinterpret_cast<float*>(rows + rl.pads) + team * 8 * (p.T * 33);
        const int other_pads = kSumWarps * p.T * 33;
        int turn = 0;
        // of the matrices that ldmatrix takes: rows 0-7 and 8-15 of one part, then of the next
        const uint32_t words = base + kHead + (block >> 1) * (kFewTile * 128) + (r0 + ((lane >> 3) & 1) * 8 + (lane & 7)) * 128;
        uint32_t part_at[2];
#pragma unroll
        for (int u2 = 0; u2 < 2; ++u2) part_at[u2] = ((half * 4 + u2 * 2 + (lane >> 4)) ^ (lane & 7)) << 4;
        // part 4 unit + i4 of a hidden row lies at 4 (unit ^ row % 2) + i4
        const int odd = (g8 & 1) * 64;
        const unsigned char* const x_even = rows + g8 * 256 + i4 * 16 + odd;
        const unsigned char* const x_odd = x_even - 2 * odd;
        Ring q;
        for (int tile = blockIdx.x; tile < p.vtiles; tile += gridDim.x) {
            float acc[2][4] = {};
            for (int st = 0; st < stages; ++st) {
                wait_one(b.full[q.slot], q.parity);
                __syncwarp();
                const int kb = 8 * st + block;
                if (kb < p.kblocks) {
                    const uint32_t offset = q.slot * p.stage_bytes;
                    const unsigned char* const stage = smem + kHead + offset;
                    uint32_t w[2][2][4];
#pragma unroll
                    for (int u2 = 0; u2 < 2; ++u2)
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt) ldmatrix4(w[u2][mt], words + offset + mt * 16 * 128 + part_at[u2]);
                    const int x_at = kb * (N * 256);
                    const int g0 = block * (kBlockCols / GROUP);   // the block's first group in the stage
                    float d[2][4];
                    uint32_t z[4];   // rows g8, + 8, + 16, + 24
                    __half2 z1[4], z16[4];
#pragma unroll
                    for (int unit = 0; unit < 4; ++unit) {   // 32 columns
                        if (unit % kUnits == 0) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) d[i / 4][i % 4] = 0.f;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                z[k] = p.zeros ? (stage + lay.zeros)[(g0 + unit / kUnits) * kFewTile + r0 + g8 + 8 * k] : 8u;
                                if (!PAIRS) zero_points(z[k], z1[k], z16[k]);
                            }
                        }
                        uint32_t a[2][2][4];
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                            for (int down = 0; down < 2; ++down) {
                                const uint32_t word = w[unit >> 1][mt][2 * (unit & 1) + down];
                                if (PAIRS) widen_word(word, a[mt][down]);
                                else widen_word(word, z1[2 * mt + down], z16[2 * mt + down], a[mt][down]);
                            }
                        const uint4 x = *reinterpret_cast<const uint4*>((unit & 1 ? x_odd : x_even) + x_at + unit * 64);
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt) {
                            mma_m16n8k16(d[mt], a[mt][0][0], a[mt][1][0], a[mt][0][1], a[mt][1][1], x.x, x.y);
                            mma_m16n8k16(d[mt], a[mt][0][2], a[mt][1][2], a[mt][0][3], a[mt][1][3], x.z, x.w);
                        }
                        // ---- a group's end: its sums, less the zero points', scaled
                        const int gl = g0 + unit / kUnits;
                        if ((unit + 1) % kUnits == 0 && st * kPerStage + gl < p.groups) {
                            const int at = gl * kFewTile + r0 + g8;
                            float s[4];
                            if (p.scale_dtype == LMLOSS_FP16) {
#pragma unroll
                                for (int k = 0; k < 4; ++k) s[k] = Fp16::widen(reinterpret_cast<const uint16_t*>(stage + lay.scales)[at + 8 * k]);
                            } else if (p.scale_dtype == LMLOSS_BF16) {
#pragma unroll
                                for (int k = 0; k < 4; ++k) s[k] = Bf16::widen(reinterpret_cast<const uint16_t*>(stage + lay.scales)[at + 8 * k]);
                            } else {
#pragma unroll
                                for (int k = 0; k < 4; ++k) s[k] = reinterpret_cast<const float*>(stage + lay.scales)[at + 8 * k];
                            }
                            float2 sums{};
                            if (PAIRS) sums = *reinterpret_cast<const float2*>(all_sums + (st * kPerStage + gl) * N + 2 * i4);
#pragma unroll
                            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const int r = 2 * mt + (k >> 1);
                                    acc[mt][k] = fmaf(s[r], PAIRS ? fmaf(-static_cast<float>(z[r]), k & 1 ? sums.y : sums.x, d[mt][k]) : d[mt][k], acc[mt][k]);
                                }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&b.empty[q.slot]));
                q.next(p.qstages);
            }
            // ---- a team's eight warps together, and out along the table's rows, a warp a hidden row; the other warps
            // go on to the next tile, whose sums go elsewhere
            float* const here = pads + turn * other_pads;
            turn ^= 1;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int mt = i / 4, k = i % 4, n = 2 * i4 + (k & 1);
                float x = acc[mt][k];
                // (a pair's lower part is operand row n + 4, of the thread two on)
                if (PAIRS) x = fmaf(__shfl_down_sync(0xffffffffu, x, 2), 1.f / 2048.f, x);
                if (n < p.T) here[(block * p.T + n) * 33 + mt * 16 + (k >> 1) * 8 + g8] = x;
            }
            asm volatile("bar.sync %0, 256;" ::"r"(team + 1) : "memory");
            const int64_t v = static_cast<int64_t>(tile) * kFewTile + r0 + lane;
            for (int n = block; n < p.T; n += 8) {
                float x = 0.f;
#pragma unroll
                for (int w = 0; w < 8; ++w) x += here[(w * p.T + n) * 33 + lane];
                if (v < p.V) {
                    if (b.odd[n]) store_plain(p, n, v);
                    else store_logit(p, n, v, x * (PAIRS ? 0x1p24f : 0x1p14f) / hidden_scale(__uint_as_float(b.top[n])) * p.scale);
                }
            }
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

template <int GROUP, bool PAIRS>
lmloss_status launch(LogitsParams& p, const TableMaps& maps, lmloss_vocab_ctx* h, cudaStream_t stream)
{
    const StageLayout lay(kFewTile, kFewCols, p.shift, p.scale_bytes, p.zeros != nullptr);
    const RowsLayout rl(kFewRows, p.T, p.kblocks, p.groups);
    p.stage_bytes = lay.bytes;
    p.qstages = std::min<int>(kMaxStages, (kMaxShared - kHead - rl.bytes) / lay.bytes);
    auto* fn = rows_kernel<GROUP, PAIRS>;
    constexpr uint32_t bit = 1u << (8 + (GROUP == 32 ? 0 : (GROUP == 64 ? 1 : 2)) + (PAIRS ? 3 : 0));
    if (!(h->limits_raised & bit)) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared) != cudaSuccess) {
            cudaGetLastError();
            return LMLOSS_ERR_CUDA;
        }
        h->limits_raised |= bit;
    }
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(p.vtiles, h->num_sms));
    fn<<<grid, kRowsThreads, kHead + p.qstages * lay.bytes + rl.bytes, stream>>>(p, maps);
    return vocab_launch_err();
}

}  // namespace

bool few_rows_fit(const LogitsParams& p)
{
    const int64_t rows = static_cast<int64_t>(p.T) * (p.pairs ? 2 : 1), N = kFewRows;
    if (rows > kFewRows || N * p.kblocks * 256 > kMaxShared) return false;   // (which leaves 1800 parts of a row)
    return kHead + RowsLayout(static_cast<int>(N), p.T, p.kblocks, p.groups).bytes +
               2 * StageLayout(kFewTile, kFewCols, p.shift, p.scale_bytes, p.zeros != nullptr).bytes <= kMaxShared;
}

lmloss_status launch_few_rows(LogitsParams& p, const TableMaps& maps, lmloss_vocab_ctx* h, cudaStream_t stream)
{
    p.N = kFewRows;
    auto by_group = [&](auto pairs) {
        constexpr bool kPairs = decltype(pairs)::value;
        if (p.shift == 5) return launch<32, kPairs>(p, maps, h, stream);
        if (p.shift == 6) return launch<64, kPairs>(p, maps, h, stream);
        return launch<128, kPairs>(p, maps, h, stream);
    };
    return p.pairs ? by_group(std::true_type{}) : by_group(std::false_type{});
}

}  // namespace lmloss
