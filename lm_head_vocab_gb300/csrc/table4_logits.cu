// Logits from hidden rows and a vocabulary table in 4 bits.
//
//   logits[t][v] = scale sum_g s[g][v] sum_{c in g} x[t][c] (q[v][c] - z[g][v])
//
// The whole numbers q - z are exact in fp16, and so is a hidden row in fp16 once a power of two brings its
// largest value to 2^14 (bf16 and fp16: what underflows is below 2^-35 of that; fp32 as a pair of fp16,
// within 2^-23 of the largest of a group of columns and 2^-46 of the row's).  So the tensor cores sum exact products within a group, in fp32, and a group's sum is scaled
// by s and added to the others in fp32 registers: no weight is rounded.
//
// Up to 8 operand rows go to a kernel of independent warps (table4_rows.cu); a pair counts as two.  For more a first
// kernel lays the hidden rows out, and in the one here a block takes 128 rows of the table and 16, 32, 64 or 128
// operand rows at a time.  Its parts, each a step of a ring ahead of the next:
//   one warp        copies 128 rows x 256 columns of the table, their scales and zeros  (TMA, HBM)
//   one warp        copies the hidden rows' 128 columns, laid out for the product       (bulk copies, L2)
//   8 warps         widen 4 bits to fp16, a thread a row, into tensor memory            (operand A)
//   2 warps         multiply, [128 x 128] by [128 x N] in turn, a sum for each group
//   4 or 8 warps    read a group's sums from tensor memory, a thread a row, and add them scaled
//
// 128256 x 4096 in groups of 128: 16 rows 74 us, 64 rows 117, 512 rows 454 (1180 TFLOP/s, 0.60 of what a bf16 product
// reaches), 1024 rows 892.  Bound by the instructions of the parts together, 60% of the issue slots, and by the
// handing on between them: without the products, the reading of sums or the writing of operands it takes 2 to 5%
// less.  So, too, smaller groups cost (512 rows by 64: 785 us, by 32: 1245): a sum's barriers take as long as its
// products, some 500 clocks a block.  With 8 groups' columns added before they are scaled that would be gone, and
// so would the exactness.
#include <algorithm>
#include <cmath>

#include "table4_logits.cuh"

namespace lmloss {
namespace {

constexpr int kMaxRows = 1024;               // hidden rows a launch
constexpr int kMany = 128;                   // operand rows of a block's product at most
constexpr uint32_t kHeader = 5120;           // barriers and factors, before the stages

constexpr int kRows = 128;                   // rows of the table a block takes at once
constexpr int kStageCols = 256;              // columns of it that a stage holds

// The kernel's shapes, by N operand rows.  Up to 32 two blocks share an SM.
template <int N>
struct Shape {
    static constexpr int kBlocks = N > 32 ? 1 : 2;           // of an SM
    static constexpr int kWidenWarps = 8;                    // two groups, which take blocks of columns in turn
    static constexpr int kSplit = N > 32 ? 2 : 1;            // parts of the operand rows
    static constexpr int kOwn = N / kSplit;                  // operand rows that a thread adds up
    static constexpr int kAddWarps = 4 * kSplit;
    static constexpr int kFirstFew = kWidenWarps + kAddWarps;   // then: table, hidden rows, products of either turn
    static constexpr int kThreads = (kFirstFew + 4) * 32;
    // tensor memory: A kAhead of either turn, then D kSums of either turn.  (With one A of a turn what widens waited
    // for its products: 1100 clocks a block of columns, for 64 operand rows as for 128.)
    static constexpr int kSums = N > 64 ? 1 : (N > 16 ? 2 : 4), kAhead = N > 32 ? 2 : 1;
    // whether sums of small groups go by lots, with one barrier a lot: where there is room for more than one, and
    // registers for the loop
    static constexpr bool kLots = N == 16 || N == 64;
    static constexpr uint32_t kD = 128 * kAhead, kColumns = N > 32 ? 512 : 256;
    static_assert(kD + 2 * kSums * N <= kColumns, "tensor memory");
    // registers a thread of each part where 64 sums do not fit an even share: in all what the block was launched with
    static constexpr bool kUneven = kOwn == 64;
    static constexpr int kWidenRegs = 72, kAddRegs = 136, kFewRegs = 40;
    static_assert(!kUneven || kWidenWarps * kWidenRegs + kAddWarps * kAddRegs + 4 * kFewRegs <= kThreads / 32 * (65536 / kThreads / 8 * 8), "registers");
};

struct HiddenParams {
    const void* x;
    int64_t ld;
    int D, kblocks;
    int N, per;
    int lanes;                   // 8 columns each, of a table's group
    int own;                     // operand rows of a thread's sums: pairs lie within them
    unsigned char* out;
    float* inverse;
};

// A block a row.  Eight columns go to a 16-byte part in the order 0 4 1 5 2 6 3 7, as the table's words widen, the
// places 1 5 and 3 7 divided by 16.
template <class X>
__global__ void __launch_bounds__(256) hidden_kernel(const __grid_constant__ HiddenParams p)
{
    grid_dep_launch();
    __shared__ float red[8];
    __shared__ int odd[8];
    const int tid = threadIdx.x, row = blockIdx.x;
    const typename X::raw* x = static_cast<const typename X::raw*>(p.x) + row * p.ld;
    constexpr bool kPair = X::kBytes == 4;
    float top = 0.f;   // of what is finite
    bool finite = true;
    for (int c = tid * 8; c < p.D; c += 256 * 8) {
        Pack<X, 8> v;
        bool others;
        load_part<X>(x, c, p.D, v);
        top = fmaxf(top, part_top<X>(v, others));
        finite = finite && !others;
    }
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    finite = __all_sync(0xffffffffu, finite);
    if ((tid & 31) == 0) {
        red[tid >> 5] = top;
        odd[tid >> 5] = finite ? 0 : 1;
    }
    __syncthreads();
    for (int w = 0; w < 8; ++w) {
        top = fmaxf(top, red[w]);
        finite &= odd[w] == 0;
    }
    const float scale = hidden_scale(top);
    if (tid == 0) p.inverse[row] = finite ? 1.f / scale : NAN;
    const int block = row / p.per;
    int n = row - block * p.per;
    if (kPair) n += n / (p.own / 2) * (p.own / 2);
    unsigned char* out = p.out + static_cast<int64_t>(block) * p.kblocks * (p.N * 256);
    for (int u = tid; u < p.kblocks * 16; u += 256) {
        uint4 hi, lo;
        float sum, sum_lo;
        Pack<X, 8> v;
        load_part<X>(x, 8 * u, p.D, v);
        bool others;
        const float largest = kPair ? group_top(p.lanes, part_top<X>(v, others)) : 0.f;
        hidden_part<X, kPair>(v, finite ? scale : 0.f, largest, hi, lo, sum, sum_lo);
        // [2][N][128 bytes] for each block of columns, swizzled as mma_desc_128b wants it
        const int part = u & 7;
        auto place = [&](int r) { return reinterpret_cast<uint4*>(out + (static_cast<int64_t>(u >> 3) * p.N + r) * 128 + ((part ^ (r & 7)) << 4)); };
        *place(n) = hi;
        if (kPair) *place(n + p.own / 2) = lo;
    }
}

// ------------------------------------------------------------------- main
// A block's head: barriers, and the factors of all hidden rows.
struct __align__(16) LogitsBarriers {
    uint64_t q_full[kMaxStages], q_empty[kMaxStages], x_full[kMaxStages], x_empty[kMaxStages];
    uint64_t a_full[2][2], a_empty[2][2], d_full[2][4], d_empty[2][4];   // of either turn
    uint32_t tmem;
    int failed;
    int odd;                     // whether any row is not finite
    float factor[kMaxRows];      // NaN: the row is not finite
};
static_assert(sizeof(LogitsBarriers) <= kHeader, "head");

template <int N>
__global__ void __launch_bounds__(Shape<N>::kThreads, Shape<N>::kBlocks)
    logits_kernel(const __grid_constant__ LogitsParams p, const __grid_constant__ TableMaps maps)
{
    using Sh = Shape<N>;
    constexpr int kSums = Sh::kSums, kOwn = Sh::kOwn;
    constexpr uint32_t kIdesc = mma_f16_idesc(N);
    constexpr uint32_t kXBytes = N * 256;
    extern __shared__ __align__(1024) unsigned char smem[];
    LogitsBarriers& b = *reinterpret_cast<LogitsBarriers*>(smem);
    const uint32_t base = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const StageLayout lay(kRows, kStageCols, p.shift, p.scale_bytes, p.zeros != nullptr);
    const uint32_t xbase = base + kHeader + p.qstages * p.stage_bytes;
    const int gs = 1 << p.shift, per_stage = kStageCols >> p.shift;
    const int stages = (p.kblocks + 1) / 2;
    const int tiles = p.vtiles * p.tblocks;

    if (tid == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(smem_addr(&b.q_full[i]), 1);
            mbar_init(smem_addr(&b.q_empty[i]), Sh::kFirstFew);
            mbar_init(smem_addr(&b.x_full[i]), 1);
            mbar_init(smem_addr(&b.x_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            for (int d = 0; d < 2; ++d) {
                mbar_init(smem_addr(&b.a_full[i][d]), 4);
                mbar_init(smem_addr(&b.a_empty[i][d]), 1);
            }
            for (int d = 0; d < 4; ++d) {
                mbar_init(smem_addr(&b.d_full[i][d]), 1);
                mbar_init(smem_addr(&b.d_empty[i][d]), Sh::kAddWarps);
            }
        }
        b.failed = 0;
        b.odd = 0;
        fence_mbar_init();
    }
    if (warp == Sh::kFirstFew + 2) tmem_alloc(smem_addr(&b.tmem), Sh::kColumns);
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = b.tmem;

    auto wait_one = [&](uint64_t& bar, uint32_t parity) {
        if (!mbar_sleep_bounded(smem_addr(&bar), parity, kWaitLimitCycles, &b.failed)) set_error(p.err, kErrTimeout);
    };
    // by a whole warp, together again after it
    auto wait = [&](uint64_t& bar, uint32_t parity) {
        wait_one(bar, parity);
        __syncwarp();
    };

    if (warp < Sh::kWidenWarps) {
        // ---- widen: a thread a row, every second block of columns
        if (Sh::kUneven) reg_dealloc<Sh::kWidenRegs>();
        const int mine = warp >> 2, row = tid & 127;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21) + mine * Sh::kAhead * 64;
        Ring q, a;
        int turn = 0;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
#pragma unroll 1
            for (int st = 0; st < stages; ++st) {
                wait(b.q_full[q.slot], q.parity);
                const unsigned char* const stage = smem + kHeader + q.slot * p.stage_bytes;
                const unsigned char* const zeros = stage + lay.zeros;
                const int blocks = min(2, p.kblocks - 2 * st);
#pragma unroll 1
                for (int kb = 0; kb < blocks; ++kb, turn ^= 1) {
                    if (turn != mine) continue;
                    uint4 w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint4*>(stage + row * 128 + (((kb * 4 + i) ^ (row & 7)) << 4));
                    wait(b.a_empty[mine][a.slot], a.parity ^ 1u);
                    tcgen05_after_sync();
                    const uint32_t to = lanes + a.slot * 64;
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        uint32_t r[32];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int unit = part * 2 + i;   // 32 columns
                            float z = 8.f;
                            if (p.zeros) z = static_cast<float>(zeros[(((kb * 4 + unit) * 32) >> p.shift) * kRows + row]);
                            const __half2 z1 = __float2half2_rn(fmaf(z, 0x1p-14f, 0x1p-4f)), z16 = __float2half2_rn(fmaf(z, 0x1p-10f, 0x1p-4f));
                            widen_word(w[unit].x, z1, z16, r + 16 * i);
                            widen_word(w[unit].y, z1, z16, r + 16 * i + 4);
                            widen_word(w[unit].z, z1, z16, r + 16 * i + 8);
                            widen_word(w[unit].w, z1, z16, r + 16 * i + 12);
                        }
                        tmem_store32(to + part * 32, r);
                    }
                    tmem_wait_store();
                    tcgen05_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&b.a_full[mine][a.slot]));
                    a.next(Sh::kAhead);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&b.q_empty[q.slot]));
                q.next(p.qstages);
            }
        }
        // the products have read them: nothing arrives after the block's end
        for (int i = 0; i < Sh::kAhead; ++i, a.next(Sh::kAhead)) wait(b.a_empty[mine][a.slot], a.parity ^ 1u);
    } else if (warp < Sh::kFirstFew) {
        // ---- add the groups' sums
        if (Sh::kUneven) reg_alloc<Sh::kAddRegs>();
        const int own0 = ((warp - Sh::kWidenWarps) >> 2) * kOwn, row = tid & 127;
        const uint32_t quarter = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        const uint32_t from = quarter + Sh::kD + own0;
        Ring q;
        bool waited = false;
        int turn = 0;                        // of the block of columns
        uint32_t taken0 = 0, taken1 = 0;     // lots read so far of either turn
        const int of_block = kBlockCols >> p.shift, lot = Sh::kLots ? min(kSums, of_block) : 1;
        const uint32_t slots = kSums / lot;  // (of lots of more than one group: 1 or 2)
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const int vt = tile / p.tblocks, tb = tile - vt * p.tblocks;
            uint64_t acc[kOwn / 2];
#pragma unroll
            for (int i = 0; i < kOwn / 2; ++i) acc[i] = f2_pack(0.f, 0.f);
#pragma unroll 1
            for (int st = 0; st < stages; ++st) {
                wait(b.q_full[q.slot], q.parity);
                const unsigned char* const scales = smem + kHeader + q.slot * p.stage_bytes + lay.scales;
                const int n = min(per_stage, p.groups - st * per_stage);
                // small loops: the five parts of a block share the instruction cache
                auto scale_of = [&](int g) { return widen_any(scales, p.scale_dtype, g * kRows + row); };
                auto add = [&](uint32_t at, float s) {
                    const uint64_t s2 = f2_pack(s, s);
#pragma unroll
                    for (int c = 0; c < kOwn; c += 16) {
                        float f[16];
                        tmem_load16(at + c, f);
                        tmem_wait_load(f);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            uint64_t& x = acc[(c + i) / 2];
                            x = f2_fma(s2, f2_pack(f[i], f[i + 1]), x);
                        }
                    }
                };
                if (!Sh::kLots || lot == 1) {
#pragma unroll 1
                    for (int g = 0; g < n; ++g) {
                        const uint32_t taken = turn ? taken1 : taken0, slot = taken % static_cast<uint32_t>(kSums);
                        const float s = scale_of(g);
                        wait(b.d_full[turn][slot], taken / static_cast<uint32_t>(kSums) & 1u);
                        tcgen05_after_sync();
                        add(from + (turn * kSums + slot) * N, s);
                        tcgen05_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&b.d_empty[turn][slot]));
                        taken0 += turn ^ 1;
                        taken1 += turn;
                        if (((g + 1) << p.shift) % kBlockCols == 0 || g + 1 == n) turn ^= 1;   // the block of columns' last
                    }
                } else {
                    // the lots of the stage's two blocks of columns in turn, so that the one's products run while the
                    // other's sums are read
#pragma unroll 1
                    for (int i = 0; i < 2 * of_block; i += lot) {
                        const int second = i & lot ? 1 : 0, side = turn ^ second;
                        int g = second * of_block + (i - second * lot) / 2;
                        if (g >= n) continue;
                        const uint32_t taken = side ? taken1 : taken0, slot = taken & (slots - 1);
                        wait(b.d_full[side][slot], taken >> (slots - 1) & 1u);
                        tcgen05_after_sync();
                        uint32_t at = from + (side * kSums + slot * lot) * N;
                        const int end = min(g + lot, n);
#pragma unroll 1
                        for (; g < end; ++g, at += N) add(at, scale_of(g));
                        tcgen05_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&b.d_empty[side][slot]));
                        taken0 += side ^ 1;
                        taken1 += side;
                    }
                    if (p.kblocks - 2 * st == 1) turn ^= 1;   // a stage of one block of columns
                }
                if (lane == 0) mbar_arrive(smem_addr(&b.q_empty[q.slot]));
                q.next(p.qstages);
            }
            if (!waited) {
                grid_dep_wait();
                // each warp for itself
                bool odd = false;
                for (int t = lane; t < p.T; t += 32) {
                    const float f = p.inverse[t];
                    odd = odd || f != f;
                    b.factor[t] = f * 0x1p7f;
                }
                if (odd) b.odd = 1;
                __syncwarp();
                waited = true;
            }
            // this thread's hidden rows of the block's
            const int own = p.pairs ? kOwn / 2 : kOwn, t0 = tb * p.per + own0 / kOwn * own, rows = min(own, p.T - t0);
            const int64_t v = static_cast<int64_t>(vt) * kRows + row;
            if (v < p.V) {
                auto all = [&](auto type) {
                    using O = decltype(type);
                    typename O::raw* to = static_cast<typename O::raw*>(p.out) + static_cast<int64_t>(t0) * p.ld_out + v;
                    auto put = [&](int i, float x) {
                        if (i < rows) *to = static_cast<typename O::raw>(O::round(x * 0x1p7f * b.factor[t0 + i] * p.scale));
                        to += p.ld_out;
                    };
#pragma unroll
                    for (int i = 0; i < kOwn / 4; ++i) {
                        float a, c, e, f;
                        f2_unpack(acc[i], a, c);
                        if (p.pairs) {
                            f2_unpack(acc[i + kOwn / 4], e, f);
                            a = fmaf(e, 1.f / 2048.f, a);
                            c = fmaf(f, 1.f / 2048.f, c);
                        }
                        put(2 * i, a);
                        put(2 * i + 1, c);
                    }
                    if (!p.pairs) {
#pragma unroll
                        for (int i = kOwn / 4; i < kOwn / 2; ++i) {
                            float a, c;
                            f2_unpack(acc[i], a, c);
                            put(2 * i, a);
                            put(2 * i + 1, c);
                        }
                    }
                };
                if (p.out_dtype == LMLOSS_BF16) all(Bf16{});
                else if (p.out_dtype == LMLOSS_FP16) all(Fp16{});
                else all(Fp32{});
            }
            if (b.odd && v < p.V)
                for (int i = 0; i < rows; ++i)
                    if (b.factor[t0 + i] != b.factor[t0 + i]) store_plain(p, t0 + i, v);
            __syncwarp();
        }
    } else {
        if (Sh::kUneven) reg_dealloc<Sh::kFewRegs>();
        if (warp == Sh::kFirstFew) {
            // ---- the table
            if (lane == 0) {
                Ring q;
                for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x)
                    for (int st = 0; st < stages; ++st) {
                        wait_one(b.q_empty[q.slot], q.parity ^ 1u);
                        const uint32_t bar = smem_addr(&b.q_full[q.slot]);
                        mbar_arrive_expect_tx(bar, lay.copied);
                        copy_table(p, lay, maps, kRows, st, 1, tile / p.tblocks * kRows, base + kHeader + q.slot * p.stage_bytes, bar);
                        q.next(p.qstages);
                    }
            }
            __syncwarp();
        } else if (warp == Sh::kFirstFew + 1) {
            // ---- the hidden rows
            if (lane == 0) {
                grid_dep_wait();
                Ring x;
                for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
                    const unsigned char* from = p.x + static_cast<int64_t>(tile % p.tblocks) * p.kblocks * kXBytes;
                    for (int kb = 0; kb < p.kblocks; ++kb) {
                        wait_one(b.x_empty[x.slot], x.parity ^ 1u);
                        const uint32_t bar = smem_addr(&b.x_full[x.slot]);
                        mbar_arrive_expect_tx(bar, kXBytes);
                        bulk_load(xbase + x.slot * kXBytes, from + static_cast<int64_t>(kb) * kXBytes, kXBytes, bar);
                        x.next(p.xstages);
                    }
                }
                // the products have read them all: nothing arrives after the block's end
                for (int i = 0; i < p.xstages; ++i, x.next(p.xstages)) wait_one(b.x_empty[x.slot], x.parity ^ 1u);
            }
            __syncwarp();
        } else {
            // ---- the products, every second block of columns: one warp waits for its operands while the other's
            // products run.  (The tensor cores take few products ahead: by one warp, three waits a block of
            // columns left them idle half the time.)
            const uint32_t leader = elect_one();
            const int mine = warp - (Sh::kFirstFew + 2);
            auto multiply = [&](auto count) {
                constexpr int kSteps = decltype(count)::value;   // a group's, 16 columns each
                constexpr int kGroups = 8 / kSteps;              // of a block of columns
                constexpr int kLot = Sh::kLots ? (kGroups < kSums ? kGroups : kSums) : 1, kSlots = kSums / kLot;
                Ring x, a, d;
                int turn = 0;
                for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
                    int left = p.groups;
#pragma unroll 1
                    for (int kb = 0; kb < p.kblocks; ++kb, left -= kGroups, turn ^= 1, x.next(p.xstages)) {
                        if (turn != mine) continue;
                        wait(b.x_full[x.slot], x.parity);
                        const uint64_t desc = mma_desc_128b(xbase + x.slot * kXBytes);
                        wait(b.a_full[mine][a.slot], a.parity);
                        const uint32_t from = tmem + (mine * Sh::kAhead + a.slot) * 64;
#pragma unroll
                        for (int g0 = 0; g0 < kGroups; g0 += kLot) {
                            if (g0 >= left) break;
                            wait(b.d_empty[mine][d.slot], d.parity ^ 1u);
                            tcgen05_after_sync();
#pragma unroll
                            for (int g = g0; g < g0 + kLot; ++g) {
                                if (g >= left) break;
                                const uint32_t to = tmem + Sh::kD + (mine * kSums + d.slot * kLot + g - g0) * N;
#pragma unroll
                                for (int k = 0; k < kSteps; ++k) {
                                    const int step = g * kSteps + k;   // 64 columns lie in one run of N rows
                                    const uint64_t at = desc + (step >> 2) * (N * 128 / 16) + (step & 3) * 2;
                                    if (k == 0) mma_f16_ts<false>(to, from + step * 8, at, kIdesc, leader);
                                    else mma_f16_ts<true>(to, from + step * 8, at, kIdesc, leader);
                                }
                            }
                            mma_commit(smem_addr(&b.d_full[mine][d.slot]), leader);
                            d.next(kSlots);
                        }
                        mma_commit(smem_addr(&b.a_empty[mine][a.slot]), leader);
                        mma_commit(smem_addr(&b.x_empty[x.slot]), leader);
                        a.next(Sh::kAhead);
                    }
                }
            };
            if (gs == 128) multiply(std::integral_constant<int, 8>{});
            else if (gs == 64) multiply(std::integral_constant<int, 4>{});
            else multiply(std::integral_constant<int, 2>{});
        }
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (b.failed && tid == 0) {
        // copies and products may be in flight: give them their time
        const long long start = clock64();
        while (clock64() - start < 20000000) {
        }
    }
    __syncthreads();
    if (warp == Sh::kFirstFew + 2) tmem_free(tmem, Sh::kColumns);
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

int64_t kblocks_of(int64_t D) { return (D + kBlockCols - 1) / kBlockCols; }

// Workspace of a launch's hidden rows: the operand rows as fp16, padded to whole blocks, and a factor for each.
struct HiddenSpace {
    size_t inverse, total;
};
HiddenSpace hidden_space(int64_t T, int64_t D, bool pairs)
{
    const int64_t rows = std::min<int64_t>(T, kMaxRows) * (pairs ? 2 : 1);
    const int64_t padded = (rows + kMany - 1) / kMany * kMany, k = kblocks_of(D);
    HiddenSpace w{};
    w.inverse = vocab_align(static_cast<size_t>(padded * k * kBlockCols * 2));
    w.total = w.inverse + vocab_align(static_cast<size_t>(rows) * 4);
    return w;
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

bool table_maps(const lmloss_table4& t, int rows, int columns, TableMaps* maps)
{
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    auto map = [&](CUtensorMap* to, CUtensorMapDataType type, void* base, int64_t across, int64_t down, int64_t stride, int box_across,
                   int box_down, CUtensorMapSwizzle swizzle) {
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(across), static_cast<cuuint64_t>(down)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
        const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_across), static_cast<cuuint32_t>(box_down)}, steps[2] = {1, 1};
        return encode(to, type, 2, base, dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const int es = float_bytes(t.scale_dtype), n = columns / t.group;
    const int64_t G = (t.D + t.group - 1) / t.group;
    return map(&maps->values, CU_TENSOR_MAP_DATA_TYPE_UINT8, t.values, (t.D + 1) / 2, t.V, t.ld_values, 128, rows, CU_TENSOR_MAP_SWIZZLE_128B) &&
           map(&maps->scales, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT32, t.scales, t.V, G, t.ld_scales * es, rows,
               n, CU_TENSOR_MAP_SWIZZLE_NONE) &&
           (!t.zeros || map(&maps->zeros, CU_TENSOR_MAP_DATA_TYPE_UINT8, t.zeros, t.V, G, t.ld_zeros, rows, n, CU_TENSOR_MAP_SWIZZLE_NONE));
}

template <int N>
lmloss_status launch_many_rows(LogitsParams& p, const TableMaps& maps, lmloss_vocab_ctx* h, cudaStream_t stream)
{
    const StageLayout lay(kRows, kStageCols, p.shift, p.scale_bytes, p.zeros != nullptr);
    // of the SM's 228 KB each block takes 1 more than it asks for
    const uint32_t shared = Shape<N>::kBlocks == 1 ? kMaxShared : kMaxShared / 2 - 1024;
    p.stage_bytes = lay.bytes;
    p.xstages = N == 128 ? 3 : (N == 32 ? 4 : 6);
    p.qstages = std::min<int>(kMaxStages, (shared - kHeader - p.xstages * N * 256) / lay.bytes);
    constexpr uint32_t bit = 1u << (N == 16 ? 17 : (N == 32 ? 18 : (N == 64 ? 19 : 20)));
    if (!(h->limits_raised & bit)) {
        if (cudaFuncSetAttribute(logits_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared) != cudaSuccess) {
            cudaGetLastError();
            return LMLOSS_ERR_CUDA;
        }
        h->limits_raised |= bit;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(static_cast<int64_t>(p.vtiles) * p.tblocks, Shape<N>::kBlocks * h->num_sms)));
    cfg.blockDim = dim3(Shape<N>::kThreads);
    cfg.dynamicSmemBytes = kHeader + p.qstages * lay.bytes + p.xstages * N * 256;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, logits_kernel<N>, p, maps) != cudaSuccess) {
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
    *bytes = hidden_space(a->T, a->table.D, true).total;   // pairs take the most
    return LMLOSS_OK;
}

lmloss_status lmloss_table4_logits(lmloss_vocab_handle h, const lmloss_table4_logits_args* a, cudaStream_t stream)
{
    if (!h) return LMLOSS_ERR_INVALID_ARG;
    lmloss_status st = check_logits(a, true);
    if (st != LMLOSS_OK) return st;
    if (a->T == 0) return LMLOSS_OK;
    const bool pairs = a->hidden_dtype == LMLOSS_FP32;
    const HiddenSpace w = hidden_space(a->T, a->table.D, pairs);
    VocabDeviceGuard g(h->device);
    if (!g.ok) return LMLOSS_ERR_CUDA;
    for (int64_t t0 = 0; t0 < a->T; t0 += kMaxRows) {
        const int T = static_cast<int>(std::min<int64_t>(a->T - t0, kMaxRows));
        LogitsParams p{};
        p.values = a->table.values;
        p.ld_values = a->table.ld_values;
        p.scales = static_cast<const unsigned char*>(a->table.scales);
        p.ld_scales = a->table.ld_scales;
        p.zeros = a->table.zeros;
        p.ld_zeros = a->table.ld_zeros;
        p.V = static_cast<int>(a->table.V);
        p.D = static_cast<int>(a->table.D);
        p.shift = table4_params(a->table).shift;
        p.scale_dtype = a->table.scale_dtype;
        p.scale_bytes = float_bytes(a->table.scale_dtype);
        p.groups = static_cast<int>((a->table.D + a->table.group - 1) / a->table.group);
        p.kblocks = static_cast<int>(kblocks_of(a->table.D));
        p.T = T;
        p.pairs = pairs;
        p.hidden = static_cast<const unsigned char*>(a->hidden) + t0 * a->ld_hidden * float_bytes(a->hidden_dtype);
        p.ld_hidden = a->ld_hidden;
        p.hidden_dtype = a->hidden_dtype;
        p.out = static_cast<unsigned char*>(a->logits) + t0 * a->ld_logits * float_bytes(a->logits_dtype);
        p.ld_out = a->ld_logits;
        p.out_dtype = a->logits_dtype;
        p.scale = a->scale;
        p.err = h->err;
        const int operands = T * (pairs ? 2 : 1);
        // (few rows are pairs whatever their type where these fit: see table4_rows.cu)
        p.pairs = pairs || 2 * T <= kFewRows;
        const bool few = few_rows_fit(p) && (p.pairs || a->logits_dtype != LMLOSS_FP32);
        if (!few) {
            // (a first launch that is not of few rows is the call's: nothing has been launched yet)
            if (w.total > h->ws_bytes) return LMLOSS_ERR_INVALID_ARG;
            p.pairs = pairs;
        }
        const int rows = few ? kFewTile : kRows;
        p.vtiles = static_cast<int>((a->table.V + rows - 1) / rows);
        TableMaps maps{};
        if (!table_maps(a->table, rows, few ? kFewCols : kStageCols, &maps)) return LMLOSS_ERR_CUDA;
        if (few) {
            st = launch_few_rows(p, maps, h, stream);
        } else {
            HiddenParams x{};
            x.x = p.hidden;
            x.ld = p.ld_hidden;
            x.D = p.D;
            x.kblocks = p.kblocks;
            x.lanes = (1 << p.shift) / 8;
            x.N = p.N = operands <= 16 ? 16 : (operands <= 32 ? 32 : (operands <= 64 ? 64 : kMany));
            x.per = p.per = pairs ? p.N / 2 : p.N;
            x.own = p.N > 32 ? p.N / 2 : p.N;
            x.out = h->ws;
            x.inverse = reinterpret_cast<float*>(h->ws + w.inverse);
            p.tblocks = (T + p.per - 1) / p.per;
            p.x = x.out;
            p.inverse = x.inverse;
            switch (a->hidden_dtype) {
            case LMLOSS_BF16: hidden_kernel<Bf16><<<T, 256, 0, stream>>>(x); break;
            case LMLOSS_FP16: hidden_kernel<Fp16><<<T, 256, 0, stream>>>(x); break;
            default: hidden_kernel<Fp32><<<T, 256, 0, stream>>>(x); break;
            }
            if ((st = vocab_launch_err()) == LMLOSS_OK)
                st = p.N == 16 ? launch_many_rows<16>(p, maps, h, stream)
                               : (p.N == 32 ? launch_many_rows<32>(p, maps, h, stream)
                                             : (p.N == 64 ? launch_many_rows<64>(p, maps, h, stream) : launch_many_rows<kMany>(p, maps, h, stream)));
        }
        if (st != LMLOSS_OK) return st;
    }
    return LMLOSS_OK;
}

}  // extern "C"
