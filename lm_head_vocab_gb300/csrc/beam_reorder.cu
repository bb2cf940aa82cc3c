// Reordering of the beams' states: row b * K_out + m of every state becomes its row
// b * K + parents[b, m].  Nothing is computed: the kernel is bound by memory, each
// surviving beam's run of bytes read once and each new one written once.  In
// place, beams that keep their slot are not touched at all.
//
// Measured (GB300, copy bandwidth 6.69 TB/s): 8 caches of 64 beams x 8 heads x 1531 of 2048
// positions x 128 bf16 into the other buffer, 5 of 8 beams surviving, 380 us = 6.9 TB/s
// (a beam taken twice is read once from DRAM); 4 caches of 64 x 4 x 777 x 80 in place, 2 of 4
// beams moving, 20 us = 6.3 TB/s; token histories, 2.7 us.
#include <algorithm>
#include <climits>
#include <numeric>

#include "vocab_common.cuh"

namespace lmloss {
namespace {

constexpr int kMaxK = LMLOSS_MAX_BEAMS;
constexpr int kThreads = 128;
constexpr int kStates = 16;                  // states of one launch
constexpr int kColumns = 4;                  // units a thread moves of each run
constexpr int kMoves = 8;                    // runs on their way at a time

struct State {
    const unsigned char* src;
    unsigned char* dst;
    int64_t src_row, dst_row;
    int64_t src_outer[3], dst_outer[3];
    int64_t units;               // of a run
    unsigned chunks;             // blocks over a run
    unsigned first;              // first block of this state in the launch
    unsigned outer[3];
    int unit;                    // bytes moved at a time: 16, 8, 4, 2 or 1
    int in_place;
};

struct ReorderParams {
    State st[kStates];
    int n;
    int B, K, K_out;
    const int32_t* parents;
    int* err;
};

// What a block moves: runs from and to these byte offsets.
struct Moves {
    int64_t src[kMaxK], dst[kMaxK];
    int n;
};

// C columns of at most kMoves / C runs, all on their way at once.
template <class U, int C>
__device__ __forceinline__ void move_few(const Moves& mv, const unsigned char* src, unsigned char* dst, int64_t u0, int64_t units)
{
    constexpr int N = kMoves / C;
    const int n = mv.n;
#pragma unroll 1
    for (int x = 0; x < kColumns; x += C) {
        const int64_t u = u0 + x * kThreads + threadIdx.x;
        U v[C][N];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (j < n && u + c * kThreads < units)
                    v[c][j] = *reinterpret_cast<const U*>(src + (u + c * kThreads) * sizeof(U) + mv.src[j]);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (j < n && u + c * kThreads < units)
                    *reinterpret_cast<U*>(dst + (u + c * kThreads) * sizeof(U) + mv.dst[j]) = v[c][j];
    }
}

// Units [u0, u0 + kThreads * kColumns) of the runs.  A thread reads and writes its own
// columns only.  In place, every run that another slot takes is read before any slot is
// written: in registers where there are few, else through shared memory.
template <class U>
__device__ __forceinline__ void move_runs(const Moves& mv, const unsigned char* src, unsigned char* dst, int64_t u0,
                                          int64_t units, bool in_place, unsigned char* stage)
{
    const int n = mv.n;
    if (n <= 2) return move_few<U, 4>(mv, src, dst, u0, units);
    if (n <= 4) return move_few<U, 2>(mv, src, dst, u0, units);
    if (n <= kMoves) return move_few<U, 1>(mv, src, dst, u0, units);
#pragma unroll 1
    for (int x = 0; x < kColumns; ++x) {
        const int64_t u = u0 + x * kThreads + threadIdx.x;
        if (u >= units) return;
        const unsigned char* from = src + u * sizeof(U);
        unsigned char* to = dst + u * sizeof(U);
        if (in_place) {
            U* own = reinterpret_cast<U*>(stage) + threadIdx.x;
#pragma unroll 4
            for (int j = 0; j < n; ++j) own[j * kThreads] = *reinterpret_cast<const U*>(from + mv.src[j]);
            for (int j = 0; j < n; ++j) *reinterpret_cast<U*>(to + mv.dst[j]) = own[j * kThreads];
            continue;
        }
        for (int j0 = 0; j0 < n; j0 += kMoves) {
            U v[kMoves];
#pragma unroll
            for (int j = 0; j < kMoves; ++j)
                if (j0 + j < n) v[j] = *reinterpret_cast<const U*>(from + mv.src[j0 + j]);
#pragma unroll
            for (int j = 0; j < kMoves; ++j)
                if (j0 + j < n) *reinterpret_cast<U*>(to + mv.dst[j0 + j]) = v[j];
        }
    }
}

__global__ void __launch_bounds__(kThreads) beam_reorder_kernel(const __grid_constant__ ReorderParams p)
{
    extern __shared__ __align__(16) unsigned char stage[];   // [K][kThreads] units, in place only
    __shared__ Moves mv;
    int i = 0;
    while (i + 1 < p.n && blockIdx.x >= p.st[i + 1].first) ++i;
    const State& st = p.st[i];
    unsigned k = blockIdx.x - st.first;
    const unsigned chunk = k % st.chunks;
    k /= st.chunks;
    const unsigned b = k % static_cast<unsigned>(p.B);
    const unsigned o = k / static_cast<unsigned>(p.B);
    const unsigned o2 = o % st.outer[2], o1 = o / st.outer[2] % st.outer[1], o0 = o / st.outer[2] / st.outer[1];
    if (threadIdx.x < 32) {
        // the slots that something is moved to, in order
        int n = 0;
        for (int m0 = 0; m0 < p.K_out; m0 += 32) {
            const int m = m0 + static_cast<int>(threadIdx.x);
            bool moved = false;
            int q = 0;
            if (m < p.K_out) {
                q = p.parents[static_cast<int64_t>(b) * p.K_out + m];
                moved = q >= 0 && q < p.K;
                if (!moved) set_error(p.err, kErrBadParent);
                if (st.in_place && q == m) moved = false;
            }
            const unsigned who = __ballot_sync(0xffffffffu, moved);
            if (moved) {
                const int at = n + __popc(who & ((1u << threadIdx.x) - 1u));
                mv.src[at] = q * st.src_row;
                mv.dst[at] = m * st.dst_row;
            }
            n += __popc(who);
        }
        if (threadIdx.x == 0) mv.n = n;
    }
    __syncthreads();
    const unsigned char* src = st.src + static_cast<int64_t>(b) * p.K * st.src_row + o0 * st.src_outer[0] +
                               o1 * st.src_outer[1] + o2 * st.src_outer[2];
    unsigned char* dst = st.dst + static_cast<int64_t>(b) * p.K_out * st.dst_row + o0 * st.dst_outer[0] +
                         o1 * st.dst_outer[1] + o2 * st.dst_outer[2];
    const int64_t u0 = static_cast<int64_t>(chunk) * (kThreads * kColumns);
    switch (st.unit) {
    case 16: move_runs<uint4>(mv, src, dst, u0, st.units, st.in_place, stage); break;
    case 8: move_runs<uint2>(mv, src, dst, u0, st.units, st.in_place, stage); break;
    case 4: move_runs<uint32_t>(mv, src, dst, u0, st.units, st.in_place, stage); break;
    case 2: move_runs<uint16_t>(mv, src, dst, u0, st.units, st.in_place, stage); break;
    default: move_runs<uint8_t>(mv, src, dst, u0, st.units, st.in_place, stage); break;
    }
}

// ------------------------------------------------------------------- host
// The last byte offset that a side of a state reaches, or -1 if it passes 2^62.
int64_t reach(int64_t row_stride, int64_t rows, const int64_t* outer, const int64_t* outer_stride, int64_t inner)
{
    __int128 r = static_cast<__int128>(rows - 1) * row_stride + inner;
    for (int i = 0; i < 3; ++i) r += static_cast<__int128>(outer[i] - 1) * outer_stride[i];
    return r > (static_cast<__int128>(1) << 62) ? -1 : static_cast<int64_t>(r);
}

// No byte of one side of a state is one of the other's.  The sides may lie interleaved (halves of
// a double buffer with the halves inside a row): where all strides above some size are multiples
// of g, each side's bytes are those of a block of the smaller dimensions, repeated every so many
// times g, so the two are apart if such blocks are, modulo g.
bool apart(const lmloss_beam_state& s, int64_t rows, int64_t rows_out, int64_t reach_src, int64_t reach_dst)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(s.src), d = reinterpret_cast<uintptr_t>(s.dst);
    if (a + static_cast<uintptr_t>(reach_src) <= d || d + static_cast<uintptr_t>(reach_dst) <= a) return true;
    const int64_t stride[2][4] = {{s.src_row_stride, s.src_outer_stride[0], s.src_outer_stride[1], s.src_outer_stride[2]},
                                  {s.dst_row_stride, s.dst_outer_stride[0], s.dst_outer_stride[1], s.dst_outer_stride[2]}};
    const int64_t count[2][4] = {{rows, s.outer[0], s.outer[1], s.outer[2]}, {rows_out, s.outer[0], s.outer[1], s.outer[2]}};
    for (int i = 0; i < 8; ++i) {
        // what counts as large: a stride of either side, and all above it
        const int64_t least = stride[i / 4][i % 4];
        if (least == 0) continue;
        int64_t g = 0, block[2] = {s.inner, s.inner};
        for (int x = 0; x < 2; ++x)
            for (int k = 0; k < 4; ++k) {
                if (count[x][k] < 2) continue;
                if (stride[x][k] >= least) g = std::gcd(g, stride[x][k]);
                else block[x] += (count[x][k] - 1) * stride[x][k];
            }
        if (g == 0) continue;
        const uint64_t u = static_cast<uint64_t>(g);
        const int64_t from = a <= d ? static_cast<int64_t>((d - a) % u) : static_cast<int64_t>((u - (a - d) % u) % u);
        if (block[0] <= from && block[1] <= g - from) return true;
    }
    return false;
}

bool empty(const lmloss_beam_state& s)
{
    return s.inner == 0 || s.outer[0] == 0 || s.outer[1] == 0 || s.outer[2] == 0;
}

// States move side by side, so none may write what another reads or writes.  Seen where the two begin
// at the same byte, by a table of up to kTabled states' dst at a time (comparing all pairs took 40 us
// for 160 states, a launch's time and more).
bool apart_from_one_another(const lmloss_beam_state* states, int n)
{
    constexpr int kTabled = 512;
    int32_t table[4 * kTabled];
    for (int first = 0; first < n; first += kTabled) {
        const int last = std::min(n, first + kTabled);
        int bits = 3;
        while ((1 << bits) < 4 * (last - first)) ++bits;
        std::fill_n(table, 1 << bits, -1);
        // the place of the state whose dst is p, or where it would be
        auto find = [&](const void* p) {
            uint64_t at = (reinterpret_cast<uintptr_t>(p) * 0x9e3779b97f4a7c15ull) >> (64 - bits);
            while (table[at] >= 0 && states[table[at]].dst != p) at = (at + 1) & ((1u << bits) - 1);
            return table + at;
        };
        for (int i = first; i < last; ++i) {
            if (empty(states[i])) continue;
            int32_t* held = find(states[i].dst);
            if (*held < 0) *held = i;
        }
        for (int i = 0; i < n; ++i) {
            if (empty(states[i])) continue;
            const int writes = *find(states[i].dst), read = *find(states[i].src);
            if (read >= 0 && read != i) return false;
            // one state given twice, not in place, is written twice alike
            if (writes >= 0 && states[writes].src != states[i].src) return false;
        }
    }
    return true;
}

lmloss_status check_states(const lmloss_beam_state* states, int32_t n, int64_t B, int32_t K, int32_t K_out)
{
    if (n < 0 || (n > 0 && !states) || B < 0 || K < 1 || K_out < 1) return LMLOSS_ERR_INVALID_ARG;
    if (K > LMLOSS_MAX_BEAMS || K_out > LMLOSS_MAX_BEAMS) return LMLOSS_ERR_INVALID_ARG;
    if (B > (int64_t(1) << 24)) return LMLOSS_ERR_UNSUPPORTED;
    for (int i = 0; i < n; ++i) {
        const lmloss_beam_state& s = states[i];
        if (s.inner < 0 || s.src_row_stride < 0 || s.dst_row_stride < 0) return LMLOSS_ERR_INVALID_ARG;
        for (int k = 0; k < 3; ++k) {
            if (s.outer[k] < 0 || s.src_outer_stride[k] < 0 || s.dst_outer_stride[k] < 0) return LMLOSS_ERR_INVALID_ARG;
            if (s.outer[k] > INT_MAX) return LMLOSS_ERR_UNSUPPORTED;
        }
        if (B == 0 || empty(s)) continue;
        if (!s.src || !s.dst) return LMLOSS_ERR_INVALID_ARG;
        // neighbouring runs of dst are apart
        if (B * K_out > 1 && s.dst_row_stride < s.inner) return LMLOSS_ERR_INVALID_ARG;
        for (int k = 0; k < 3; ++k)
            if (s.outer[k] > 1 && s.dst_outer_stride[k] < s.inner) return LMLOSS_ERR_INVALID_ARG;
        if (s.src == s.dst) {
            if (K != K_out || s.src_row_stride != s.dst_row_stride) return LMLOSS_ERR_INVALID_ARG;
            for (int k = 0; k < 3; ++k)
                if (s.outer[k] > 1 && s.src_outer_stride[k] != s.dst_outer_stride[k]) return LMLOSS_ERR_INVALID_ARG;
        }
        const int64_t rs = reach(s.src_row_stride, B * K, s.outer, s.src_outer_stride, s.inner);
        const int64_t rd = reach(s.dst_row_stride, B * K_out, s.outer, s.dst_outer_stride, s.inner);
        if (rs < 0 || rd < 0) return LMLOSS_ERR_INVALID_ARG;
        if (s.src != s.dst && !apart(s, B * K, B * K_out, rs, rd)) return LMLOSS_ERR_INVALID_ARG;
    }
    return B == 0 || apart_from_one_another(states, n) ? LMLOSS_OK : LMLOSS_ERR_INVALID_ARG;
}

// the widest unit that every run starts at and is a multiple of
int unit_of(const lmloss_beam_state& s)
{
    uint64_t all = reinterpret_cast<uintptr_t>(s.src) | reinterpret_cast<uintptr_t>(s.dst) |
                   static_cast<uint64_t>(s.inner) | static_cast<uint64_t>(s.src_row_stride) |
                   static_cast<uint64_t>(s.dst_row_stride);
    for (int k = 0; k < 3; ++k)
        if (s.outer[k] > 1)
            all |= static_cast<uint64_t>(s.src_outer_stride[k]) | static_cast<uint64_t>(s.dst_outer_stride[k]);
    int u = 16;
    while (all & static_cast<uint64_t>(u - 1)) u /= 2;
    return u;
}

}  // namespace
}  // namespace lmloss

using namespace lmloss;

extern "C" {

lmloss_status lmloss_beam_check_states(const lmloss_beam_state* states, int32_t n, int64_t B, int32_t K, int32_t K_out)
{
    return check_states(states, n, B, K, K_out);
}

lmloss_status lmloss_beam_reorder(lmloss_vocab_handle h, const lmloss_beam_state* states, int32_t n,
                                  const int32_t* parents, int64_t B, int32_t K, int32_t K_out, cudaStream_t stream)
{
    if (!h) return LMLOSS_ERR_INVALID_ARG;
    lmloss_status st = check_states(states, n, B, K, K_out);
    if (st != LMLOSS_OK) return st;
    if (B > 0 && n > 0 && !parents) return LMLOSS_ERR_INVALID_ARG;
    if (B == 0) return LMLOSS_OK;
    // block counts first: nothing is launched if one state is too large
    for (int i = 0; i < n; ++i) {
        const lmloss_beam_state& s = states[i];
        if (empty(s)) continue;
        const __int128 blocks = static_cast<__int128>((s.inner / unit_of(s) + kThreads * kColumns - 1) / (kThreads * kColumns)) * B *
                                s.outer[0] * s.outer[1] * s.outer[2];
        if (blocks > INT_MAX / kStates) return LMLOSS_ERR_UNSUPPORTED;
    }
    VocabDeviceGuard g(h->device);
    if (!g.ok) return LMLOSS_ERR_CUDA;
    for (int i = 0; i < n;) {
        ReorderParams p{};
        p.B = static_cast<int>(B);
        p.K = K;
        p.K_out = K_out;
        p.parents = parents;
        p.err = h->err;
        int64_t blocks = 0;
        bool staged = false;
        for (; i < n && p.n < kStates; ++i) {
            const lmloss_beam_state& s = states[i];
            if (empty(s)) continue;
            State& d = p.st[p.n++];
            d.src = static_cast<const unsigned char*>(s.src);
            d.dst = static_cast<unsigned char*>(s.dst);
            d.src_row = s.src_row_stride;
            d.dst_row = s.dst_row_stride;
            for (int k = 0; k < 3; ++k) {
                d.outer[k] = static_cast<unsigned>(s.outer[k]);
                d.src_outer[k] = s.src_outer_stride[k];
                d.dst_outer[k] = s.dst_outer_stride[k];
            }
            d.unit = unit_of(s);
            d.units = s.inner / d.unit;
            d.chunks = static_cast<unsigned>((d.units + kThreads * kColumns - 1) / (kThreads * kColumns));
            d.in_place = s.src == s.dst;
            staged = staged || (d.in_place && K > kMoves);
            d.first = static_cast<unsigned>(blocks);
            blocks += static_cast<int64_t>(d.chunks) * B * s.outer[0] * s.outer[1] * s.outer[2];
        }
        if (blocks == 0) continue;
        size_t smem = staged ? static_cast<size_t>(K) * kThreads * 16 : 0;
        if (smem > 48 * 1024 &&
            cudaFuncSetAttribute(beam_reorder_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 LMLOSS_MAX_BEAMS * kThreads * 16) != cudaSuccess) {
            cudaGetLastError();
            return LMLOSS_ERR_CUDA;
        }
        beam_reorder_kernel<<<static_cast<unsigned>(blocks), kThreads, smem, stream>>>(p);
        if ((st = vocab_launch_err()) != LMLOSS_OK) return st;
    }
    return LMLOSS_OK;
}

}  // extern "C"
