// A vocabulary table in 4 bits: made from float weights, and looked up.
//
//   w[v][c] = s[g][v] (q[v][c] - z[g][v]),  g = c / group
//
// Making a table reads the weights and writes half a byte for each; the lookup reads half a byte for each column
// and writes the row.  Both would be bound by memory, and are where elements are wide: 128256 x 4096 made from fp32
// in groups of 32, 361 us (1.00 of the copy's rate); the whole table to fp32, 355 us (1.00).  Otherwise by
// instructions: made from bf16 in groups of 128, 258 us (0.76; 77% of the issue slots, 15 instructions a
// weight and lane); 32767 of 151936 x 2048 to bf16, 39 us (0.66).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "table4.cuh"

namespace lmloss {

lmloss_status table4_check(const lmloss_table4& t, bool pointers)
{
    if (t.V < 1 || t.D < 1 || (t.group != 32 && t.group != 64 && t.group != 128)) return LMLOSS_ERR_INVALID_ARG;
    if (!float_dtype(t.scale_dtype)) return LMLOSS_ERR_INVALID_ARG;
    if (t.V > (int64_t(1) << 31) - (1 << 16) || t.D > (int64_t(1) << 20)) return LMLOSS_ERR_UNSUPPORTED;
    if (!pointers) return LMLOSS_OK;
    if (!t.values || !t.scales || !aligned16(t.values) || !aligned16(t.scales) || !aligned16(t.zeros))
        return LMLOSS_ERR_INVALID_ARG;
    if (t.ld_values < (t.D + 1) / 2 || t.ld_values % 16 || t.ld_values > (int64_t(1) << 32)) return LMLOSS_ERR_INVALID_ARG;
    if (t.ld_scales < t.V || t.ld_scales > (int64_t(1) << 32) || t.ld_scales * float_bytes(t.scale_dtype) % 16)
        return LMLOSS_ERR_INVALID_ARG;
    if (t.zeros && (t.ld_zeros < t.V || t.ld_zeros > (int64_t(1) << 32) || t.ld_zeros % 16)) return LMLOSS_ERR_INVALID_ARG;
    return LMLOSS_OK;
}

namespace {

// Rows and their vectors over threads without divisions: a block is `across` vectors (a power of two) of
// 256 / across rows, kDeep times down.
constexpr int kDeep = 4;

struct Spread {
    int log_across;
    int blocks_across;           // blocks along a row
    int64_t down;                // rows of a block
    explicit Spread(int64_t vectors)   // at least one
    {
        log_across = 4;          // a group's threads are neighbours
        while (log_across < 8 && (int64_t(1) << log_across) < vectors) ++log_across;
        blocks_across = static_cast<int>((vectors + (int64_t(1) << log_across) - 1) >> log_across);
        down = kDeep << (8 - log_across);
    }
    // rows of a launch: whole blocks within the grid's limit
    int64_t most() const { return ((int64_t(1) << 31) - 1) / blocks_across * down; }
};

// max and min that keep a NaN
__device__ __forceinline__ float keep_max(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float keep_min(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// ---------------------------------------------------------------- quantize
struct QuantizeParams {
    Table4 t;
    const void* weight;
    const unsigned char* weight_end;
    int64_t ld;
    int64_t rows;
    int aligned;                 // rows begin on 16-byte boundaries
    int log_across, blocks_across;
    int* err;
};

// The whole number nearest to a quotient, halves to the even one, from q = a r + 1.5 2^23 rounded (r = 1 / s), which
// may be one off next to a half.  The remainder a - q s is exact in fp32 there: a multiple of half a step of s,
// and at most about s / 2.
__device__ __forceinline__ float settle(float q, float a, float s)
{
    const float rest = fmaf(-q, s, a), half = 0.5f * s;
    const bool odd = __float_as_uint(q + 12582912.f) & 1u;
    if (fabsf(rest) > half || (fabsf(rest) == half && odd)) q += rest > 0.f ? 1.f : -1.f;
    return q;
}

// x / D rounded once, where the remainder does not underflow: a product with the rounded reciprocal is one step off at
// most, and its exact remainder settles that (Markstein, 1990; checked for 7 and 15 over all significands).
template <int D>
__device__ __forceinline__ float quotient_by(float x)
{
    if (x < 0x1p-90f) return __fdiv_rn(x, static_cast<float>(D));
    constexpr float r = 1.f / D;
    const float q = __fmul_rn(x, r);
    return fmaf(fmaf(-q, static_cast<float>(D), x), r, q);
}

// The largest (or least) of each of kDeep rows over a group's threads: the thread of quad q leaves with row q's.
template <class F>
__device__ __forceinline__ float over_group(const float (&x)[kDeep], int lanes, F&& most)
{
    static_assert(kDeep == 4, "a quad's threads");
    const bool two = threadIdx.x & 2, one = threadIdx.x & 1;
    const float a = most(two ? x[2] : x[0], __shfl_xor_sync(0xffffffffu, two ? x[0] : x[2], 2));
    const float b = most(two ? x[3] : x[1], __shfl_xor_sync(0xffffffffu, two ? x[1] : x[3], 2));
    float m = most(one ? b : a, __shfl_xor_sync(0xffffffffu, one ? a : b, 1));
    if (lanes > 4) m = most(m, __shfl_xor_sync(0xffffffffu, m, 4));
    if (lanes > 8) m = most(m, __shfl_xor_sync(0xffffffffu, m, 8));
    return m;
}

// Two numbers of 16 bits at once, as max and min that keep a NaN
template <class W>
__device__ __forceinline__ uint32_t keep_max2(uint32_t a, uint32_t b)
{
    uint32_t r;
    if constexpr (W::kIndex == Bf16::kIndex) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <class W>
__device__ __forceinline__ uint32_t keep_min2(uint32_t a, uint32_t b)
{
    uint32_t r;
    if constexpr (W::kIndex == Bf16::kIndex) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A thread takes 8 columns of kDeep rows; a group's 4, 8 or 16 neighbouring threads share its extremes, and of each
// quad a thread works out one row's scale, reciprocal and zero point.  The quotients, in pairs:
//   weights and scales of 16 bits   two corrections bring a quotient within 2^-22 of a w / s that is n + 1/2 or at
//                                   least 2^-14 away from it (of significands below 2^11, w / s - n - 1/2 has a
//                                   denominator below 2^14), and exactly to n + 1/2: nothing is left to settle
//   others                          one product, settled where one of the eight lies within 2^-20 of a half
// Quotients of 16-bit weights are halves often (their largest is a multiple of seven in one group of seven): with one
// product, settled, and extremes of one row at a time, 128256 x 4096 took 418 us.
template <class W, class S, bool ZEROS>
__global__ void __launch_bounds__(256) quantize_kernel(const __grid_constant__ QuantizeParams p)
{
    const Table4& t = p.t;
    const int64_t down = blockIdx.x / static_cast<unsigned>(p.blocks_across);
    const int along = static_cast<int>(blockIdx.x - static_cast<unsigned>(down) * static_cast<unsigned>(p.blocks_across));
    const int c = ((along << p.log_across) + (threadIdx.x & ((1 << p.log_across) - 1))) * 8;
    const int rows_a_pass = 256 >> p.log_across;
    const int64_t v0 = down * (kDeep * rows_a_pass) + (threadIdx.x >> p.log_across);
    const int lanes = (1 << t.shift) / 8, g = c >> t.shift;
    const int rows = static_cast<int>(min(p.rows - v0, static_cast<int64_t>(kDeep * rows_a_pass)));   // from v0 on
    const bool whole = c + 8 <= t.D;
    const unsigned char* const base = static_cast<const unsigned char*>(p.weight);
    const unsigned char* at = base + (v0 * p.ld + c) * W::kBytes;
    const int64_t step = p.ld * rows_a_pass * W::kBytes;

    Pack<W, 8> in[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k, at += step) {
        in[k].zero();
        if (k * rows_a_pass >= rows) continue;
        if (p.aligned && whole) {
            in[k].load(at);
        } else if (whole && inside_blocks<W, 8>(at, base, p.weight_end)) {
            constexpr int kVecs = 8 * W::kBytes / 16 + 1;
            const uint4* a = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(at) & ~uintptr_t(15));
            uint4 x[kVecs];
#pragma unroll
            for (int i = 0; i < kVecs; ++i) x[i] = __ldg(a + i);
            shift_blocks<W, 8>(in[k], x, static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at)));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < t.D) in[k].set(i, W::widen(reinterpret_cast<const typename W::raw*>(at)[i]));
        }
    }
    float lo[kDeep], hi[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
        if constexpr (W::kBytes == 2) {
            uint32_t high = 0, low = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                high = keep_max2<W>(high, ZEROS ? in[k].w[i] : in[k].w[i] & 0x7fff7fffu);
                if (ZEROS) low = keep_min2<W>(low, in[k].w[i]);
            }
            hi[k] = keep_max(W::widen(static_cast<uint16_t>(high)), W::widen(static_cast<uint16_t>(high >> 16)));
            lo[k] = ZEROS ? keep_min(W::widen(static_cast<uint16_t>(low)), W::widen(static_cast<uint16_t>(low >> 16))) : 0.f;
        } else {
            lo[k] = hi[k] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = in[k].get(i);
                hi[k] = keep_max(hi[k], ZEROS ? x : fabsf(x));
                if (ZEROS) lo[k] = keep_min(lo[k], x);
            }
        }
    }
    // this thread's row of the group
    constexpr float kMagic = 12582912.f;   // x + kMagic - kMagic is the whole number nearest to x
    const int quad = threadIdx.x & 3;
    const float top = over_group(hi, lanes, keep_max), bottom = ZEROS ? over_group(lo, lanes, keep_min) : 0.f, range = top - bottom;
    float own = S::widen(static_cast<typename S::raw>(S::round(quotient_by<ZEROS ? 15 : 7>(range)))), own_z = ZEROS ? 0.f : 8.f;
    // not finite: a weight, or the scale in its type.  (top - bottom may pass fp32's range too.)
    const bool bad = !(own < INFINITY) || !(top < INFINITY) || !(bottom > -INFINITY);
    // a scale whose reciprocal passes fp32's range is brought up, with its weights
    const bool tiny = own < 0x1p-100f && W::kIndex != Fp16::kIndex;
    const float up = tiny ? 0x1p100f : 1.f;
    float own_r = __frcp_rn(own * up);
    if (ZEROS && !bad && own > 0.f) {
        const float below = -bottom * up;
        own_z = fminf(fmaxf(settle(fmaf(below, own_r, kMagic) - kMagic, below, own * up), 0.f), 15.f);
    }
    if ((threadIdx.x & (lanes - 1)) < 4 && quad * rows_a_pass < rows && c - quad * 8 < t.D) {
        const int64_t v = v0 + quad * rows_a_pass;
        static_cast<typename S::raw*>(t.scales)[g * t.ld_scales + v] = static_cast<typename S::raw>(S::round(bad ? NAN : own));
        if (ZEROS) t.zeros[g * t.ld_zeros + v] = static_cast<uint8_t>(own_z);
        if (bad) set_error(p.err, kErrRange);
    }
    // Taken one by one, told by the sign: a group of zeros or with a number that is not finite; one brought up; one
    // whose scale lost bits in its type's subnormals, so that quotients may be out of range.
    if (bad) own = 0.f;
    if (own == 0.f || tiny || !(range < own * (ZEROS ? 15.2f : 7.4f))) own_r = -own_r;
    uint8_t* out = t.values + v0 * t.ld_values + c / 2;
    const int64_t out_step = t.ld_values * rows_a_pass;
#pragma unroll
    for (int k = 0; k < kDeep; ++k, out += out_step) {
        const int from = (threadIdx.x & 28) + k;
        const float s = __shfl_sync(0xffffffffu, own, from), r = __shfl_sync(0xffffffffu, own_r, from);
        const float z = ZEROS ? __shfl_sync(0xffffffffu, own_z, from) : 8.f, least = -z, largest = 15.f - z;
        if (k * rows_a_pass >= rows || c >= t.D) continue;
        uint64_t x2[4];   // of columns i and i + 4
        bool one_by_one = r < 0.f;
        if (!one_by_one) {
            const uint64_t s2 = f2_pack(-s, -s), r2 = f2_pack(r, r), magic2 = f2_pack(kMagic, kMagic), unmagic2 = f2_pack(-kMagic, -kMagic);
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t a = f2_pack(in[k].get(i), in[k].get(i + 4));
                if constexpr (W::kBytes == 2 && S::kBytes == 2) {
                    const uint64_t q = f2_mul(a, r2);
                    x2[i] = f2_add(f2_add(f2_fma(f2_fma(q, s2, a), r2, q), magic2), unmagic2);
                } else {
                    x2[i] = f2_add(f2_fma(a, r2, magic2), unmagic2);
                    float e0, e1;
                    f2_unpack(f2_fma(x2[i], s2, a), e0, e1);
                    most = fmaxf(fmaxf(most, fabsf(e0)), fabsf(e1));
                }
                if (ZEROS) {   // (one more than 15 where both ends round up)
                    float x0, x1;
                    f2_unpack(x2[i], x0, x1);
                    x2[i] = f2_pack(fminf(x0, largest), fminf(x1, largest));
                }
            }
            one_by_one = (W::kBytes != 2 || S::kBytes != 2) && !(most < s * 0.4999995f);
        }
        if (one_by_one) {
            float x[8];
            const float lift = s < 0x1p-100f && W::kIndex != Fp16::kIndex ? 0x1p100f : 1.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = in[k].get(i) * lift;
                x[i] = s == 0.f ? 0.f : fminf(fmaxf(settle(fmaf(a, fabsf(r), kMagic) - kMagic, a, s * lift), least), largest);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x2[i] = f2_pack(x[i], x[i + 4]);
        }
        // four numbers make one below 2^16, exact in fp32; z is added to all four at once
        const uint64_t sixteen2 = f2_pack(16.f, 16.f);
        const float more = fmaf(z, 4369.f, 8388608.f);
        float low, high;
        f2_unpack(f2_add(f2_fma(f2_fma(f2_fma(x2[3], sixteen2, x2[2]), sixteen2, x2[1]), sixteen2, x2[0]), f2_pack(more, more)), low, high);
        uint32_t word = __byte_perm(__float_as_uint(low), __float_as_uint(high), 0x5410);
        if (whole) {
            *reinterpret_cast<uint32_t*>(out) = word;
        } else {
            word &= (1u << (4 * (t.D - c))) - 1u;
            for (int i = 0; c + 2 * i < t.D; ++i) out[i] = static_cast<uint8_t>(word >> (8 * i));
        }
    }
}

// ------------------------------------------------------------------ lookup
struct LookupParams {
    Table4 t;
    const void* ids;
    int ids32;
    int T;
    void* rows;
    int64_t ld_rows;
    float scale;
    int log_across, blocks_across;
    int* err;
};

// scale (s (q - z)) of a word's eight numbers, in pairs.  A number's nibble, as a byte, under the exponent of 2^23 is
// 2^23 + q; less 2^23 + z it is exact.  (By shifts and masks, number by number, 32767 rows of 2048 took 41.5 us for 39.)
__device__ __forceinline__ void eight_numbers(uint32_t w, float s, float z, float scale, float (&x)[8])
{
    const uint32_t even = w & 0x0f0f0f0fu, odd = w >> 4 & 0x0f0f0f0fu;
    const float less = -8388608.f - z;
    const uint64_t less2 = f2_pack(less, less), s2 = f2_pack(s, s), scale2 = f2_pack(scale, scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(__byte_perm(even, 0x4b000000u, 0x7440 + i)), b = __uint_as_float(__byte_perm(odd, 0x4b000000u, 0x7440 + i));
        f2_unpack(f2_mul(scale2, f2_mul(s2, f2_add(f2_pack(a, b), less2))), x[2 * i], x[2 * i + 1]);
    }
}

// Whole aligned rows: a thread takes a word, 8 columns, of kDeep rows, and writes 16-byte vectors.  Of fp32 those are
// two; neighbouring threads exchange words so that each of their stores fills a 32-byte sector together.
template <class R, class S>
__global__ void __launch_bounds__(256) lookup_words_kernel(const __grid_constant__ LookupParams p)
{
    const Table4& t = p.t;
    const unsigned down = blockIdx.x / static_cast<unsigned>(p.blocks_across);
    const int along = static_cast<int>(blockIdx.x - down * static_cast<unsigned>(p.blocks_across));
    const int c = ((along << p.log_across) + (threadIdx.x & ((1 << p.log_across) - 1))) * 8;
    const int rows_a_pass = 256 >> p.log_across;
    const int row0 = static_cast<int>(down) * (kDeep * rows_a_pass) + (threadIdx.x >> p.log_across);
    const bool in = c < t.D;
    const typename S::raw* const scales = static_cast<const typename S::raw*>(t.scales) + static_cast<int64_t>(in ? c >> t.shift : 0) * t.ld_scales;
    const uint8_t* const zeros = t.zeros ? t.zeros + static_cast<int64_t>(in ? c >> t.shift : 0) * t.ld_zeros : nullptr;
    int64_t id[kDeep];
    uint32_t word[kDeep];
    float s[kDeep], z[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
        const int row = row0 + k * rows_a_pass;
        id[k] = row >= p.T ? LMLOSS_IGNORE_INDEX
                           : (p.ids32 ? static_cast<int64_t>(static_cast<const int32_t*>(p.ids)[row]) : static_cast<const int64_t*>(p.ids)[row]);
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
        word[k] = 0;
        s[k] = z[k] = 0.f;
        if (!in || id[k] < 0 || id[k] >= t.V) {
            if (id[k] != LMLOSS_IGNORE_INDEX && (id[k] < 0 || id[k] >= t.V)) {
                set_error(p.err, kErrBadTarget);
                s[k] = NAN;
            }
            continue;
        }
        word[k] = __ldg(reinterpret_cast<const uint32_t*>(t.values + id[k] * t.ld_values + (c >> 1)));
        s[k] = S::widen(__ldg(scales + id[k]));
        z[k] = zeros ? static_cast<float>(__ldg(zeros + id[k])) : 8.f;
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
        const int row = row0 + k * rows_a_pass;
        // 2^23 + q, less 2^23 + z: exact
        const float off = 8388608.f + z[k];
        auto value = [&](uint32_t w, int i) { return p.scale * (s[k] * (__uint_as_float((w >> (4 * i) & 15u) | 0x4b000000u) - off)); };
        if constexpr (R::kBytes == 2) {
            if (!in || row >= p.T) continue;
            float x[8];
            eight_numbers(word[k], s[k], z[k], p.scale, x);
            Pack<R, 8> v;
            v.set_all(x);
            v.store(static_cast<typename R::raw*>(p.rows) + static_cast<int64_t>(row) * p.ld_rows + c);
        } else {
            const bool odd = threadIdx.x & 1;
            const uint32_t other = __shfl_xor_sync(0xffffffffu, word[k], 1);
            const uint32_t first = (odd ? other : word[k]) >> (odd ? 16 : 0), second = (odd ? word[k] : other) >> (odd ? 16 : 0);
            if (row >= p.T) continue;
            float* const out = static_cast<float*>(p.rows) + static_cast<int64_t>(row) * p.ld_rows + (c & ~15) + (odd ? 4 : 0);
            Pack<R, 4> v;
            float x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = value(first, i);
            v.set_all(x);
            if ((c & ~15) < t.D) v.store(out);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = value(second, i);
            v.set_all(x);
            if ((c | 8) < t.D) v.store(out + 8);
        }
    }
}

// Rows at any alignment: a warp takes 32 neighbouring words of kDeep rows and writes the 31 vectors (of fp32, pairs of
// vectors) that lie on 16-byte boundaries of the row, each put together from a word's numbers and the last of the word
// before, which the neighbouring thread has.  The warp before ends with this one's first word.
// (By vectors on their own, with two words, two groups and a scale for each number, it took 45 instructions a
// number: 32003 x 1001 to fp32, 79 us.  Of fp32, with half a sector written at a time, 37.6, and 33.6 so.)
template <class R, class S>
__global__ void __launch_bounds__(256) lookup_shifted_kernel(const __grid_constant__ LookupParams p)
{
    constexpr int kWords = 8 * R::kBytes / 4;                // of 8 numbers in the result's type
    constexpr int kUnit = 16 / R::kBytes;                    // numbers of a vector
    const Table4& t = p.t;
    const int lane = threadIdx.x & 31;
    const unsigned warp = blockIdx.x * 8u + (threadIdx.x >> 5), down = warp / static_cast<unsigned>(p.blocks_across);
    const int along = static_cast<int>(warp - down * static_cast<unsigned>(p.blocks_across));
    const int k8 = along * 31 + lane - 1, c = k8 * 8;        // the thread's word and its first column
    const bool in = k8 >= 0 && c < t.D;
    const int row0 = static_cast<int>(down) * kDeep;
    if (row0 >= p.T) return;
    const typename S::raw* const scales = static_cast<const typename S::raw*>(t.scales) + static_cast<int64_t>(in ? c >> t.shift : 0) * t.ld_scales;
    const uint8_t* const zeros = t.zeros ? t.zeros + static_cast<int64_t>(in ? c >> t.shift : 0) * t.ld_zeros : nullptr;
    int64_t id[kDeep];
    uint32_t word[kDeep];
    float s[kDeep], z[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
        const int row = row0 + k;
        id[k] = row >= p.T ? LMLOSS_IGNORE_INDEX
                           : (p.ids32 ? static_cast<int64_t>(static_cast<const int32_t*>(p.ids)[row]) : static_cast<const int64_t*>(p.ids)[row]);
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
        word[k] = 0;
        s[k] = z[k] = 0.f;
        if (id[k] != LMLOSS_IGNORE_INDEX && (id[k] < 0 || id[k] >= t.V)) {
            set_error(p.err, kErrBadTarget);
            s[k] = NAN;
        } else if (in && id[k] >= 0) {
            word[k] = __ldg(reinterpret_cast<const uint32_t*>(t.values + id[k] * t.ld_values + (c >> 1)));
            s[k] = S::widen(__ldg(scales + id[k]));
            z[k] = zeros ? static_cast<float>(__ldg(zeros + id[k])) : 8.f;
        }
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
        const int row = row0 + k;
        if (row >= p.T) break;
        typename R::raw* const out = static_cast<typename R::raw*>(p.rows) + static_cast<int64_t>(row) * p.ld_rows;
        const int off = static_cast<int>((reinterpret_cast<uintptr_t>(out) & 15u) / R::kBytes);   // numbers of the row's first vector before it
        float x[8];
        eight_numbers(word[k], s[k], z[k], p.scale, x);
        Pack<R, 8> own;
        own.set_all(x);
        // the last `off` of the word before, then this one's: w[0] begins 16 bytes before this word's numbers
        uint32_t w[kWords + 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(0xffffffffu, own.w[kWords - 4 + i], 1);
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[4 + i] = own.w[i];
        const int sh = 16 - off * R::kBytes;   // bytes to leave out: 16 where rows are aligned
        Pack<R, 8> v;
        auto leave_out = [&](auto words) {     // (a row's, so that a warp goes one way)
            constexpr int kOut = decltype(words)::value;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const int next = i + kOut + 1 < kWords + 4 ? i + kOut + 1 : kWords + 3;   // (of 16 bytes none is needed)
                v.w[i] = R::kBytes == 4 ? w[i + kOut] : __funnelshift_r(w[i + kOut], w[next], (sh & 2) * 8);
            }
        };
        switch (sh >> 2) {
        case 0: leave_out(std::integral_constant<int, 0>{}); break;
        case 1: leave_out(std::integral_constant<int, 1>{}); break;
        case 2: leave_out(std::integral_constant<int, 2>{}); break;
        case 3: leave_out(std::integral_constant<int, 3>{}); break;
        default: leave_out(std::integral_constant<int, 4>{});
        }
        // numbers [first, first + 8) of the row; the thread behind its last word has what that word leaves
        const int first = c - off;
        auto put = [&](int from, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
            if (from >= 0 && from + kUnit <= t.D) {
                *reinterpret_cast<uint4*>(out + from) = make_uint4(w0, w1, w2, w3);
            } else {
                const uint32_t some[4] = {w0, w1, w2, w3};
#pragma unroll
                for (int i = 0; i < kUnit; ++i)
                    if (from + i >= 0 && from + i < t.D) {
                        if constexpr (R::kBytes == 4) out[from + i] = some[i];
                        else out[from + i] = static_cast<typename R::raw>(some[i / 2] >> (16 * (i & 1)));
                    }
            }
        };
        if constexpr (R::kBytes == 2) {
            if (lane > 0) put(first, v.w[0], v.w[1], v.w[2], v.w[3]);
        } else {
            // two neighbours write the one's 32 bytes, then the other's: whole sectors at once
            const bool odd = lane & 1;
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = __shfl_xor_sync(0xffffffffu, odd ? v.w[i] : v.w[4 + i], 1);
            if (lane > 1) put(odd ? first - 4 : first, odd ? y[0] : v.w[0], odd ? y[1] : v.w[1], odd ? y[2] : v.w[2], odd ? y[3] : v.w[3]);
            put(odd ? first + 4 : first + 8, odd ? v.w[4] : y[0], odd ? v.w[5] : y[1], odd ? v.w[6] : y[2], odd ? v.w[7] : y[3]);
        }
    }
}

lmloss_status check_quantize(const lmloss_table4_quantize_args* a)
{
    if (!a) return LMLOSS_ERR_INVALID_ARG;
    const lmloss_status st = table4_check(a->table, true);
    if (st != LMLOSS_OK) return st;
    if (!float_dtype(a->weight_dtype) || a->ld_weight < a->table.D || a->ld_weight > INT64_MAX / 16 / a->table.V) return LMLOSS_ERR_INVALID_ARG;
    if (!a->weight || reinterpret_cast<uintptr_t>(a->weight) % float_bytes(a->weight_dtype)) return LMLOSS_ERR_INVALID_ARG;
    return LMLOSS_OK;
}

lmloss_status check_lookup(const lmloss_table4_lookup_args* a)
{
    if (!a) return LMLOSS_ERR_INVALID_ARG;
    const lmloss_status st = table4_check(a->table, true);
    if (st != LMLOSS_OK) return st;
    if (a->T < 0 || a->ld_rows < a->table.D || !float_dtype(a->rows_dtype) || !std::isfinite(a->scale)) return LMLOSS_ERR_INVALID_ARG;
    if (a->ids_dtype != LMLOSS_INT64 && a->ids_dtype != LMLOSS_INT32) return LMLOSS_ERR_INVALID_ARG;
    if (a->T >= (int64_t(1) << 30)) return LMLOSS_ERR_UNSUPPORTED;
    if (a->T > 0) {
        if (a->ld_rows > INT64_MAX / 16 / a->T) return LMLOSS_ERR_INVALID_ARG;
        if (!a->ids || reinterpret_cast<uintptr_t>(a->ids) % (a->ids_dtype == LMLOSS_INT64 ? 8 : 4)) return LMLOSS_ERR_INVALID_ARG;
        if (!a->rows || reinterpret_cast<uintptr_t>(a->rows) % float_bytes(a->rows_dtype)) return LMLOSS_ERR_INVALID_ARG;
    }
    return LMLOSS_OK;
}

template <class F>
void by_type(int32_t dtype, F&& f)
{
    if (dtype == LMLOSS_BF16) f(Bf16{});
    else if (dtype == LMLOSS_FP16) f(Fp16{});
    else f(Fp32{});
}

}  // namespace
}  // namespace lmloss

using namespace lmloss;

extern "C" {

lmloss_status lmloss_table4_check(const lmloss_table4* t) { return t ? table4_check(*t, true) : LMLOSS_ERR_INVALID_ARG; }
lmloss_status lmloss_table4_check_quantize_args(const lmloss_table4_quantize_args* a) { return check_quantize(a); }
lmloss_status lmloss_table4_check_lookup_args(const lmloss_table4_lookup_args* a) { return check_lookup(a); }

lmloss_status lmloss_table4_quantize(lmloss_vocab_handle h, const lmloss_table4_quantize_args* a, cudaStream_t stream)
{
    if (!h) return LMLOSS_ERR_INVALID_ARG;
    const lmloss_status st = check_quantize(a);
    if (st != LMLOSS_OK) return st;
    VocabDeviceGuard g(h->device);
    if (!g.ok) return LMLOSS_ERR_CUDA;
    const Spread all((a->table.D + a->table.group - 1) / a->table.group * (a->table.group / 8));
    const int64_t most = all.most();
    for (int64_t v0 = 0; v0 < a->table.V; v0 += most) {
        QuantizeParams p{};
        p.t = table4_params(a->table);
        p.rows = std::min<int64_t>(a->table.V - v0, most);
        p.t.values += v0 * a->table.ld_values;
        p.t.scales = static_cast<unsigned char*>(p.t.scales) + v0 * float_bytes(a->table.scale_dtype);
        if (p.t.zeros) p.t.zeros += v0;
        p.weight = static_cast<const unsigned char*>(a->weight) + v0 * a->ld_weight * float_bytes(a->weight_dtype);
        p.weight_end = static_cast<const unsigned char*>(p.weight) + ((p.rows - 1) * a->ld_weight + a->table.D) * float_bytes(a->weight_dtype);
        p.ld = a->ld_weight;
        p.aligned = aligned16(p.weight) && a->ld_weight * float_bytes(a->weight_dtype) % 16 == 0;
        p.log_across = all.log_across;
        p.blocks_across = all.blocks_across;
        p.err = h->err;
        const unsigned grid = static_cast<unsigned>(all.blocks_across * ((p.rows + all.down - 1) / all.down));
        by_type(a->weight_dtype, [&](auto w) {
            by_type(a->table.scale_dtype, [&](auto s) {
                if (p.t.zeros) quantize_kernel<decltype(w), decltype(s), true><<<grid, 256, 0, stream>>>(p);
                else quantize_kernel<decltype(w), decltype(s), false><<<grid, 256, 0, stream>>>(p);
            });
        });
        const lmloss_status launched = vocab_launch_err();
        if (launched != LMLOSS_OK) return launched;
    }
    return LMLOSS_OK;
}

lmloss_status lmloss_table4_lookup(lmloss_vocab_handle h, const lmloss_table4_lookup_args* a, cudaStream_t stream)
{
    if (!h) return LMLOSS_ERR_INVALID_ARG;
    const lmloss_status st = check_lookup(a);
    if (st != LMLOSS_OK) return st;
    if (a->T == 0) return LMLOSS_OK;
    VocabDeviceGuard g(h->device);
    if (!g.ok) return LMLOSS_ERR_CUDA;
    const int E = 16 / float_bytes(a->rows_dtype);
    // (of fp32, 16 columns at a time: they lie in one group)
    const bool words = a->table.D % 8 == 0 && (a->table.D % 16 == 0 || E == 8) && aligned16(a->rows) && a->ld_rows % E == 0;
    Spread all((a->table.D + 7) / 8);
    if (!words) {
        // warps: 31 words each, and one behind the last for what shifts out of it
        all.blocks_across = static_cast<int>(((a->table.D + 7) / 8 + 1 + 30) / 31);
        all.down = kDeep;
    }
    const int64_t most = all.most();
    for (int64_t t0 = 0; t0 < a->T; t0 += most) {
        LookupParams p{};
        p.t = table4_params(a->table);
        p.ids = static_cast<const unsigned char*>(a->ids) + t0 * (a->ids_dtype == LMLOSS_INT64 ? 8 : 4);
        p.ids32 = a->ids_dtype == LMLOSS_INT32;
        p.T = static_cast<int>(std::min<int64_t>(a->T - t0, most));
        p.rows = static_cast<unsigned char*>(a->rows) + t0 * a->ld_rows * float_bytes(a->rows_dtype);
        p.ld_rows = a->ld_rows;
        p.scale = a->scale;
        p.log_across = all.log_across;
        p.blocks_across = all.blocks_across;
        p.err = h->err;
        const int64_t pieces = all.blocks_across * ((p.T + all.down - 1) / all.down);   // blocks, or warps
        const unsigned grid = static_cast<unsigned>(words ? pieces : (pieces + 7) / 8);
        by_type(a->rows_dtype, [&](auto r) {
            by_type(a->table.scale_dtype, [&](auto s) {
                if (words) lookup_words_kernel<decltype(r), decltype(s)><<<grid, 256, 0, stream>>>(p);
                else lookup_shifted_kernel<decltype(r), decltype(s)><<<grid, 256, 0, stream>>>(p);
            });
        });
        const lmloss_status launched = vocab_launch_err();
        if (launched != LMLOSS_OK) return launched;
    }
    return LMLOSS_OK;
}

}  // extern "C"
