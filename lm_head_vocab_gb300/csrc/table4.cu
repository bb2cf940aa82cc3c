// A vocabulary table in 4 bits: made from float weights, and looked up.
//
//   w[v][c] = s[g][v] (q[v][c] - z[g][v]),  g = c / group
//
// Both are bound by memory: making a table reads the weights and writes half a byte for each; the lookup reads half a byte for each column
// and writes the row.
#include <algorithm>
#include <cmath>

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

// ---------------------------------------------------------------- quantize
struct QuantizeParams {
    Table4 t;
    const void* weight;
    int64_t ld;
    int64_t chunks;              // runs of 8 columns of a row, to whole groups
    int64_t total;               // of all rows
    int* err;
};

// A thread takes 8 columns; a group's 4, 8 or 16 neighbouring threads share its extremes.
template <class W, class S>
__global__ void __launch_bounds__(256) quantize_kernel(const __grid_constant__ QuantizeParams p)
{
    const Table4& t = p.t;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const bool in = i < p.total;
    const int64_t v = in ? i / p.chunks : 0;
    const int c = static_cast<int>(in ? i - v * p.chunks : 0) * 8;
    const int lanes = (1 << t.shift) / 8;
    float x[8];
    const typename W::raw* w = static_cast<const typename W::raw*>(p.weight) + v * p.ld + c;
    if (in && c + 8 <= t.D && (reinterpret_cast<uintptr_t>(w) & 15u) == 0) {
        Pack<W, 8> q;
        q.load(w);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = q.get(k);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = in && c + k < t.D ? W::widen(w[k]) : 0.f;
    }
    // extremes; NaN and infinities show up in `sum`
    float lo = 0.f, hi = 0.f, sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        lo = fminf(lo, x[k]);
        hi = fmaxf(hi, x[k]);
        sum += x[k] * 0.f;
    }
    for (int o = 1; o < lanes; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    const float ideal = t.zeros ? __fdiv_rn(hi - lo, 15.f) : __fdiv_rn(fmaxf(hi, -lo), 7.f);
    const typename S::raw sr = static_cast<typename S::raw>(S::round(ideal));
    float s = S::widen(sr);
    const bool bad = !(sum == 0.f) || !(s < INFINITY);
    float z = 0.f;
    if (bad || s == 0.f) {
        // all weights count as 0
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = 0.f;
    } else {
        // nearest whole numbers of exact quotients: q = rint(x / s) may be one off where the quotient is within a
        // rounding of a half; the remainder x - q s says so
        auto nearest = [&](float a) {
            float q = rintf(__fdiv_rn(a, s));
            if (fabsf(q) < 64.f) {
                const double r = fma(-static_cast<double>(q), static_cast<double>(s), static_cast<double>(a)), half = 0.5 * static_cast<double>(s);
                const bool odd = fmodf(q, 2.f) != 0.f;
                if (r > half || (r == half && odd)) q += 1.f;
                else if (r < -half || (r == -half && odd)) q -= 1.f;
            }
            return q;
        };
        if (t.zeros) {
            z = fminf(fmaxf(nearest(-lo), 0.f), 15.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = fminf(fmaxf(nearest(x[k]) + z, 0.f), 15.f) - z;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = fminf(fmaxf(nearest(x[k]), -8.f), 7.f);
        }
    }
    if (!in) return;
    const float zero = t.zeros ? z : 8.f;
    uint32_t word = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (c + k < t.D) word |= static_cast<uint32_t>(x[k] + zero) << (4 * k);
    uint8_t* out = t.values + v * t.ld_values + c / 2;
    if (c + 8 <= t.D) {
        *reinterpret_cast<uint32_t*>(out) = word;
    } else {
        for (int k = 0; c + 2 * k < t.D; ++k) out[k] = static_cast<uint8_t>(word >> (8 * k));
    }
    if ((c & ((1 << t.shift) - 1)) == 0) {
        const int g = c >> t.shift;
        static_cast<typename S::raw*>(t.scales)[g * t.ld_scales + v] = bad ? static_cast<typename S::raw>(S::round(NAN)) : sr;
        if (t.zeros) t.zeros[g * t.ld_zeros + v] = static_cast<uint8_t>(z);
        if (bad) set_error(p.err, kErrRange);
    }
}

// ------------------------------------------------------------------ lookup
struct LookupParams {
    Table4 t;
    const void* ids;
    int ids32;
    void* rows;
    int64_t ld_rows;
    float scale;
    int64_t chunks;              // vectors of a row
    int64_t total;
    int* err;
};

// A thread takes the 8 columns (4 of fp32) of one 16-byte vector of a row that is written; at a row's ends,
// where a vector reaches past them, columns go one by one.
template <class R, class S>
__global__ void __launch_bounds__(256) lookup_kernel(const __grid_constant__ LookupParams p)
{
    constexpr int E = 16 / R::kBytes;
    const Table4& t = p.t;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= p.total) return;
    const int64_t row = i / p.chunks;
    typename R::raw* out = static_cast<typename R::raw*>(p.rows) + row * p.ld_rows;
    const int c0 = static_cast<int>(i - row * p.chunks) * E - static_cast<int>((reinterpret_cast<uintptr_t>(out) & 15u) / R::kBytes);
    if (c0 >= t.D) return;
    const int64_t id = p.ids32 ? static_cast<int64_t>(static_cast<const int32_t*>(p.ids)[row]) : static_cast<const int64_t*>(p.ids)[row];
    const bool ok = id >= 0 && id < t.V;
    if (!ok && id != LMLOSS_IGNORE_INDEX) set_error(p.err, kErrBadTarget);
    const float other = ok || id == LMLOSS_IGNORE_INDEX ? 0.f : NAN;
    const uint8_t* q = t.values + (ok ? id : 0) * t.ld_values;
    auto column = [&](int c) {
        if (!ok) return other;
        const int g = c >> t.shift;
        const float w = table4_scale<S>(t, g, id) * (static_cast<float>(q[c >> 1] >> (4 * (c & 1)) & 15) - table4_zero(t, g, id));
        return p.scale * w;
    };
    if (c0 < 0 || c0 + E > t.D) {
        for (int k = 0; k < E; ++k)
            if (c0 + k >= 0 && c0 + k < t.D) out[c0 + k] = static_cast<typename R::raw>(R::round(column(c0 + k)));
        return;
    }
    float x[E];
#pragma unroll
    for (int k = 0; k < E; ++k) x[k] = column(c0 + k);
    Pack<R, E> v;
    v.set_all(x);
    v.store(out + c0);
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
    const int64_t chunks = (a->table.D + a->table.group - 1) / a->table.group * (a->table.group / 8);
    // whole rows a launch, within the grid's limit
    const int64_t most = std::max<int64_t>(((int64_t(1) << 31) - 1) / chunks * 256, 1);
    for (int64_t v0 = 0; v0 < a->table.V; v0 += most) {
        QuantizeParams p{};
        p.t = table4_params(a->table);
        const int64_t rows = std::min<int64_t>(a->table.V - v0, most);
        p.t.values += v0 * a->table.ld_values;
        p.t.scales = static_cast<unsigned char*>(p.t.scales) + v0 * float_bytes(a->table.scale_dtype);
        if (p.t.zeros) p.t.zeros += v0;
        p.weight = static_cast<const unsigned char*>(a->weight) + v0 * a->ld_weight * float_bytes(a->weight_dtype);
        p.ld = a->ld_weight;
        p.chunks = chunks;
        p.total = rows * chunks;
        p.err = h->err;
        const unsigned grid = static_cast<unsigned>((p.total + 255) / 256);
        by_type(a->weight_dtype, [&](auto w) {
            by_type(a->table.scale_dtype, [&](auto s) { quantize_kernel<decltype(w), decltype(s)><<<grid, 256, 0, stream>>>(p); });
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
    const int64_t chunks = (a->table.D + 2 * E - 2) / E;   // one more where a row starts inside a vector
    const int64_t most = ((int64_t(1) << 31) - 1) / chunks * 256;
    for (int64_t t0 = 0; t0 < a->T; t0 += most) {
        LookupParams p{};
        p.t = table4_params(a->table);
        p.ids = static_cast<const unsigned char*>(a->ids) + t0 * (a->ids_dtype == LMLOSS_INT64 ? 8 : 4);
        p.ids32 = a->ids_dtype == LMLOSS_INT32;
        p.rows = static_cast<unsigned char*>(a->rows) + t0 * a->ld_rows * float_bytes(a->rows_dtype);
        p.ld_rows = a->ld_rows;
        p.scale = a->scale;
        p.chunks = chunks;
        p.total = std::min<int64_t>(a->T - t0, most) * chunks;
        p.err = h->err;
        const unsigned grid = static_cast<unsigned>((p.total + 255) / 256);
        by_type(a->rows_dtype, [&](auto r) {
            by_type(a->table.scale_dtype, [&](auto s) { lookup_kernel<decltype(r), decltype(s)><<<grid, 256, 0, stream>>>(p); });
        });
        const lmloss_status launched = vocab_launch_err();
        if (launched != LMLOSS_OK) return launched;
    }
    return LMLOSS_OK;
}

}  // extern "C"
