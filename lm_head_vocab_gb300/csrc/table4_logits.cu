// Logits from hidden rows and a vocabulary table in 4 bits.
//
//   logits[t][v] = scale sum_g s[g][v] sum_{c in g} x[t][c] (q[v][c] - z[g][v])
//
// The products with whole numbers are summed within a group and scaled once: no weight is rounded.
#include <algorithm>
#include <cmath>

#include "table4.cuh"

namespace lmloss {
namespace {

struct LogitsParams {
    Table4 t;
    const void* x;
    int64_t ld_x;
    int T;
    void* out;
    int64_t ld_out;
    float scale;
};

constexpr int kRows = 4;         // hidden rows at once

// A warp takes one row of the table and kRows hidden rows; a lane 8 columns at a time, which lie in one group.
template <class X, class O, class S>
__global__ void __launch_bounds__(256) logits_simple_kernel(const __grid_constant__ LogitsParams p)
{
    const Table4& t = p.t;
    const int lane = threadIdx.x & 31;
    const int64_t v = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * kRows;
    if (v >= t.V) return;
    float acc[kRows] = {};
    const uint8_t* q = t.values + v * t.ld_values;
    const typename X::raw* x = static_cast<const typename X::raw*>(p.x);
    for (int c = lane * 8; c < t.D; c += 256) {
        const uint32_t word = *reinterpret_cast<const uint32_t*>(q + c / 2);
        const int g = c >> t.shift;
        const float s = table4_scale<S>(t, g, v), z = table4_zero(t, g, v);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (t0 + r >= p.T) break;
            float sum = 0.f;
            for (int k = 0; k < 8; ++k)
                if (c + k < t.D) sum = fmaf(X::widen(x[(t0 + r) * p.ld_x + c + k]), static_cast<float>(word >> (4 * k) & 15u) - z, sum);
            acc[r] = fmaf(s, sum, acc[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        for (int o = 16; o > 0; o >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
        if (lane == 0 && t0 + r < p.T)
            static_cast<typename O::raw*>(p.out)[(t0 + r) * p.ld_out + v] = static_cast<typename O::raw>(O::round(p.scale * acc[r]));
    }
}

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

lmloss_status lmloss_table4_check_logits_args(const lmloss_table4_logits_args* a) { return check_logits(a, true); }

lmloss_status lmloss_table4_logits_workspace(const lmloss_table4_logits_args* a, size_t* bytes)
{
    if (!bytes) return LMLOSS_ERR_INVALID_ARG;
    const lmloss_status st = check_logits(a, false);
    if (st != LMLOSS_OK) return st;
    *bytes = 0;
    return LMLOSS_OK;
}

lmloss_status lmloss_table4_logits(lmloss_vocab_handle h, const lmloss_table4_logits_args* a, cudaStream_t stream)
{
    if (!h) return LMLOSS_ERR_INVALID_ARG;
    const lmloss_status st = check_logits(a, true);
    if (st != LMLOSS_OK) return st;
    if (a->T == 0) return LMLOSS_OK;
    VocabDeviceGuard g(h->device);
    if (!g.ok) return LMLOSS_ERR_CUDA;
    LogitsParams p{};
    p.t = table4_params(a->table);
    p.x = a->hidden;
    p.ld_x = a->ld_hidden;
    p.T = static_cast<int>(a->T);
    p.out = a->logits;
    p.ld_out = a->ld_logits;
    p.scale = a->scale;
    const int64_t most = 65535 * kRows;
    for (int64_t t0 = 0; t0 < a->T; t0 += most) {
        p.T = static_cast<int>(std::min<int64_t>(a->T - t0, most));
        p.x = static_cast<const unsigned char*>(a->hidden) + t0 * a->ld_hidden * float_bytes(a->hidden_dtype);
        p.out = static_cast<unsigned char*>(a->logits) + t0 * a->ld_logits * float_bytes(a->logits_dtype);
        const dim3 grid(static_cast<unsigned>((a->table.V + 7) / 8), static_cast<unsigned>((p.T + kRows - 1) / kRows));
        by_type(a->hidden_dtype, [&](auto x) {
            by_type(a->logits_dtype, [&](auto o) {
                by_type(a->table.scale_dtype, [&](auto s) {
                    logits_simple_kernel<decltype(x), decltype(o), decltype(s)><<<grid, 256, 0, stream>>>(p);
                });
            });
        });
        const lmloss_status launched = vocab_launch_err();
        if (launched != LMLOSS_OK) return launched;
    }
    return LMLOSS_OK;
}

}  // extern "C"
