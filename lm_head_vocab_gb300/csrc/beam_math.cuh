// What a beam step computes for the order of its candidates beside the rows' sums: logarithms,
// powers, and bounds in fp32 on the rank keys.  The same on the host.
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>

#include "vocab_common.cuh"

namespace lmloss {
namespace {

__host__ __device__ inline uint32_t bits_of(float x)
{
    uint32_t b;
    memcpy(&b, &x, sizeof b);
    return b;
}
__host__ __device__ inline float float_of(uint32_t b)
{
    float x;
    memcpy(&x, &b, sizeof x);
    return x;
}
__host__ __device__ inline double double_of(uint64_t b)
{
    double x;
    memcpy(&x, &b, sizeof x);
    return x;
}

// ln(hi + lo) for a sum of at least 1, within 3e-9 (2.3e-9 the most seen), from fp32 operations alone but
// for its last three additions (fp64 runs at a sixty-fourth of fp32's rate here).
// hi + lo = 2^e f with f in [0.7, 1.42), ln f = 2 artanh(q) with q = (f - 1) / (f + 1):
// q is carried as a quotient and its remainder, the series' higher terms in fp32.
__host__ __device__ inline double log_of_sum(float hi, float lo)
{
    if (!(hi < INFINITY)) return static_cast<double>(hi);   // NaN
    int e = static_cast<int>(bits_of(hi) >> 23) - 127;
    float scale = float_of(static_cast<uint32_t>(127 - e) << 23);
    if (hi * scale > 1.4142135f) {
        ++e;
        scale *= 0.5f;
    }
    const float f = hi * scale, g = lo * scale;
    const float num = f - 1.f, den = f + 1.f, den_lo = (f - (den - 1.f)) + g;
    const float q = num / den;
    const float rest = (fmaf(-q, den, num) + fmaf(-q, den_lo, g)) / den;
    const float q2 = q * q;
    const float t = q2 * fmaf(q2, fmaf(q2, fmaf(q2, fmaf(q2, 1.f / 11, 1.f / 9), 1.f / 7), 0.2f), 1.f / 3);
    return fma(static_cast<double>(e), 0.693147180559945309417, 2.0 * static_cast<double>(q)) +
           static_cast<double>(2.f * fmaf(q, t, rest));
}

// n^a for n >= 1 and a > 0, within 3e-9 (1 + a) of itself: e^(a ln n) = 2^i e^r with
// |r| <= ln 2 / 2, the series to r^8 (what follows is below 2e-10), its terms from r^3 on in
// fp32; the logarithm's error counts a times.  (fp64's pow took 10 us of a step's 20.)
__host__ __device__ inline double power(int n, double a)
{
    if (a == 1.0) return static_cast<double>(n);
    const float hi = static_cast<float>(n);
    const double y = a * log_of_sum(hi, static_cast<float>(n - static_cast<int64_t>(hi)));
    const float i = rintf(static_cast<float>(y) * kLog2e);
    // near the range's end, and past it the largest value, by which a row's candidates keep their order
    if (!(i < 1000.f)) return fmin(pow(static_cast<double>(n), a), 1.7976931348623157e308);
    const double r = fma(static_cast<double>(i), -0.693147180559945309417, y);
    const float f = static_cast<float>(r);
    const float tail = f * f * f *
                       fmaf(f, fmaf(f, fmaf(f, fmaf(f, fmaf(f, 1.f / 40320, 1.f / 5040), 1.f / 720), 1.f / 120), 1.f / 24), 1.f / 6);
    const double e = 1.0 + (r + (0.5 * r * r + static_cast<double>(tail)));
    return e * double_of(static_cast<uint64_t>(static_cast<int64_t>(i) + 1023) << 52);
}

// Bounds on the rank key (base + z) / d of a candidate: its fp32 value, inv = 1 / d, and at most
// six roundings of 2^-24 of the terms.  From d = 1e30 on there are none: near fp32's range inv
// loses bits, then all of them, and the value says nothing of the rank.
__host__ __device__ inline void rank_bounds(float base, float z, float inv, float& low, float& high)
{
    const float x = (base + z) * inv, err = (fabsf(base) + fabsf(z)) * inv * 4.8e-7f + 1e-37f;
    const bool fine = fabsf(x) < INFINITY && err < INFINITY && inv > 1e-30f;
    low = fine ? x - err : -INFINITY;
    high = fine ? x + err : INFINITY;
}

}  // namespace
}  // namespace lmloss
