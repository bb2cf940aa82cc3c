// A vocabulary table in 4 bits, as the kernels see it.
#pragma once

#include "vocab_common.cuh"

namespace lmloss {
namespace {

// w[v][c] = scales[g][v] (q[v][c] - zeros[g][v]), g = c / group
struct Table4 {
    uint8_t* values;
    int64_t ld_values;
    void* scales;
    int64_t ld_scales;
    uint8_t* zeros;
    int64_t ld_zeros;
    int V, D;
    int shift;                   // log2 of the group
};

inline Table4 table4_params(const lmloss_table4& t)
{
    Table4 p{};
    p.values = t.values;
    p.ld_values = t.ld_values;
    p.scales = t.scales;
    p.ld_scales = t.ld_scales;
    p.zeros = t.zeros;
    p.ld_zeros = t.ld_zeros;
    p.V = static_cast<int>(t.V);
    p.D = static_cast<int>(t.D);
    p.shift = t.group == 32 ? 5 : (t.group == 64 ? 6 : 7);
    return p;
}

}  // namespace

// Shared by the table's entry points: everything but the pointers, or with them.
lmloss_status table4_check(const lmloss_table4& t, bool pointers);

}  // namespace lmloss
