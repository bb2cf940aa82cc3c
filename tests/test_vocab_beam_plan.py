"""The parts that a beam step cuts its rows into, on the host: every column belongs to one part, also
at the largest vocabularies, where the last part ends past 2^31 columns if nothing stops it."""
import math

import pytest
import torch

from tests import vocab_host

PROGRAM = r"""
#include <cstdio>
#include "beam_plan.cuh"
using namespace lmloss;

int main()
{
    const int64_t longest = (int64_t(1) << 31) - (1 << 16);
    const int64_t sizes[] = {1, 7, 2047, 8192, 8193, 128256, 262144, (1 << 24) + 5, longest - (1 << 24), longest - (1 << 20),
                             longest - 8192, longest - 1, longest};
    const int shapes[][2] = {{1, 1}, {1, 2}, {1, 4}, {1, 5}, {1, 17}, {1, 64}, {3, 1}, {2, 8}, {64, 8}, {700, 1}, {1000, 64}};
    const int types[] = {LMLOSS_BF16, LMLOSS_FP16, LMLOSS_FP32};
    long plans = 0;
    for (int64_t V : sizes)
        for (auto& shape : shapes)
            for (int type : types)
                for (int sms : {1, 16, 132, 148, 152, 160}) {
                    lmloss_beam_args a{};
                    a.B = shape[0];
                    a.K = shape[1];
                    a.M = 64;
                    a.V = a.ld = V;
                    a.dtype = type;
                    BeamPlan P{};
                    if (plan_beam(&a, sms, P) != LMLOSS_OK) continue;
                    ++plans;
                    const int64_t cols = int64_t(P.vpt) * kThreads * (16 / float_bytes(type)), size = P.tiles * cols;
                    // a part begins inside the row, and what a block adds to a column stays in 32 bits
                    if (size > (int64_t(1) << 31) - 1 || (P.slices - 1) * size >= V || V + cols > (int64_t(1) << 31) - 1) {
                        std::printf("V %ld B %ld K %d sms %d: %d parts of %ld columns\n", long(V), long(a.B), a.K, sms, P.slices, long(size));
                        return 1;
                    }
                    for (int part = 0; part < P.slices; ++part) {
                        const int64_t begin = part * size, want = std::min(begin + size, V);
                        const int end = part_end(part * P.tiles * int(cols), P.tiles, int(cols), int(V));
                        if (end != want || (part + 1 == P.slices && end != V)) {
                            std::printf("V %ld B %ld K %d type %d sms %d: part %d of %d ends at %d, not %ld\n", long(V), long(a.B),
                                        a.K, type, sms, part, P.slices, end, long(want));
                            return 1;
                        }
                    }
                }
    std::printf("%ld\n", plans);
    return 0;
}
"""


def test_parts_cover_every_row(tmp_path):
    # all but the shapes whose parts are too many for one launch
    assert int(vocab_host.run(tmp_path, PROGRAM)[0]) > 2000


@pytest.mark.gpu
@pytest.mark.parametrize("short", [0, 8191])
def test_the_last_columns_of_the_longest_row(short):
    import __graft_entry__
    __graft_entry__.build()
    from lm_head_vocab_gb300 import VocabOps
    V = (1 << 31) - (1 << 16) - short
    ops = VocabOps(0, max_tokens=0, max_rows=1, max_vocab=V)
    z = torch.full((1, V), -30.0, device="cuda", dtype=torch.bfloat16)
    z[0, V - 1], z[0, V - 2], z[0, 7] = 5.0, 3.0, 4.0
    r = ops.beam_step(z, torch.zeros(1, 1, device="cuda"), num_candidates=4)
    assert ops.device_error() == 0
    assert r.tokens[0].tolist() == [V - 1, 7, V - 2, 0]
    lse = math.log(math.exp(5) + math.exp(4) + math.exp(3) + (V - 3) * math.exp(-30))
    # fewer than 2^12 additions in a chain, each within 2^-24 of the sum; ex2 and its argument within 2^-19
    assert abs(r.lse.item() - lse) < 2.0 ** -12 + 2.0 ** -18
    for got, x in zip(r.scores[0].tolist(), (5, 4, 3, -30)):
        assert abs(got - (x - lse)) < 2.0 ** -12 + 2.0 ** -18
    ops.close()
