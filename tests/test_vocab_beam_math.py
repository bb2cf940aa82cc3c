"""The logarithms, powers and bounds by which a beam step orders its candidates, on the host against
fp64 and long double."""
import pytest

from tests import vocab_host

HEAD = r"""
#include <cstdio>
#include <random>
#include "beam_math.cuh"
using namespace lmloss;
"""

BOUNDS = HEAD + r"""
// every rank key lies within the fp32 bounds by which candidates are dropped
int main()
{
    std::mt19937_64 gen(1);
    std::uniform_real_distribution<double> u(0, 1);
    const double alphas[] = {0.1, 0.6, 1.0, 2.5, 7.0, 8.5, 9.0, 10.0, 10.5, 10.7, 11.0, 12.5, 30.0, 85.0, 100.0, 400.0};
    for (double alpha : alphas)
        for (int i = 0; i < 200000; ++i) {
            const int n = i < 100 ? i + 1 : static_cast<int>(std::exp(u(gen) * std::log(2e6)));
            const double base = -std::exp(u(gen) * 25 - 12);
            const float z = static_cast<float>(i % 3 == 0 ? -base : (u(gen) - 0.5) * std::exp(u(gen) * 12 - 6));
            const double d = power(n, alpha), rank = (base + static_cast<double>(z)) / d;
            float low, high;
            rank_bounds(static_cast<float>(base), z, 1.f / static_cast<float>(d), low, high);
            if (!(low <= rank && rank <= high)) {
                std::printf("alpha %g, length %d, base %.9g, logit %.9g: %.9g is not in [%.9g, %.9g]\n", alpha, n, base, z, rank, low, high);
                return 1;
            }
        }
    return 0;
}
"""


def test_rank_keys_lie_within_their_bounds(tmp_path):
    vocab_host.run(tmp_path, BOUNDS)
