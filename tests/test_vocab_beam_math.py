"""The logarithms, powers and bounds by which a beam step orders its candidates, on the host against
fp64 and long double."""
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


ERRORS = HEAD + r"""
// largest error of the logarithm, then for each exponent largest relative error of the power
int main()
{
    std::mt19937_64 gen(2);
    std::uniform_real_distribution<double> u(0, 1);
    double worst = 0;
    for (int i = 0; i < 3000000; ++i) {
        const float hi = i < 100000 ? 1 + i * 1e-5f : static_cast<float>(std::exp(u(gen) * 22));
        const float lo = static_cast<float>(hi * (u(gen) - 0.5) * 1.1920929e-7);
        worst = std::max(worst, static_cast<double>(std::fabs(log_of_sum(hi, lo) - std::log(static_cast<long double>(hi) + lo))));
    }
    std::printf("0 %g\n", worst);
    for (double a : {0.01, 0.1, 0.3, 0.6, 0.9, 1.0, 1.5, 2.0, 2.5, 5.0, 10.0, 16.0, 40.0, 50.0, 60.0}) {
        double w = 0;
        for (int i = 1; i < 200000; ++i) {
            const int n = i < 100000 ? i : 100000 + static_cast<int>(u(gen) * 2147383647.0);
            const long double exact = std::pow(static_cast<long double>(n), static_cast<long double>(a));
            if (exact < 1.7e308L) w = std::max(w, static_cast<double>(std::fabs(power(n, a) / exact - 1)));
        }
        std::printf("%g %g\n", a, w);
    }
    return 0;
}
"""


def test_logarithm_and_power_are_as_close_as_they_say(tmp_path):
    # what beam_math.cuh states: 3e-9, and of itself 3e-9 (1 + exponent)
    for line in vocab_host.run(tmp_path, ERRORS):
        a, error = map(float, line.split())
        assert error <= 3e-9 * (1 + a), line
