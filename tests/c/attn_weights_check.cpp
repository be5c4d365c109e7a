// The attention kernels' scale factors (attn_weights.hpp) built for the host:
// for every scale a cache may hold, in any order, no operation is invalid (a
// NaN), the factors are finite, and a weight's factor and the sum's undo each
// other.  Prints the failures, "ok" if there are none.
#include <cfenv>
#include <cmath>
#include <cstdio>

#define __device__
#define __forceinline__ inline
#include "attn_weights.hpp"

using namespace qg;

int main()
{
    const float scales[] = {0.0f, 0x1p-100f, 1e-9f, 0.03f, 1.0f, 1e9f, 0x1p100f};
    const float factors[] = {0x1p-149f, 1e-30f, 0.18f, 1e10f, 3.4e38f};
    int bad = 0;
    std::feclearexcept(FE_ALL_EXCEPT);
    for (volatile float ks : scales)
        for (volatile float c2 : factors) {
            volatile float kc = score_factor(ks, c2), x = -INFINITY;
            x = x * kc;
            if (!(kc > 0 && std::isfinite(kc) && x == -INFINITY))
                ++bad, std::printf("score factor %g of %g, %g\n", kc, ks, c2);
        }
    // log2 R: between the least and the largest scale, and the lag of two maxima
    for (volatile float log2R = -109.0f; log2R <= 108.0f; log2R += 7.75f)
        for (volatile float s : scales) {
            volatile float h = held_scale(s), R = std::exp2(log2R);
            volatile float shift = run_shift(std::log2(h), log2R), back = run_back(R, 1.0f / h);
            if (!(h > 0 && std::isfinite(shift) && std::isfinite(back)))
                ++bad, std::printf("scale %g under %g: %g, %g\n", s, R, shift, back);
            volatile float both = back < 0x1p-126f ? 0.0f : shift + std::log2(back);
            if (!(std::fabs(both) < 1e-4f))
                ++bad, std::printf("scale %g under %g: factors give 2^%g\n", s, R, both);
        }
    if (std::fetestexcept(FE_INVALID))
        ++bad, std::printf("an invalid operation\n");
    if (!bad)
        std::printf("ok\n");
    return bad != 0;
}
