// Whether the layer's second product for one token takes its own form: never with more workgroups than a
// dispatch counts, at any number of choices, columns and row length that the layer takes.
#include <cstdio>
#include <cstdlib>

#include "../../rotated_bit_linear_amd/csrc/kernels.hpp"

using namespace convrot;

static void require(bool ok, const char *what, int64_t S, int64_t N, int64_t F)
{
    if (!ok) { std::printf("failed: %s at %lld choices, %lld columns, %lld long\n", what, (long long)S, (long long)N, (long long)F); std::exit(1); }
}

int main()
{
    int taken = 0;
    for (int64_t S = 1; S <= kMostChoices; S++)
        for (int lg = 0; lg <= 28; lg++)
            for (int64_t N = (1ll << lg) - 1; N <= (1ll << lg) + 1 && N <= 1ll << 28; N++)
                for (int64_t F = 256; F <= 8192; F += 256) {
                    if (N < 1) continue;
                    const int64_t threads = S * ((N + 127) / 128) * 256;     // a dispatch counts them in 32 bits
                    const bool fits = experts_row_fits(1, S, N, F);
                    require(!fits || threads <= 0xFFFFFFFFll, "more workgroups than a dispatch counts", S, N, F);
                    require(fits == (F <= 4096 && threads <= 0xFFFFFFFFll), "form", S, N, F);
                    require(!experts_row_fits(2, S, N, F), "two tokens", S, N, F);
                    taken += fits;
                }
    std::printf("ok %d\n", taken);
    return 0;
}
