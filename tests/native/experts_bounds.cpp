// The places and rows that the experts' product takes from device data, walked on the host for plans
// that hold anything: no place outside the order, no row outside its matrix.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "../../rotated_bit_linear_amd/csrc/experts.hpp"

using namespace convrot;

static void require(bool ok, const char *what)
{
    if (!ok) { std::printf("failed: %s\n", what); std::exit(1); }
}

int main()
{
    std::mt19937 rng(7);
    auto pick = [&](int lo, int hi) { return (int)(lo + (int64_t)(rng() % (uint32_t)((int64_t)hi - lo + 1))); };
    const int odd[] = {-2147483647 - 1, -1, 0, 1, 2147483647};
    int64_t walked = 0;
    for (int round = 0; round < 3000; round++) {
        const int E = pick(1, 70), S = pick(1, 300), lg = pick(4, 8), top_k = pick(1, 32);
        std::vector<int32_t> offsets(E + 1), rows(S);
        for (auto &o : offsets) o = rng() % 5 ? pick(-5, S + 5) : odd[rng() % 5];
        for (auto &r : rows) r = rng() % 5 ? pick(-3, S + 3) : odd[rng() % 5];
        if (round % 3 == 0) {                    // a plan as it should be
            for (auto &o : offsets) o = pick(0, S);
            for (int i = 1; i <= E; i++) offsets[i] = offsets[i] > offsets[i - 1] ? offsets[i] : offsets[i - 1];
        }
        ExpertsGemm g{};
        g.rows = rows.data(); g.S = S; g.M = pick(1, S); g.gather = pick(0, 1) * top_k; g.scatter = pick(0, 1);
        int64_t blocks = 0;
        for (int e = 0; e < E; e++) {
            const int lo = expert_offset(offsets.data(), e, S), hi = expert_offset(offsets.data(), e + 1, S);
            require(lo >= 0 && lo <= S && hi >= 0 && hi <= S, "offset");
            const int n = expert_blocks(lo, hi, lg);
            blocks += n;
            for (int b = 0; b < n; b++) {
                const int first = block_place(lo, b, lg);
                require(first >= lo && first < hi, "block");
                for (int i = first; i < first + (1 << lg) && i < hi; i++) {
                    const int named = named_row(g, i), from = row_from(g, i, named), to = row_to(g, i, named);
                    require(from >= -1 && from < g.M, "row of A");
                    require(to >= -1 && to < S, "row of C");
                    walked++;
                }
            }
        }
        if (round % 3 == 0) require(blocks <= most_blocks(S, E, lg), "more blocks than the launch has");
    }
    for (int round = 0; round < 300; round++) {  // every tile of an expert once, in range
        const int blocks = pick(1, 40), n_tiles = pick(1, 30), band = pick(1, 16);
        std::vector<int> seen(blocks * n_tiles);
        for (int i = 0; i < blocks * n_tiles; i++) {
            const TilePlace p = place_in_bands(i, blocks, n_tiles, band);
            require(p.block >= 0 && p.block < blocks && p.column >= 0 && p.column < n_tiles, "tile");
            require(seen[p.block * n_tiles + p.column]++ == 0, "tile twice");
        }
    }
    std::printf("ok %lld\n", (long long)walked);
    return 0;
}
