// The append's walk over pages (kv8.hpp) on the host, with runs that are shorter, as long and
// longer than the bound the launch is sized by: every token below the bound is taken once, at its
// own place; no other token is; a workgroup never has more tokens of a page than it holds; and the
// 16-byte stores of a whole page happen only where one head is held at a time, so that every thread's
// store lies on that head's page.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "../../rotated_bit_linear_amd/csrc/kv8.hpp"

using namespace convrot;

int main()
{
    int bad = 0;
    const std::vector<int> sizes = {1, 2, 3, 4, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200};
    for (int max_new : sizes)
        for (int n : sizes)
            for (int past : {0, 1, 32, 63, 64, 65, 100})
                for (int short_by : {0, 1}) {                   // 1: a cache too short for the run
                    const int64_t kv = short_by ? n - 1 : past + n, first = short_by ? 0 : past;
                    const int32_t cu[2] = {3, (int32_t)(3 + n)}, lens[1] = {(int32_t)kv};
                    const Batch s{cu, lens, nullptr, 8, 8, 3 + n};
                    std::vector<int> taken(n, 0);
                    const int NT = 1 << append_log_tokens(max_new), HP = 64 / NT;
                    for (int64_t visit = 0; visit < append_visits(max_new); visit++) {
                        PageRun r;
                        if (!append_page_run(s, 0, max_new, visit, r)) continue;
                        bad += r.stored != (short_by == 0);
                        bad += r.nt < 1 || r.nt > NT || r.off0 < 0 || r.off0 + r.nt > kPage;
                        // teams of a workgroup: token `team % NT`, head slot `team / NT` of HP
                        for (int team = 0; team < 64; team++) {
                            const int tk = team % NT, slot = team / NT;
                            if (tk >= r.nt || slot != 0) continue;
                            const int64_t i = r.row0 + tk - 3;
                            bad += i < 0 || i >= n;
                            if (i < 0 || i >= n) continue;
                            taken[i]++;
                            bad += r.page * kPage + r.off0 + tk != first + i;
                        }
                        if (r.nt == kPage) bad += HP != 1;      // 64 teams: head slots 0 .. HP - 1 on this page's head
                    }
                    for (int64_t i = 0; i < n; i++) bad += taken[i] != (i < max_new ? 1 : 0);
                }
    std::printf(bad ? "%d wrong\n" : "ok %d\n", bad);
    return bad != 0;
}
