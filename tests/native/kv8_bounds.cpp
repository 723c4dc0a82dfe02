// The bounds that the cache kernels take from device data (kv8.hpp), on the host: whatever the
// batch's arrays hold, rows stay inside [0, T), lengths inside the page table and page ids
// inside the cache.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "../../rotated_bit_linear_amd/csrc/kv8.hpp"

using namespace convrot;

int main()
{
    const int32_t lo = -2147483647 - 1, hi = 2147483647;
    const std::vector<int32_t> bounds = {lo, -1, 0, 1, 5, 9, 10, 11, hi};
    const std::vector<int32_t> ids = {lo, -1, 0, 6, 7, hi};
    int bad = 0;
    for (int32_t a : bounds)
        for (int32_t b : bounds)
            for (int32_t kv : {lo, -1, 0, 1, 64, 191, 192, 193, hi})
                for (int32_t id : ids) {
                    const int32_t cu[2] = {a, b}, lens[1] = {kv}, table[3] = {id, id, id};
                    const Batch s{cu, lens, table, 3, 7, 10};
                    int64_t t0, n;
                    batch_rows(s, 0, t0, n);
                    const bool ok = a >= 0 && b >= a && b <= 10;
                    bad += n != (ok ? b - a : 0);
                    bad += n > 0 && (t0 < 0 || t0 + n > 10);
                    const int64_t l = batch_kv(s, 0);
                    bad += l < 0 || l > 192 || (kv >= 0 && kv <= 192 && l != kv);
                    for (int64_t p = -1; p <= 3; p++) {
                        const int64_t got = batch_page(s, 0, p);
                        bad += got != ((p >= 0 && p < 3 && id >= 0 && id < 7) ? id : -1);
                    }
                }
    std::printf(bad ? "%d wrong\n" : "ok %d\n", bad);
    return bad != 0;
}
