// The 8-bit key/value cache: what its writer (rope_cache.hip) and its readers (attn_kv8.hip)
// share.
//
// Pages of kPage tokens.  Keys: [page][kv head][token][D] bytes, values [page][kv head][D][token]
// bytes (dim-major: the 16 consecutive tokens of one dim that a lane of the P V product needs
// are then one 16-byte load), E4M3 codes (OCP: bias 7, largest 448, 0x7F and 0xFF NaN).  One
// FP32 scale per page and kv head for the keys and one for the values: value = code * scale.
// The writer's scales are powers of two (2^-126 for a page of zeros), so that a page whose scale grows
// is rescaled without rounding (but for codes that fall below E4M3's normal range).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace convrot {

constexpr int kPage = 64;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

// the ragged batch: queries of sequence b are rows cu[b] .. cu[b+1]-1; rows outside [0, T) or
// out of order count as none
struct Batch {
    const int32_t *cu;
    const int32_t *kv_lens;
    const int32_t *table;     // page ids [B, ld_table]
    int64_t ld_table;         // pages a sequence may have
    int64_t n_pages;
    int64_t T;
};

__host__ __device__ inline void batch_rows(const Batch &s, int b, int64_t &t0, int64_t &n)
{
    t0 = s.cu[b];
    const int64_t t1 = s.cu[b + 1];
    n = (t0 >= 0 && t1 >= t0 && t1 <= s.T) ? t1 - t0 : 0;
}

// tokens in the cache, never more than the table has pages for
__host__ __device__ inline int64_t batch_kv(const Batch &s, int b)
{
    const int64_t l = s.kv_lens[b], cap = s.ld_table * kPage;
    return l < 0 ? 0 : l < cap ? l : cap;
}

// id of page p of sequence b, or -1 where the table names no page of the cache
__host__ __device__ inline int64_t batch_page(const Batch &s, int b, int64_t p)
{
    if (p < 0 || p >= s.ld_table) return -1;
    const int64_t id = s.table[(int64_t)b * s.ld_table + p];
    return id >= 0 && id < s.n_pages ? id : -1;
}

// ---- the append's walk: a workgroup takes one page of one sequence ----

// pages that a run of max_new tokens may touch, wherever it starts in its first one
__host__ __device__ inline int64_t append_visits(int64_t max_new) { return (max_new + kPage - 2) / kPage + 1; }

// log2 of the tokens that a workgroup holds at a time: at least max_new, or a page
__host__ __device__ inline int append_log_tokens(int64_t max_new)
{
    int l = 0;
    while ((1 << l) < max_new && (1 << l) < kPage) l++;
    return l;
}

// the new tokens of a sequence that lie on the visit-th page of its run
struct PageRun {
    int64_t page;    // position / kPage
    int64_t row0;    // row of the first of them
    int nt, off0;    // how many, and where on the page they start
    bool stored;     // the cache is long enough to hold the run
};

// False where there are none.  Of a run longer than max_new the first max_new tokens count: the launch
// is sized for those, so nt never exceeds the tokens that a workgroup holds.
__host__ __device__ inline bool append_page_run(const Batch &s, int b, int max_new, int64_t visit, PageRun &r)
{
    int64_t t0, n;
    batch_rows(s, b, t0, n);
    const int64_t kv = s.kv_lens[b];
    r.stored = kv >= n;
    const int64_t first = kv >= n ? kv - n : 0;              // position of the first new token
    const int m = (int)n < max_new ? (int)n : max_new;      // rows are counted in 31 bits
    const int64_t end = first + m;
    r.page = first / kPage + visit;
    const int64_t lo = first > r.page * kPage ? first : r.page * kPage;
    const int64_t hi = end < (r.page + 1) * kPage ? end : (r.page + 1) * kPage;
    if (lo >= hi) return false;
    r.nt = (int)(hi - lo);
    r.off0 = (int)(lo - r.page * kPage);
    r.row0 = t0 + (lo - first);
    return true;
}

}  // namespace convrot
