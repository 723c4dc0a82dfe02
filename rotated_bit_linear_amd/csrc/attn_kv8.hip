// Attention over the 8-bit paged cache (layout and scales: kv8.hpp).
//   O[r] = sum_j p[r, j] V[j] / sum_j p[r, j],  p[r, j] = exp(sm_scale Q[r] . K[j])
// over the keys j that row r sees: j < kv_len, and with `causal` j <= kv_len - n + i for token
// i of its sequence's n.  Rows are (token, query head of the group) pairs of one key/value
// head, so a group shares every key and value that is read.  A row that sees no key gives 0.
//
// Both kernels compute S^T = K Q^T and O^T = V^T P^T on the matrix cores.  A lane then holds
// one query row (a column of S^T) with several keys in its registers: the softmax statistics
// are in-lane operations and one exchange between the lanes of a column, and the lane's own
// P values are, packed to 16 bits, its operand of the second product with no data movement:
// the contraction may take keys in any order, so V^T is presented in the order in which S^T
// leaves them.
// Precision: codes are exact in bf16 and fp16, products accumulate in FP32, maximum and sum
// are FP32.  P is rounded to fp16 whatever the queries' type (half a step is at most 2^-11 of
// p, and 2^-25 below 2^-14; the second product takes the codes as fp16): in bf16, half a
// step is 2^-8, and a row that one key dominates would be off by that twice.
// Scales: a page's key scale joins the factor of the exponent's argument, its value scale vs
// the exponent: P holds p * vs / 2^at, and a row's accumulators sums of p v / 2^at.  `at` follows the
// smallest scale so far (2^at <= vs, so P is at least p and loses no more bits than p would);
// it rises where a row's own P would leave fp16 (2^14), and stays where the row's accumulators would
// pass 2^100, beside which the page does not count.  It is a power of two, so that moving it
// rounds nothing, and each row has its own: what one row weighs takes no bits from another.
// The running maximum is only raised when some row's scores exceed it by 8 (in log2): until
// then p is at most 2^8, which FP32 sums and fp16 hold without loss, and the accumulators need
// no rescaling.
// Masked places: scores are selected, not added to, so NaN or infinite codes of keys that a
// row does not see leave it alone; values beyond kv_len are zeroed.  On a page that every row of the
// tile sees whole, a NaN code goes through the product into its element.  On any other page NaN
// codes are zeroed before the product, and where there were some, such pages are read again at the
// end and the elements of the rows that see them set to NaN.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kernels.hpp"
#include "kv8.hpp"

namespace convrot {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct AttnArgs {
    const uint16_t *q;
    uint16_t *out;
    int64_t ld_q, ld_out;
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
    Batch batch;
    int B, Hq, Hkv, G;       // G = Hq / Hkv
    int row_blocks;          // blocks of query rows a sequence and key/value head
    int whole, tail, splits; // blocks done by one workgroup each, then blocks split into runs of pages
    int64_t pages_per_split;
    float factor;            // sm_scale * log2(e)
    int causal;
    float *part_o;           // of the split blocks' rows [split][part_rows][D]: a run's own result
    float2 *part_ml;         // [split][part_rows] (its maximum, its sum of p)
    int64_t part_rows;       // rows of the split blocks, or of the whole batch (by_token)
    int by_token;            // a row's part lies at its token and head, not at its place in the block
};

// 16-bit operand types: bf16 (0) or fp16 (1)
template <int DT> struct Half;
template <> struct Half<0> {
    using V8 = bf16x8;
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        bf16x2 r;
        r[0] = (__bf16)a;
        r[1] = (__bf16)b;
        return __builtin_bit_cast(uint32_t, r);
    }
    template <bool HI> static __device__ __forceinline__ uint32_t widen(uint32_t w)
    {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
    }
    static __device__ __forceinline__ f32x16 mfma32(u32x4v a, u32x4v b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(V8, a), __builtin_bit_cast(V8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x4 mfma16(u32x4v a, u32x4v b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(V8, a), __builtin_bit_cast(V8, b), c, 0, 0, 0);
    }
};
template <> struct Half<1> {
    using V8 = f16x8;
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        f16x2 r;
        r[0] = (_Float16)a;
        r[1] = (_Float16)b;
        return __builtin_bit_cast(uint32_t, r);
    }
    template <bool HI> static __device__ __forceinline__ uint32_t widen(uint32_t w)
    {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
    }
    static __device__ __forceinline__ f32x16 mfma32(u32x4v a, u32x4v b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(V8, a), __builtin_bit_cast(V8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x4 mfma16(u32x4v a, u32x4v b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(V8, a), __builtin_bit_cast(V8, b), c, 0, 0, 0);
    }
};

// 8 codes (two words) to 8 16-bit values
template <int DT>
__device__ __forceinline__ u32x4v widen8(uint32_t lo, uint32_t hi)
{
    return u32x4v{Half<DT>::template widen<false>(lo), Half<DT>::template widen<true>(lo),
                  Half<DT>::template widen<false>(hi), Half<DT>::template widen<true>(hi)};
}

// 0x80 in each byte that holds a NaN code
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// 0xFF in those bytes
__device__ __forceinline__ uint32_t spread_bytes(uint32_t b) { return (b << 1) - (b >> 7); }
// the bytes of a word that hold tokens below `left` (word w of a run of tokens)
__device__ __forceinline__ uint32_t below_bytes(int left)
{
    return left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
}

// whether the first `left` tokens of one dim (64 codes) hold a NaN code
__device__ __forceinline__ bool nan_among(const uint8_t *codes, int left)
{
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < kPage / 16; i++) {
        const u32x4v c = *reinterpret_cast<const u32x4v *>(codes + 16 * i);
#pragma unroll
        for (int w = 0; w < 4; w++) bad |= nan_bytes(c[w] & below_bytes(left - 16 * i - 4 * w));
    }
    return bad != 0;
}

// the larger of the two lanes l and l ^ 32, in both
__device__ __forceinline__ float both_halves_max(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// a value the compiler cannot derive from earlier ones: what follows from it is computed where
// it is needed instead of staying in registers over the main loop
__device__ __forceinline__ int opaque_lane(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// pins the computation of v to this place (the compiler would sink it out of the products' shadow)
__device__ __forceinline__ void stay(float &v) { asm volatile("" : "+v"(v)); }

// waits for all of this wave's LDS operations
__device__ __forceinline__ void lds_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// a barrier that waits for this wave's LDS operations but the last `younger` (its operand reads)
template <int younger>
__device__ __forceinline__ void barrier_but()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(%0)" ::"n"(younger) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// 16 codes at a uniform address, kept in scalar registers, and a lane's 32-bit offset
typedef const __attribute__((address_space(1))) uint8_t *global_u8;
typedef const __attribute__((address_space(1))) u32x4v *global_u32x4;
__device__ __forceinline__ u32x4v load_codes(const uint8_t *base, uint32_t off)
{
    global_u8 p = (global_u8)base;
    asm volatile("" : "+s"(p));
    return *(global_u32x4)(p + off);
}

// what a kernel only reads, at uniform addresses: scalar loads, whatever it stores elsewhere
typedef const __attribute__((address_space(4))) int32_t *scalar_i32;
typedef const __attribute__((address_space(4))) float *scalar_f32;

constexpr float kLow = -3.4028235e38f;   // running maximum before the first key: below no finite score
constexpr float kSlack = 8.0f;    // log2: how far scores may exceed the running maximum
constexpr float kMostP = 14.0f;   // log2 of the largest P

// the factor of a page's scores: above zero, so that a masked score stays minus infinity
__device__ __forceinline__ float score_factor(float factor, float ks) { return fmaxf(factor * ks, 0x1p-149f); }

// A row's reference for the values: its accumulators hold sums of p v / 2^at.  The lanes of a row hold
// the same; where all rows of the wave do, a page is compared with it by one scalar.
struct ValueRef {
    int at = 128;                 // above any scale: the first page's is taken
    int common = kNone;           // `at` of every lane, or kNone
    int exp = 128;                // the current page's scale: 2^(exp + frac), 0 <= frac < 1 (uniform)
    float frac = 0.0f;
    float shift = 0.0f;           // log2 of its ratio to 2^at, joins the exponents
    float weight = 1.0f;          // what turns the page's sum of P into a sum of p
    static constexpr int kNone = 1 << 20;
    __device__ __forceinline__ void page(float vs)
    {
        vs = fmaxf(vs, 0x1p-149f);
        exp = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_frexp_expf(vs) - 1);
        frac = __builtin_amdgcn_logf(2.0f * __builtin_amdgcn_frexp_mantf(vs));
        aim();
    }
    __device__ __forceinline__ void aim()
    {
        // below -64 P is zero in any case, and its FP32 sum still holds p
        shift = fmaxf(frac + (float)(exp - at), -64.0f);
        weight = __builtin_amdgcn_exp2f(-shift);
    }
    // false: for every row 2^at is at most the page's scale, and P stays below 2^kMostP
    __device__ __forceinline__ bool stray() const { return (uint32_t)(exp - common) >= (uint32_t)(kMostP - kSlack); }
    // whether a row's scores (at most `over` above its maximum) ask for another `at`
    __device__ __forceinline__ bool off(float over) const { return exp < at || over + shift > kMostP; }
    // moves `at` down to the page's scale, as far as accumulators of magnitude `top` allow, or up to
    // it where its largest P would exceed 2^kMostP; returns by how many powers of two they grow
    __device__ __forceinline__ int move(float top, float over)
    {
        const int room = top > 0.0f ? max(100 - __builtin_amdgcn_frexp_expf(top), 0) : 1024;
        const int from = at;
        if (exp < at) at = max(exp, at - room);
        else if (over + shift > kMostP) at = exp;
        const int first = __builtin_amdgcn_readfirstlane(at);
        common = __builtin_amdgcn_ballot_w64(at != first) == 0 ? first : kNone;
        aim();
        return from - at;
    }
};

// per-sequence facts of a workgroup (the launch's limits keep n * G and the keys within an int)
struct Seq {
    int64_t t0;
    int n, kv, rows;
};
__device__ __forceinline__ Seq load_seq(const AttnArgs &a, int b)
{
    Seq s;
    int64_t n;
    batch_rows(a.batch, b, s.t0, n);
    s.n = (int)n;
    s.kv = (int)batch_kv(a.batch, b);
    s.rows = s.n * a.G;
    return s;
}
// what a workgroup does: block `block` of the rows of sequence b and key/value head hk; the whole
// cache (split < 0), or its run `split` (part: which of the split blocks it is)
struct Task {
    int b, hk, block, split, part;
};
// The longest rows (causal) come first.  Workgroups go to the eight XCDs in turn, and a sequence's
// key/value head stays on one of them where there are eight heads or a multiple: its keys and
// values are then read into one L2, and every XCD has its share of each sequence.  With other
// numbers of heads sequences of different lengths would load the XCDs unevenly, so there the
// units move on by one each row of whole blocks (4 ragged prompts of up to 2000 tokens, 16 query and 2
// key/value heads of 64: 66 us without, 47 with).
__device__ __forceinline__ Task task_of(const AttnArgs &a, int id)
{
    Task t;
    t.split = -1;
    t.part = 0;
    int w = id;
    if (id >= a.whole) {
        const int i = id - a.whole;
        t.split = i / a.tail;
        t.part = i % a.tail;
        w = a.whole + t.part;
    }
    const int units = a.B * a.Hkv, row = w / units;
    int unit = w % units;
    if (a.B > 1 && a.Hkv % 8 != 0 && (row + 1) * units <= a.whole) unit = (unit + row) % units;
    t.block = a.row_blocks - 1 - row;
    t.b = unit / a.Hkv;
    t.hk = unit % a.Hkv;
    return t;
}

// where the result of a run for row r (r0 the block's first, `per` its rows) goes
__device__ __forceinline__ int64_t part_of(const AttnArgs &a, const Task &t, const Seq &s, int r, int r0, int per)
{
    const int tok = r / a.G;
    const int64_t at = a.by_token ? (s.t0 + tok) * a.Hq + t.hk * a.G + (r - tok * a.G) : (int64_t)t.part * per + (r - r0);
    return t.split * a.part_rows + at;
}

// the sequence that token t belongs to, or -1: of those that begin at or before it the last,
// sought by 64 lanes at once; where the bounds are not in order, one after the other
__device__ __forceinline__ int sequence_of(const AttnArgs &a, int64_t t, int lane)
{
    auto holds = [&](int b) __attribute__((always_inline)) {
        int64_t t0, n;
        batch_rows(a.batch, b, t0, n);
        return t >= t0 && t < t0 + n;
    };
    int lo = 0, n = a.B;
    while (n > 1) {
        const int step = (n + 63) / 64;
        const bool begun = lane * step < n && a.batch.cu[lo + lane * step] <= t;
        const int k = max(__popcll(__builtin_amdgcn_ballot_w64(begun)) - 1, 0);
        lo += k * step;
        n = min(step, n - k * step);
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    if (holds(lo)) return lo;
    for (int b = 0; b < a.B; b += 64) {
        const uint64_t found = __builtin_amdgcn_ballot_w64(b + lane < a.B && holds(b + lane));
        if (found) return b + __builtin_ctzll(found);
    }
    return -1;
}

// number of keys that token i of the sequence sees
__device__ __forceinline__ int visible(const AttnArgs &a, const Seq &s, int i)
{
    return a.causal ? max(s.kv - s.n + i + 1, 0) : s.kv;
}

}  // namespace

// ------------------------------------------------------------------ prompts: many rows ----
// One workgroup: 32 query rows in each of 4 waves over a run of pages.  A page is
// read once into registers, widened to 16 bits, and written to one of two LDS tiles in the
// order in which the matrix operands want it; rows are padded by 16 bytes so that the 16
// lanes of a read cover all banks.
// Software pipeline over halves of a page (32 keys): a step issues the score products of the
// next half, the softmax of this one under them, this half's second products, and under
// those the writes of half a page to come into LDS; one barrier a step.  That half page's codes
// are converted in front of the first product, with the wait for their loads: waves that only
// stage share the conversions, and the compiler moves them above the branch.
// 32 rows a wave: with 64 a wave reads its operands half as often, but needs 512 registers, and
// one wave a SIMD has nothing to issue under its products (3.7 ms against 2.85 below).
// Measured: 19989 tokens on 19989, 14 heads of 128, bf16: 2.81 to 3.00 ms on different boxes, 950 to
// 1020 TFLOP/s (a library product of 8192^3 bf16: 1434); causal prompts of up to 4096 tokens, 32
// and 8 heads: 381 to 416 us, 870 to 950; three sequences of up to 515 new tokens over 10515, 12
// heads of 64, fp16: 55 us and 9 for the join, bound by the vector units (the softmax of a score
// costs the same for half the products).  Counters of the first: matrix cores busy 50 % of the
// cycles, vector units 50 (an exponential takes two slots), LDS 44 and 6 in bank conflicts: the two
// units' work follows more than it overlaps.  A wave issues 49 % of its time, waits 31 for a busy
// unit and 20 for data and at barriers.
constexpr int kWaves = 4, kRowsBlock = 32 * kWaves;

template <int DT, int D>
__global__ __launch_bounds__(256, D == 64 ? 3 : 2) void attn_rows_kernel(AttnArgs a)
{
    constexpr int KROW = 2 * D + 16, VROW = 2 * kPage + 16;   // bytes of a widened row of keys, of values
    constexpr int KQ = D / 64, VQ = D / 64;             // 16-byte code loads a thread and tile
    constexpr int ROWS = kRowsBlock;
    __shared__ __attribute__((aligned(16))) uint8_t ldsK[2][kPage * KROW];
    __shared__ __attribute__((aligned(16))) uint8_t ldsV[2][D * VROW];
    __shared__ uint32_t nan_codes;                      // NaN codes were cleared from a page

    const Task task = task_of(a, blockIdx.x);
    const int b = task.b, hk = task.hk;
    const Seq s = load_seq(a, b);
    const int r0 = task.block * ROWS;
    if (r0 >= s.rows) return;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;

    // keys seen by this lane's rows, by the block's last row (the loop's end) and by all of its rows
    const int last = min(r0 + ROWS, s.rows) - 1;
    const int lim_all = visible(a, s, r0 / a.G);
    const int pages = (visible(a, s, last / a.G) + kPage - 1) / kPage;
    const int p0 = task.split < 0 ? 0 : (int)(task.split * a.pages_per_split);
    const int p1 = task.split < 0 || task.split + 1 == a.splits ? pages : (int)min((int64_t)pages, p0 + a.pages_per_split);
    if (task.split >= 0 && p0 >= p1) return;               // no row of the block looks here

    const bool busy = r0 + wave * 32 < s.rows;     // a wave without rows only stages
    int lim;
    u32x4v q[D / 16];
    {
        // rows past the last repeat it and are not stored
        const int r = min(r0 + wave * 32 + col, s.rows - 1), i_tok = r / a.G;
        lim = visible(a, s, i_tok);
#pragma unroll
        for (int k = 0; k < D / 16; k++)
            q[k] = *reinterpret_cast<const u32x4v *>(a.q + (s.t0 + i_tok) * a.ld_q + (hk * a.G + (r - i_tok * a.G)) * D +
                                                     16 * k + 8 * half);
    }

    // ---- staging: codes of a page in registers, then widened in LDS ----
    // where the table names no page, page 0 is read and nobody sees its keys
    auto page_of = [&](int32_t id, bool &ok) __attribute__((always_inline)) {
        id = __builtin_amdgcn_readfirstlane(id);
        ok = id >= 0 && id < a.batch.n_pages;
        return (int64_t)(ok ? id : 0) * a.Hkv + hk;
    };
    // entry of page p in the table (p below the length, hence inside the table)
    const int32_t *table = a.batch.table + (int64_t)b * a.batch.ld_table;
    const int k_row = tid >> 2, k_off = (tid & 3) * (D / 4);
    auto load_k = [&](int64_t at, u32x4v (&r)[KQ]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < KQ; i++)
            r[i] = load_codes(a.k + at * (kPage * D), k_row * D + k_off + 16 * i);
    };
    auto load_v = [&](int64_t at, u32x4v (&r)[VQ]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < VQ; i++)
            r[i] = load_codes(a.v + at * (kPage * D), 16 * (tid + 256 * i));
    };
    // the i-th of the 2 KQ 16-byte chunks that a thread widens of a tile
    auto store_k = [&](const u32x4v (&r)[KQ], int buf, int i) __attribute__((always_inline)) {
        *reinterpret_cast<u32x4v *>(ldsK[buf] + k_row * KROW + 2 * k_off + 16 * i) =
            widen8<DT>(r[i >> 1][2 * (i & 1)], r[i >> 1][2 * (i & 1) + 1]);
    };
    auto store_v = [&](const u32x4v (&r)[VQ], int buf, int i) __attribute__((always_inline)) {
        // 16 tokens of one dim: words 0, 2 for lanes 0-31, then 1, 3 for lanes 32-63
        *reinterpret_cast<u32x4v *>(ldsV[buf] + ((tid >> 2) + 64 * (i >> 1)) * VROW + 32 * (tid & 3) + 16 * (i & 1)) =
            widen8<1>(r[i >> 1][i & 1], r[i >> 1][2 + (i & 1)]);
    };
    // values of a page that some row does not see whole: nothing beyond the cache, no NaN codes
    auto clean_v = [&](u32x4v (&r)[VQ], int p) __attribute__((always_inline)) {
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < VQ; i++) {
            const int left = s.kv - p * kPage - 16 * (tid & 3);
#pragma unroll
            for (int w = 0; w < 4; w++) {
                const uint32_t x = r[i][w] & below_bytes(left - 4 * w);
                const uint32_t bad = nan_bytes(x);
                any |= bad;
                r[i][w] = x & ~spread_bytes(bad);
            }
        }
        if (any) nan_codes = 1;
    };

    // ---- the parts of a page ----
    f32x16 o[D / 32];
#pragma unroll
    for (int d = 0; d < D / 32; d++)
#pragma unroll
        for (int e = 0; e < 16; e++) o[d][e] = 0.0f;
    float m = kLow, l = 0.0f, mx = 0.0f;
    ValueRef ref;
    // operand i of the score products with 32 keys (half kb of a tile), of the second products
    const int lane_k = col * KROW + 16 * half, lane_v = col * VROW + 16 * half;
    auto read_k = [&](int buf, int kb, int i) __attribute__((always_inline)) {
        return *reinterpret_cast<const u32x4v *>(ldsK[buf] + lane_k + 32 * kb * KROW + 32 * i);
    };
    auto read_v = [&](int buf, int kb, int i) __attribute__((always_inline)) {
        const int j = i / (D / 32), d = i % (D / 32);
        return *reinterpret_cast<const u32x4v *>(ldsV[buf] + lane_v + 32 * d * VROW + 32 * (2 * kb + j));
    };
    auto mask = [&](f32x16 &x, int p, int kb, bool ok) __attribute__((always_inline)) {
        const int left = (ok ? lim - p * kPage : 0) - 32 * kb - 4 * half;
#pragma unroll
        for (int e = 0; e < 16; e++) x[e] = 8 * (e >> 2) + (e & 3) < left ? x[e] : -__builtin_inff();
    };
    float top;                                          // largest score of the half page so far
    auto max_of = [&](const f32x16 &x, int e0, int e1) __attribute__((always_inline)) {
#pragma unroll
        for (int e = e0; e < e1; e++) top = e == 0 ? x[0] : fmaxf(top, x[e]);
        stay(top);
    };
    // the maximum of the scores about to be added, and the reference of their values: rescales
    // what is there where they move (rare)
    auto raise = [&]() __attribute__((always_inline)) {
        if (__builtin_expect(__builtin_amdgcn_ballot_w64(mx > m + kSlack) != 0, 0)) {
            const float m1 = fmaxf(m, mx), f = __builtin_amdgcn_exp2f(m - m1);
            m = m1;
            l *= f;
#pragma unroll
            for (int d = 0; d < D / 32; d++)
#pragma unroll
                for (int e = 0; e < 16; e++) o[d][e] *= f;
        }
        if (__builtin_expect(ref.stray(), 0)) {
            if (__builtin_amdgcn_ballot_w64(ref.off(mx - m)) != 0) {
                float most = 0.0f;
#pragma unroll
                for (int d = 0; d < D / 32; d++)
#pragma unroll
                    for (int e = 0; e < 16; e++) most = fmaxf(most, fabsf(o[d][e]));
                const int by = ref.move(both_halves_max(most), mx - m);
#pragma unroll
                for (int d = 0; d < D / 32; d++)
#pragma unroll
                    for (int e = 0; e < 16; e++) o[d][e] = __builtin_amdgcn_ldexpf(o[d][e], by);
            }
        }
    };
    u32x4v pk[2];
    float sum;
    auto softmax = [&](const f32x16 &x, float c, int e0, int e1) __attribute__((always_inline)) {
#pragma unroll
        for (int e = e0; e < e1; e += 2) {
            const float y = __builtin_amdgcn_exp2f(fmaf(x[e], c, ref.shift - m));
            const float z = __builtin_amdgcn_exp2f(fmaf(x[e + 1], c, ref.shift - m));
            sum = e == 0 ? y + z : sum + (y + z);
            pk[e >> 3][(e >> 1) & 3] = Half<1>::pack(y, z);
        }
        stay(sum);
    };
    // A step: softmax of x (half kb of page p, tile bv of the values) and its second products;
    // scores of the next half into y (half kb ^ 1 of tile bk of the keys); one tile's widening
    // in quarters by `widen`; the first operands of the step after it (half kb of tile bk1).
    // Written out in the order of issue: per matrix product the operand AHEAD of it is
    // read, and as much vector work follows as the product takes.
    constexpr int NQ = D / 16, NV = D / 16, AHEAD = D == 64 ? 3 : 4, RING = D == 64 ? 4 : 8;
    // what the barrier after a step may leave outstanding: operand reads for the next step, but no more
    // than follow the step's last staging write (its widening ends half way through the second products)
    constexpr int LEFT = AHEAD < NV / 2 ? AHEAD : NV / 2;
    static_assert(LEFT <= NV - NV / 2 && LEFT <= AHEAD, "a staging write must not be left outstanding");
    u32x4v f[RING];
    auto step = [&](int kb, const f32x16 &x, f32x16 &y, float c, int bk, int bv, int bk1,
                    auto widen) __attribute__((always_inline)) {
        if (!busy) {                                    // uniform in the wave
#pragma unroll
            for (int i = 0; i < NV / 2; i++) widen(i);
            lds_done();                                 // no operand reads follow that the barrier may leave out
            return;
        }
        __builtin_amdgcn_s_setprio(1);                  // a wave at its products before one at its scales and barriers
#pragma unroll
        for (int t = 0; t < NQ + NV; t++) {
            const int u = t + AHEAD;
            f[u % RING] = u < NQ ? read_k(bk, kb ^ 1, u) : u < NQ + NV ? read_v(bv, kb, u - NQ) : read_k(bk1, kb, u - NQ - NV);
            if (t < NQ) {
                if (t == 0)
#pragma unroll
                    for (int e = 0; e < 16; e++) y[e] = 0.0f;
                y = Half<DT>::mfma32(f[t % RING], q[t], y);
                softmax(x, c, t * (16 / NQ), (t + 1) * (16 / NQ));
            } else {
                const int i = t - NQ;
                o[i % (D / 32)] = Half<1>::mfma32(f[t % RING], pk[i / (D / 32)], o[i % (D / 32)]);
                if (i < NV / 2) widen(i);
                else max_of(y, (i - NV / 2) * (32 / NV), (i - NV / 2 + 1) * (32 / NV));
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_setprio(0);
        l = fmaf(sum, ref.weight, l);
    };

    if (tid == 0) nan_codes = 0;
    __syncthreads();
    if (p0 < p1) {
        u32x4v kr[KQ], vr[VQ];
        auto masked = [&](int p, bool ok) __attribute__((always_inline)) { return (p + 1) * kPage > lim_all || !ok; };
        const int pl = p1 - 1;                          // the last page stands in where there is none (never used)
        // pages p, p + 1, p + 2: where they are, and the scales of the first two
        bool ok, ok1, ok2;
        int64_t at = page_of(table[p0], ok), at1 = page_of(table[min(p0 + 1, pl)], ok1);
        int64_t at2 = page_of(table[min(p0 + 2, pl)], ok2);
        int32_t id3 = table[min(p0 + 3, pl)];
        float c = score_factor(a.factor, a.k_scale[at]);
        // page 0 stands in for a page that is not there: its scale is not this sequence's
        if (ok) ref.page(a.v_scale[at]);
        float ks1 = a.k_scale[at1], vs1 = a.v_scale[at1];
        f32x16 sa, sb;
        {
            u32x4v k0[KQ], v0[VQ], k1[KQ];              // all in flight together
            load_k(at, k0);
            load_v(at, v0);
            load_k(at1, k1);
            load_v(at1, vr);
            if (masked(p0, ok)) clean_v(v0, p0);
#pragma unroll
            for (int i = 0; i < 2 * KQ; i++) {
                store_k(k0, 0, i);
                store_v(v0, 0, i);
                store_k(k1, 1, i);
            }
        }
        load_k(at2, kr);
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 16; e++) sa[e] = 0.0f;
#pragma unroll
        for (int t = 0; t < NQ; t++) sa = Half<DT>::mfma32(read_k(0, 0, t), q[t], sa);
        if (masked(p0, ok)) mask(sa, p0, 0, ok);
        max_of(sa, 0, 16);
        mx = both_halves_max(top) * c;
#pragma unroll
        for (int t = 0; t < AHEAD; t++) f[t] = read_k(0, 1, t);
        for (int p = p0; p < pl; p++) {
            const int cur = (p - p0) & 1, nxt = cur ^ 1;
            // ---- keys 0..31 of page p; the scores of its keys 32..63; values p + 1 staged ----
            raise();
            if (masked(p + 1, ok1)) {
                clean_v(vr, p + 1);
                lds_done();                             // its note is written
            }
            barrier_but<LEFT>();                        // values p are staged; values p - 1 are read
            step(0, sa, sb, c, cur, cur, nxt, [&](int i) __attribute__((always_inline)) { store_v(vr, nxt, i); });
            load_v(at2, vr);
            if (masked(p, ok)) {
                mask(sb, p, 1, ok);
                max_of(sb, 0, 16);
            }
            mx = both_halves_max(top) * c;
            raise();
            barrier_but<LEFT>();                        // keys p + 1 are staged; keys p are read
            // ---- keys 32..63; the scores of keys 0..31 of page p + 1; keys p + 2 staged ----
            step(1, sb, sa, c, nxt, cur, nxt, [&](int i) __attribute__((always_inline)) { store_k(kr, cur, i); });
            ok = ok1;
            c = score_factor(a.factor, ks1);
            if (ok) ref.page(vs1);
            if (masked(p + 1, ok)) {
                mask(sa, p + 1, 0, ok);
                max_of(sa, 0, 16);
            }
            mx = both_halves_max(top) * c;
            ks1 = a.k_scale[at2];
            vs1 = a.v_scale[at2];
            ok1 = ok2;
            at2 = page_of(id3, ok2);
            id3 = table[min(p + 4, pl)];
            load_k(at2, kr);
        }
        // ---- the last page ----
        const int cur = (pl - p0) & 1;
        raise();
        __syncthreads();
        step(0, sa, sb, c, cur, cur, cur, [](int) {});
        if (masked(pl, ok)) {
            mask(sb, pl, 1, ok);
            max_of(sb, 0, 16);
        }
        mx = both_halves_max(top) * c;
        raise();
        softmax(sb, c, 0, 16);
        l = fmaf(sum, ref.weight, l);
#pragma unroll
        for (int i = 0; i < NV; i++)
            o[i % (D / 32)] = Half<1>::mfma32(read_v(cur, 1, i), pk[i / (D / 32)], o[i % (D / 32)]);
        if (__builtin_expect(nan_codes != 0, 0)) {      // uniform; the notes lie before the last barrier
            uint64_t hit = 0;                           // bit 16 d + e: element e of o[d]
            for (int pg = max(p0, lim_all / kPage); pg < p1; pg++) {
                bool there;
                const int64_t page = page_of(table[pg], there);
                if (!there) continue;
                const int left = lim - pg * kPage;
                for (int i = 0; i < D / 2; i++) {
                    const int dim = 32 * (i >> 4) + 8 * ((i >> 2) & 3) + 4 * half + (i & 3);
                    if (nan_among(a.v + (page * D + dim) * kPage, left)) hit |= (uint64_t)1 << i;
                }
            }
#pragma unroll
            for (int d = 0; d < D / 32; d++)
#pragma unroll
                for (int e = 0; e < 16; e++) o[d][e] = (hit >> (16 * d + e)) & 1 ? __builtin_nanf("") : o[d][e];
        }
    }

    // ---- the lane's row (found again rather than kept): dims 32 d + 8 g + 4 half + 0..3 ----
    const float total = l + __shfl_xor(l, 32);
    const int r = r0 + opaque_lane(wave * 32 + col);
    if (r >= s.rows) return;
    // the average first, then its power of two: sums of p v may pass FP32 where their average does not
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    auto value = [&](float x) __attribute__((always_inline)) { return __builtin_amdgcn_ldexpf(x * inv, ref.at); };
    if (task.split >= 0) {
        const int64_t at = part_of(a, task, s, r, r0, ROWS);
        float *po = a.part_o + at * D;
#pragma unroll
        for (int d = 0; d < D / 32; d++)
#pragma unroll
            for (int g = 0; g < 4; g++)
                *reinterpret_cast<f32x4 *>(po + 32 * d + 8 * g + 4 * half) =
                    f32x4{value(o[d][4 * g]), value(o[d][4 * g + 1]), value(o[d][4 * g + 2]), value(o[d][4 * g + 3])};
        if (half == 0) a.part_ml[at] = float2{m, total};
        return;
    }
    uint16_t *po = a.out + (s.t0 + r / a.G) * a.ld_out + (hk * a.G + r % a.G) * D;
#pragma unroll
    for (int d = 0; d < D / 32; d++)
#pragma unroll
        for (int g = 0; g < 4; g++)
            *reinterpret_cast<u32x2v *>(po + 32 * d + 8 * g + 4 * half) =
                u32x2v{Half<DT>::pack(value(o[d][4 * g]), value(o[d][4 * g + 1])),
                       Half<DT>::pack(value(o[d][4 * g + 2]), value(o[d][4 * g + 3]))};
}

// ------------------------------------------------------------- single tokens: few rows ----
// Up to 16 query rows of a key/value head are one operand of the 16 x 16 matrix instructions;
// the cache is the other, read straight from memory into registers in operand order (no LDS,
// every code read once): the rows of a 16-key block of S^T may be any keys, so block kb takes
// keys 16 a + 4 kb + r in rows 4 a + r, which leaves each lane with the 16 consecutive keys
// 16 (lane / 16) ..; the 16 bytes of V^T at those keys are the lane's operands of two P V
// steps.  Likewise each 16-byte load of K covers two steps of the contraction over D.
// The four waves of a workgroup take the pages of its run in turn and join through LDS; runs
// of one row are joined by attn_join_kernel.
// Bound by the cache's bytes: twelve waves a compute unit keep a whole page each in flight, the
// page after it asked for by an id that is there already.  Values are read once by whole cache
// lines, past the caches; a load of K takes halves of lines (D = 128), whose other halves
// non-temporal loads would fetch again: 384 us, with both so 405, with neither 413.
// Measured, 32 query and 8 key/value heads of 128: 64 sequences of 32768 tokens 653 us (6.6 TB/s),
// of up to 32768 tokens 382 us (6.0); one of 131072 47 us (54 on inputs that change), of 4097 12 us
// with its join (8 and 4, both a launch and four dependent loads long).
constexpr int kFewRows = 16;

template <int DT, int D>
__global__ __launch_bounds__(256, 3) void attn_few_kernel(AttnArgs a)
{
    constexpr int C = D / 64;                            // 64-byte column runs of a key
    __shared__ float lo[4][kFewRows][D + 4];
    __shared__ float lm[4][kFewRows], ll[4][kFewRows];

    const Task task = task_of(a, blockIdx.x);
    const int b = task.b, hk = task.hk;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int p0 = task.split < 0 ? 0 : (int)(task.split * a.pages_per_split);

    // ---- a page's codes and scales ----
    // the table's entry for page p, or for its last one (never used: no page lies past the table)
    const scalar_i32 table = (scalar_i32)(a.batch.table + (int64_t)b * a.batch.ld_table);
    auto entry = [&](int64_t p) __attribute__((always_inline)) { return table[min(p, a.batch.ld_table - 1)]; };
    auto there = [&](int32_t id) __attribute__((always_inline)) { return id >= 0 && id < a.batch.n_pages; };
    const int krow = 16 * (col >> 2) + (col & 3);        // + 4 kb
    u32x4v kr[4][C], vr[D / 16];
    float ks, vs;
    auto load_page = [&](int32_t id) __attribute__((always_inline)) {
        const int64_t at = (int64_t)(there(id) ? id : 0) * a.Hkv + hk;   // page 0 stands in where there is none
        const uint8_t *kp = a.k + at * (kPage * D) + krow * D + 16 * quarter;
        const uint8_t *vp = a.v + at * (kPage * D) + col * kPage + 16 * quarter;
#pragma unroll
        for (int kb = 0; kb < 4; kb++)
#pragma unroll
            for (int c = 0; c < C; c++) kr[kb][c] = *reinterpret_cast<const u32x4v *>(kp + 4 * kb * D + 64 * c);
#pragma unroll
        for (int d = 0; d < D / 16; d++) vr[d] = __builtin_nontemporal_load(reinterpret_cast<const u32x4v *>(vp + 16 * d * kPage));
        ks = ((scalar_f32)a.k_scale)[at];
        vs = ((scalar_f32)a.v_scale)[at];
    };
    // the first page is on its way before the lengths are looked at: inside the cache, whatever
    // the table's unused places hold
    int32_t id = entry((int64_t)p0 + wave), id1 = entry((int64_t)p0 + wave + 4);
    const Seq s = load_seq(a, b);
    load_page(id);
    asm volatile("" ::: "memory");                       // not moved behind the next branch
    const int r0 = task.block * kFewRows;
    if (r0 >= s.rows) return;
    const int r = min(r0 + col, s.rows - 1);             // rows past the last repeat it and are not stored
    const int i_tok = r / a.G, head = hk * a.G + (r - i_tok * a.G);
    const int last = min(r0 + kFewRows, s.rows) - 1;
    const int lim = visible(a, s, i_tok);
    const int lim_all = visible(a, s, r0 / a.G);
    const int pages = (visible(a, s, last / a.G) + kPage - 1) / kPage;
    const int p1 = task.split < 0 || task.split + 1 == a.splits ? pages : (int)min((int64_t)pages, p0 + a.pages_per_split);
    if (task.split >= 0 && p0 >= p1) return;

    // queries: dims 64 c + 16 quarter + 8 u ..
    u32x4v q[C][2];
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
        for (int u = 0; u < 2; u++)
            q[c][u] = *reinterpret_cast<const u32x4v *>(a.q + (s.t0 + i_tok) * a.ld_q + head * D + 64 * c +
                                                        16 * quarter + 8 * u);

    f32x4 o[D / 16];
#pragma unroll
    for (int d = 0; d < D / 16; d++) o[d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float m = kLow, l = 0.0f;
    ValueRef ref;
    bool nan_codes = false;                              // NaN codes were cleared from a page of this wave

    for (int p = p0 + wave; p < p1; p += 4) {
        if (there(id)) {                                 // uniform in the wave
            f32x4 sc[4];
#pragma unroll
            for (int kb = 0; kb < 4; kb++) {
                sc[kb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < C; c++) {
                    sc[kb] = Half<DT>::mfma16(widen8<DT>(kr[kb][c][0], kr[kb][c][1]), q[c][0], sc[kb]);
                    sc[kb] = Half<DT>::mfma16(widen8<DT>(kr[kb][c][2], kr[kb][c][3]), q[c][1], sc[kb]);
                }
            }
            if ((p + 1) * kPage > lim_all) {                 // some row does not see all of the page
                uint32_t bad = 0;
                const int inside = s.kv - p * kPage - 16 * quarter;
#pragma unroll
                for (int d = 0; d < D / 16; d++)
#pragma unroll
                    for (int w = 0; w < 4; w++) {
                        const uint32_t x = vr[d][w] & below_bytes(inside - 4 * w);
                        const uint32_t n = nan_bytes(x);
                        bad |= n;
                        vr[d][w] = x & ~spread_bytes(n);
                    }
                nan_codes |= __builtin_amdgcn_ballot_w64(bad != 0) != 0;
                const int left = lim - p * kPage - 16 * quarter;
#pragma unroll
                for (int e = 0; e < 16; e++) sc[e >> 2][e & 3] = e < left ? sc[e >> 2][e & 3] : -__builtin_inff();
            }
            const float c = score_factor(a.factor, ks);
            float mx = sc[0][0];
#pragma unroll
            for (int e = 1; e < 16; e++) mx = fmaxf(mx, sc[e >> 2][e & 3]);
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32)) * c;
            if (__builtin_expect(__builtin_amdgcn_ballot_w64(mx > m + kSlack) != 0, 0)) {
                const float m1 = fmaxf(m, mx), f = __builtin_amdgcn_exp2f(m - m1);
                m = m1;
                l *= f;
#pragma unroll
                for (int d = 0; d < D / 16; d++) o[d] *= f;
            }
            ref.page(vs);
            if (__builtin_expect(ref.stray(), 0)) {
                if (__builtin_amdgcn_ballot_w64(ref.off(mx - m)) != 0) {
                    float most = 0.0f;
#pragma unroll
                    for (int d = 0; d < D / 16; d++)
#pragma unroll
                        for (int e = 0; e < 4; e++) most = fmaxf(most, fabsf(o[d][e]));
                    most = fmaxf(most, __shfl_xor(most, 16));
                    const int by = ref.move(fmaxf(most, __shfl_xor(most, 32)), mx - m);
#pragma unroll
                    for (int d = 0; d < D / 16; d++)
#pragma unroll
                        for (int e = 0; e < 4; e++) o[d][e] = __builtin_amdgcn_ldexpf(o[d][e], by);
                }
            }
            const float shift = ref.shift - m;
            float sum = 0.0f;
            u32x4v pk[2];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const float x = __builtin_amdgcn_exp2f(fmaf(sc[e >> 2][e & 3], c, shift));
                const float y = __builtin_amdgcn_exp2f(fmaf(sc[e >> 2][(e & 3) + 1], c, shift));
                sum += x + y;
                pk[e >> 3][(e >> 1) & 3] = Half<1>::pack(x, y);
            }
            l = fmaf(sum, ref.weight, l);
#pragma unroll
            for (int d = 0; d < D / 16; d++) {
                o[d] = Half<1>::mfma16(widen8<1>(vr[d][0], vr[d][1]), pk[0], o[d]);
                o[d] = Half<1>::mfma16(widen8<1>(vr[d][2], vr[d][3]), pk[1], o[d]);
            }
        }
        if (p + 4 >= p1) break;
        id = id1;
        load_page(id);
        id1 = entry((int64_t)p + 8);                     // a page ahead of its use
    }

    if (__builtin_expect(nan_codes, 0)) {                // uniform in the wave
        uint32_t hit = 0;                                // bit 4 d + e: element e of o[d]
        for (int p = p0 + wave; p < p1; p += 4) {
            const int32_t at = entry(p);
            if ((p + 1) * kPage <= lim_all || !there(at)) continue;
            const uint8_t *vp = a.v + ((int64_t)at * a.Hkv + hk) * (kPage * D);
            for (int i = 0; i < D / 4; i++)
                if (nan_among(vp + (16 * (i >> 2) + 4 * quarter + (i & 3)) * kPage, lim - p * kPage)) hit |= 1u << i;
        }
#pragma unroll
        for (int d = 0; d < D / 16; d++)
#pragma unroll
            for (int e = 0; e < 4; e++) o[d][e] = (hit >> (4 * d + e)) & 1 ? __builtin_nanf("") : o[d][e];
    }

    // ---- join the waves' averages: row `col`, dims 16 d + 4 quarter .. ----
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    const float mean = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int d = 0; d < D / 16; d++) {
        f32x4 x;
#pragma unroll
        for (int e = 0; e < 4; e++) x[e] = __builtin_amdgcn_ldexpf(o[d][e] * mean, ref.at);
        *reinterpret_cast<f32x4 *>(&lo[wave][col][16 * d + 4 * quarter]) = x;
    }
    if (quarter == 0) { lm[wave][col] = m; ll[wave][col] = l; }
    __syncthreads();
    const int n_rows = last - r0 + 1;
    for (int i = tid; i < n_rows * (D / 2); i += 256) {
        const int rr = i / (D / 2), d = 2 * (i % (D / 2));
        float top = kLow, x = 0.0f, y = 0.0f, sum = 0.0f, f[4];
#pragma unroll
        for (int w = 0; w < 4; w++) top = fmaxf(top, lm[w][rr]);
#pragma unroll
        for (int w = 0; w < 4; w++) {
            f[w] = ll[w][rr] * __builtin_amdgcn_exp2f(lm[w][rr] - top);
            sum += f[w];
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int w = 0; w < 4; w++) {
            x = fmaf(lo[w][rr][d], f[w] * inv, x);
            y = fmaf(lo[w][rr][d + 1], f[w] * inv, y);
        }
        const int gr = r0 + rr, tok = gr / a.G;
        const int hd = hk * a.G + (gr - tok * a.G);
        if (task.split >= 0) {
            const int64_t at = part_of(a, task, s, gr, r0, kFewRows);
            *reinterpret_cast<float2 *>(a.part_o + at * D + d) = float2{x, y};
            if (d == 0) a.part_ml[at] = float2{top, sum};
        } else {
            *reinterpret_cast<uint32_t *>(a.out + (s.t0 + tok) * a.ld_out + (int64_t)hd * D + d) = Half<DT>::pack(x, y);
        }
    }
}

// --------------------------------------------------------------- joining the splits ----
// W waves per row of the split blocks: the runs that hold keys the row sees, two (D = 128) or four
// at a time in 16-byte loads, a fixed order of sums; the waves' sums through LDS.
template <int DT, int D, int W>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int rows)
{
    constexpr int L = D / 4, P = 64 / L;                 // lanes of a run's row, runs a wave takes at once
    __shared__ float part[4][D];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), dim = 4 * (lane % L);
    const int64_t id = (int64_t)blockIdx.x * (4 / W) + wave / W;
    const int64_t stride = a.part_rows;
    if (id >= stride) return;                            // whole workgroups where waves share a row
    Task task;
    int tok, r;
    if (a.by_token) {
        const int t = (int)((uint32_t)id / (uint32_t)a.Hq), head = (int)id - t * a.Hq, units = a.B * a.Hkv;
        task.b = sequence_of(a, t, lane);
        if (task.b < 0) return;
        task.hk = head / a.G;
        tok = t - a.batch.cu[task.b];
        r = tok * a.G + head - task.hk * a.G;
        // in a block that the launch has, and one of the split ones (those are not moved on)
        const int block = r / rows;
        if (block >= a.row_blocks) return;
        if ((int64_t)(a.row_blocks - 1 - block) * units + task.b * a.Hkv + task.hk < a.whole) return;
    } else {
        task = task_of(a, a.whole + (int)(id / rows));
        r = task.block * rows + (int)(id % rows);
        tok = r / a.G;
    }
    const Seq s = load_seq(a, task.b);
    if (r >= s.rows) return;
    const int64_t pages = (visible(a, s, tok) + kPage - 1) / kPage;
    const int n = (int)min((pages + a.pages_per_split - 1) / a.pages_per_split, (int64_t)a.splits);
    // the first 64 runs' maxima and sums stay in the lanes
    const float2 own = lane < n ? a.part_ml[lane * stride + id] : float2{kLow, 0.0f};
    float top = own.x;
    for (int i = lane + 64; i < n; i += 64) top = fmaxf(top, a.part_ml[i * stride + id].x);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    float sum = own.y * __builtin_amdgcn_exp2f(own.x - top);
    for (int i = lane + 64; i < n; i += 64) {
        const float2 ml = a.part_ml[i * stride + id];
        sum = fmaf(ml.y, __builtin_amdgcn_exp2f(ml.x - top), sum);
    }
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int i = wave % W * P + lane / L; i < n; i += W * P) {
        const float2 ml = a.part_ml[i * stride + id];
        const float f = ml.y * __builtin_amdgcn_exp2f(ml.x - top) * inv;
        const f32x4 o = *reinterpret_cast<const f32x4 *>(a.part_o + (i * stride + id) * D + dim);
#pragma unroll
        for (int e = 0; e < 4; e++) acc[e] = fmaf(o[e], f, acc[e]);
    }
#pragma unroll
    for (int x = L; x < 64; x <<= 1) {
#pragma unroll
        for (int e = 0; e < 4; e++) acc[e] += __shfl_xor(acc[e], x);
    }
    if constexpr (W > 1) {
        if (lane < L) {
#pragma unroll
            for (int e = 0; e < 4; e++) part[wave][dim + e] = acc[e];
        }
        __syncthreads();
        if (wave != 0) return;
#pragma unroll
        for (int w = 1; w < W; w++)
#pragma unroll
            for (int e = 0; e < 4; e++) acc[e] += part[w][dim + e];
    }
    if (lane >= L) return;                               // they hold the same sums
    uint16_t *po = a.out + (s.t0 + tok) * a.ld_out + (task.hk * a.G + (r - tok * a.G)) * D + dim;
    *reinterpret_cast<u32x2v *>(po) = u32x2v{Half<DT>::pack(acc[0], acc[1]), Half<DT>::pack(acc[2], acc[3])};
}

// ----------------------------------------------------------------------- launching ----

AttnPlan plan_attn_kv8(int64_t T, int64_t B, int64_t max_q, int64_t max_kv, int Hq, int Hkv, int D, int cus)
{
    AttnPlan p{};
    p.splits = p.pages_per_split = p.row_blocks = 1;
    if (T == 0 || B == 0 || max_q == 0 || Hq == 0) return p;
    const int64_t rows = max_q * (Hq / Hkv);
    p.few = rows <= kFewRows;
    const int per = p.few ? kFewRows : kRowsBlock;
    p.row_blocks = (rows + per - 1) / per;
    const int64_t pages = max_kv > 0 ? (max_kv + kPage - 1) / kPage : 1;
    if (B > kMostBlocks / Hkv / p.row_blocks) {          // more than a launch counts: refused by the caller
        p.whole = kMostBlocks + 1;
        return p;
    }
    const int64_t base = B * Hkv * p.row_blocks;
    p.whole = base;
    if (p.few) {
        // Where the blocks fill the device (three workgroups a compute unit), runs short enough to
        // even out ragged lengths, but of 16 pages: 64 sequences of up to 32768 tokens, 8
        // key/value heads, 403 us in sixteen workgroups a compute unit, 431 in eight, 412 in 32 (before later steps).
        // Else enough runs to fill it once, at least 8 while that is within sixteen, of a page a
        // wave or more: one sequence of 131072 tokens in 96 runs 51 us, in 512 105 us (before later steps).
        const int64_t slots = 3 * (int64_t)cus, fine = 16 * (int64_t)cus / base;
        int64_t n = fine;
        if (base < slots) {
            n = (slots + base - 1) / base;
            if (n < 8) n = fine < 8 ? fine : 8;
        }
        const int64_t most = pages / (base >= slots ? 16 : 4);
        if (n > most) n = most;
        if (n > 1) {
            p.whole = 0;
            p.splits = n;
        }
    } else {
        // Rounds of workgroups over the device, each as long as its pages and a start worth three.
        // Either every block is split, or only those left over by whole rounds (the device then
        // shares them out).  The FP32 parts are written and read: in the time of a page the device
        // moves about 10 KiB a compute unit.
        const int64_t slots = (D == 64 ? 3 : 2) * (int64_t)cus;
        // Of the blocks, those that have rows: full ones, and about half a block a sequence.  Up to 515,
        // 311 and 106 rows over up to 10515 keys, 12 heads of 64: 73 us by these, 93 by all blocks; 30
        // sequences of up to 46 rows over 14183, 16 and 4 heads of 128: 166 against 205; the other way
        // 44 of up to 74 over 1547, 56 and 8 heads of 64: 68 against 61.
        const int64_t full = Hkv * (T * (Hq / Hkv) / per + (B + 1) / 2), busy = full < base ? (full < 1 ? 1 : full) : base;
        auto rounds = [&](int64_t blocks) { return ((int64_t)((double)blocks * busy / base) + slots - 1) / slots; };
        int64_t best = rounds(base) * (pages + 3) * 95 / 100;                 // splitting has to save 5 %
        for (const int64_t whole : {(int64_t)0, (int64_t)((double)(busy / slots * slots) * base / busy)}) {
            const int64_t tail = base - whole;
            if (tail == 0) continue;
            for (int64_t n = 2; n <= pages / 8 && n <= 64; n++) {
                const int64_t join = (int64_t)(2.0 * n * tail * busy / base * kRowsBlock * D * 4 / (10240.0 * cus));
                const int64_t cost = rounds(whole) * (pages + 3) + rounds(tail * n) * ((pages + n - 1) / n + 3) + join;
                if (cost < best) {
                    best = cost;
                    p.whole = whole;
                    p.splits = n;
                }
            }
        }
    }
    p.tail = base - p.whole;
    if (p.tail > 0) {
        p.pages_per_split = (pages + p.splits - 1) / p.splits;
        p.splits = (pages + p.pages_per_split - 1) / p.pages_per_split;
        // Parts lie in the order of the blocks, whose rows the join finds without a search.  Blocks are
        // counted for the longest run of queries, so a long prompt among short ones may have many times
        // more than there are rows: above 16 MiB, parts then lie by token and head (one prompt of 2048
        // tokens and 63 single ones, 32 and 8 heads of 128, over 32768: 3.7 GB by blocks, 0.18 so; 5
        // sequences of up to 4 tokens over 7997, 96 and 12 heads of 64: 30 us by blocks, 24 so).
        const int64_t row = (int64_t)p.splits * (D + 2) * 4;
        p.part_rows = p.tail * per;
        p.by_token = p.part_rows > T * Hq && p.part_rows > (16 << 20) / row;
        if (p.by_token) p.part_rows = T * Hq;
        p.off_ml = (size_t)p.splits * (size_t)p.part_rows * D * 4;
        p.bytes = (size_t)p.part_rows * (size_t)row;
        // many runs: four waves a row
        p.join_waves = p.splits > 8 ? 4 : 1;
        p.join_groups = p.join_waves == 4 ? p.part_rows : (p.part_rows + 3) / 4;
    }
    return p;
}

template <int DT, int D>
static hipError_t launch_attn(const AttnArgs &a, const AttnPlan &p, hipStream_t st)
{
    const int64_t blocks = p.whole + p.tail * p.splits;
    if (blocks > kMostBlocks || p.join_groups > kMostBlocks) return hipErrorInvalidValue;
    if (p.few) hipLaunchKernelGGL((attn_few_kernel<DT, D>), dim3((unsigned)blocks), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((attn_rows_kernel<DT, D>), dim3((unsigned)blocks), dim3(256), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.tail == 0) return e;
    const int rows = p.few ? kFewRows : kRowsBlock;
    const dim3 grid((unsigned)p.join_groups);
    if (p.join_waves == 4) hipLaunchKernelGGL((attn_join_kernel<DT, D, 4>), grid, dim3(256), 0, st, a, rows);
    else hipLaunchKernelGGL((attn_join_kernel<DT, D, 1>), grid, dim3(256), 0, st, a, rows);
    return hipGetLastError();
}

hipError_t launch_attn_kv8(const AttnLaunch &l, hipStream_t st)
{
    AttnArgs a{};
    a.q = static_cast<const uint16_t *>(l.q);
    a.out = static_cast<uint16_t *>(l.out);
    a.ld_q = l.ld_q; a.ld_out = l.ld_out;
    a.k = l.cache.k; a.v = l.cache.v; a.k_scale = l.cache.k_scale; a.v_scale = l.cache.v_scale;
    a.batch = Batch{l.cu, l.kv_lens, l.cache.table, l.cache.ld_table, l.cache.n_pages, l.T};
    a.B = (int)l.B; a.Hq = l.Hq; a.Hkv = l.Hkv; a.G = l.Hq / l.Hkv;
    a.row_blocks = (int)l.plan.row_blocks;
    a.whole = (int)l.plan.whole; a.tail = (int)l.plan.tail; a.splits = (int)l.plan.splits;
    a.pages_per_split = l.plan.pages_per_split;
    a.factor = l.sm_scale * 1.4426950408889634f;
    a.causal = l.causal;
    a.part_rows = l.plan.part_rows;
    a.by_token = l.plan.by_token;
    a.part_o = static_cast<float *>(l.workspace);
    a.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(l.workspace) + l.plan.off_ml);
    if (l.D == 128) return l.dtype == 0 ? launch_attn<0, 128>(a, l.plan, st) : launch_attn<1, 128>(a, l.plan, st);
    return l.dtype == 0 ? launch_attn<0, 64>(a, l.plan, st) : launch_attn<1, 64>(a, l.plan, st);
}

}  // namespace convrot
