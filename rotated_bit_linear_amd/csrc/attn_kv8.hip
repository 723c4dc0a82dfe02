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
// are FP32.  P is rounded to the type of the queries (half a step, 2^-9 or 2^-12 of each
// p; errors of different keys are independent), as is the output.
// Scales: a page's key scale joins the factor of the exponent's argument, its value scale
// the exponent: P holds p * vs / vref, vref the largest value scale so far (the accumulators
// are rescaled when it grows), so 16-bit P never overflows.  A value scale below 2^-64 vref
// counts as 2^-64 vref.
// The running maximum is only raised when some row's scores exceed it by 8 (in log2): until
// then p is at most 2^8, which FP32 sums and both 16-bit types hold without loss, and the
// accumulators need no rescaling.
// Masked places: scores are selected, not added to, so NaN or infinite codes of keys that a
// row does not see leave it alone; values beyond kv_len are zeroed, and where some row of
// the tile does not see a key whose value holds a NaN code, the codes are zeroed and the NaN
// put into the scores of the rows that do see it.
#include <hip/hip_runtime.h>
#include <stdint.h>

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
    int row_blocks, splits;
    int64_t pages_per_split;
    float factor;            // sm_scale * log2(e)
    int causal;
    float *part_o;           // [split][T][Hq][D], times 2^(m) sums of p v (splits > 1)
    float2 *part_ml;         // [split][T][Hq] (running maximum, sum)
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
// one bit a byte (bits 0..3)
__device__ __forceinline__ uint32_t gather_bits(uint32_t b) { return (((b >> 7) & 0x01010101u) * 0x01020408u) >> 24; }
// the bytes of a word that hold tokens below `left` (word w of a run of tokens)
__device__ __forceinline__ uint32_t below_bytes(int left)
{
    return left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
}

constexpr float kLow = -1e30f;    // running maximum before the first key
constexpr float kSlack = 8.0f;    // log2: how far scores may exceed the running maximum

// the factor of a page's scores and the shift of its exponents
__device__ __forceinline__ float score_factor(float factor, float ks) { return fmaxf(factor * ks, 1e-37f); }

// per-sequence facts of a workgroup
struct Seq {
    int64_t t0, n, kv, rows;
};
__device__ __forceinline__ Seq load_seq(const AttnArgs &a, int b)
{
    Seq s;
    batch_rows(a.batch, b, s.t0, s.n);
    s.kv = batch_kv(a.batch, b);
    s.rows = s.n * a.G;
    return s;
}
// number of keys that token i of the sequence sees
__device__ __forceinline__ int64_t visible(const AttnArgs &a, const Seq &s, int64_t i)
{
    if (!a.causal) return s.kv;
    const int64_t l = s.kv - s.n + i + 1;
    return l < 0 ? 0 : l;
}

}  // namespace

// ------------------------------------------------------------------ prompts: many rows ----
// One workgroup: 32 query rows in each of 4 waves over a run of pages.  A page is read once
// into registers (while the page before it is multiplied), widened to 16 bits, and written to
// one of two LDS tiles in the order in which the matrix operands want it; chunks of 16 bytes
// are swizzled by row so that the 16 lanes of a read cover all banks.
constexpr int kRowsWave = 32, kWaves = 4, kRowsBlock = kRowsWave * kWaves;

template <int DT, int D>
__global__ __launch_bounds__(256, 2) void attn_rows_kernel(AttnArgs a)
{
    constexpr int TILE = kPage * D * 2;                 // bytes of a widened tile
    constexpr int KQ = D / 64, VQ = D / 64;             // 16-byte code loads a thread and tile
    constexpr int KC = D / 8;                           // 16-byte chunks of a widened key row
    __shared__ __attribute__((aligned(1024))) uint8_t ldsK[2][TILE];
    __shared__ __attribute__((aligned(1024))) uint8_t ldsV[2][TILE];
    __shared__ uint32_t nan_keys[3][2];                 // keys of a tile whose values hold NaN codes

    // longest rows first (causal), key/value heads apart by the XCDs' stride
    const int units = a.B * a.Hkv;
    const int unit = blockIdx.x % units, rest = blockIdx.x / units;
    const int split = rest % a.splits, block = a.row_blocks - 1 - rest / a.splits;
    const int b = unit / a.Hkv, hk = unit % a.Hkv;
    const Seq s = load_seq(a, b);
    const int64_t r0 = (int64_t)block * kRowsBlock;
    if (r0 >= s.rows) return;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int col = lane & 31, half = lane >> 5;
    const int64_t r = r0 + wave * kRowsWave + col;
    const bool valid = r < s.rows;
    const int64_t i_tok = valid ? r / a.G : 0;
    const int head = hk * a.G + (valid ? (int)(r - i_tok * a.G) : 0);
    const int64_t row = s.t0 + i_tok;

    // keys seen: by this row, by the block's last row (the loop's end) and by all of its rows
    const int64_t last = (r0 + kRowsBlock < s.rows ? r0 + kRowsBlock : s.rows) - 1;
    const int lim = valid ? (int)visible(a, s, i_tok) : 0;
    const int lim_all = (int)visible(a, s, r0 / a.G);
    const int pages = ((int)visible(a, s, last / a.G) + kPage - 1) / kPage;
    const int p0 = (int)(split * a.pages_per_split);
    const int p1 = split + 1 == a.splits ? pages : (int)min((int64_t)pages, p0 + a.pages_per_split);
    if (a.splits > 1 && p0 >= p1) return;               // no row of the block looks here

    u32x4v q[D / 16];
#pragma unroll
    for (int k = 0; k < D / 16; k++)
        q[k] = valid ? *reinterpret_cast<const u32x4v *>(a.q + row * a.ld_q + (int64_t)head * D + 16 * k + 8 * half)
                     : u32x4v{0u, 0u, 0u, 0u};

    // ---- staging ----
    u32x4v kreg[KQ], vreg[VQ];
    float ks_next = 0.0f, vs_next = 0.0f;
    bool ok_next = false;
    const int k_row = tid >> 2, k_off = (tid & 3) * (D / 4);
    auto load = [&](int p) {
        // where the table names no page, page 0 is read and nobody sees its keys
        const int64_t id = batch_page(a.batch, b, p);
        ok_next = id >= 0;
        const int64_t at = (ok_next ? id : 0) * a.Hkv + hk;
        const uint8_t *kp = a.k + at * (kPage * D), *vp = a.v + at * (kPage * D);
#pragma unroll
        for (int i = 0; i < KQ; i++) kreg[i] = *reinterpret_cast<const u32x4v *>(kp + k_row * D + k_off + 16 * i);
#pragma unroll
        for (int i = 0; i < VQ; i++) vreg[i] = *reinterpret_cast<const u32x4v *>(vp + 16 * (tid + 256 * i));
        ks_next = a.k_scale[at];
        vs_next = a.v_scale[at];
    };
    auto store = [&](int p, int buf, int slot) {
        if ((p + 1) * kPage > lim_all) {                // some row does not see all of the page
#pragma unroll
            for (int i = 0; i < VQ; i++) {
                const int u = tid + 256 * i, j = u & 3;
                const int left = (int)s.kv - p * kPage - 16 * j;
#pragma unroll
                for (int w = 0; w < 4; w++) {
                    uint32_t x = vreg[i][w] & below_bytes(left - 4 * w);
                    const uint32_t bad = nan_bytes(x);
                    if (bad) {
                        atomicOr(&nan_keys[slot][j >> 1], gather_bits(bad) << (16 * (j & 1) + 4 * w));
                        x &= ~spread_bytes(bad);
                    }
                    vreg[i][w] = x;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < KQ; i++) {
            const int c = k_off / 8 + 2 * i;            // chunk in the key's row
            const int sw = KC == 16 ? (k_row & 15) : ((k_row >> 1) & 7);
            uint8_t *dst = ldsK[buf] + k_row * (2 * D);
            *reinterpret_cast<u32x4v *>(dst + ((c ^ sw) << 4)) = widen8<DT>(kreg[i][0], kreg[i][1]);
            *reinterpret_cast<u32x4v *>(dst + (((c + 1) ^ sw) << 4)) = widen8<DT>(kreg[i][2], kreg[i][3]);
        }
#pragma unroll
        for (int i = 0; i < VQ; i++) {                  // 16 tokens of one dim: words 0, 2 for lanes 0-31, 1, 3 for 32-63
            const int u = tid + 256 * i, d = u >> 2, j = u & 3;
            const int sw = (d >> 1) & 7;
            uint8_t *dst = ldsV[buf] + d * (2 * kPage);
            *reinterpret_cast<u32x4v *>(dst + (((2 * j) ^ sw) << 4)) = widen8<DT>(vreg[i][0], vreg[i][2]);
            *reinterpret_cast<u32x4v *>(dst + (((2 * j + 1) ^ sw) << 4)) = widen8<DT>(vreg[i][1], vreg[i][3]);
        }
    };

    f32x16 o[D / 32];
#pragma unroll
    for (int d = 0; d < D / 32; d++)
#pragma unroll
        for (int e = 0; e < 16; e++) o[d][e] = 0.0f;
    float m = kLow, l = 0.0f, vref = kMinScale;

    if (tid < 6) (&nan_keys[0][0])[tid] = 0;
    float ks = 0.0f, vs = 0.0f;
    bool ok = false;
    if (p0 < p1) {
        load(p0);
        __syncthreads();
        store(p0, 0, 0);
        ks = ks_next; vs = vs_next; ok = ok_next;
    }
    __syncthreads();

    int slot = 0;
    for (int p = p0; p < p1; p++) {
        const int buf = (p - p0) & 1, slot1 = slot == 2 ? 0 : slot + 1, slot2 = slot1 == 2 ? 0 : slot1 + 1;
        if (tid < 2) nan_keys[slot2][tid] = 0;          // read a page ago, written a page from now
        const bool more = p + 1 < p1;
        if (more) load(p + 1);

        f32x16 sc[2];
#pragma unroll
        for (int kb = 0; kb < 2; kb++) {
#pragma unroll
            for (int e = 0; e < 16; e++) sc[kb][e] = 0.0f;
            const int kr = 32 * kb + col;
            const int sw = KC == 16 ? (kr & 15) : ((kr >> 1) & 7);
            const uint8_t *src = ldsK[buf] + kr * (2 * D);
#pragma unroll
            for (int k = 0; k < D / 16; k++)
                sc[kb] = Half<DT>::mfma32(*reinterpret_cast<const u32x4v *>(src + (((2 * k + half) ^ sw) << 4)), q[k], sc[kb]);
        }
        if ((p + 1) * kPage > lim_all || !ok) {         // masks: uniform in the workgroup
            const int left = ok ? lim - p * kPage : 0;
#pragma unroll
            for (int kb = 0; kb < 2; kb++) {
                const uint32_t bad = nan_keys[slot][kb];
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    const int key = 8 * (e >> 2) + 4 * half + (e & 3);
                    const float x = (bad >> key) & 1 ? __uint_as_float(0x7fc00000u) : sc[kb][e];
                    sc[kb][e] = 32 * kb + key < left ? x : -__builtin_inff();
                }
            }
        }
        const float c = score_factor(a.factor, ks);
        float mx = sc[0][0];
#pragma unroll
        for (int e = 1; e < 32; e++) mx = fmaxf(mx, sc[e >> 4][e & 15]);
        mx = fmaxf(mx, __shfl_xor(mx, 32)) * c;
        if (__builtin_amdgcn_ballot_w64(mx > m + kSlack) != 0) {
            const float m1 = fmaxf(m, mx), f = __builtin_amdgcn_exp2f(m - m1);
            m = m1;
            l *= f;
#pragma unroll
            for (int d = 0; d < D / 32; d++)
#pragma unroll
                for (int e = 0; e < 16; e++) o[d][e] *= f;
        }
        const float vsx = fmaxf(fmaxf(vs, kMinScale), vref * 0x1p-64f);
        if (vsx > vref) {                               // uniform
            const float f = vref / vsx;
            vref = vsx;
#pragma unroll
            for (int d = 0; d < D / 32; d++)
#pragma unroll
                for (int e = 0; e < 16; e++) o[d][e] *= f;
        }
        const float shift = __builtin_amdgcn_logf(vsx / vref) - m;
        float sum = 0.0f;
        u32x4v pk[4];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            const float x = __builtin_amdgcn_exp2f(fmaf(sc[e >> 4][e & 15], c, shift));
            const float y = __builtin_amdgcn_exp2f(fmaf(sc[e >> 4][(e & 15) + 1], c, shift));
            sum += x + y;
            pk[e >> 3][(e >> 1) & 3] = Half<DT>::pack(x, y);
        }
        l = fmaf(sum, vref / vsx, l);
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int d = 0; d < D / 32; d++) {
                const int vr = 32 * d + col;
                const uint8_t *src = ldsV[buf] + vr * (2 * kPage) + (((2 * j + half) ^ ((vr >> 1) & 7)) << 4);
                o[d] = Half<DT>::mfma32(*reinterpret_cast<const u32x4v *>(src), pk[j], o[d]);
            }
        if (more) {
            store(p + 1, buf ^ 1, slot1);
            ks = ks_next; vs = vs_next; ok = ok_next;
        }
        slot = slot1;
        __syncthreads();
    }

    // ---- the lane's row: dims 32 d + 8 g + 4 half + 0..3 ----
    l += __shfl_xor(l, 32);
    if (!valid) return;
    if (a.splits > 1) {
        float *po = a.part_o + (((int64_t)split * a.batch.T + row) * a.Hq + head) * D;
#pragma unroll
        for (int d = 0; d < D / 32; d++)
#pragma unroll
            for (int g = 0; g < 4; g++)
                *reinterpret_cast<f32x4 *>(po + 32 * d + 8 * g + 4 * half) =
                    f32x4{o[d][4 * g] * vref, o[d][4 * g + 1] * vref, o[d][4 * g + 2] * vref, o[d][4 * g + 3] * vref};
        if (half == 0) a.part_ml[((int64_t)split * a.batch.T + row) * a.Hq + head] = float2{m, l};
        return;
    }
    const float inv = l == 0.0f ? 0.0f : vref / l;
    uint16_t *po = a.out + row * a.ld_out + (int64_t)head * D;
#pragma unroll
    for (int d = 0; d < D / 32; d++)
#pragma unroll
        for (int g = 0; g < 4; g++)
            *reinterpret_cast<u32x2v *>(po + 32 * d + 8 * g + 4 * half) =
                u32x2v{Half<DT>::pack(o[d][4 * g] * inv, o[d][4 * g + 1] * inv),
                       Half<DT>::pack(o[d][4 * g + 2] * inv, o[d][4 * g + 3] * inv)};
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
// Bound by the cache's bytes: the waves keep a whole page each in flight.
constexpr int kFewRows = 16;

template <int DT, int D>
__global__ __launch_bounds__(256) void attn_few_kernel(AttnArgs a)
{
    constexpr int C = D / 64;                            // 64-byte column runs of a key
    __shared__ float lo[4][kFewRows][D + 4];
    __shared__ float lm[4][kFewRows], ll[4][kFewRows];

    const int units = a.B * a.Hkv;
    const int unit = blockIdx.x % units, rest = blockIdx.x / units;
    const int block = rest % a.row_blocks, split = rest / a.row_blocks;
    const int b = unit / a.Hkv, hk = unit % a.Hkv;
    const Seq s = load_seq(a, b);
    const int64_t r0 = (int64_t)block * kFewRows;
    if (r0 >= s.rows) return;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int64_t r = r0 + col;
    const bool valid = r < s.rows;
    const int64_t i_tok = valid ? r / a.G : 0;
    const int head = hk * a.G + (valid ? (int)(r - i_tok * a.G) : 0);
    const int64_t last = (r0 + kFewRows < s.rows ? r0 + kFewRows : s.rows) - 1;
    const int lim = valid ? (int)visible(a, s, i_tok) : 0;
    const int lim_all = (int)visible(a, s, r0 / a.G);
    const int pages = ((int)visible(a, s, last / a.G) + kPage - 1) / kPage;
    const int p0 = (int)(split * a.pages_per_split);
    const int p1 = split + 1 == a.splits ? pages : (int)min((int64_t)pages, p0 + a.pages_per_split);
    if (a.splits > 1 && p0 >= p1) return;

    // queries: dims 64 c + 16 quarter + 8 u ..
    u32x4v q[C][2];
#pragma unroll
    for (int c = 0; c < C; c++)
#pragma unroll
        for (int u = 0; u < 2; u++)
            q[c][u] = valid ? *reinterpret_cast<const u32x4v *>(a.q + (s.t0 + i_tok) * a.ld_q + (int64_t)head * D +
                                                                 64 * c + 16 * quarter + 8 * u)
                            : u32x4v{0u, 0u, 0u, 0u};

    f32x4 o[D / 16];
#pragma unroll
    for (int d = 0; d < D / 16; d++) o[d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float m = kLow, l = 0.0f, vref = kMinScale;

    const int krow = 16 * (col >> 2) + (col & 3);        // + 4 kb
    for (int p = p0 + wave; p < p1; p += 4) {
        const int64_t id = batch_page(a.batch, b, p);
        if (id < 0) continue;                            // no such page (wave-uniform)
        const int64_t at = id * a.Hkv + hk;
        const uint8_t *kp = a.k + at * (kPage * D) + krow * D + 16 * quarter;
        const uint8_t *vp = a.v + at * (kPage * D) + col * kPage + 16 * quarter;
        u32x4v kr[4][C], vr[D / 16];
#pragma unroll
        for (int kb = 0; kb < 4; kb++)
#pragma unroll
            for (int c = 0; c < C; c++) kr[kb][c] = *reinterpret_cast<const u32x4v *>(kp + 4 * kb * D + 64 * c);
#pragma unroll
        for (int d = 0; d < D / 16; d++) vr[d] = *reinterpret_cast<const u32x4v *>(vp + 16 * d * kPage);
        const float ks = a.k_scale[at], vs = a.v_scale[at];

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
            uint32_t bad = 0;                            // this lane's 16 keys whose values hold NaN codes
            const int inside = (int)s.kv - p * kPage - 16 * quarter;
#pragma unroll
            for (int d = 0; d < D / 16; d++)
#pragma unroll
                for (int w = 0; w < 4; w++) {
                    uint32_t x = vr[d][w] & below_bytes(inside - 4 * w);
                    const uint32_t n = nan_bytes(x);
                    bad |= gather_bits(n) << (4 * w);
                    vr[d][w] = x & ~spread_bytes(n);
                }
#pragma unroll
            for (int x = 1; x < 16; x <<= 1) bad |= __shfl_xor(bad, x);   // over the dims of the other lanes
            const int left = lim - p * kPage - 16 * quarter;
#pragma unroll
            for (int kb = 0; kb < 4; kb++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int key = 4 * kb + e;
                    const float x = (bad >> key) & 1 ? __uint_as_float(0x7fc00000u) : sc[kb][e];
                    sc[kb][e] = key < left ? x : -__builtin_inff();
                }
        }
        const float c = score_factor(a.factor, ks);
        float mx = sc[0][0];
#pragma unroll
        for (int e = 1; e < 16; e++) mx = fmaxf(mx, sc[e >> 2][e & 3]);
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32)) * c;
        if (__builtin_amdgcn_ballot_w64(mx > m + kSlack) != 0) {
            const float m1 = fmaxf(m, mx), f = __builtin_amdgcn_exp2f(m - m1);
            m = m1;
            l *= f;
#pragma unroll
            for (int d = 0; d < D / 16; d++) o[d] *= f;
        }
        const float vsx = fmaxf(fmaxf(vs, kMinScale), vref * 0x1p-64f);
        if (vsx > vref) {                                // uniform
            const float f = vref / vsx;
            vref = vsx;
#pragma unroll
            for (int d = 0; d < D / 16; d++) o[d] *= f;
        }
        const float shift = __builtin_amdgcn_logf(vsx / vref) - m;
        float sum = 0.0f;
        u32x4v pk[2];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const float x = __builtin_amdgcn_exp2f(fmaf(sc[e >> 2][e & 3], c, shift));
            const float y = __builtin_amdgcn_exp2f(fmaf(sc[e >> 2][(e & 3) + 1], c, shift));
            sum += x + y;
            pk[e >> 3][(e >> 1) & 3] = Half<DT>::pack(x, y);
        }
        l = fmaf(sum, vref / vsx, l);
#pragma unroll
        for (int d = 0; d < D / 16; d++) {
            o[d] = Half<DT>::mfma16(widen8<DT>(vr[d][0], vr[d][1]), pk[0], o[d]);
            o[d] = Half<DT>::mfma16(widen8<DT>(vr[d][2], vr[d][3]), pk[1], o[d]);
        }
    }

    // ---- join the waves: row `col`, dims 16 d + 4 quarter .. ----
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
#pragma unroll
    for (int d = 0; d < D / 16; d++)
        *reinterpret_cast<f32x4 *>(&lo[wave][col][16 * d + 4 * quarter]) =
            f32x4{o[d][0] * vref, o[d][1] * vref, o[d][2] * vref, o[d][3] * vref};
    if (quarter == 0) { lm[wave][col] = m; ll[wave][col] = l; }
    __syncthreads();
    const int n_rows = (int)(last - r0) + 1;
    for (int i = tid; i < n_rows * (D / 2); i += 256) {
        const int rr = i / (D / 2), d = 2 * (i % (D / 2));
        float top = kLow, x = 0.0f, y = 0.0f, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; w++) top = fmaxf(top, lm[w][rr]);
#pragma unroll
        for (int w = 0; w < 4; w++) {
            const float f = __builtin_amdgcn_exp2f(lm[w][rr] - top);
            x = fmaf(lo[w][rr][d], f, x);
            y = fmaf(lo[w][rr][d + 1], f, y);
            sum = fmaf(ll[w][rr], f, sum);
        }
        const int64_t gr = r0 + rr, tok = gr / a.G;
        const int hd = hk * a.G + (int)(gr - tok * a.G);
        if (a.splits > 1) {
            const int64_t at = ((int64_t)split * a.batch.T + s.t0 + tok) * a.Hq + hd;
            *reinterpret_cast<float2 *>(a.part_o + at * D + d) = float2{x, y};
            if (d == 0) a.part_ml[at] = float2{top, sum};
        } else {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            *reinterpret_cast<uint32_t *>(a.out + (s.t0 + tok) * a.ld_out + (int64_t)hd * D + d) =
                Half<DT>::pack(x * inv, y * inv);
        }
    }
}

// --------------------------------------------------------------- joining the splits ----
// One wave per query row: the runs that hold keys the row sees, in order.
template <int DT, int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t rid = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (rid >= a.batch.T * a.Hq) return;
    const int64_t row = rid / a.Hq;
    // the sequence of this row (the rows of sequence b start at cu[b])
    int b = 0;
    for (int step = 1 << 30; step > 0; step >>= 1)
        if (b + step < a.B && a.batch.cu[b + step] <= row) b += step;
    const Seq s = load_seq(a, b);
    if (row < s.t0 || row >= s.t0 + s.n) return;         // a row of no sequence
    const int lim = (int)visible(a, s, row - s.t0);
    const int64_t pages = (lim + kPage - 1) / kPage;
    int64_t n = (pages + a.pages_per_split - 1) / a.pages_per_split;
    if (n > a.splits) n = a.splits;
    const int64_t stride = a.batch.T * a.Hq;
    float top = kLow;
    for (int64_t i = lane; i < n; i += 64) top = fmaxf(top, a.part_ml[i * stride + rid].x);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    constexpr int E = D / 64;
    float acc[E] = {}, sum = 0.0f;
    for (int64_t i = 0; i < n; i++) {
        const float2 ml = a.part_ml[i * stride + rid];
        const float f = __builtin_amdgcn_exp2f(ml.x - top);
        sum = fmaf(ml.y, f, sum);
#pragma unroll
        for (int e = 0; e < E; e++) acc[e] = fmaf(a.part_o[(i * stride + rid) * D + E * lane + e], f, acc[e]);
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t *po = a.out + row * a.ld_out + (rid - row * a.Hq) * D + E * lane;
    if constexpr (E == 2) *reinterpret_cast<uint32_t *>(po) = Half<DT>::pack(acc[0] * inv, acc[1] * inv);
    else *po = (uint16_t)Half<DT>::pack(acc[0] * inv, 0.0f);
}

// ----------------------------------------------------------------------- launching ----

AttnPlan plan_attn_kv8(int64_t T, int64_t B, int64_t max_q, int64_t max_kv, int Hq, int Hkv, int D, int cus)
{
    AttnPlan p{};
    p.splits = p.pages_per_split = p.row_blocks = 1;
    if (T == 0 || B == 0 || max_q == 0 || Hq == 0) return p;
    const int64_t rows = max_q * (Hq / Hkv);
    p.few = rows <= 2 * kFewRows;
    const int per = p.few ? kFewRows : kRowsBlock;
    p.row_blocks = (rows + per - 1) / per;
    const int64_t pages = max_kv > 0 ? (max_kv + kPage - 1) / kPage : 1;
    const int64_t base = B * Hkv * p.row_blocks;
    // workgroups wanted, and the fewest pages that are worth one
    const int64_t want = (p.few ? 8 : 2) * (int64_t)cus, least = p.few ? 4 : 8;
    int64_t splits = (want + base - 1) / base;
    if (splits > pages / least) splits = pages / least;
    if (splits < 1) splits = 1;
    p.pages_per_split = (pages + splits - 1) / splits;
    p.splits = (pages + p.pages_per_split - 1) / p.pages_per_split;
    if (p.splits > 1) {
        p.off_ml = (((size_t)p.splits * (size_t)T * Hq * D * 4) + 255) & ~(size_t)255;
        p.bytes = p.off_ml + (size_t)p.splits * (size_t)T * Hq * 8;
    }
    return p;
}

template <int DT, int D>
static hipError_t launch_attn(const AttnArgs &a, bool few, hipStream_t st)
{
    const int64_t blocks = (int64_t)a.B * a.Hkv * a.row_blocks * a.splits;
    if (blocks > (int64_t)(UINT32_MAX / 256)) return hipErrorInvalidValue;
    if (few) hipLaunchKernelGGL((attn_few_kernel<DT, D>), dim3((unsigned)blocks), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((attn_rows_kernel<DT, D>), dim3((unsigned)blocks), dim3(256), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    hipLaunchKernelGGL((attn_join_kernel<DT, D>), dim3((unsigned)((a.batch.T * a.Hq + 3) / 4)), dim3(256), 0, st, a);
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
    a.row_blocks = (int)l.plan.row_blocks; a.splits = (int)l.plan.splits;
    a.pages_per_split = l.plan.pages_per_split;
    a.factor = l.sm_scale * 1.4426950408889634f;
    a.causal = l.causal;
    a.part_o = static_cast<float *>(l.workspace);
    a.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(l.workspace) + l.plan.off_ml);
    if (l.D == 128) return l.dtype == 0 ? launch_attn<0, 128>(a, l.plan.few, st) : launch_attn<1, 128>(a, l.plan.few, st);
    return l.dtype == 0 ? launch_attn<0, 64>(a, l.plan.few, st) : launch_attn<1, 64>(a, l.plan.few, st);
}

}  // namespace convrot
