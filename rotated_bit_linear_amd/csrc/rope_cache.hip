// Rotary embedding over several position axes, the per-head RMS norm of queries and keys, and
// the append of keys and values to the 8-bit paged cache, in one launch over the rows that a
// QKV projection writes.
//   per token and head: x' = x * w / sqrt(mean(x^2) + eps)           (where weights are given)
//   pair i of D/2, angle f = pos[axis[i]] * freq[i]:
//     (a, b) -> (a cos f - b sin f, b cos f + a sin f)
//   with (a, b) = (x[i], x[i + D/2]), or (x[2i], x[2i+1]) for interleaved pairs.
// Queries are rounded to their type; rotated keys and the values are quantized from FP32 to
// E4M3 against their page's scale, the smallest power of two that keeps the page's largest
// magnitude within 448.  A page that already holds older tokens keeps its scale or grows it;
// then the older codes are rescaled by that power of two.
// Angles: pos * freq reaches 10^6 rad and more, where FP32 has lost the fraction of the turn;
// it is taken in FP64 turns, whose fraction goes to the FP32 sine and cosine instructions
// (arguments in turns; at most 1.2e-7 off, two FP32 half steps of 1, over 4 million points).
//
// Bound by HBM: two bytes in, two (queries) or one (keys, values) out an element.  One page of
// one sequence and a run of heads per workgroup, so a page's maximum, its scale and its codes
// have one owner (no atomics on memory, the same result every time), and the sines of a token
// are shared by the run.  A team of D/16 lanes holds one token of one head, 8 pairs a lane;
// the 64 teams of a workgroup cover NT tokens of 64 / NT heads at once, NT from the longest
// run of new tokens (a single token a sequence leaves a team per head).
// Measured: 19989 tokens, 56 + 56 + 56 heads of 128, bf16, norms, three axes: 280 to 317 us (4.5 to
// 5.1 TB/s; a 1 GiB copy runs at 5.1); 7 ragged prompts of up to 1500 tokens, 24 + 8 + 8 heads of
// 64: 18 us; 64 single tokens, 32 + 8 + 8 heads of 128: 8 us, a chain of dependent loads.
#include <hip/hip_runtime.h>
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <stdint.h>

#include "elem_load.hpp"
#include "kernels.hpp"
#include "kv8.hpp"

namespace convrot {

struct RopeArgs {
    const void *qkv;
    int64_t ld_qkv;
    void *q_out;
    int64_t ld_q;
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    const float *q_weight, *k_weight;
    const int32_t *pos;
    int64_t ld_pos;
    const double *freq;
    const int32_t *axis;
    Batch batch;
    int n_axes;
    int Hq, Hkv;
    int max_new;         // tokens of a run that are processed
    int visits;          // pages that so many tokens may touch
    int log_tokens;      // of NT
    int q_chunks, kv_chunks;   // workgroups that share a page's heads (each takes every so-manieth)
    uint32_t q_blocks;
    float eps;
};

// sum over the lanes of a team (4 or 8 neighbouring lanes), the same bits in each
template <int TEAM>
__device__ __forceinline__ float team_sum(float x)
{
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0xB1, 0xF, 0xF, true));   // quad_perm 1,0,3,2
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x4E, 0xF, 0xF, true));   // quad_perm 2,3,0,1
    if constexpr (TEAM == 8)
        x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x141, 0xF, 0xF, true));  // row_half_mirror
    return x;
}

// The 16 elements of lane c of a team: elements 8c.. and D/2 + 8c.. (halves), or 16c..
// (interleaved); decoded, pair i is (x[i], x[8 + i]) either way.  Ordinary loads: interleaved,
// each takes halves of 32-byte runs, which non-temporal ones fetch twice (7 ragged prompts of
// up to 1500 tokens, 40 heads of 64, 21.5 against 18.1 us; no difference for whole lines).
struct Raw16 { u32x4v a, b; };
template <int D, bool IL>
__device__ __forceinline__ Raw16 fetch16(const uint16_t *head, int c)
{
    return {*reinterpret_cast<const u32x4v *>(head + (IL ? 16 * c : 8 * c)),
            *reinterpret_cast<const u32x4v *>(head + (IL ? 16 * c + 8 : D / 2 + 8 * c))};
}
template <int DT, bool IL>
__device__ __forceinline__ void decode16(const Raw16 &r, float (&x)[16])
{
    float y[16];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        y[i] = Elem<DT>::cvt((uint16_t)(r.a[i >> 1] >> (16 * (i & 1))));
        y[8 + i] = Elem<DT>::cvt((uint16_t)(r.b[i >> 1] >> (16 * (i & 1))));
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
        x[i] = IL ? y[2 * i] : y[i];
        x[8 + i] = IL ? y[2 * i + 1] : y[8 + i];
    }
}

template <int DT>
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    if constexpr (DT == 0)
        return (uint32_t)__bfloat16_as_ushort(__float2bfloat16(lo)) | ((uint32_t)__bfloat16_as_ushort(__float2bfloat16(hi)) << 16);
    else
        return (uint32_t)__half_as_ushort(__float2half(lo)) | ((uint32_t)__half_as_ushort(__float2half(hi)) << 16);
}

// What turns the 8 pairs of a lane: the norm's weights times cosine and sine,
// (a, b) -> r (a ca - b sb, b cb + a sa)
struct Turn { float ca[8], sa[8], cb[8], sb[8]; };

// 1 / sqrt(mean(x^2) + eps) of the head that a team holds.  Where FP32 squares overflow or vanish (bf16
// and eps reach there), x is moved by a power of two first, and eps with it.
template <int D>
__device__ __forceinline__ float team_rstd(float (&x)[16], float eps)
{
    auto mean = [&]() __attribute__((always_inline)) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i++) s = fmaf(x[i], x[i], s);
        return team_sum<D / 16>(s) * (1.0f / D);
    };
    float m = mean() + eps;
    if (__builtin_expect(!(m >= 0x1p-100f && m <= 0x1p100f), 0)) {
        const float k = m < 1.0f ? 0x1p70f : 0x1p-70f;
#pragma unroll
        for (int i = 0; i < 16; i++) x[i] *= k;
        m = mean() + eps * k * k;
    }
    return 1.0f / sqrtf(m);
}

__device__ __forceinline__ void turn16(float (&x)[16], const Turn &t, float r)
{
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float a = x[i], b = x[8 + i];
        x[i] = fmaf(a, t.ca[i], -(b * t.sb[i])) * r;
        x[8 + i] = fmaf(b, t.cb[i], a * t.sa[i]) * r;
    }
}

// largest finite magnitude of 16 values, as its bits (a NaN is passed over by the maximum; an
// infinity shows in it, and then each value is looked at)
__device__ __forceinline__ uint32_t amax16(const float (&x)[16])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i++) m = fmaxf(m, fabsf(x[i]));
    if (__builtin_expect(m == __builtin_inff(), 0)) {
        m = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i++) m = fabsf(x[i]) < __builtin_inff() ? fmaxf(m, fabsf(x[i])) : m;
    }
    return __float_as_uint(m);
}

// smallest power of two s >= 2^-126 with amax <= 448 s, from the bits of amax (448 = 1.75 * 2^8)
__device__ __forceinline__ float page_scale(uint32_t amax)
{
    const int e = (int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}

// four E4M3 codes of x * inv, round to nearest even (the conversion gives NaN for NaN and infinity)
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, r, true);
    return (uint32_t)r;
}

__device__ __forceinline__ uint8_t rescale1(uint8_t code, float f)
{
    const float x = __builtin_amdgcn_cvt_f32_fp8((int)code, 0) * f;
    return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, x, 0, false);
}

// IL: interleaved pairs
template <int DT, int D, bool IL>
__global__ __launch_bounds__(4 * D, 4) void rope_append_kernel(RopeArgs a)
{
    constexpr int TEAM = D / 16, TEAMS = 64;
    constexpr int VROW = kPage + 4;                        // bytes per dim of the transposed tile
    __shared__ uint32_t amax[3][2][TEAMS];                 // [step mod 3][keys, values][head slot]
    __shared__ __attribute__((aligned(16))) uint8_t vtile[D * VROW];

    // ---- this workgroup's page, tokens and heads ----
    // (all queries first: keys and values beside them measured 12 % slower)
    const bool is_q = blockIdx.x < a.q_blocks;
    const int chunks = is_q ? a.q_chunks : a.kv_chunks;
    const uint32_t id = is_q ? blockIdx.x : blockIdx.x - a.q_blocks;
    const int chunk = id % chunks, visit = id / chunks % a.visits, b = id / chunks / a.visits;
    PageRun run;
    if (!append_page_run(a.batch, b, a.max_new, visit, run)) return;
    const int nt = run.nt, off0 = run.off0;

    const int NT = 1 << a.log_tokens, HP = TEAMS >> a.log_tokens;   // tokens and heads at a time
    const int tid = threadIdx.x, c = tid % TEAM, team = tid / TEAM;
    const int tk = team & (NT - 1), slot = team >> a.log_tokens;

    // ---- cosine and sine of this lane's pairs, shared by the workgroup's heads ----
    const float *weight = is_q ? a.q_weight : a.k_weight;
    const bool live = tk < nt;
    const int64_t row = run.row0 + tk;
    const int64_t page = is_q ? 0 : batch_page(a.batch, b, run.page);
    if (!is_q && (!run.stored || page < 0)) return;        // nowhere to put them
    const uint16_t *qkv = static_cast<const uint16_t *>(a.qkv) + row * a.ld_qkv;
    const int step = chunks * HP, h0 = chunk * HP;         // heads h0 + slot, + step, ...
    // the first head's loads, under the sines
    Raw16 r0{}, r1{};
    if (live && h0 + slot < (is_q ? a.Hq : a.Hkv)) {
        r0 = fetch16<D, IL>(qkv + ((is_q ? 0 : a.Hq) + h0 + slot) * D, c);
        if (!is_q) r1 = fetch16<D, false>(qkv + (a.Hq + a.Hkv + h0 + slot) * D, c);
    }
    // every table entry in flight at once; of the positions all axes' are loaded and one selected,
    // so that no load waits for another
    float wa[8], wb[8];
    double freq[8];
    uint32_t axis[8];
    int32_t at[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; i++) wa[i] = wb[i] = 1.0f;
    if (weight) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            wa[i] = weight[IL ? 16 * c + 2 * i : 8 * c + i];
            wb[i] = weight[IL ? 16 * c + 2 * i + 1 : D / 2 + 8 * c + i];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
        freq[i] = a.freq[8 * c + i];
        axis[i] = a.axis[8 * c + i];
    }
    if (live) {
#pragma unroll
        for (int i = 0; i < 4; i++) at[i] = a.pos[row * a.ld_pos + min(i, a.n_axes - 1)];
    }
    Turn turn;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int32_t pos = axis[i] == 0 ? at[0] : axis[i] == 1 ? at[1] : axis[i] == 2 ? at[2] : at[3];   // beyond: the last
        const double turns = (double)pos * (freq[i] * 0.15915494309189533577);                         // 1 / (2 pi)
        const float part = (float)(turns - rint(turns));
        const float si = __builtin_amdgcn_sinf(part), co = __builtin_amdgcn_cosf(part);
        turn.ca[i] = wa[i] * co;
        turn.sa[i] = wa[i] * si;
        turn.cb[i] = wb[i] * co;
        turn.sb[i] = wb[i] * si;
    }
    if (is_q) {
        if (!live) return;                                 // whole teams, no barrier on this side
        const int64_t at = run.row0 + opaque(tk);          // found again: not kept over the other side's loop
        const uint16_t *src = static_cast<const uint16_t *>(a.qkv) + at * a.ld_qkv;
        uint16_t *out = static_cast<uint16_t *>(a.q_out) + at * a.ld_q;
        for (int h = h0 + slot; h < a.Hq; h += step) {
            float x[16];
            decode16<DT, IL>(r0, x);
            if (h + step < a.Hq) r0 = fetch16<D, IL>(src + (h + step) * D, c);
            turn16(x, turn, weight ? team_rstd<D>(x, a.eps) : 1.0f);
            uint16_t *o = out + h * D;
            u32x4v s0, s1;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                s0[i] = IL ? pack16<DT>(x[i], x[8 + i]) : pack16<DT>(x[2 * i], x[2 * i + 1]);
                s1[i] = IL ? pack16<DT>(x[4 + i], x[12 + i]) : pack16<DT>(x[8 + 2 * i], x[9 + 2 * i]);
            }
            *reinterpret_cast<u32x4v *>(o + (IL ? 16 * c : 8 * c)) = s0;
            *reinterpret_cast<u32x4v *>(o + (IL ? 16 * c + 8 : D / 2 + 8 * c)) = s1;
        }
        return;
    }

    // ---- keys and values ----
    int set = 0;
    for (int i = tid; i < 6 * TEAMS; i += 4 * D) (&amax[0][0][0])[i] = 0;
    __syncthreads();
    for (int hb = h0; hb < a.Hkv; hb += step) {
        const int h = hb + slot;
        const bool on = live && h < a.Hkv;
        float k[16], v[16];
        decode16<DT, IL>(r0, k);
        decode16<DT, false>(r1, v);
        if (live && h + step < a.Hkv) {
            r0 = fetch16<D, IL>(qkv + (a.Hq + h + step) * D, c);
            r1 = fetch16<D, false>(qkv + (a.Hq + a.Hkv + h + step) * D, c);
        }
        if (on) {
            turn16(k, turn, weight ? team_rstd<D>(k, a.eps) : 1.0f);
            atomicMax(&amax[set][0][slot], amax16(k));
            atomicMax(&amax[set][1][slot], amax16(v));
        }
        __syncthreads();
        float sk = page_scale(amax[set][0][slot]), sv = page_scale(amax[set][1][slot]);
        // the last step's set, read before this barrier, is used again after the next one
        const int last = set == 0 ? 2 : set - 1;
        if (tid < 2 * TEAMS) (&amax[last][0][0])[tid] = 0;
        set = set == 2 ? 0 : set + 1;
        const int64_t at = page * a.Hkv + h;
        uint8_t *kp = a.k + at * (kPage * D), *vp = a.v + at * (kPage * D);
        if (off0 > 0) {                                    // older tokens (uniform): the scale only grows
            float fk = 1.0f, fv = 1.0f;
            if (h < a.Hkv) {
                const float ok = a.k_scale[at], ov = a.v_scale[at];
                sk = fmaxf(ok, sk);
                sv = fmaxf(ov, sv);
                fk = ok / sk;
                fv = ov / sv;
            }
            __syncthreads();                               // every lane has the old scales
            const int lane = opaque(tk * TEAM + c), lanes = NT * TEAM;   // this head's lanes
            if (fk != 1.0f)
                for (int i = lane; i < off0 * D; i += lanes) kp[i] = rescale1(kp[i], fk);
            if (fv != 1.0f)
                for (int i = lane; i < off0 * D; i += lanes) {
                    uint8_t *q = vp + (i / off0) * kPage + i % off0;
                    *q = rescale1(*q, fv);
                }
        }
        const float ik = 1.0f / sk, iv = 1.0f / sv;
        // a full page of one head at a time (nt is at most NT, so HP is 1): values through LDS
        const bool whole = nt == kPage && HP == 1;
        if (on) {
            if (tk == 0 && c == 0) {
                a.k_scale[at] = sk;
                a.v_scale[at] = sv;
            }
            const int tt = off0 + tk;
            uint8_t *o = kp + opaque(tt * D), *gv = vp + opaque(8 * c * kPage + tt);   // not kept over the loop
            uint8_t *lv = vtile + opaque(8 * c * VROW + tt);
            if constexpr (IL) {
                u32x4v s;
#pragma unroll
                for (int i = 0; i < 4; i++) s[i] = encode4(k[2 * i], k[8 + 2 * i], k[2 * i + 1], k[9 + 2 * i], ik);
                *reinterpret_cast<u32x4v *>(o + 16 * c) = s;
            } else {
                u32x2v s0, s1;
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    s0[i] = encode4(k[4 * i], k[4 * i + 1], k[4 * i + 2], k[4 * i + 3], ik);
                    s1[i] = encode4(k[8 + 4 * i], k[9 + 4 * i], k[10 + 4 * i], k[11 + 4 * i], ik);
                }
                *reinterpret_cast<u32x2v *>(o + 8 * c) = s0;
                *reinterpret_cast<u32x2v *>(o + D / 2 + 8 * c) = s1;
            }
#pragma unroll
            for (int g = 0; g < 4; g++) {                  // v: registers 0..7 dims 8c.., 8..15 dims D/2 + 8c..
                const uint32_t e = encode4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3], iv);
                const int d = (g >= 2 ? D / 2 : 0) + 4 * (g & 1);          // + 8 c
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (whole) lv[(d + i) * VROW] = (uint8_t)(e >> (8 * i));
                    else gv[(d + i) * kPage] = (uint8_t)(e >> (8 * i));
                }
            }
        }
        if (whole) {                                       // uniform
            __syncthreads();
            const uint32_t *s = reinterpret_cast<const uint32_t *>(vtile + (tid >> 2) * VROW + 16 * (tid & 3));
            *reinterpret_cast<u32x4v *>(vp + 16 * tid) = u32x4v{s[0], s[1], s[2], s[3]};
            // the next step's first barrier orders these reads before its writes of the tile
        }
    }
}

template <int DT, int D>
static hipError_t launch_rope(RopeArgs a, int64_t B, int64_t max_new, bool interleaved, int cus, hipStream_t st)
{
    constexpr int TEAMS = 64;
    a.max_new = (int)max_new;
    a.log_tokens = append_log_tokens(max_new);
    const int hp = TEAMS >> a.log_tokens;
    a.visits = (int)append_visits(max_new);
    // heads per workgroup: a multiple of those it takes at a time, as many as leave four
    // workgroups for every compute unit (the sines are then shared by more heads), at most 8
    // steps (19989 tokens, 56 heads: 318 us with 16, 301 with 8; 8 heads with 4: 50 us, with 2: 58)
    const int64_t pages = B * a.visits;
    auto chunks = [&](int run) { return (a.Hq + run - 1) / run + (a.Hkv + run - 1) / run; };
    int run = hp;
    while (run < 8 * hp && pages * chunks(2 * run) >= 4 * (int64_t)cus) run *= 2;
    a.q_chunks = (a.Hq + run - 1) / run;
    a.kv_chunks = (a.Hkv + run - 1) / run;
    const int64_t blocks = pages * chunks(run);
    if (blocks > (int64_t)(UINT32_MAX / (4 * D))) return hipErrorInvalidValue;
    a.q_blocks = (uint32_t)(pages * a.q_chunks);
    if (interleaved) hipLaunchKernelGGL((rope_append_kernel<DT, D, true>), dim3((unsigned)blocks), dim3(4 * D), 0, st, a);
    else hipLaunchKernelGGL((rope_append_kernel<DT, D, false>), dim3((unsigned)blocks), dim3(4 * D), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_rope_append_kv8(const RopeLaunch &r, hipStream_t st)
{
    RopeArgs a{};
    a.qkv = r.qkv; a.ld_qkv = r.ld_qkv; a.q_out = r.q_out; a.ld_q = r.ld_q;
    a.k = r.cache.k; a.v = r.cache.v; a.k_scale = r.cache.k_scale; a.v_scale = r.cache.v_scale;
    a.q_weight = r.q_weight; a.k_weight = r.k_weight;
    a.pos = r.pos; a.ld_pos = r.ld_pos; a.freq = r.freq; a.axis = r.axis;
    a.batch = Batch{r.cu, r.kv_lens, r.cache.table, r.cache.ld_table, r.cache.n_pages, r.T};
    a.n_axes = r.n_axes; a.Hq = r.Hq; a.Hkv = r.Hkv; a.eps = r.eps;
    const bool il = r.interleaved != 0;
    if (r.D == 128) return r.dtype == 0 ? launch_rope<0, 128>(a, r.B, r.max_new, il, r.cus, st) : launch_rope<1, 128>(a, r.B, r.max_new, il, r.cus, st);
    return r.dtype == 0 ? launch_rope<0, 64>(a, r.B, r.max_new, il, r.cus, st) : launch_rope<1, 64>(a, r.B, r.max_new, il, r.cus, st);
}

}  // namespace convrot
