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
// it is taken in FP64 turns, whose fraction goes to FP32 sine and cosine.
//
// Bound by HBM: two bytes in, two (queries) or one (keys, values) out an element.  One page of
// one sequence and a run of heads per workgroup, so a page's maximum, its scale and its codes
// have one owner (no atomics on memory, the same result every time), and the sines of a token
// are shared by the run.  A team of D/16 lanes holds one token of one head, 8 pairs a lane;
// teams of a workgroup cover NT tokens of 256 / (NT * D/16) heads at once, NT from the
// longest run of new tokens (a single token a sequence leaves a team per head).
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
    int visits;          // pages that the longest run of new tokens may touch
    int tokens;          // NT, a power of two
    int q_run, kv_run;   // heads per workgroup
    int q_chunks, chunks;
    float eps;
    int interleaved;
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
// (interleaved); in registers pair i is (x[i], x[8 + i]) either way.
template <int DT, int D>
__device__ __forceinline__ void load16(const uint16_t *head, int c, int interleaved, float (&x)[16])
{
    const u32x4v *p0 = reinterpret_cast<const u32x4v *>(head + (interleaved ? 16 * c : 8 * c));
    const u32x4v *p1 = reinterpret_cast<const u32x4v *>(head + (interleaved ? 16 * c + 8 : D / 2 + 8 * c));
    const u32x4v a = __builtin_nontemporal_load(p0), b = __builtin_nontemporal_load(p1);
    float y[16];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        y[i] = Elem<DT>::cvt((uint16_t)(a[i >> 1] >> (16 * (i & 1))));
        y[8 + i] = Elem<DT>::cvt((uint16_t)(b[i >> 1] >> (16 * (i & 1))));
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
        x[i] = interleaved ? y[2 * i] : y[i];
        x[8 + i] = interleaved ? y[2 * i + 1] : y[8 + i];
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

template <int D>
__device__ __forceinline__ void norm16(float (&x)[16], const float (&w)[16], float eps)
{
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i++) s = fmaf(x[i], x[i], s);
    s = team_sum<D / 16>(s);
    const float r = 1.0f / sqrtf(s * (1.0f / D) + eps);
#pragma unroll
    for (int i = 0; i < 16; i++) x[i] = x[i] * r * w[i];
}

__device__ __forceinline__ void turn16(float (&x)[16], const float (&co)[8], const float (&si)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float a = x[i], b = x[8 + i];
        x[i] = fmaf(a, co[i], -(b * si[i]));
        x[8 + i] = fmaf(b, co[i], a * si[i]);
    }
}

// largest finite magnitude of 16 values
__device__ __forceinline__ uint32_t amax16(const float (&x)[16])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const uint32_t u = __float_as_uint(x[i]) & 0x7fffffffu;
        m = max(m, u < 0x7f800000u ? u : 0u);
    }
    return m;
}

// smallest power of two s >= 2^-126 with amax <= 448 s, from the bits of amax (448 = 1.75 * 2^8)
__device__ __forceinline__ float page_scale(uint32_t amax)
{
    const int e = (int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}

// four E4M3 codes of x * inv, round to nearest even; a value that is not finite gives NaN
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv)
{
    auto val = [inv](float x) {
        return (__float_as_uint(x) & 0x7fffffffu) < 0x7f800000u ? x * inv : __uint_as_float(0x7fc00000u);
    };
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(val(a), val(b), 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(val(c), val(d), r, true);
    return (uint32_t)r;
}

__device__ __forceinline__ uint8_t rescale1(uint8_t code, float f)
{
    const float x = __builtin_amdgcn_cvt_f32_fp8((int)code, 0) * f;
    return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, x, 0, false);
}

// NI: rounds of NT tokens that a page may take
template <int DT, int D, int NI>
__global__ __launch_bounds__(256) void rope_append_kernel(RopeArgs a)
{
    constexpr int TEAM = D / 16, TEAMS = 256 / TEAM;
    constexpr int VROW = kPage + 4;                        // bytes per dim of the transposed tile
    __shared__ uint32_t amax[2][2][TEAMS];                 // [step parity][keys, values][head slot]
    __shared__ __attribute__((aligned(16))) uint8_t vtile[D * VROW];

    // ---- this workgroup's page, tokens and heads ----
    int64_t id = blockIdx.x;
    const int chunk = (int)(id % a.chunks);
    id /= a.chunks;
    const int visit = (int)(id % a.visits), b = (int)(id / a.visits);
    int64_t t0, n;
    batch_rows(a.batch, b, t0, n);
    if (n == 0) return;
    const int64_t kv = a.batch.kv_lens[b];
    const int64_t first = kv >= n ? kv - n : 0;            // position of the first new token
    const int64_t pg = first / kPage + visit;
    const int64_t lo = first > pg * kPage ? first : pg * kPage;
    const int64_t hi = first + n < (pg + 1) * kPage ? first + n : (pg + 1) * kPage;
    if (lo >= hi) return;
    const int nt = (int)(hi - lo), off0 = (int)(lo - pg * kPage);
    const int64_t row0 = t0 + (lo - first);

    const int NT = a.tokens, HP = TEAMS / NT;              // tokens and heads at a time
    const int tid = threadIdx.x, c = tid % TEAM, team = tid / TEAM;
    const int tk = team % NT, slot = team / NT;
    const bool il = a.interleaved != 0;

    // ---- cosine and sine of this lane's pairs, shared by the workgroup's heads ----
    float co[NI][8], si[NI][8];
    bool live[NI];
#pragma unroll
    for (int j = 0; j < NI; j++) {
        const int tt = tk + j * NT;
        live[j] = tt < nt;
        if (!live[j]) continue;
        const int32_t *p = a.pos + (row0 + tt) * a.ld_pos;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int ax = min((uint32_t)a.axis[8 * c + i], (uint32_t)(a.n_axes - 1));
            const double turns = (double)p[ax] * (a.freq[8 * c + i] * 0.15915494309189533577);   // 1 / (2 pi)
            sincospif(2.0f * (float)(turns - rint(turns)), &si[j][i], &co[j][i]);
        }
    }

    const bool is_q = chunk < a.q_chunks;
    const float *weight = is_q ? a.q_weight : a.k_weight;
    float w[16];
    if (weight) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            w[i] = weight[il ? 16 * c + 2 * i : 8 * c + i];
            w[8 + i] = weight[il ? 16 * c + 2 * i + 1 : D / 2 + 8 * c + i];
        }
    }
    const uint16_t *qkv = static_cast<const uint16_t *>(a.qkv);

    if (is_q) {
        const int h1 = min((chunk + 1) * a.q_run, a.Hq);
        for (int h = chunk * a.q_run + slot; h < h1; h += HP) {
#pragma unroll
            for (int j = 0; j < NI; j++) {
                if (!live[j]) continue;                    // whole teams
                const int64_t row = row0 + tk + j * NT;
                float x[16];
                load16<DT, D>(qkv + row * a.ld_qkv + (int64_t)h * D, c, il, x);
                if (weight) norm16<D>(x, w, a.eps);
                turn16(x, co[j], si[j]);
                uint16_t *o = static_cast<uint16_t *>(a.q_out) + row * a.ld_q + (int64_t)h * D;
                u32x4v s0, s1;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    s0[i] = il ? pack16<DT>(x[i], x[8 + i]) : pack16<DT>(x[2 * i], x[2 * i + 1]);
                    s1[i] = il ? pack16<DT>(x[4 + i], x[12 + i]) : pack16<DT>(x[8 + 2 * i], x[9 + 2 * i]);
                }
                *reinterpret_cast<u32x4v *>(o + (il ? 16 * c : 8 * c)) = s0;
                *reinterpret_cast<u32x4v *>(o + (il ? 16 * c + 8 : D / 2 + 8 * c)) = s1;
            }
        }
        return;
    }

    // ---- keys and values ----
    const int64_t page = batch_page(a.batch, b, pg);
    if (kv < n || page < 0) return;                        // nowhere to put them
    const int kc = chunk - a.q_chunks;
    const int h0 = kc * a.kv_run, h1 = min(h0 + a.kv_run, a.Hkv);
    int parity = 0;
    if (tid < 4 * TEAMS) (&amax[0][0][0])[tid] = 0;
    __syncthreads();
    for (int hb = h0; hb < h1; hb += HP) {
        const int h = hb + slot;
        const bool on = h < h1;
        float k[NI][16], v[NI][16];
        uint32_t mk = 0, mv = 0;
#pragma unroll
        for (int j = 0; j < NI; j++) {
            if (!on || !live[j]) continue;
            const uint16_t *r = qkv + (row0 + tk + j * NT) * a.ld_qkv;
            load16<DT, D>(r + (int64_t)(a.Hq + h) * D, c, il, k[j]);
            load16<DT, D>(r + (int64_t)(a.Hq + a.Hkv + h) * D, c, 0, v[j]);
            if (weight) norm16<D>(k[j], w, a.eps);
            turn16(k[j], co[j], si[j]);
            mk = max(mk, amax16(k[j]));
            mv = max(mv, amax16(v[j]));
        }
        if (on && (live[0])) {
            atomicMax(&amax[parity][0][slot], mk);
            atomicMax(&amax[parity][1][slot], mv);
        }
        __syncthreads();
        const float need_k = page_scale(amax[parity][0][slot]), need_v = page_scale(amax[parity][1][slot]);
        if (tid < 2 * TEAMS) (&amax[parity ^ 1][0][0])[tid] = 0;   // the next step's (read before the last barrier)
        parity ^= 1;
        float sk = need_k, sv = need_v;
        const int64_t at = page * a.Hkv + h;
        uint8_t *kp = a.k + at * (kPage * D), *vp = a.v + at * (kPage * D);
        float fk = 1.0f, fv = 1.0f;
        if (on && off0 > 0) {                              // older tokens: the scale only grows
            const float ok = a.k_scale[at], ov = a.v_scale[at];
            sk = fmaxf(ok, need_k);
            sv = fmaxf(ov, need_v);
            fk = ok / sk;
            fv = ov / sv;
        }
        __syncthreads();                                   // every lane has the old scales
        if (on) {
            const int lane = tk * TEAM + c, lanes = NT * TEAM;   // this head's lanes
            if (fk != 1.0f)
                for (int i = lane; i < off0 * D; i += lanes) kp[i] = rescale1(kp[i], fk);
            if (fv != 1.0f)
                for (int i = lane; i < off0 * D; i += lanes) {
                    uint8_t *q = vp + (i / off0) * kPage + i % off0;
                    *q = rescale1(*q, fv);
                }
            if (lane == 0) {
                a.k_scale[at] = sk;
                a.v_scale[at] = sv;
            }
        }
        const float ik = 1.0f / sk, iv = 1.0f / sv;
        const bool whole = nt == kPage && HP == 1;         // a full page of one head: values through LDS
#pragma unroll
        for (int j = 0; j < NI; j++) {
            if (!on || !live[j]) continue;
            const int tt = off0 + tk + j * NT;
            uint8_t *o = kp + tt * D;
            const float(&x)[16] = k[j];
            if (il) {
                u32x4v s;
#pragma unroll
                for (int i = 0; i < 4; i++) s[i] = encode4(x[2 * i], x[8 + 2 * i], x[2 * i + 1], x[9 + 2 * i], ik);
                *reinterpret_cast<u32x4v *>(o + 16 * c) = s;
            } else {
                u32x2v s0, s1;
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    s0[i] = encode4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3], ik);
                    s1[i] = encode4(x[8 + 4 * i], x[9 + 4 * i], x[10 + 4 * i], x[11 + 4 * i], ik);
                }
                *reinterpret_cast<u32x2v *>(o + 8 * c) = s0;
                *reinterpret_cast<u32x2v *>(o + D / 2 + 8 * c) = s1;
            }
#pragma unroll
            for (int g = 0; g < 4; g++) {                  // v: registers 0..7 dims 8c.., 8..15 dims D/2 + 8c..
                const uint32_t e = encode4(v[j][4 * g], v[j][4 * g + 1], v[j][4 * g + 2], v[j][4 * g + 3], iv);
                const int d = (g >= 2 ? D / 2 : 0) + 8 * c + 4 * (g & 1);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (whole) vtile[(d + i) * VROW + tt] = (uint8_t)(e >> (8 * i));
                    else vp[(d + i) * kPage + tt] = (uint8_t)(e >> (8 * i));
                }
            }
        }
        if (whole) {                                       // uniform
            __syncthreads();
            for (int i = tid; i < D * 4; i += 256) {
                const uint32_t *s = reinterpret_cast<const uint32_t *>(vtile + (i >> 2) * VROW + 16 * (i & 3));
                *reinterpret_cast<u32x4v *>(vp + 16 * i) = u32x4v{s[0], s[1], s[2], s[3]};
            }
            // the next step's first barrier orders these reads before its writes of the tile
        }
    }
}

template <int DT, int D>
static hipError_t launch_rope(RopeArgs a, int64_t B, int64_t max_new, int cus, hipStream_t st)
{
    constexpr int TEAMS = 256 / (D / 16);
    int nt = 1;
    while (nt < max_new && nt < kPage && nt < TEAMS) nt *= 2;
    a.tokens = nt;
    const int hp = TEAMS / nt;
    a.visits = (int)((max_new + kPage - 2) / kPage + 1);
    // heads per workgroup: a multiple of those it takes at a time, as many as leave four
    // workgroups for every compute unit (the sines are then shared by more heads), at most 8 steps
    const int64_t pages = B * a.visits;
    auto chunks = [&](int run) { return (a.Hq + run - 1) / run + (a.Hkv + run - 1) / run; };
    int run = hp;
    while (run < 8 * hp && pages * chunks(2 * run) >= 4 * (int64_t)cus) run *= 2;
    a.q_run = a.kv_run = run;
    a.q_chunks = (a.Hq + run - 1) / run;
    a.chunks = chunks(run);
    const int64_t blocks = pages * a.chunks;
    if (blocks > (int64_t)(UINT32_MAX / 256)) return hipErrorInvalidValue;
    if (max_new > nt) hipLaunchKernelGGL((rope_append_kernel<DT, D, kPage / TEAMS < 1 ? 1 : kPage / TEAMS>), dim3((unsigned)blocks), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((rope_append_kernel<DT, D, 1>), dim3((unsigned)blocks), dim3(256), 0, st, a);
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
    a.n_axes = r.n_axes; a.Hq = r.Hq; a.Hkv = r.Hkv; a.eps = r.eps; a.interleaved = r.interleaved;
    if (r.D == 128) return r.dtype == 0 ? launch_rope<0, 128>(a, r.B, r.max_new, r.cus, st) : launch_rope<1, 128>(a, r.B, r.max_new, r.cus, st);
    return r.dtype == 0 ? launch_rope<0, 64>(a, r.B, r.max_new, r.cus, st) : launch_rope<1, 64>(a, r.B, r.max_new, r.cus, st);
}

}  // namespace convrot
