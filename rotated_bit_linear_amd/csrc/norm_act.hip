// RMS norm of a residual stream fused into the S8 activation preparation:
//   h = round(x + r) to the stream's type (r optional; h written when asked for),
//   y[k] = h[k] * w[k] * rstd, rstd = 1 / sqrt(mean(h^2) + eps),
//   ConvRot256 of y and its row quantization.
// The rotation is linear and a row's codes do not change when the row is multiplied by a
// constant, so rstd never touches an element: with z the butterflies of h * w (before the
// 1/16), the codes are those of z and the scale is (max|z| / 16 / 127) * rstd.  That leaves
// one pass and one barrier a row (the maximum of |z| and the sum of squares are reduced
// together; normalising first would need the sum before the rotation and the maximum after
// it), and codes that depend on no order of summation: products and butterflies are the
// FP32 operations of the definition, bit for bit.
// The sum of squares is held in FP64: the squares of FP32 values are exact there, so neither
// large rows (|h| above 1.8e19) overflow nor small ones vanish, and the sum's order changes
// x_scale by at most an ulp.  One FP64 FMA an element is hidden under the loads.
//
// Bound by HBM: x, r and h in two (four) bytes and one byte of code an element; without a
// residual, 16-bit rows come as near to the vector units' rate (27 operations an element).
// Work split: a 16-lane group per 256-column block as in row_prep.hpp, whole rows in registers
// up to 64 blocks (K_pad 16384; two blocks a group spill beside the second operand and the
// weights), several short rows a workgroup, the next rows requested while this one is rotated;
// longer rows are streamed twice.
// Measured: 19989 x 5376 bf16 with a residual 136 us (5.5 TB/s, a 1 GiB copy runs at 5.1), without
// 62 (5.2); 4096 x 14336 fp32 43 (6.9, partly from the last-level cache; 47 to 50 on rows not
// there); 21841 x 5377 bf16 173 (4.8); 4096 x 20000 bf16, streamed twice, 175 (3.3); one row 4.3.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "elem_load.hpp"
#include "kernels.hpp"
#include "row_prep.hpp"

namespace convrot {

template <int DT>
struct NormArgs {
    using T = typename Elem<DT>::T;
    const T *x;              // no restrict: sum may be x or r (each element is read before it is written)
    const T *r;
    T *sum;
    const float *w;
    int64_t ld_x, ld_r, ld_sum;
    int64_t K;
    double eps;
};

// Elements [k0, k0 + 16) of a row.  Past K: zeros in whole 16-byte chunks; what a chunk holds
// beyond K is cut by cut_segment once the loads have arrived.  Such a chunk may be read where
// another row follows (a row's stride covers it, `more`); the last row's elements are read one
// by one, from clamped places, all in flight at once.
// Ordinary loads: a segment is two or four 16-byte loads, each of which touches every cache
// line of the wave's run, and non-temporal ones fetch lines again that are still wanted
// (19989 x 5376 bf16 with a residual 157 against 141 us, 4096 x 14336 fp32 76 against 50 us).
template <int DT>
__device__ __forceinline__ void fetch_stream(const typename Elem<DT>::T *row, int64_t k0, int64_t K, bool more, RawSeg<DT> &r)
{
    constexpr int NW = DT == 2 ? 4 : 2;                      // 16-byte chunks
    if (k0 + 16 <= K) {
#pragma unroll
        for (int c = 0; c < NW; c++) r.w[c] = *(reinterpret_cast<const u32x4 *>(row + k0) + c);
        return;
    }
    if (k0 >= K || more) {
        const int rem = opaque(k0 < K ? (int)(K - k0) : 0);
#pragma unroll
        for (int c = 0; c < NW; c++) {
            if (16 / NW * c < rem) r.w[c] = *(reinterpret_cast<const u32x4 *>(row + k0) + c);
            else r.w[c] = u32x4{0u, 0u, 0u, 0u};
        }
        return;
    }
    const int rem = opaque((int)(K - k0));                   // 1 .. 15
    uint32_t e[16];
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const auto *p = row + k0 + min(i, rem - 1);
        if constexpr (DT == 2) e[i] = __float_as_uint(*p);
        else e[i] = *p;
    }
    if constexpr (DT == 2) {
#pragma unroll
        for (int i = 0; i < 16; i++) r.w[i >> 2][i & 3] = e[i];
    } else {
#pragma unroll
        for (int i = 0; i < 16; i += 2) r.w[i >> 3][(i >> 1) & 3] = e[i] | (e[i + 1] << 16);
    }
}

// zeros past K
template <int DT>
__device__ __forceinline__ void cut_segment(int64_t k0, int64_t K, RawSeg<DT> &r)
{
    if (k0 + 16 <= K || k0 >= K) return;
    const int rem = opaque((int)(K - k0));                   // 1 .. 15; its comparisons are not kept over the rows
    if constexpr (DT == 2) {
#pragma unroll
        for (int i = 0; i < 16; i++) r.w[i >> 2][i & 3] = i < rem ? r.w[i >> 2][i & 3] : 0u;
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) r.w[i >> 2][i & 3] &= 2 * i + 1 < rem ? 0xffffffffu : 2 * i < rem ? 0xffffu : 0u;
    }
}

// h = x + r of one segment, in FP32 and rounded to the stream's type (raw bytes in r0)
template <int DT>
__device__ __forceinline__ void add_segment(RawSeg<DT> &r0, const RawSeg<DT> &r1)
{
    if constexpr (DT == 2) {
#pragma unroll
        for (int i = 0; i < 16; i++)
            r0.w[i >> 2][i & 3] = __float_as_uint(__uint_as_float(r0.w[i >> 2][i & 3]) + __uint_as_float(r1.w[i >> 2][i & 3]));
    } else {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float a = seg_elem<DT>(r0, i) + seg_elem<DT>(r1, i);
            const float b = seg_elem<DT>(r0, i + 1) + seg_elem<DT>(r1, i + 1);
            uint32_t lo, hi;
            if constexpr (DT == 0) {
                lo = __bfloat16_as_ushort(__float2bfloat16(a));
                hi = __bfloat16_as_ushort(__float2bfloat16(b));
            } else {
                lo = __half_as_ushort(__float2half(a));
                hi = __half_as_ushort(__float2half(b));
            }
            r0.w[i >> 3][(i >> 1) & 3] = lo | (hi << 16);
        }
    }
}

// a segment's raw bytes to row + k0: 16-byte stores below K, the chunk across K in 8, 4 and 2
// bytes (28567 rows of 4111 bf16 with stores of 15 single elements: 262 us)
template <int DT>
__device__ __forceinline__ void store_seg(typename Elem<DT>::T *row, int64_t k0, int64_t K, const RawSeg<DT> &r)
{
    constexpr int NW = DT == 2 ? 4 : 2, E = 16 / NW;         // chunks, elements of one
    uint8_t *to = reinterpret_cast<uint8_t *>(row + k0);
    if (k0 + 16 <= K) {
#pragma unroll
        for (int c = 0; c < NW; c++) *(reinterpret_cast<u32x4 *>(to) + c) = r.w[c];
        return;
    }
    if (k0 >= K) return;
    const int rem = opaque((int)(K - k0));                   // 1 .. 15
#pragma unroll
    for (int c = 0; c < NW; c++) {
        const int n = rem - E * c;                           // elements of this chunk below K
        if (n >= E) {
            *(reinterpret_cast<u32x4 *>(to) + c) = r.w[c];
        } else if (n > 0) {
            const int bytes = n * (16 / E);
            uint32_t w = r.w[c][0];                          // the word after those stored so far
            uint8_t *at = to + 16 * c;
            if (bytes & 8) {
                *reinterpret_cast<uint2 *>(at) = make_uint2(r.w[c][0], r.w[c][1]);
                w = r.w[c][2];
                at += 8;
            }
            if (bytes & 4) {
                *reinterpret_cast<uint32_t *>(at) = w;
                w = (bytes & 8) ? r.w[c][3] : r.w[c][1];
                at += 4;
            }
            if (bytes & 2) *reinterpret_cast<uint16_t *>(at) = (uint16_t)w;
        }
    }
}

struct NormWeights { float c[16]; };

// weights of a segment (1 where there are none); past K cut_weights follows
__device__ __forceinline__ void load_weights(const float *w, int64_t k0, int64_t K, NormWeights &n)
{
    if (w && k0 + 16 <= K) {
        __builtin_memcpy(n.c, w + k0, 64);               // 4-byte aligned
        return;
    }
    const int rem = opaque((int)(K - k0 < 16 ? K - k0 : 16));
#pragma unroll
    for (int i = 0; i < 16; i++) n.c[i] = 1.0f;
    if (w && rem > 0) {
#pragma unroll
        for (int i = 0; i < 16; i++) n.c[i] = w[k0 + min(i, rem - 1)];
    }
}

// 0 past K: an element there is 0, but the weight may be an infinity or a NaN
__device__ __forceinline__ void cut_weights(int64_t k0, int64_t K, NormWeights &n)
{
    if (k0 + 16 <= K) return;
    const int rem = (int)(K - k0);
#pragma unroll
    for (int i = 0; i < 16; i++) n.c[i] = i < rem ? n.c[i] : 0.0f;
}

// sum over the 16 lanes of a group, the same bits in every lane (the DPP exchanges of group16_umax)
__device__ __forceinline__ double group16_sum(double v)
{
    auto step = [](double x, auto ctrl) {
        constexpr int C = decltype(ctrl)::value;
        const uint64_t b = (uint64_t)__double_as_longlong(x);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, C, 0xF, 0xF, true);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), C, 0xF, 0xF, true);
        return x + __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
    };
    v = step(v, std::integral_constant<int, 0xB1>{});
    v = step(v, std::integral_constant<int, 0x4E>{});
    v = step(v, std::integral_constant<int, 0x141>{});
    return step(v, std::integral_constant<int, 0x140>{});
}

__device__ __forceinline__ float norm_scale(const RowQuant &q, double sumsq, int64_t K, double eps)
{
    if (q.scale == 0.0f) return 0.0f;            // a zero row, whatever rstd is
    return q.scale * (float)(1.0 / sqrt(sumsq / (double)K + eps));
}

// decoded segment: v = h * w, and the squares of h added to ss
template <int DT>
__device__ __forceinline__ void weigh(const RawSeg<DT> &h, const NormWeights &w, float (&v)[16], double &ss)
{
    decode_seg<DT>(h, v);
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const double d = (double)v[i];
        ss = __builtin_fma(d, d, ss);
        v[i] = v[i] * w.c[i];
    }
}

// computes v and ss here, so that what they came from is no longer needed
__device__ __forceinline__ void pin(float (&v)[16], double &ss)
{
#pragma unroll
    for (int i = 0; i < 16; i++) asm volatile("" : "+v"(v[i]));
    asm volatile("" : "+v"(ss));
}

// LDS of a workgroup of G groups: G transpose tiles, then two sets (for alternate rows) of G
// sums and G maxima
__host__ __device__ constexpr size_t norm_lds_bytes(int groups)
{
    return (size_t)groups * (kTileStrideF * sizeof(float) + 2 * (sizeof(double) + sizeof(float)));
}

struct NormReduce {
    double *sums;
    uint32_t *maxs;
    __device__ __forceinline__ NormReduce(float *lds, int G, int parity)
    {
        double *d = reinterpret_cast<double *>(lds + G * kTileStrideF);
        sums = d + parity * G;
        maxs = reinterpret_cast<uint32_t *>(d + 2 * G) + parity * G;
    }
    // this group's part in, the row's maximum and sum out (groups g0 .. g0 + n - 1, n <= 64)
    __device__ __forceinline__ void put(int grp, int t, float zmax, double ss)
    {
        zmax = group16_max(zmax);
        ss = group16_sum(ss);
        if (t == 0) { sums[grp] = ss; maxs[grp] = __float_as_uint(zmax); }
    }
    __device__ __forceinline__ float row_max(int g0, int n, int t) const
    {
        uint32_t z = 0;
        for (int i = t; i < n; i += 16) z = max(z, maxs[g0 + i]);
        return __uint_as_float(group16_umax(z));
    }
    __device__ __forceinline__ double row_sum(int g0, int n, int t) const
    {
        double s = 0.0;
        for (int i = t; i < n; i += 16) s += sums[g0 + i];
        return group16_sum(s);
    }
};

// Rows of nb <= 64 blocks, one 16-lane group each, rpw rows a workgroup.
template <int DT, bool kRes>
__global__ __launch_bounds__(1024) void norm_rows_kernel(NormArgs<DT> a, int64_t n_rows, int nb, int rpw,
                                                         int8_t *__restrict__ out, int64_t ld_out,
                                                         float *__restrict__ scale, int natural)
{
    extern __shared__ float lds[];
    const int grp = threadIdx.x >> 4, t = threadIdx.x & 15;
    const int G = blockDim.x >> 4;
    float *tile = lds + grp * kTileStrideF;
    const int slot = grp / nb, b = grp - slot * nb;
    const bool active = slot < rpw;
    const int64_t k0 = ((int64_t)b * 16 + t) * 16;
    NormWeights w;
    load_weights(a.w, k0, a.K, w);

    RawSeg<DT> x = {}, r = {};                       // zero in lanes that hold no row: they store nothing
    auto fetch = [&](int64_t row) {
        if (!active || row >= n_rows) return;
        fetch_stream<DT>(a.x + row * a.ld_x, k0, a.K, row + 1 < n_rows, x);
        if constexpr (kRes) fetch_stream<DT>(a.r + row * a.ld_r, k0, a.K, row + 1 < n_rows, r);
    };
    const int64_t step = (int64_t)gridDim.x * rpw;
    int64_t base = (int64_t)blockIdx.x * rpw;
    fetch(base + slot);
    cut_weights(k0, a.K, w);
    int parity = 0;
    // codes are stored after the next row's arrival: a wait for its loads would also wait for
    // stores issued after them
    bool pending = false;
    int8_t *dst = out;
    u32x4 codes = {};
    for (; base < n_rows; base += step) {
        const int64_t row = base + slot;
        const bool live = active && row < n_rows;
        float v[16], zmax = 0.0f;
        double ss = 0.0;
        cut_segment<DT>(k0, a.K, x);
        if constexpr (kRes) {
            cut_segment<DT>(k0, a.K, r);
            add_segment<DT>(x, r);
            if (live && a.sum) store_seg<DT>(a.sum + row * a.ld_sum, k0, a.K, x);
        }
        weigh<DT>(x, w, v, ss);
        pin(v, ss);                                  // x is free: the next row lands in the same registers
        if (pending) __builtin_nontemporal_store(codes, reinterpret_cast<u32x4 *>(dst));
        fetch(row + step);
        hadamard256(v, tile, t, natural != 0);
#pragma unroll
        for (int i = 0; i < 16; i++) zmax = fmaxf(zmax, fabsf(v[i]));
        NormReduce red(lds, G, parity);
        red.put(grp, t, zmax, ss);
        __syncthreads();
        parity ^= 1;
        pending = live;
        if (!live) continue;                         // whole 16-lane groups: the DPP steps stay inside active rows
        const RowQuant rq = row_quant<8>(red.row_max(slot * nb, nb, t));
        dst = out + row * ld_out + 16 * (16 * (int64_t)b + t);
        store_codes(v, rq, reinterpret_cast<int8_t *>(&codes));
        if (b == 0) {
            const double s = red.row_sum(slot * nb, nb, t);
            if (t == 0) scale[row] = norm_scale(rq, s, a.K, a.eps);
        }
    }
    if (pending) __builtin_nontemporal_store(codes, reinterpret_cast<u32x4 *>(dst));
}

// Rows streamed twice: pass 1 forms h (and writes it), its squares and the rotated maximum;
// pass 2 reads h (the one written, or x and r again), rotates and quantizes.
template <int DT, bool kRes>
__global__ __launch_bounds__(1024) void norm_two_pass_kernel(NormArgs<DT> a, int64_t n_rows, int nb,
                                                             int8_t *__restrict__ out, int64_t ld_out,
                                                             float *__restrict__ scale, int natural)
{
    extern __shared__ float lds[];
    const int grp = threadIdx.x >> 4, t = threadIdx.x & 15;
    const int G = blockDim.x >> 4;
    float *tile = lds + grp * kTileStrideF;
    const int slices = (nb + G - 1) / G;
    auto fetch = [&](const typename Elem<DT>::T *p, int64_t ld, int64_t row, int64_t k0, RawSeg<DT> &seg) {
        fetch_stream<DT>(p + row * ld, k0, a.K, row + 1 < n_rows, seg);
        cut_segment<DT>(k0, a.K, seg);
    };
    int parity = 0;
    for (int64_t row = blockIdx.x; row < n_rows; row += gridDim.x) {
        float v[16], zmax = 0.0f;
        double ss = 0.0;
        NormWeights w;
        for (int s = 0; s < slices; s++) {
            const int64_t k0 = ((int64_t)(s * G + grp) * 16 + t) * 16;
            RawSeg<DT> x, r;
            fetch(a.x, a.ld_x, row, k0, x);
            if constexpr (kRes) {
                fetch(a.r, a.ld_r, row, k0, r);
                add_segment<DT>(x, r);
                if (a.sum) store_seg<DT>(a.sum + row * a.ld_sum, k0, a.K, x);
            }
            load_weights(a.w, k0, a.K, w);
            cut_weights(k0, a.K, w);
            weigh<DT>(x, w, v, ss);
            hadamard256(v, tile, t, natural != 0);
#pragma unroll
            for (int i = 0; i < 16; i++) zmax = fmaxf(zmax, fabsf(v[i]));
        }
        NormReduce red(lds, G, parity);
        red.put(grp, t, zmax, ss);
        __syncthreads();
        parity ^= 1;
        const RowQuant rq = row_quant<8>(red.row_max(0, G, t));
        for (int s = 0; s < slices; s++) {
            const int b = s * G + grp;
            const int64_t k0 = ((int64_t)b * 16 + t) * 16;
            RawSeg<DT> x, r;
            if (kRes && a.sum) {
                fetch(a.sum, a.ld_sum, row, k0, x);   // this thread's own stores
            } else {
                fetch(a.x, a.ld_x, row, k0, x);
                if constexpr (kRes) {
                    fetch(a.r, a.ld_r, row, k0, r);
                    add_segment<DT>(x, r);
                }
            }
            double unused = 0.0;
            load_weights(a.w, k0, a.K, w);
            cut_weights(k0, a.K, w);
            weigh<DT>(x, w, v, unused);
            hadamard256(v, tile, t, natural != 0);
            if (b < nb) store_codes<8>(v, rq, out + row * ld_out, b, t);
        }
        if (grp == 0) {
            const double s = red.row_sum(0, G, t);
            if (t == 0) scale[row] = norm_scale(rq, s, a.K, a.eps);
        }
    }
}

template <int DT, bool kRes>
static hipError_t launch_norm(const NormArgs<DT> &a, int64_t M, int8_t *out, int64_t ld_out, float *scale,
                              bool force_two_pass, bool natural, int cus, hipStream_t st)
{
    const int nb = (int)((a.K + 255) / 256);
    if (force_two_pass || nb > kMaxGroupsWide) {
        const int slices = (nb + kMaxGroups1 - 1) / kMaxGroups1;
        const int threads = ((nb + slices - 1) / slices + 3) / 4 * 64;
        const dim3 grid((unsigned)(M < kTwoPassMaxGrid ? M : kTwoPassMaxGrid));
        hipLaunchKernelGGL((norm_two_pass_kernel<DT, kRes>), grid, dim3(threads), norm_lds_bytes(threads / 16), st, a,
                           M, nb, out, ld_out, scale, natural);
        return hipGetLastError();
    }
    // rows a workgroup: the fewest rounds over the device, 4 waves of this kernel a SIMD, of which
    // a workgroup of 4 waves or more takes equally many on each (short batches: a row each; long
    // ones: the packing that leaves the fewest lanes idle).  25530 rows of 4600 bf16: one row in 5
    // waves, as 16 waves a compute unit would suggest, 232 us, three in 14 180 us
    int rpw = 1;
    int64_t best = INT64_MAX;
    for (int n = 1; n * nb <= kMaxGroupsWide; n++) {
        const int waves = (n * nb + 3) / 4, groups = waves < 4 ? 16 / waves : 4 / ((waves + 3) / 4);
        const int64_t at_once = (int64_t)cus * groups * n, rounds = (M + at_once - 1) / at_once;
        if (rounds < best) { best = rounds; rpw = n; }
    }
    const int threads = (rpw * nb + 3) / 4 * 64;
    const size_t lds = norm_lds_bytes(threads / 16);
    const RowPrepShape s{threads, 1, false, false};
    const void *k = reinterpret_cast<const void *>(&norm_rows_kernel<DT, kRes>);
    const dim3 grid((unsigned)row_prep_grid((M + rpw - 1) / rpw, s, k, lds));
    hipLaunchKernelGGL((norm_rows_kernel<DT, kRes>), grid, dim3(threads), lds, st, a, M, nb, rpw, out, ld_out, scale,
                       natural);
    return hipGetLastError();
}

template <int DT>
static hipError_t launch_norm_dt(const void *x, int64_t ld_x, const void *r, int64_t ld_r, void *sum, int64_t ld_sum,
                                 const float *w, float eps, int64_t M, int64_t K, int8_t *out, int64_t ld_out,
                                 float *scale, bool two_pass, bool natural, int cus, hipStream_t st)
{
    using T = typename Elem<DT>::T;
    const NormArgs<DT> a{static_cast<const T *>(x), static_cast<const T *>(r), static_cast<T *>(sum), w, ld_x, ld_r,
                         ld_sum, K, (double)eps};
    return r ? launch_norm<DT, true>(a, M, out, ld_out, scale, two_pass, natural, cus, st)
             : launch_norm<DT, false>(a, M, out, ld_out, scale, two_pass, natural, cus, st);
}

hipError_t launch_quant_act_rmsnorm(const void *x, int dtype, int64_t ld_x, const void *r, int64_t ld_r, void *sum,
                                    int64_t ld_sum, const float *w, float eps, int64_t M, int64_t K, int8_t *x_s8,
                                    int64_t ld_s8, float *x_scale, bool two_pass, bool transposed, int cus,
                                    hipStream_t st)
{
    switch (dtype) {
    case 0: return launch_norm_dt<0>(x, ld_x, r, ld_r, sum, ld_sum, w, eps, M, K, x_s8, ld_s8, x_scale, two_pass, !transposed, cus, st);
    case 1: return launch_norm_dt<1>(x, ld_x, r, ld_r, sum, ld_sum, w, eps, M, K, x_s8, ld_s8, x_scale, two_pass, !transposed, cus, st);
    case 2: return launch_norm_dt<2>(x, ld_x, r, ld_r, sum, ld_sum, w, eps, M, K, x_s8, ld_s8, x_scale, two_pass, !transposed, cus, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace convrot
