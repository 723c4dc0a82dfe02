// Products of the experts' rows with the experts' 4-bit weights:
//   C[r, n] = ((float)sum_k A[s, k] W_e[n, k] * a_scale[s]) * b_scale[e, n] (+ bias[e, n])
// for the rows of each expert e, s the row of A and r the row of C that a place in the order names;
// with SwiGLU, swish of the first half of the columns times the second half.
// Weights and sums as in gemm_s8s4.hip: nibbles widened to bytes 16 q, int32 sums of 16 q a.
#include <hip/hip_runtime.h>
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <stdint.h>

#include "experts.hpp"
#include "kernels.hpp"
#include "swiglu.hpp"

namespace convrot {
namespace {

typedef int32_t v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4i widen(uint32_t d0, uint32_t d1)
{
    constexpr uint32_t hi = 0xF0F0F0F0u;
    return v4i{(int32_t)((d0 << 4) & hi), (int32_t)(d0 & hi), (int32_t)((d1 << 4) & hi), (int32_t)(d1 & hi)};
}

// four neighbouring columns n .. n+3 of a row, rounded once to the output type
template <int OUT>
__device__ __forceinline__ void store4(void *C, int64_t at, const v4f &v, const v4i &raw, int left, bool vec)
{
    if constexpr (OUT == 0 || OUT == 1) {
        uint16_t *out = static_cast<uint16_t *>(C) + at;
        uint16_t h[4];
#pragma unroll
        for (int r = 0; r < 4; r++) {
            if constexpr (OUT == 0) h[r] = __bfloat16_as_ushort(__float2bfloat16(v[r]));
            else h[r] = __half_as_ushort(__float2half(v[r]));
        }
        if (vec && left >= 4) {
            *reinterpret_cast<uint2 *>(out) = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
            return;
        }
#pragma unroll
        for (int r = 0; r < 4; r++)
            if (r < left) out[r] = h[r];
    } else {
        uint32_t *out = static_cast<uint32_t *>(C) + at;
        if (vec && left >= 4) {
            if constexpr (OUT == 3) *reinterpret_cast<v4i *>(out) = raw;
            else *reinterpret_cast<v4f *>(out) = v;
            return;
        }
#pragma unroll
        for (int r = 0; r < 4; r++)
            if (r < left) out[r] = OUT == 3 ? (uint32_t)raw[r] : __float_as_uint(v[r]);
    }
}

// A workgroup takes 16 MT rows of an expert and 32 weight rows (with SwiGLU 16 gates and their 16
// values); its four waves share out K, each in whole lines of the weight, and add their sums in LDS.
// Both operands go straight to registers in the order of the matrix instruction (16 x 16 x 64, weight
// first): quarter q of a wave's lanes takes bytes 16 q of 64 of a packed row, two groups of 16 codes, one
// for each of two instructions, and the activation's bytes of the same columns.
constexpr int kWaves = 4, kTileN = 32;

template <int OUT, int MT, bool SWIGLU>
__global__ __launch_bounds__(64 * kWaves)
void experts_few_kernel(const ExpertsGemm g)
{
    __shared__ v4i sums[kWaves][2 * MT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, q = lane >> 4;
    constexpr int LG = MT == 1 ? 4 : 5;
    ExpertBlock blk;
    if (!find_block(g.offsets, g.E, g.S, LG, (int)(blockIdx.x / g.n_tiles), lane, blk)) return;
    const int half = SWIGLU ? g.N >> 1 : 0;
    const int n0 = (int)(blockIdx.x % g.n_tiles) * (SWIGLU ? kTileN / 2 : kTileN);
    const int n_end = SWIGLU ? half : g.N;

    const uint8_t *wp[2];
#pragma unroll
    for (int f = 0; f < 2; f++) {
        const int n = min(n0 + (SWIGLU ? 0 : 16 * f) + col, n_end - 1) + (SWIGLU && f ? half : 0);
        wp[f] = g.B + (int64_t)blk.e * g.stride_b + (int64_t)n * g.ldb + 16 * q;
    }
    const int8_t *ap[MT];
#pragma unroll
    for (int m = 0; m < MT; m++) {
        const int i = blk.row + 16 * m + col;
        const int r = i < blk.end ? row_from(g, i) : -1;
        ap[m] = g.A + (int64_t)max(r, 0) * g.lda + 64 * (q >> 1) + 16 * (q & 1);
    }
    v4i acc[2][MT];
#pragma unroll
    for (int f = 0; f < 2; f++)
#pragma unroll
        for (int m = 0; m < MT; m++) acc[f][m] = v4i{0, 0, 0, 0};

    for (int kb = wave; kb < g.K_pad / 256; kb += kWaves) {
        v4i w[2][2], a[MT][4];
#pragma unroll
        for (int f = 0; f < 2; f++)
#pragma unroll
            for (int s = 0; s < 2; s++) w[f][s] = *reinterpret_cast<const v4i *>(wp[f] + kb * 128 + s * 64);
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int s = 0; s < 4; s++)
                a[m][s] = *reinterpret_cast<const v4i *>(ap[m] + (int64_t)kb * 256 + (s >> 1) * 128 + (s & 1) * 32);
#pragma unroll
        for (int s = 0; s < 4; s++)
#pragma unroll
            for (int f = 0; f < 2; f++) {
                const v4i wide = widen((uint32_t)w[f][s >> 1][2 * (s & 1)], (uint32_t)w[f][s >> 1][2 * (s & 1) + 1]);
#pragma unroll
                for (int m = 0; m < MT; m++)
                    acc[f][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wide, a[m][s], acc[f][m], 0, 0, 0);
            }
    }
#pragma unroll
    for (int f = 0; f < 2; f++)
#pragma unroll
        for (int m = 0; m < MT; m++) sums[wave][2 * m + f][lane] = acc[f][m];
    __syncthreads();

    // lane l of a fragment holds row l % 16 and columns 4 (l / 16) .. +3
    const bool vec = g.vec;
    auto total = [&](int p) {
        v4i t = sums[0][p][lane];
#pragma unroll
        for (int w = 1; w < kWaves; w++) t += sums[w][p][lane];
        return t >> 4;
    };
    auto scaled = [&](const v4i &t, float sa, int n, int left) {
        v4f v;
        const int64_t at = (int64_t)blk.e * g.N + n;
#pragma unroll
        for (int r = 0; r < 4; r++) {
            v[r] = r < left ? ((float)t[r] * sa) * g.sb[at + r] : 0.0f;
            if (g.bias && r < left) v[r] += g.bias[at + r];
        }
        return v;
    };
    for (int p = wave; p < (SWIGLU ? MT : 2 * MT); p += kWaves) {
        const int m = SWIGLU ? p : p >> 1;
        const int i = blk.row + 16 * m + col;
        const int from = i < blk.end ? row_from(g, i) : -1, to = i < blk.end ? row_to(g, i) : -1;
        const int n = n0 + (SWIGLU ? 0 : 16 * (p & 1)) + 4 * q;
        const int left = n_end - n;
        if (from < 0 || to < 0 || left <= 0) continue;
        const float sa = OUT == 3 ? 0.0f : g.sa[from];
        const int64_t at = (int64_t)to * g.ldc + n;
        if constexpr (SWIGLU) {
            const v4f a = scaled(total(2 * m), sa, n, left), b = scaled(total(2 * m + 1), sa, half + n, left);
            v4f o;
#pragma unroll
            for (int r = 0; r < 4; r++) {
                o[r] = swiglu_elem(a[r], b[r]);
                // the product is rounded to FP32 before it is rounded to fp16, as everywhere in this
                // library: without this the compiler makes one rounding of the two (v_fma_mixlo_f16)
                if constexpr (OUT == 1) asm("" : "+v"(o[r]));
            }
            store4<OUT>(g.C, at, o, v4i{}, left, vec);
        } else {
            const v4i t = total(p);
            store4<OUT>(g.C, at, OUT == 3 ? v4f{} : scaled(t, sa, n, left), t, left, vec);
        }
    }
}

template <int OUT, bool SWIGLU>
hipError_t launch_few(const ExpertsGemm &g, int mt, int64_t blocks, hipStream_t st)
{
    const dim3 grid((unsigned)(blocks * g.n_tiles)), threads(64 * kWaves);
    if (mt == 1) hipLaunchKernelGGL((experts_few_kernel<OUT, 1, SWIGLU>), grid, threads, 0, st, g);
    else hipLaunchKernelGGL((experts_few_kernel<OUT, 2, SWIGLU>), grid, threads, 0, st, g);
    return hipGetLastError();
}

}  // namespace

// Many rows an expert on average: tiles through LDS.
static bool tiled(int64_t S, int64_t E) { return S > 32 * E; }
static int lg_rows(int64_t S, int64_t E) { return S <= 16 * E ? 4 : 5; }

int64_t experts_gemm_blocks(int64_t S, int64_t E, int64_t N, bool)
{
    if (tiled(S, E)) return 2 * experts_tile_blocks(S, E, N);
    return most_blocks(S, E, lg_rows(S, E)) * ((N + kTileN - 1) / kTileN);
}

hipError_t launch_gemm_experts(ExpertsGemm g, int out_dtype, bool swiglu, hipStream_t st)
{
    if (tiled(g.S, g.E)) return launch_experts_tile(g, out_dtype, swiglu, st);
    const int lg = lg_rows(g.S, g.E);
    g.n_tiles = (g.N + kTileN - 1) / kTileN;
    const int es = out_dtype < 2 ? 2 : 4;
    g.vec = (uintptr_t)g.C % (4 * es) == 0 && g.ldc % 4 == 0;
    const int64_t blocks = most_blocks(g.S, g.E, lg);
    const int mt = 1 << (lg - 4);
    switch (out_dtype) {
    case 0: return swiglu ? launch_few<0, true>(g, mt, blocks, st) : launch_few<0, false>(g, mt, blocks, st);
    case 1: return swiglu ? launch_few<1, true>(g, mt, blocks, st) : launch_few<1, false>(g, mt, blocks, st);
    case 2: return swiglu ? launch_few<2, true>(g, mt, blocks, st) : launch_few<2, false>(g, mt, blocks, st);
    case 3: return swiglu ? hipErrorInvalidValue : launch_few<3, false>(g, mt, blocks, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace convrot
