// The experts' second product for one token: each of its choices is one row, and there is nothing to sort.
//
// A workgroup takes one choice and 128 weight rows, 32 a wave.  It rotates and quantizes the choice's row
// between the products for itself, while the first weights are on their way from memory: a launch less (one
// token, 8 of 64 experts, 5376 and 1792 wide: 35.4 -> 32.5 us).  The codes then lie in LDS, so a wave only
// waits for its own weights: no barrier a step.  Bound by HBM and by the launch.
// Products as in gemm_experts.hip: 16 x 16 x 64 with the weights first; all 16 columns are the one row.
// (The first product in this form, its row copied to LDS, takes 2.5 us more than with both operands in the
// ring; gemm_experts.hip keeps it.)
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "elem_load.hpp"
#include "gemm_experts.hpp"
#include "kernels.hpp"
#include "row_prep.hpp"

namespace convrot {
namespace {

using gemm::store4;
using gemm::v4f;
using gemm::v4i;
using gemm::wait_vm;
using gemm::widen;

constexpr int kWaves = 4, kTileN = 32 * kWaves;
static_assert(kTileN == kRowTile, "the launch's count of workgroups");
constexpr int kStep = kTileN * 128, kDepth = 3;       // LDS bytes of a step of 256 columns, steps of the ring
constexpr int kMostEach = 4, kMostCodes = 256 * kWaves * kMostEach;   // blocks of 256 a wave prepares; columns
static_assert(kMostCodes == kRowMostCodes, "the longest row");

__device__ __forceinline__ int swz_w(int r) { return (r >> 1) & 7; }

__device__ __forceinline__ float xor_lane(float v, int m)
{
    const int x = (int)__float_as_uint(v);
    switch (m) {
    case 1: return __uint_as_float(__builtin_amdgcn_update_dpp(0, x, 0xB1, 0xF, 0xF, true));     // quad_perm 1 0 3 2
    case 2: return __uint_as_float(__builtin_amdgcn_update_dpp(0, x, 0x4E, 0xF, 0xF, true));     // quad_perm 2 3 0 1
    case 8: return __uint_as_float(__builtin_amdgcn_update_dpp(0, x, 0x128, 0xF, 0xF, true));    // row_ror 8
    default: return __shfl_xor(v, m);
    }
}

// a barrier that waits for LDS alone: the weights stay in flight
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    gemm::barrier();
    asm volatile("" ::: "memory");
}

// Codes of the row h [F] in natural order, columns past F zero, to LDS; returns its scale.  The operations are
// those of the activation's preparation, one by one: butterflies of the pairs j, j + h for h = 1 .. 128
// (element 4 lane + i of a block), the row's maximum, row_quant and its codes.  after_loads: what is issued
// behind the row's loads.
template <int DT, class Issue>
__device__ __forceinline__ float prepare_row(const typename Elem<DT>::T *h, int F, int blocks, int8_t *codes,
                                             uint32_t *tops, int lane, int wave, Issue after_loads)
{
    typedef typename Elem<DT>::T T;
    typedef T T4 __attribute__((ext_vector_type(4)));
    T4 raw[kMostEach];
    float v[kMostEach][4];
#pragma unroll
    for (int n = 0; n < kMostEach; n++) {
        const int at = 256 * (kWaves * n + wave) + 4 * lane;
        raw[n] = T4{0, 0, 0, 0};
        if (at < F) raw[n] = *reinterpret_cast<const T4 *>(h + at);   // rows are whole 16 bytes long
    }
    after_loads();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < kMostEach; n++)
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[n][i] = 256 * (kWaves * n + wave) + 4 * lane + i < F ? Elem<DT>::cvt(raw[n][i]) : 0.0f;
    float top = 0.0f;
#pragma unroll
    for (int n = 0; n < kMostEach; n++) {
        if (kWaves * n + wave >= blocks) break;
        float(&x)[4] = v[n];
        const float a0 = x[0] + x[1], a1 = x[0] - x[1], a2 = x[2] + x[3], a3 = x[2] - x[3];
        x[0] = a0 + a2; x[2] = a0 - a2; x[1] = a1 + a3; x[3] = a1 - a3;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float o = xor_lane(x[i], m);
                x[i] = lane & m ? o - x[i] : x[i] + o;
            }
#pragma unroll
        for (int i = 0; i < 4; i++) top = fmaxf(top, fabsf(x[i]));
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, xor_lane(top, m));
    if (lane == 0) tops[wave] = __float_as_uint(top);
    lds_barrier();
    uint32_t all = tops[0];                           // magnitudes: their bits are in their order
#pragma unroll
    for (int w = 1; w < kWaves; w++) all = all > tops[w] ? all : tops[w];
    const RowQuant q = row_quant<8>(__uint_as_float(all));
#pragma unroll
    for (int n = 0; n < kMostEach; n++) {
        if (kWaves * n + wave >= blocks) break;
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; i++) c[i] = code_bits((q.folded ? v[n][i] : (v[n][i] * 0.0625f) * 0x1p64f) * q.mult);
        *reinterpret_cast<uint32_t *>(codes + 256 * (kWaves * n + wave) + 4 * lane) = pack_low_bytes(c[0], c[1], c[2], c[3]);
    }
    return q.scale;
}

// A holds the rows between the products, of OUT's type, lda elements each, one a choice.
template <int OUT>
__global__ __launch_bounds__(64 * kWaves)
void experts_row_kernel(const ExpertsGemm g)
{
    __shared__ __attribute__((aligned(1024))) int8_t ring[kDepth * kStep];
    __shared__ __attribute__((aligned(16))) int8_t codes[kMostCodes];
    __shared__ uint32_t tops[kWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, q = lane >> 4;
    const int slot = (int)(blockIdx.x / (uint32_t)g.n_tiles);
    const uint32_t e = (uint32_t)g.ids[slot] - (uint32_t)g.first;
    if (e >= (uint32_t)g.E) return;
    const int nk = g.K_pad / 256;
    const int n0 = ((int)(blockIdx.x % (uint32_t)g.n_tiles) * kWaves + wave) * 32;
    auto weight_row = [&](int r) { return min(n0 + r, g.N - 1); };
    // scales and biases of the columns 4 q .. +3 of each fragment, and the row, before the weights: loads
    // return in order
    v4f sb[2], bias[2];
#pragma unroll
    for (int f = 0; f < 2; f++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const int64_t at = (int64_t)e * g.N + weight_row(16 * f + 4 * q + r);
            sb[f][r] = g.sb[at];
            bias[f][r] = g.bias ? g.bias[at] : 0.0f;
        }
    const int8_t *wsrc[4];                            // where the next step lies
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int r = 8 * j + (lane >> 3);
        wsrc[j] = reinterpret_cast<const int8_t *>(g.B) + (int64_t)e * g.stride_b + (int64_t)weight_row(r) * g.ldb +
                  (((lane & 7) ^ swz_w(r)) << 4);
    }
    auto issue = [&](int at) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            __builtin_amdgcn_global_load_lds(wsrc[j], ring + at + wave * 4096 + j * 1024, 16, 0, 2);   // non-temporal
            wsrc[j] += 128;
        }
    };
    auto issue_first = [&]() {
#pragma unroll
        for (int s = 0; s < kDepth - 1; s++)
            if (s < nk) issue(s * kStep);
    };
    const auto *h = reinterpret_cast<const typename Elem<OUT>::T *>(g.A) + (int64_t)slot * g.lda;
    const float sa = prepare_row<OUT>(h, g.K, nk, codes, tops, lane, wave, issue_first);
    lds_barrier();

    const uint32_t base = (uint32_t)(uintptr_t)ring + wave * 4096 + col * 128;
    uint32_t adr_w[2], adr_a = (uint32_t)(uintptr_t)codes + 64 * (q >> 1) + 16 * (q & 1);
#pragma unroll
    for (int t = 0; t < 2; t++) adr_w[t] = base + (((4 * t + q) ^ swz_w(col)) << 4);
    auto lds = [](uint32_t a) { return *reinterpret_cast<const __attribute__((address_space(3))) v4i *>(a); };
    v4i acc[2] = {v4i{0, 0, 0, 0}, v4i{0, 0, 0, 0}};
    int at = 0, ahead = (kDepth - 1) * kStep;
    for (int k = 0; k < nk; k++) {
        // the wave's own loads of step k are done; the steps behind it may be in flight
        if (k + 1 < nk) wait_vm<4 * (kDepth - 2)>();
        else wait_vm<0>();
        asm volatile("" ::: "memory");                // no read of LDS before the wait
        v4i w[2][2], a[2][2];
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int f = 0; f < 2; f++) {
                w[t][f] = lds(adr_w[t] + at + f * 2048);
                a[t][f] = lds(adr_a + t * 128 + f * 32);
            }
        if (k + kDepth - 1 < nk) issue(ahead);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int f = 0; f < 2; f++)
                    acc[f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                        widen((uint32_t)w[t][f][2 * h], (uint32_t)w[t][f][2 * h + 1]), a[t][h], acc[f], 0, 0, 0);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        at = at == (kDepth - 1) * kStep ? 0 : at + kStep;
        ahead = ahead == (kDepth - 1) * kStep ? 0 : ahead + kStep;
        adr_a += 256;
    }

    // every column of a fragment is the row; lane 16 q stores columns 4 q .. +3
    if (col != 0) return;
    const int64_t row = (int64_t)slot * g.ldc;
#pragma unroll
    for (int f = 0; f < 2; f++) {
        v4f v;
#pragma unroll
        for (int r = 0; r < 4; r++) {
            v[r] = ((float)(acc[f][r] >> 4) * sa) * sb[f][r];
            if (g.bias) v[r] += bias[f][r];
        }
        const int n = n0 + 16 * f + 4 * q;
        if (n < g.N) store4<OUT>(g.C, row + n, v, v4i{}, g.N - n, g.vec);
    }
}

template <int OUT>
hipError_t launch_row_of(const ExpertsGemm &g, hipStream_t st)
{
    const dim3 grid((unsigned)((int64_t)g.S * g.n_tiles)), threads(64 * kWaves);
    hipLaunchKernelGGL((experts_row_kernel<OUT>), grid, threads, 0, st, g);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_experts_row(ExpertsGemm g, int out_dtype, hipStream_t st)
{
    g.n_tiles = (g.N + kTileN - 1) / kTileN;
    const int es = out_dtype < 2 ? 2 : 4;
    g.vec = (uintptr_t)g.C % (4 * es) == 0 && g.ldc % 4 == 0;
    switch (out_dtype) {
    case 0: return launch_row_of<0>(g, st);
    case 1: return launch_row_of<1>(g, st);
    case 2: return launch_row_of<2>(g, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace convrot
