// The experts' products for many rows an expert: 256 rows x 256 weight rows a workgroup, the ring and the
// waits of gemm_s8s4.hip, with the rows of A gathered, the rows of C scattered, and SwiGLU in the epilogue.
//
// A tile's rows are those of one expert, up to 256; 64 a wave.  Waves beyond the expert's last row only
// move data: an expert's last tile costs the matrix cores what its rows need, in steps of 64.
// With SwiGLU a tile is 128 gates and their 128 values, dealt to the waves so that a wave holds both of a
// column: its 128 weight rows are 64 gates and 64 values.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "experts.hpp"
#include "gemm_experts.hpp"
#include "kernels.hpp"
#include "swiglu.hpp"

namespace convrot {
namespace {

using gemm::v4i;
using gemm::widen;
using gemm::v16i;

constexpr int W_M = 4, W_N = 2;                 // waves along M (rows), N (weight rows)
constexpr int T_M = 64, T_N = 128;              // wave tile
constexpr int F_M = T_M / 32, F_N = T_N / 32;
constexpr int BM = W_M * T_M, BN = W_N * T_N;
constexpr int LG_BM = 8;
static_assert(BM == 1 << LG_BM && BN == 256, "tile");
constexpr int BK = 128, NSTAGE = 3, KS = BK / 32;
constexpr int NWAVE = W_M * W_N, NTHREAD = 64 * NWAVE;
constexpr int ROW_A = BK, ROW_B = BK / 2;
constexpr int SA = BM * ROW_A, SB = BN * ROW_B;
constexpr int B_BASE = NSTAGE * SA;
constexpr int PIECES_A = SA / 1024, PIECES_B = SB / 1024, PPW = (PIECES_A + PIECES_B) / NWAVE;
static_assert((PIECES_A + PIECES_B) % NWAVE == 0, "DMA pieces split evenly over the waves");
// behind the ring: where each row of the tile goes and its scale, the weight rows' scales and biases
constexpr int MAPS = NSTAGE * (SA + SB);
constexpr int POOL = MAPS + 4 * BM * 4;
static_assert(POOL <= 160 * 1024 && NWAVE * gemm::EPI_BYTES <= MAPS, "LDS");

__device__ __forceinline__ int swz_a(int r) { return (r ^ (r >> 3)) & 7; }
__device__ __forceinline__ int swz_b(int r) { return ((r >> 1) ^ (r >> 2)) & 3; }

template <int OUT>
__device__ __forceinline__ void put4(int8_t *dst, const float (&v)[4])
{
    if constexpr (OUT == 2) {
        *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
    } else if constexpr (OUT == 0) {
        const __hip_bfloat16 h[4] = {__float2bfloat16(v[0]), __float2bfloat16(v[1]), __float2bfloat16(v[2]), __float2bfloat16(v[3])};
        *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<const uint2 *>(h);
    } else {
        const __half h[4] = {__float2half(v[0]), __float2half(v[1]), __float2half(v[2]), __float2half(v[3])};
        *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<const uint2 *>(h);
    }
}

template <int OUT, bool SWIGLU>
__global__ __launch_bounds__(NTHREAD, 1)
void experts_tile_kernel(const ExpertsGemm g)
{
    __shared__ __attribute__((aligned(1024))) int8_t pool[POOL];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / W_N, wn = wave % W_N;

    const int blocks = count_blocks(g.offsets, g.E, g.S, LG_BM, lane);
    if ((int64_t)blockIdx.x >= (int64_t)blocks * g.n_tiles) return;
    int tm, tn;
    gemm::tile_of(blockIdx.x, blocks, g.n_tiles, tm, tn);
    ExpertBlock blk;
    if (!find_block(g.offsets, g.E, g.S, LG_BM, tm, lane, blk)) return;
    const int rows = min(blk.end - blk.row, BM);
    const int cols = SWIGLU ? g.N >> 1 : g.N;         // columns of C
    constexpr int BC = SWIGLU ? BN / 2 : BN;
    const int n0 = tn * BC;
    // weight row of row r of the tile: with SwiGLU 64 gates and their 64 values a wave
    auto weight_row = [&](int r) {
        if constexpr (SWIGLU) return min(n0 + ((r >> 7) << 6) + (r & 63), cols - 1) + ((r >> 6 & 1) ? cols : 0);
        else return min(n0 + r, cols - 1);
    };

    // ---- DMA assignment (gemm_s8s4.hip): rows that are none read the tile's first row ----
    const int8_t *gsrc[PPW];
    int ldst[PPW], kstep[PPW];
#pragma unroll
    for (int j = 0; j < PPW; j++) {
        const int p = wave * PPW + j;
        if (p < PIECES_A) {
            const int r = 8 * p + (lane >> 3);
            const int i = blk.row + (r < rows ? r : 0), from = row_from(g, i, named_row(g, i));
            gsrc[j] = g.A + (int64_t)max(from, 0) * g.lda + (((lane & 7) ^ swz_a(r)) << 4);
            ldst[j] = p * 1024;
            kstep[j] = BK;
        } else {
            const int q = p - PIECES_A;
            const int r = 16 * q + (lane >> 2);
            gsrc[j] = reinterpret_cast<const int8_t *>(g.B) + (int64_t)blk.e * g.stride_b + (int64_t)weight_row(r) * g.ldb +
                      (((lane & 3) ^ swz_b(r)) << 4);
            ldst[j] = B_BASE + q * 1024;
            kstep[j] = BK / 2;
        }
    }
    int *const map_to = reinterpret_cast<int *>(pool + MAPS);
    float *const map_sa = reinterpret_cast<float *>(pool + MAPS) + BM;
    float *const map_sb = map_sa + BM, *const map_bias = map_sb + BN;
    if (tid < BM) {
        const int i = blk.row + (tid < rows ? tid : 0), named = named_row(g, i);
        const int from = tid < rows ? row_from(g, i, named) : -1;
        map_to[tid] = from < 0 ? -1 : row_to(g, i, named);
        map_sa[tid] = OUT != 3 && from >= 0 ? g.sa[from] : 0.0f;
    } else {
        const int r = tid - BM;
        const int64_t n = (int64_t)blk.e * g.N + weight_row(r);
        map_sb[r] = OUT != 3 ? g.sb[n] : 0.0f;
        map_bias[r] = g.bias ? g.bias[n] : 0.0f;
    }

    const bool k_rev = gemm::k_reversed(blockIdx.x);
    const int nk = g.K_pad / BK;                      // even, >= 2
    auto issue = [&](int s, int kt) {
        const int64_t ks = k_rev ? nk - 1 - kt : kt;
#pragma unroll
        for (int j = 0; j < PPW; j++) {
            const int stage_off = ldst[j] < B_BASE ? s * SA : s * SB;
            __builtin_amdgcn_global_load_lds(gsrc[j] + ks * kstep[j], pool + ldst[j] + stage_off, 16, 0, 0);
        }
    };

    const int frow = lane & 31, fhalf = lane >> 5;
    uint32_t adrA[KS][F_M], adrA2[KS][F_M], adrB[KS / 2][F_N];
#pragma unroll
    for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int i = 0; i < F_M; i++) {
            const int r = wm * T_M + i * 32 + frow;
            adrA[ks][i] = (uint32_t)(uintptr_t)pool + r * ROW_A + (((2 * ks + fhalf) ^ swz_a(r)) << 4);
            adrA2[ks][i] = adrA[ks][i] + 2 * SA;
        }
#pragma unroll
    for (int pp = 0; pp < KS / 2; pp++)
#pragma unroll
        for (int j = 0; j < F_N; j++) {
            const int r = wn * T_N + j * 32 + frow;
            adrB[pp][j] = (uint32_t)(uintptr_t)pool + B_BASE + r * ROW_B + (((2 * pp + fhalf) ^ swz_b(r)) << 4);
        }
    v16i acc[F_M][F_N];
#pragma unroll
    for (int i = 0; i < F_M; i++)
#pragma unroll
        for (int j = 0; j < F_N; j++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[i][j][r] = 0;

    v4i fa[2][F_M], fb[2][F_N], braw[F_N];
    auto lds = [](uint32_t a) { return reinterpret_cast<const __attribute__((address_space(3))) v4i *>(a); };
    auto read_a = [&](int s, int ks, int slot) {
#pragma unroll
        for (int i = 0; i < F_M; i++) fa[slot][i] = s == 2 ? *lds(adrA2[ks][i]) : *lds(adrA[ks][i] + s * SA);
    };
    auto read_b = [&](int s, int pp) {
#pragma unroll
        for (int j = 0; j < F_N; j++) braw[j] = *lds(adrB[pp][j] + s * SB);
    };
    auto widen_b = [&]() {
#pragma unroll
        for (int j = 0; j < F_N; j++) {
            fb[0][j] = widen((uint32_t)braw[j][0], (uint32_t)braw[j][1]);
            fb[1][j] = widen((uint32_t)braw[j][2], (uint32_t)braw[j][3]);
        }
    };
    auto mfmas = [&](int slot, int t0, int t1) {
#pragma unroll
        for (int t = 0; t < F_M * F_N; t++) {
            if (t < t0 || t >= t1) continue;
            const int i = t / F_N, j = t % F_N;
            acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[slot][j], fa[slot][i], acc[i][j], 0, 0, 0);
        }
    };

    // the steps, waits and barriers of gemm_s8s4.hip; the maps are written before the first barrier
#pragma unroll
    for (int s = 0; s < NSTAGE; s++) issue(s, min(s, nk - 1));
    __builtin_amdgcn_s_waitcnt(gemm::waitcnt_vm((NSTAGE - 1) * PPW));
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    gemm::barrier();
    asm volatile("" ::: "memory");
    constexpr int NMF = F_M * F_N;
    using C0 = std::integral_constant<int, 0>;
    using C1 = std::integral_constant<int, 1>;
    using C2 = std::integral_constant<int, 2>;
    if (wm * T_M < rows) {
        read_a(0, 0, 0);
        read_b(0, 0);
        auto step = [&](auto S_, int k) {
            constexpr int S = decltype(S_)::value;
            constexpr int NX = (S + 1) % NSTAGE;
#pragma unroll
            for (int ks = 0; ks < KS; ks++) {
                if (ks % 2 == 0) widen_b();
                if (ks < KS - 1) {
                    read_a(S, ks + 1, (ks + 1) & 1);
                    if (ks == 1) read_b(S, 1);
                    mfmas(ks & 1, 0, NMF);
                    __builtin_amdgcn_sched_barrier(0);
                } else {
                    mfmas(ks & 1, 0, 1);
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    __builtin_amdgcn_s_waitcnt(gemm::waitcnt_vm(PPW));
                    gemm::barrier();
                    asm volatile("" ::: "memory");    // no read of LDS before the barrier
                    read_a(NX, 0, 0);
                    read_b(NX, 0);
                    mfmas(ks & 1, 1, NMF);
                    if (k + 1 < nk) issue(S, min(k + NSTAGE, nk - 1));
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        };
        int kt = 0;
        for (; kt + NSTAGE <= nk; kt += NSTAGE) {
            step(C0{}, kt);
            step(C1{}, kt + 1);
            step(C2{}, kt + 2);
        }
        if (kt < nk) step(C0{}, kt);
        if (kt + 1 < nk) step(C1{}, kt + 1);
    } else {
        int s = 0;
        for (int kt = 0; kt < nk; kt++) {
            __builtin_amdgcn_s_waitcnt(gemm::waitcnt_vm(PPW));
            gemm::barrier();
            if (kt + 1 < nk) issue(s, min(kt + NSTAGE, nk - 1));
            s = s == NSTAGE - 1 ? 0 : s + 1;
        }
    }
    __builtin_amdgcn_s_waitcnt(gemm::waitcnt_vm(0));
    __builtin_amdgcn_s_waitcnt(gemm::waitcnt_lgkm0());
    gemm::barrier();                                  // every wave is done with the ring
    asm volatile("" ::: "memory");
    if (wm * T_M >= rows) return;

    // ---- epilogue: by 32 rows, through this wave's part of the idle ring, to the rows of C ----
    constexpr int ES = OUT < 2 ? 2 : 4;
    constexpr int WC = SWIGLU ? T_N / 2 : T_N;        // columns of C a wave
    constexpr int CB = WC * ES < 256 ? WC * ES : 256; // bytes a row and chunk
    constexpr int NC = CB / ES, FJ = SWIGLU ? F_N / 2 : F_N;
    int8_t *const etile = pool + wave * gemm::EPI_BYTES;
    const float *const sb = map_sb + wn * T_N, *const bias = map_bias + wn * T_N;
    const int nbase = n0 + wn * WC;
#pragma unroll
    for (int i = 0; i < F_M; i++) {
        const float sa = map_sa[wm * T_M + i * 32 + frow];
#pragma unroll
        for (int c = 0; c < WC / NC; c++) {
#pragma unroll
            for (int jj = 0; jj < NC / 32; jj++) {
                const int j = c * (NC / 32) + jj;
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const int nl = jj * 32 + 8 * q + 4 * fhalf;   // column inside the chunk
                    const int nw = j * 32 + 8 * q + 4 * fhalf;    // weight row inside the wave's
                    int8_t *dst = etile + frow * gemm::EPI_STRIDE + nl * ES;
                    if constexpr (OUT == 3) {
                        *reinterpret_cast<v4i *>(dst) = v4i{acc[i][j][4 * q] >> 4, acc[i][j][4 * q + 1] >> 4,
                                                            acc[i][j][4 * q + 2] >> 4, acc[i][j][4 * q + 3] >> 4};
                    } else {
                        auto scaled = [&](const v16i &t, int n, float (&v)[4]) {
                            const float4 s4 = *reinterpret_cast<const float4 *>(sb + n);
                            v[0] = ((float)(t[4 * q] >> 4) * sa) * s4.x;
                            v[1] = ((float)(t[4 * q + 1] >> 4) * sa) * s4.y;
                            v[2] = ((float)(t[4 * q + 2] >> 4) * sa) * s4.z;
                            v[3] = ((float)(t[4 * q + 3] >> 4) * sa) * s4.w;
                            if (g.bias) {
                                const float4 b4 = *reinterpret_cast<const float4 *>(bias + n);
                                v[0] += b4.x; v[1] += b4.y; v[2] += b4.z; v[3] += b4.w;
                            }
                        };
                        float v[4];
                        scaled(acc[i][j], nw, v);
                        if constexpr (SWIGLU) {
                            float b[4];
                            scaled(acc[i][j + FJ], nw + T_N / 2, b);
#pragma unroll
                            for (int r = 0; r < 4; r++) {
                                v[r] = swiglu_elem(v[r], b[r]);
                                // rounded to FP32 first, as everywhere (gemm_experts.hip)
                                if constexpr (OUT == 1) asm("" : "+v"(v[r]));
                            }
                        }
                        put4<OUT>(dst, v);
                    }
                }
            }
            gemm::wave_sync();
            constexpr int PR = CB / 16;               // 16-byte pieces a row
#pragma unroll
            for (int t = 0; t < 32 * PR / 64; t++) {
                const int p = lane + 64 * t;
                const int row = p / PR, cc = p % PR;
                const uint4 v = *reinterpret_cast<const uint4 *>(etile + row * gemm::EPI_STRIDE + cc * 16);
                const int to = map_to[wm * T_M + i * 32 + row];
                const int n = nbase + c * NC + cc * (16 / ES);
                if (to < 0 || n >= cols) continue;
                int8_t *out = static_cast<int8_t *>(g.C) + ((int64_t)to * g.ldc + n) * ES;
                if (g.vec && n + 16 / ES <= cols) {
                    // written once: it must not evict what other workgroups still read from L2
                    __builtin_nontemporal_store(gemm::u32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<gemm::u32x4 *>(out));
                } else {
                    const int8_t *vb = reinterpret_cast<const int8_t *>(&v);
#pragma unroll
                    for (int el = 0; el < 16 / ES; el++)
                        if (n + el < cols) {
                            if constexpr (ES == 2) reinterpret_cast<uint16_t *>(out)[el] = reinterpret_cast<const uint16_t *>(vb)[el];
                            else reinterpret_cast<uint32_t *>(out)[el] = reinterpret_cast<const uint32_t *>(vb)[el];
                        }
                }
            }
            gemm::wave_sync();
        }
    }
}

template <int OUT, bool SWIGLU>
hipError_t launch_one(const ExpertsGemm &g, hipStream_t st)
{
    const dim3 grid((unsigned)(most_blocks(g.S, g.E, LG_BM) * g.n_tiles));
    hipLaunchKernelGGL((experts_tile_kernel<OUT, SWIGLU>), grid, dim3(NTHREAD), 0, st, g);
    return hipGetLastError();
}

}  // namespace

int64_t experts_tile_blocks(int64_t S, int64_t E, int64_t N) { return most_blocks(S, E, LG_BM) * ((N + BN - 1) / BN); }

hipError_t launch_experts_tile(ExpertsGemm g, int out_dtype, bool swiglu, hipStream_t st)
{
    g.n_tiles = (g.N + BN - 1) / BN;
    g.vec = (uintptr_t)g.C % 16 == 0 && g.ldc * (out_dtype < 2 ? 2 : 4) % 16 == 0;
    switch (out_dtype) {
    case 0: return swiglu ? launch_one<0, true>(g, st) : launch_one<0, false>(g, st);
    case 1: return swiglu ? launch_one<1, true>(g, st) : launch_one<1, false>(g, st);
    case 2: return swiglu ? launch_one<2, true>(g, st) : launch_one<2, false>(g, st);
    case 3: return swiglu ? hipErrorInvalidValue : launch_one<3, false>(g, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace convrot
