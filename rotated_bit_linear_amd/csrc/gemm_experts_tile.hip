// The experts' products for many rows an expert: 128 rows x 256 weight rows a workgroup through LDS by direct
// loads, the products of gemm_s8s4.hip, with the rows of A gathered, the rows of C scattered, and SwiGLU in the
// epilogue.
//
// A tile's rows are those of one expert; 64 a wave.  Waves beyond the expert's last row only move data.
// With SwiGLU a tile is 128 gates and their 128 values, dealt to the waves so that a wave holds both of a
// column: its 128 weight rows are 64 gates and 64 values.
// Two workgroups run on a compute unit: one looks its rows up, or stores, while the other multiplies, and last
// tiles waste less than those of 256 rows.  In their 80 KB each, A, which comes from far, has three steps of
// the ring and the weights, which other tiles on the XCD read too, two; three of A beside two of the weights
// take 4096 x 8 slots on 64 experts, 1792 -> 5376, from 420 to 386 us.  Against one workgroup a unit with 256 x
// 256 tiles and three steps of both (64 experts, 5376 -> 2 x 1792 with SwiGLU and 1792 -> 5376, us): 200 rows
// an expert 380 -> 336 and 215 -> 190, 512 rows 725 -> 668 and 424 -> 385, 2500 rows 3015 -> 2965 and 1783 ->
// 1660 (2080 and 1860 TOPS).  Bound, at 2500 rows, by the power limit: 1.82 and 1.92 GHz of 2.4, the matrix cores
// busy 55 and 47 % of the cycles; at 512 rows (the second product: 41 % at 2.20 GHz) more by the steps' own chain.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "experts.hpp"
#include "gemm_experts.hpp"
#include "kernels.hpp"
#include "swiglu.hpp"

namespace convrot {
namespace {

using gemm::v4i;
using gemm::widen;
using gemm::v16i;

constexpr int W_M = 2, W_N = 2;                 // waves along M (rows), N (weight rows)
constexpr int T_M = 64, T_N = 128;              // wave tile
constexpr int F_M = T_M / 32, F_N = T_N / 32;
constexpr int BM = W_M * T_M, BN = W_N * T_N;
constexpr int LG_BM = 7;
constexpr int kBand = 8;                        // blocks of rows that walk the columns together
static_assert(BM == 1 << LG_BM && BN == 256, "tile");
constexpr int BK = 128, DA = 3, DB = 2, KS = BK / 32;      // steps of the ring of A and of the weights
constexpr int NWAVE = W_M * W_N, NTHREAD = 64 * NWAVE;
constexpr int ROW_A = BK, ROW_B = BK / 2;
constexpr int SA = BM * ROW_A, SB = BN * ROW_B;
constexpr int B_BASE = DA * SA, POOL = B_BASE + DB * SB;
constexpr int PA = SA / 1024 / NWAVE, PB = SB / 1024 / NWAVE;   // direct loads of a wave and step
// once the ring is idle, behind the waves' tiles: where each row goes and its scale, the weight rows' scales
// and biases
constexpr int MAPS = NWAVE * gemm::EPI_BYTES;
static_assert(2 * POOL <= 160 * 1024 && MAPS + 2 * (BM + BN) * 4 <= POOL && NTHREAD == BN && BM <= NTHREAD, "LDS");

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
__global__ __launch_bounds__(NTHREAD, 2)
void experts_tile_kernel(const ExpertsGemm g)
{
    __shared__ __attribute__((aligned(1024))) int8_t pool[POOL];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / W_N, wn = wave % W_N;

    const int blocks = count_blocks(g.offsets, g.E, g.S, LG_BM, lane);
    // Workgroup i runs on XCD i % 8, and each XCD takes an eighth of the tiles, in the order of the experts; an
    // expert's go by bands of 8 blocks of rows, so that the 64 tiles that run on an XCD at once are 8 x 8 of one
    // expert and read the fewest bytes (against the dense GEMM's order, which knows no experts: 2500 rows an
    // expert 1711 -> 1659 us and 3014 -> 2966; bands of 4 and 16: 1672, 1692)
    const int64_t tiles = (int64_t)blocks * g.n_tiles, part = (tiles + gemm::NUM_XCD - 1) / gemm::NUM_XCD;
    const int turn = (int)(blockIdx.x / gemm::NUM_XCD);
    const int64_t tile = (int64_t)(blockIdx.x % gemm::NUM_XCD) * part + turn;
    if (turn >= part || tile >= tiles) return;
    ExpertBlock blk;
    if (!find_block(g.offsets, g.E, g.S, LG_BM, (int)(tile / g.n_tiles), lane, blk)) return;
    const TilePlace place = place_in_bands(blk.nth * g.n_tiles + (int)(tile % g.n_tiles), blk.blocks, g.n_tiles, kBand);
    blk.row += (place.block - blk.nth) << LG_BM;
    const int rows = min(blk.end - blk.row, BM);
    const int cols = SWIGLU ? g.N >> 1 : g.N;         // columns of C
    constexpr int BC = SWIGLU ? BN / 2 : BN;
    const int n0 = place.column * BC;
    // weight row of row r of the tile: with SwiGLU 64 gates and their 64 values a wave
    auto weight_row = [&](int r) {
        if constexpr (SWIGLU) return min(n0 + ((r >> 7) << 6) + (r & 63), cols - 1) + ((r >> 6 & 1) ? cols : 0);
        else return min(n0 + r, cols - 1);
    };

    // direct loads of a step: 8 rows of A or 16 weight rows each; rows that are none read the tile's first row
    const int8_t *a_src[PA], *b_src[PB];
#pragma unroll
    for (int j = 0; j < PA; j++) {
        const int r = 8 * (wave * PA + j) + (lane >> 3);
        const int i = blk.row + (r < rows ? r : 0), from = row_from(g, i, named_row(g, i));
        a_src[j] = g.A + (int64_t)max(from, 0) * g.lda + (((lane & 7) ^ swz_a(r)) << 4);
    }
#pragma unroll
    for (int j = 0; j < PB; j++) {
        const int r = 16 * (wave * PB + j) + (lane >> 2);
        b_src[j] = reinterpret_cast<const int8_t *>(g.B) + (int64_t)blk.e * g.stride_b + (int64_t)weight_row(r) * g.ldb +
                   (((lane & 3) ^ swz_b(r)) << 4);
    }
    // thread t: row t of the tile, weight row t
    int to = -1;
    float sa = 0.0f, sb, bias;
    if (tid < rows) {
        const int i = blk.row + tid, named = named_row(g, i), from = row_from(g, i, named);
        to = from < 0 ? -1 : row_to(g, i, named);
        if (OUT != 3 && from >= 0) sa = g.sa[from];
    }
    {
        const int64_t n = (int64_t)blk.e * g.N + weight_row(tid);
        sb = OUT != 3 ? g.sb[n] : 0.0f;
        bias = g.bias ? g.bias[n] : 0.0f;
    }

    // every second time its 64 tiles an XCD walks K from the end, which its cache still holds
    const bool k_rev = turn >> 6 & 1;
    const int nk = g.K_pad / BK;                      // even, >= 2
    auto issue_a = [&](int at, int kt) {
        const int64_t ks = k_rev ? nk - 1 - kt : kt;
#pragma unroll
        for (int j = 0; j < PA; j++)
            __builtin_amdgcn_global_load_lds(a_src[j] + ks * BK, pool + at + (wave * PA + j) * 1024, 16, 0, 0);
    };
    auto issue_b = [&](int at, int kt) {
        const int64_t ks = k_rev ? nk - 1 - kt : kt;
#pragma unroll
        for (int j = 0; j < PB; j++)
            __builtin_amdgcn_global_load_lds(b_src[j] + ks * (BK / 2), pool + B_BASE + at + (wave * PB + j) * 1024, 16, 0, 0);
    };

    const int frow = lane & 31, fhalf = lane >> 5;
    uint32_t adrA[KS][F_M], adrB[KS / 2][F_N];
#pragma unroll
    for (int ks = 0; ks < KS; ks++)
#pragma unroll
        for (int i = 0; i < F_M; i++) {
            const int r = wm * T_M + i * 32 + frow;
            adrA[ks][i] = (uint32_t)(uintptr_t)pool + r * ROW_A + (((2 * ks + fhalf) ^ swz_a(r)) << 4);
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
    auto read_a = [&](int at, int ks, int slot) {
#pragma unroll
        for (int i = 0; i < F_M; i++) fa[slot][i] = *lds(adrA[ks][i] + at);
    };
    auto read_b = [&](int at, int pp) {
#pragma unroll
        for (int j = 0; j < F_N; j++) braw[j] = *lds(adrB[pp][j] + at);
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

    // the first wait leaves step 1 and A's step 2 in flight
    issue_b(0, 0);
    issue_a(0, 0);
    issue_b(SB, 1);
    issue_a(SA, 1);
    if (nk > 2) {
        issue_a(2 * SA, 2);
        __builtin_amdgcn_s_waitcnt(gemm::waitcnt_vm(2 * PA + PB));
    } else {
        __builtin_amdgcn_s_waitcnt(gemm::waitcnt_vm(PA + PB));
    }
    gemm::barrier();
    asm volatile("" ::: "memory");
    constexpr int NMF = F_M * F_N;
    int at_a = 0, at_b = 0;
    // step k + 1 has arrived everywhere (behind its loads in flight: A's of step k + 2), and all have read step k
    auto next_step = [&](int k) {
        if (k + 2 < nk) __builtin_amdgcn_s_waitcnt(gemm::waitcnt_vm(PA));
        else __builtin_amdgcn_s_waitcnt(gemm::waitcnt_vm(0));
        gemm::barrier();
        asm volatile("" ::: "memory");                // no read of LDS before the barrier
    };
    auto refill = [&](int k, int a, int b) {
        if (k + 2 < nk) issue_b(b, k + 2);
        if (k + 3 < nk) issue_a(a, k + 3);
    };
    auto advance = [&]() {
        at_a = at_a == (DA - 1) * SA ? 0 : at_a + SA;
        at_b ^= SB;
    };
    if (wm * T_M < rows) {
        read_a(0, 0, 0);
        read_b(0, 0);
        for (int k = 0; k < nk; k++) {
#pragma unroll
            for (int ks = 0; ks < KS; ks++) {
                if (ks % 2 == 0) widen_b();
                if (ks < KS - 1) {
                    read_a(at_a, ks + 1, (ks + 1) & 1);
                    if (ks == 1) read_b(at_b, 1);
                    mfmas(ks & 1, 0, NMF);
                    __builtin_amdgcn_sched_barrier(0);
                } else {
                    mfmas(ks & 1, 0, 1);
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    next_step(k);
                    const int a = at_a, b = at_b;
                    advance();
                    read_a(at_a, 0, 0);
                    read_b(at_b, 0);
                    mfmas(ks & 1, 1, NMF);
                    refill(k, a, b);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    } else {
        for (int k = 0; k < nk; k++) {
            next_step(k);
            refill(k, at_a, at_b);
            advance();
        }
    }
    __builtin_amdgcn_s_waitcnt(gemm::waitcnt_vm(0));
    __builtin_amdgcn_s_waitcnt(gemm::waitcnt_lgkm0());
    gemm::barrier();                                  // every wave is done with the ring
    asm volatile("" ::: "memory");
    int *const map_to = reinterpret_cast<int *>(pool + MAPS);
    float *const map_sa = reinterpret_cast<float *>(pool + MAPS) + BM;
    float *const map_sb = map_sa + BM, *const map_bias = map_sb + BN;
    if (tid < BM) {
        map_to[tid] = to;
        map_sa[tid] = sa;
    }
    map_sb[tid] = sb;
    map_bias[tid] = bias;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    gemm::barrier();
    asm volatile("" ::: "memory");
    if (wm * T_M >= rows) return;

    // ---- epilogue: by 32 rows, through this wave's part of the idle ring, to the rows of C ----
    constexpr int ES = OUT < 2 ? 2 : 4;
    constexpr int WC = SWIGLU ? T_N / 2 : T_N;        // columns of C a wave
    constexpr int CB = WC * ES < 256 ? WC * ES : 256; // bytes a row and chunk
    constexpr int NC = CB / ES, FJ = SWIGLU ? F_N / 2 : F_N;
    int8_t *const etile = pool + wave * gemm::EPI_BYTES;
    const float *const w_sb = map_sb + wn * T_N, *const w_bias = map_bias + wn * T_N;
    const int nbase = n0 + wn * WC;
#pragma unroll
    for (int i = 0; i < F_M; i++) {
        const float row_sa = map_sa[wm * T_M + i * 32 + frow];
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
                            const float4 s4 = *reinterpret_cast<const float4 *>(w_sb + n);
                            v[0] = ((float)(t[4 * q] >> 4) * row_sa) * s4.x;
                            v[1] = ((float)(t[4 * q + 1] >> 4) * row_sa) * s4.y;
                            v[2] = ((float)(t[4 * q + 2] >> 4) * row_sa) * s4.z;
                            v[3] = ((float)(t[4 * q + 3] >> 4) * row_sa) * s4.w;
                            if (g.bias) {
                                const float4 b4 = *reinterpret_cast<const float4 *>(w_bias + n);
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
    const dim3 grid((unsigned)experts_tile_blocks(g.S, g.E, g.N));
    hipLaunchKernelGGL((experts_tile_kernel<OUT, SWIGLU>), grid, dim3(NTHREAD), 0, st, g);
    return hipGetLastError();
}

}  // namespace

int64_t experts_tile_blocks(int64_t S, int64_t E, int64_t N)
{
    const int64_t tiles = most_blocks(S, E, LG_BM) * ((N + BN - 1) / BN);
    return (tiles + gemm::NUM_XCD - 1) / gemm::NUM_XCD * gemm::NUM_XCD;
}

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
