// Products of the experts' rows with the experts' 4-bit weights:
//   C[r, n] = ((float)sum_k A[s, k] W_e[n, k] * a_scale[s]) * b_scale[e, n] (+ bias[e, n])
// for the rows of each expert e, s the row of A and r the row of C that a place in the order names;
// with SwiGLU, swish of the first half of the columns times the second half.
// Weights and sums as in gemm_s8s4.hip: nibbles widened to bytes 16 q, int32 sums of 16 q a.
#include <hip/hip_runtime.h>
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "experts.hpp"
#include "gemm_experts.hpp"
#include "kernels.hpp"
#include "swiglu.hpp"

namespace convrot {
namespace {

using gemm::store4;
using gemm::v4f;
using gemm::v4i;
using gemm::wait_vm;
using gemm::widen;

// A workgroup takes up to 64 rows of an expert and 128 weight rows, 32 a wave (with SwiGLU 16 gates and their
// 16 values), and walks K in steps of 256 codes: whole lines of the weight.  Loaded to registers in the order
// of the matrix instruction, neighbouring lanes would take 16 bytes of different rows, which the texture unit
// works off a lane's line at a time; so both operands go to LDS by direct loads in which eight (weight) and
// sixteen (activation) lanes share a row.  A wave's weight rows are its own, the activation's are shared: one
// barrier a step.  The rings' 80 KB let two workgroups run on a compute unit: three steps of weights, three of
// the activation for up to 32 rows and two for 64, whose rows lie in L2 (48 rows an expert, 3584 x 5376: 156 us
// with two steps of both, 151 so, 148 without conflicts of LDS banks).  Slower: one workgroup with twice the
// ring; several tiles of weight rows a workgroup without a pause between them (64 tokens on 64 experts, 5376 x
// 1792: 57 us, 110 and 59).
constexpr int kWaves = 4, kTileN = 32 * kWaves, kLgRows = 6;
constexpr int kStepW = kTileN * 128;                  // LDS bytes of a step's weight rows
constexpr int kRing = 80 * 1024;

// Places of 16-byte chunks: those that the 16 lanes of a fragment read together cover all 64 banks.  A weight row
// has 8 (two rows to the banks), an activation row 16.
__device__ __forceinline__ int swz_w(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int swz_a(int r) { return r & 15; }

// until step k of the first DA - 1 is done: behind its activation loads are the later ones of the prologue (RM
// a step) and k steps
template <int RM, int DA, int J = 0>
__device__ __forceinline__ void wait_first(int k)
{
    constexpr int N = (DA - 2 - J) * RM + J * (4 + RM);
    if constexpr (J == DA - 2) wait_vm<N>();
    else if (k == J) wait_vm<N>();
    else wait_first<RM, DA, J + 1>(k);
}

// What a workgroup of the stream kernel does, the same for every number of rows.
struct Stream {
    const ExpertsGemm &g;
    ExpertBlock blk;
    int slots;               // without a plan: the slot of place `lane`
    int tile;                // which 128 weight rows
    int lane, wave;
    int8_t *pool;
};

// Products of up to 16 RM rows over rings of DW steps of weights and DA of the activation.  Weights that nobody
// else reads go past the caches (64 tokens on 64 experts, 3584 x 5376: 106 -> 95 us, 6.5 TB/s); where an expert
// has several blocks its weights come from the cache the next time (777 tokens on 60: 31 us, not 36).
template <int OUT, bool SWIGLU, int RM, int DW, int DA>
__device__ __forceinline__ void stream(const Stream &x)
{
    constexpr int kStepA = RM * 4096, RING_A = DW * kStepW;  // LDS bytes of a step's rows, and where their ring is
    static_assert(RING_A + DA * kStepA <= kRing && DA >= 2 && DA <= 3 && (DW == DA || DW == DA + 1), "rings");
    constexpr int WC = SWIGLU ? 16 : 32;                     // columns of C a wave
    const ExpertsGemm &g = x.g;
    const ExpertBlock blk = x.blk;
    const int lane = x.lane, wave = x.wave, col = lane & 15, q = lane >> 4;
    int8_t *const pool = x.pool;
    const int n_end = SWIGLU ? g.N >> 1 : g.N, nk = g.K_pad / 256;
    const int n0 = (x.tile * kWaves + wave) * WC;
    const bool once = blk.blocks == 1;

    // the rows that the plan names are requested before everything else: loads return in order.  Place of the
    // lane's direct load j of the activation (places behind the last read the first one), and of its row of
    // the result's fragment m
    auto place_a = [&](int j) {
        const int i = blk.row + 16 * j + 4 * wave + (lane >> 4);
        return i < blk.end ? i : blk.row;
    };
    auto place_c = [&](int m) { return min(blk.row + 16 * m + col, blk.end - 1); };
    int named_a[4], named_c[4];
#pragma unroll
    for (int m = 0; m < RM; m++) {
        named_a[m] = g.ids ? __shfl(x.slots, place_a(m)) : named_row(g, place_a(m));
        named_c[m] = g.ids ? __shfl(x.slots, place_c(m)) : named_row(g, place_c(m));
    }

    auto weight_row = [&](int r) {                           // row r of the wave's 32
        return SWIGLU ? min(n0 + (r & 15), n_end - 1) + (r >> 4) * n_end : min(n0 + r, n_end - 1);
    };
    // scales and biases of the columns 4 q .. +3 of each fragment
    v4f sb[2], bias[2];
#pragma unroll
    for (int f = 0; f < 2; f++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const int64_t at = (int64_t)blk.e * g.N + weight_row(16 * f + 4 * q + r);
            sb[f][r] = OUT != 3 ? g.sb[at] : 0.0f;
            bias[f][r] = g.bias ? g.bias[at] : 0.0f;
        }
    const int8_t *wsrc[4];                                   // where the next step lies
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int r = 8 * j + (lane >> 3);
        wsrc[j] = reinterpret_cast<const int8_t *>(g.B) + (int64_t)blk.e * g.stride_b + (int64_t)weight_row(r) * g.ldb +
                  (((lane & 7) ^ swz_w(r)) << 4);
    }
    auto issue_w = [&](int at) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            int8_t *dst = pool + at + wave * 4096 + j * 1024;
            if (once) __builtin_amdgcn_global_load_lds(wsrc[j], dst, 16, 0, 2);     // non-temporal
            else __builtin_amdgcn_global_load_lds(wsrc[j], dst, 16, 0, 0);
            wsrc[j] += 128;
        }
    };
#pragma unroll
    for (int s = 0; s < DW - 1; s++)
        if (s < nk) issue_w(s * kStepW);

    const int8_t *asrc[4];
#pragma unroll
    for (int j = 0; j < RM; j++) {
        const int r = 16 * j + 4 * wave + (lane >> 4);
        asrc[j] = g.A + (int64_t)max(row_from(g, place_a(j), named_a[j]), 0) * g.lda + (((lane & 15) ^ swz_a(r)) << 4);
    }
    auto issue_a = [&](int at) {
#pragma unroll
        for (int j = 0; j < RM; j++) {
            __builtin_amdgcn_global_load_lds(asrc[j], pool + RING_A + at + j * 4096 + wave * 1024, 16, 0, 0);
            asrc[j] += 256;
        }
    };
#pragma unroll
    for (int s = 0; s < DA - 1; s++)
        if (s < nk) issue_a(s * kStepA);

    int to[4];
    float sa[4];
#pragma unroll
    for (int m = 0; m < RM; m++) {
        const int i = place_c(m), from = row_from(g, i, named_c[m]);
        const bool there = blk.row + 16 * m + col < blk.end && from >= 0;
        to[m] = there ? row_to(g, i, named_c[m]) : -1;
        sa[m] = OUT != 3 && there ? g.sa[from] : 0.0f;
    }

    // LDS addresses of stage 0: weight chunk 4 t + q of row 16 f + col; activation chunk 8 t + 4 (q / 2) +
    // q % 2 + 2 h of row 16 m + col (h: which of a chunk's two groups of codes)
    const uint32_t base = (uint32_t)(uintptr_t)pool;
    uint32_t adr_w[2], adr_a[2][2];
#pragma unroll
    for (int t = 0; t < 2; t++) {
        adr_w[t] = base + wave * 4096 + col * 128 + (((4 * t + q) ^ swz_w(col)) << 4);
#pragma unroll
        for (int h = 0; h < 2; h++)
            adr_a[t][h] = base + RING_A + col * 256 + (((8 * t + 4 * (q >> 1) + (q & 1) + 2 * h) ^ swz_a(col)) << 4);
    }
    auto lds = [](uint32_t a) { return *reinterpret_cast<const __attribute__((address_space(3))) v4i *>(a); };
    v4i acc[2][RM];
#pragma unroll
    for (int f = 0; f < 2; f++)
#pragma unroll
        for (int m = 0; m < RM; m++) acc[f][m] = v4i{0, 0, 0, 0};
    struct Half { v4i w[2], a[RM][2]; };
    auto read = [&](Half &h_, uint32_t at_w, uint32_t at, int t) {
#pragma unroll
        for (int f = 0; f < 2; f++) h_.w[f] = lds(adr_w[t] + at_w + f * 2048);
#pragma unroll
        for (int m = 0; m < RM; m++)
#pragma unroll
            for (int h = 0; h < 2; h++) h_.a[m][h] = lds(adr_a[t][h] + at + m * 4096);
    };
    auto multiply = [&](const Half &h_) {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int f = 0; f < 2; f++) {
                const v4i wide = widen((uint32_t)h_.w[f][2 * h], (uint32_t)h_.w[f][2 * h + 1]);
#pragma unroll
                for (int m = 0; m < RM; m++)
                    acc[f][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wide, h_.a[m][h], acc[f][m], 0, 0, 0);
            }
    };

    // From 2 (DW - 1) steps on, waits leave in flight what was issued behind step k's loads; other loads in between
    // only make the first ones wait for more.
    const bool exact_waits = nk >= 2 * (DW - 1);
    int at_w = 0, next_w = (DW - 1) * kStepW, at_a = 0, next_a = (DA - 1) * kStepA;
    for (int k = 0; k < nk; k++) {
        // step k's loads are done: this wave's, and behind the barrier all; and all have read step k - 1
        if (!exact_waits) wait_vm<0>();
        else if (k < DA - 1) wait_first<RM, DA>(k);
        else if (k + 1 < nk) wait_vm<(DA - 2) * (4 + RM) + (DW - DA) * 4>();
        else wait_vm<0>();
        gemm::barrier();
        asm volatile("" ::: "memory");                       // no read of LDS before the barrier
        Half a, b;
        read(a, at_w, at_a, 0);
        read(b, at_w, at_a, 1);
        if (k + DA - 1 < nk) issue_a(next_a);
        if (k + DW - 1 < nk) issue_w(next_w);
        __builtin_amdgcn_sched_barrier(0);
        multiply(a);
        multiply(b);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        at_w = at_w == (DW - 1) * kStepW ? 0 : at_w + kStepW;
        next_w = next_w == (DW - 1) * kStepW ? 0 : next_w + kStepW;
        at_a = at_a == (DA - 1) * kStepA ? 0 : at_a + kStepA;
        next_a = next_a == (DA - 1) * kStepA ? 0 : next_a + kStepA;
    }

    // lane l of a fragment holds row l % 16 and columns 4 (l / 16) .. +3
    auto scaled = [&](const v4i &t, float s, int f) {
        v4f v;
#pragma unroll
        for (int r = 0; r < 4; r++) {
            v[r] = ((float)t[r] * s) * sb[f][r];
            if (g.bias) v[r] += bias[f][r];
        }
        return v;
    };
#pragma unroll
    for (int m = 0; m < RM; m++) {
        const int64_t row = (int64_t)to[m] * g.ldc;
        if constexpr (SWIGLU) {
            const int n = n0 + 4 * q;
            const v4f a = scaled(acc[0][m] >> 4, sa[m], 0), b = scaled(acc[1][m] >> 4, sa[m], 1);
            v4f o;
#pragma unroll
            for (int r = 0; r < 4; r++) {
                o[r] = swiglu_elem(a[r], b[r]);
                // the product is rounded to FP32 before it is rounded to fp16, as everywhere in this
                // library: without this the compiler makes one rounding of the two (v_fma_mixlo_f16)
                if constexpr (OUT == 1) asm("" : "+v"(o[r]));
            }
            if (to[m] >= 0 && n < n_end) store4<OUT>(g.C, row + n, o, v4i{}, n_end - n, g.vec);
        } else {
#pragma unroll
            for (int f = 0; f < 2; f++) {
                const int n = n0 + 16 * f + 4 * q;
                const v4i t = acc[f][m] >> 4;
                if (to[m] >= 0 && n < n_end)
                    store4<OUT>(g.C, row + n, OUT == 3 ? v4f{} : scaled(t, sa[m], f), t, n_end - n, g.vec);
            }
        }
    }
}

// The b-th expert among the choices of up to 64 slots, in the order of their first slots: a wave's own plan.
// Lane p gets the slot of the expert's place p.
__device__ __forceinline__ bool find_choice(const ExpertsGemm &g, int b, int lane, ExpertBlock &blk, int &slots)
{
    const uint32_t id = lane < g.S ? (uint32_t)g.ids[lane] - (uint32_t)g.first : ~0u;
    uint64_t left = __builtin_amdgcn_ballot_w64(id < (uint32_t)g.E), mine;
    while (true) {
        if (left == 0) return false;
        const uint32_t e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        mine = __builtin_amdgcn_ballot_w64(id == e);
        if (b-- == 0) {
            blk.e = (int)e;
            break;
        }
        left &= ~mine;
    }
    blk.row = 0;
    blk.end = __popcll(mine);
    blk.blocks = 1;
    blk.nth = 0;
    const uint64_t below = (1ull << lane) - 1;
    const int place = mine >> lane & 1 ? __popcll(mine & below) : blk.end + __popcll(~mine & below);
    slots = __builtin_amdgcn_ds_permute(place << 2, lane);
    return true;
}

template <int OUT, bool SWIGLU>
__global__ __launch_bounds__(64 * kWaves)
void experts_stream_kernel(const ExpertsGemm g)
{
    __shared__ __attribute__((aligned(1024))) int8_t pool[kRing];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    ExpertBlock blk;
    const int b = (int)(blockIdx.x / g.n_tiles);
    int slots = 0;
    if (!(g.ids ? find_choice(g, b, lane, blk, slots) : find_block(g.offsets, g.E, g.S, kLgRows, b, lane, blk))) return;
    int tile = (int)(blockIdx.x % g.n_tiles);
    if (blk.blocks > 1) {
        // Workgroup i runs on XCD i % 8.  The blocks of an expert take a tile of its weights on the same XCD, one
        // after another, so that all but the first find it in that XCD's cache: 8 tiles at a time, then the rest
        // (777 tokens on 60 experts: 31.4 -> 30.2 us, 100 rows an expert: 230 -> 224).
        const int j = blk.nth * g.n_tiles + tile, whole = g.n_tiles & ~(gemm::NUM_XCD - 1);
        const int left = j - whole * blk.blocks, run = gemm::NUM_XCD * blk.blocks;
        tile = left < 0 ? j / run * gemm::NUM_XCD + j % gemm::NUM_XCD : whole + left % (g.n_tiles - whole);
        const int nth = left < 0 ? j % run / gemm::NUM_XCD : left / (g.n_tiles - whole);
        blk.row += (nth - blk.nth) << kLgRows;
    }
    const Stream x{g, blk, slots, tile, lane, wave, pool};
    const int rows = blk.end - blk.row;
    if (rows <= 16) stream<OUT, SWIGLU, 1, 3, 3>(x);
    else if (rows <= 32) stream<OUT, SWIGLU, 2, 3, 3>(x);
    else stream<OUT, SWIGLU, 4, 3, 2>(x);
}

template <int OUT, bool SWIGLU>
hipError_t launch_stream(const ExpertsGemm &g, hipStream_t st)
{
    const int64_t blocks = g.ids ? (g.S < g.E ? g.S : g.E) : most_blocks(g.S, g.E, kLgRows);
    const dim3 grid((unsigned)(blocks * g.n_tiles));
    hipLaunchKernelGGL((experts_stream_kernel<OUT, SWIGLU>), grid, dim3(64 * kWaves), 0, st, g);
    return hipGetLastError();
}

// Many rows an expert on average: 128-row tiles, whose waves share the weights in LDS.  64 experts, bf16, us
// for 3584 x 5376 and 5376 x 1792, by streams and by tiles: 72 rows an expert 171 and 107, 207 and 111; 88 rows
// 197 and 122, 210 and 113; 100 rows 214 and 133, 218 and 118.  The average is over the experts here and counts
// every slot, also those of experts elsewhere: how many fall here only the device knows (8 of 64 experts here, 128
// tokens of 8 choices: 45 us by tiles, 16 by streams).
bool tiled(int64_t S, int64_t E) { return S > 88 * E; }

}  // namespace

int64_t experts_gemm_blocks(int64_t S, int64_t E, int64_t N)
{
    if (tiled(S, E)) return experts_tile_blocks(S, E, N);
    return most_blocks(S, E, kLgRows) * ((N + kTileN - 1) / kTileN);
}

hipError_t launch_gemm_experts(ExpertsGemm g, int out_dtype, bool swiglu, hipStream_t st)
{
    if (g.ids && g.S > kOwnPlan) return hipErrorInvalidValue;
    if (tiled(g.S, g.E)) return launch_experts_tile(g, out_dtype, swiglu, st);
    g.n_tiles = (g.N + kTileN - 1) / kTileN;
    const int es = out_dtype < 2 ? 2 : 4;
    g.vec = (uintptr_t)g.C % (4 * es) == 0 && g.ldc % 4 == 0;
    switch (out_dtype) {
    case 0: return swiglu ? launch_stream<0, true>(g, st) : launch_stream<0, false>(g, st);
    case 1: return swiglu ? launch_stream<1, true>(g, st) : launch_stream<1, false>(g, st);
    case 2: return swiglu ? launch_stream<2, true>(g, st) : launch_stream<2, false>(g, st);
    case 3: return swiglu ? hipErrorInvalidValue : launch_stream<3, false>(g, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace convrot
