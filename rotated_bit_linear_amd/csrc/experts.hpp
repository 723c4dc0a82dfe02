// What the kernels of a layer of experts share.  A slot is one choice of one token: slot t * k + j is
// choice j of token t.  The plan lists the slots by expert: those of expert e are
// rows[offsets[e] .. offsets[e+1]-1].
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.hpp"

namespace convrot {

// sum over lanes 0 .. own of a wave
__device__ __forceinline__ int wave_scan(int x)
{
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, true);   // row_shr 1, 2, 4, 8: within 16 lanes
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // lane 15 of rows 0, 2 to rows 1, 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // lane 31 to rows 2, 3
    return x;
}

// An offset as it lies on the device, held within the slots that there are.
__host__ __device__ inline int expert_offset(const int32_t *offsets, int i, int S)
{
    const int o = offsets[i];
    return o < 0 ? 0 : o < S ? o : S;
}

// blocks of 2^lg places that a run lo .. hi-1 is cut into, and the first place of its i-th
__host__ __device__ inline int expert_blocks(int lo, int hi, int lg) { return hi > lo ? (int)(((int64_t)hi - lo + (1 << lg) - 1) >> lg) : 0; }
__host__ __device__ inline int block_place(int lo, int i, int lg) { return lo + (i << lg); }

// row of A and row of C of a place, -1 where the plan names none; `named` is rows[i], where there are rows
__host__ __device__ inline int row_from(const ExpertsGemm &g, int i, int named)
{
    const int r = g.gather ? (int)((uint32_t)named / (uint32_t)g.gather) : i;
    return r >= 0 && r < g.M ? r : -1;
}
__host__ __device__ inline int row_to(const ExpertsGemm &g, int i, int named)
{
    const int r = g.scatter ? named : i;
    return r >= 0 && r < g.S ? r : -1;
}
__host__ __device__ inline int named_row(const ExpertsGemm &g, int i) { return g.gather || g.scatter ? g.rows[i] : 0; }

// blocks of all experts, found by each wave
__device__ __forceinline__ int count_blocks(const int32_t *offsets, int E, int S, int lg, int lane)
{
    int n = 0;
    for (int c = lane; c < E; c += 64)
        n += expert_blocks(expert_offset(offsets, c, S), expert_offset(offsets, c + 1, S), lg);
    return __builtin_amdgcn_readlane(wave_scan(n), 63);
}

// Block b of the experts' rows: block counts follow from the offsets, which only the device knows, so
// every wave finds its own.  False where there are fewer blocks.  Whatever the offsets hold,
// 0 <= row < end <= S.
struct ExpertBlock {
    int e, row, end;         // expert, the block's first place in the order, and the end of the expert's
    int blocks, nth;         // blocks of the expert, and which of them this one is
};
__device__ __forceinline__ bool find_block(const int32_t *offsets, int E, int S, int lg, int b, int lane,
                                           ExpertBlock &out)
{
    int before = 0;
    for (int c = 0; c < E; c += 64) {
        const int i = c + lane;
        const int lo = i < E ? expert_offset(offsets, i, S) : 0, hi = i < E ? expert_offset(offsets, i + 1, S) : 0;
        const int n = expert_blocks(lo, hi, lg);
        const int upto = before + wave_scan(n);
        const uint64_t past = __builtin_amdgcn_ballot_w64(upto > b);
        if (past) {
            const int l = __builtin_ctzll(past);
            out.e = c + l;
            out.end = __builtin_amdgcn_readlane(hi, l);
            out.blocks = __builtin_amdgcn_readlane(n, l);
            const int first = __builtin_amdgcn_readlane(upto, l) - out.blocks;
            out.nth = b - first;
            out.row = block_place(__builtin_amdgcn_readlane(lo, l), out.nth, lg);
            return true;
        }
        before = __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

// Tile i of an expert's blocks of rows x n_tiles columns, taken by bands of `band` blocks, each band column by
// column.
struct TilePlace {
    int block, column;
};
__host__ __device__ inline TilePlace place_in_bands(int i, int blocks, int n_tiles, int band)
{
    const int nth = i / (band * n_tiles), left = blocks - nth * band, high = left < band ? left : band;
    const int j = i - nth * band * n_tiles;
    return {nth * band + j % high, j / high};
}

// blocks of 2^lg rows that S slots of E experts come to at most
inline int64_t most_blocks(int64_t S, int64_t E, int lg) { return S <= E ? S : E + ((S - E) >> lg); }

}  // namespace convrot
