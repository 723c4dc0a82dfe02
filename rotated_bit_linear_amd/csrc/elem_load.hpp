// Loads of activation rows in segments of 16 elements, shared by the row preparation kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <stdint.h>

#include "row_prep.hpp"

namespace convrot {

template <int DT> struct Elem;
template <> struct Elem<0> {   // bf16: the upper half of a binary32
    using T = uint16_t;
    static __device__ __forceinline__ float cvt(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
};
template <> struct Elem<1> {   // fp16: exact widening
    using T = uint16_t;
    static __device__ __forceinline__ float cvt(uint16_t h) { return __half2float(__ushort_as_half(h)); }
};
template <> struct Elem<2> {   // fp32
    using T = float;
    static __device__ __forceinline__ float cvt(float f) { return f; }
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Raw bytes of 16 consecutive elements: 32 bytes for 16-bit types, 64 for fp32.
template <int DT> struct RawSeg {
    u32x4 w[DT == 2 ? 4 : 2];
};

// Fetch elements [k0, k0+16) of a row with logical length K: vector loads when the whole
// segment lies below K and the row permits 16-byte loads (non-temporal: the activation is
// read once; ordinary with kKeep, for the first pass over a row that is read twice),
// element loads for a segment straddling K, nothing at all past K.
template <int DT, bool kKeep = false>
__device__ __forceinline__ void fetch_seg(const typename Elem<DT>::T *row, int64_t k0, int64_t K, bool aligned,
                                          RawSeg<DT> &r)
{
    constexpr int NW = DT == 2 ? 4 : 2;
    if (aligned && k0 + 16 <= K) {
#pragma unroll
        for (int c = 0; c < NW; c++) {
            const u32x4 *src = reinterpret_cast<const u32x4 *>(row + k0) + c;
            if constexpr (kKeep) r.w[c] = *src;
            else r.w[c] = __builtin_nontemporal_load(src);
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < NW; c++) r.w[c] = u32x4{0u, 0u, 0u, 0u};
    if (k0 >= K) return;
    const int rem = opaque((int)(K - k0 < 16 ? K - k0 : 16));   // elements below K
    if constexpr (DT == 2) {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(row + k0);
#pragma unroll
        for (int i = 0; i < 16; i++)
            if (i < rem) r.w[i >> 2][i & 3] = p[i];
    } else {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(row + k0);
#pragma unroll
        for (int i = 0; i < 16; i++)
            if (i < rem) r.w[i >> 3][(i >> 1) & 3] |= (uint32_t)p[i] << (16 * (i & 1));
    }
}

// element i (0..15) of a fetched segment
template <int DT>
__device__ __forceinline__ float seg_elem(const RawSeg<DT> &r, int i)
{
    if constexpr (DT == 2) {
        return __uint_as_float(r.w[i >> 2][i & 3]);
    } else {
        const uint32_t w = r.w[i >> 3][(i >> 1) & 3];
        return Elem<DT>::cvt((uint16_t)((i & 1) ? (w >> 16) : (w & 0xffffu)));
    }
}

template <int DT>
__device__ __forceinline__ void decode_seg(const RawSeg<DT> &r, float (&v)[16])
{
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = seg_elem<DT>(r, i);
}

}  // namespace convrot
