// What the experts' products share: weight codes as bytes, and stores of a lane's columns.
#pragma once

#include <hip/hip_runtime.h>
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <stdint.h>

#include "gemm_common.hpp"

namespace convrot {
namespace gemm {

typedef float v4f __attribute__((ext_vector_type(4)));

// weight codes of two dwords as bytes 16 q, in k order (gemm_s8s4.hip)
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

template <int N>
__device__ __forceinline__ void wait_vm() { __builtin_amdgcn_s_waitcnt(waitcnt_vm(N)); }

}  // namespace gemm
}  // namespace convrot
