// The SwiGLU element and the exponential in it, shared by the activation preparation and the experts'
// product.
#pragma once

#include <hip/hip_runtime.h>

namespace convrot {

// ------------------------------------------------------ reproducible exponential ----

// E(x) ~ exp(x) from IEEE basic operations only: Cody & Waite (1980) reduction
// x = k ln2 + r, k = rint(x log2 e), ln2 = C1 + C2 with C1 holding 15 significant bits,
// then the degree-7 Taylor polynomial of exp(r) in Horner form with fused multiply-adds,
// then the exact scaling by 2^k.  Coefficients: RN(1/n!).  By definition E(x) = +inf for
// x > 89 and E(x) = 0 for x < -104.
//
// The steps are evaluated on x clamped to [-200, 200] with no further selects: inside
// [-104, 89] nothing changes; for x in (89, 200] the reduction gives k >= 128 with
// p >= 1.32 (k = 128) or p >= 0.70 (k > 128), so p * 2^k overflows to +inf; for x in
// [-200, -104) it gives p * 2^k < 2^-150, which rounds to 0.  A NaN argument gives NaN
// or, if the clamp returns a bound, a finite value; the callers below only use E(-a)
// inside a product with a, which is NaN either way.
__device__ __forceinline__ float repro_exp_nan_free(float x)
{
    const float kLog2e = 0x1.715476p+0f;
    const float kC1 = 0x1.62e4p-1f;
    const float kC2 = 0x1.7f7d1cp-20f;
    const float xc = __builtin_amdgcn_fmed3f(x, -200.0f, 200.0f);
    const float kf = rintf(xc * kLog2e);
    float r = fmaf(-kf, kC1, xc);
    r = fmaf(-kf, kC2, r);
    float p = 0x1.a01a02p-13f;             // 1/7!
    p = fmaf(p, r, 0x1.6c16c2p-10f);       // 1/6!
    p = fmaf(p, r, 0x1.111112p-7f);        // 1/5!
    p = fmaf(p, r, 0x1.555556p-5f);        // 1/4!
    p = fmaf(p, r, 0x1.555556p-3f);        // 1/3!
    p = fmaf(p, r, 0x1.0p-1f);             // 1/2!
    p = fmaf(p, r, 1.0f);
    p = fmaf(p, r, 1.0f);
    return __builtin_amdgcn_ldexpf(p, (int)kf);
}

// 1 / d for 1 <= d < 2^126, correctly rounded: the hardware reciprocal estimate refined by
// one Newton step in fused multiply-adds (Markstein's correction).  The tests check it
// against IEEE division for every d that an fp32 gate can produce here.
__device__ __forceinline__ float recip_refined(float d)
{
    const float y = __builtin_amdgcn_rcpf(d);
    const float e = fmaf(-d, y, 1.0f);
    return fmaf(e, y, y);
}

constexpr float kRecipLimit = 0x1p126f;   // d at or above: IEEE division (gate below about -87.3)

// The SwiGLU element: swish(a) * b with swish(a) = a * sigma(a), sigma(a) = 1 / (1 + E(-a)),
// every operation rounded once as written.
__device__ __forceinline__ float swiglu_exact(float a, float b)
{
    const float d = 1.0f + repro_exp_nan_free(-a);
    return (a * (1.0f / d)) * b;
}

// Same value; the refined reciprocal where it is exact, IEEE division for the lanes (a
// wave-uniform branch, practically never taken) whose denominator is 2^126 or more.
__device__ __forceinline__ float swiglu_elem(float a, float b)
{
    const float d = 1.0f + repro_exp_nan_free(-a);
    float o = (a * recip_refined(d)) * b;
    const bool far = !(d < kRecipLimit);
    if (__builtin_amdgcn_ballot_w64(far) != 0) {
        if (far) o = (a * (1.0f / d)) * b;
    }
    return o;
}

}  // namespace convrot
