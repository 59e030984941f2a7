// recurrence.cuh -- pieces that the prompt and single-token kernels share: element loads and
// the decay factor e^g in more than single precision.
#pragma once

#include "tv_internal.cuh"

namespace tv {
namespace rec {

// A number >= 0 as the unevaluated sum hi + lo of two floats.  hi is rounded down, and lo is above
// 0 wherever hi is (2^-149 at least): an infinite x stays x in x hi + x lo, where a lo of 0 or
// below would make NaN of it.
struct Pair {
    float hi, lo;
};

// 2^(n + f) for whole n and |f| <= 0.5, from the series of e^t - 1 at t = f ln 2 (|t| <= 0.35:
// the first term left out, t^9 / 9!, is below 2^-32).  The sum 1 + (e^t - 1) is kept as a pair,
// so the relative error is that of e^t - 1: 2^-24 for f = 0.5, and falling with f.  A decay that
// is applied row after row is close to 1, and there an error of 2^-24 each time would add up.
__device__ __forceinline__ Pair exp2_pair(float n, float f) {
    const float t = f * 0.693147180559945309f;
    float p = 1.f / 40320.f;
    p = fmaf(p, t, 1.f / 5040.f);
    p = fmaf(p, t, 1.f / 720.f);
    p = fmaf(p, t, 1.f / 120.f);
    p = fmaf(p, t, 1.f / 24.f);
    p = fmaf(p, t, 1.f / 6.f);
    p = fmaf(p, t, 0.5f);
    p = fmaf(p, t, 1.f);
    const float r = t * p;
    Pair e;
    e.hi = __fadd_rd(1.f, r);
    e.lo = r - (e.hi - 1.f);
    const int k = (int)fminf(fmaxf(n, -252.f), 254.f), k0 = k / 2, k1 = k - k0;  // two factors
    const float s0 = __int_as_float((k0 + 127) << 23), s1 = __int_as_float((k1 + 127) << 23);
    e.hi = e.hi * s0 * s1;
    e.lo = e.lo * s0 * s1;
    if (n < -252.f) e.hi = e.lo = 0.f;
    if (e.hi > 0.f) e.lo = fmaxf(e.lo, __int_as_float(1));  // (past 2^128 both may be infinite)
    return e;
}

// e^g for any g; NaN stays NaN.
__device__ __forceinline__ Pair exp_pair(float g) {
    if (g != g) return {g, g};
    const float x = fminf(fmaxf(g, -1000.f), 1000.f);  // (beyond: 0 or infinity all the same)
    const float log2e = 1.44269502f, rest = 1.92596303e-8f;
    const float y = x * log2e, lo = fmaf(x, rest, fmaf(x, log2e, -y));
    const float n = rintf(y);
    return exp2_pair(n, (y - n) + lo);
}

__device__ __forceinline__ float4 load4(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}

__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
}

// Element i of an output of either type.
__device__ __forceinline__ void store_out(void *out, bool f32, size_t i, float x) {
    if (f32)
        static_cast<float *>(out)[i] = x;
    else
        static_cast<__nv_bfloat16 *>(out)[i] = __float2bfloat16_rn(x);
}

}  // namespace rec
}  // namespace tv
