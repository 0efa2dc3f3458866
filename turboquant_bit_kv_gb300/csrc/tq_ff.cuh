// Double-float arithmetic: a value as the unevaluated sum h + l of two
// float32, |l| at most half an ulp of h: about 48 significant bits from the
// float32 pipes, for the few rows where float32 alone cannot decide (GB300's
// double-precision pipe has one sixty-fourth of the float32 rate).  The sums
// and products are the error-free transformations of Knuth (TwoSum) and of
// the fused multiply-add (TwoProduct).
#pragma once

#include "tq_device.cuh"

namespace tq {

struct ff {
    float h, l;
};

__device__ __forceinline__ ff ff_of(float h, float l = 0.f) { return {h, l}; }

// h + l renormalised, |l| below |h|.
__device__ __forceinline__ ff ff_quick(float h, float l) {
    const float s = __fadd_rn(h, l);
    return {s, __fsub_rn(l, __fsub_rn(s, h))};
}

__device__ __forceinline__ ff ff_add(ff a, ff b) {
    float s, e;
    two_sum(a.h, b.h, s, e);
    return ff_quick(s, e + (a.l + b.l));
}

// a + b and a^2 of float32, exact.
__device__ __forceinline__ ff ff_sum(float a, float b) {
    ff r;
    two_sum(a, b, r.h, r.l);
    return r;
}
__device__ __forceinline__ ff ff_square(float a) {
    const float p = __fmul_rn(a, a);
    return {p, fmaf(a, a, -p)};
}

__device__ __forceinline__ ff ff_neg(ff a) { return {-a.h, -a.l}; }
__device__ __forceinline__ ff ff_sub(ff a, ff b) { return ff_add(a, ff_neg(b)); }

__device__ __forceinline__ ff ff_mul(ff a, ff b) {
    const float p = __fmul_rn(a.h, b.h);
    return ff_quick(p, __fadd_rn(fmaf(a.h, b.h, -p), fmaf(a.h, b.l, __fmul_rn(a.l, b.h))));
}

__device__ __forceinline__ ff ff_scale(ff a, float b) {   // a float32 factor
    const float p = __fmul_rn(a.h, b);
    return ff_quick(p, __fadd_rn(fmaf(a.h, b, -p), __fmul_rn(a.l, b)));
}

// Square root of a positive value: one Newton step from the float32 root.
__device__ __forceinline__ ff ff_sqrt(ff a) {
    const float s = sqrtf(a.h);
    const float r = __fadd_rn(fmaf(-s, s, a.h), a.l);   // the first difference is exact
    return ff_quick(s, r / (2.f * s));
}

// fp16 of a non-negative value, one rounding to nearest even.
__device__ __forceinline__ unsigned short ff_half(ff a) {
    if (!(a.h < 65536.f)) return __half_as_ushort(__float2half_rn(a.h));
    const __half d = __float2half_rd(a.h);   // a lies in [d, u] up to a.l, which the midpoint sees
    const unsigned short b = __half_as_ushort(d);
    const float lo = __half2float(d), hi = b + 1 >= 0x7C00 ? 65536.f : __half2float(__ushort_as_half((unsigned short)(b + 1)));
    const float t = (a.h - 0.5f * (lo + hi)) + a.l;
    if (t > 0.f) return (unsigned short)(b + 1);
    // (a.h on d itself with a.l below it still rounds to d)
    if (t < 0.f) return b;
    return (unsigned short)(b + (b & 1));
}

}  // namespace tq
