// Rotary positions on the device: reduction of the angle and the sine and
// cosine of one (token, pair).
//
// The angle of pair i at position t is t * f_i radians.  A rope holds f_i as
// a 64-bit fraction of a turn, F_i = f_i / (2 pi) * 2^64 mod 2^64, so that
// the low 64 bits of t * F_i are the angle modulo one turn, off by |t| 2^-64
// turns at most (F_i is rounded to a whole number): positions up to 2^37 lose
// nothing that float32 could hold (a float32 product t * f_i is off by up to
// 0.06 rad at t = 10^6), and negative positions work by two's complement.
#pragma once

#include <stdint.h>

#include "tq.h"
#include "tq_ff.cuh"

namespace tq {

constexpr int kRopePairs = 64;

// Angle modulo one turn, in 2^-64 turns.
__device__ __forceinline__ uint64_t rope_turns(uint64_t turn, int64_t pos) { return turn * (uint64_t)pos; }

// Sine and cosine of an angle given in 2^-64 turns.  The two top bits (after
// adding half a quarter turn) pick the quarter, the rest is a signed angle in
// [-pi/4, pi/4], where the Taylor series through x^9 and x^10 are below 2^-29
// of their true values (x^11 / 11! and x^12 / 12! at pi/4).
__device__ __forceinline__ void rope_sincos(uint64_t frac, float &s, float &c) {
    const uint32_t hi = (uint32_t)((frac + (1ull << 31)) >> 32);
    const uint32_t q = (hi + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(hi - (q << 30)) * 1.4629180792671596e-09f;   // 2 pi / 2^32
    const float x2 = x * x;
    float ps = fmaf(x2, 2.7557319223985893e-06f, -1.9841269841269841e-04f);   // 1/9!, -1/7!
    ps = fmaf(x2, ps, 8.3333333333333333e-03f);                               // 1/5!
    ps = fmaf(x2, ps, -1.6666666666666667e-01f);                              // -1/3!
    ps = fmaf(x * x2, ps, x);
    float pc = fmaf(x2, -2.7557319223985888e-07f, 2.4801587301587302e-05f);   // -1/10!, 1/8!
    pc = fmaf(x2, pc, -1.3888888888888889e-03f);                              // -1/6!
    pc = fmaf(x2, pc, 4.1666666666666664e-02f);                               // 1/4!
    pc = fmaf(x2, pc, -0.5f);
    pc = fmaf(x2, pc, 1.f);
    const float sa = (q & 1u) ? pc : ps, ca = (q & 1u) ? ps : pc;
    s = (q & 2u) ? -sa : sa;
    c = ((q + 1u) & 2u) ? -ca : ca;
}

// 1 / (n (n + 1)), n = 1 .. 20.
static __constant__ double kRopeInverse[20] = {
    1. / 2,   1. / 6,   1. / 12,  1. / 20,  1. / 30,  1. / 42,  1. / 56,  1. / 72,  1. / 90,  1. / 110,
    1. / 132, 1. / 156, 1. / 182, 1. / 210, 1. / 240, 1. / 272, 1. / 306, 1. / 342, 1. / 380, 1. / 420};

// The same in double precision (series through x^21 and x^20, below 2^-70 of
// their values at pi/4), in few instructions: for rare rows.
__device__ __forceinline__ void rope_sincos_double(uint64_t frac, double &s, double &c) {
    const uint32_t q = (uint32_t)((frac + (1ull << 61)) >> 62);
    const double x = (double)(int64_t)(frac - ((uint64_t)q << 62)) * 3.4061215800300735e-19;   // 2 pi / 2^64
    const double x2 = x * x;
    // sin x / x = 1 - x2 / (2 3) (1 - x2 / (4 5) (...)), cos x = 1 - x2 / (1 2) (1 - x2 / (3 4) (...))
    double ps = 1.0, pc = 1.0;
#pragma unroll 1
    for (int k = 9; k >= 0; --k) {
        ps = fma(-x2 * kRopeInverse[2 * k + 1], ps, 1.0);
        pc = fma(-x2 * kRopeInverse[2 * k], pc, 1.0);
    }
    ps *= x;
    s = (q & 1u) ? pc : ps;
    c = (q & 1u) ? ps : pc;
    if (q & 2u) s = -s;
    if ((q + 1u) & 2u) c = -c;
}

// The same in double-float arithmetic: the angle exact, the series' terms
// through x^7 in double-float, the rest (below 2^-18 and good to 2^-21 of
// itself, series through x^13) in float32: off by less than 2^-38.
__device__ __forceinline__ void rope_sincos_ff(uint64_t frac, ff &s, ff &c) {
    const uint32_t q = (uint32_t)((frac + (1ull << 61)) >> 62);
    const int64_t r = (int64_t)(frac - ((uint64_t)q << 62));
    const float f1 = __int2float_rn((int)(r >> 32));
    const int64_t rest = r - ((int64_t)f1 << 32);          // below 2^40 in size
    const float f2 = (float)(int)(rest >> 16) * 1.52587890625e-05f + (float)(int)(rest & 0xFFFF) * 2.3283064365386963e-10f;
    // times 2 pi / 2^32, as two float32
    const ff x = ff_mul(ff_quick(f1, f2), ff_of(1.46291807926715967e-09f, 1.46291807926715967e-09 - (double)1.46291807926715967e-09f));
    const ff z = ff_mul(x, x), z2 = ff_mul(z, z), z3 = ff_mul(z2, z);
    const float z4 = z2.h * z2.h;
    const ff one = {1.f, 0.f};
    const ff k6 = {1.66666666666666667e-01f, (float)(1.66666666666666667e-01 - (double)1.66666666666666667e-01f)};
    const ff k24 = {4.16666666666666667e-02f, (float)(4.16666666666666667e-02 - (double)4.16666666666666667e-02f)};
    const ff k120 = {8.33333333333333333e-03f, (float)(8.33333333333333333e-03 - (double)8.33333333333333333e-03f)};
    const ff k720 = {1.38888888888888889e-03f, (float)(1.38888888888888889e-03 - (double)1.38888888888888889e-03f)};
    const ff k5040 = {1.98412698412698413e-04f, (float)(1.98412698412698413e-04 - (double)1.98412698412698413e-04f)};
    // sin x = x (1 - z / 6 + z^2 / 120 - z^3 / 7! + z^4 (1 / 9! - z / 11! + z^2 / 13!))
    const float ts = z4 * fmaf(z.h, fmaf(z.h, 1.60590438368216146e-10f, -2.50521083854417188e-08f), 2.75573192239858907e-06f);
    const ff ps = ff_mul(x, ff_add(ff_sub(one, ff_mul(z, k6)),
                                   ff_add(ff_sub(ff_mul(z2, k120), ff_mul(z3, k5040)), ff_of(ts))));
    // cos x = 1 - z / 2 + z^2 / 24 - z^3 / 6! + z^4 (1 / 8! - z / 10! + z^2 / 12!)
    const float tc = z4 * fmaf(z.h, fmaf(z.h, 2.08767569878680990e-09f, -2.75573192239858907e-07f), 2.48015873015873016e-05f);
    const ff pc = ff_add(ff_sub(one, ff_scale(z, 0.5f)),
                         ff_add(ff_sub(ff_mul(z2, k24), ff_mul(z3, k720)), ff_of(tc)));
    s = (q & 1u) ? pc : ps;
    c = (q & 1u) ? ps : pc;
    if (q & 2u) s = ff_neg(s);
    if ((q + 1u) & 2u) c = ff_neg(c);
}

// Argument check of a caller's rope (host).
inline bool rope_ok(const tq_rope *r) {
    if (r->head_dim != 128 || r->rot_dim < 32 || r->rot_dim > 128 || (r->rot_dim & 31)) return false;
    if (r->style != TQ_ROPE_HALF && r->style != TQ_ROPE_ADJACENT) return false;
    if (r->axes < 1 || r->axes > 3) return false;
    for (int i = 0; i < r->rot_dim / 2; ++i)
        if (r->axis[i] >= r->axes) return false;
    return true;
}

}  // namespace tq
