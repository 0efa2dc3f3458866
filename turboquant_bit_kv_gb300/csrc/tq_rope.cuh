// Rotary positions on the device: exact angle reduction and the sine and
// cosine of one (token, pair).
//
// The angle of pair i at position t is t * f_i radians.  A rope holds f_i as
// a 64-bit fraction of a turn, F_i = f_i / (2 pi) * 2^64 mod 2^64, so that
// the low 64 bits of t * F_i are the angle modulo one turn with an error of
// at most t * 2^-65 turns: far positions lose nothing (a float32 product
// t * f_i is off by up to 0.06 rad at t = 10^6), and negative positions work
// by two's complement.
#pragma once

#include <stdint.h>

#include "tq.h"

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

// The same in double precision.
__device__ __forceinline__ void rope_sincos_double(uint64_t frac, double &s, double &c) {
    sincospi((double)(int64_t)frac * 1.0842021724855044e-19 /* 2^-63 */, &s, &c);
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
