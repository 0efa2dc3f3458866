// Rows of 128 elements of float32, bf16 or fp16 taken 8 elements at a time, and
// the check that no two rows of an output share an element (shared by the
// rotary kernels).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "tq.h"
#include "tq_device.cuh"

namespace tq {
namespace {

template <int DT>
struct Elem;
template <>
struct Elem<TQ_F32> {
    static constexpr int kVecs = 2;   // 16-byte vectors of 8 elements
};
template <>
struct Elem<TQ_BF16> {
    static constexpr int kVecs = 1;
};
template <>
struct Elem<TQ_F16> {
    static constexpr int kVecs = 1;
};

template <int DT>
__device__ __forceinline__ void unpack8(const uint4 (&v)[Elem<DT>::kVecs], float (&f)[8]) {
    if constexpr (DT == TQ_F32) {
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    } else {
        const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == TQ_BF16) {
                f[2 * i] = bf16_bits_lo(w[i]);
                f[2 * i + 1] = bf16_bits_hi(w[i]);
            } else {
                const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                f[2 * i] = h.x;
                f[2 * i + 1] = h.y;
            }
        }
    }
}

template <int DT>
__device__ __forceinline__ void pack8(const float (&f)[8], uint4 (&v)[Elem<DT>::kVecs]) {
    if constexpr (DT == TQ_F32) {
        v[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        v[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == TQ_BF16) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&b);
            } else {
                const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Whether two of the rows of kD elements at i s + j t, i < n, j < m, share an
// element (they would be written twice, in any order).
bool rows_overlap(int64_t n, int64_t s, int64_t m, int64_t t) {
    if ((n > 1 && s < kD) || (m > 1 && t < kD)) return true;
    if (n <= 1 || m <= 1) return false;
    if ((s - kD) / t >= m - 1 || (t - kD) / s >= n - 1) return false;   // all j before the next i, or the other way round
    if (n > m) return rows_overlap(m, t, n, s);
    for (int64_t i = 1; i < n; ++i) {   // the j nearest to row (i, 0)
        const __int128 at = (__int128)i * s;
        const int64_t near = (int64_t)((at + t / 2) / t), j = near < 1 ? 1 : (near < m ? near : m - 1);
        const __int128 d = at - (__int128)j * t;
        if (d < kD && d > -kD) return true;
        if (near >= m) return false;   // (further i are further away)
    }
    return false;
}

}  // namespace
}  // namespace tq
