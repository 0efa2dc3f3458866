// tq_norm_rope_apply: the heads of queries and keys normalised one by one and
// turned by rotary positions, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w,  then pair (a, b) of y becomes
//   (a cos t - b sin t, b cos t + a sin t), t = pos[axis] * f,
//
// in float32 from the loaded element to the stored one, rounded once.  Every
// element is read and written once, which is the floor; separate calls for the
// two norms and the two rotations would move it four times.
//
// Eight threads hold a head's row (16 elements each): three shuffles add its
// squares up.  A group of eight takes up to kWalk heads of one token, queries or
// keys, so that the sines of a thread's 8 pairs and their products with the
// weights are worked out once for all of them: a head then costs two packed
// products an element.
#include <cmath>

#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_rope.cuh"
#include "tq_rows.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256;

struct NormRopeArgs {
    const uint8_t *x[2];                             // queries, keys
    uint8_t *out[2];
    const void *weight[2];                           // [128] of weight_dtype, or null (ones)
    const int64_t *pos;
    int64_t n_tok, pos_axis;
    int64_t tok[2], head[2], o_tok[2], o_head[2];    // strides in bytes
    int heads[2], groups[2], walk;                   // groups: of at most walk heads
    int weight_dtype;
    float eps;
};

// 1 / sqrt(mean of the row's squares + eps), from this thread's 16 elements
// and its 7 neighbours'.  A sum that leaves float32's range is taken again
// from elements scaled down (such a mean is far above eps).
__device__ __forceinline__ float inverse_rms(const float2 (&x)[8], float eps, unsigned group) {
    auto sum = [&](float f) {
        float2 s = make_float2(0.f, 0.f), t = s;
        const float2 f2 = make_float2(f, f);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 a = f == 1.f ? x[i] : __fmul2_rn(x[i], f2), b = f == 1.f ? x[i + 1] : __fmul2_rn(x[i + 1], f2);
            s = __ffma2_rn(a, a, s);
            t = __ffma2_rn(b, b, t);
        }
        float r = (s.x + s.y) + (t.x + t.y);
#pragma unroll
        for (int m = 1; m < 8; m <<= 1) r += __shfl_xor_sync(group, r, m);
        return r;
    };
    const float s = sum(1.f);
    if (s <= 3.0e38f) return rsqrtf(fmaf(s, 1.f / 128.f, eps));
    return rsqrtf(sum(0x1p-80f) * (1.f / 128.f)) * 0x1p-80f;   // (NaN or infinite elements: NaN, or 0 times infinity)
}

__device__ __forceinline__ float weight_at(const void *w, int dtype, int e) {
    if (!w) return 1.f;
    if (dtype == TQ_F32) return static_cast<const float *>(w)[e];
    if (dtype == TQ_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[e]);
    return __half2float(static_cast<const __half *>(w)[e]);
}

// Thread (token, group of heads, chunk c of 8): the row's 16 elements of chunk c
// are two runs of 8, at elements e0 and e1.
template <int DT, bool HALF>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ tq_rope rope,
                                                             const __grid_constant__ NormRopeArgs a) {
    constexpr int NV = Elem<DT>::kVecs, ES = DT == TQ_F32 ? 4 : 2;
    const int c = threadIdx.x & 7;
    const unsigned lanes = 0xFFu << (threadIdx.x & 24);   // the threads of this row
    const int per_tok = a.groups[0] + a.groups[1];
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 8) + (threadIdx.x >> 3), n = unit / per_tok;
    if (n >= a.n_tok) return;
    int first = (int)(unit - n * per_tok);
    const int which = first >= a.groups[0];
    first = (first - (which ? a.groups[0] : 0)) * a.walk;
    const int end = min(first + a.walk, a.heads[which]);
    const int pairs = rope.rot_dim / 2;
    const bool turned = 8 * c < pairs;   // chunks past the rotated elements are normalised only
    const int e0 = HALF && turned ? 8 * c : 16 * c;
    const int e1 = HALF && turned ? pairs + 8 * c : 16 * c + 8;
    const int64_t head = a.head[which], o_head = a.o_head[which];
    const uint8_t *x = a.x[which] + n * a.tok[which];
    uint8_t *o = a.out[which] + n * a.o_tok[which];
    // heads go by in batches, loaded at once; other warps' loads run meanwhile
    constexpr int kBatch = DT == TQ_F32 ? 2 : 4;
    uint4 va[kBatch][NV], vb[kBatch][NV];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (h0 + u < end) {
                const uint8_t *xr = x + (h0 + u) * head;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    va[u][i] = __ldcs(reinterpret_cast<const uint4 *>(xr + e0 * ES) + i);
                    vb[u][i] = __ldcs(reinterpret_cast<const uint4 *>(xr + e1 * ES) + i);
                }
            }
        }
    };
    load(first);
    // elements 2k, 2k + 1 of the 16 become (themselves) * p + (the others of their pairs) * q
    float2 p[8], q[8];
    {
        const void *w = a.weight[which];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            p[k] = make_float2(weight_at(w, a.weight_dtype, e0 + 2 * k), weight_at(w, a.weight_dtype, e0 + 2 * k + 1));
            p[k + 4] = make_float2(weight_at(w, a.weight_dtype, e1 + 2 * k), weight_at(w, a.weight_dtype, e1 + 2 * k + 1));
        }
        if (turned) {
            int64_t ps[3];
#pragma unroll
            for (int i = 0; i < 3; ++i) ps[i] = a.pos[(i < rope.axes ? i : 0) * a.pos_axis + n];
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                float sn[2], cs[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int ax = rope.axis[8 * c + k + e];
                    rope_sincos(rope_turns(rope.turn[8 * c + k + e], ax == 0 ? ps[0] : ax == 1 ? ps[1] : ps[2]), sn[e], cs[e]);
                }
                if constexpr (HALF) {
                    // pairs k, k + 1: element k of the first run with element k of the second
                    const float2 wa = p[k / 2], wb = p[k / 2 + 4];
                    p[k / 2] = make_float2(wa.x * cs[0], wa.y * cs[1]);
                    q[k / 2] = make_float2(-wb.x * sn[0], -wb.y * sn[1]);
                    p[k / 2 + 4] = make_float2(wb.x * cs[0], wb.y * cs[1]);
                    q[k / 2 + 4] = make_float2(wa.x * sn[0], wa.y * sn[1]);
                } else {
                    // pair k: elements 2k, 2k + 1 of the 16
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 w2 = p[k + e];
                        p[k + e] = make_float2(w2.x * cs[e], w2.y * cs[e]);
                        q[k + e] = make_float2(-w2.y * sn[e], w2.x * sn[e]);
                    }
                }
            }
        }
    }
    for (int h0 = first; h0 < end; h0 += kBatch) {
        if (h0 > first) load(h0);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (h0 + u < end) {
                float f[8], g[8];
                unpack8<DT>(va[u], f);
                unpack8<DT>(vb[u], g);
                float2 y[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    y[k] = make_float2(f[2 * k], f[2 * k + 1]);
                    y[k + 4] = make_float2(g[2 * k], g[2 * k + 1]);
                }
                const float r = inverse_rms(y, a.eps, lanes);
                const float2 r2 = make_float2(r, r);
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = __fmul2_rn(y[k], r2);
                float2 z[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 other = HALF ? y[k ^ 4] : make_float2(y[k].y, y[k].x);
                    z[k] = turned ? __ffma2_rn(y[k], p[k], __fmul2_rn(other, q[k])) : __fmul2_rn(y[k], p[k]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    f[2 * k] = z[k].x;
                    f[2 * k + 1] = z[k].y;
                    g[2 * k] = z[k + 4].x;
                    g[2 * k + 1] = z[k + 4].y;
                }
                uint4 ra[NV], rb[NV];
                pack8<DT>(f, ra);
                pack8<DT>(g, rb);
                uint8_t *orow = o + (h0 + u) * o_head;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    __stcs(reinterpret_cast<uint4 *>(orow + e0 * ES) + i, ra[i]);
                    __stcs(reinterpret_cast<uint4 *>(orow + e1 * ES) + i, rb[i]);
                }
            }
        }
    }
}

template <int DT>
int launch(const tq_rope &rope, const NormRopeArgs &a, unsigned grid, cudaStream_t st) {
    if (rope.style == TQ_ROPE_HALF)
        norm_rope_kernel<DT, true><<<grid, kThreads, 0, st>>>(rope, a);
    else
        norm_rope_kernel<DT, false><<<grid, kThreads, 0, st>>>(rope, a);
    return launch_status();
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" int tq_norm_rope_apply(const void *q, int q_heads, int64_t q_tok_stride, int64_t q_head_stride,
                                  const void *k, int k_heads, int64_t k_tok_stride, int64_t k_head_stride, int dtype,
                                  int64_t n_tok, const void *q_weight, const void *k_weight, int weight_dtype,
                                  float eps, const int64_t *pos, int64_t pos_axis_stride, const tq_rope *rope,
                                  void *q_out, int64_t q_out_tok_stride, int64_t q_out_head_stride, void *k_out,
                                  int64_t k_out_tok_stride, int64_t k_out_head_stride, void *stream) {
    if (n_tok < 0 || q_heads < 0 || k_heads < 0 || (int64_t)q_heads + k_heads <= 0) return TQ_ERR_ARG;
    if (!(eps >= 0x1p-100f) || !std::isfinite(eps)) return TQ_ERR_ARG;
    const int es = dtype_bytes(dtype);
    if (!es || !dtype_bytes(weight_dtype) || (rope && !rope_ok(rope))) return TQ_ERR_UNSUPPORTED;
    if ((int64_t)q_heads + k_heads > (1 << 26)) return TQ_ERR_UNSUPPORTED;
    if (n_tok == 0) return TQ_OK;
    if ((q_heads && (!q || !q_out)) || (k_heads && (!k || !k_out)) || (rope && !pos)) return TQ_ERR_ARG;
    if (q_tok_stride < 0 || q_head_stride < 0 || k_tok_stride < 0 || k_head_stride < 0 || q_out_tok_stride < 0 ||
        q_out_head_stride < 0 || k_out_tok_stride < 0 || k_out_head_stride < 0 || pos_axis_stride < 0)
        return TQ_ERR_ARG;
    const int64_t strides = q_tok_stride | q_head_stride | k_tok_stride | k_head_stride | q_out_tok_stride |
                            q_out_head_stride | k_out_tok_stride | k_out_head_stride;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(pos, 8) ||
        !aligned(q_weight, dtype_bytes(weight_dtype)) || !aligned(k_weight, dtype_bytes(weight_dtype)) ||
        ((strides * es) & 15))
        return TQ_ERR_ALIGN;
    if ((q_heads && rows_overlap(n_tok, q_out_tok_stride, q_heads, q_out_head_stride)) ||
        (k_heads && rows_overlap(n_tok, k_out_tok_stride, k_heads, k_out_head_stride)))
        return TQ_ERR_ARG;
    tq_rope none = {};   // no pair turns
    NormRopeArgs a = {};
    a.x[0] = static_cast<const uint8_t *>(q);
    a.x[1] = static_cast<const uint8_t *>(k);
    a.out[0] = static_cast<uint8_t *>(q_out);
    a.out[1] = static_cast<uint8_t *>(k_out);
    a.weight[0] = q_weight;
    a.weight[1] = k_weight;
    a.pos = pos;
    a.n_tok = n_tok;
    a.pos_axis = pos_axis_stride;
    a.tok[0] = q_tok_stride * es;
    a.tok[1] = k_tok_stride * es;
    a.head[0] = q_head_stride * es;
    a.head[1] = k_head_stride * es;
    a.o_tok[0] = q_out_tok_stride * es;
    a.o_tok[1] = k_out_tok_stride * es;
    a.o_head[0] = q_out_head_stride * es;
    a.o_head[1] = k_out_head_stride * es;
    a.heads[0] = q_heads;
    a.heads[1] = k_heads;
    a.weight_dtype = weight_dtype;
    a.eps = eps;
    // heads of a group: with few tokens every head has threads of its own; once the groups fill the
    // GPU (about 256 per SM) they walk up to 8 heads
    int walk = 1;
    while (walk < 8 && n_tok * ((int64_t)q_heads + k_heads) > (int64_t)sm_count() * 256 * walk) walk *= 2;
    a.walk = walk;
    a.groups[0] = (q_heads + walk - 1) / walk;
    a.groups[1] = (k_heads + walk - 1) / walk;
    constexpr int per = kThreads / 8;
    const int64_t per_tok = a.groups[0] + a.groups[1];
    if (n_tok > INT64_MAX / per_tok - per) return TQ_ERR_UNSUPPORTED;
    const int64_t grid = (n_tok * per_tok + per - 1) / per;
    if (grid > 0x7FFFFFFF) return TQ_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const tq_rope &r = rope ? *rope : none;
    switch (dtype) {
        case TQ_BF16: return launch<TQ_BF16>(r, a, (unsigned)grid, st);
        case TQ_F16: return launch<TQ_F16>(r, a, (unsigned)grid, st);
        default: return launch<TQ_F32>(r, a, (unsigned)grid, st);
    }
}
