// tq_norm_rope_apply: the heads of queries and keys normalised one by one and
// turned by rotary positions, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w,  then pair (a, b) of y becomes
//   (a cos t - b sin t, b cos t + a sin t), t = pos[axis] * f,
//
// in float32 from the loaded element to the stored one, rounded once.  Every
// element is read and written once, which is the floor; separate calls for the
// two norms and the two rotations would move it four times.  Eight threads
// hold a head's row (16 elements each): three shuffles add its squares up, and
// a thread takes the sines of its 8 pairs once and walks the heads of its
// token with them, queries and keys alike.
#include <cmath>

#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_rope.cuh"
#include "tq_rows.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256;

struct NormRopeArgs {
    const uint8_t *q, *k;
    uint8_t *q_out, *k_out;
    const void *q_weight, *k_weight;                 // [128] of weight_dtype, or null (ones)
    const int64_t *pos;
    int64_t n_tok, q_tok, q_head, k_tok, k_head;     // strides in bytes (pos: elements)
    int64_t qo_tok, qo_head, ko_tok, ko_head, pos_axis;
    int q_heads, heads, slots;                       // heads: q's and k's; slots: as in tq_rope_apply
    int weight_dtype;
    float eps;
};

// 1 / sqrt(mean of the row's squares + eps), from this thread's 16 elements
// and its 7 neighbours'.  A sum that leaves float32's range is taken again
// from elements scaled down (such a mean is far above eps).
__device__ __forceinline__ float inverse_rms(const float (&a)[8], const float (&b)[8], float eps, unsigned group) {
    auto sum = [&](float f) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = a[i] * f, y = b[i] * f;
            s = fmaf(x, x, s);
            s = fmaf(y, y, s);
        }
#pragma unroll
        for (int m = 1; m < 8; m <<= 1) s += __shfl_xor_sync(group, s, m);
        return s;
    };
    const float s = sum(1.f);
    if (s <= 3.0e38f) return rsqrtf(fmaf(s, 1.f / 128.f, eps));
    return rsqrtf(sum(0x1p-80f) * (1.f / 128.f)) * 0x1p-80f;   // (NaN or infinite elements: NaN, or 0 times infinity)
}

template <int DT, bool HALF>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ tq_rope rope,
                                                             const __grid_constant__ NormRopeArgs a) {
    constexpr int NV = Elem<DT>::kVecs, ES = DT == TQ_F32 ? 4 : 2;
    __shared__ uint64_t turn[kRopePairs];
    __shared__ uint8_t axis[kRopePairs];
    __shared__ __align__(16) float weight[2][kD];
    if (threadIdx.x < kRopePairs) {
        turn[threadIdx.x] = rope.turn[threadIdx.x];
        axis[threadIdx.x] = rope.axis[threadIdx.x];
    }
    for (int i = threadIdx.x; i < 2 * kD; i += kThreads) {
        const void *w = i < kD ? a.q_weight : a.k_weight;
        const int e = i & (kD - 1);
        float v = 1.f;
        if (w) {
            if (a.weight_dtype == TQ_F32) v = static_cast<const float *>(w)[e];
            else if (a.weight_dtype == TQ_BF16) v = __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[e]);
            else v = __half2float(static_cast<const __half *>(w)[e]);
        }
        weight[i / kD][e] = v;
    }
    __syncthreads();
    const int c = threadIdx.x & 7, row = threadIdx.x >> 3;
    const unsigned group = 0xFFu << (threadIdx.x & 24);   // the threads of this row
    const int slot = row % a.slots;
    const int64_t n = (int64_t)blockIdx.x * (kThreads / 8 / a.slots) + row / a.slots;
    if (n >= a.n_tok) return;
    const int pairs = rope.rot_dim / 2;
    const bool turned = 8 * c < pairs;   // chunks past the rotated elements are normalised only
    const int e0 = HALF && turned ? 8 * c : 16 * c;
    const int e1 = HALF && turned ? pairs + 8 * c : 16 * c + 8;
    const uint8_t *q = a.q + n * a.q_tok, *k = a.k + n * a.k_tok;
    uint8_t *qo = a.q_out + n * a.qo_tok, *ko = a.k_out + n * a.ko_tok;
    constexpr int kBatch = DT == TQ_F32 ? 2 : 4;
    uint4 va[kBatch][NV], vb[kBatch][NV];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = h0 + u * a.slots;
            if (h < a.heads) {
                const uint8_t *xr = h < a.q_heads ? q + h * a.q_head : k + (h - a.q_heads) * a.k_head;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    va[u][i] = __ldcs(reinterpret_cast<const uint4 *>(xr + e0 * ES) + i);
                    vb[u][i] = __ldcs(reinterpret_cast<const uint4 *>(xr + e1 * ES) + i);
                }
            }
        }
    };
    load(slot);
    float sn[8], cs[8];
    if (turned) {
        int64_t p[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) p[i] = a.pos[(i < rope.axes ? i : 0) * a.pos_axis + n];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int ax = axis[8 * c + i];
            const int64_t t = ax == 0 ? p[0] : ax == 1 ? p[1] : p[2];
            rope_sincos(rope_turns(turn[8 * c + i], t), sn[i], cs[i]);
        }
    }
    for (int h0 = slot; h0 < a.heads; h0 += kBatch * a.slots) {
        uint4 ra[kBatch][NV], rb[kBatch][NV];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = h0 + u * a.slots;
            if (h < a.heads) {
                float fa[8], fb[8], ga[8], gb[8];
                unpack8<DT>(va[u], fa);
                unpack8<DT>(vb[u], fb);
                const float r = inverse_rms(fa, fb, a.eps, group);
                const float *w = weight[h < a.q_heads ? 0 : 1];
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float4 w0 = *reinterpret_cast<const float4 *>(w + e0 + i);
                    const float4 w1 = *reinterpret_cast<const float4 *>(w + e1 + i);
                    const float x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        fa[i + e] = fa[i + e] * r * x0[e];
                        fb[i + e] = fb[i + e] * r * x1[e];
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if constexpr (HALF) {
                        ga[i] = turned ? fmaf(fa[i], cs[i], -(fb[i] * sn[i])) : fa[i];
                        gb[i] = turned ? fmaf(fb[i], cs[i], fa[i] * sn[i]) : fb[i];
                    } else {
                        // pair i of the chunk: elements 2i, 2i + 1 of its 16
                        float *src = i < 4 ? fa : fb, *dst = i < 4 ? ga : gb;
                        const int m = 2 * (i & 3);
                        dst[m] = turned ? fmaf(src[m], cs[i], -(src[m + 1] * sn[i])) : src[m];
                        dst[m + 1] = turned ? fmaf(src[m + 1], cs[i], src[m] * sn[i]) : src[m + 1];
                    }
                }
                pack8<DT>(ga, ra[u]);
                pack8<DT>(gb, rb[u]);
            }
        }
        load(h0 + kBatch * a.slots);   // (rows in place: other heads than the ones written now)
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int h = h0 + u * a.slots;
            if (h < a.heads) {
                uint8_t *orow = h < a.q_heads ? qo + h * a.qo_head : ko + (h - a.q_heads) * a.ko_head;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    __stcs(reinterpret_cast<uint4 *>(orow + e0 * ES) + i, ra[u][i]);
                    __stcs(reinterpret_cast<uint4 *>(orow + e1 * ES) + i, rb[u][i]);
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
    NormRopeArgs a;
    a.q = static_cast<const uint8_t *>(q);
    a.k = static_cast<const uint8_t *>(k);
    a.q_out = static_cast<uint8_t *>(q_out);
    a.k_out = static_cast<uint8_t *>(k_out);
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.pos = pos;
    a.n_tok = n_tok;
    a.q_tok = q_tok_stride * es;
    a.q_head = q_head_stride * es;
    a.k_tok = k_tok_stride * es;
    a.k_head = k_head_stride * es;
    a.qo_tok = q_out_tok_stride * es;
    a.qo_head = q_out_head_stride * es;
    a.ko_tok = k_out_tok_stride * es;
    a.ko_head = k_out_head_stride * es;
    a.pos_axis = pos_axis_stride;
    a.q_heads = q_heads;
    a.heads = q_heads + k_heads;
    a.weight_dtype = weight_dtype;
    a.eps = eps;
    // head slots of a block (32 rows of 8 threads): with few tokens every head has threads of its
    // own; once the rows fill the GPU (about 256 per SM) a thread walks up to 8 heads
    int slots = 32;
    while (slots > 1 && (slots / 2 >= a.heads ||
                         (slots * 4 >= a.heads && n_tok * slots > (int64_t)sm_count() * 256)))
        slots /= 2;
    a.slots = slots;
    const int64_t per = kThreads / 8 / slots, grid = (n_tok + per - 1) / per;
    if (grid > 0x7FFFFFFF) return TQ_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const tq_rope &r = rope ? *rope : none;
    switch (dtype) {
        case TQ_BF16: return launch<TQ_BF16>(r, a, (unsigned)grid, st);
        case TQ_F16: return launch<TQ_F16>(r, a, (unsigned)grid, st);
        default: return launch<TQ_F32>(r, a, (unsigned)grid, st);
    }
}
