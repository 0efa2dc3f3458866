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
// squares up.  A group of eight takes up to eight heads of one token, queries or
// keys, so that the sines of a thread's 8 pairs are worked out once for all of
// them.  All its heads are requested at once into shared memory: 192 KB an SM on
// their way, and no registers held for them.  A row is requested as it lies, 128
// bytes by the eight threads at a time, whichever of them needs which (a thread's
// own elements are 32 bytes apart or more where they are float32 or adjacent
// pairs: half of each sector, twice; 16411 tokens x 40 heads 71 us in bf16 and
// 141 in float32).  float32 rows leave the same way (101 us, as the threads hold
// them 102 to 108; bf16 54, through shared memory 55.5).
// HBM bounds it: bf16 (336 MB) in 53.6 us, 0.93 of the measured copy rate,
// float32 in 101, 0.98 (requested into registers 63.8 us at 16 warps an SM;
// sixteen threads a row, which need fewer, 78).  Blocks are small and take the
// memory that their heads need, so that a few thousand tokens are one even wave:
// 2049 tokens x 32 heads 7.6 us (with blocks of 256 threads 2 us more).
#include <cmath>
#include <type_traits>

#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_rope.cuh"
#include "tq_rows.cuh"

namespace tq {
namespace {

constexpr int kThreads = 128;

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

// Heads of a group: as many as 32 KB hold for a block.
template <int DT>
__host__ __device__ constexpr int heads_walked() {
    return DT == TQ_F32 ? 4 : 8;
}

// step(0), step(1), ... step(N - 1), each with its number as a constant.
template <int I, int N, class Step>
__device__ __forceinline__ void walk_heads(Step step) {
    if constexpr (I < N) {
        step(std::integral_constant<int, I>());
        walk_heads<I + 1, N>(step);
    }
}

// Thread (token, group of heads, chunk c of 8): the row's 16 elements of chunk c
// are two runs of 8, at elements e0 and e1.
template <int DT, bool HALF>
__global__ void __launch_bounds__(kThreads, 6) norm_rope_kernel(const __grid_constant__ tq_rope rope,
                                                                const __grid_constant__ NormRopeArgs a) {
    constexpr int NV = Elem<DT>::kVecs, ES = DT == TQ_F32 ? 4 : 2;
    // weights of the 16 elements of each chunk, four at a time side by side
    __shared__ float4 weight[2][4][8];
    const int pairs = rope.rot_dim / 2;
    auto runs = [&](int c, int &e0, int &e1) {
        const bool turned = 8 * c < pairs;
        e0 = HALF && turned ? 8 * c : 16 * c;
        e1 = HALF && turned ? pairs + 8 * c : 16 * c + 8;
    };
    if (threadIdx.x < 64) {
        const int which = threadIdx.x >> 5, j = (threadIdx.x >> 3) & 3, c = threadIdx.x & 7;
        int e0, e1;
        runs(c, e0, e1);
        const int e = (j < 2 ? e0 : e1) + 4 * (j & 1);
        const void *w = a.weight[which];
        weight[which][j][c] = make_float4(weight_at(w, a.weight_dtype, e), weight_at(w, a.weight_dtype, e + 1),
                                          weight_at(w, a.weight_dtype, e + 2), weight_at(w, a.weight_dtype, e + 3));
    }
    const int c = threadIdx.x & 7;
    const unsigned lanes = 0xFFu << (threadIdx.x & 24);   // the threads of this row
    const int per_tok = a.groups[0] + a.groups[1];
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 8) + (threadIdx.x >> 3), n = unit / per_tok;
    int first = (int)(unit - n * per_tok);
    const int which = first >= a.groups[0];
    first = (first - (which ? a.groups[0] : 0)) * a.walk;
    const int end = n < a.n_tok ? min(first + a.walk, a.heads[which]) : 0;
    const bool turned = 8 * c < pairs;   // chunks past the rotated elements are normalised only
    int e0, e1;
    runs(c, e0, e1);
    const int64_t head = a.head[which], o_head = a.o_head[which];
    const uint8_t *x = a.x[which] + n * a.tok[which];
    uint8_t *o = a.out[which] + n * a.o_tok[which];
    // the group's heads: vector v of head u's row at [u][group of threads][place(v)], where eight threads
    // meet all banks whether they read v apart by 1, 2 or 4
    extern __shared__ uint4 held[];
    constexpr int kWalk = heads_walked<DT>(), kRow = 16 * NV;
    auto row_of = [&](int u) { return held + (u * (kThreads / 8) + (threadIdx.x >> 3)) * kRow; };
    auto place = [](int v) { return v ^ (v >> 3); };
#pragma unroll
    for (int u = 0; u < kWalk; ++u) {
        if (first + u < end) {
            const uint8_t *xr = x + (first + u) * head;
#pragma unroll
            for (int i = 0; i < 2 * NV; ++i) {
                const int v = 8 * i + c;
                const uint32_t dst = (uint32_t)__cvta_generic_to_shared(row_of(u) + place(v));
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(xr + 16 * v) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    float2 sn[4], cs[4];   // of the chunk's pairs 2k, 2k + 1
    if (turned && end > 0) {
        int64_t ps[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) ps[i] = a.pos[(i < rope.axes ? i : 0) * a.pos_axis + n];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i0 = 8 * c + 2 * k, a0 = rope.axis[i0], a1 = rope.axis[i0 + 1];
            rope_sincos(rope_turns(rope.turn[i0], a0 == 0 ? ps[0] : a0 == 1 ? ps[1] : ps[2]), sn[k].x, cs[k].x);
            rope_sincos(rope_turns(rope.turn[i0 + 1], a1 == 0 ? ps[0] : a1 == 1 ? ps[1] : ps[2]), sn[k].y, cs[k].y);
        }
    }
    __syncthreads();
    walk_heads<0, kWalk>([&](auto at) {
        constexpr int u = decltype(at)::value;
        asm volatile("cp.async.wait_group %0;" ::"n"(kWalk - 1 - u) : "memory");
        if (first + u >= end) return;
        __syncwarp(lanes);
        uint4 *row = row_of(u);
        uint4 va[NV], vb[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            va[i] = row[place(e0 * ES / 16 + i)];
            vb[i] = row[place(e1 * ES / 16 + i)];
        }
        float f[8], g[8];
        unpack8<DT>(va, f);
        unpack8<DT>(vb, g);
        float2 y[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            y[k] = make_float2(f[2 * k], f[2 * k + 1]);
            y[k + 4] = make_float2(g[2 * k], g[2 * k + 1]);
        }
        const float r = inverse_rms(y, a.eps, lanes);
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 w = weight[which][j][c];
            y[2 * j] = __fmul2_rn(__fmul2_rn(y[2 * j], r2), make_float2(w.x, w.y));
            y[2 * j + 1] = __fmul2_rn(__fmul2_rn(y[2 * j + 1], r2), make_float2(w.z, w.w));
        }
        if (turned) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (HALF) {
                    // pairs 2k, 2k + 1: elements 2k, 2k + 1 of both runs
                    const float2 p = y[k], q = y[k + 4], ns = make_float2(-sn[k].x, -sn[k].y);
                    y[k] = __ffma2_rn(p, cs[k], __fmul2_rn(q, ns));
                    y[k + 4] = __ffma2_rn(q, cs[k], __fmul2_rn(p, sn[k]));
                } else {
                    // pair 2k + e: elements 4k + 2e, 4k + 2e + 1 of the 16
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float s1 = e ? sn[k].y : sn[k].x, c1 = e ? cs[k].y : cs[k].x;
                        const float2 p = y[2 * k + e];
                        y[2 * k + e] = __ffma2_rn(p, make_float2(c1, c1), __fmul2_rn(make_float2(p.y, p.x), make_float2(-s1, s1)));
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[2 * k] = y[k].x;
            f[2 * k + 1] = y[k].y;
            g[2 * k] = y[k + 4].x;
            g[2 * k + 1] = y[k + 4].y;
        }
        uint4 ra[NV], rb[NV];
        pack8<DT>(f, ra);
        pack8<DT>(g, rb);
        uint8_t *orow = o + (first + u) * o_head;
        if constexpr (NV == 2) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                row[place(e0 * ES / 16 + i)] = ra[i];
                row[place(e1 * ES / 16 + i)] = rb[i];
            }
            __syncwarp(lanes);
#pragma unroll
            for (int i = 0; i < 2 * NV; ++i)
                __stcs(reinterpret_cast<uint4 *>(orow) + 8 * i + c, row[place(8 * i + c)]);
        } else {
            __stcs(reinterpret_cast<uint4 *>(orow + e0 * ES), ra[0]);
            __stcs(reinterpret_cast<uint4 *>(orow + e1 * ES), rb[0]);
        }
    });
}

template <int DT, bool HALF>
int launch_style(const tq_rope &rope, const NormRopeArgs &a, unsigned grid, cudaStream_t st) {
    constexpr int each = 2 * Elem<DT>::kVecs * 16 * kThreads;
    static int done[64] = {0};
    if (set_smem_limit((const void *)norm_rope_kernel<DT, HALF>, heads_walked<DT>() * each, done) != TQ_OK)
        return TQ_ERR_CUDA;
    norm_rope_kernel<DT, HALF><<<grid, kThreads, a.walk * each, st>>>(rope, a);
    return launch_status();
}

template <int DT>
int launch(const tq_rope &rope, const NormRopeArgs &a, unsigned grid, cudaStream_t st) {
    return rope.style == TQ_ROPE_HALF ? launch_style<DT, true>(rope, a, grid, st) : launch_style<DT, false>(rope, a, grid, st);
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
    if ((int64_t)q_heads + k_heads > (1 << 26) || n_tok > ((int64_t)1 << 36)) return TQ_ERR_UNSUPPORTED;
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
    // GPU (128 per SM; on 2049 tokens x 32 heads 7.6 us, with 256 10.2, with 64 8.4) they walk as many
    // heads as a block holds
    int walk = 1;
    const int most = dtype == TQ_F32 ? heads_walked<TQ_F32>() : heads_walked<TQ_BF16>();
    while (walk < most && n_tok * ((int64_t)q_heads + k_heads) > (int64_t)sm_count() * 128 * walk) walk *= 2;
    a.walk = walk;
    a.groups[0] = (q_heads + walk - 1) / walk;
    a.groups[1] = (k_heads + walk - 1) / walk;
    constexpr int per = kThreads / 8;
    const int64_t per_tok = a.groups[0] + a.groups[1];
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
