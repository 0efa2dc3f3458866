// Rotary positions with one to three axes: the host-side tables
// (tq_rope_load, tq_rope_set_freqs) and tq_rope_apply.
//
// tq_rope_apply: pair i = (a, b) of every head of token n becomes
// (a cos t - b sin t, b cos t + a sin t), t = pos[axis(i)][n] * f_i, in
// float32, rounded once to the rows' type.  Each element is read and written
// once (the floor; the positions are 8 bytes per token and axis): a thread
// owns 8 pairs of one token, takes their sines and cosines once and walks
// the token's heads with them, so the trigonometry (about 25 instructions a
// pair) is shared by all the heads it visits.
#include <cmath>
#include <cstring>

#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_rope.cuh"
#include "tq_rows.cuh"

namespace tq {
namespace {

constexpr int kThreads = 256;

struct RopeArgs {
    const uint8_t *x;
    uint8_t *out;
    const int64_t *pos;
    int64_t n_tok, x_tok, x_head, o_tok, o_head, pos_axis;   // strides in bytes (pos: elements)
    int heads, slots;                                        // head slots of a block: each walks heads slot, slot + slots, ...
};

// Thread (token, head slot, chunk c of 8): the row's 16 elements of chunk c
// are two runs of 8, at elements e0 and e1.
template <int DT, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ tq_rope rope,
                                                        const __grid_constant__ RopeArgs a) {
    constexpr int NV = Elem<DT>::kVecs, ES = DT == TQ_F32 ? 4 : 2;
    __shared__ uint64_t turn[kRopePairs];
    __shared__ uint8_t axis[kRopePairs];
    if (threadIdx.x < kRopePairs) {
        turn[threadIdx.x] = rope.turn[threadIdx.x];
        axis[threadIdx.x] = rope.axis[threadIdx.x];
    }
    __syncthreads();
    const int c = threadIdx.x & 7, row = threadIdx.x >> 3;
    const int slot = row % a.slots;
    const int64_t n = (int64_t)blockIdx.x * (kThreads / 8 / a.slots) + row / a.slots;
    if (n >= a.n_tok) return;
    const int pairs = rope.rot_dim / 2;
    const bool turned = 8 * c < pairs;   // chunks past the rotated elements are copied
    const int e0 = HALF && turned ? 8 * c : 16 * c;
    const int e1 = HALF && turned ? pairs + 8 * c : 16 * c + 8;
    const uint8_t *x = a.x + n * a.x_tok;
    uint8_t *o = a.out + n * a.o_tok;
    // heads go by in batches of kBatch; a batch is loaded before the sines (and the batch before it) are needed
    constexpr int kBatch = DT == TQ_F32 ? 2 : 4;
    uint4 va[kBatch][NV], vb[kBatch][NV];
    auto load = [&](int h0) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int h = h0 + q * a.slots;
            if (h < a.heads) {
                const uint8_t *xr = x + h * a.x_head;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    va[q][i] = __ldcs(reinterpret_cast<const uint4 *>(xr + e0 * ES) + i);
                    vb[q][i] = __ldcs(reinterpret_cast<const uint4 *>(xr + e1 * ES) + i);
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
        for (int k = 0; k < 8; ++k) {
            const int ax = axis[8 * c + k];
            const int64_t t = ax == 0 ? p[0] : ax == 1 ? p[1] : p[2];
            rope_sincos(rope_turns(turn[8 * c + k], t), sn[k], cs[k]);
        }
    }
    for (int h0 = slot; h0 < a.heads; h0 += kBatch * a.slots) {
        uint4 ra[kBatch][NV], rb[kBatch][NV];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                ra[q][i] = va[q][i];
                rb[q][i] = vb[q][i];
            }
            if (turned && h0 + q * a.slots < a.heads) {
                float fa[8], fb[8], ga[8], gb[8];
                unpack8<DT>(ra[q], fa);
                unpack8<DT>(rb[q], fb);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if constexpr (HALF) {
                        ga[k] = fmaf(fa[k], cs[k], -(fb[k] * sn[k]));
                        gb[k] = fmaf(fb[k], cs[k], fa[k] * sn[k]);
                    } else {
                        // pair k of the chunk: elements 2k, 2k + 1 of its 16
                        float *src = k < 4 ? fa : fb, *dst = k < 4 ? ga : gb;
                        const int m = 2 * (k & 3);
                        dst[m] = fmaf(src[m], cs[k], -(src[m + 1] * sn[k]));
                        dst[m + 1] = fmaf(src[m + 1], cs[k], src[m] * sn[k]);
                    }
                }
                pack8<DT>(ga, ra[q]);
                pack8<DT>(gb, rb[q]);
            }
        }
        load(h0 + kBatch * a.slots);   // (rows in place: other heads than the ones written now)
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int h = h0 + q * a.slots;
            if (h < a.heads) {
                uint8_t *orow = o + h * a.o_head;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    __stcs(reinterpret_cast<uint4 *>(orow + e0 * ES) + i, ra[q][i]);
                    __stcs(reinterpret_cast<uint4 *>(orow + e1 * ES) + i, rb[q][i]);
                }
            }
        }
    }
}

template <int DT>
int launch(const tq_rope &rope, const RopeArgs &a, unsigned grid, cudaStream_t st) {
    if (rope.style == TQ_ROPE_HALF)
        rope_kernel<DT, true><<<grid, kThreads, 0, st>>>(rope, a);
    else
        rope_kernel<DT, false><<<grid, kThreads, 0, st>>>(rope, a);
    return launch_status();
}

// f radians per position as a fraction of a turn in 2^-64 units, modulo one
// turn: f / (2 pi) as the exact product with a two-term 1 / (2 pi).
uint64_t turn_of(double f) {
    const double hi = 0.15915494309189535, lo = -9.839338337591243e-18;   // 1 / (2 pi)
    const double p = f * hi, e = std::fma(f, hi, -p) + f * lo;
    double whole;
    const double frac = std::modf(p, &whole);   // exact
    const double a = std::ldexp(frac, 64), b = std::ldexp(e, 64);
    // a lies in (-2^64, 2^64): as a sum of two halves it fits signed integers
    const double ah = std::floor(std::ldexp(a, -32)), al = a - std::ldexp(ah, 32);
    return ((uint64_t)(int64_t)ah << 32) + (uint64_t)(int64_t)std::nearbyint(al) + (uint64_t)(int64_t)std::nearbyint(b);
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" int tq_rope_set_freqs(tq_rope *rope, const double *freqs) {
    if (!rope || !freqs) return TQ_ERR_ARG;
    if (!rope_ok(rope)) return TQ_ERR_UNSUPPORTED;
    for (int i = 0; i < rope->rot_dim / 2; ++i)
        if (!(std::fabs(freqs[i]) <= 1024.0)) return TQ_ERR_ARG;
    for (int i = 0; i < rope->rot_dim / 2; ++i) rope->turn[i] = turn_of(freqs[i]);
    return TQ_OK;
}

extern "C" int tq_rope_load(int head_dim, int rot_dim, double base, int style, int axes, const int *sections,
                            int interleaved, tq_rope *out) {
    if (!out || !sections) return TQ_ERR_ARG;
    if (!(base > 1.0) || !std::isfinite(base)) return TQ_ERR_ARG;
    if (head_dim != kD || rot_dim < 32 || rot_dim > kD || (rot_dim & 31) || axes < 1 || axes > 3 ||
        (style != TQ_ROPE_HALF && style != TQ_ROPE_ADJACENT))
        return TQ_ERR_UNSUPPORTED;
    const int pairs = rot_dim / 2;
    int sum = 0;
    for (int i = 0; i < axes; ++i) {
        if (sections[i] < 0 || sections[i] > pairs) return TQ_ERR_ARG;
        if (interleaved && i > 0 && axes * sections[i] > pairs) return TQ_ERR_ARG;
        sum += sections[i];
    }
    if (sum != pairs) return TQ_ERR_ARG;
    tq_rope r;
    std::memset(&r, 0, sizeof(r));
    r.head_dim = head_dim;
    r.rot_dim = rot_dim;
    r.style = style;
    r.axes = axes;
    double freqs[kRopePairs];
    for (int i = 0, a = 0, used = 0; i < pairs; ++i, ++used) {
        if (interleaved) {
            const int j = i % axes;
            r.axis[i] = (uint8_t)(j > 0 && i < axes * sections[j] ? j : 0);
        } else {
            while (used == sections[a]) {
                ++a;
                used = 0;
            }
            r.axis[i] = (uint8_t)a;
        }
        freqs[i] = std::pow(base, -2.0 * i / rot_dim);
    }
    const int st = tq_rope_set_freqs(&r, freqs);
    if (st != TQ_OK) return st;
    *out = r;
    return TQ_OK;
}

extern "C" int tq_rope_apply(const void *x, int dtype, int64_t n_tok, int heads, int64_t x_tok_stride,
                             int64_t x_head_stride, const int64_t *pos, int64_t pos_axis_stride, const tq_rope *rope,
                             void *out, int64_t out_tok_stride, int64_t out_head_stride, void *stream) {
    if (!rope || n_tok < 0 || heads <= 0) return TQ_ERR_ARG;
    const int es = dtype_bytes(dtype);
    if (!es || !rope_ok(rope)) return TQ_ERR_UNSUPPORTED;
    if (n_tok == 0) return TQ_OK;
    if (!x || !pos || !out || x_tok_stride < 0 || x_head_stride < 0 || out_tok_stride < 0 || out_head_stride < 0 ||
        pos_axis_stride < 0)
        return TQ_ERR_ARG;
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(pos, 8) || ((x_tok_stride * es) & 15) ||
        ((x_head_stride * es) & 15) || ((out_tok_stride * es) & 15) || ((out_head_stride * es) & 15))
        return TQ_ERR_ALIGN;
    if (rows_overlap(n_tok, out_tok_stride, heads, out_head_stride)) return TQ_ERR_ARG;
    RopeArgs a;
    a.x = static_cast<const uint8_t *>(x);
    a.out = static_cast<uint8_t *>(out);
    a.pos = pos;
    a.n_tok = n_tok;
    a.x_tok = x_tok_stride * es;
    a.x_head = x_head_stride * es;
    a.o_tok = out_tok_stride * es;
    a.o_head = out_head_stride * es;
    a.pos_axis = pos_axis_stride;
    a.heads = heads;
    // head slots of a block (32 rows of 8 threads): with few tokens every head has threads of its
    // own; once the rows fill the GPU (about 256 per SM) a thread walks up to 8 heads
    int slots = 32;
    while (slots > 1 &&
           (slots / 2 >= heads || (slots * 4 >= heads && n_tok * slots > (int64_t)sm_count() * 256)))
        slots /= 2;
    a.slots = slots;
    const int64_t per = kThreads / 8 / slots, grid = (n_tok + per - 1) / per;
    if (grid > 0x7FFFFFFF) return TQ_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case TQ_BF16: return launch<TQ_BF16>(*rope, a, (unsigned)grid, st);
        case TQ_F16: return launch<TQ_F16>(*rope, a, (unsigned)grid, st);
        default: return launch<TQ_F32>(*rope, a, (unsigned)grid, st);
    }
}
