// Quantise-on-insert of new tokens: rotary positions on the keys, then keys
// and values rotated (H D), normalised, quantised and packed into the cache's
// blocks, all heads of all tokens in one launch (tq_insert_kv).
//
// For each key row k of token n: x = rope(k, pos[n]) (float32, never rounded
// in between), nrm = ||x||, y = H (D x) / (sqrt(128) nrm), code_j =
// #{i : b_i <= y_j}, block = [fp16 nrm][packed codes]; a value row the same
// without rope.  Each row is read once and each block written once (the floor:
// 256 + 66 bytes for a 16-bit row at 4 bits); the rotation, 7 x 128 additions
// a row, and the quantiser, about 8 instructions an element, make instruction
// issue the bound.
//
// Layout.  A CTA takes 16 tokens and four warps; a warp takes the 16 tokens
// of one head at a time, two threads per row (element map of fwht_pair128, in
// which elements j and j + 64 of a row are the two halves of one packed
// pair).  The sines and cosines of the 16 tokens are computed once per CTA
// and shared by its heads; the sign diagonal D is folded in: the rows' sign
// bits are flipped as they are unpacked, and the sine of a pair whose two
// signs differ is negated.
//
// Codes.  The quantiser works in v = 63 y: adding 1.5 * 2^23 rounds v to an
// integer whose low 7 bits select one of 128 cells; a cell holds at most one
// boundary b (checked on the host) and the number of boundaries below it, and
// the sign of v - b finishes the count.  The table has 16 copies (one per
// lane of a half warp), so the 8-byte loads meet no bank conflict.
//
// Borders.  Decisions are those of 64-bit arithmetic (y rounded once to
// float32 and compared with the float32 boundaries), although the row is
// transformed in float32: a row with a coordinate closer to a boundary than
// kEps (far above the float32 error), a norm close to a rounding border of
// fp16 or a sum of squares outside float32's safe range is taken again by its
// whole warp in double precision (about 0.4% of rows).
#include <cmath>
#include <cstring>

#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_rope.cuh"

namespace tq {
namespace {

constexpr int kTok = 16;             // tokens of a CTA
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kGrid = 63.f;        // cells per unit of y
// Distance to a boundary, in v = 63 y, below which a row is decided in double
// precision: 2e-6 of a coordinate's standard deviation (1 / sqrt(128)).  The
// float32 path is off by about 1.2e-7 of it (rms: rope, seven butterfly
// stages and the scale, each half an ulp of partial sums of the row's size).
constexpr float kEps = 2e-6f * kGrid * 0.08838834764831845f;

enum { kRopeNone = 0, kRopeHalf1, kRopeHalf2, kRopeHalf3, kRopeHalf4, kRopeAdjacent };

struct Side {
    const uint8_t *x;       // rows
    uint8_t *blocks;
    int64_t tok, head;      // row strides in bytes
    int64_t n_blocks;
    float b[15];            // boundaries
    int bits;
    int style;              // kRope*
};

struct InsertArgs {
    Side side[2];           // keys, values
    const int64_t *pos, *dst;
    int64_t n_tok, pos_axis, dst_head;
    int heads, heads_per_cta, groups;   // groups of heads per token tile
    uint32_t signs[4];
};

struct Shared {
    uint2 cells[128 * 16];                    // (boundary, boundaries below + 1) x 16 copies
    float2 cs[kRopePairs][kTok];              // (cos, sin'), sin' negated where the pair's signs differ
    alignas(16) uint16_t stage[kWarps][kTok * 33 + 8];   // packed blocks of a warp's 16 rows
    double2 cs64[kWarps][kRopePairs];         // a row's cos and sin (double-precision path)
};

template <int DT>
struct Row {
    static constexpr int kVecs = DT == TQ_F32 ? 2 : 1;
    static constexpr int kBytes = DT == TQ_F32 ? 4 : 2;
};

// Element e of a row as a double.
template <int DT>
__device__ __forceinline__ double elem_double(const uint8_t *row, int e) {
    if constexpr (DT == TQ_F32) return (double)reinterpret_cast<const float *>(row)[e];
    else if constexpr (DT == TQ_BF16)
        return (double)__uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(row)[e] << 16);
    else
        return (double)__half2float(reinterpret_cast<const __half *>(row)[e]);
}

// One row by a whole warp in double precision: lane l holds elements
// 4 l .. 4 l + 3.  Returns the fp16 norm; code[i] is the code of element
// 4 l + i.
template <int DT>
__device__ __noinline__ uint32_t row_double(const uint8_t *row, const Side &sd, const tq_rope &rope,
                                            const InsertArgs &a, int64_t tok, double2 *cs64, uint32_t (&code)[4]) {
    const int lane = threadIdx.x & 31;
    double v[4];
    if (sd.style != kRopeNone) {
        const int pairs = rope.rot_dim / 2;
        for (int i = lane; i < pairs; i += 32) {
            const int64_t t = a.pos[rope.axis[i] * a.pos_axis + tok];
            double s, c;
            rope_sincos_double(rope_turns(rope.turn[i], t), s, c);
            cs64[i] = make_double2(c, s);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = 4 * lane + i;
            v[i] = elem_double<DT>(row, e);
            if (e < 2 * pairs) {
                const bool half = sd.style != kRopeAdjacent;
                const int pr = half ? (e < pairs ? e : e - pairs) : e >> 1;
                const bool second = half ? e >= pairs : (e & 1) != 0;
                const int other = half ? (second ? e - pairs : e + pairs) : e ^ 1;
                const double2 t = cs64[pr];
                const double o = elem_double<DT>(row, other);
                v[i] = fma(v[i], t.x, second ? o * t.y : -o * t.y);
            }
        }
        __syncwarp();
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = elem_double<DT>(row, 4 * lane + i);
    }
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) ss = fma(v[i], v[i], ss);
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    const double nrm = sqrt(ss);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if ((a.signs[lane >> 3] >> (4 * (lane & 7) + i)) & 1u) v[i] = -v[i];
    const double x0 = v[0] + v[1], x1 = v[0] - v[1], x2 = v[2] + v[3], x3 = v[2] - v[3];
    v[0] = x0 + x2;
    v[2] = x0 - x2;
    v[1] = x1 + x3;
    v[3] = x1 - x3;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double o = __shfl_xor_sync(0xffffffffu, v[i], m);
            v[i] = (lane & m) ? o - v[i] : v[i] + o;
        }
    }
    const double f = ss > 0.0 ? 1.0 / (nrm * 11.313708498984761) : 0.0;   // sqrt(128)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float y = (float)(v[i] * f);
        uint32_t n = 0;
        for (int j = 0; j < (1 << sd.bits) - 1; ++j) n += sd.b[j] <= y ? 1u : 0u;
        code[i] = n;
    }
    return __half_as_ushort(__double2half(nrm));
}

// fp16 norm of a row by a whole warp, from its unrotated elements (rope keeps
// the norm), in double precision.
template <int DT>
__device__ __noinline__ uint32_t norm_double(const uint8_t *row) {
    const int lane = threadIdx.x & 31;
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double v = elem_double<DT>(row, 4 * lane + i);
        ss = fma(v, v, ss);
    }
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    return __half_as_ushort(__double2half(sqrt(ss)));
}

// Rotary positions on a row in the layout of fwht_pair128: element 16 c + 8 h
// + k is p[c & 3][k].x (c < 4) or .y.
template <int M>
__device__ __forceinline__ void rope_half(float2 (&p)[4][8], const float2 (*cs)[kTok], int tok, int h) {
#pragma unroll
    for (int c = 0; c < M; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 t = cs[16 * c + 8 * h + k][tok];
            float &fa = c < 4 ? p[c & 3][k].x : p[c & 3][k].y;
            float &fb = c + M < 4 ? p[(c + M) & 3][k].x : p[(c + M) & 3][k].y;
            const float va = fa, vb = fb;
            fa = fmaf(va, t.x, -(vb * t.y));
            fb = fmaf(vb, t.x, va * t.y);
        }
}

__device__ __forceinline__ void rope_adjacent(float2 (&p)[4][8], const float2 (*cs)[kTok], int tok, int h) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            const int i = 8 * c + 4 * h + k / 2;
            const float2 t = cs[i][tok], u = cs[i + 32][tok];   // elements below and from 64 on
            const float2 va = p[c][k], vb = p[c][k + 1];
            p[c][k] = make_float2(fmaf(va.x, t.x, -(vb.x * t.y)), fmaf(va.y, u.x, -(vb.y * u.y)));
            p[c][k + 1] = make_float2(fmaf(vb.x, t.x, va.x * t.y), fmaf(vb.y, u.x, va.y * u.y));
        }
}

// Codes of this thread's 64 elements of a row, packed: for chunk c (0..7) and
// element 16 c + 8 h + k the BITS-wide field k of w[c].  Returns the smallest
// |v - b| met.
template <int BITS>
__device__ __forceinline__ float quantise(const float2 (&p)[4][8], float scale, const uint2 *cells, uint32_t (&w)[8]) {
    float near = 1.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        uint32_t acc = 0;
#pragma unroll
        for (int k = 7; k >= 0; --k) {
            const float u = c < 4 ? p[c & 3][k].x : p[c & 3][k].y;
            const uint32_t cell = __float_as_uint(fmaf(u, scale, 12582912.f + 64.f)) & 127u;
            const uint2 e = cells[cell * 16];
            const float t = fmaf(u, scale, -__uint_as_float(e.x));
            near = fminf(near, fabsf(t));
            acc = (acc << BITS) + e.y + (uint32_t)(__float_as_int(t) >> 31);
        }
        w[c] = acc;
    }
    return near;
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 4) insert_kernel(const __grid_constant__ tq_rope rope,
                                                             const __grid_constant__ InsertArgs a, int sides, int first) {
    constexpr int NV = Row<DT>::kVecs, ES = Row<DT>::kBytes;
    extern __shared__ __align__(16) uint8_t dsmem[];
    Shared &sm = *reinterpret_cast<Shared *>(dsmem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = lane & 1, r = lane >> 1;
    const Side &sd = a.side[first + blockIdx.x % sides];
    const int64_t unit = blockIdx.x / sides;
    const int64_t tok0 = unit / a.groups * kTok;
    const int head0 = (int)(unit % a.groups) * a.heads_per_cta;
    const int bits = sd.bits, levels = 1 << bits, bytes = 2 + 16 * bits;
    const int64_t tok = min64(tok0 + r, a.n_tok - 1);   // this thread's token

    static_assert(kThreads == 128, "a thread per cell");
    {
        uint32_t below = 0;
        float edge = 3.0e38f;   // a cell without a boundary: v - edge < 0 for every v
        for (int j = 0; j < levels - 1; ++j) {
            const float v = sd.b[j] * kGrid;
            const int at = (int)(__float_as_uint(v + (12582912.f + 64.f)) & 127u);
            if (at < tid) ++below;
            if (at == tid) edge = v;
        }
        const uint2 e = make_uint2(__float_as_uint(edge), below + 1);
#pragma unroll
        for (int i = 0; i < 16; ++i) sm.cells[tid * 16 + ((i + tid) & 15)] = e;
    }
    if (sd.style != kRopeNone) {
        for (int i = tid; i < kRopePairs * kTok; i += kThreads) {
            const int pr = i / kTok, t = i % kTok;
            float s = 0.f, c = 1.f;
            if (pr < rope.rot_dim / 2) {
                const int64_t n = min64(tok0 + t, a.n_tok - 1);
                rope_sincos(rope_turns(rope.turn[pr], a.pos[rope.axis[pr] * a.pos_axis + n]), s, c);
                const int ea = sd.style == kRopeAdjacent ? 2 * pr : pr;
                const int eb = sd.style == kRopeAdjacent ? ea + 1 : pr + rope.rot_dim / 2;
                if (((a.signs[ea >> 5] >> (ea & 31)) ^ (a.signs[eb >> 5] >> (eb & 31))) & 1u) s = -s;
            }
            sm.cs[pr][t] = make_float2(c, s);
        }
    }
    __syncthreads();

    const int64_t dst = tok0 + r < a.n_tok ? a.dst[tok] : -1;
    uint16_t *stage = sm.stage[warp];
    const uint2 *cells = sm.cells + (lane & 15);
    const int head_end = min(head0 + a.heads_per_cta, a.heads);
    for (int head = head0 + warp; head < head_end; head += kWarps) {
        const uint8_t *row = sd.x + tok * sd.tok + head * sd.head;
        uint4 raw[8][NV];
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                raw[c][i] = __ldcs(reinterpret_cast<const uint4 *>(row + (16 * c + 8 * h) * ES) + i);
        float2 p[4][8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            // elements 16 c + 8 h .. + 7: their signs are bits 16 (c & 1) + 8 h .. of word c / 2
            const uint32_t sg = a.signs[c >> 1] >> (16 * (c & 1) + 8 * h);
            float f[8];
            if constexpr (DT == TQ_F32) {
                const uint32_t w[8] = {raw[c][0].x, raw[c][0].y, raw[c][0].z, raw[c][0].w,
                                       raw[c][NV - 1].x, raw[c][NV - 1].y, raw[c][NV - 1].z, raw[c][NV - 1].w};
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(w[k] ^ ((sg << (31 - k)) & 0x80000000u));
            } else {
                uint32_t w[4] = {raw[c][0].x, raw[c][0].y, raw[c][0].z, raw[c][0].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    w[k] ^= ((sg << (15 - 2 * k)) & 0x8000u) | ((sg << (30 - 2 * k)) & 0x80000000u);
                    if constexpr (DT == TQ_BF16) {
                        f[2 * k] = bf16_bits_lo(w[k]);
                        f[2 * k + 1] = bf16_bits_hi(w[k]);
                    } else {
                        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
                        f[2 * k] = x.x;
                        f[2 * k + 1] = x.y;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (c < 4) p[c & 3][k].x = f[k];
                else p[c & 3][k].y = f[k];
            }
        }
        switch (sd.style) {
            case kRopeHalf4: rope_half<4>(p, sm.cs, r, h); break;
            case kRopeHalf3: rope_half<3>(p, sm.cs, r, h); break;
            case kRopeHalf2: rope_half<2>(p, sm.cs, r, h); break;
            case kRopeHalf1: rope_half<1>(p, sm.cs, r, h); break;
            case kRopeAdjacent: rope_adjacent(p, sm.cs, r, h); break;
            default: break;
        }
        float2 acc2[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            acc2[c] = __fmul2_rn(p[c][0], p[c][0]);
#pragma unroll
            for (int k = 1; k < 8; ++k) acc2[c] = __ffma2_rn(p[c][k], p[c][k], acc2[c]);
        }
        const float2 a01 = add2(add2(acc2[0], acc2[1]), add2(acc2[2], acc2[3]));
        float ss = a01.x + a01.y;
        ss += __shfl_xor_sync(0xffffffffu, ss, 1);
        fwht_pair128(p, h ? -1.f : 1.f);
        const float nrm = sqrtf(ss);
        // 2^-100 .. 2^100: squares neither underflow nor overflow (false for a NaN as well)
        const bool safe = ss >= 7.888609052210118e-31f && ss <= 1.2676506002282294e30f;
        const float scale = kGrid * 0.08838834764831845f / nrm;
        uint32_t w[8];
        float near = bits == 4 ? quantise<4>(p, scale, cells, w)
                               : bits == 3 ? quantise<3>(p, scale, cells, w) : quantise<2>(p, scale, cells, w);
        uint32_t todo = __ballot_sync(0xffffffffu, !safe || near < kEps);
        todo = (todo | (todo >> 1)) & 0x55555555u;   // either thread of a row speaks for it
        uint32_t ties = __ballot_sync(0xffffffffu, near_fp16_tie_fast(nrm)) & 0x55555555u & ~todo;

        // stage the 16 blocks: half word 0 the norm, then the codes
        uint16_t *blk = stage + r * (bytes / 2);
        if (h == 0) blk[0] = __half_as_ushort(__float2half_rn(nrm));
        if (bits == 4) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                blk[1 + 4 * c + 2 * h] = (uint16_t)w[c];
                blk[2 + 4 * c + 2 * h] = (uint16_t)(w[c] >> 16);
            }
        } else if (bits == 2) {
#pragma unroll
            for (int c = 0; c < 8; ++c) blk[1 + 2 * c + h] = (uint16_t)w[c];
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                uint32_t lo = 0, hi = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    lo |= ((w[c] >> (3 * k)) & 3u) << (2 * k);
                    hi |= ((w[c] >> (3 * k + 2)) & 1u) << k;
                }
                blk[1 + 2 * c + h] = (uint16_t)lo;
                reinterpret_cast<uint8_t *>(blk)[34 + 2 * c + h] = (uint8_t)hi;
            }
        }
        __syncwarp();
        while (ties) {
            const int l = __ffs(ties) - 1, rr = l >> 1;
            ties &= ties - 1;
            const int64_t t = min64(tok0 + rr, a.n_tok - 1);
            const uint32_t nb = norm_double<DT>(sd.x + t * sd.tok + head * sd.head);
            if (lane == 0) stage[rr * (bytes / 2)] = (uint16_t)nb;
            __syncwarp();
        }
        while (todo) {
            const int l = __ffs(todo) - 1, rr = l >> 1;
            todo &= todo - 1;
            const int64_t t = min64(tok0 + rr, a.n_tok - 1);
            uint32_t code[4];
            const uint32_t nb = row_double<DT>(sd.x + t * sd.tok + head * sd.head, sd, rope, a, t, sm.cs64[warp], code);
            uint16_t *b = stage + rr * (bytes / 2);
            if (lane == 0) b[0] = (uint16_t)nb;
            if (bits == 4) {
                b[1 + lane] = (uint16_t)(code[0] | (code[1] << 4) | (code[2] << 8) | (code[3] << 12));
            } else {
                const uint32_t lo = (code[0] & 3u) | ((code[1] & 3u) << 2) | ((code[2] & 3u) << 4) | ((code[3] & 3u) << 6);
                reinterpret_cast<uint8_t *>(b)[2 + lane] = (uint8_t)lo;
                if (bits == 3) {
                    uint32_t hi = (code[0] >> 2) | ((code[1] >> 2) << 1) | ((code[2] >> 2) << 2) | ((code[3] >> 2) << 3);
                    hi |= __shfl_down_sync(0xffffffffu, hi, 1) << 4;
                    if (!(lane & 1)) reinterpret_cast<uint8_t *>(b)[34 + lane / 2] = (uint8_t)hi;
                }
            }
            __syncwarp();
        }

        // store: 16 consecutive block slots at a 16-byte boundary leave as one run, else block by block
        const int64_t slot = dst < 0 ? -1 : dst + head * a.dst_head;
        const bool ok = slot >= 0 && slot < sd.n_blocks;
        const int64_t slot0 = __shfl_sync(0xffffffffu, slot, 0);
        uint8_t *out0 = sd.blocks + slot0 * bytes;
        const bool run = __all_sync(0xffffffffu, ok && slot == slot0 + r) && ((uintptr_t)out0 & 15) == 0;
        if (run) {
            for (int i = lane; i < bytes; i += 32)
                reinterpret_cast<uint4 *>(out0)[i] = reinterpret_cast<const uint4 *>(stage)[i];
        } else {
            const uint32_t okm = __ballot_sync(0xffffffffu, ok);
            for (int q = 0; q < kTok; ++q) {
                if (!((okm >> (2 * q)) & 1u)) continue;
                const int64_t s = __shfl_sync(0xffffffffu, slot, 2 * q);
                uint16_t *o = reinterpret_cast<uint16_t *>(sd.blocks + s * bytes);
                const uint16_t *b = stage + q * (bytes / 2);
                for (int i = lane; i < bytes / 2; i += 32) o[i] = b[i];
            }
        }
        __syncwarp();
    }
}

template <int DT>
int launch(const tq_rope &rope, const InsertArgs &a, int sides, int first, unsigned grid, cudaStream_t st) {
    static int done[64] = {0};
    if (set_smem_limit((const void *)insert_kernel<DT>, (int)sizeof(Shared), done) != TQ_OK) return TQ_ERR_CUDA;
    insert_kernel<DT><<<grid, kThreads, sizeof(Shared), st>>>(rope, a, sides, first);
    return launch_status();
}

// The quantiser's cells hold at most one boundary each, and no boundary lies
// within 1/64 of a cell's edge (a coordinate near it is then always compared
// with it).  True of the codebooks of tq_codebook_load.
bool cells_ok(const tq_codebook *cb) {
    int last = -1;
    for (int i = 0; i < cb->levels - 1; ++i) {
        const float v = cb->boundaries[i] * kGrid;
        if (!(std::fabs(v) < 62.f)) return false;
        const float n = std::nearbyint(v);
        if (std::fabs(v - n) > 0.5f - 1.f / 64.f) return false;
        const int cell = (int)n + 64;
        if (cell <= last) return false;
        last = cell;
    }
    return true;
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" int tq_insert_kv(const void *k, int64_t k_tok_stride, int64_t k_head_stride, const void *v,
                            int64_t v_tok_stride, int64_t v_head_stride, int dtype, int64_t n_tok, int heads,
                            const int64_t *pos, int64_t pos_axis_stride, const tq_rope *rope, const tq_codebook *kcb,
                            const tq_codebook *vcb, tq_signs signs, uint8_t *k_blocks, uint8_t *v_blocks,
                            int64_t n_blocks, const int64_t *dst, int64_t dst_head_stride, void *stream) {
    if (n_tok < 0 || heads <= 0 || n_blocks < 0 || dst_head_stride < 0) return TQ_ERR_ARG;
    if ((k != nullptr) != (k_blocks != nullptr) || (v != nullptr) != (v_blocks != nullptr)) return TQ_ERR_ARG;
    if ((k && !kcb) || (v && !vcb) || (rope && !pos)) return TQ_ERR_ARG;
    const int es = dtype_bytes(dtype);
    if (!es) return TQ_ERR_UNSUPPORTED;
    if (rope && !rope_ok(rope)) return TQ_ERR_UNSUPPORTED;
    InsertArgs a;
    std::memset(&a, 0, sizeof(a));
    const void *xs[2] = {k, v};
    uint8_t *outs[2] = {k_blocks, v_blocks};
    const tq_codebook *cbs[2] = {kcb, vcb};
    const int64_t tok[2] = {k_tok_stride, v_tok_stride}, head[2] = {k_head_stride, v_head_stride};
    for (int i = 0; i < 2; ++i) {
        if (!xs[i]) continue;
        if (!codebook_ok(cbs[i]) || !cells_ok(cbs[i])) return TQ_ERR_UNSUPPORTED;
        if (tok[i] < 0 || head[i] < 0) return TQ_ERR_ARG;
        if (!aligned(xs[i], 16) || ((tok[i] * es) & 15) || ((head[i] * es) & 15) || !aligned(outs[i], 2))
            return TQ_ERR_ALIGN;
        Side &s = a.side[i];
        s.x = static_cast<const uint8_t *>(xs[i]);
        s.blocks = outs[i];
        s.tok = tok[i] * es;
        s.head = head[i] * es;
        s.n_blocks = n_blocks;
        s.bits = cbs[i]->bits;
        for (int j = 0; j < 15; ++j) s.b[j] = j < cbs[i]->levels - 1 ? cbs[i]->boundaries[j] : 0.f;
        s.style = kRopeNone;
        if (i == 0 && rope)
            s.style = rope->style == TQ_ROPE_ADJACENT ? (int)kRopeAdjacent : kRopeHalf1 + rope->rot_dim / 32 - 1;
    }
    if (n_tok == 0 || (!k && !v)) return TQ_OK;
    if (!dst) return TQ_ERR_ARG;
    if (!aligned(dst, 8) || (rope && !aligned(pos, 8))) return TQ_ERR_ALIGN;
    if (rope && pos_axis_stride < 0) return TQ_ERR_ARG;
    a.pos = pos;
    a.pos_axis = pos_axis_stride;
    a.dst = dst;
    a.dst_head = dst_head_stride;
    a.n_tok = n_tok;
    a.heads = heads;
    for (int i = 0; i < 4; ++i) a.signs[i] = signs.w[i];
    const int sides = (k != nullptr) + (v != nullptr), first = k ? 0 : 1;
    const int64_t tiles = (n_tok + kTok - 1) / kTok;
    // all heads of a token tile in one CTA share its sines; with few tiles four heads a CTA fill more SMs
    a.heads_per_cta = tiles * sides >= (int64_t)sm_count() * 4 ? heads : (heads < kWarps ? heads : kWarps);
    a.groups = (heads + a.heads_per_cta - 1) / a.heads_per_cta;
    const int64_t grid = tiles * a.groups * sides;
    if (grid > 0x7FFFFFFF) return TQ_ERR_UNSUPPORTED;
    tq_rope none;
    if (!rope) std::memset(&none, 0, sizeof(none));
    const tq_rope &r = rope ? *rope : none;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case TQ_BF16: return launch<TQ_BF16>(r, a, sides, first, (unsigned)grid, st);
        case TQ_F16: return launch<TQ_F16>(r, a, sides, first, (unsigned)grid, st);
        default: return launch<TQ_F32>(r, a, sides, first, (unsigned)grid, st);
    }
}
