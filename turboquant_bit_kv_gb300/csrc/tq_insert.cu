// Quantise-on-insert of new tokens: rotary positions on the keys, then keys
// and values rotated (H D), normalised, quantised and packed into the cache's
// blocks, all heads of all tokens in one launch (tq_insert_kv).
//
// For each key row k of token n: x = rope(k, pos[n]) (float32, never rounded
// in between), nrm = ||x||, y = H (D x) / (sqrt(128) nrm), code_j =
// #{i : b_i <= y_j}, block = [fp16 nrm][packed codes]; a value row the same
// without rope.  Each row is read once and each block written once (the floor:
// 256 + 66 bytes for a 16-bit row at 4 bits).  Instruction issue is what
// bounds the kernel, and the quantiser (about 6.5 instructions an element) the
// largest part of it.
//
// Layout.  A CTA takes 16 tokens and four warps; a warp takes the 16 tokens
// of one head at a time as the 16 rows of m16n8k16 products.  Thread (g, t) =
// (lane / 4, lane % 4) holds elements 32 c + 8 t .. + 7 (c = 0 .. 3) of rows g
// and g + 8.  H factors over the bits of the element index: bits 0, 1, 3 and 4
// are the k index of a product with the 16 x 16 Hadamard matrix (eight k-tiles
// of 16 elements, +-1 operands, exact), bits 2, 5 and 6 number the k-tiles and
// are three butterfly stages on the accumulators, which a thread holds all of:
// the transform costs no shuffle and no shared memory.  The columns are ordered
// so that a thread gets back the elements whose inputs it held.  Rows of 16-bit
// elements enter as they are; rotated (or float32) rows are scaled by a power
// of two to a norm of about 2^9 and split x = hi + lo into two fp16 parts (22
// bits; the float32 accumulation keeps 24).
//
// The sines and cosines of the 16 tokens are computed once per CTA and shared
// by its heads; the sign diagonal D is folded in: the rows' sign bits are
// flipped as they are loaded, and the sine of a pair whose two signs differ is
// negated.
//
// Codes.  The quantiser works in v = 63 y: adding 1.5 * 2^16 + 64.5 leaves v
// + 64.5 with seven fraction bits in the low mantissa bits, so that one AND
// gives the cell floor(v + 64.5) of 128 times the 128 bytes of its table row; a
// cell holds at most one boundary b (checked on the host) and the number of
// boundaries below it, and the sign of v - b finishes the count.  A row has 16
// copies (one per lane of a half warp), so the 8-byte loads meet no bank
// conflict.
//
// Borders.  Decisions are those of 64-bit arithmetic (y rounded once to
// float32 and compared with the float32 boundaries), although the row is
// transformed in float32: a row with a coordinate closer to a boundary, or a
// norm closer to a rounding border of fp16, than float32 arithmetic can be off
// whatever the row holds (the bounds below; up to 0.8% of rows for the codes,
// 0.2 to 0.4% for the norms) is listed, and when the CTA is through its tiles the
// listed rows are taken again, one by each of its warps (four for their norms
// alone): in float32 once more, and each coordinate near a boundary as one sum
// in double-float.  Rows of a sum of squares outside float32's safe range go
// through double precision.  (The double-precision pipe has one sixty-fourth of
// the float32 rate.  Of the 289 us of a prompt of 131072 tokens x 8 heads the
// listed rows are about 34: 23 more than with borders at the furthest wrong
// decision seen on random rows, which rows made for it get past.  Between the
// tiles, whenever 8, 16 or 32 rows are listed, they cost 77, 51 and 8 us more
// than at the end: their code is then fetched again.)  A CTA whose list
// overflows takes all its rows again.
//
// Few rows go to a kernel of their own, a warp per row (insert_few_kernel).
//
// CTAs are persistent, four per SM, each on keys or on values; a warp's next
// rows are on their way to shared memory (each thread copies what it will read
// itself) while it works on the current ones.
#include <cmath>
#include <cstring>

#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_rope.cuh"

namespace tq {
namespace {

constexpr int kTok = 16;             // tokens of a tile
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kGrid = 63.f;        // cells per unit of y
constexpr float kUnit = 5.568465901844061f;   // 63 / sqrt(128): a standard deviation in v = 63 y
// How far a coordinate can be off in float32, from the operations it goes
// through, all errors at their largest and in the same direction.  In units of
// u = 2^-24 of a coordinate's standard deviation (the row's norm / sqrt(128));
// the sizes of a row's elements add up to sqrt(128) = 11.3 of its norm at most,
// the norms of its 64 pairs to 8:
//   rope      24.3  sine and cosine, as a vector off by 2.15 u (all 2^32 angles
//                   evaluated), add up to sqrt(2) times that in a pair's sum
//             22.6  products and sums, 2 sqrt(2) u a pair
//   split     22.6  two fp16 parts: 2 u of each element
//   products  22.6  sums of 16 terms by the tensor cores, cut to 24 bits; they
//              1.4  also cut each term at 2^-25 of the largest one's power of two
//                   (as measured, sum by sum), which the lower parts' sum can
//                   lose by; terms within 2^14 of the largest lose nothing, and a
//                   smaller one takes more from the sizes' sum than its cut adds
//   stages    11.3  each butterfly stage but the last: three after the products,
//                   seven in insert_few_kernel
// and, times the coordinate (the outermost boundary b at most): the norm 4.5 (10
// more from the products where it is taken from their results; few rows 4), its
// inverse 1.5, the constant and its product 1.6, the boundary in v 1, the
// rounding of y to float32 1, the last stage 1.  Each sum is raised by a
// hundredth and more for products of these errors.  (Rows whose errors do add up
// are easily made: pairs all alike at one angle are decided wrongly up to 2e-6
// of a standard deviation away.  Rows of random elements: 4.3e-7 in 1.2e9
// coordinates.)
struct Bound {
    float row, level;   // and times b
};
constexpr Bound kBoundRope = {118.f, 11.5f};     // rotated rows: 116.2 + 10.6 b
constexpr Bound kBoundSplit = {71.f, 11.5f};     // float32 rows without rope: 69.2 + 10.6 b
constexpr Bound kBoundDirect = {46.f, 22.f};     // 16-bit rows without rope: 45.2 + 20.6 b
constexpr Bound kBoundFewRope = {117.f, 11.5f};  // insert_few_kernel: 114.8 + 10.1 b
constexpr Bound kBoundFew = {69.f, 11.5f};       // 67.9 + 10.1 b

// How far a norm can be off, in units of its last float32 place (u of it at
// least): 4.5 (few rows 4) from the sum of squares, 1.5 from its inverse root, 1
// from their product, 10 more where the squares are of the products' results.
constexpr uint32_t kTieUlps = 8, kTieUlpsDirect = 18;

// Rows per SM, keys and values together, up to which a warp takes a row
// (insert_few_kernel).  us, against insert_kernel's, for bfloat16 keys with
// rotary positions in 4 bits and values in 2, 8 heads, by tokens: 16 4.2 / 11.5,
// 256 7.4 / 12.3, 512 9.0 / 12.8, 768 (81 rows per SM) 10.7 / 13.1, 1024 12.6 /
// 13.4, 1280 14.6 / 13.6, 2048 20.1 / 14.3.  Keys alone cross at 75, without
// rotary positions at 130 rows per SM.
constexpr int kFewRows = 80;

enum { kRopeNone = 0, kRopeHalf1, kRopeHalf2, kRopeHalf3, kRopeHalf4, kRopeAdjacent };

struct Side {
    const uint8_t *x;       // rows
    uint8_t *blocks;
    int64_t tok, head;      // row strides in bytes
    int64_t n_blocks;
    float b[15];            // boundaries
    float eps, eps_few;     // distance to a boundary, in v = 63 y, below which a coordinate is decided again; the
                            // same for insert_few_kernel's arithmetic
    uint32_t ulps;          // distance of the norm to a rounding border of fp16 below which it is rounded again
    int bits;
    int style;              // kRope*
};

struct InsertArgs {
    Side side[2];           // keys, values
    const int64_t *pos, *dst;
    int64_t n_tok, pos_axis, dst_head;
    int units;              // of a side: (tile group, head group) pairs
    int heads, heads_per_cta, groups;   // groups of heads per tile group
    int tiles;              // token tiles of a CTA at once: 4, 2 or 1 for 1, 2 or more heads
    int list;               // rows of either kind that a CTA can list
    int ctas[2];            // of each side
    uint32_t signs[4];
};

constexpr int kStage = kTok * 33 + 8;    // half words a warp stages its 16 blocks in (and the 128 values of a
                                         // row taken again)

struct Listed {     // a row to take again
    int unit;
    uint32_t row;   // head * 64 + token of the unit
};

struct Shared {
    uint2 cells[128 * 16];                    // (boundary, boundaries below + 1) x 16 copies
    alignas(16) uint16_t stage[kWarps][kStage];
    uint4 in[kWarps][8][32];                  // the next rows (16-bit types), as their threads read them
    uint4 flip[4][4];                         // sign bits of the 16-bit elements 32 c + 8 t .. + 7
    uint64_t turn[kRopePairs];                // the rope, and whether a pair's two signs differ (bit 2 of axis)
    uint8_t axis[kRopePairs];
    int listed[2];                            // rows to list: for their norms, and whole
    // cosines and sines (negated where the pair's two signs differ) of two
    // neighbouring pairs, (c, c', s, s'); unit u of token n and thread t at
    // [(u * 16 + n) * 4 + t].  Halves: unit 4 c + k holds pairs 32 c + 8 t + 2 k and the next.
    // Adjacent: unit 2 c + k holds pairs 16 c + 4 t + 2 k and the next.  A table per token tile, then the lists
    // of rows for their norms and of whole rows.
    alignas(16) float4 cs[][8 * kTok * 4];
};
__device__ __forceinline__ Listed *list_of(Shared &sm, int tiles) { return reinterpret_cast<Listed *>(sm.cs + tiles); }

template <int DT>
struct Row {
    static constexpr int kVecs = DT == TQ_F32 ? 2 : 1;
    static constexpr int kBytes = DT == TQ_F32 ? 4 : 2;
};

// Element e of a row.
template <int DT>
__device__ __forceinline__ float elem(const uint8_t *row, int e) {
    if constexpr (DT == TQ_F32) return reinterpret_cast<const float *>(row)[e];
    else if constexpr (DT == TQ_BF16)
        return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(row)[e] << 16);
    else
        return __half2float(reinterpret_cast<const __half *>(row)[e]);
}

// Rows taken again.  The code is kept small and in loops, values in shared
// memory: it runs seldom, and fetching instructions that are not in a cache
// costs more than executing them (unrolled, two rows of the same arithmetic
// took 20 us).

// Codes of elements 4 l .. 4 l + 3 (byte i of code) into a block.
__device__ __forceinline__ void write_codes(uint8_t *block, int bits, uint32_t code, int lane) {
    if (bits == 4) {
        code |= code >> 4;   // bytes 0 and 2 hold two codes each
        reinterpret_cast<uint16_t *>(block)[1 + lane] = (uint16_t)((code & 0xFFu) | ((code >> 8) & 0xFF00u));
        return;
    }
    const uint32_t low = code & 0x03030303u;
    block[2 + lane] = (uint8_t)(low | (low >> 6) | (low >> 12) | (low >> 18));
    if (bits == 3) {
        const uint32_t top = (code >> 2) & 0x01010101u;
        uint32_t hi = (top | (top >> 7) | (top >> 14) | (top >> 21)) & 15u;
        hi |= __shfl_down_sync(0xffffffffu, hi, 1) << 4;
        if (!(lane & 1)) block[34 + lane / 2] = (uint8_t)hi;
    }
}

// A value of either arithmetic, for the code that the two share.
__device__ __forceinline__ double add_(double a, double b) { return a + b; }
__device__ __forceinline__ ff add_(ff a, ff b) { return ff_add(a, b); }
__device__ __forceinline__ double neg_(double a) { return -a; }
__device__ __forceinline__ ff neg_(ff a) { return ff_neg(a); }
__device__ __forceinline__ double mul_(double a, double b) { return a * b; }
__device__ __forceinline__ ff mul_(ff a, ff b) { return ff_mul(a, b); }
__device__ __forceinline__ double scale_(double a, float b) { return a * (double)b; }
__device__ __forceinline__ ff scale_(ff a, float b) { return ff_scale(a, b); }
__device__ __forceinline__ double shfl_(double a, int m) { return __shfl_xor_sync(0xffffffffu, a, m); }
__device__ __forceinline__ ff shfl_(ff a, int m) {
    return {__shfl_xor_sync(0xffffffffu, a.h, m), __shfl_xor_sync(0xffffffffu, a.l, m)};
}
__device__ __forceinline__ void load_(double &v, float x) { v = (double)x; }
__device__ __forceinline__ void load_(ff &v, float x) { v = ff_of(x); }
__device__ __forceinline__ void sincos_(uint64_t f, double &s, double &c) { rope_sincos_double(f, s, c); }
__device__ __forceinline__ void sincos_(uint64_t f, ff &s, ff &c) { rope_sincos_ff(f, s, c); }

// One row by a warp in the arithmetic N: H (D x) of the rotated row into
// v[128]; the sum of the row's squares is returned.
template <int DT, class N>
__device__ __forceinline__ N transform_row(const uint8_t *row, const Side &sd, const tq_rope &rope, const InsertArgs &a,
                                           int64_t tok, N *v) {
    const int lane = threadIdx.x & 31;
    const int pairs = sd.style == kRopeNone ? 0 : rope.rot_dim / 2;
#pragma unroll 1
    for (int pr = lane; pr < kRopePairs; pr += 32) {
        const bool turned = pr < pairs, half = turned && sd.style != kRopeAdjacent;
        const int ea = half ? pr : 2 * pr, eb = half ? pr + pairs : 2 * pr + 1;
        const float xa = elem<DT>(row, ea), xb = elem<DT>(row, eb);
        N ra, rb;
        load_(ra, xa);
        load_(rb, xb);
        if (turned) {
            N s, c;
            sincos_(rope_turns(rope.turn[pr], a.pos[rope.axis[pr] * a.pos_axis + tok]), s, c);
            ra = add_(scale_(c, xa), scale_(s, -xb));
            rb = add_(scale_(c, xb), scale_(s, xa));
        }
        v[ea] = ra;
        v[eb] = rb;
    }
    __syncwarp();
    N ss;
    load_(ss, 0.f);
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const N x = v[32 * i + lane];
        ss = add_(ss, mul_(x, x));
        if ((a.signs[i] >> lane) & 1u) v[32 * i + lane] = neg_(x);
    }
#pragma unroll 1
    for (int m = 1; m < 32; m <<= 1) ss = add_(ss, shfl_(ss, m));
#pragma unroll 1
    for (int h = 1; h < kD; h <<= 1) {
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int n = 32 * q + lane, i = ((n & ~(h - 1)) << 1) | (n & (h - 1));
            const N x = v[i], y = v[i + h];
            v[i] = add_(x, y);
            v[i + h] = add_(x, neg_(y));
        }
    }
    __syncwarp();
    return ss;
}

// A row outside float32's safe range (not of zeros), in double precision.
template <int DT>
__device__ __noinline__ void range_row(const uint8_t *row, uint8_t *block, const Side &sd, const tq_rope &rope,
                                       const InsertArgs &a, int64_t tok, double *v) {
    const int lane = threadIdx.x & 31;
    const double nrm = sqrt(transform_row<DT, double>(row, sd, rope, a, tok, v));
    const double f = 1.0 / (nrm * 11.313708498984761);   // sqrt(128)
    uint32_t code = 0;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const float y = (float)(v[4 * lane + i] * f);
#pragma unroll 1
        for (int j = 0; j < (1 << sd.bits) - 1; ++j) code += sd.b[j] <= y ? 1u << (8 * i) : 0u;
    }
    if (lane == 0) *reinterpret_cast<__half *>(block) = __double2half(nrm);
    write_codes(block, sd.bits, code, lane);
}

// A row whose codes float32 does not decide, in double-float.
template <int DT>
__device__ __noinline__ void near_row(const uint8_t *row, uint8_t *block, const Side &sd, const tq_rope &rope,
                                      const InsertArgs &a, int64_t tok, ff *v) {
    const int lane = threadIdx.x & 31;
    const ff nrm = ff_sqrt(transform_row<DT, ff>(row, sd, rope, a, tok, v));
    if (lane == 0) *reinterpret_cast<uint16_t *>(block) = ff_half(nrm);
    // y >= b after its rounding to float32 where v >= b' sqrt(128) nrm, b' half way to b's lower neighbour;
    // lane j has boundary j
    const float b = sd.b[lane < 15 ? lane : 14];
    const uint32_t w = __float_as_uint(b);
    const float under = b == 0.f ? 0.f : __uint_as_float(b > 0.f ? w - 1 : w + 1);
    const ff k = ff_mul(nrm, ff_of(11.313708498984761f, (float)(11.313708498984761 - (double)11.313708498984761f)));
    const ff mine = ff_mul(k, ff_of(b, b == 0.f ? 0.f : 0.5f * (under - b)));
    ff x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = v[4 * lane + i];
    uint32_t code = 0;
#pragma unroll 1
    for (int j = 0; j < (1 << sd.bits) - 1; ++j) {
        const float eh = __shfl_sync(0xffffffffu, mine.h, j), el = __shfl_sync(0xffffffffu, mine.l, j);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            // (of two renormalised values the larger high part, then the larger low part)
            code += x[i].h > eh || (x[i].h == eh && x[i].l >= el) ? 1u << (8 * i) : 0u;
    }
    write_codes(block, sd.bits, code, lane);
}

// The few coordinates of a row that float32 does not decide, in double-float:
// coordinate j is a sum over the row's pairs, so it costs one reduction and no
// transform.
// near: bits i of the lane's elements 4 lane + i to decide, cell[i] the number
// of boundaries below their cells.  Returns the lane's codes; the norm is
// rounded again as well.
__device__ __noinline__ uint32_t decide_few(float x0, float x1, float x2, float x3, uint32_t near, uint32_t cell,
                                            uint32_t code, uint64_t angle0, uint64_t angle1, int partner, uint32_t flip,
                                            int pairs, const Side &sd, uint8_t *block) {
    const int lane = threadIdx.x & 31;
    // two pairs (A, B) of the row, of elements ia and ia + apart: adjacent ones, or of the halves (the lane of the
    // upper half has the second two of the four pairs that both hold elements of)
    const bool half = partner >= 0 && sd.style != kRopeAdjacent, upper = half && partner < lane;
    const int from = half ? partner : lane;
    const float o0 = __shfl_sync(0xffffffffu, upper ? x0 : x2, from);
    const float o1 = __shfl_sync(0xffffffffu, upper ? x1 : x3, from);
    const uint32_t other = __shfl_sync(0xffffffffu, flip, from);
    const float A[2] = {!half ? x0 : upper ? o0 : x0, !half ? x2 : upper ? o1 : x1};
    const float B[2] = {!half ? x1 : upper ? x2 : o0, !half ? x3 : upper ? x3 : o1};
    const uint32_t fa = !half ? (flip & 1u) | (flip >> 1 & 2u) : upper ? other >> 2 : flip;   // (bit z)
    const uint32_t fb = !half ? (flip >> 1 & 1u) | (flip >> 2 & 2u) : upper ? flip >> 2 : other;
    const int ia = upper ? 4 * from + 2 : 4 * lane, next = half ? 1 : 2, apart = half ? pairs : 1;
    ff s[2], c[2];
#pragma unroll 1
    for (int z = 0; z < 2; ++z) {
        ff sz = {0.f, 0.f}, cz = {1.f, 0.f};
        if (partner >= 0) rope_sincos_ff(z ? angle1 : angle0, sz, cz);
        if (z) s[1] = sz, c[1] = cz;
        else s[0] = sz, c[0] = cz;
    }
    ff squares = ff_add(ff_add(ff_square(x0), ff_square(x1)), ff_add(ff_square(x2), ff_square(x3)));
    uint32_t who = __ballot_sync(0xffffffffu, near != 0);
    bool first = true;
    do {
        const int src = who ? __ffs(who) - 1 : 0;
        const uint32_t bits = __shfl_sync(0xffffffffu, near, src);
        const int e = bits ? __ffs(bits) - 1 : 0, j = 4 * src + e;
        ff v = ff_of(0.f), ss = squares;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            // +-(A c - B s) +- (B c + A s) = c (+-A +- B) + s (+-A -+ B)
            const int at = ia + z * next;
            const bool na = (__popc(at & j) ^ (fa >> z)) & 1, nb = (__popc((at + apart) & j) ^ (fb >> z)) & 1;
            const ff p = ff_sum(na ? -A[z] : A[z], nb ? -B[z] : B[z]), q = ff_sum(nb ? -A[z] : A[z], na ? B[z] : -B[z]);
            v = ff_add(v, ff_add(ff_mul(c[z], p), ff_mul(s[z], q)));
        }
#pragma unroll 1
        for (int m = 1; m < 32; m <<= 1) {
            v = ff_add(v, shfl_(v, m));
            ss = ff_add(ss, shfl_(ss, m));
        }
        const ff nrm = ff_sqrt(ss);
        if (first && lane == 0) *reinterpret_cast<uint16_t *>(block) = ff_half(nrm);
        first = false;
        if (lane == src && near) {   // y >= b as in near_row
            const int below = (int)((cell >> (8 * e)) & 0xFFu);
            const float b = sd.b[below];
            const uint32_t w = __float_as_uint(b);
            const float under = b == 0.f ? 0.f : __uint_as_float(b > 0.f ? w - 1 : w + 1);
            const ff k = ff_mul(nrm, ff_of(11.313708498984761f, (float)(11.313708498984761 - (double)11.313708498984761f)));
            const ff edge = ff_mul(k, ff_of(b, b == 0.f ? 0.f : 0.5f * (under - b)));
            const uint32_t c = (uint32_t)below + (v.h > edge.h || (v.h == edge.h && v.l >= edge.l) ? 1u : 0u);
            code = (code & ~(0xFFu << (8 * e))) | c << (8 * e);
            near &= near - 1;
        }
        who = __ballot_sync(0xffffffffu, near != 0);
    } while (who);
    return code;
}

// What a lane needs of the rope and the signs: the turns of two pairs (adjacent
// elements, or halves, where the lane of the upper half, its partner's elements
// + rot_dim / 2, takes the second two of the four that both need).
struct FewLane {
    uint64_t turn[2];
    int axis[2];
    int partner;
    bool turned, upper, adj;
    uint32_t flip;
};

__device__ __forceinline__ FewLane few_lane(const Side &sd, const tq_rope &rope, const InsertArgs &a) {
    const int lane = threadIdx.x & 31;
    const int span = sd.style == kRopeNone ? 0 : rope.rot_dim / 8;   // lanes of half the rotated elements
    FewLane w;
    w.turned = lane < 2 * span;
    w.upper = lane >= span;
    w.adj = sd.style == kRopeAdjacent;
    w.partner = !w.turned || w.adj ? lane : w.upper ? lane - span : lane + span;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        const int p = (w.adj ? 2 * lane : w.upper ? 4 * (lane - span) + 2 : 4 * lane) + z;
        w.turn[z] = w.turned ? rope.turn[p] : 0;
        w.axis[z] = w.turned ? rope.axis[p] : 0;
    }
    w.flip = a.signs[lane >> 3] >> (4 * (lane & 7));
    return w;
}

// A lane's elements of a row and the row's positions, as loaded.
struct FewIn {
    uint4 raw;
    int64_t pos[3];
};

template <int DT>
__device__ __forceinline__ FewIn few_load(const uint8_t *row, int64_t tok, const Side &sd, const tq_rope &rope,
                                          const InsertArgs &a) {
    const int lane = threadIdx.x & 31;
    FewIn n;
    n.raw = make_uint4(0, 0, 0, 0);
    if constexpr (DT == TQ_F32) {
        n.raw = __ldcs(reinterpret_cast<const uint4 *>(row) + lane);
    } else {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(row) + lane);
        n.raw.x = v.x;
        n.raw.y = v.y;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
        n.pos[i] = sd.style == kRopeNone ? 0 : a.pos[(i < rope.axes ? i : 0) * a.pos_axis + tok];
    return n;
}

// One row by a warp into its block.  cells: the quantiser's, entry c at (128 c)
// >> shift; again: space for 128 values in double.
template <int DT>
__device__ __forceinline__ void few_row(const FewIn &n, const FewLane &w, const uint8_t *cells, int shift,
                                        const uint8_t *row, uint8_t *block, const Side &sd, const tq_rope &rope,
                                        const InsertArgs &a, int64_t tok, void *again) {
    const int lane = threadIdx.x & 31, bits = sd.bits;
    const uint4 raw = n.raw;
    const int64_t (&pos)[3] = n.pos;
    // a row of zeros (sign bits aside: of both elements of a word of 16-bit types)
    if (!__any_sync(0xffffffffu, (raw.x | raw.y | raw.z | raw.w) & (DT == TQ_F32 ? 0x7FFFFFFFu : 0x7FFF7FFFu))) {
        if (lane == 0) *reinterpret_cast<uint16_t *>(block) = 0;
        const uint2 e = *reinterpret_cast<const uint2 *>(cells + ((64 * 128) >> shift));   // the cell of 0
        write_codes(block, bits, 0x01010101u * (e.y - (__uint_as_float(e.x) > 0.f)), lane);
        return;
    }
    float x[4];
    if constexpr (DT == TQ_F32) {
        x[0] = __uint_as_float(raw.x);
        x[1] = __uint_as_float(raw.y);
        x[2] = __uint_as_float(raw.z);
        x[3] = __uint_as_float(raw.w);
    } else if constexpr (DT == TQ_BF16) {
        x[0] = bf16_bits_lo(raw.x);
        x[1] = bf16_bits_hi(raw.x);
        x[2] = bf16_bits_lo(raw.y);
        x[3] = bf16_bits_hi(raw.y);
    } else {
        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&raw.x));
        const float2 q = __half22float2(*reinterpret_cast<const __half2 *>(&raw.y));
        x[0] = p.x;
        x[1] = p.y;
        x[2] = q.x;
        x[3] = q.y;
    }
    const float4 in = make_float4(x[0], x[1], x[2], x[3]);
    float ss = fmaf(x[0], x[0], x[1] * x[1]) + fmaf(x[2], x[2], x[3] * x[3]);   // (rope keeps the norm)
    uint64_t angle[2] = {0, 0};
    if (sd.style != kRopeNone) {
        float s[2], c[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            angle[z] = rope_turns(w.turn[z], w.axis[z] == 0 ? pos[0] : w.axis[z] == 1 ? pos[1] : pos[2]);
            rope_sincos(angle[z], s[z], c[z]);
        }
        if (w.adj) {
            if (w.turned)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const float xa = x[2 * z], xb = x[2 * z + 1];
                    x[2 * z] = fmaf(xa, c[z], -(xb * s[z]));
                    x[2 * z + 1] = fmaf(xb, c[z], xa * s[z]);
                }
        } else {
            float so[2], co[2], o[4];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                so[z] = __shfl_sync(0xffffffffu, s[z], w.partner);
                co[z] = __shfl_sync(0xffffffffu, c[z], w.partner);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = __shfl_sync(0xffffffffu, x[i], w.partner);
            if (w.turned)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool mine = (i >= 2) == w.upper;
                    const float si = mine ? s[i & 1] : so[i & 1], ci = mine ? c[i & 1] : co[i & 1];
                    x[i] = fmaf(x[i], ci, o[i] * (w.upper ? si : -si));
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(__float_as_uint(x[i]) ^ ((w.flip >> i) << 31));
    {
        const float p = x[0] + x[1], q = x[0] - x[1], r = x[2] + x[3], d = x[2] - x[3];
        x[0] = p + r;
        x[1] = q + d;
        x[2] = p - r;
        x[3] = q - d;
    }
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, m);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float o = __shfl_xor_sync(0xffffffffu, x[i], m);
            x[i] = o + (lane & m ? -x[i] : x[i]);
        }
    }
    // norm, ranges and codes as in insert_kernel
    float inv;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(ss));
    inv = fmaf(inv * fmaf(-ss * inv, inv, 1.f), 0.5f, inv);
    const float nrm = ss * inv, scale = kUnit * inv;
    const bool wild = !(ss >= 7.888609052210118e-31f && ss <= 1.2676506002282294e30f);
    const bool tie = ((__float_as_uint(nrm) & 0x1FFFu) - (0x1000u - kTieUlps)) <= 2 * kTieUlps ||
                     !(nrm >= 6.103515625e-05f && nrm < 65504.f);
    uint32_t near = 0, code = 0, cell = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float v = fmaf(x[i], scale, 98304.f + 64.5f);
        const uint2 e = *reinterpret_cast<const uint2 *>(cells + ((__float_as_uint(v) & 0x3F80u) >> shift));
        const float d = fmaf(x[i], scale, -__uint_as_float(e.x));
        near |= fabsf(d) < sd.eps_few ? 1u << i : 0u;
        cell |= (e.y - 1) << (8 * i);
        code |= ((e.y + (uint32_t)(__float_as_int(d) >> 31)) & 15u) << (8 * i);
    }
    if (wild) {
        range_row<DT>(row, block, sd, rope, a, tok, static_cast<double *>(again));
    } else {
        const uint32_t who = __ballot_sync(0xffffffffu, near != 0);
        if (who == 0 && !tie) {
            if (lane == 0) *reinterpret_cast<__half *>(block) = __float2half_rn(nrm);
        } else if (__popc(who) <= 4) {
            code = decide_few(in.x, in.y, in.z, in.w, near, cell, code, angle[0], angle[1], w.turned ? w.partner : -1,
                              w.flip, rope.rot_dim / 2, sd, block);
        }
        if (__popc(who) <= 4) write_codes(block, bits, code, lane);
        else near_row<DT>(row, block, sd, rope, a, tok, static_cast<ff *>(again));
    }
}

// Norms of four rows (rope keeps them), one per eight lanes.
template <int DT>
__device__ __noinline__ void norm_rows(const uint8_t *row, uint8_t *block, bool write) {
    const int l = threadIdx.x & 7;
    ff ss = ff_of(0.f);
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
        const ff x = ff_of(elem<DT>(row, 16 * l + i));
        ss = ff_add(ss, ff_mul(x, x));
    }
#pragma unroll 1
    for (int m = 1; m < 8; m <<= 1) ss = ff_add(ss, shfl_(ss, m));
    if (write && l == 0) *reinterpret_cast<uint16_t *>(block) = ff_half(ff_sqrt(ss));
}

// The listed rows of the CTA, a warp each (four for their norms alone).  If the
// list overflowed (inputs of many zeros, say), all its rows.
template <int DT>
__device__ __noinline__ void finish(int which, const tq_rope &rope, const InsertArgs &a) {
    extern __shared__ __align__(16) uint8_t dsmem[];
    Shared &sm = *reinterpret_cast<Shared *>(dsmem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Side &sd = a.side[which];
    const uint8_t *cells = reinterpret_cast<const uint8_t *>(sm.cells);
    uint16_t *stage = sm.stage[warp];
    const int ties = sm.listed[0], whole = sm.listed[1];
    const int64_t bytes = 2 + 16 * sd.bits;
    const int cta = blockIdx.x - (which ? a.ctas[0] : 0), step = a.ctas[which], span = kTok * a.tiles;
    auto block_of = [&](int64_t tok, int head) { return sd.blocks + (a.dst[tok] + head * a.dst_head) * bytes; };
    auto row_of = [&](int64_t tok, int head) { return sd.x + tok * sd.tok + head * sd.head; };
    auto token_of = [&](int unit, int t) { return (int64_t)(unit / a.groups) * span + t; };
    const Listed *list = list_of(sm, a.tiles);
    auto find = [&](const Listed &e, int64_t &tok, int &head) {
        tok = token_of(e.unit, (int)(e.row & 63u));
        head = (int)(e.row >> 6);
    };
    // this warp's next row: of the list, or of all the CTA's
    const bool all = max(ties, whole) > a.list;
    int unit = cta, in_unit = warp, in_group = 0;
    int at = warp;
    auto next = [&](int64_t &tok, int &head) {
        if (!all) {
            if (at >= whole) return false;
            find(list[a.list + at], tok, head);
            at += kWarps;
            return true;
        }
        while (unit < a.units) {
            const int head0 = unit % a.groups * a.heads_per_cta, heads = min(a.heads_per_cta, a.heads - head0);
            tok = token_of(unit, in_unit);
            if (in_unit >= span || tok >= a.n_tok) {
                unit += step;
                in_unit = warp;
                in_group = 0;
            } else if (in_group == heads) {
                in_unit += kWarps;
                in_group = 0;
            } else {
                head = head0 + in_group++;
                const int64_t dst = a.dst[tok], slot = dst < 0 ? -1 : dst + head * a.dst_head;
                if (slot >= 0 && slot < sd.n_blocks) return true;
            }
        }
        return false;
    };
    const FewLane lane_part = few_lane(sd, rope, a);
    int64_t tok = 0;
    int head = 0;
    FewIn in;
    bool more = next(tok, head);
    if (more) in = few_load<DT>(row_of(tok, head), tok, sd, rope, a);
    while (more) {   // (the next row on its way while this one is taken)
        const FewIn now = in;
        const int64_t t = tok;
        const int h = head;
        more = next(tok, head);
        if (more) in = few_load<DT>(row_of(tok, head), tok, sd, rope, a);
        few_row<DT>(now, lane_part, cells, 0, row_of(t, h), block_of(t, h), sd, rope, a, t, stage);
        __syncwarp();
    }
    if (all) return;
    for (int i = 4 * warp; i < ties; i += 4 * kWarps) {
        const int q = i + (lane >> 3);
        find(list[q < ties ? q : i], tok, head);
        norm_rows<DT>(row_of(tok, head), block_of(tok, head), q < ties);
    }
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// (a, b) <- (a cos - b sin, b cos + a sin) for two pairs at once.
__device__ __forceinline__ void turn2(float2 &a, float2 &b, const float4 &t) {
    const float2 c = make_float2(t.x, t.y), s = make_float2(t.z, t.w), n = make_float2(-t.z, -t.w);
    const float2 va = a, vb = b;
    a = fma2(va, c, mul2(vb, n));
    b = fma2(vb, c, mul2(va, s));
}

// A row's elements in a thread: x[c][k] holds elements 32 c + 8 t + 2 k, + 1.
typedef float2 RowPart[4][4];

// Rotary positions on a thread's part of a row; cs: the row's token in the
// table of sines, [unit * 64].
__device__ __forceinline__ void rope_row(RowPart &x, int style, const float4 *cs, int t) {
    if (style == kRopeHalf4) {          // pairs (e, e + 64)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k) turn2(x[c][k], x[c + 2][k], cs[(4 * c + k) * 64]);
    } else if (style == kRopeAdjacent) {   // pairs (e, e + 1): e even
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                const float4 w = cs[(2 * c + k / 2) * 64];
                const float2 a = x[c][k], b = x[c][k + 1];
                x[c][k] = make_float2(fmaf(a.x, w.x, -(a.y * w.z)), fmaf(a.y, w.x, a.x * w.z));
                x[c][k + 1] = make_float2(fmaf(b.x, w.y, -(b.y * w.w)), fmaf(b.y, w.y, b.x * w.w));
            }
    } else if (style == kRopeHalf2) {   // pairs (e, e + 32)
#pragma unroll
        for (int k = 0; k < 4; ++k) turn2(x[0][k], x[1][k], cs[k * 64]);
    } else if (style == kRopeHalf1) {   // pairs (e, e + 16): thread t with t ^ 2
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 w = cs[k * 64 - (t & 2)];   // pair index modulo 16: thread t & 1
            float2 o;
            o.x = __shfl_xor_sync(0xffffffffu, x[0][k].x, 2);
            o.y = __shfl_xor_sync(0xffffffffu, x[0][k].y, 2);
            const float2 s = (t & 2) ? make_float2(w.z, w.w) : make_float2(-w.z, -w.w);
            x[0][k] = fma2(x[0][k], make_float2(w.x, w.y), mul2(o, s));
        }
    } else if (style == kRopeHalf3) {
        // pairs (e, e + 48): the partner of chunk c's element lies in thread t ^ 2, chunk (c + 1) % 3 for
        // t < 2, (c + 2) % 3 for the others; pair index e or e - 48
        const bool hi = (t & 2) != 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float2 o[3];
#pragma unroll
            for (int c = 0; c < 3; ++c) {
                const float2 send = hi ? x[(c + 1) % 3][k] : x[(c + 2) % 3][k];
                o[c].x = __shfl_xor_sync(0xffffffffu, send.x, 2);
                o[c].y = __shfl_xor_sync(0xffffffffu, send.y, 2);
            }
#pragma unroll
            for (int c = 0; c < 3; ++c) {
                // first of its pair: chunk 0, and chunk 1 for t < 2
                const bool second = c == 2 || (c == 1 && hi);
                // pair 32 c' + 8 t' + 2 k: chunk 0 as it is; chunk 1: t < 2 as it is, else pair 8 (t - 2);
                // chunk 2: t < 2 pair 8 (t + 2), else 32 + 8 (t - 2)
                const int unit = c == 0 ? 0 : (c == 1 ? (hi ? 0 : 1) : (hi ? 1 : 0));
                const int shift = c == 0 ? 0 : (c == 1 ? (hi ? -2 : 0) : (hi ? -2 : 2));
                const float4 w = cs[(4 * unit + k) * 64 + shift];
                const float2 s = second ? make_float2(w.z, w.w) : make_float2(-w.z, -w.w);
                x[c][k] = fma2(x[c][k], make_float2(w.x, w.y), mul2(o[c], s));
            }
        }
    }
}

template <bool BF16>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with the accumulator starting at zero.
template <bool BF16>
__device__ __forceinline__ void mma16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Accumulators: [c][s][n-tile][4]; entries 0, 1 (row g) and 2, 3 (row g + 8)
// are elements 32 c + 8 t + 4 s + 2 nt, + 1.
typedef float Acc[4][2][2][4];

// The butterflies over element bits 2 (s), 5 and 6 (c).
__device__ __forceinline__ void butterflies(Acc &u) {
    auto step = [](float (&a)[4], float (&b)[4]) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const float2 x = make_float2(a[i], a[i + 1]), y = make_float2(b[i], b[i + 1]);
            const float2 p = add2(x, y), m = sub2(x, y);
            a[i] = p.x;
            a[i + 1] = p.y;
            b[i] = m.x;
            b[i + 1] = m.y;
        }
    };
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
        for (int c = 0; c < 4; ++c) step(u[c][0][nt], u[c][1][nt]);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            step(u[0][s][nt], u[1][s][nt]);
            step(u[2][s][nt], u[3][s][nt]);
            step(u[0][s][nt], u[2][s][nt]);
            step(u[1][s][nt], u[3][s][nt]);
        }
    }
}

// Codes of a thread's 32 elements of row R (0: g, 1: g + 8), the BITS-wide
// field k of w[c] element 32 c + 8 t + k.  Returns the smallest |v - b| met.
template <int BITS, int R>
__device__ __forceinline__ float quantise(const Acc &u, float scale, const uint8_t *cells, uint32_t lane8,
                                          uint32_t (&w)[4]) {
    float near = 1.f;
    const float2 s2 = make_float2(scale, scale), m2 = make_float2(98304.f + 64.5f, 98304.f + 64.5f);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t acc = 0;
#pragma unroll
        for (int q = 3; q >= 0; --q) {
            const float2 x = make_float2(u[c][q >> 1][q & 1][2 * R], u[c][q >> 1][q & 1][2 * R + 1]);
            const float2 v = fma2(x, s2, m2);
            const uint2 e1 = *reinterpret_cast<const uint2 *>(cells + ((__float_as_uint(v.y) & 0x3F80u) | lane8));
            const uint2 e0 = *reinterpret_cast<const uint2 *>(cells + ((__float_as_uint(v.x) & 0x3F80u) | lane8));
            const float t1 = fmaf(x.y, scale, -__uint_as_float(e1.x)), t0 = fmaf(x.x, scale, -__uint_as_float(e0.x));
            near = fminf(fminf(near, fabsf(t1)), fabsf(t0));
            acc = (acc << BITS) + e1.y + (uint32_t)(__float_as_int(t1) >> 31);
            acc = (acc << BITS) + e0.y + (uint32_t)(__float_as_int(t0) >> 31);
        }
        w[c] = acc;
    }
    return near;
}

// Quantise and stage one row: half word 0 of its block the norm, then the codes.
template <int BITS, int R>
__device__ __forceinline__ float pack_row(const Acc &u, float scale, const uint8_t *cells, uint32_t lane8,
                                          uint16_t *blk, int t) {
    uint32_t w[4];
    const float near = quantise<BITS, R>(u, scale, cells, lane8, w);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if constexpr (BITS == 4) {
            blk[1 + 8 * c + 2 * t] = (uint16_t)w[c];
            blk[2 + 8 * c + 2 * t] = (uint16_t)(w[c] >> 16);
        } else if constexpr (BITS == 2) {
            blk[1 + 4 * c + t] = (uint16_t)w[c];
        } else {
            uint32_t lo = 0, hi = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                lo |= ((w[c] >> (3 * k)) & 3u) << (2 * k);
                hi |= ((w[c] >> (3 * k + 2)) & 1u) << k;
            }
            blk[1 + 4 * c + t] = (uint16_t)lo;
            reinterpret_cast<uint8_t *>(blk)[34 + 4 * c + t] = (uint8_t)hi;
        }
    }
    return near;
}

// One float2 as two fp16 parts, hi + lo.
__device__ __forceinline__ void split2(float2 x, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x.x, x.y);
    const float2 r = sub2(x, __half22float2(h));
    const __half2 l = __floats2half2_rn(r.x, r.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 4) insert_kernel(const __grid_constant__ tq_rope rope,
                                                             const __grid_constant__ InsertArgs a) {
    constexpr int NV = Row<DT>::kVecs, ES = Row<DT>::kBytes;
    extern __shared__ __align__(16) uint8_t dsmem[];
    Shared &sm = *reinterpret_cast<Shared *>(dsmem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int which = (int)blockIdx.x < a.ctas[0] ? 0 : 1;
    const Side &sd = a.side[which];
    const int cta = blockIdx.x - (which ? a.ctas[0] : 0), step = a.ctas[which];
    const int bits = sd.bits, levels = 1 << bits, bytes = 2 + 16 * bits, style = sd.style;
    // the warps of a tile take its heads in turn
    const int hw = kWarps / a.tiles, tile = warp / hw;

    // rows of a unit: a tile of 16 tokens, and the heads of a group in this warp's turn
    const bool one_group = a.groups == 1;
    auto group_of = [&](int unit) { return one_group ? 0 : unit % a.groups; };
    auto tile_of = [&](int unit) { return ((int64_t)(one_group ? unit : unit / a.groups) * a.tiles + tile) * kTok; };
    auto head_of = [&](int unit) { return group_of(unit) * a.heads_per_cta + warp % hw; };
    auto head_end = [&](int unit) { return min((group_of(unit) + 1) * a.heads_per_cta, a.heads); };
    // the two rows of this thread: its 8 elements of chunk c at + 32 c
    auto rows_of = [&](int64_t tok0, const uint8_t *(&p)[2]) {
#pragma unroll
        for (int r = 0; r < 2; ++r) p[r] = sd.x + min64(tok0 + g + 8 * r, a.n_tok - 1) * sd.tok + 8 * t * ES;
    };
    // copies of the rows of (rows, head) to this thread's places
    auto fetch = [&](const uint8_t *const (&rows)[2], int head) {
        if constexpr (DT != TQ_F32) {
            const int64_t at = head * sd.head;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint8_t *p = rows[r] + at;
#pragma unroll
                for (int c = 0; c < 4; ++c) cp_async16(&sm.in[warp][4 * r + c][lane], p + 32 * c * ES);
            }
            cp_async_commit();
        }
    };
    int unit = cta;
    int head = 0;
    // the next (unit, head) of this warp from (u, h) on that has rows; u past the end if none
    auto settle = [&](int &u, int &h) {
        while (u < a.units && (h >= head_end(u) || tile_of(u) >= a.n_tok)) {
            u += step;
            if (u < a.units) h = head_of(u);
        }
    };
    if (unit < a.units) {
        head = head_of(unit);
        int u = unit;
        int h = head;
        settle(u, h);
        if (u < a.units) {
            const uint8_t *rows[2];
            rows_of(tile_of(u), rows);
            fetch(rows, h);
        }
    }

    // the 16 x 16 Hadamard matrix as B fragments: k = (thread t, j) in, n = (thread g / 2, j = 2 nt + g % 2)
    // out; j = 0, 1 in b[nt][0], 2, 3 in b[nt][1]; 1.0 of the products' type
    constexpr bool kBf = DT == TQ_BF16;
    const bool direct = DT != TQ_F32 && style == kRopeNone;
    uint32_t bf[2][2];
    {
        const uint32_t one = direct && kBf ? 0x3F80u : 0x3C00u;
        const int tt = __popc(t & (g >> 1));
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int jo = 2 * nt + (g & 1);
                const uint32_t n0 = (tt + __popc((2 * q) & jo)) & 1, n1 = (tt + __popc((2 * q + 1) & jo)) & 1;
                bf[nt][q] = (one | n0 << 15) | (one | n1 << 15) << 16;
            }
    }
    uint16_t *stage = sm.stage[warp];
    const uint8_t *cells = reinterpret_cast<const uint8_t *>(sm.cells);
    const uint32_t lane8 = (lane & 15) * 8;

    for (; unit < a.units; unit += step) {
        const int64_t tok0 = tile_of(unit);
        const int64_t my = tok0 + (lane & 15);
        const int64_t dst = my < a.n_tok ? a.dst[my] : -1;   // of token lane % 16
        // positions of this thread's token (tid / 4 % 16) of tile v of the unit, on their way while the tables are
        // built and the other warps finish
        const int64_t first = tile_of(unit) - tile * kTok;
        int64_t pos[3] = {0, 0, 0};
        auto positions = [&](int v) {
            const int64_t at = min64(first + v * kTok + ((tid >> 2) & 15), a.n_tok - 1);
#pragma unroll
            for (int i = 0; i < 3; ++i) pos[i] = a.pos[(i < rope.axes ? i : 0) * a.pos_axis + at];
        };
        if (style != kRopeNone) positions(0);
        if (unit == cta) {
            static_assert(kThreads == 128, "a thread per cell");
            {
                uint32_t below = 0;
                float edge = 3.0e38f;   // a cell without a boundary: v - edge < 0 for every v
                for (int j = 0; j < levels - 1; ++j) {
                    const float v = sd.b[j] * kGrid;
                    const int at = (int)floorf(v + 64.5f);
                    if (at < tid) ++below;
                    if (at == tid) edge = v;
                }
                const uint2 e = make_uint2(__float_as_uint(edge), below + 1);
#pragma unroll
                for (int i = 0; i < 16; ++i) sm.cells[tid * 16 + ((i + tid) & 15)] = e;
            }
            if (tid < 64) {   // word k of chunk c, thread t: elements 32 c + 8 t + 2 k, + 1
                const int e = 2 * tid, c = e >> 5, th = (e >> 3) & 3, k = (e >> 1) & 3;
                const uint32_t s2 = a.signs[e >> 5] >> (e & 31);
                reinterpret_cast<uint32_t *>(&sm.flip[c][th])[k] = (s2 & 1u) << 15 | (s2 & 2u) << 30;
            }
            if (tid < 2) sm.listed[tid] = 0;
            if (tid < kRopePairs && style != kRopeNone) {
                const int pairs = rope.rot_dim / 2;
                const int ea = style == kRopeAdjacent ? 2 * tid : tid, eb = style == kRopeAdjacent ? ea + 1 : tid + pairs;
                const uint32_t differ = tid < pairs ? ((a.signs[ea >> 5] >> (ea & 31)) ^ (a.signs[eb >> 5] >> (eb & 31))) & 1u : 0u;
                // (past the rotated elements: no angle)
                sm.turn[tid] = tid < pairs ? rope.turn[tid] : 0;
                sm.axis[tid] = (uint8_t)((tid < pairs ? rope.axis[tid] : 0) | differ << 2);
            }
        }
        if (style != kRopeNone) {
            const bool adj = style == kRopeAdjacent;
            const int th = tid & 3;
            __syncthreads();   // the rope's copy is there, and the last unit's table no longer read
            for (int v = 0; v < a.tiles; ++v) {
                if (v > 0) positions(v);
#pragma unroll
                for (int u = 0; u < 4; ++u) {   // its units tid / 64, + 2, ...
                    const int unit8 = 2 * u + (tid >> 6);
                    const int p0 = adj ? 16 * (unit8 >> 1) + 4 * th + 2 * (unit8 & 1) : 32 * (unit8 >> 2) + 8 * th + 2 * (unit8 & 3);
                    float s[2], c[2];
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const uint32_t ax = sm.axis[p0 + z];
                        const int64_t p = (ax & 3u) == 0 ? pos[0] : (ax & 3u) == 1 ? pos[1] : pos[2];
                        rope_sincos(rope_turns(sm.turn[p0 + z], p), s[z], c[z]);
                        if (ax & 4u) s[z] = -s[z];
                    }
                    sm.cs[v][u * 128 + tid] = make_float4(c[0], c[1], s[0], s[1]);
                }
            }
        }
        if (style != kRopeNone || unit == cta) __syncthreads();
        const int hend = tok0 < a.n_tok ? head_end(unit) : 0;
        const uint8_t *rows[2];
        rows_of(tok0, rows);
        for (head = head_of(unit); head < hend; head += hw) {
            uint4 raw[2][4][NV];
            if constexpr (DT == TQ_F32) {
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < NV; ++i)
                            raw[r][c][i] =
                                __ldcs(reinterpret_cast<const uint4 *>(rows[r] + head * sd.head + 32 * c * ES) + i);
            } else {
                cp_async_wait<0>();
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int c = 0; c < 4; ++c) raw[r][c][0] = sm.in[warp][4 * r + c][lane];
                if (head + hw < hend) {
                    fetch(rows, head + hw);
                } else {
                    int u = unit;
                    int h = head + hw;
                    settle(u, h);
                    if (u < a.units) {
                        const uint8_t *next[2];
                        rows_of(tile_of(u), next);
                        fetch(next, h);
                    }
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint4 f = sm.flip[c][t];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        raw[r][c][0].x ^= f.x;
                        raw[r][c][0].y ^= f.y;
                        raw[r][c][0].z ^= f.z;
                        raw[r][c][0].w ^= f.w;
                    }
                }
            }
            Acc u;
            // sums of squares of rows g and g + 8 (of the whole row after the quad's shuffles)
            float ss[2], post[2] = {1.f, 1.f};   // (post: the inverse of a row's factor)
            if (direct) {
                if constexpr (DT != TQ_F32) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            const uint4 x = raw[0][c][0], y = raw[1][c][0];
                            mma16_first<kBf>(u[c][0][nt], x.x, y.x, x.y, y.y, bf[nt][0], bf[nt][1]);
                            mma16_first<kBf>(u[c][1][nt], x.z, y.z, x.w, y.w, bf[nt][0], bf[nt][1]);
                        }
                }
                // a product with the 16 x 16 matrix has 16 times the row's sum of squares
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float2 q[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 x = make_float2(u[c][i >> 1][i & 1][2 * r], u[c][i >> 1][i & 1][2 * r + 1]);
                            q[c] = i ? fma2(x, x, q[c]) : mul2(x, x);
                        }
                    q[0] = add2(add2(q[0], q[1]), add2(q[2], q[3]));
                    ss[r] = q[0].x + q[0].y;
                    ss[r] += __shfl_xor_sync(0xffffffffu, ss[r], 1);
                    ss[r] += __shfl_xor_sync(0xffffffffu, ss[r], 2);
                    ss[r] *= 0.0625f;
                }
            } else {
                RowPart x[2];
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint4 v0 = raw[r][c][0], v1 = raw[r][c][NV - 1];
                        if constexpr (DT == TQ_F32) {
                            const uint4 f = sm.flip[c][t];
                            const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
                            const uint32_t m[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                x[r][c][k] = make_float2(__uint_as_float(w[2 * k] ^ (m[k] << 16)),
                                                         __uint_as_float(w[2 * k + 1] ^ (m[k] & 0x80000000u)));
                        } else {
                            const uint32_t w[4] = {v0.x, v0.y, v0.z, v0.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if constexpr (kBf) x[r][c][k] = make_float2(bf16_bits_lo(w[k]), bf16_bits_hi(w[k]));
                                else x[r][c][k] = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
                            }
                        }
                    }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float2 q[4];   // (the norm is that of the row before its rotation)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k) q[c] = k ? fma2(x[r][c][k], x[r][c][k], q[c]) : mul2(x[r][c][k], x[r][c][k]);
                    q[0] = add2(add2(q[0], q[1]), add2(q[2], q[3]));
                    ss[r] = q[0].x + q[0].y;
                    ss[r] += __shfl_xor_sync(0xffffffffu, ss[r], 1);
                    ss[r] += __shfl_xor_sync(0xffffffffu, ss[r], 2);
                    // power of two that brings the norm to [2^9, 2^10.5): half the exponent of the sum of
                    // squares (rows outside the safe range are redone, whatever comes of it here)
                    const int e = (int)(__float_as_uint(ss[r]) >> 23) - 127;
                    const float pre = __uint_as_float((uint32_t)(127 + 9 - (e >> 1)) << 23);
                    post[r] = __uint_as_float((uint32_t)(127 - 9 + (e >> 1)) << 23);
                    rope_row(x[r], style, sm.cs[tile] + (g + 8 * r) * 4 + t, t);
                    const float2 p2 = make_float2(pre, pre);
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[r][i >> 2][i & 3] = mul2(x[r][i >> 2][i & 3], p2);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        uint32_t hi[2][2], lo[2][2];
#pragma unroll
                        for (int r = 0; r < 2; ++r)
#pragma unroll
                            for (int q = 0; q < 2; ++q) split2(x[r][c][2 * s + q], hi[r][q], lo[r][q]);
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            // (the lower parts first: a sum loses places of its largest term's size)
                            mma16_first<false>(u[c][s][nt], lo[0][0], lo[1][0], lo[0][1], lo[1][1], bf[nt][0], bf[nt][1]);
                            mma16<false>(u[c][s][nt], hi[0][0], hi[1][0], hi[0][1], hi[1][1], bf[nt][0], bf[nt][1]);
                        }
                    }
            }
            butterflies(u);
            bool redo[2], tie[2];
            float nrm[2], near[2], sc[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                // 1 / norm: the hardware's estimate and one Newton step (2^-23)
                float inv;
                asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(ss[r]));
                inv = fmaf(inv * fmaf(-ss[r] * inv, inv, 1.f), 0.5f, inv);
                nrm[r] = ss[r] * inv;
                sc[r] = kUnit * inv * post[r];
                // 2^-100 .. 2^100: squares neither underflow nor overflow (false for a NaN as well)
                redo[r] = !(ss[r] >= 7.888609052210118e-31f && ss[r] <= 1.2676506002282294e30f);
                tie[r] = ((__float_as_uint(nrm[r]) & 0x1FFFu) - (0x1000u - sd.ulps)) <= 2 * sd.ulps ||
                         !(nrm[r] >= 6.103515625e-05f && nrm[r] < 65504.f);   // (or outside fp16's normal range)
            }
            uint16_t *blkA = stage + g * (bytes / 2), *blkB = stage + (g + 8) * (bytes / 2);
            if (t == 0) {
                blkA[0] = __half_as_ushort(__float2half_rn(nrm[0]));
                blkB[0] = __half_as_ushort(__float2half_rn(nrm[1]));
            }
            if (bits == 4) {
                near[0] = pack_row<4, 0>(u, sc[0], cells, lane8, blkA, t);
                near[1] = pack_row<4, 1>(u, sc[1], cells, lane8, blkB, t);
            } else if (bits == 3) {
                near[0] = pack_row<3, 0>(u, sc[0], cells, lane8, blkA, t);
                near[1] = pack_row<3, 1>(u, sc[1], cells, lane8, blkB, t);
            } else {
                near[0] = pack_row<2, 0>(u, sc[0], cells, lane8, blkA, t);
                near[1] = pack_row<2, 1>(u, sc[1], cells, lane8, blkB, t);
            }
            __syncwarp();

            // store: 16 consecutive block slots at a 16-byte boundary leave as one run, else block by block
            const int64_t slot = dst < 0 ? -1 : dst + head * a.dst_head;
            const bool ok = slot >= 0 && slot < sd.n_blocks;
            const int64_t slot0 = __shfl_sync(0xffffffffu, slot, 0);
            uint8_t *out0 = sd.blocks + slot0 * bytes;
            const bool run = __all_sync(0xffffffffu, ok && slot == slot0 + (lane & 15)) && ((uintptr_t)out0 & 15) == 0;
            const uint32_t okm = __ballot_sync(0xffffffffu, ok);
            if (run) {
                for (int i = lane; i < bytes; i += 32)
                    reinterpret_cast<uint4 *>(out0)[i] = reinterpret_cast<const uint4 *>(stage)[i];
            } else {
                for (int q = 0; q < kTok; ++q) {
                    const int64_t s = __shfl_sync(0xffffffffu, slot, q);
                    if (!((okm >> q) & 1u)) continue;
                    uint16_t *o = reinterpret_cast<uint16_t *>(sd.blocks + s * bytes);
                    const uint16_t *b = stage + q * (bytes / 2);
                    for (int i = lane; i < bytes / 2; i += 32) o[i] = b[i];
                }
            }

            // rows to take again: bits 4 g .. of a mask for rows g and g + 8 (any thread of the quad speaks for its
            // row)
            uint32_t todo[2], ties[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                uint32_t m = __ballot_sync(0xffffffffu, redo[r] || near[r] < sd.eps);
                m |= m >> 1;
                todo[r] = (m | m >> 2) & 0x11111111u;
                ties[r] = __ballot_sync(0xffffffffu, tie[r]) & 0x11111111u;
            }
            if (todo[0] | todo[1] | ties[0] | ties[1]) {
                // lane n < 16 lists row n: for its norm, or whole
                const int bit = 4 * (lane & 7), odd = lane & 8;
                const bool whole = ((odd ? todo[1] : todo[0]) >> bit) & 1u, tied = ((odd ? ties[1] : ties[0]) >> bit) & 1u;
                if (lane < kTok && ok && (whole || tied)) {
                    const int at = atomicAdd(&sm.listed[whole ? 1 : 0], 1);
                    if (at < a.list)
                        list_of(sm, a.tiles)[whole ? a.list + at : at] = {unit, (uint32_t)head << 6 | (tile * kTok + lane)};
                }
            }
            __syncwarp();
        }
    }
    __syncthreads();
    finish<DT>(which, rope, a);
}

// Few rows: latency is what counts.  A warp per row, four elements per lane,
// the rotary partner and five of the transform's seven stages by shuffles; all
// loads are under way while the CTA fills the quantiser's cells (one copy: a
// warp's few lookups can bear the conflicts).  The whole call is then launch,
// one memory latency and about 400 instructions, 3.3 us for 16 tokens x 8 heads
// without a row that float32 does not decide, 4.2 with some (most calls of 256
// rows have one), where insert_kernel's tile takes 11.5.  Six CTAs per SM in all
// (four took 1024 tokens the same, eight 8% longer, one CTA for every four rows
// half as long again).
struct SmallShared {
    uint2 cells[128];                         // as Shared's, one copy
    alignas(16) ff again[kWarps][kD];         // values of a row taken again
};

template <int DT>
__global__ void __launch_bounds__(kThreads) insert_few_kernel(const __grid_constant__ tq_rope rope,
                                                              const __grid_constant__ InsertArgs a) {
    __shared__ SmallShared sm;
    const int tid = threadIdx.x, warp = tid >> 5;
    const Side &sd = a.side[a.side[0].x ? blockIdx.y : 1];
    const int bits = sd.bits;
    const uint32_t rows = (uint32_t)a.n_tok * (uint32_t)a.heads;
    uint32_t id = blockIdx.x * kWarps + warp;
    // what a row needs from memory, on its way while the cells are filled
    const uint8_t *row = nullptr;
    int64_t tok = 0, dst = -1;
    int head = 0;
    FewIn in;
    auto load = [&]() {
        const uint32_t n = id / (uint32_t)a.heads;
        tok = n;
        head = (int)(id - n * (uint32_t)a.heads);
        row = sd.x + tok * sd.tok + head * sd.head;
        in = few_load<DT>(row, tok, sd, rope, a);
        dst = a.dst[tok];
    };
    if (id < rows) load();
    const FewLane w = few_lane(sd, rope, a);
    {
        uint32_t below = 0;
        float edge = 3.0e38f;   // as in insert_kernel
        for (int j = 0; j < (1 << bits) - 1; ++j) {
            const float v = sd.b[j] * kGrid;
            const int at = (int)floorf(v + 64.5f);
            if (at < tid) ++below;
            if (at == tid) edge = v;
        }
        sm.cells[tid] = make_uint2(__float_as_uint(edge), below + 1);
    }
    __syncthreads();

    const uint8_t *cells = reinterpret_cast<const uint8_t *>(sm.cells);
    for (; id < rows; id += gridDim.x * kWarps) {
        if (row == nullptr) load();
        const int64_t slot = dst < 0 ? -1 : dst + head * a.dst_head;
        if (slot >= 0 && slot < sd.n_blocks) {
            few_row<DT>(in, w, cells, 4, row, sd.blocks + slot * (2 + 16 * bits), sd, rope, a, tok, sm.again[warp]);
            __syncwarp();
        }
        row = nullptr;
    }
}

template <int DT>
int launch_few(const tq_rope &rope, const InsertArgs &a, int sides, cudaStream_t st) {
    const int64_t ctas = (a.n_tok * a.heads + kWarps - 1) / kWarps;
    const dim3 grid((unsigned)min64(ctas, (int64_t)sm_count() * 6 / sides), (unsigned)sides);
    insert_few_kernel<DT><<<grid, kThreads, 0, st>>>(rope, a);
    return launch_status();
}

template <int DT>
int launch(const tq_rope &rope, const InsertArgs &a, cudaStream_t st) {
    const int smem = (int)(sizeof(Shared) + (size_t)a.tiles * sizeof(float4) * 8 * kTok * 4 + 2 * a.list * sizeof(Listed));
    static int done[64] = {0};
    if (set_smem_limit((const void *)insert_kernel<DT>, smem, done) != TQ_OK) return TQ_ERR_CUDA;
    insert_kernel<DT><<<a.ctas[0] + a.ctas[1], kThreads, smem, st>>>(rope, a);
    return launch_status();
}

int launch_part(int dtype, const tq_rope &rope, const InsertArgs &a, int sides, cudaStream_t st) {
    const bool small = a.n_tok <= (int64_t)sm_count() * kFewRows / ((int64_t)a.heads * sides);
    switch (dtype) {
        case TQ_BF16: return small ? launch_few<TQ_BF16>(rope, a, sides, st) : launch<TQ_BF16>(rope, a, st);
        case TQ_F16: return small ? launch_few<TQ_F16>(rope, a, sides, st) : launch<TQ_F16>(rope, a, st);
        default: return small ? launch_few<TQ_F32>(rope, a, sides, st) : launch<TQ_F32>(rope, a, st);
    }
}

// A bound for a codebook, in v.
float border(const Bound &e, const tq_codebook *cb) {
    float b = 0.f;
    for (int i = 0; i < cb->levels - 1; ++i) b = std::fmax(b, std::fabs(cb->boundaries[i]) * 11.3137085f);
    return (e.row + e.level * b) * 5.9604645e-8f * kUnit;
}

// The quantiser's cells hold at most one boundary each, and no boundary lies
// within 1/64 of a cell's edge (a coordinate near it is then always compared
// with it).  True of the codebooks of tq_codebook_load.
bool cells_ok(const tq_codebook *cb) {
    int last = -1;
    for (int i = 0; i < cb->levels - 1; ++i) {
        const float v = cb->boundaries[i] * kGrid;
        if (!(std::fabs(v) < 62.f)) return false;
        const float n = std::floor(v + 64.5f);
        if (std::fabs(v + 64.f - n) > 0.5f - 1.f / 64.f) return false;
        const int cell = (int)n;
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
    if (heads >= 1 << 26) return TQ_ERR_UNSUPPORTED;   // (Listed)
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
        const bool direct = s.style == kRopeNone && dtype != TQ_F32;
        s.ulps = direct ? kTieUlpsDirect : kTieUlps;
        s.eps = border(s.style != kRopeNone ? kBoundRope : direct ? kBoundDirect : kBoundSplit, cbs[i]);
        s.eps_few = border(s.style != kRopeNone ? kBoundFewRope : kBoundFew, cbs[i]);
    }
    if (n_tok == 0 || (!k && !v)) return TQ_OK;
    if (!dst) return TQ_ERR_ARG;
    if (!aligned(dst, 8) || (rope && !aligned(pos, 8))) return TQ_ERR_ALIGN;
    if (rope && pos_axis_stride < 0) return TQ_ERR_ARG;
    a.pos = pos;
    a.pos_axis = pos_axis_stride;
    a.dst = dst;
    a.dst_head = dst_head_stride;
    a.heads = heads;
    for (int i = 0; i < 4; ++i) a.signs[i] = signs.w[i];
    // token tiles of a CTA: its four warps share a tile's sines, or take a tile each where heads are few
    a.tiles = heads == 1 ? 4 : heads == 2 ? 2 : 1;
    // the lists: what four CTAs leave of 196 KB of shared memory (with more of it, and less L1, float32 rows take 15%
    // longer)
    a.list = a.tiles > 1 ? 128 : 190;
    const int sides = (k != nullptr) + (v != nullptr);
    const int64_t slots = (int64_t)sm_count() * 4;
    // a rotated key costs about half as much again as a value
    const int64_t share = sides == 1 ? slots : a.side[0].style == kRopeNone ? slots / 2 : slots * 3 / 5;
    // A launch takes 80 rows of a CTA for every place of a list at most: of random rows up to 0.8% come on one, and a
    // CTA whose list overflows takes all its rows again, four times as long.  Half a million tokens x 8 heads.
    const int64_t fewest = sides == 1 ? slots : min64(share, slots - share);
    const int64_t most = max64(64, (int64_t)a.list * 80 * fewest / heads & ~(int64_t)63);
    tq_rope none;
    if (!rope) std::memset(&none, 0, sizeof(none));
    for (int64_t done = 0; done < n_tok; done += most) {
        a.n_tok = min64(most, n_tok - done);
        const int64_t tiles = (a.n_tok + (int64_t)kTok * a.tiles - 1) / (kTok * a.tiles);
        // with few tiles, four heads a CTA fill more SMs
        a.heads_per_cta = heads <= kWarps || tiles * sides >= slots ? heads : kWarps;
        a.groups = (heads + a.heads_per_cta - 1) / a.heads_per_cta;
        if (tiles * a.groups > 0x3FFFFFFF) return TQ_ERR_UNSUPPORTED;
        a.units = (int)(tiles * a.groups);
        a.ctas[0] = k ? (int)min64(a.units, share) : 0;
        a.ctas[1] = v ? (int)min64(a.units, k ? slots - share : slots) : 0;
        const int status = launch_part(dtype, rope ? *rope : none, a, sides, static_cast<cudaStream_t>(stream));
        if (status != TQ_OK) return status;
        for (Side &s : a.side)
            if (s.x) s.x += a.n_tok * s.tok;
        if (rope) a.pos += a.n_tok;
        a.dst += a.n_tok;
    }
    return TQ_OK;
}
