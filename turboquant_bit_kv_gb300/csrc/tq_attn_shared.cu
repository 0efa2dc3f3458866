// tq_attn_decode_shared: one query token per sequence over a packed cache
// whose first part, a prefix, is the same for the whole batch.
//
//   o_b = sum_t softmax(s_b)_t v_t over the prefix's tokens and sequence b's own,
//   s_t = scale * n_t <R q, c[code_t]>,  values summed in the rotated domain,
//   o = R^T (sum) / sqrt(128) at the end.
//
// A sequence at a time, the prefix would be read and its codes looked up once
// per sequence; looking them up is what bounds the decode attention.  Together,
// the B x G query rows of a KV head meet the same keys, so the prefix is two
// dense products on the 5th-generation tensor cores and every code is turned
// into a number once per 256 rows.  The sequences' own tokens go through the
// decode attention's kernel (tq_attn_mma.cuh) as they are; a merge adds the two
// parts up: each part of the context leaves the maximum, the sum and the sum of
// values of its softmax, and those join exactly.
//
// Four launches, chained as programmatic dependents: query prep (rotated once,
// as operand tiles and as fragments), own tokens, prefix, merge.  The prefix
// comes second because its start (tensor memory, the first blocks and their
// levels) needs nothing of the others and goes on while the own tokens end; the
// other way round 17 sequences behind 10007 tokens take 44.0 us, so 42.2 (64 behind
// 32769: 81.9 and 81.3).
//
// The prefix kernel.  A CTA takes 256 query rows (two tiles of 128, one
// stream each) or, where a KV head has an odd tile, 128 (both streams take that
// tile, every other key tile each), and a range of the prefix in tiles of 128
// keys:
//   S[128 rows x 128 keys] = Q K^T   Q split hi + lo into fp16, K single fp16
//   O[128 rows x 128 dims] += P V    P split hi + lo, in tensor memory, V single
// accumulated in float32 in tensor memory.  Centroids are fp16 under a common
// factor that makes their roundings small (attn_centroid_factor: at most 2^-18
// / 2^-15 / 2^-13.5 of the level for 2 / 3 / 4 bits), so one product with K
// does where the decode kernel's own factor of 1 needs two.  Key norms scale
// the scores, value norms the probabilities.
//
// Tensor memory: S of stream x at column 128 x, O at 256 + 128 x.  P takes the
// place of S: a thread reads 32 scores of its row and writes their
// probabilities' hi (16 columns) and lo parts over them.  The products are
// issued in the order P V of one stream, S of the same stream's next tile, then
// the other stream, so one stream's softmax runs while the other's products do.
//
// Roles (576 threads, one CTA per SM):
//   warps 0-3, 4-7    rows of stream 0, 1: a thread a row (its tensor-memory
//       lane), in one pass over its scores.  The reference of a row's exponents
//       moves only when 32 keys' largest score plus the tile's largest value
//       norm (in log2) exceeds it by more than 8, so O is rarely rescaled, and P
//       times the value norm stays below 2^8 (as held, 2^15) whatever the norms
//       are.
//   warps 8-11, 12-15    a thread a key, a thread a value: codes to fp16 in
//       registers (byte permutes over the levels' bytes; no lookups in shared
//       memory, which the products keep busy), into the swizzled K and V tiles.
//       The key warps also unpack both norms, which the rows want first.
//   warp 16    bulk copies: the query tiles, then the packed blocks.
//   warp 17    issues the products.
// Every wait is bounded; one that gives up is recorded (tq_device_status).
//
// What bounds it: 256 rows x 128 keys are 4096 cycles of products and take some
// 6400: a stream's scores, softmax and values follow one another, a row's 128
// keys take its thread 2300 to 3000 cycles (two thirds of all instructions; the
// levels of 256 blocks are the rest), and shared memory serves the products and
// the levels' stores at once.  64 sequences of 28/4 heads behind 32769 tokens of
// 3 bits: 63 us of the call's 81, the tensor pipe active for 51 % of them, 40 %
// of the issue slots used.
#include <cmath>

#include "tq_attn.cuh"
#include "tq_attn_mma.h"
#include "tq_internal.h"
#include "tq_tc.cuh"

namespace tq {

int launch_attn_mma_scores_k2(const AttnArgs &a, MmaPlan &plan, int vb, int nt, bool paged, cudaStream_t st);
int launch_attn_mma_scores_k3(const AttnArgs &a, MmaPlan &plan, int vb, int nt, bool paged, cudaStream_t st);
int launch_attn_mma_scores_k4(const AttnArgs &a, MmaPlan &plan, int vb, int nt, bool paged, cudaStream_t st);
int launch_attn_prep_mma(const AttnArgs &a, const MmaPlan &plan, int qjl, cudaStream_t st);

namespace {

constexpr int kShKeys = 128;                 // keys per tile
constexpr int kShRows = 128;                 // rows per stream
constexpr int kShRowWarps = 8, kShKeyWarps = 4;
constexpr int kShValueWarp = kShRowWarps + kShKeyWarps;   // (the first of as many)
constexpr int kShProducer = kShValueWarp + kShKeyWarps, kShMma = kShProducer + 1;
constexpr int kShThreads = 32 * (kShMma + 1);
constexpr uint32_t kShCols = 512, kShColO = 256;
constexpr int kShNormSlots = 8;
constexpr int kShNormSlot = (2 * kShKeys + 4) * 4;   // key norms | value norms | four maxima of log2 value norm
constexpr float kShUp = 128.f;               // P is held times this

// mbarriers
enum {
    kQFull = 0,        // query tiles landed
    kKFull = 1,        // [2] packed key blocks landed
    kKEmpty = 3,       // [2] ... and turned into the operand tile
    kVFull = 5,        // [2]
    kVEmpty = 7,       // [2]
    kKReady = 9,       // [2] operand tile of keys written (4 key warps)
    kKFree = 11,       // [2] the products that read it completed
    kVReady = 13,      // [2]
    kVFree = 15,       // [2]
    kNReady = 17,      // [8] norms of a tile written
    kSReady = 25,      // [2] stream's scores in tensor memory
    kPReady = 27,      // [2] stream's P in their place (4 row warps)
    kODone = 29,       // [2] stream's last product completed
    kDrain = 31,
    kShBars = 32
};

// Shared memory, from a 1024-byte aligned base.  A KV head's even tiles of
// rows: Q of the two streams, one K and one V tile; an odd one: Q, and a K and
// a V tile for each stream.  32 KB apiece: hi and lo of Q, K, V.
template <int KB, int VB>
struct ShSmem {
    static constexpr int kTile = 32768;
    static constexpr int kKBlk = 6 * kTile;                          // packed key blocks, kNK stages
    static constexpr int kKBytes = kShKeys * (2 + 16 * KB), kVBytes = kShKeys * (2 + 16 * VB);
    static constexpr int kRest = kShNormSlots * kShNormSlot + kShBars * 8 + 16 + 1024;
    // value blocks two tiles ahead (their norms are wanted before the tile's turn), key blocks too where
    // there is room
    static constexpr int kNV = 2;
    static constexpr int kNK = kKBlk + 2 * kKBytes + 2 * kVBytes + kRest <= 232448 ? 2 : 1;
    static constexpr int kVBlk = kKBlk + kNK * kKBytes;
    static constexpr int kNorm = kVBlk + kNV * kVBytes;              // [kShNormSlots]
    static constexpr int kBars = kNorm + kShNormSlots * kShNormSlot;
    static constexpr int kSlot = kBars + kShBars * 8;                // tensor-memory base, failure flag
    static constexpr int kTotal = kSlot + 16 + 1024;
    static_assert(kTotal <= 232448, "shared memory of one CTA");
    static_assert(kNorm % 16 == 0 && kBars % 8 == 0, "alignment");
};

// Partition of the prefix's work: per KV head `pairs` CTAs' worth of 256 rows in
// s2 ranges of the prefix each and, with an odd tile, one of 128 in s1 ranges.
struct SharedPlan {
    int tiles, pairs, odd, s2, s1, per_head, ctas;
    int most;   // CTAs of no plan for this prefix or a shorter one are more
};

struct SharedArgs {
    const uint8_t *q;         // operand tiles [Hkv][tiles][hi, lo][32 KB]
    const uint8_t *k, *v;     // the prefix's blocks [Hkv][cap], or pools with a table
    const int32_t *table;
    const int32_t *len;       // tokens of the prefix (null: P)
    float *part;              // [ctas][2][128][132]
    int rows, Hkv, P, cap, page;
    SharedPlan plan;
    float k_norm;             // 1 / the key centroids' factor
    uint32_t kt[4], vt[4];    // bytes of the levels (level_bytes)
    int drop;                 // test hook: the copies' barriers wait for an arrival that never comes
};

__device__ __forceinline__ int shared_len(const int32_t *len, int P) {
    if (!len) return P;
    const int n = *len;
    return n < 0 ? 0 : (n > P ? P : n);
}

// Range w of n tiles cut into W = min(ranges, n) equal parts.
__device__ __forceinline__ void shared_range(int n, int ranges, int w, int &lo, int &hi) {
    const int W = n < ranges ? n : ranges;
    lo = w < W ? (int)((int64_t)w * n / W) : 0;
    hi = w < W ? (int)(((int64_t)w + 1) * n / W) : 0;
}

__device__ __forceinline__ uint32_t sh_prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

__device__ __forceinline__ uint32_t sh_lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t sh_lds16(uint32_t addr) {
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ void sh_sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void sh_bulk(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Shared-memory descriptor of an operand tile in the 128-byte swizzle layout.
__device__ __forceinline__ uint64_t sh_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// kind::f16, float32 accumulator, fp16 operands, M = N = 128; mn: B is MN-major.
__host__ __device__ constexpr uint32_t sh_idesc(uint32_t mn) {
    return (1u << 4) | (mn << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
}

// D (+)= A B, A in tensor memory (rows in lanes, two fp16 a column).
__device__ __forceinline__ void sh_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::
            "r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One lane of a converged warp.  Products are issued under it, group by group,
// by a warp that otherwise runs as a whole: their operands are then the same
// in every lane, and cost no instructions to bring into uniform registers.
__device__ __forceinline__ bool sh_elect() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// 2^x (the special-function unit's approximation, a few ulp; 2^-inf = 0).
__device__ __forceinline__ float sh_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (hi, lo) fp16 parts of two floats of at most 2^15: hi the ten leading bits after the first, lo what is left of
// them, x = hi + lo to about 2^-21 (2^-25 where x is below fp16's normal numbers).
__device__ __forceinline__ void sh_split(float2 x, uint32_t &hi, uint32_t &lo) {
    const float2 t = make_float2(__uint_as_float(__float_as_uint(x.x) & 0xFFFFE000u),
                                 __uint_as_float(__float_as_uint(x.y) & 0xFFFFE000u));
    const float2 r = __ffma2_rn(t, make_float2(-1.f, -1.f), x);   // (exact)
    const __half2 h = __floats2half2_rn(t.x, t.y), l = __floats2half2_rn(r.x, r.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

// ---- codes to fp16 levels.  A byte permute picks four bytes by the four low
// nibbles of its selector, each from eight: the levels' high and low bytes,
// which two more permutes put together into two pairs.  Tables t: 2 bits: high
// bytes, low bytes of the four levels; 3 bits: high bytes (two words), low
// bytes (two words) of the eight; 4 bits: the same of the eight positive levels
// (the other half mirrored, their sign set).  The order in which the dims come
// out is the one that costs least; operand_place gives a dim's place, and Q
// and the sums of values follow it.

// Eight levels as four words of two, from a selector of eight nibbles (3, 4 bits).
template <int BITS>
__device__ __forceinline__ void levels8(const uint32_t (&t)[4], uint32_t sel, uint32_t raw, uint32_t (&o)[4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t s = h ? sel >> 16 : sel;
        uint32_t hb = sh_prmt(t[0], t[1], s);
        const uint32_t lb = sh_prmt(t[2], t[3], s);
        if constexpr (BITS == 4) {
            // bit 3 of a nibble copies the byte's top bit into all of it: 0xFF for the upper half, else
            // 0x80; bit 6 of that, inverted, is the sign
            const uint32_t r = sh_prmt(0x80808080u, 0x80808080u, h ? raw >> 16 : raw);
            hb |= ~(r << 1) & 0x80808080u;
        }
        o[2 * h] = sh_prmt(lb, hb, 0x5140u);
        o[2 * h + 1] = sh_prmt(lb, hb, 0x7362u);
    }
}

// Levels of 32 dims of 3-bit codes, in the operand's order: l0, l1 the low
// plane's words of dims 0 .. 15 and 16 .. 31, h the high plane's.  Selector j
// takes dims 4 i + j into its nibbles 2 i and dims 16 + 4 i + j into 2 i + 1: the
// low plane's bits lie in l0's and l1's bytes i, and the high plane's four
// nibbles of 16 dims are spread to bytes once for all four selectors.
__device__ __forceinline__ void levels32(const uint32_t (&t)[4], uint32_t l0, uint32_t l1, uint32_t h, uint32_t (&o)[16]) {
    const uint32_t p = sh_prmt(h, 0, 0x1100u), q = sh_prmt(h, 0, 0x3322u);
    const uint32_t u = (p & 0x000F000Fu) | ((p >> 4) & 0x0F000F00u) | ((q << 4) & 0x00F000F0u) | (q & 0xF000F000u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t b = j < 2 ? l1 << (4 - 2 * j) : l1 >> (2 * j - 4);
        const uint32_t c = j < 2 ? u << (2 - j) : u >> (j - 2);
        uint32_t e[4];
        levels8<3>(t, ((l0 >> (2 * j)) & 0x03030303u) | (b & 0x30303030u) | (c & 0x44444444u), 0, e);
#pragma unroll
        for (int k = 0; k < 4; ++k) o[4 * j + k] = e[k];
    }
}

// Levels of 16 dims of 2- or 4-bit codes as eight words of two, in the operand's
// order: w the code words of those dims (4 bits: two, 2 bits: one).
template <int BITS>
__device__ __forceinline__ void levels16(const uint32_t (&t)[4], uint32_t w0, uint32_t w1, uint32_t (&o)[8]) {
    if constexpr (BITS == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w = i ? w1 : w0;
            const uint32_t flip = ((~w >> 3) & 0x11111111u) * 7u;   // the lower half counts down
            uint32_t q[4];
            levels8<4>(t, (w ^ flip) & 0x77777777u, w, q);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[4 * i + k] = q[k];
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // the codes of dims 4 i + k in bytes; nibbles code + 4 (low byte), code (high byte) pick a level whole
            const uint32_t d = ((w0 >> (2 * k)) & 0x03030303u) * 17u | 0x04040404u;
            o[2 * k] = sh_prmt(t[0], t[1], d);
            o[2 * k + 1] = sh_prmt(t[0], t[1], d >> 16);
        }
    }
}

// A block's codes (block at shared address blk, 2-byte aligned) into row r of an
// operand tile at `tile`, 32 dims at a time (rolled: straight-line code for a
// whole row would be fetched anew for every tile).
template <int BITS>
__device__ __forceinline__ void dequant_row(const uint32_t (&t)[4], uint32_t blk, uint32_t tile, int r) {
    constexpr int NW = BITS == 4 ? 4 : 2;   // words per 32 dims (3 bits: of the low plane)
    const uint32_t at = blk + 2, base = at & ~3u, sh = (at & 3u) * 8u;
    const uint32_t row = tile + r * 128;
#pragma unroll 1
    for (int g = 0; g < 4; ++g) {
        uint32_t raw[NW + 1], w[NW], hp = 0;
#pragma unroll
        for (int i = 0; i <= NW; ++i) raw[i] = sh_lds32(base + 4 * NW * g + 4 * i);
#pragma unroll
        for (int i = 0; i < NW; ++i) w[i] = __funnelshift_r(raw[i], raw[i + 1], sh);
        if constexpr (BITS == 3)
            hp = __funnelshift_r(sh_lds32(base + 32 + 4 * g), sh_lds32(base + 36 + 4 * g), sh);
        const uint32_t half = row + (g >> 1) * 16384;
        uint32_t o[16];
        if constexpr (BITS == 3) {
            levels32(t, w[0], w[1], hp, o);
        } else {
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                uint32_t e[8];
                levels16<BITS>(t, w[(a * NW / 2) % NW], w[(a * NW / 2 + 1) % NW], e);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[8 * a + k] = e[k];
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            sh_sts128(half + ((((uint32_t)(4 * (g & 1) + k)) ^ (r & 7)) << 4), o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
    }
}

// A row's softmax over a tile of 128 keys.  m: the reference of its exponents
// (-inf before the first finite score), l: the sum of 2^(s - m).
struct RowState {
    float m, l;
};

// The reference moves up by `up` (a whole number; 0 for rows that stay) or is
// set: what the row has summed up, the stream's O (of the tiles before, if any)
// and the `done` keys of this tile whose P is written already are scaled down.
// Rare: out of line.
__device__ __noinline__ void move_reference(uint32_t s_col, uint32_t o_col, bool scale_o, int done, float f) {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");   // P of the keys done
    if (scale_o) {
#pragma unroll 1
        for (int c = 0; c < 128; c += 16) {
            uint32_t w[16];
            tc_ld16(o_col + c, w);
            tc_wait_ld();
#pragma unroll
            for (int q = 0; q < 16; ++q) w[q] = __float_as_uint(__uint_as_float(w[q]) * f);
            tc_st16(o_col + c, w);
        }
    }
    const __half2 f2 = __float2half2_rn(f);   // (a power of two: exact, or below what P holds)
#pragma unroll 1
    for (int c = 0; c < done; c += 16) {
        uint32_t w[16];
        tc_ld16(s_col + c, w);
        tc_wait_ld();
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const __half2 p = __hmul2(*reinterpret_cast<const __half2 *>(&w[q]), f2);
            w[q] = *reinterpret_cast<const uint32_t *>(&p);
        }
        tc_st16(s_col + c, w);
    }
}

// The row's scores, 32 keys at a time: P = 2^(s - m) times the value norms, as
// fp16 hi and lo parts, over the scores.  kn, vn: norms of the tile's keys and
// values, lv: log2 of the largest value norm.  m is kept above every s + lv - 8,
// so that P times 2^7 stays below 2^15.  TAIL: only `valid` keys are there
// (the others have the value norm 0).
template <bool TAIL>
__device__ __forceinline__ void row_tile(RowState &st, uint32_t s_col, uint32_t o_col, bool scale_o, const float *kn,
                                         const float *vn, float lv, int valid) {
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
        float s[32];
        tc_ld32(s_col + c, s);
        tc_wait_ld();
        // no finite score so far: scores are -inf (P 0) or NaN (which stays NaN)
        float mref = st.m == -INFINITY ? 0.f : st.m;
        const float2 m2 = make_float2(-mref, -mref);
        float mx = -INFINITY, my = -INFINITY;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float4 n = reinterpret_cast<const float4 *>(kn + c)[q];
            const float2 x = __ffma2_rn(make_float2(s[4 * q], s[4 * q + 1]), make_float2(n.x, n.y), m2);
            const float2 y = __ffma2_rn(make_float2(s[4 * q + 2], s[4 * q + 3]), make_float2(n.z, n.w), m2);
            s[4 * q] = x.x;
            s[4 * q + 1] = x.y;
            s[4 * q + 2] = y.x;
            s[4 * q + 3] = y.y;
            if constexpr (TAIL) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + 4 * q + e >= valid) s[4 * q + e] = -INFINITY;
            }
            mx = fmaxf(fmaxf(mx, s[4 * q]), s[4 * q + 1]);
            my = fmaxf(fmaxf(my, s[4 * q + 2]), s[4 * q + 3]);
        }
        const float top = fmaxf(mx, my) + lv;   // (above m)
        const bool set = st.m == -INFINITY && top > -INFINITY;
        const bool move = set || top > 8.f;
        if (__any_sync(0xffffffffu, move)) {
            const float up = move ? ceilf(top) : 0.f;
            const float f = set || !move ? 1.f : exp2f(-up);   // (unset: nothing has been summed up)
            move_reference(s_col, o_col, scale_o, c, f);
            st.l *= f;
            sum = make_float2(sum.x * f, sum.y * f);
            if (move) st.m = mref + up;
#pragma unroll
            for (int q = 0; q < 32; ++q) s[q] -= up;
        }
        uint32_t wh[16], wl[16];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float4 v = reinterpret_cast<const float4 *>(vn + c)[q];
            const float2 p = make_float2(sh_ex2(s[4 * q]), sh_ex2(s[4 * q + 1]));
            const float2 r = make_float2(sh_ex2(s[4 * q + 2]), sh_ex2(s[4 * q + 3]));
            sum = __fadd2_rn(sum, __fadd2_rn(p, r));
            sh_split(__fmul2_rn(p, make_float2(v.x, v.y)), wh[2 * q], wl[2 * q]);
            sh_split(__fmul2_rn(r, make_float2(v.z, v.w)), wh[2 * q + 1], wl[2 * q + 1]);
        }
        tc_st16(s_col + c, wh);
        tc_st16(s_col + c + 16, wl);
    }
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    st.l += sum.x + sum.y;
}

template <int KB, int VB>
__global__ void __launch_bounds__(kShThreads, 1) attn_shared_kernel(const __grid_constant__ SharedArgs a) {
    using S = ShSmem<KB, VB>;
    extern __shared__ __align__(16) uint8_t sh_smem_raw[];
    const uint32_t raw_s = (uint32_t)__cvta_generic_to_shared(sh_smem_raw);
    const uint32_t base_s = (raw_s + 1023u) & ~1023u;
    uint8_t *smem = sh_smem_raw + (base_s - raw_s);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int i) { return base_s + S::kBars + 8u * (uint32_t)i; };
    volatile int *fail_s = reinterpret_cast<volatile int *>(smem + S::kSlot + 4);
    float *norms = reinterpret_cast<float *>(smem + S::kNorm);

    // ---- the CTA's rows and key tiles
    const SharedPlan &p = a.plan;
    const int kvh = blockIdx.x / p.per_head, in = blockIdx.x % p.per_head;
    const bool two = in < p.pairs * p.s2;
    const int qt = two ? 2 * (in / p.s2) : 2 * p.pairs;   // first tile of rows
    const int len = shared_len(a.len, a.P);
    int tile0, tile1;
    shared_range((len + kShKeys - 1) / kShKeys, two ? p.s2 : p.s1, two ? in % p.s2 : in - p.pairs * p.s2, tile0, tile1);
    const int nt = tile1 - tile0;
    // operand tiles: Q of stream x, and key / value tiles of stage st
    auto q_at = [&](int x) { return base_s + (two ? x : 0) * 2 * S::kTile; };
    auto k_at = [&](int st) { return base_s + (two ? 4 : 2 + 2 * st) * S::kTile; };
    auto v_at = [&](int st) { return k_at(st) + S::kTile; };
    // tile i of the CTA: its operand stage, and how often that has been used before
    auto stage = [&](int i) { return two ? 0 : i & 1; };
    auto use = [&](int i) { return two ? i : i >> 1; };

    if (tid == 0) {
        const int extra = a.drop ? 1 : 0;   // (test hook)
        tc_mbar_init(bar(kQFull), 1 + extra);
        for (int s = 0; s < 2; ++s) {
            tc_mbar_init(bar(kKFull + s), 1 + extra);
            tc_mbar_init(bar(kVFull + s), 1 + extra);
            tc_mbar_init(bar(kKEmpty + s), kShKeyWarps);
            tc_mbar_init(bar(kVEmpty + s), 2 * kShKeyWarps);   // (values, and their norms)
            tc_mbar_init(bar(kKReady + s), kShKeyWarps);
            tc_mbar_init(bar(kVReady + s), kShKeyWarps);
            tc_mbar_init(bar(kKFree + s), two ? 2 : 1);
            tc_mbar_init(bar(kVFree + s), two ? 2 : 1);
            tc_mbar_init(bar(kSReady + s), 1);
            tc_mbar_init(bar(kPReady + s), 4);
            tc_mbar_init(bar(kODone + s), 1);
        }
        for (int s = 0; s < kShNormSlots; ++s) tc_mbar_init(bar(kNReady + s), kShKeyWarps);
        tc_mbar_init(bar(kDrain), 1);
        *fail_s = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base_s + S::kSlot),
                     "r"(kShCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + S::kSlot);
    asm volatile("griddepcontrol.launch_dependents;");

    // a bounded wait; one that gives up is recorded, and the caller's role makes no further waits
    auto wait = [&](bool &ok, int b, uint32_t parity) {
        if (ok && !tc_mbar_wait(bar(b), parity & 1u)) {
            ok = false;
            *fail_s = 1;
            note_wait_failed();
        }
    };

    if (warp == kShProducer) {
        // ---- copies: lane l takes piece l of a tile (one, or one for each page it meets: 17 at most)
        bool ok = true;
        // the query tiles come from the prep kernel (which the own tokens' has waited for); the blocks do not,
        // and the first go ahead
        auto queries = [&]() {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            if (nt > 0 && lane == 0) {
                const int n = two ? 4 : 2;
                const uint8_t *src = a.q + ((int64_t)kvh * p.tiles + qt) * (2 * S::kTile);
                tc_mbar_expect_tx(bar(kQFull), (uint32_t)(n * S::kTile));
                for (int i = 0; i < n; ++i)
                    sh_bulk(base_s + i * S::kTile, src + (int64_t)i * S::kTile, S::kTile, bar(kQFull));
            }
        };
        if (nt == 0) queries();   // (waits, as every CTA does: who waits for this grid counts on the end of those before)
        for (int i = 0; i < nt && ok; ++i) {
            const int t0 = (tile0 + i) * kShKeys;
            const int end = min(t0 + kShKeys, (len + 7) & ~7);
            int64_t slot = 0;
            int from = t0, n = 0;
            if (!a.table) {
                slot = (int64_t)kvh * a.cap + t0;
                n = lane == 0 ? end - t0 : 0;
            } else {
                const int64_t pg = t0 / a.page + lane;
                const int64_t lo = pg * a.page > t0 ? pg * a.page : t0, hi = min64((pg + 1) * a.page, end);
                if (lo < hi) {
                    from = (int)lo;
                    n = (int)(hi - lo);
                    slot = ((int64_t)a.table[pg] * a.Hkv + kvh) * a.page + (lo - pg * a.page);
                }
            }
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const int ns = kv ? S::kNV : S::kNK, s = i % ns, bytes = (kv ? S::kVBytes : S::kKBytes) / kShKeys;
                if (i >= ns) wait(ok, (kv ? kVEmpty : kKEmpty) + s, (uint32_t)(i / ns - 1));
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t full = bar((kv ? kVFull : kKFull) + s);
                if (lane == 0) tc_mbar_expect_tx(full, (uint32_t)((end - t0) * bytes));
                __syncwarp();
                const uint32_t dst = base_s + (kv ? S::kVBlk + s * S::kVBytes : S::kKBlk + s * S::kKBytes);
                if (n > 0) sh_bulk(dst + (from - t0) * bytes, (kv ? a.v : a.k) + slot * bytes, (uint32_t)(n * bytes), full);
            }
            if (i == 0) queries();
        }
    } else if (warp == kShMma) {
        // ---- the products: item e is stream e & 1's tile e >> 1 (two) or tile e
        bool ok = true;
        const int items = two ? 2 * nt : nt;
        auto tile_of = [&](int e) { return two ? e >> 1 : e; };
        auto warp_wait = [&](int b, uint32_t parity) {
            wait(ok, b, parity);
            ok = __all_sync(0xffffffffu, ok);
        };
        auto scores = [&](int e) {
            const int i = tile_of(e), x = e & 1, st = stage(i);
            if (!two || x == 0) warp_wait(kKReady + st, (uint32_t)use(i));
            if (!ok) return;
            tc_fence_after();
            const uint32_t d = tmem + 128u * (uint32_t)x;
            const uint64_t kd = sh_desc(k_at(st), 16, 1024), qd = sh_desc(q_at(x), 16, 1024);
            if (sh_elect()) {
#pragma unroll
                for (int n = 0; n < 16; ++n) {   // 16 dims at a time: with the hi parts of Q, then the lo parts
                    const uint32_t off = ((n & 7) >> 2) * (16384 / 16) + (n & 3) * (32 / 16);
                    tc_mma(d, qd + off + (n >> 3) * (S::kTile / 16), kd + off, sh_idesc(0), n > 0);
                }
                tc_commit(bar(kSReady + x));
                tc_commit(bar(kKFree + st));
            }
            __syncwarp();
        };
        auto values = [&](int e) {
            const int i = tile_of(e), x = e & 1, st = stage(i);
            if (!two || x == 0) warp_wait(kVReady + st, (uint32_t)use(i));
            warp_wait(kPReady + x, (uint32_t)(e >> 1));
            if (!ok) return;
            tc_fence_after();
            const uint32_t pa = tmem + 128u * (uint32_t)x, d = tmem + kShColO + 128u * (uint32_t)x;
            const uint64_t vd = sh_desc(v_at(st), 16384, 1024);
            if (sh_elect()) {
#pragma unroll
                for (int n = 0; n < 16; ++n)   // 16 keys at a time: of 32, the hi parts, then the lo parts
                    sh_mma_ts(d, pa + 8u * n, vd + (4096 / 16) * (n >> 2) + (2048 / 16) * (n & 1), sh_idesc(1),
                              e > 1 || n > 0);
                tc_commit(bar(kVFree + st));
                if (e + 2 >= items) tc_commit(bar(kODone + x));
            }
            __syncwarp();
        };
        if (items > 0) warp_wait(kQFull, 0);
        for (int e = 0; e < 2 && e < items; ++e) scores(e);
        for (int e = 0; e < items && ok; ++e) {
            values(e);
            if (ok && e + 2 < items) scores(e + 2);
        }
        // before teardown: every product issued here has completed
        if (sh_elect()) tc_commit(bar(kDrain));
        __syncwarp();
        tc_mbar_wait(bar(kDrain), 0u);
    } else if (warp >= kShValueWarp) {
        // ---- value warps: thread = key of the tile
        const int k = tid - 32 * kShValueWarp;
        bool ok = true;
        for (int i = 0; i < nt; ++i) {
            const int st = stage(i), u = use(i), sv = i % S::kNV;
            const uint32_t vblk = base_s + S::kVBlk + sv * S::kVBytes + k * (2 + 16 * VB);
            wait(ok, kVFull + sv, (uint32_t)(i / S::kNV));
            if (u >= 1) wait(ok, kVFree + st, (uint32_t)(u - 1));
            dequant_row<VB>(a.vt, vblk, v_at(st), k);
            // the tiles were written by ordinary stores and are read by the tensor cores
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                tc_mbar_arrive(bar(kVEmpty + sv));
                tc_mbar_arrive(bar(kVReady + st));
            }
        }
    } else if (warp >= kShRowWarps) {
        // ---- key warps: thread = key of the tile; its value's norm too, which the rows want with the scores
        const int k = tid - 32 * kShRowWarps;
        bool ok = true;
        for (int i = 0; i < nt; ++i) {
            const int st = stage(i), u = use(i);
            const int sk = i % S::kNK, sv = i % S::kNV;
            const uint32_t kblk = base_s + S::kKBlk + sk * S::kKBytes + k * (2 + 16 * KB);
            wait(ok, kKFull + sk, (uint32_t)(i / S::kNK));
            wait(ok, kVFull + sv, (uint32_t)(i / S::kNV));
            // (the norms of tile i - 8 have been read: the last wait for a stage says that the products of tile
            // i - 4, or a later one, are done, and P of tile i - 6 came before them)
            const bool live = (tile0 + i) * kShKeys + k < len;
            float *nm = norms + (i % kShNormSlots) * (kShNormSlot / 4);
            const float kn = __half2float(__ushort_as_half((unsigned short)sh_lds16(kblk)));
            const float vn = __half2float(__ushort_as_half((unsigned short)sh_lds16(
                base_s + S::kVBlk + sv * S::kVBytes + k * (2 + 16 * VB))));
            nm[k] = live ? kn * a.k_norm : 0.f;
            nm[kShKeys + k] = live ? vn * kShUp : 0.f;
            // the largest value norm, in [2^-14, 2^16] whatever it is
            float lv = live ? fminf(fmaxf(vn, 0x1p-14f), 0x1p16f) : 0x1p-14f;
            lv = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(lv)));   // (positive: ordered as integers)
            if (lane == 0) nm[2 * kShKeys + warp - kShRowWarps] = log2f(lv);
            __syncwarp();
            if (lane == 0) {
                tc_mbar_arrive(bar(kVEmpty + sv));
                tc_mbar_arrive(bar(kNReady + i % kShNormSlots));
            }
            if (u >= 1) wait(ok, kKFree + st, (uint32_t)(u - 1));
            dequant_row<KB>(a.kt, kblk, k_at(st), k);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                tc_mbar_arrive(bar(kKEmpty + sk));
                tc_mbar_arrive(bar(kKReady + st));
            }
        }
    } else {
        // ---- row warps: thread = row of stream x, keys of the stream's tiles
        const int x = warp >> 2, r = tid & 127;
        const uint32_t lane_t = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t s_col = lane_t + 128u * (uint32_t)x, o_col = lane_t + kShColO + 128u * (uint32_t)x;
        const int mine = two ? nt : (nt - x + 1) >> 1;
        RowState state = {-INFINITY, 0.f};
        bool ok = true;
        for (int t = 0; t < mine; ++t) {
            const int i = two ? t : 2 * t + x;
            const float *nm = norms + (i % kShNormSlots) * (kShNormSlot / 4);
            wait(ok, kNReady + i % kShNormSlots, (uint32_t)(i / kShNormSlots));
            wait(ok, kSReady + x, (uint32_t)t);
            tc_fence_after();
            const int nvalid = len - (tile0 + i) * kShKeys;   // (of 128)
            const float4 lv4 = *reinterpret_cast<const float4 *>(nm + 2 * kShKeys);
            const float lv = fmaxf(fmaxf(lv4.x, lv4.y), fmaxf(lv4.z, lv4.w));
            // (the stream's products before this tile's scores have completed: O may be scaled)
            if (nvalid < kShKeys) row_tile<true>(state, s_col, o_col, t > 0, nm, nm + kShKeys, lv, nvalid);
            else row_tile<false>(state, s_col, o_col, t > 0, nm, nm + kShKeys, lv, kShKeys);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) tc_mbar_arrive(bar(kPReady + x));
        }
        // ---- this row's partial: reference, sum, sums of values by dim
        float m_ref = state.m, l = state.l;
        if (mine > 0) wait(ok, kODone + x, 0);
        tc_fence_after();
        // Rows are put together in shared memory (where the queries were: every product has completed) and
        // leave as one copy a stream, as far as there are rows.
        auto rows_sync = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kShRowWarps) : "memory"); };
        float *own = reinterpret_cast<float *>(smem) + (two ? x * kShRows + r : r) * kPartialFloats;
        // 32 columns of sums to dims: place -> dim, the inverse of operand_place
        auto put = [&](float *out, const float (&o)[32]) {
            float d[32];
#pragma unroll
            for (int q = 0; q < 32; ++q)
                d[VB == 4 ? q : VB == 3 ? 16 * (q & 1) + 4 * ((q >> 1) & 3) + (q >> 3) : (q & 16) + 4 * (q & 3) + ((q >> 2) & 3)] = o[q];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                reinterpret_cast<float4 *>(out)[q] = make_float4(d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]);
        };
        // NaN marks a failed wait, of the roles that these rows' numbers come from too
        if (!ok || *fail_s) l = __int_as_float(0x7fc00000);
        rows_sync();
        if (two) {
            own[0] = m_ref;
            own[1] = l;
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
                float o[32];
                if (mine > 0) {   // (the whole warp)
                    tc_ld32(o_col + c, o);
                    tc_wait_ld();
                }
#pragma unroll
                for (int q = 0; q < 32; ++q) o[q] = mine > 0 ? o[q] * (1.f / kShUp) : 0.f;
                put(own + 4 + c, o);
            }
        } else {
            // both streams' sums of a row lie in its lane: join them, each thread half of the dims
            float2 *stat = reinterpret_cast<float2 *>(smem + S::kKBlk);   // (the packed blocks' place)
            stat[x * kShRows + r] = make_float2(m_ref, l);
            rows_sync();
            const float2 s0 = stat[r], s1 = stat[kShRows + r];
            const float M = fmaxf(s0.x, s1.x);
            const float f0 = s0.x == -INFINITY ? 0.f : exp2f(s0.x - M), f1 = s1.x == -INFINITY ? 0.f : exp2f(s1.x - M);
            if (x == 0) {
                // (a sum that is not finite, of scores that are not, shows whatever its maximum)
                own[0] = M;
                own[1] = (s0.x == -INFINITY ? s0.y : f0 * s0.y) + (s1.x == -INFINITY ? s1.y : f1 * s1.y);
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 64 * x; c < 64 * x + 64; c += 32) {
                float o[32], o1[32];
                if (nt > 0) tc_ld32(lane_t + kShColO + c, o);
                if (nt > 1) tc_ld32(lane_t + kShColO + 128 + c, o1);
                tc_wait_ld();
#pragma unroll
                for (int q = 0; q < 32; ++q)
                    o[q] = ((nt > 0 ? o[q] * f0 : 0.f) + (nt > 1 ? o1[q] * f1 : 0.f)) * (1.f / kShUp);
                put(own + 4 + c, o);
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        rows_sync();
        const int streams = two ? 2 : 1;
        if (r == 0 && x < streams) {
            const int rows = min(kShRows, a.rows - (qt + x) * kShRows);
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                             a.part + (int64_t)(2 * blockIdx.x + x) * kShRows * kPartialFloats),
                         "r"(base_s + (uint32_t)(x * kShRows * kPartialFloats * 4)),
                         "r"((uint32_t)(rows * kPartialFloats * 4))
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // (before the memory is given back)
        }
    }

    // ---- teardown: every product completed (the issuing thread waited for its last commit), every
    // tensor-memory access completed; copies still in flight after a failed wait land first
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*fail_s) {
        if (tid == 0) spin_ns(100000000ull);
        __syncthreads();
    }
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kShCols) : "memory");
}

struct MergeArgs {
    const float *part, *own;
    const int32_t *len, *seq_lens;
    const int2 *live;
    void *out;
    int P, Hq, Hkv, G, out_dtype;
    SharedPlan plan;
    float out_scale;
    uint32_t signs[4];
};

constexpr int kMergeWarps = 2;
constexpr int kMergeDepth = 16;  // slots a warp has on their way at once

// One CTA for one (sequence, query head): 32 slots at a time, the prefix's, then
// the own tokens'.  Both warps take the maxima and sums of all of them, a lane a
// slot, and the sums of values of half of them, a lane four dims, all requested
// at once (reading what other SMs have just written costs a round trip through
// L2; four warps of eight slots took 0.8 us more on 1792 rows, eight of four 4
// us); their sums of values meet in shared memory, and the first turns the
// output back.
__global__ void __launch_bounds__(32 * kMergeWarps) attn_shared_merge_kernel(const __grid_constant__ MergeArgs a) {
    __shared__ __align__(16) float accs[kMergeWarps][kD];
    const int b = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, kvh = h / a.G, g = h % a.G;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const SharedPlan &p = a.plan;
    const int row = b * a.G + g, tile = row / kShRows;
    const bool two = tile < 2 * p.pairs;
    const int n = (shared_len(a.len, a.P) + kShKeys - 1) / kShKeys, ranges = two ? p.s2 : p.s1;
    const float *part = a.part + ((int64_t)(kvh * p.per_head + (two ? (tile >> 1) * p.s2 : p.pairs * p.s2)) * 2 * kShRows +
                                  (two ? (tile & 1) * kShRows : 0) + row % kShRows) * kPartialFloats;
    const bool empty = a.seq_lens && a.seq_lens[b] < 0;
    const int before = empty ? 0 : (n < ranges ? n : ranges);
    const int64_t j = (int64_t)b * a.Hkv + kvh;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int2 met = __ldcg(a.live + j);
    const int total = before + (empty ? 0 : met.y);
    const float *own = a.own + ((met.x + j) * a.G + g) * kPartialFloats;
    auto slot = [&](int s) {
        return s < before ? part + s * ((int64_t)2 * kShRows * kPartialFloats)
                          : own + (int64_t)(s - before) * a.G * kPartialFloats;
    };
    float M = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < total; s0 += 32) {
        float ms = -INFINITY, ls = 0.f;
        if (s0 + lane < total) {
            const float2 v = __ldcg(reinterpret_cast<const float2 *>(slot(s0 + lane)));
            ms = v.x;
            ls = v.y;
        }
        float4 x[kMergeDepth];
#pragma unroll
        for (int i = 0; i < kMergeDepth; ++i) {
            const int s = s0 + warp + kMergeWarps * i;
            x[i] = s < total ? __ldcg(reinterpret_cast<const float4 *>(slot(s) + 4) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float Mn = ms;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) Mn = fmaxf(Mn, __shfl_xor_sync(0xffffffffu, Mn, o));
        Mn = fmaxf(M, Mn);
        // (a slot without a finite score has the sum 0, or NaN, which shows)
        const float w = ms == -INFINITY ? 0.f : exp2f(ms - Mn);
        const float f = M == -INFINITY ? 0.f : exp2f(M - Mn);
        float lb = ms == -INFINITY ? ls : w * ls;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) lb += __shfl_xor_sync(0xffffffffu, lb, o);
        l = (M == -INFINITY ? l : l * f) + lb;
        M = Mn;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
        for (int i = 0; i < kMergeDepth; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, warp + kMergeWarps * i);
            acc = make_float4(fmaf(wi, x[i].x, acc.x), fmaf(wi, x[i].y, acc.y), fmaf(wi, x[i].z, acc.z),
                              fmaf(wi, x[i].w, acc.w));
        }
    }
    reinterpret_cast<float4 *>(accs[warp])[lane] = acc;
    __syncthreads();
    if (warp) return;
    const float lt = l;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kMergeWarps; ++i) {
        const float4 x = reinterpret_cast<const float4 *>(accs[i])[lane];
        v[0] += x.x;
        v[1] += x.y;
        v[2] += x.z;
        v[3] += x.w;
    }
    // o = D H (sums / l) / sqrt(128), 0 where nothing was seen (a NaN l, of a failed copy too, shows)
    const bool seen = lt > 0.f || lt != lt;
    const float inv = a.out_scale / lt;
    const float x0 = v[0] + v[1], x1 = v[0] - v[1], x2 = v[2] + v[3], x3 = v[2] - v[3];
    v[0] = x0 + x2;
    v[2] = x0 - x2;
    v[1] = x1 + x3;
    v[3] = x1 - x3;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float o = __shfl_xor_sync(0xffffffffu, v[k], m);
            v[k] = (lane & m) ? (o - v[k]) : (v[k] + o);
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int d = 4 * lane + k;
        v[k] = seen ? v[k] * inv : 0.f;
        if ((a.signs[d >> 5] >> (d & 31)) & 1u) v[k] = -v[k];
    }
    const int64_t at = (int64_t)blockIdx.x * kD + 4 * lane;
    if (a.out_dtype == TQ_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        uint32_t o[2];
        if (a.out_dtype == TQ_BF16) {
            const __nv_bfloat162 e = __floats2bfloat162_rn(v[0], v[1]), f = __floats2bfloat162_rn(v[2], v[3]);
            o[0] = *reinterpret_cast<const uint32_t *>(&e);
            o[1] = *reinterpret_cast<const uint32_t *>(&f);
        } else {
            const __half2 e = __floats2half2_rn(v[0], v[1]), f = __floats2half2_rn(v[2], v[3]);
            o[0] = *reinterpret_cast<const uint32_t *>(&e);
            o[1] = *reinterpret_cast<const uint32_t *>(&f);
        }
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.out) + 2 * at) = make_uint2(o[0], o[1]);
    }
}

// Ranges of the prefix: of all counts that give every CTA a tile, the one whose
// slowest SM is done first, a pair's CTA taking two units a tile, and about
// three for its start and end.  The counts tried for a shorter prefix are the
// first of a longer one's, so the last bounds the CTAs of both.
SharedPlan shared_plan(int sms, int B, int Hq, int Hkv, int P) {
    SharedPlan p;
    const int64_t rows = (int64_t)B * (Hq / Hkv);
    p.tiles = (int)((rows + kShRows - 1) / kShRows);
    p.pairs = p.tiles / 2;
    p.odd = p.tiles & 1;
    const int64_t n = ((int64_t)P + kShKeys - 1) / kShKeys;
    int64_t best = INT64_MAX;
    p.s2 = 1;
    p.most = 0;
    for (int64_t s = 1; s <= n && s <= 2 * (int64_t)sms; ++s) {
        const int64_t ctas = Hkv * (p.pairs * s + (p.pairs ? (s + 1) / 2 : s) * p.odd);
        const int64_t cost = (ctas + sms - 1) / sms * (3 + (p.pairs ? 2 : 1) * ((n + s - 1) / s));
        if (cost < best) {
            best = cost;
            p.s2 = (int)s;
        }
        p.most = (int)ctas;   // (grows with s)
        if (ctas > 4 * (int64_t)sms) break;
    }
    p.s1 = p.pairs ? (p.s2 + 1) / 2 : p.s2;
    p.per_head = p.pairs * p.s2 + p.odd * p.s1;
    p.ctas = Hkv * p.per_head;
    return p;
}

int64_t most_workers(int B, int Hkv, int T) {
    return min64((int64_t)B * Hkv * ((T + kMmaChunk - 1) / kMmaChunk), (int64_t)kMmaMaxWarpsPerSm * sm_count());
}

// Workspace: the prefix's partials | the own tokens' [W + B Hkv][G][132] | query fragments [B Hkv] | query tiles |
// segments' workers [B Hkv][2], in floats.  Room for p.most CTAs: what holds a
// prefix holds every shorter one.
struct Layout {
    int64_t own, frag, tiles, live, floats;
    Layout(const SharedPlan &p, int B, int Hq, int Hkv, int64_t W) {
        const int64_t segs = (int64_t)B * Hkv;
        own = (int64_t)p.most * 2 * kShRows * kPartialFloats;
        frag = own + (W + segs) * (Hq / Hkv) * kPartialFloats;
        tiles = (frag + segs * kFragWords + 3) & ~(int64_t)3;
        live = tiles + (int64_t)Hkv * p.tiles * (2 * 32768 / 4);
        floats = live + ((segs * 2 + 3) & ~(int64_t)3);
    }
};

bool shape_ok(int B, int Hq, int Hkv, int P, int T) {
    return B > 0 && Hq > 0 && Hkv > 0 && P > 0 && T > 0 && Hq % Hkv == 0;
}

// What the kernels' 32-bit indices hold.
bool size_ok(int B, int Hq, int Hkv, int P, int T) {
    return Hq / Hkv <= 8 && P <= kMmaMaxTokens && T <= kMmaMaxTokens && (int64_t)B * Hq <= (1 << 24) &&
           (int64_t)B * Hkv * ((T + kMmaChunk - 1) / kMmaChunk) <= 0x7FFFFFFF;
}

template <int KB, int VB>
int launch_shared(const SharedArgs &a, cudaStream_t st) {
    using S = ShSmem<KB, VB>;
    static int done[64] = {0};
    if (set_smem_limit((const void *)attn_shared_kernel<KB, VB>, S::kTotal, done) != TQ_OK) return TQ_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.plan.ctas);
    cfg.blockDim = dim3(kShThreads);
    cfg.dynamicSmemBytes = S::kTotal;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, attn_shared_kernel<KB, VB>, a));
}

template <int KB>
int launch_shared_v(const SharedArgs &a, int vb, cudaStream_t st) {
    return vb == 2 ? launch_shared<KB, 2>(a, st) : vb == 3 ? launch_shared<KB, 3>(a, st) : launch_shared<KB, 4>(a, st);
}

// The bytes from which levels16 takes a codebook's levels times f.
void level_bytes(const tq_codebook *cb, float f, uint32_t (&t)[4]) {
    for (int i = 0; i < 4; ++i) t[i] = 0;
    const int n = cb->bits == 4 ? 8 : cb->levels, from = cb->bits == 4 ? 8 : 0;
    for (int i = 0; i < n; ++i) {
        const __half h = __float2half_rn(cb->centroids[from + i] * f);
        uint16_t w;
        static_assert(sizeof(h) == sizeof(w), "fp16");
        __builtin_memcpy(&w, &h, 2);
        // 2 bits: word 0 high bytes, 1 low bytes; else words 0, 1 high bytes, 2, 3 low bytes
        t[i / 4] |= (uint32_t)(w >> 8) << (8 * (i % 4));
        t[(cb->bits == 2 ? 1 : 2) + i / 4] |= (uint32_t)(w & 255) << (8 * (i % 4));
    }
}

// The mirrored half of a 4-bit codebook is taken from the other.
bool symmetric(const tq_codebook *cb) {
    if (cb->bits != 4) return true;
    for (int i = 0; i < 8; ++i)
        if (!(cb->centroids[8 + i] > 0.f) || cb->centroids[7 - i] != -cb->centroids[8 + i]) return false;
    return true;
}

}  // namespace

int wait_failed_shared(unsigned *v, bool clear) { return read_wait_failed(v, clear); }

}  // namespace tq

using namespace tq;

extern "C" size_t tq_attn_shared_workspace_bytes(int B, int Hq, int Hkv, int P, int T) {
    if (!shape_ok(B, Hq, Hkv, P, T) || !size_ok(B, Hq, Hkv, P, T)) return 0;
    const SharedPlan p = shared_plan(sm_count(), B, Hq, Hkv, P);
    return (size_t)Layout(p, B, Hq, Hkv, most_workers(B, Hkv, T)).floats * sizeof(float);
}

extern "C" int tq_attn_decode_shared(const void *q, int q_dtype, const uint8_t *k_prefix, const uint8_t *v_prefix,
                                     const int32_t *prefix_table, int P_cap, int P, const int32_t *prefix_len,
                                     const uint8_t *k_blocks, const tq_codebook *kcb, const uint8_t *v_blocks,
                                     const tq_codebook *vcb, const int32_t *block_table, int64_t table_row_stride,
                                     int max_pages, int page_tokens, const int32_t *seq_lens, int B, int Hq, int Hkv,
                                     int T_cap, int T, float scale, tq_signs signs, void *out, int out_dtype,
                                     void *workspace, size_t workspace_bytes, void *stream) {
    if (!q || !k_prefix || !v_prefix || !k_blocks || !kcb || !v_blocks || !vcb || !out || !workspace) return TQ_ERR_ARG;
    if (!shape_ok(B, Hq, Hkv, P, T) || P > P_cap || !std::isfinite(scale)) return TQ_ERR_ARG;
    if (!prefix_table != !block_table) return TQ_ERR_ARG;
    const bool paged = block_table != nullptr;
    if (paged) {
        if (max_pages <= 0 || page_tokens <= 0 || (int64_t)max_pages * page_tokens < T ||
            table_row_stride < (B > 1 ? max_pages : 0) || table_row_stride > 0x7FFFFFFF)
            return TQ_ERR_ARG;
        if (page_tokens & 7) return TQ_ERR_UNSUPPORTED;
    } else if (T > T_cap || (T_cap & 7) || (P_cap & 7)) {
        return TQ_ERR_ARG;
    }
    if (!size_ok(B, Hq, Hkv, P, T)) return TQ_ERR_UNSUPPORTED;
    if (dtype_bytes(q_dtype) == 0 || dtype_bytes(out_dtype) == 0) return TQ_ERR_UNSUPPORTED;
    if (!codebook_ok(kcb) || !codebook_ok(vcb) || !symmetric(kcb) || !symmetric(vcb)) return TQ_ERR_UNSUPPORTED;
    if (!aligned(q, dtype_bytes(q_dtype)) || !aligned(k_prefix, 16) || !aligned(v_prefix, 16) ||
        !aligned(k_blocks, 16) || !aligned(v_blocks, 16) || !aligned(out, 16) || !aligned(workspace, 16) ||
        !aligned(prefix_table, 4) || !aligned(prefix_len, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4))
        return TQ_ERR_ALIGN;
    const SharedPlan sp = shared_plan(sm_count(), B, Hq, Hkv, P);
    const Layout at(sp, B, Hq, Hkv, most_workers(B, Hkv, T));
    if (workspace_bytes < (size_t)at.floats * sizeof(float)) return TQ_ERR_WORKSPACE;

    const int kb = kcb->bits, vb = vcb->bits, G = Hq / Hkv;
    MmaPlan plan = mma_plan(B, Hq, Hkv, T, kb, vb, false, G);
    float *ws = static_cast<float *>(workspace);
    plan.frag_off = at.frag - at.own;
    const float kf = attn_centroid_factor(kcb), vf = attn_centroid_factor(vcb);

    AttnArgs a = {};   // the own tokens
    a.drop = drop_copies();
    a.q = q;
    a.q_dtype = q_dtype;
    a.k = k_blocks;
    a.v = v_blocks;
    a.seq_lens = seq_lens;
    a.ws = ws + at.own;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = G;
    a.T_cap = paged ? (T + 7) & ~7 : T_cap;
    a.T = T;
    a.qscale = scale * 1.4426950408889634f;
    for (int i = 0; i < 16; ++i) {
        a.kc[i] = kcb->centroids[i];
        a.vc[i] = vcb->centroids[i] * vf;
    }
    for (int i = 0; i < 4; ++i) a.signs[i] = signs.w[i];
    a.table = block_table;
    a.max_pages = (int)table_row_stride;
    a.page = page_tokens;
    a.live = reinterpret_cast<int2 *>(ws + at.live);
    a.workers = plan.W;
    a.q_tiles = reinterpret_cast<uint8_t *>(ws + at.tiles);
    a.q_tile_count = sp.tiles;
    a.q_tile_bits = kb;

    SharedArgs s = {};
    s.q = a.q_tiles;
    s.k = k_prefix;
    s.v = v_prefix;
    s.table = prefix_table;
    s.len = prefix_len;
    s.part = ws;
    s.rows = B * G;
    s.Hkv = Hkv;
    s.P = P;
    s.cap = P_cap;
    s.page = page_tokens;
    s.plan = sp;
    s.k_norm = 1.f / kf;
    level_bytes(kcb, kf, s.kt);
    level_bytes(vcb, vf, s.vt);
    s.drop = a.drop;

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int r = launch_attn_prep_mma(a, plan, 0, st);
    if (r != TQ_OK) return r;
    const int nt = G <= 4 ? 1 : 2;
    r = kb == 2 ? launch_attn_mma_scores_k2(a, plan, vb, nt, paged, st)
                : kb == 3 ? launch_attn_mma_scores_k3(a, plan, vb, nt, paged, st)
                          : launch_attn_mma_scores_k4(a, plan, vb, nt, paged, st);
    if (r != TQ_OK) return r;
    r = kb == 2 ? launch_shared_v<2>(s, vb, st) : kb == 3 ? launch_shared_v<3>(s, vb, st) : launch_shared_v<4>(s, vb, st);
    if (r != TQ_OK) return r;

    MergeArgs m = {};
    m.part = s.part;
    m.own = a.ws;
    m.len = prefix_len;
    m.seq_lens = seq_lens;
    m.live = a.live;
    m.out = out;
    m.P = P;
    m.Hq = Hq;
    m.Hkv = Hkv;
    m.G = G;
    m.out_dtype = out_dtype;
    m.plan = sp;
    m.out_scale = 0.08838834764831845f / vf;
    for (int i = 0; i < 4; ++i) m.signs[i] = signs.w[i];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * Hq));
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, attn_shared_merge_kernel, m));
}
