// Eviction from a packed cache by accumulated attention weight:
// tq_evict_select picks the tokens of each (sequence, KV head) that stay,
// tq_evict_compact moves their blocks and weights together in place.
//
// Both run a thread-block cluster per (sequence, KV head) row, its CTAs
// sharing the row's tokens: rows are few (8 for one sequence of 8 KV heads),
// the GPU has 152 SMs, and the steps between which a row has to agree
// (histograms, "everybody has read") are then cluster barriers instead of
// kernel boundaries or spins on memory.
#include <cooperative_groups.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace cg = cooperative_groups;

namespace tq {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kSelCached = 40 * 1024;      // keys of a CTA's chunk held in shared memory (160 KB)
constexpr int kSelChunk = 20 * 1024;       // keys a CTA gets before a row takes more CTAs
constexpr int kSelLeast = 8192;           // (while SMs would stay idle)
constexpr int kMaxCluster = 8;             // portable cluster size

// ---- selection
//
// Of the tokens that are not kept anyway (the first, the last), the m largest
// weights.  On order-preserving keys, a histogram of the top 11 bits finds the
// bin that the m-th largest key lies in; a second pass over the keys counts what lies in
// higher bins and lists the keys of that bin, and two more rounds of 11 and 10
// bits over the list find the m-th largest key K itself.  Everything above K
// stays and, of the tokens equal to K, the ones of lowest index: each warp has a
// contiguous piece of the row's tokens and knows how many stay before it, so a
// last pass writes the indices in order.  Weights are read from memory once
// (chunks beyond kSelCached keys are read again from L2) and the indices
// written once: 4 bytes in a token, 4 out a kept one.  What bounds it is what
// every CTA does whatever its keys (three histograms cleared, searched and
// merged, the cluster's meetings) and the latency of one key per lane and
// iteration: 256 rows of up to 32769 tokens, 2.8 million keys in the 108 that
// have more than 16384, take 16.7 million warp instructions, 190 per 32 keys.

// Key of a weight: ascending with it as unsigned integers, -0 equal to +0,
// every NaN above +inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(w + 0.f);   // -0 + 0 = +0
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

struct SelArgs {
    const float *weights;
    const int32_t *seq_lens;
    int32_t *kept, *new_lens;
    int64_t row_stride;
    int Hkv, T, keep, first, last, cached;   // cached: shared-memory keys of a CTA (0: none)
};

constexpr int kSelList = 4096;     // keys of the threshold's bin that a CTA can list

struct SelShared {
    uint32_t hist[3][kBins];
    uint32_t key[kSelList];        // listed keys, and the warps whose pieces they are of
    uint8_t of[kSelList];
    uint32_t part[kSelWarps];
    uint32_t found[2];             // digit of the m-th largest key, keys above it
    uint32_t above[kSelWarps], equal[kSelWarps];   // per warp's piece
    uint32_t sums[2];              // this CTA's larger and equal tokens
    uint32_t listed;
};

__device__ __forceinline__ uint32_t warp_sum(uint32_t v) { return __reduce_add_sync(0xffffffffu, v); }

// The digit (of WIDTH bits) that the m-th largest key has and how many keys
// have larger ones, from the row's histograms hist of all its CTAs: each adds
// its bins that are not empty to the first CTA's, and all read those.
template <int WIDTH>
__device__ __forceinline__ void find_digit(cg::cluster_group &cl, SelShared &s, uint32_t *hist, uint32_t &m,
                                           uint32_t &prefix) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kNum = 1 << WIDTH, kPer = kNum / kSelThreads;
    // thread t holds the bins of digits kNum - 1 - kPer t downwards
    uint32_t *all = cl.map_shared_rank(hist, 0);
    if (cl.num_blocks() > 1) {
        __syncthreads();
        if (cl.block_rank() > 0) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const int at = kNum - 1 - (tid * kPer + e);
                if (hist[at]) atomicAdd(all + at, hist[at]);
            }
        }
    }
    cl.sync();
    uint32_t cnt[kPer], sum = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        cnt[e] = all[kNum - 1 - (tid * kPer + e)];
        sum += cnt[e];
    }
    uint32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) s.part[warp] = inc;
    __syncthreads();
    uint32_t before = inc - sum + warp_sum(lane < warp ? s.part[lane] : 0u);
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        if (before < m && before + cnt[e] >= m) {   // exactly one bin
            s.found[0] = (uint32_t)(kNum - 1 - (tid * kPer + e));
            s.found[1] = before;
        }
        before += cnt[e];
    }
    __syncthreads();
    prefix = (prefix << WIDTH) | s.found[0];
    m -= s.found[1];
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ SelArgs a) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ SelShared s;
    static_assert(kSelWarps == 32 && kSelThreads == 1024, "a lane per warp, a thread per bin of 10 bits");
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int64_t row = blockIdx.x / C;
    const int b = (int)(row / a.Hkv);
    int L = a.T;
    if (a.seq_lens) {
        const int sl = a.seq_lens[b];
        L = sl < 0 ? 0 : (sl > a.T ? a.T : sl);
    }
    int32_t *kept = a.kept + row * a.keep;
    if (row % a.Hkv == 0 && rank == 0 && tid == 0) a.new_lens[b] = L < a.keep ? L : a.keep;
    if (L <= a.keep) {   // (the whole cluster)
        for (int i = rank * kSelThreads + tid; i < a.keep; i += C * kSelThreads) kept[i] = i < L ? i : -1;
        return;
    }
    // kept anyway: the first and the last tokens
    for (int i = rank * kSelThreads + tid; i < a.first; i += C * kSelThreads) kept[i] = i;
    for (int i = rank * kSelThreads + tid; i < a.last; i += C * kSelThreads) kept[a.keep - a.last + i] = L - a.last + i;
    uint32_t m = (uint32_t)(a.keep - a.first - a.last);   // to find among the others
    if (m == 0) return;
    kept += a.first;
    // the others: tokens a.first + 0 .. R - 1, this CTA's lo .. lo + n - 1 of them, this warp's p0 .. p1 - 1
    // of those (a multiple of 32 each)
    const int R = L - a.first - a.last;
    const int chunk = (R + C - 1) / C, lo = min(rank * chunk, R), n = min(R - lo, chunk);
    const float *w = a.weights + row * a.row_stride + a.first + lo;
    const bool cached = n <= a.cached;
    const int piece = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int p0 = min(warp * piece, n), p1 = min(p0 + piece, n);

    for (int i = tid; i < 3 * kBins; i += kSelThreads) (&s.hist[0][0])[i] = 0;
    if (tid == 0) s.listed = 0;
    cl.sync();   // (the first CTA's bins are empty before the others add to them)
    // pass 1: keys, and the histogram of their top 11 bits
#pragma unroll 8
    for (int i0 = p0; i0 < p1; i0 += 32) {
        const int i = i0 + lane;
        const bool in = i < p1;
        const uint32_t k = in ? weight_key(__ldcs(w + i)) : 0;
        if (in && cached) keys[i] = k;
        // one add for the lanes that share the first lane's digit (ties and zeros are common)
        const uint32_t d = k >> 21, lead = __shfl_sync(0xffffffffu, d, 0);
        const uint32_t same = __ballot_sync(0xffffffffu, in && d == lead);
        if (lane == 0) atomicAdd(&s.hist[0][d], (uint32_t)__popc(same));
        else if (in && d != lead) atomicAdd(&s.hist[0][d], 1u);
    }
    uint32_t prefix = 0;
    find_digit<11>(cl, s, s.hist[0], m, prefix);
    // pass 2: keys of higher bins counted, those of the bin listed and their next digit counted
    const uint32_t top = prefix;
    uint32_t above = 0;
#pragma unroll 4
    for (int i0 = p0; i0 < p1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < p1 ? (cached ? keys[i] : weight_key(__ldg(w + i))) : 0;
        above += (k >> 21) > top;
        if (i < p1 && (k >> 21) == top) {
            const uint32_t at = atomicAdd(&s.listed, 1u);
            if (at < kSelList) {
                s.key[at] = k;
                s.of[at] = (uint8_t)warp;
            }
            atomicAdd(&s.hist[1][(k >> 10) & 2047u], 1u);
        }
    }
    above = warp_sum(above);
    if (lane == 0) {
        s.above[warp] = above;
        s.equal[warp] = 0;
    }
    find_digit<11>(cl, s, s.hist[1], m, prefix);
    // the last digit, over the list, or over the keys again where they did not fit
    const uint32_t listed = s.listed;
    const bool fits = listed <= kSelList;
    auto key = [&](int i) { return cached ? keys[i] : weight_key(__ldg(w + i)); };
    if (fits) {
        for (uint32_t i = tid; i < listed; i += kSelThreads)
            if ((s.key[i] >> 10) == prefix) atomicAdd(&s.hist[2][s.key[i] & 1023u], 1u);
    } else {
        for (int i = p0 + lane; i < p1; i += 32)
            if ((key(i) >> 10) == prefix) atomicAdd(&s.hist[2][key(i) & 1023u], 1u);
    }
    find_digit<10>(cl, s, s.hist[2], m, prefix);
    // prefix: the threshold key; m: how many of the tokens equal to it stay.  The bin's keys by piece:
    if (fits) {
        for (uint32_t i = tid; i < listed; i += kSelThreads) {
            const uint32_t k = s.key[i];
            if (k > prefix) atomicAdd(&s.above[s.of[i]], 1u);
            else if (k == prefix) atomicAdd(&s.equal[s.of[i]], 1u);
        }
    } else {
        uint32_t more = 0, equal = 0;
        for (int i = p0 + lane; i < p1; i += 32) {
            const uint32_t k = key(i);
            more += k > prefix && (k >> 21) == top;
            equal += k == prefix;
        }
        more = warp_sum(more);
        equal = warp_sum(equal);
        if (lane == 0) {
            s.above[warp] += more;
            s.equal[warp] = equal;
        }
    }
    __syncthreads();
    if (warp < 2) {
        const uint32_t t = warp_sum(warp == 0 ? s.above[lane] : s.equal[lane]);
        if (lane == 0) s.sums[warp] = t;
    }
    cl.sync();
    uint32_t na = 0, ne = 0;   // larger and equal tokens before this warp's piece
    for (int p = 0; p < rank; ++p) {
        const uint32_t *o = cl.map_shared_rank(&s.sums[0], p);
        na += o[0];
        ne += o[1];
    }
    na += warp_sum(lane < warp ? s.above[lane] : 0u);
    ne += warp_sum(lane < warp ? s.equal[lane] : 0u);
    const uint32_t under = (1u << lane) - 1u;
    const int token0 = a.first + lo;
#pragma unroll 4
    for (int i0 = p0; i0 < p1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < p1 ? key(i) : 0;
        const bool eq = k == prefix && i < p1;
        const uint32_t ma = __ballot_sync(0xffffffffu, k > prefix), me = __ballot_sync(0xffffffffu, eq);
        const uint32_t ra = na + __popc(ma & under);
        if (me == 0) {
            if (k > prefix) kept[ra + min(ne, m)] = token0 + i;
        } else {
            const uint32_t re = ne + __popc(me & under);
            if (k > prefix || (eq && re < m)) kept[ra + min(re, m)] = token0 + i;
            ne += __popc(me);
        }
        na += __popc(ma);
    }
    cl.sync();   // no CTA leaves while others still read its sums
}

// ---- compaction
//
// Token j of a row takes the block of token kept[j] >= j (ascending), in
// place.  The row goes by in steps of (CTAs x tile) tokens: a step's blocks
// are read into shared memory, the cluster meets, and the step's blocks are
// written.  A block that a step writes lies at or below every source of the
// following steps (kept[j] >= j), so the only order to keep is "all reads of
// a step before its writes".  Every kept block is read once and written once;
// tiles in which nothing moves are left alone.
//
// Blocks of 34, 50, 66 ... bytes start at any even address.  WIDE (cache and
// pages multiples of 8 tokens, so that eight blocks are a multiple of 16
// bytes; aligned bases): a block is read as the aligned 16-byte pieces that
// it lies in, with the bytes around it, and written as part of a group of
// eight blocks that starts and ends on a 16-byte boundary, its 16-byte pieces
// put together from the aligned words around them in shared memory.  Otherwise
// (and for blocks below 16 bytes) half words are read and written one by one.
constexpr int kMovThreads = 1024;          // of a CTA that has an SM to itself; 256 where four share one
constexpr int kMovSmem = 56 * 1024;        // shared memory of a CTA of 256 threads
constexpr int kMovMaxBytes = 512;          // of a block

struct MovArgs {
    uint8_t *blocks[2];
    float *weights;
    const int32_t *kept, *new_lens, *table;
    int64_t w_stride;
    int bytes[2];                          // of a block (0: no such cache)
    int pieces[2];                         // 16-byte pieces that a block may lie in
    int pitch[2];                          // shared-memory bytes of a token
    uint32_t inv_half[2], inv_piece[2];    // ceil(2^32 / n) of the half words of a block, the pieces
    int Hkv, T, T_cap, keep, max_pages, page, num_pages, tile;
};

__device__ __forceinline__ int div_by(uint32_t p, uint32_t inv) { return inv ? (int)__umulhi(p, inv) : (int)p; }

// 16 bytes at a 2-byte aligned shared-memory address.
__device__ __forceinline__ void lds16_a2(const uint8_t *p, uint32_t (&v)[4]) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(p);
    const uint32_t *w = reinterpret_cast<const uint32_t *>(p - (at & 2u));
    const uint32_t sh = (at & 2u) * 8u;
    uint32_t x[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) x[i] = w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __funnelshift_r(x[i], x[i + 1], sh);
}

template <bool WIDE>
__global__ void __launch_bounds__(kMovThreads, 1) compact_kernel(const __grid_constant__ MovArgs a) {
    extern __shared__ __align__(16) uint8_t mov_smem[];
    int64_t *src = reinterpret_cast<int64_t *>(mov_smem);      // [tile] source slot
    int64_t *dst = src + a.tile;                               // [tile] own slot, -1: not in the pool
    uint8_t *stage0 = reinterpret_cast<uint8_t *>(dst + a.tile);
    float *sw = reinterpret_cast<float *>(stage0 + (size_t)a.tile * (a.pitch[0] + a.pitch[1]));
    uint32_t *place = reinterpret_cast<uint32_t *>(sw + a.tile);   // [2][tile] where a token's block starts in the stage
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, threads = blockDim.x, C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int64_t row = blockIdx.x / C;
    const int b = (int)(row / a.Hkv), h = (int)(row % a.Hkv);
    const int32_t *kept = a.kept + row * a.keep;
    const int per = C * a.tile;
    // this thread's first index of a step, requested one step ahead (the first along with the length)
    auto index_at = [&](int j) { return j < a.keep ? kept[j] : 0; };
    int ahead = index_at(rank * a.tile + tid);
    const int nl = a.new_lens[b];
    const int n = nl < 0 ? 0 : (nl > a.keep ? a.keep : (nl > a.T ? a.T : nl));
    float *w = a.weights ? a.weights + row * a.w_stride : nullptr;
    // ascending indices that end where they would without a gap: nothing moves
    const int steps = n == 0 || kept[n - 1] == n - 1 ? 0 : (n + per - 1) / per;

    auto slot = [&](int t) -> int64_t {
        if (!a.table) return row * a.T_cap + t;
        const int pg = t / a.page;
        const int id = a.table[(int64_t)b * a.max_pages + pg];
        if (id < 0 || id >= a.num_pages) return -1;
        return ((int64_t)id * a.Hkv + h) * a.page + (t - pg * a.page);
    };
    for (int t = 0; t < steps; ++t) {
        const int base = t * per + rank * a.tile;
        const int cnt = max(0, min(a.tile, n - base));
        const bool moves = cnt > 0 && kept[base + cnt - 1] != base + cnt - 1;   // (a step in which nothing moves)
        if (moves) {
            for (int i = tid; i < cnt; i += threads) {
                const int j = base + i;
                int from = i == tid ? ahead : kept[j];
                if (from < j || from >= a.T) from = j;   // not a place to take from: it stays
                const int64_t own = slot(j);
                int64_t s = from == j ? own : slot(from);
                if (s < 0) {
                    s = own;
                    from = j;
                }
                src[i] = s;
                dst[i] = own;
#pragma unroll
                for (int side = 0; side < 2; ++side)
                    place[side * a.tile + i] =
                        (uint32_t)(i * a.pitch[side] + (WIDE ? (int)((uint32_t)s * (uint32_t)a.bytes[side] & 15u) : 0));
                reinterpret_cast<int *>(sw)[i] = own < 0 ? j : from;   // (its weight: once the blocks are requested)
            }
            ahead = index_at(base + per + tid);
            __syncthreads();
            uint8_t *stage = stage0;
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                const int bytes = a.bytes[side];
                if (bytes == 0) continue;
                const uint8_t *cache = a.blocks[side];
                if (WIDE) {
                    const int np = a.pieces[side], total = cnt * np;
                    for (int p0 = tid; p0 < total; p0 += 4 * threads) {
                        uint4 v[4];
                        int at[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int p = p0 + u * threads;
                            at[u] = -1;
                            if (p < total) {
                                const int i = div_by(p, a.inv_piece[side]), q = p - i * np;
                                const int64_t s = src[i], first = s * bytes;
                                const int skew = (int)(first & 15);
                                if (s >= 0 && q * 16 < skew + bytes) {
                                    at[u] = i * a.pitch[side] + q * 16;
                                    v[u] = *reinterpret_cast<const uint4 *>(cache + (first - skew) + q * 16);
                                }
                            }
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            if (at[u] >= 0) *reinterpret_cast<uint4 *>(stage + at[u]) = v[u];
                    }
                } else {
                    const int hw = bytes / 2, total = cnt * hw;
#pragma unroll 8
                    for (int p = tid; p < total; p += threads) {
                        const int i = div_by(p, a.inv_half[side]), k = p - i * hw;
                        if (src[i] >= 0)
                            *reinterpret_cast<uint16_t *>(stage + i * a.pitch[side] + 2 * k) =
                                reinterpret_cast<const uint16_t *>(cache)[src[i] * hw + k];
                    }
                }
                stage += a.tile * a.pitch[side];
            }
            if (w)
                for (int i = tid; i < cnt; i += threads) sw[i] = w[reinterpret_cast<const int *>(sw)[i]];
        } else {
            ahead = index_at(base + per + tid);
        }
        cl.sync();   // every CTA has read its blocks of this step
        if (moves) {
            const uint8_t *stage = stage0;
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                const int bytes = a.bytes[side], hw = bytes / 2;
                if (bytes == 0) continue;
                uint8_t *cache = a.blocks[side];
                const uint32_t *at = place + side * a.tile;
                const int words = WIDE ? cnt * bytes / 16 : 0;   // whole 16-byte pieces of the tile
                for (int x = tid; x < words; x += threads) {
                    // piece x: half words 8 x .. 8 x + 7 of the tile, of block i from its k-th on, the last
                    // 8 - r of them perhaps of the next block (blocks have 8 at least)
                    const int i = div_by(8 * x, a.inv_half[side]), k = 8 * x - i * hw, r = hw - k, o = i & ~7;
                    uint32_t v[4];
                    lds16_a2(stage + at[i] + 2 * k, v);
                    if (r < 8) {
                        uint32_t u[4];
                        lds16_a2(stage + at[i + 1] - 2 * r, u);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            v[q] = 2 * q >= r ? u[q] : (2 * q + 1 >= r ? (v[q] & 0xFFFFu) | (u[q] & 0xFFFF0000u) : v[q]);
                    }
                    if (dst[o] >= 0)
                        *reinterpret_cast<uint4 *>(cache + dst[o] * bytes + (8 * x - o * hw) * 2) =
                            make_uint4(v[0], v[1], v[2], v[3]);
                }
                const int total = cnt * hw;
                for (int p = words * 8 + tid; p < total; p += threads) {
                    const int i = div_by(p, a.inv_half[side]), k = p - i * hw;
                    if (dst[i] >= 0)
                        reinterpret_cast<uint16_t *>(cache)[dst[i] * hw + k] =
                            *reinterpret_cast<const uint16_t *>(stage + at[i] + 2 * k);
                }
                stage += a.tile * a.pitch[side];
            }
            if (w)
                for (int i = tid; i < cnt; i += threads) w[base + i] = sw[i];
            __syncthreads();   // the next step's blocks take this one's place
        }
    }
    // vacated slots start from zero again (all reads lie before the last meeting)
    if (w)
        for (int t = n + rank * threads + tid; t < a.T; t += C * threads) w[t] = 0.f;
}

template <class K, class A>
int launch_cluster(K kernel, int64_t rows, int C, int threads, size_t smem, cudaStream_t st, const A &args) {
    if (rows * C > 0x7FFFFFFF) return TQ_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, kernel, args));
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" int tq_evict_select(const float *weights, int64_t row_stride, const int32_t *seq_lens, int B, int Hkv, int T,
                               int keep, int first, int last, int32_t *kept, int32_t *new_lens, void *stream) {
    if (!weights || !kept || !new_lens) return TQ_ERR_ARG;
    if (B <= 0 || Hkv <= 0 || T < 1 || keep < 1 || first < 0 || last < 0 || (int64_t)first + last > keep ||
        row_stride < T)
        return TQ_ERR_ARG;
    if (T > (1 << 30) || keep > (1 << 30)) return TQ_ERR_UNSUPPORTED;   // (indices plus a cluster's threads fit int)
    if (seq_lens == new_lens) return TQ_ERR_ARG;   // other rows still read the old lengths
    if (!aligned(weights, 4) || !aligned(kept, 4) || !aligned(new_lens, 4) || !aligned(seq_lens, 4)) return TQ_ERR_ALIGN;
    const int64_t rows = (int64_t)B * Hkv;
    // CTAs per row: a chunk of at most kSelChunk keys each; while SMs would stay idle, of kSelLeast.  (A
    // cluster's meetings cost more than its CTAs save: 256 rows of 32769 take 30 us with two CTAs a row,
    // 42 with four, 87 with eight.)
    int C = 1;
    while (C < kMaxCluster &&
           ((T + C - 1) / C > kSelChunk || (rows * C * 2 <= sm_count() && (T + C - 1) / C > kSelLeast)))
        C *= 2;
    const int chunk = (T + C - 1) / C;
    SelArgs a;
    a.weights = weights;
    a.seq_lens = seq_lens;
    a.kept = kept;
    a.new_lens = new_lens;
    a.row_stride = row_stride;
    a.Hkv = Hkv;
    a.T = T;
    a.keep = keep;
    a.first = first;
    a.last = last;
    a.cached = chunk <= kSelCached ? chunk : 0;
    const size_t smem = (size_t)a.cached * 4;
    static int done[64] = {0};
    if (set_smem_limit((const void *)select_kernel, kSelCached * 4, done) != TQ_OK) return TQ_ERR_CUDA;
    return launch_cluster(select_kernel, rows, C, kSelThreads, smem, static_cast<cudaStream_t>(stream), a);
}

extern "C" int tq_evict_compact(uint8_t *k_blocks, int k_block_bytes, uint8_t *v_blocks, int v_block_bytes,
                                float *weights, int64_t weights_row_stride, const int32_t *kept, int keep,
                                const int32_t *new_lens, const int32_t *block_table, int max_pages, int page_tokens,
                                int num_pages, int B, int Hkv, int T_cap, int T, void *stream) {
    if (!k_blocks || !kept || !new_lens) return TQ_ERR_ARG;
    if (B <= 0 || Hkv <= 0 || T < 1 || keep < 1 || k_block_bytes <= 0 || (v_blocks && v_block_bytes <= 0))
        return TQ_ERR_ARG;
    if (weights && weights_row_stride < T) return TQ_ERR_ARG;
    if (T > (1 << 30)) return TQ_ERR_UNSUPPORTED;
    if (block_table) {
        if (max_pages <= 0 || page_tokens <= 0 || num_pages <= 0 || (int64_t)max_pages * page_tokens < T) return TQ_ERR_ARG;
    } else if (T > T_cap) {
        return TQ_ERR_ARG;
    }
    const int vbytes = v_blocks ? v_block_bytes : 0;
    if ((k_block_bytes & 1) || (vbytes & 1)) return TQ_ERR_ALIGN;
    if (k_block_bytes > kMovMaxBytes || vbytes > kMovMaxBytes) return TQ_ERR_UNSUPPORTED;
    if (!aligned(k_blocks, 2) || !aligned(v_blocks, 2) || !aligned(weights, 4) || !aligned(kept, 4) ||
        !aligned(new_lens, 4) || !aligned(block_table, 4))
        return TQ_ERR_ALIGN;
    MovArgs a;
    a.blocks[0] = k_blocks;
    a.blocks[1] = v_blocks;
    a.weights = weights;
    a.kept = kept;
    a.new_lens = new_lens;
    a.table = block_table;
    a.w_stride = weights_row_stride;
    const bool wide = aligned(k_blocks, 16) && aligned(v_blocks, 16) && ((block_table ? page_tokens : T_cap) & 7) == 0 &&
                      k_block_bytes >= 16 && (vbytes == 0 || vbytes >= 16);
    const int bytes[2] = {k_block_bytes, vbytes};
    auto inverse = [](int n) { return n < 2 ? 0u : (uint32_t)(((1ull << 32) + n - 1) / n); };
    int token = 2 * 8 + 4 + 2 * 4;   // shared memory of a token
    for (int i = 0; i < 2; ++i) {
        a.bytes[i] = bytes[i];
        a.pieces[i] = bytes[i] ? (bytes[i] + 14 + 15) / 16 : 0;
        a.pitch[i] = wide ? a.pieces[i] * 16 : bytes[i];
        a.inv_half[i] = inverse(bytes[i] / 2);
        a.inv_piece[i] = inverse(a.pieces[i]);
        token += a.pitch[i];
    }
    a.Hkv = Hkv;
    a.T = T;
    a.T_cap = T_cap;
    a.keep = keep;
    a.max_pages = max_pages;
    a.page = page_tokens;
    a.num_pages = num_pages;
    const int64_t rows = (int64_t)B * Hkv;
    const int m = keep < T ? keep : T;
    // CTAs per row: doubled while there are fewer than the GPU holds (four per SM; the last doubling may pass that,
    // 128 rows get 1024 CTAs for 608 places) and each still gets 64 tokens.  Few CTAs take an SM's shared memory and
    // threads each, so that a row goes by in few steps (2 rows of 29281 to 22908: 66 us in eight steps, 29 in two)
    int C = 1;
    while (C < kMaxCluster && rows * C < 4 * (int64_t)sm_count() && m > C * 64) C *= 2;
    int share = 4;   // CTAs per SM
    while (share > 1 && rows * C * 2 <= (int64_t)sm_count() * share) share /= 2;
    // tokens of a CTA and step: the shared memory's worth at most, the steps of equal size, groups of eight
    const int most = (kMovSmem * (4 / share) / token) & ~7;
    const int steps = (m + C * most - 1) / (C * most);
    a.tile = ((m + C * steps - 1) / (C * steps) + 7) & ~7;
    const size_t smem = (size_t)a.tile * token;
    const int threads = kMovThreads / share;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    static int done[2][64] = {{0}};
    if (wide) {
        if (set_smem_limit((const void *)compact_kernel<true>, 4 * kMovSmem, done[0]) != TQ_OK) return TQ_ERR_CUDA;
        return launch_cluster(compact_kernel<true>, rows, C, threads, smem, st, a);
    }
    if (set_smem_limit((const void *)compact_kernel<false>, 4 * kMovSmem, done[1]) != TQ_OK) return TQ_ERR_CUDA;
    return launch_cluster(compact_kernel<false>, rows, C, threads, smem, st, a);
}
