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
constexpr int kMaxCluster = 8;             // portable cluster size

// ---- selection
//
// Of the tokens that are not kept anyway (the first, the last), the m
// largest weights: three rounds of an 11-, 11- and 10-bit radix select on
// order-preserving keys find the m-th largest key K exactly, every CTA of the
// row adding up all the row's histograms by itself; then everything above K
// stays and, of the tokens equal to K, the ones of lowest index.  Weights are
// read from memory once (chunks beyond kSelCached keys are read again from
// L2) and the indices written once: 4 bytes in a token, 4 out a kept one.

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

struct SelShared {
    uint32_t hist[3][kBins];
    uint32_t part[kSelWarps];
    uint32_t found[3];             // digit of the m-th largest key, keys above it, total
    uint32_t above[kSelWarps], equal[kSelWarps];
    uint32_t sums[2];              // this CTA's kept-anyway or larger, and equal tokens
};

__device__ __forceinline__ uint32_t warp_sum(uint32_t v) { return __reduce_add_sync(0xffffffffu, v); }

__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ SelArgs a) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ SelShared s;
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
    const float *w = a.weights + row * a.row_stride;
    const int chunk = (L + C - 1) / C;
    const int lo = min(rank * chunk, L), n = min(L - lo, chunk);   // this CTA's tokens lo .. lo + n - 1
    const int first = a.first, last0 = L - a.last;                 // tokens first .. last0 - 1 are ranked
    const bool cached = n <= a.cached;
    auto key = [&](int i) { return cached ? keys[i] : weight_key(__ldg(w + lo + i)); };
    auto ranked = [&](int i) { return lo + i >= first && lo + i < last0; };

    for (int i = tid; i < 3 * kBins; i += kSelThreads) (&s.hist[0][0])[i] = 0;
    __syncthreads();
    // keys below a prefix mask: round r counts the digits of the keys whose higher digits match
    uint32_t prefix = 0, m = (uint32_t)(a.keep - a.first - a.last);   // the m-th largest is sought, m >= 1
    const bool none = m == 0;
    constexpr int shift[3] = {21, 10, 0};
    constexpr int width[3] = {11, 11, 10};
    if (!none) {
#pragma unroll
        for (int r = 0; r < 3; ++r) {
            const int steps = (n + kSelThreads - 1) / kSelThreads;
#pragma unroll 4
            for (int q = 0; q < steps; ++q) {
                const int i = q * kSelThreads + tid;
                bool in = i < n;
                uint32_t k = 0;
                if (in) {
                    if (r == 0) {
                        k = weight_key(__ldcs(w + lo + i));
                        if (cached) keys[i] = k;
                    } else {
                        k = key(i);
                    }
                    in = ranked(i) && (r == 0 || (k >> (shift[r] + width[r])) == prefix);
                }
                const uint32_t d = (k >> shift[r]) & ((1u << width[r]) - 1u);
                if (r > 0) {   // few keys share the higher digits
                    if (in) atomicAdd(&s.hist[r][d], 1u);
                    continue;
                }
                // one add for the lanes that share the first such lane's digit (ties and zeros are common)
                const uint32_t live = __ballot_sync(0xffffffffu, in);
                if (live) {
                    const uint32_t lead = __shfl_sync(0xffffffffu, d, __ffs(live) - 1);
                    const uint32_t same = __ballot_sync(0xffffffffu, in && d == lead);
                    if (lane == __ffs(live) - 1) atomicAdd(&s.hist[r][d], (uint32_t)__popc(same));
                    else if (in && d != lead) atomicAdd(&s.hist[r][d], 1u);
                }
            }
            cl.sync();
            // the row's histogram, from the top: thread t holds the bins of digits top - 2 t and top - 2 t - 1
            constexpr int kPer = kBins / kSelThreads;
            const int bins = 1 << width[r];
            uint32_t cnt[kPer] = {}, sum = 0;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const int at = bins - 1 - (tid * kPer + e);
                if (at >= 0) {
                    for (int p = 0; p < C; ++p) cnt[e] += cl.map_shared_rank(&s.hist[r][0], p)[at];
                }
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
            if (before < m && before + sum >= m) {   // exactly one thread
                uint32_t acc = before;
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    if (acc < m && acc + cnt[e] >= m) {
                        s.found[0] = (uint32_t)(bins - 1 - (tid * kPer + e));
                        s.found[1] = acc;
                    }
                    acc += cnt[e];
                }
            }
            __syncthreads();
            prefix = (prefix << width[r]) | s.found[0];
            m -= s.found[1];
            __syncthreads();
        }
    }
    // prefix: the threshold key; m: how many of the tokens equal to it stay (those of lowest index)
    // class of token i: kept anyway or larger (1), equal to the threshold (2), evicted (0)
    auto cls = [&](int i) -> int {
        if (!ranked(i)) return 1;
        if (none) return 0;
        const uint32_t k = key(i);
        return k > prefix ? 1 : (k == prefix ? 2 : 0);
    };
    // each warp takes a contiguous piece of the chunk, a multiple of 32 tokens
    const int piece = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int p0 = min(warp * piece, n), p1 = min(p0 + piece, n);
    uint32_t above = 0, equal = 0;
    for (int i = p0 + lane; i < p1; i += 32) {
        const int c = cls(i);
        above += c == 1;
        equal += c == 2;
    }
    above = warp_sum(above);
    equal = warp_sum(equal);
    if (lane == 0) {
        s.above[warp] = above;
        s.equal[warp] = equal;
    }
    __syncthreads();
    if (warp < 2) {
        const uint32_t t = warp_sum(warp == 0 ? s.above[lane] : s.equal[lane]);
        if (lane == 0) s.sums[warp] = t;
    }
    cl.sync();
    uint32_t na = 0, ne = 0;   // tokens of either class before this warp's piece
    for (int p = 0; p < rank; ++p) {
        const uint32_t *o = cl.map_shared_rank(&s.sums[0], p);
        na += o[0];
        ne += o[1];
    }
    static_assert(kSelWarps == 32, "a lane per warp");
    na += warp_sum(lane < warp ? s.above[lane] : 0u);
    ne += warp_sum(lane < warp ? s.equal[lane] : 0u);
    for (int i0 = p0; i0 < p1; i0 += 32) {
        const int i = i0 + lane;
        const int c = i < p1 ? cls(i) : 0;
        const uint32_t ma = __ballot_sync(0xffffffffu, c == 1), me = __ballot_sync(0xffffffffu, c == 2);
        const uint32_t under = (1u << lane) - 1u;
        const uint32_t ra = na + __popc(ma & under), re = ne + __popc(me & under);
        if (c == 1 || (c == 2 && re < m)) kept[ra + min(re, m)] = lo + i;
        na += __popc(ma);
        ne += __popc(me);
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
// eight blocks that starts and ends on a 16-byte boundary, its pieces put
// together from half words in shared memory.  Otherwise half words are
// read and written one by one.
constexpr int kMovThreads = 256;
constexpr int kMovSmem = 56 * 1024;        // four CTAs per SM: enough reads in flight
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

template <bool WIDE>
__global__ void __launch_bounds__(kMovThreads, 4) compact_kernel(const __grid_constant__ MovArgs a) {
    extern __shared__ __align__(16) uint8_t mov_smem[];
    int64_t *src = reinterpret_cast<int64_t *>(mov_smem);      // [tile] source slot
    int64_t *dst = src + a.tile;                               // [tile] own slot, -1: not in the pool
    uint8_t *stage0 = reinterpret_cast<uint8_t *>(dst + a.tile);
    float *sw = reinterpret_cast<float *>(stage0 + (size_t)a.tile * (a.pitch[0] + a.pitch[1]));
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int64_t row = blockIdx.x / C;
    const int b = (int)(row / a.Hkv), h = (int)(row % a.Hkv);
    const int32_t *kept = a.kept + row * a.keep;
    const int nl = a.new_lens[b];
    const int n = nl < 0 ? 0 : (nl > a.keep ? a.keep : (nl > a.T ? a.T : nl));
    float *w = a.weights ? a.weights + row * a.w_stride : nullptr;
    const int per = C * a.tile;
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
        const bool moves = cnt > 0 && kept[base + cnt - 1] != base + cnt - 1;
        if (moves) {
            for (int i = tid; i < cnt; i += kMovThreads) {
                const int j = base + i;
                int from = kept[j];
                if (from < j || from >= a.T) from = j;   // not a place to take from: it stays
                const int64_t own = slot(j);
                int64_t s = from == j ? own : slot(from);
                if (s < 0) {
                    s = own;
                    from = j;
                }
                src[i] = s;
                dst[i] = own;
                if (w) sw[i] = w[own < 0 ? j : from];
            }
            __syncthreads();
            uint8_t *stage = stage0;
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                const int bytes = a.bytes[side];
                if (bytes == 0) continue;
                const uint8_t *cache = a.blocks[side];
                if (WIDE) {
                    const int np = a.pieces[side], total = cnt * np;
                    for (int p0 = tid; p0 < total; p0 += 4 * kMovThreads) {
                        uint4 v[4];
                        int at[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int p = p0 + u * kMovThreads;
                            at[u] = -1;
                            if (p < total) {
                                const int i = div_by(p, a.inv_piece[side]), q = p - i * np;
                                const int64_t s = src[i];
                                if (s >= 0) {
                                    const int64_t first = s * bytes, piece = (first >> 4) + q;
                                    if (piece * 16 < first + bytes) {
                                        at[u] = i * a.pitch[side] + q * 16;
                                        v[u] = *reinterpret_cast<const uint4 *>(cache + piece * 16);
                                    }
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
                    for (int p = tid; p < total; p += kMovThreads) {
                        const int i = div_by(p, a.inv_half[side]), k = p - i * hw;
                        if (src[i] >= 0)
                            *reinterpret_cast<uint16_t *>(stage + i * a.pitch[side] + 2 * k) =
                                reinterpret_cast<const uint16_t *>(cache)[src[i] * hw + k];
                    }
                }
                stage += a.tile * a.pitch[side];
            }
        }
        cl.sync();   // every CTA has read its blocks of this step
        if (moves) {
            const uint8_t *stage = stage0;
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                const int bytes = a.bytes[side], hw = bytes / 2, pitch = a.pitch[side];
                if (bytes == 0) continue;
                uint8_t *cache = a.blocks[side];
                const int words = WIDE ? cnt * bytes / 16 : 0;   // whole 16-byte pieces of the tile
                for (int x = tid; x < words; x += kMovThreads) {
                    // piece x holds half words 8 x .. 8 x + 7 of the tile, of at most two blocks that matter
                    const int i = div_by(8 * x, a.inv_half[side]), k = 8 * x - i * hw;
                    const int o = (i & ~7);
                    uint32_t v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t e[2];
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            int ii = i, kk = k + 2 * q + z;
                            while (kk >= hw) {
                                kk -= hw;
                                ++ii;
                            }
                            const uint32_t skew = (uint32_t)(src[ii] * bytes) & 15u;
                            e[z] = *reinterpret_cast<const uint16_t *>(stage + ii * pitch + skew + 2 * kk);
                        }
                        v[q] = e[0] | (e[1] << 16);
                    }
                    if (dst[o] >= 0)
                        *reinterpret_cast<uint4 *>(cache + dst[o] * bytes + (int64_t)(8 * x - o * hw) * 2) =
                            make_uint4(v[0], v[1], v[2], v[3]);
                }
                const int total = cnt * hw;
                for (int p = words * 8 + tid; p < total; p += kMovThreads) {
                    const int i = div_by(p, a.inv_half[side]), k = p - i * hw;
                    const uint32_t skew = WIDE ? (uint32_t)(src[i] * bytes) & 15u : 0u;
                    if (dst[i] >= 0)
                        reinterpret_cast<uint16_t *>(cache)[dst[i] * hw + k] =
                            *reinterpret_cast<const uint16_t *>(stage + i * pitch + skew + 2 * k);
                }
                stage += a.tile * pitch;
            }
            if (w)
                for (int i = tid; i < cnt; i += kMovThreads) w[base + i] = sw[i];
            __syncthreads();   // the next step's blocks take this one's place
        }
    }
    // vacated slots start from zero again (all reads lie before the last meeting)
    if (w)
        for (int t = n + rank * kMovThreads + tid; t < a.T; t += C * kMovThreads) w[t] = 0.f;
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
    if (cudaLaunchKernelEx(&cfg, kernel, args) != cudaSuccess) {
        cudaGetLastError();
        return TQ_ERR_CUDA;
    }
    return launch_status();
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
    if (T > (1 << 30)) return TQ_ERR_UNSUPPORTED;
    if (seq_lens == new_lens) return TQ_ERR_ARG;   // other rows still read the old lengths
    if (!aligned(weights, 4) || !aligned(kept, 4) || !aligned(new_lens, 4) || !aligned(seq_lens, 4)) return TQ_ERR_ALIGN;
    const int64_t rows = (int64_t)B * Hkv;
    // CTAs per row: a chunk of at most kSelChunk keys each; while SMs would stay idle, of 8192
    int C = 1;
    while (C < kMaxCluster &&
           ((T + C - 1) / C > kSelChunk || (rows * C * 2 <= sm_count() && (T + C - 1) / C > 8192)))
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
    const bool wide = aligned(k_blocks, 16) && aligned(v_blocks, 16) && ((block_table ? page_tokens : T_cap) & 7) == 0;
    const int bytes[2] = {k_block_bytes, vbytes};
    auto inverse = [](int n) { return n < 2 ? 0u : (uint32_t)(((1ull << 32) + n - 1) / n); };
    int token = 2 * 8 + 4;   // shared memory of a token
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
    // CTAs per row: while the GPU holds more (four per SM) and each still gets 64 tokens
    int C = 1;
    while (C < kMaxCluster && rows * C < 4 * (int64_t)sm_count() && m > C * 64) C *= 2;
    // tokens of a CTA and step: the shared memory's worth at most, the steps of equal size, groups of eight
    const int most = (kMovSmem / token) & ~7;
    const int steps = (m + C * most - 1) / (C * most);
    a.tile = ((m + C * steps - 1) / (C * steps) + 7) & ~7;
    const size_t smem = (size_t)a.tile * token;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    static int done[2][64] = {{0}};
    if (wide) {
        if (set_smem_limit((const void *)compact_kernel<true>, kMovSmem, done[0]) != TQ_OK) return TQ_ERR_CUDA;
        return launch_cluster(compact_kernel<true>, rows, C, kMovThreads, smem, st, a);
    }
    if (set_smem_limit((const void *)compact_kernel<false>, kMovSmem, done[1]) != TQ_OK) return TQ_ERR_CUDA;
    return launch_cluster(compact_kernel<false>, rows, C, kMovThreads, smem, st, a);
}
