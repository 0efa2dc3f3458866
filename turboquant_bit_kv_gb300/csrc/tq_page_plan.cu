// tq_page_plan: block tables, slots and positions of a serving step from its
// requests' lengths, on the GPU.
//
// Requests in order: c tokens cached, m new ones, h pages held.  A request
// needs max(0, ceil((c + m) / page) - h) pages and takes them from the end of
// the list of free ones while there are enough; the first that goes short, and
// all after it that need any, take none.  So the pages taken before a request
// are a running sum of needs, whoever is refused, and one scan over the
// requests settles it.  Then token i of a request sits in slot
// table[(c + i) / page] * Hkv * page + (c + i) % page.
//
// There is next to nothing to move (16 bytes a token, 24 a request): the call
// is launch, load latency and two scans.  One CTA does the requests, 1024 at a
// time, with their pages entered by all its threads; it does the tokens too
// where there are few (one launch), else a grid of its own does, launched as a
// programmatic dependent.
#include <cstdint>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kThreads = 1024;
constexpr int kTokenThreads = 256;
// Tokens that the requests' CTA does itself.
constexpr int64_t kFewTokens = 4096;

struct PlanArgs {
    const int32_t *cached, *fresh, *held, *free_pages, *free_count;
    const int64_t *pos_start;
    int32_t *table, *new_held, *new_count, *seq_lens, *tok_start;
    int64_t *dst, *pos;
    int64_t row, n_tok, most;    // row: of the table; most: tokens a row's pages hold
    int B, Hkv, page, max_pages, n_free;
};

// Inclusive sums of x over the CTA's threads, in order, and the sum of all.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t *warps, int64_t &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += v;
    }
    __syncthreads();   // (the sums of the scan before have been read)
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    int64_t s = warps[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += v;
    }
    all = __shfl_sync(0xffffffffu, s, 31);
    const int64_t before = __shfl_sync(0xffffffffu, s, (warp + 31) & 31);
    return x + (warp ? before : 0);
}

// First of the n ascending values that is above x (n if none is).
template <class T>
__device__ __forceinline__ int first_above(const T *v, int n, T x) {
    int lo = 0;
    while (n > 0) {
        const int half = n >> 1;
        if (v[lo + half] <= x) {
            lo += half + 1;
            n -= half + 1;
        } else {
            n = half;
        }
    }
    return lo;
}

// Slot and position of token n, token i of request b.
__device__ __forceinline__ void place(const PlanArgs &a, int64_t n, int b, int64_t i, int64_t c, bool ok) {
    const int64_t t = c + i, pg = t / a.page;
    a.dst[n] = ok ? (int64_t)a.table[b * a.row + pg] * a.Hkv * a.page + (t - pg * a.page) : -1;
    a.pos[n] = (a.pos_start ? a.pos_start[b] : c) + i;
}

__global__ void __launch_bounds__(kThreads) plan_requests_kernel(const __grid_constant__ PlanArgs a, int tokens_too) {
    __shared__ int64_t warps[32];
    __shared__ int64_t last_tok[kThreads], last_page[kThreads];   // past the request's last token / page taken
    __shared__ int64_t top;
    __shared__ int32_t held_s[kThreads], ok_s[kThreads], cached_s[kThreads];
    asm volatile("griddepcontrol.launch_dependents;");
    const int count = min(max(*a.free_count, 0), a.n_free);
    int64_t toks = 0, pages = 0, taken = 0;   // before this round's requests; pages: needed, taken: given
    if (threadIdx.x == 0) a.tok_start[0] = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        const bool live = b < a.B;
        const int32_t c = live ? max(a.cached[b], 0) : 0, m = live ? max(a.fresh[b], 0) : 0;
        const int32_t h = live ? min(max(a.held[b], 0), a.max_pages) : 0;
        const int64_t total = (int64_t)c + m;
        int64_t all;
        const int64_t end = toks + block_scan(m, warps, all);
        const bool fits = total <= a.most && end <= a.n_tok;
        const int64_t first = toks;
        toks += all;
        int64_t need = fits && m > 0 ? (total + a.page - 1) / a.page - h : 0;
        if (need < 0) need = 0;
        const int64_t upto = pages + block_scan(need, warps, all);
        const bool ok = fits && (need == 0 || upto <= count);
        pages += all;
        if (!ok) need = 0;
        last_tok[threadIdx.x] = end;
        last_page[threadIdx.x] = upto;
        held_s[threadIdx.x] = h;
        ok_s[threadIdx.x] = ok;
        cached_s[threadIdx.x] = c;
        if (threadIdx.x == 0) top = taken;
        __syncthreads();
        // sums only grow: those up to the list's length are the pages taken, the last of them all that are
        if (upto <= count && (threadIdx.x == kThreads - 1 || last_page[threadIdx.x + 1] > count)) top = upto;
        if (live) {
            a.tok_start[b + 1] = (int32_t)min64(end, 0x7FFFFFFF);
            a.new_held[b] = h + (int32_t)need;
            a.seq_lens[b] = ok ? (int32_t)total : c;
        }
        __syncthreads();
        const int64_t before = taken;
        taken = top;
        for (int64_t p = before + threadIdx.x; p < taken; p += kThreads) {
            const int r = first_above(last_page, kThreads, p);
            a.table[(b0 + r) * a.row + held_s[r] + (p - (r ? last_page[r - 1] : before))] = a.free_pages[count - 1 - p];
        }
        if (tokens_too) {
            __syncthreads();
            const int64_t stop = min64(toks, a.n_tok);
            for (int64_t n = first + threadIdx.x; n < stop; n += kThreads) {
                const int r = first_above(last_tok, kThreads, n);
                place(a, n, b0 + r, n - (r ? last_tok[r - 1] : first), cached_s[r], ok_s[r]);
            }
        }
    }
    if (threadIdx.x == 0) *a.new_count = count - (int32_t)taken;
    if (tokens_too) {
        for (int64_t n = toks + threadIdx.x; n < a.n_tok; n += kThreads) {
            a.dst[n] = -1;
            a.pos[n] = 0;
        }
    }
}

__global__ void __launch_bounds__(kTokenThreads) plan_tokens_kernel(const __grid_constant__ PlanArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t all = min64(a.tok_start[a.B], a.n_tok);
    const int64_t step = (int64_t)gridDim.x * kTokenThreads;
    for (int64_t n = (int64_t)blockIdx.x * kTokenThreads + threadIdx.x; n < a.n_tok; n += step) {
        if (n >= all) {
            a.dst[n] = -1;
            a.pos[n] = 0;
            continue;
        }
        const int b = first_above(a.tok_start + 1, a.B, (int32_t)n);
        const int64_t c = max(a.cached[b], 0);
        place(a, n, b, n - a.tok_start[b], c, a.seq_lens[b] == c + a.fresh[b]);
    }
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" int tq_page_plan(const int32_t *cached_lens, const int32_t *fresh_lens, const int64_t *pos_start, int B,
                            int Hkv, int page_tokens, int32_t *block_table, int64_t table_row_stride, int max_pages,
                            const int32_t *held, int32_t *new_held, const int32_t *free_pages, int n_free,
                            const int32_t *free_count, int32_t *new_free_count, int32_t *seq_lens, int32_t *tok_start,
                            int64_t *dst, int64_t *pos, int64_t n_tok, void *stream) {
    if (B <= 0 || Hkv <= 0 || page_tokens <= 0 || max_pages <= 0 || n_free < 0 || n_tok < 0) return TQ_ERR_ARG;
    if (!cached_lens || !fresh_lens || !block_table || !held || !new_held || !free_count || !new_free_count ||
        !seq_lens || !tok_start || (n_free && !free_pages) || (n_tok && (!dst || !pos)))
        return TQ_ERR_ARG;
    if (table_row_stride < (B > 1 ? max_pages : 0)) return TQ_ERR_ARG;
    // (new_held may be held, new_free_count free_count: they are read before they are written)
    const void *in[] = {cached_lens, fresh_lens, held, free_count, free_pages, pos_start};
    const void *out[] = {seq_lens, tok_start, dst, pos, block_table};
    for (const void *o : out)
        for (const void *i : in)
            if (o && o == i) return TQ_ERR_ARG;
    if (n_tok > 0x7FFFFFFF || B > (1 << 24)) return TQ_ERR_UNSUPPORTED;
    if (!aligned(cached_lens, 4) || !aligned(fresh_lens, 4) || !aligned(block_table, 4) || !aligned(held, 4) ||
        !aligned(new_held, 4) || !aligned(free_pages, 4) || !aligned(free_count, 4) || !aligned(new_free_count, 4) ||
        !aligned(seq_lens, 4) || !aligned(tok_start, 4) || !aligned(dst, 8) || !aligned(pos, 8) ||
        !aligned(pos_start, 8))
        return TQ_ERR_ALIGN;
    PlanArgs a;
    a.cached = cached_lens;
    a.fresh = fresh_lens;
    a.held = held;
    a.free_pages = free_pages;
    a.free_count = free_count;
    a.pos_start = pos_start;
    a.table = block_table;
    a.new_held = new_held;
    a.new_count = new_free_count;
    a.seq_lens = seq_lens;
    a.tok_start = tok_start;
    a.dst = dst;
    a.pos = pos;
    a.row = table_row_stride;
    a.n_tok = n_tok;
    const int64_t most = (int64_t)max_pages * page_tokens;
    a.most = most < 0x7FFFFFFF ? most : 0x7FFFFFFF;
    a.B = B;
    a.Hkv = Hkv;
    a.page = page_tokens;
    a.max_pages = max_pages;
    a.n_free = n_free;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool few = n_tok <= kFewTokens;
    plan_requests_kernel<<<1, kThreads, 0, st>>>(a, few ? 1 : 0);
    const int r = launch_status();
    if (r != TQ_OK || few) return r;
    const int64_t blocks = (n_tok + kTokenThreads - 1) / kTokenThreads, most_blocks = (int64_t)sm_count() * 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks < most_blocks ? blocks : most_blocks));
    cfg.blockDim = dim3(kTokenThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, plan_tokens_kernel, a));
}
