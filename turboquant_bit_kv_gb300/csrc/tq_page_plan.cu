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
// is launch, load latency and scans.  So every CTA scans all requests, 1024 at a
// time, and places the tokens of its own range: a page that its request has just
// taken is known from the scan, and entered by the request's first token in it.
// Few tokens are one CTA's.  With more, no CTA may write what another still
// reads: where the state is updated in place (new_held is held, or
// new_free_count free_count), a second launch of one CTA, a programmatic
// dependent that has scanned by the time the first is done, writes those two;
// else the first CTA does (257 requests of 12001 tokens 4.2 us, in place 4.75; 512
// of 196496 5.3 and 6.0).
#include <cstdint>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kThreads = 1024;
// Up to kFewTokens are one CTA's (64 requests of 1000 tokens: one launch 4.3 us,
// two 4.7; of 2048: 5.5 and 4.7), else a CTA takes kTokens at least (of 8192:
// 4.4 us; with 1024 a CTA 4.8, with 2048 6.1).
constexpr int64_t kFewTokens = 1024, kTokens = 512;

struct PlanArgs {
    const int32_t *cached, *fresh, *held, *free_pages, *free_count;
    const int64_t *pos_start;
    int32_t *table, *new_held, *new_count, *seq_lens, *tok_start;
    int64_t *dst, *pos;
    int64_t row, n_tok, most;    // row: of the table; most: tokens a row's pages hold
    int64_t per;                 // tokens of a CTA
    int B, Hkv, page, max_pages, n_free;
};

// What a launch writes: kPlace the tokens, pages, lengths and first tokens, kState new_held and new_free_count.
enum { kPlace = 1, kState = 2 };

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

template <int WHAT>
__global__ void __launch_bounds__(kThreads) page_plan_kernel(const __grid_constant__ PlanArgs a) {
    __shared__ int64_t warps[32];
    // of a round's requests: past their last token, cached tokens, pages held (negative: -1 - them, of a refused
    // one), pages that those before have taken
    __shared__ int32_t end_s[kThreads], cached_s[kThreads], held_s[kThreads], page_s[kThreads];
    __shared__ int32_t given;
    asm volatile("griddepcontrol.launch_dependents;");
    const int count = min(max(*a.free_count, 0), a.n_free);
    const int64_t lo = (int64_t)blockIdx.x * a.per, hi = min64(lo + a.per, a.n_tok);   // this CTA's tokens
    int64_t toks = 0, pages = 0;   // of the requests before this round; pages: needed
    if (threadIdx.x == 0) given = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        const bool live = b < a.B;
        const int32_t c = live ? max(a.cached[b], 0) : 0, m = live ? max(a.fresh[b], 0) : 0;
        const int32_t h = live ? min(max(a.held[b], 0), a.max_pages) : 0;
        const int64_t total = (int64_t)c + m, first = toks;
        int64_t all;
        const int64_t end = toks + block_scan(m, warps, all);
        toks += all;
        const bool fits = total <= a.most && end <= a.n_tok;
        int64_t need = fits && m > 0 ? (total + a.page - 1) / a.page - h : 0;
        if (need < 0) need = 0;
        const int64_t upto = pages + block_scan(need, warps, all);
        pages += all;
        const bool ok = fits && (need == 0 || upto <= count);
        if (WHAT & kPlace) {
            end_s[threadIdx.x] = (int32_t)min64(end, 0x7FFFFFFF);
            cached_s[threadIdx.x] = c;
            held_s[threadIdx.x] = ok ? h : -1 - h;
            page_s[threadIdx.x] = ok && need > 0 ? (int32_t)(upto - need) : 0;   // (at most count)
            if (live && blockIdx.x == 0) {
                a.tok_start[b + 1] = (int32_t)min64(end, 0x7FFFFFFF);
                a.seq_lens[b] = ok ? (int32_t)total : c;
            }
        }
        if ((WHAT & kState) && blockIdx.x == 0) {
            // sums only grow: those up to the list's length are the pages taken, the last of them all that are
            if (!(WHAT & kPlace) && b0 == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
            if (live) a.new_held[b] = h + (ok ? (int32_t)need : 0);
            if (ok && need > 0) atomicMax(&given, (int32_t)upto);
        }
        if (WHAT & kPlace) {
            __syncthreads();
            const int64_t from = max64(lo, first), stop = min64(hi, toks);
            for (int64_t n = from + threadIdx.x; n < stop; n += kThreads) {
                // the first request that ends past token n
                int r = 0;
#pragma unroll
                for (int half = kThreads / 2; half > 0; half >>= 1)
                    if (end_s[r + half - 1] <= n) r += half;
                const int64_t i = n - (r ? end_s[r - 1] : first), base = cached_s[r], t = base + i;
                const int32_t held = held_s[r];
                int64_t slot = -1;
                if (held >= 0) {
                    const int32_t pg = (int32_t)(t / a.page), off = (int32_t)(t - (int64_t)pg * a.page);
                    int32_t *row = a.table + (b0 + r) * a.row;
                    const int32_t *taken = a.free_pages + (count - 1 - page_s[r]) + held;   // entry e: taken[-e]
                    int32_t id;
                    if (pg < held) {
                        id = row[pg];
                    } else {
                        id = taken[-pg];
                        if (off == 0 || i == 0) row[pg] = id;
                        if (i == 0)
                            for (int32_t e = held; e < pg; ++e) row[e] = taken[-e];   // (fewer held than cached)
                    }
                    slot = (int64_t)id * a.Hkv * a.page + off;
                }
                a.dst[n] = slot;
                a.pos[n] = (a.pos_start ? a.pos_start[b0 + r] : base) + i;
            }
        }
    }
    if (WHAT & kPlace) {
        for (int64_t n = max64(lo, toks) + threadIdx.x; n < hi; n += kThreads) {
            a.dst[n] = -1;
            a.pos[n] = 0;
        }
        if (threadIdx.x == 0 && blockIdx.x == 0) a.tok_start[0] = 0;
    }
    if ((WHAT & kState) && blockIdx.x == 0) {
        __syncthreads();
        if (threadIdx.x == 0) *a.new_count = count - given;
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
    for (const void *i : in)
        if (i && ((i == new_held && i != held) || (i == new_free_count && i != free_count))) return TQ_ERR_ARG;
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
    // a CTA an SM at most: each scans all requests
    const int64_t even = (n_tok + sm_count() - 1) / sm_count();
    a.per = few ? kFewTokens : (even > kTokens ? even : kTokens);
    const unsigned ctas = few ? 1 : (unsigned)((n_tok + a.per - 1) / a.per);
    if (few || (new_held != held && new_free_count != free_count)) {
        page_plan_kernel<kPlace | kState><<<ctas, kThreads, 0, st>>>(a);
        return launch_status();
    }
    page_plan_kernel<kPlace><<<ctas, kThreads, 0, st>>>(a);
    const int r = launch_status();
    if (r != TQ_OK) return r;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, page_plan_kernel<kState>, a));
}
