// Decode attention that also adds up the attention weights
// (tq_attn_decode_weights): the accumulators from which tokens are chosen for
// eviction.
//
//   s_{g,t} = scale * n_t <R q_g, c[code_t]>,  p_g = softmax_t(s_g),
//   o_g = R^T sum_t p_{g,t} nv_t cV[vcode_t],  w_t <- decay w_t + sum_g p_{g,t}
//
// over the G query heads of a KV head.  A weight needs the softmax's final
// maximum and sum, which a single pass over a split context does not have:
// the attention kernel writes its scores (4 G bytes a token, next to 68 to
// 132 bytes of packed blocks) on its way, and the kernel that merges the
// splits turns them into weights.  Computing the scores a second time would
// cost the keys' lookups again, which is what bounds the attention kernel.
// Three launches as in tq_attn_decode (query prep, attention, merge), chained
// as programmatic dependents.
//
// The work is split over the chunks that hold tokens, not over the longest
// context, so a batch of different lengths takes as long as its tokens (16
// sequences of 0 to 8192 tokens, 55% of them: 49 us before).
//
// Every weight is written by one thread, its heads added in order, so results
// do not depend on timing.  Scores, statistics and weights are float32.
#include <cmath>
#include <cstring>
#include <mutex>

#include "tq_attn.cuh"
#include "tq_attn_combine.cuh"
#include "tq_attn_mma.h"
#include "tq_internal.h"

namespace tq {

int launch_attn_mma_scores_k2(const AttnArgs &a, MmaPlan &plan, int vb, int nt, bool paged, cudaStream_t st);
int launch_attn_mma_scores_k3(const AttnArgs &a, MmaPlan &plan, int vb, int nt, bool paged, cudaStream_t st);
int launch_attn_mma_scores_k4(const AttnArgs &a, MmaPlan &plan, int vb, int nt, bool paged, cudaStream_t st);
int launch_attn_prep_mma(const AttnArgs &a, const MmaPlan &plan, int qjl, cudaStream_t st);

// A common factor for a codebook's centroids under which their fp16 roundings
// are smallest (the values, and the keys of a shared prefix, enter the tensor cores
// as fp16; the factor is taken out again later): the best of 2^14 factors in [1, 2).
// The codebook is antisymmetric, so L / 2 magnitudes have to fall close to
// fp16 numbers at once: the worst rounding drops from 2^-12 to about 2^-18
// (2 bits), 2^-15 (3 bits), 2^-13.5 (4 bits).
float attn_centroid_factor(const tq_codebook *cb) {
    static std::mutex mu;
    static tq_codebook known[5];
    static float factor[5];
    std::lock_guard<std::mutex> lock(mu);
    const int n = cb->bits;
    if (factor[n] != 0.f && std::memcmp(known[n].centroids, cb->centroids, sizeof(float) * cb->levels) == 0)
        return factor[n];
    float best = 1.f, err = INFINITY;
    for (int i = 0; i < (1 << 14); ++i) {
        const float f = 1.f + i / 16384.f;
        float e = 0.f;
        for (int q = 0; q < cb->levels; ++q) {
            const float c = std::fabs(cb->centroids[q]) * f;
            if (!(c > 0.f)) continue;
            int ex;
            const float m = std::frexp(c, &ex) * 2048.f;   // 11 significant bits
            e = std::fmax(e, std::fabs(m - std::nearbyint(m)) / m);
        }
        if (e < err) {
            err = e;
            best = f;
        }
    }
    known[n] = *cb;
    factor[n] = best;
    return best;
}

namespace {

constexpr int kMergeBatch = 16;      // slots a merging thread loads at once (one round covers 16 x groups)

struct WeightsArgs {
    const float *ws;
    const float *scores;
    const int32_t *seq_lens;
    const int2 *live;
    float *weights;
    void *out;
    int64_t w_stride;
    int64_t per;
    int Hq, Hkv, G, T, B, parts;   // parts: weights CTAs per segment, of per tokens each (a multiple of 32)
    int out_dtype;
    float decay, out_scale;
    uint32_t signs[4];
};

// Weights of tokens t0 .. end - 1 of a segment from its scores and its heads'
// (maximum, 1 / sum): a warp takes two chunks of 32 tokens at a time, G rows of
// 32 scores each, one coalesced load a row.  stats() fills ml (all threads of
// the CTA run it) while the first scores are on their way.
template <int G, class Stats>
__device__ __forceinline__ void add_weights(const float *scores, const float (*ml)[2], float *w, int t0, int end,
                                            float decay, Stats stats) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    float mx[G], inv[G];
    bool first = true;
    for (int c = t0 / kMmaChunk + 2 * warp; first || c * kMmaChunk < end; c += 2 * nw) {
        float s[2][G], old[2] = {0.f, 0.f};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int t = (c + u) * kMmaChunk + lane;
            const float *row = scores + (int64_t)(c + u) * (kMmaChunk * G) + lane;
            if (t < end) {
#pragma unroll
                for (int g = 0; g < G; ++g) s[u][g] = __ldcs(row + g * kMmaChunk);
                if (decay != 0.f) old[u] = __ldcs(w + t);
            }
        }
        if (first) {
            stats();
#pragma unroll
            for (int g = 0; g < G; ++g) {
                mx[g] = ml[g][0];
                inv[g] = ml[g][1];
            }
            first = false;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int t = (c + u) * kMmaChunk + lane;
            if (t < end) {
                float p = 0.f;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    float e;   // (weights below 2^-126 count as 0)
                    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(s[u][g] - mx[g]));
                    p = fmaf(e, inv[g], p);
                }
                w[t] = fmaf(old[u], decay, p);
            }
        }
    }
}

// CTAs [0, B Hq): the merge of one (sequence, query head).  The rest: the
// weights of a.per tokens of one segment (sequence, KV head): the
// final maximum and sum of its heads, one warp per head over the segment's
// slots, then a chunk of 32 tokens per warp at a time, the first scores
// requested before (1 x 1001 tokens 12.9 -> 12.2 us a call, 64 x 32769 512 ->
// 505).  The lengths are the caller's, so they are read before the attention
// kernel is waited for; the CTAs of the merge all wait, so the grid ends after
// it.
__global__ void __launch_bounds__(kAttnThreads * kCombineMaxGroups, 2) attn_weights_kernel(
    const __grid_constant__ WeightsArgs a, const __grid_constant__ MmaPlan plan) {
    const int heads = a.B * a.Hq;
    const bool merge = (int)blockIdx.x < heads;
    const int64_t unit = blockIdx.x - heads;
    const int64_t j = merge ? (blockIdx.x / a.Hq) * a.Hkv + blockIdx.x % a.Hq / a.G : unit / a.parts;
    const int b = (int)(j / a.Hkv);
    int L = a.T;
    if (a.seq_lens) {
        const int sl = a.seq_lens[b];
        L = sl < 0 ? 0 : (sl > a.T ? a.T : sl);
    }
    const int64_t t0 = merge ? 0 : unit % a.parts * a.per;
    if (t0 >= L && !merge) return;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the segment's slots: the workers whose ranges meet its chunks
    const int2 met = __ldcg(a.live + j);
    const int nslots = met.y;
    const float *slots = a.ws + (met.x + j) * a.G * kPartialFloats;   // [nslots][G]
    if (merge) {
        const int64_t at = (int64_t)blockIdx.x * kD;
        combine_mma<kMergeBatch>(
            slots + blockIdx.x % a.G * kPartialFloats, a.G * kPartialFloats, nslots, 1, a.out_scale, a.signs[0],
            a.signs[1], a.signs[2], a.signs[3], [&](int d, float v) {
                if (a.out_dtype == TQ_F32) static_cast<float *>(a.out)[at + d] = v;
                else if (a.out_dtype == TQ_BF16) static_cast<__nv_bfloat16 *>(a.out)[at + d] = __float2bfloat16_rn(v);
                else static_cast<__half *>(a.out)[at + d] = __float2half_rn(v);
            });
        return;
    }
    __shared__ float ml[8][2];   // final maximum, 1 / sum
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    auto stats = [&]() {
        for (int g = warp; g < a.G; g += nw) {
            const float *base = slots + g * kPartialFloats;
            float M = -INFINITY, l = 0.f;
            for (int s = lane; s < nslots; s += 32) {
                const float *ps = base + (int64_t)s * a.G * kPartialFloats;
                const float ms = __ldcg(ps), ls = __ldcg(ps + 1);
                const float mn = fmaxf(M, ms);
                l = mn == -INFINITY ? l + ls : l * exp2f(M - mn) + ls * exp2f(ms - mn);
                M = mn;
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) {
                const float mo = __shfl_xor_sync(0xffffffffu, M, o), lo = __shfl_xor_sync(0xffffffffu, l, o);
                const float mn = fmaxf(M, mo);
                l = mn == -INFINITY ? l + lo : l * exp2f(M - mn) + lo * exp2f(mo - mn);
                M = mn;
            }
            if (lane == 0) {
                // no finite score at all: weights of 0 (a NaN sum, from a failed copy, still shows)
                const bool dead = M == -INFINITY;
                ml[g][0] = dead ? 0.f : M;
                ml[g][1] = dead ? l : 1.f / l;
            }
        }
        __syncthreads();
    };
    const int end = (int)min64(t0 + a.per, L);
    float *w = a.weights + j * a.w_stride;
    const float *sc = a.scores + j * plan.C * (kMmaChunk * a.G);
    switch (a.G) {
        case 1: add_weights<1>(sc, ml, w, (int)t0, end, a.decay, stats); break;
        case 2: add_weights<2>(sc, ml, w, (int)t0, end, a.decay, stats); break;
        case 3: add_weights<3>(sc, ml, w, (int)t0, end, a.decay, stats); break;
        case 4: add_weights<4>(sc, ml, w, (int)t0, end, a.decay, stats); break;
        case 5: add_weights<5>(sc, ml, w, (int)t0, end, a.decay, stats); break;
        case 6: add_weights<6>(sc, ml, w, (int)t0, end, a.decay, stats); break;
        case 7: add_weights<7>(sc, ml, w, (int)t0, end, a.decay, stats); break;
        default: add_weights<8>(sc, ml, w, (int)t0, end, a.decay, stats); break;
    }
}

int64_t scores_floats(int B, int Hq, int Hkv, int T) {
    return (int64_t)B * Hkv * ((T + kMmaChunk - 1) / kMmaChunk) * kMmaChunk * (Hq / Hkv);
}

// Workspace: partials [W + B Hkv][G][132] | query fragments [B Hkv] | segments' workers [B Hkv][2] | scores, in
// floats; W workers, at most kMmaMaxWarpsPerSm per SM and a chunk each.
struct Layout {
    int64_t frag, live, scores, floats;
    Layout(int B, int Hq, int Hkv, int T, int64_t W) {
        const int64_t segs = (int64_t)B * Hkv;
        frag = (W + segs) * (Hq / Hkv) * kPartialFloats;
        live = frag + segs * kFragWords;
        scores = live + ((segs * 2 + 3) & ~(int64_t)3);
        floats = scores + scores_floats(B, Hq, Hkv, T);
    }
};

int64_t most_workers(int B, int Hkv, int T) {
    return min64((int64_t)B * Hkv * ((T + kMmaChunk - 1) / kMmaChunk), (int64_t)kMmaMaxWarpsPerSm * sm_count());
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" size_t tq_attn_weights_workspace_bytes(int B, int Hq, int Hkv, int T) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || T <= 0 || T > kMmaMaxTokens || Hq % Hkv || Hq / Hkv > 8) return 0;
    return (size_t)Layout(B, Hq, Hkv, T, most_workers(B, Hkv, T)).floats * sizeof(float);
}

extern "C" int tq_attn_decode_weights(const void *q, int q_dtype, const uint8_t *k_blocks, const tq_codebook *kcb,
                                      const uint8_t *v_blocks, const tq_codebook *vcb, const int32_t *block_table,
                                      int max_pages, int page_tokens, const int32_t *seq_lens, int B, int Hq, int Hkv,
                                      int T_cap, int T, float scale, tq_signs signs, float *weights,
                                      int64_t weights_row_stride, float decay, void *out, int out_dtype,
                                      void *workspace, size_t workspace_bytes, void *stream) {
    if (!q || !k_blocks || !kcb || !v_blocks || !vcb || !weights || !out || !workspace) return TQ_ERR_ARG;
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || T < 1 || weights_row_stride < T) return TQ_ERR_ARG;
    if (!std::isfinite(scale) || !std::isfinite(decay)) return TQ_ERR_ARG;
    const bool paged = block_table != nullptr;
    if (paged) {
        if (max_pages <= 0 || page_tokens <= 0 || (int64_t)max_pages * page_tokens < T) return TQ_ERR_ARG;
        if (page_tokens & 7) return TQ_ERR_UNSUPPORTED;
    } else if (T > T_cap || (T_cap & 7)) {
        return TQ_ERR_ARG;
    }
    const int G = Hq / Hkv;
    if (G > 8 || T > kMmaMaxTokens) return TQ_ERR_UNSUPPORTED;
    if (dtype_bytes(q_dtype) == 0 || dtype_bytes(out_dtype) == 0) return TQ_ERR_UNSUPPORTED;
    if (!codebook_ok(kcb) || !codebook_ok(vcb)) return TQ_ERR_UNSUPPORTED;
    if (!aligned(q, dtype_bytes(q_dtype)) || !aligned(k_blocks, 16) || !aligned(v_blocks, 16) || !aligned(out, 16) ||
        !aligned(workspace, 16) || !aligned(weights, 4) || !aligned(seq_lens, 4) || !aligned(block_table, 4))
        return TQ_ERR_ALIGN;
    if (workspace_bytes < tq_attn_weights_workspace_bytes(B, Hq, Hkv, T)) return TQ_ERR_WORKSPACE;
    const int64_t segs = (int64_t)B * Hkv;
    int64_t per;
    const int parts = weights_parts(sm_count(), segs, T, per);
    const int64_t grid = (int64_t)B * Hq + (int64_t)B * Hkv * parts;
    if (grid > 0x7FFFFFFF || segs * ((T + kMmaChunk - 1) / kMmaChunk) > 0x7FFFFFFF) return TQ_ERR_UNSUPPORTED;

    AttnArgs a = {};
    a.drop = drop_copies();
    a.q = q;
    a.q_dtype = q_dtype;
    a.k = k_blocks;
    a.v = v_blocks;
    a.seq_lens = seq_lens;
    a.ws = static_cast<float *>(workspace);
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = G;
    a.T_cap = paged ? (T + 7) & ~7 : T_cap;
    a.T = T;
    a.qscale = scale * 1.4426950408889634f;
    const float vf = attn_centroid_factor(vcb);
    for (int i = 0; i < 16; ++i) {
        a.kc[i] = kcb->centroids[i];
        a.vc[i] = vcb->centroids[i] * vf;
    }
    for (int i = 0; i < 4; ++i) a.signs[i] = signs.w[i];
    a.table = block_table;
    a.max_pages = max_pages;
    a.page = page_tokens;

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int kb = kcb->bits, vb = vcb->bits, nt = G <= 4 ? 1 : 2;
    MmaPlan plan = mma_plan(B, Hq, Hkv, T, kb, vb, false, G);
    const Layout at(B, Hq, Hkv, T, plan.W);
    plan.frag_off = at.frag;
    a.live = reinterpret_cast<int2 *>(a.ws + at.live);
    a.workers = plan.W;
    a.scores = a.ws + at.scores;
    int r = launch_attn_prep_mma(a, plan, 0, st);
    if (r != TQ_OK) return r;
    r = kb == 2 ? launch_attn_mma_scores_k2(a, plan, vb, nt, paged, st)
                : kb == 3 ? launch_attn_mma_scores_k3(a, plan, vb, nt, paged, st)
                          : launch_attn_mma_scores_k4(a, plan, vb, nt, paged, st);
    if (r != TQ_OK) return r;
    WeightsArgs w;
    w.ws = a.ws;
    w.scores = a.scores;
    w.seq_lens = seq_lens;
    w.live = a.live;
    w.weights = weights;
    w.out = out;
    w.w_stride = weights_row_stride;
    w.Hq = Hq;
    w.Hkv = Hkv;
    w.G = G;
    w.T = T;
    w.B = B;
    w.parts = parts;
    w.per = per;
    w.out_dtype = out_dtype;
    w.decay = decay;
    w.out_scale = 0.08838834764831845f / vf;
    for (int i = 0; i < 4; ++i) w.signs[i] = signs.w[i];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    const int groups = (plan.Smax + kMergeBatch - 1) / kMergeBatch;
    cfg.blockDim = dim3(kAttnThreads * (groups < 1 ? 1 : (groups > kCombineMaxGroups ? kCombineMaxGroups : groups)));
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launch_status(cudaLaunchKernelEx(&cfg, attn_weights_kernel, w, plan));
}
