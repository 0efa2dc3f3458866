// Work partition of the tensor-core decode-attention kernels (shared by the
// launcher, the query-prep and combine kernels and the workspace size query).
#pragma once

#include <stdint.h>

#include "tq_attn.cuh"

namespace tq {

constexpr int kMmaChunk = 32;        // tokens per chunk
constexpr int kMmaMaxWarpsPerSm = 16;   // no configuration runs more warps per SM
constexpr int kMmaMaxWorkersPerSeg = 31;   // workers <= 31 x segments: at most 32 partial slots,
constexpr int kMmaMaxChunksCapped = 5;     // as long as that leaves each worker 5 chunks or fewer
// Query fragments per (sequence, KV head) segment, in 32-bit words: three
// parts (n-tiles 0 and 1 of the rotated query, the sketched query) x 32
// lanes x 16 words.
constexpr int kFragWords = 3 * 32 * 16;

// Chunks are ordered by (sequence, KV head, position); worker w (warp
// w / P of CTA w % P, so that small grids spread over every CTA) covers
// chunks [w * Ctot / W, (w + 1) * Ctot / W), W <= Ctot (never empty).  Smax
// bounds the number of workers that touch one (sequence, KV head) segment,
// i.e. the partial slots per query head.  Workspace: partials
// [B][Hq][Smax][132] floats | query fragments [B * Hkv][kFragWords] words.
struct MmaPlan {
    int C;              // chunks per segment, ceil(T / kMmaChunk)
    int64_t Ctot;       // B * Hkv * C
    int P;              // CTAs (all resident), at most W
    int W;              // workers: min(Ctot, P x warps per CTA, and on small problems the cap below)
    int Smax;           // partial slots per (sequence, query head)
    int64_t frag_off;   // float offset of the query fragments in the workspace
    int wide;           // 2-bit values, one n-tile: 16 warps per SM (else 12)
    int warps;          // warps per CTA of the configuration
};

// kb / vb: key / value bits (vb = 16: raw fp16 values); qjl: two-term
// score; G: query heads per KV head.  Workers are capped at
// kMmaMaxWorkersPerSeg per segment while that leaves each worker at most
// kMmaMaxChunksCapped chunks.  mma_plan_for takes the SM count explicitly
// (mma_plan uses the current device's).
MmaPlan mma_plan_for(int sms, int B, int Hq, int Hkv, int T, int kb, int vb, bool qjl, int G);
MmaPlan mma_plan(int B, int Hq, int Hkv, int T, int kb, int vb, bool qjl, int G);
// Workspace floats the tensor-core path needs for any T <= T_cap on a GPU of
// `sms` SMs (sms <= 0: the current device's).
int64_t mma_workspace_floats(int B, int Hq, int Hkv, int T_cap, int sms);
bool attn_mma_supported(int kb, int vb, bool qjl, int G);
int launch_attn_mma(const AttnArgs &a, MmaPlan &plan, int kb, int vb, bool qjl, cudaStream_t st);

// Worker that owns chunk x: the largest w with floor(w * Ctot / W) <= x.
__host__ __device__ inline int64_t mma_worker_of_chunk(int64_t x, const MmaPlan &p) {
    return ((x + 1) * p.W - 1) / p.Ctot;
}

// Partition of the kernels that keep the scores: the chunks that hold tokens
// only, so that every worker does the same work whatever the sequences'
// lengths.  Sequence b has live_chunks(a, b) of them for each KV head; chunk x
// of all `total` belongs to worker live_worker(x, total, W), worker w < W =
// min(plan's workers, total) has chunks [w total / W, (w + 1) total / W), never
// none, and its partial of segment j lies in slot w + j: as workers and
// segments go by in order, no two pairs share a slot, and W + B Hkv hold them
// all.
__host__ __device__ inline int live_worker(int64_t x, int64_t total, int workers) {
    const int64_t W = min64(workers, total);
    return (int)(((x + 1) * W - 1) / total);
}

__device__ __forceinline__ int live_chunks(const AttnArgs &a, int b) {
    int L = a.T;
    if (a.seq_lens) {
        const int sl = a.seq_lens[b];
        L = sl < 0 ? 0 : (sl > a.T ? a.T : sl);
    }
    return (L + kMmaChunk - 1) / kMmaChunk;
}

// Pieces of a full chunk of tokens t0 .. t0 + kMmaChunk - 1 (t0 a multiple of
// kMmaChunk) that pages of any multiple of 8 tokens cut it into, four at most:
// piece i is tokens t .. t + len - 1, len 0 where there is none.
constexpr int kMmaPieces = kMmaChunk / 8;
__host__ __device__ inline void chunk_piece(int t0, int page, int i, int &t, int &len) {
    const int64_t end = (int64_t)t0 + kMmaChunk, head = page - t0 % page;   // head: tokens to the end of the first page
    const int64_t at = i == 0 ? t0 : t0 + head + (int64_t)(i - 1) * page;
    t = at < end ? (int)at : t0;
    len = at < end ? (int)min64(i == 0 ? head : page, end - at) : 0;
}

// Most tokens of a context whose scores are kept: positions up to a round of
// the kernels' loops (64 chunks) past the last one fit 32 bits.
constexpr int kMmaMaxTokens = 0x7FFFFFFF - 8191;

// The weights' part of the merge: CTAs per segment, each of `per` tokens (a
// multiple of kMmaChunk): about 32 CTAs per SM, but no more than one for every
// kWeightsTokens tokens (each works out its heads' maximum and sum).
constexpr int kWeightsTokens = 1024;
inline int weights_parts(int sms, int64_t segs, int T, int64_t &per) {
    const int64_t wanted = ((int64_t)sms * 32 + segs - 1) / segs;
    const int64_t most = ((int64_t)T + kWeightsTokens - 1) / kWeightsTokens;
    const int64_t parts = min64(wanted, most);
    per = ((T + parts - 1) / parts + kMmaChunk - 1) / kMmaChunk * kMmaChunk;
    return (int)((T + per - 1) / per);
}

// A common factor for a codebook's centroids under which their fp16 roundings
// are smallest (tq_attn_weights.cu).
float attn_centroid_factor(const tq_codebook *cb);

// Slot groups of 128 threads in a combine CTA: one per 32 slots of Smax, at most kCombineMaxGroups.
inline int mma_combine_groups(const MmaPlan &p) {
    const int g = (p.Smax + 31) / 32;
    return g < 1 ? 1 : (g > kCombineMaxGroups ? kCombineMaxGroups : g);
}

}  // namespace tq
