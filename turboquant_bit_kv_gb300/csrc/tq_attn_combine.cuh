// The merge of the tensor-core decode attention's partials, shared by the
// combine kernels.
#pragma once

#include "tq_attn.cuh"
#include "tq_attn_mma.h"

namespace tq {

// Merge for the tensor-core kernel's partition, by one CTA for one (sequence,
// query head): the partials at base + i * stride, i < nslots.  128 x ng
// threads: thread d of slot group g reduces output dim d over batches g, g +
// ng, ... of kBatch slots.  Reading what other SMs just wrote costs a full L2
// round trip, so each thread issues every load of a batch at once (m and l of
// each slot -- the same address across the group -- and its dim of acc) and
// only then reduces, with the running max rescaled between batches; the groups
// run their rounds side by side and meet in shared memory.  rotate_back applies
// D H with the factor out_scale; store(d, value) takes the output.
template <int kBatch, class Store>
__device__ __forceinline__ void combine_mma(const float *base, int stride, int nslots, int rotate_back,
                                            float out_scale, uint32_t s0, uint32_t s1, uint32_t s2, uint32_t s3,
                                            Store store) {
    __shared__ float buf[kD];
    __shared__ float gacc[kCombineMaxGroups][kD];
    __shared__ float gml[kCombineMaxGroups][2];
    const int d = threadIdx.x & (kD - 1), grp = threadIdx.x / kD, ng = blockDim.x / kD;
    float M = -INFINITY, l = 0.f, acc = 0.f;
    for (int sb = grp * kBatch; sb < nslots; sb += ng * kBatch) {
        float mv[kBatch], lv[kBatch], xv[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const bool ok = sb + i < nslots;
            const float *ps = base + (int64_t)(sb + i) * stride;
            mv[i] = ok ? __ldcg(ps) : -INFINITY;
            lv[i] = ok ? __ldcg(ps + 1) : 0.f;
            xv[i] = ok ? __ldcg(ps + 4 + d) : 0.f;
        }
        float Mb = M;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) Mb = fmaxf(Mb, mv[i]);
        if (Mb == -INFINITY) {   // nothing finite so far: sums are 0, or NaN
#pragma unroll
            for (int i = 0; i < kBatch; ++i) l += lv[i];
            continue;
        }
        if (M != -INFINITY && Mb != M) {
            const float c = exp2f(M - Mb);
            l *= c;
            acc *= c;
        }
        M = Mb;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const float w = mv[i] == -INFINITY ? 0.f : exp2f(mv[i] - M);
            l = fmaf(w, lv[i], l);
            acc = fmaf(w, xv[i], acc);
        }
    }
    if (ng > 1) {
        // the groups' states, rescaled to their common max (every thread of a group holds the same
        // M and l)
        gacc[grp][d] = acc;
        if (d == 0) {
            gml[grp][0] = M;
            gml[grp][1] = l;
        }
        __syncthreads();
        if (grp == 0) {
            float Mt = -INFINITY;
            for (int g = 0; g < ng; ++g) Mt = fmaxf(Mt, gml[g][0]);
            l = 0.f;
            acc = 0.f;
            if (Mt != -INFINITY) {
                for (int g = 0; g < ng; ++g) {
                    const float mg = gml[g][0];
                    const float w = mg == -INFINITY ? 0.f : exp2f(mg - Mt);
                    l = fmaf(w, gml[g][1], l);
                    acc = fmaf(w, gacc[g][d], acc);
                }
            } else {
                for (int g = 0; g < ng; ++g) l += gml[g][1];
            }
        }
    }
    const float o = (l > 0.f || l != l) ? acc / l : 0.f;   // a NaN l (failed copy) propagates
    if (!rotate_back) {
        if (grp == 0) store(d, o);
        return;
    }
    // inverse rotation by group 0; every thread passes the same barriers
    if (grp == 0) buf[d] = o;
    __syncthreads();
#pragma unroll
    for (int L = 1; L < kD; L <<= 1) {
        float v = 0.f, w = 0.f;
        if (grp == 0) {
            v = buf[d];
            w = buf[d ^ L];
        }
        __syncthreads();
        if (grp == 0) buf[d] = (d & L) ? (w - v) : (v + w);
        __syncthreads();
    }
    if (grp == 0) {
        const uint32_t sw[4] = {s0, s1, s2, s3};
        const float v = buf[d] * out_scale;
        store(d, ((sw[d >> 5] >> (d & 31)) & 1u) ? -v : v);
    }
}

}  // namespace tq
