// row_stage.cuh -- what the kernels that keep rows of logits in shared memory
// share (cross-entropy, log probabilities): the NaN-propagating max, the bulk
// copies of a row's 16-byte granules, and the chain sums over a staged row.
//
// A row of floats may start anywhere mod 16 bytes: with misalignment H
// (elements) granule q is the aligned float4 of elements 4q - H .. 4q + 3 - H,
// and the profile's group g (elements 4g .. 4g+3) is the last 4 - H elements of
// granule g and the first H of granule g + 1.
#pragma once

#include "det_internal.cuh"

namespace det {
namespace {

constexpr int kXsPiece = 1024;                   // granules per bulk copy (16 KB)

__device__ __forceinline__ float warp_butterfly_sum(float s) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
    return s;
}

// The profile's row max: NaN if any element is NaN, else the largest (ties
// between +0 and -0 are bit-inert for the loss and dlogits).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The profile's group g (elements 4g .. 4g+3) from granule g (cur) and
// granule g + 1 (nxt): the last 4 - H elements of cur, then the first H of nxt.
template <int H>
__device__ __forceinline__ float4 group_of(float4 cur, float4 nxt) {
    if (H == 0) return cur;
    if (H == 1) return make_float4(cur.y, cur.z, cur.w, nxt.x);
    if (H == 2) return make_float4(cur.z, cur.w, nxt.x, nxt.y);
    return make_float4(cur.w, nxt.x, nxt.y, nxt.z);
}

__device__ __forceinline__ float comp(float4 v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Asks L2 to fetch granules [0, n) of the row whose aligned base is xa. Every
// granule holds at least one element of the row, so no byte outside the
// row's pages is touched.
__device__ __forceinline__ void prefetch_granules_l2(const float *xa, int n) {
    for (int q = 0; q < n; q += kXsPiece) {
        const int c = min(kXsPiece, n - q);
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(xa + 4 * q),
                     "r"(uint32_t(c) * 16u)
                     : "memory");
    }
}

// Thread 0: copies granules [q0, q1) of the row whose aligned base is xa into
// the same granules of buf, completing on bar.
__device__ __forceinline__ void load_granules(float4 *buf, const float *xa, int q0, int q1,
                                              uint64_t *bar) {
    const uint32_t b = smem_u32(bar);
    mbar_arrive_expect_tx(b, uint32_t(q1 - q0) * 16u);
    for (int q = q0; q < q1; q += kXsPiece) {
        const int n = min(kXsPiece, q1 - q);
        bulk_load(smem_u32(buf + q), xa + 4 * q, uint32_t(n) * 16u, b);
    }
}

__device__ __forceinline__ uint64_t l2_policy_evict_first() {
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

// load_granules of a row that is not read again: L2 may drop it first.
__device__ __forceinline__ void load_granules_last(float4 *buf, const float *xa, int q0, int q1,
                                                   uint64_t *bar, uint64_t evict_first) {
    const uint32_t b = smem_u32(bar);
    mbar_arrive_expect_tx(b, uint32_t(q1 - q0) * 16u);
    for (int q = q0; q < q1; q += kXsPiece) {
        const int n = min(kXsPiece, q1 - q);
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(buf + q)),
            "l"(xa + 4 * q), "r"(uint32_t(n) * 16u), "r"(b), "l"(evict_first)
            : "memory");
    }
}

// Stage D for a row with misalignment H: chain l (< 256) adds the exps of its
// groups g = l, l + 256, ... in ascending order. Group g is the last 4 - H
// elements of granule g and the first H of granule g + 1; both granules are
// read with 16-byte loads (consecutive chains, consecutive granules: no bank
// conflicts), one sweep ahead of the adds.
// s: the chain's value so far, for a row that comes in segments of whole sweeps.
// 16-byte load from shared memory by shared-window address: the chain runs in
// an out-of-line function, where a plain pointer would compile to a generic
// load (slower, and tracked as a long-latency access).
__device__ __forceinline__ float4 lds4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ float lds1(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

template <int H>
__device__ __noinline__ float xent_smem_chain(uint32_t buf, int V, float s = 0.0f) {
    const int l = threadIdx.x;
    const int ngroups = (V + 3) >> 2, gfull = V >> 2;
    int g = l;
    if (g < gfull) {
        float4 c0 = lds4(buf + 16u * g), c1 = H ? lds4(buf + 16u * (g + 1)) : c0;
        for (; g < gfull; g += kXentLanes) {
            const int gn = g + kXentLanes;
            float4 n0 = c0, n1 = c1;
            if (gn < gfull) {
                n0 = lds4(buf + 16u * gn);
                if (H) n1 = lds4(buf + 16u * (gn + 1));
            }
            const float4 v = group_of<H>(c0, c1);
            s = __fadd_rn(__fadd_rn(__fadd_rn(__fadd_rn(s, v.x), v.y), v.z), v.w);
            c0 = n0;
            c1 = n1;
        }
    }
    if (g < ngroups) {     // the last, partial group
        for (int j = 4 * g; j < V; ++j) s = __fadd_rn(s, lds1(buf + 4u * (j + H)));
    }
    return s;
}

}  // namespace
}  // namespace det
