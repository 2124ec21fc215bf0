// row_stage.cuh -- what the kernels that stage rows of logits in shared memory
// share (cross-entropy, log probabilities): the NaN-propagating max, the
// butterfly, a group of the profile from two granules, and L2's evict-first policy.
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

__device__ __forceinline__ uint64_t l2_policy_evict_first() {
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

// 16-byte load from shared memory by shared-window address: in an out-of-line
// function a plain pointer would compile to a generic load (slower, and tracked
// as a long-latency access).
__device__ __forceinline__ float4 lds4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

}  // namespace
}  // namespace det
