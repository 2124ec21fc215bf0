// decode.cuh -- what the kernels of decode attention share (decode.cu: each request
// for itself; decode_shared.cu: requests that share a prefix).
#pragma once

#include "det_internal.cuh"
#include "det_math.cuh"

namespace det {

namespace {

enum Loader { kTma, kCopy16, kCopy4 };

// Waits for the piece in a slot of a warp's ring of `stages`; false when the wait gave up.
// In the test suite's copy of the library (DET_TEST_DECODE_GIVE_UP) a warp gives up on
// one of its first 2 * stages pieces, which one by its CTA's number, without a look at
// it, so that it leaves healthy copies in flight.
__device__ __forceinline__ bool wait_for_piece(uint32_t bars, int slot, uint32_t phase, int stages) {
#ifdef DET_TEST_DECODE_GIVE_UP
    if (slot + stages * int(phase) == int(blockIdx.x) % (2 * stages)) return false;
#endif
    return mbar_wait_bounded(bars + 8 * slot, phase);
}

__device__ __forceinline__ float4 lds4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float lds1(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void sts1(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float butterfly32(float s) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
    return s;
}

// exp4 where the maximum is not finite.
__device__ __noinline__ float4 exp4_any(float4 x, float m) {
    return make_float4(det_exp(__fsub_rn(x.x, m)), det_exp(__fsub_rn(x.y, m)),
                       det_exp(__fsub_rn(x.z, m)), det_exp(__fsub_rn(x.w, m)));
}

// Floats as whole numbers in their order, NaN above all; 0 is below every float's.
__device__ __forceinline__ unsigned max_key(float x) {
    const unsigned b = __float_as_uint(x);
    return x != x ? 0xffffffffu : b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float max_of_key(unsigned k) {
    if (k == 0xffffffffu) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}

}  // namespace
}  // namespace det
