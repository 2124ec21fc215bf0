// decode.cu -- attention of one new token a request over a paged key-value
// cache, for sm_103a.
//
//   s_j = q K_j (fmaf chain from +0),  x_j = s_j scale,  m = max x_j,
//   e_j = exp(x_j - m),  S = the 256-chain sum of the e_j,  p_j = e_j (1/S),
//   o = sum over 256-token chunks, left to right, of fmaf chains of p_j V_j
//
// the last row of the causal attention over the same tokens, bit for bit.
//
// One CTA a request and query head: a thread a token for the scores, thread l =
// chain l for S, a thread a component for P V.
#include <algorithm>

#include "det_internal.cuh"
#include "det_math.cuh"

namespace det {
namespace {

constexpr int kThreads = 256;

struct DecodeArgs {
    int heads, kv_heads, head_dim;
    const float *q;
    int64_t ldq;
    const float *k, *v;
    int64_t num_pages, page_size, page_stride, token_stride, head_stride;
    const int32_t *table;
    int64_t max_pages, ldt;
    const int32_t *kv_lens;
    float scale;
    float *out;
    int64_t ldo;
    float *scores;            // batch * heads rows of max_len floats
    int64_t max_len;
    int32_t *dev_status;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__global__ void __launch_bounds__(kThreads) decode_kernel(DecodeArgs A) {
    __shared__ float red[kThreads / 32];
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = h / (A.heads / A.kv_heads), d = A.head_dim;
    float *o = A.out + b * A.ldo + int64_t(h) * d;
    const float *q = A.q + b * A.ldq + int64_t(h) * d;
    const int64_t n = A.kv_lens[b];
    const bool bad = n < 0 || n > A.max_len;
    const int32_t *pages = A.table + b * A.ldt;
    int lost = 0;
    if (!bad)
        for (int64_t i = tid; i * A.page_size < n; i += kThreads)
            lost |= pages[i] < 0 || pages[i] >= A.num_pages;
    lost = __syncthreads_or(lost);
    if (bad || lost) {
        for (int i = tid; i < d; i += kThreads) o[i] = __uint_as_float(0x7fc00000u);
        if (tid == 0 && A.dev_status)
            atomicOr(reinterpret_cast<int *>(A.dev_status), bad ? 1 : 2);
        return;
    }
    if (n == 0) {
        for (int i = tid; i < d; i += kThreads) o[i] = 0.0f;
        return;
    }
    auto row_of = [&](int64_t j) {
        return int64_t(pages[j / A.page_size]) * A.page_stride +
               (j % A.page_size) * A.token_stride + g * A.head_stride;
    };
    float *x = A.scores + (int64_t(b) * A.heads + h) * A.max_len;
    float m = __uint_as_float(0xff800000u);
    for (int64_t j = tid; j < n; j += kThreads) {
        const float *kr = A.k + row_of(j);
        float s = 0.0f;
        for (int i = 0; i < d; ++i) s = __fmaf_rn(q[i], kr[i], s);
        s = __fmul_rn(s, A.scale);
        x[j] = s;
        m = max_nan(m, s);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (lane == 0) red[warp] = m;
    __syncthreads();
    m = red[0];
    for (int w = 1; w < kThreads / 32; ++w) m = max_nan(m, red[w]);
    __syncthreads();
    float S = 0.0f;
    for (int64_t j = 4 * tid; j < n; j += 4 * kThreads)
        for (int64_t i = j; i < j + 4 && i < n; ++i) {
            const float e = det_exp(__fsub_rn(x[i], m));
            x[i] = e;
            S = __fadd_rn(S, e);
        }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) S = __fadd_rn(S, __shfl_xor_sync(0xffffffffu, S, off));
    if (lane == 0) red[warp] = S;
    __syncthreads();
    const float inv = __fdiv_rn(
        1.0f, __fadd_rn(__fadd_rn(__fadd_rn(red[0], red[1]), __fadd_rn(red[2], red[3])),
                        __fadd_rn(__fadd_rn(red[4], red[5]), __fadd_rn(red[6], red[7]))));
    for (int i = tid; i < d; i += kThreads) {
        float total = 0.0f;
        for (int64_t c = 0; c < n; c += kKChunk) {
            const int64_t end = c + kKChunk < n ? c + kKChunk : n;
            float part = 0.0f;
            for (int64_t j = c; j < end; ++j)
                part = __fmaf_rn(__fmul_rn(x[j], inv), A.v[row_of(j) + i], part);
            total = c ? __fadd_rn(total, part) : part;
        }
        o[i] = total;
    }
}

}  // namespace

size_t decode_workspace_bytes(int64_t batch, int64_t heads, int64_t, int64_t, int64_t max_len) {
    return size_t(batch) * size_t(heads) * size_t(max_len) * 4;
}

cudaError_t launch_decode_attention(int64_t batch, int heads, const float *q, int64_t ldq,
                                    const det_kv_cache &c, const int32_t *table,
                                    int64_t max_pages, int64_t ldt, const int32_t *kv_lens,
                                    float scale, float *out, int64_t ldo, float *workspace,
                                    int32_t *dev_status, cudaStream_t s) {
    const DecodeArgs A = {heads, int(c.kv_heads), int(c.head_dim), q, ldq, c.k, c.v, c.num_pages,
                          c.page_size, c.page_stride, c.token_stride, c.head_stride, table,
                          max_pages, ldt, kv_lens, scale, out, ldo, workspace,
                          max_pages * c.page_size, dev_status};
    decode_kernel<<<dim3(unsigned(heads), unsigned(batch)), kThreads, 0, s>>>(A);
    return cudaGetLastError();
}

}  // namespace det
