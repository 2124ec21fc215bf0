// logprob.cu -- log probabilities of given tokens under rows of logits, with
// entropy and the largest alternatives, and their gradient, for sm_103a.
//
//   m = max x_j,  e_j = exp(x_j - m),  S = the cross-entropy's 256-chain sum,
//   logp = (x_y - m) - log S,  T = sum e_j (x_j - m) over 4096 chains,
//   entropy = log S - T / S
//   dx_j = dlogp ([j == y] - p_j) - dentropy p_j ((x_j - m) - log S + entropy)
//
// The forward reads each logit once and writes a few floats a row; the gradient
// reads and writes each element once: HBM bounds both.
#include <algorithm>

#include "det_internal.cuh"
#include "det_math.cuh"

namespace det {
namespace {

constexpr int kThreads = 256;
constexpr int kTChains = 4096;
constexpr float kNaNf = __builtin_nanf("");

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float butterfly32(float s) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, off));
    return s;
}

// Order of the alternatives as a key: larger logits have larger keys, +0 and -0
// the same, NaN the largest; the lower id wins among equal keys. A 64-bit rank
// holds both.
__device__ __forceinline__ uint64_t rank_of(float x, int j) {
    uint32_t k;
    if (x != x) {
        k = 0xffffffffu;
    } else {
        const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));    // -0 -> +0
        k = b & 0x80000000u ? ~b : b | 0x80000000u;
    }
    return uint64_t(k) << 32 | uint32_t(~j);
}

struct LogprobArgs {
    int64_t rows;
    int V;
    const float *logits;
    int64_t ld;
    const int32_t *tokens;
    int top_k;
    float *logp, *entropy;
    float4 *stats;
    int32_t *top_ids;
    float *top_logp;
    int32_t *dev_status;
};

// A CTA a row, thread l = chain l; the row is read in three passes.
__global__ void __launch_bounds__(kThreads) logprob_kernel(LogprobArgs A) {
    __shared__ float T[kTChains / 4];
    __shared__ float red[32];
    __shared__ uint64_t best[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x) {
        const float *x = A.logits + row * A.ld;
        float m = x[0];
        for (int j = tid; j < A.V; j += kThreads) m = max_nan(m, x[j]);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (lane == 0) red[warp] = m;
        __syncthreads();
        m = red[0];
        for (int w = 1; w < kThreads / 32; ++w) m = max_nan(m, red[w]);
        m = __fadd_rn(m, 0.0f);          // a zero maximum is +0
        __syncthreads();
        // elements 4 (tid + 256 t) .. + 3 of sweep t lie on chains
        // 4 (tid + 256 (t mod 4)) .. + 3 of T
        float S = 0.0f, t16[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) t16[i] = 0.0f;
        for (int j0 = 4 * tid; j0 < A.V; j0 += 16 * kThreads) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int j = j0 + (i >> 2) * 4 * kThreads + (i & 3);
                if (j < A.V) {
                    const float d = __fsub_rn(x[j], m), e = det_exp(d);
                    S = __fadd_rn(S, e);
                    if (e != 0.0f) t16[i] = __fmaf_rn(e, d, t16[i]);
                }
            }
        }
        S = butterfly32(S);
        if (lane == 0) red[warp] = S;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            T[tid + i * kThreads] = __fadd_rn(
                __fadd_rn(__fadd_rn(t16[4 * i], t16[4 * i + 1]), t16[4 * i + 2]), t16[4 * i + 3]);
        __syncthreads();
        S = __fadd_rn(__fadd_rn(__fadd_rn(red[0], red[1]), __fadd_rn(red[2], red[3])),
                      __fadd_rn(__fadd_rn(red[4], red[5]), __fadd_rn(red[6], red[7])));
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float u = butterfly32(T[tid + i * kThreads]);
            if (lane == 0) red[warp + i * (kThreads / 32)] = u;
        }
        __syncthreads();
        const float Ts = butterfly32(red[lane]);
        const float logS = det_log(S);
        const float ent = __fsub_rn(logS, __fdiv_rn(Ts, S));
        if (tid == 0) {
            const int y = A.tokens[row];
            const bool none = y == -1, wrong = !none && (y < 0 || y >= A.V);
            A.logp[row] = none ? 0.0f : wrong ? kNaNf : __fsub_rn(__fsub_rn(x[y], m), logS);
            A.entropy[row] = ent;
            if (A.stats) A.stats[row] = make_float4(m, __fdiv_rn(1.0f, S), logS, ent);
            if (wrong && A.dev_status) atomicOr(reinterpret_cast<int *>(A.dev_status), 1);
        }
        // the alternatives, one at a time: the best rank below the last one
        uint64_t last = ~uint64_t(0);
        for (int k = 0; k < A.top_k; ++k) {
            uint64_t r = 0;
            for (int j = tid; j < A.V; j += kThreads) {
                const uint64_t c = rank_of(x[j], j);
                if ((c < last || k == 0) && c > r) r = c;
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) {
                const uint64_t o = __shfl_xor_sync(0xffffffffu, r, off);
                r = o > r ? o : r;
            }
            if (lane == 0) best[warp] = r;
            __syncthreads();
            for (int w = 0; w < kThreads / 32; ++w) r = best[w] > r ? best[w] : r;
            __syncthreads();
            last = r;
            if (tid == 0) {
                const int j = int(~uint32_t(r));
                A.top_ids[row * A.top_k + k] = j;
                A.top_logp[row * A.top_k + k] = __fsub_rn(__fsub_rn(x[j], m), logS);
            }
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kThreads)
    logprob_bwd_kernel(int64_t rows, int V, const float *logits, int64_t ld,
                       const int32_t *tokens, const float4 *stats, const float *dlogp,
                       const float *dentropy, float *dlogits, int64_t ldd) {
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const float4 st = stats[row];
        const int y = tokens[row];
        const bool wrong = y < -1 || y >= V;
        const float g = y == -1 || wrong ? 0.0f : dlogp[row];
        const float gH = dentropy ? dentropy[row] : 0.0f;
        for (int j = blockIdx.x * kThreads + threadIdx.x; j < V; j += gridDim.x * kThreads) {
            const float d = __fsub_rn(logits[row * ld + j], st.x);
            const float p = __fmul_rn(det_exp(d), st.y);
            float a = y == -1 ? 0.0f : __fmul_rn(g, __fsub_rn(j == y ? 1.0f : 0.0f, p));
            if (dentropy) {
                const float w =
                    p == 0.0f ? 0.0f : __fmul_rn(p, __fadd_rn(__fsub_rn(d, st.z), st.w));
                a = __fsub_rn(a, __fmul_rn(gH, w));
            }
            dlogits[row * ldd + j] = wrong ? kNaNf : a;
        }
    }
}

}  // namespace

cudaError_t launch_logprob(int64_t rows, int64_t V, const float *logits, int64_t ld,
                           const int32_t *tokens, int top_k, float *logp, float *entropy,
                           float *stats, int32_t *top_ids, float *top_logp, int32_t *dev_status,
                           cudaStream_t s) {
    const LogprobArgs A = {rows, int(V), logits, ld, tokens, top_k, logp, entropy,
                           reinterpret_cast<float4 *>(stats), top_ids, top_logp, dev_status};
    const int64_t grid = std::min<int64_t>(rows, int64_t(sm_count_current_device()) * 4);
    logprob_kernel<<<unsigned(grid), kThreads, 0, s>>>(A);
    return cudaGetLastError();
}

cudaError_t launch_logprob_bwd(int64_t rows, int64_t V, const float *logits, int64_t ld,
                               const int32_t *tokens, const float *stats, const float *dlogp,
                               const float *dentropy, float *dlogits, int64_t ldd,
                               cudaStream_t s) {
    const dim3 grid(unsigned(std::min<int64_t>((V + kThreads - 1) / kThreads, 64)),
                    unsigned(std::min<int64_t>(rows, 65535)));
    logprob_bwd_kernel<<<grid, kThreads, 0, s>>>(rows, int(V), logits, ld, tokens,
                                                 reinterpret_cast<const float4 *>(stats), dlogp,
                                                 dentropy, dlogits, ldd);
    return cudaGetLastError();
}

}  // namespace det
