// logprob.cu -- log probabilities of given tokens under rows of logits, with
// entropy and the largest alternatives, and their gradient, for sm_103a.
//
//   m = max x_j,  e_j = exp(x_j - m),  S = the cross-entropy's 256-chain sum,
//   logp = (x_y - m) - log S,  entropy = log S - T / S,
//   T = sum e_j (x_j - m): chain j mod 4096 of each 16384 elements by fmaf from
//   +0, the blocks' chains added left to right from +0, then the tree
//   dx_j = dlogp ([j == y] - p_j) - dentropy p_j ((x_j - m) - log S + entropy)
//
// The forward reads each logit once and writes a few floats a row, the gradient
// reads and writes each element once: HBM bounds both, with the exps close
// behind (about 14 instructions an element).
//
// Forward: a persistent CTA takes a row at a time in segments of whole granules
// (row_stage.cuh) through two shared-memory buffers filled by bulk copies; a row
// of at most 14,000 granules (56,000 floats; the 162M model has 50,257 ids) stays
// on chip and is read from memory once, a longer one comes a second time, from L2
// where it fits. Per segment: the max as it lands; then e in place and T's
// chains by all warps, an element's chain being fixed by the thread that owns its
// granule; then the 256 chains of S by the first 8 warps.
// The alternatives: with t the top_k-th largest of the maxima of 32 groups of
// threads, at least top_k elements are >= t, and few more; they are listed while the exps are
// formed and ranked by (value, lowest id) with a count of the better ones. A list
// that overflows (many equal logits) or a row without a finite max is done by
// top_k block-wide maxima instead. Neither way depends on the order of arrival.
// Gradient: a thread four granules of a row; the exps again from the row's m.
#include <algorithm>

#include "det_internal.cuh"
#include "det_math.cuh"
#include "row_stage.cuh"

namespace det {

// Set when a bounded wait for a row's segment gave up.
__device__ unsigned int g_logprob_watchdog;

namespace {

constexpr int kTChains = 4096;
constexpr int kTBlock = 16384;          // elements
constexpr int kSweep = kTChains / 4;    // granules that cover T's chains once
// Granules of a segment, whole sweeps of T's chains: rows of at most two segments
// stay on chip (the second buffer then holds what is left), longer ones take
// two buffers of the smaller size.
constexpr int kSegment = 7 * kSweep, kLongSegment = 6 * kSweep;
constexpr int kOnChip = 14000;          // granules of a row that stays
constexpr int kSmallRow = 1536;         // granules up to which 256 threads take a row
constexpr int kListed = 512;
constexpr unsigned kWatchdogLogprob = 64u;   // det_watchdog_status bit 6
constexpr float kInf = __builtin_inff();
static_assert(kSweep % kXentLanes == 0, "a chain goes on in the next segment");
static_assert(kOnChip <= 2 * kSegment && (kOnChip + 8) * 16 + 6144 <= 227 * 1024 &&
                  2 * (kLongSegment + 2) * 16 + 6144 <= 227 * 1024, "shared memory");

// Order of the alternatives as a key: larger logits have larger keys, +0 and -0
// the same, NaN the largest; the lower id wins among equal keys. A 64-bit rank
// holds both; 0 is below every rank.
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));    // -0 -> +0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t rank_of(float x, int j) {
    return uint64_t(key_of(x)) << 32 | uint32_t(~j);
}
__device__ __forceinline__ int id_of(uint64_t rank) { return int(~uint32_t(rank)); }

__device__ __forceinline__ uint64_t warp_max(uint64_t r) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, r, off);
        r = o > r ? o : r;
    }
    return r;
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
    int segment, segments;      // granules of a segment; segments of a row
};

struct Shared {
    uint64_t list[kListed];
    uint64_t top[32];
    uint64_t warp_best[32];
    float4 edge[32];            // T of each warp's first lane
    float red[32], tsum[32];
    float bound;                // elements at or above it are listed
    int listed;
    uint64_t bar[2];
};

// The alternatives one at a time: each thread holds the best rank of its
// elements below the last one taken; only the thread that had the winner looks
// through its elements again.
template <int NT>
__device__ __noinline__ void top_by_rounds(const float *x, int V, int top_k, Shared &sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto below = [&](uint64_t limit, bool all) {
        uint64_t r = 0;
        for (int j = tid; j < V; j += NT) {
            const uint64_t c = rank_of(x[j], j);
            if ((all || c < limit) && c > r) r = c;
        }
        return r;
    };
    uint64_t mine = below(0, true);
    for (int k = 0; k < top_k; ++k) {
        const uint64_t w = warp_max(mine);
        if (lane == 0) sh.warp_best[warp] = w;
        __syncthreads();
        uint64_t best = 0;
        for (int i = 0; i < NT / 32; ++i) best = sh.warp_best[i] > best ? sh.warp_best[i] : best;
        if (tid == 0) sh.top[k] = best;
        if (mine == best) mine = below(best, false);
        __syncthreads();
    }
}

template <int NT>
__global__ void __launch_bounds__(NT, NT == 1024 ? 1 : 4) logprob_kernel(LogprobArgs A) {
    constexpr int kWarps = NT / 32;
    constexpr int kSets = kSweep / NT;       // T's chains a thread carries: 4 a set
    extern __shared__ float4 row_buf[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = A.segments, V = A.V;
    const int loads = n <= 2 ? n : 2 * n;    // of a row
    float4 *const buf[2] = {row_buf, row_buf + A.segment + 2};
    auto start_of = [&](int64_t r) { return A.logits + r * A.ld; };
    auto shift_of = [](const float *x) {
        return int((reinterpret_cast<uintptr_t>(x) >> 2) & 3);
    };
    // load i of this CTA: row blockIdx.x + (i / loads) * gridDim.x, segment i mod
    // loads mod n, into buffer i mod 2; a segment takes along the first granule
    // of the next
    auto issue = [&](int64_t i) {
        const int64_t r = blockIdx.x + i / loads * gridDim.x;
        if (r >= A.rows) return;
        const int s = int(i % loads) % n;
        const float *x = start_of(r);
        const int h = shift_of(x), nch = (V + h + 3) >> 2;
        const int q0 = s * A.segment, q1 = min(nch, q0 + A.segment + 1);
        load_granules(buf[i & 1] - q0, x - h, q0, q1, &sh.bar[i & 1]);
    };
    if (tid == 0) {
        mbar_init(smem_u32(&sh.bar[0]), 1);
        mbar_init(smem_u32(&sh.bar[1]), 1);
        fence_mbar_init();
        issue(0);
        issue(1);
    }
    __syncthreads();
    int64_t first = 0;                       // this row's first load
    for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x, first += loads) {
        const float *x = start_of(row);
        const int h = shift_of(x), nch = (V + h + 3) >> 2;
        if (tid == 0 && n == 2 && row + gridDim.x < A.rows) {
            const float *nx = start_of(row + gridDim.x);
            prefetch_granules_l2(nx - shift_of(nx), (V + shift_of(nx) + 3) >> 2);
        }
        bool ok = true;
        auto wait = [&](int64_t i) {
            ok = mbar_wait_bounded(smem_u32(&sh.bar[i & 1]), uint32_t(i >> 1) & 1u) && ok;
        };
        // 1. the max, and each group of threads' own (elements outside the row left
        // out)
        float m = -kInf;
        for (int s = 0; s < n; ++s) {
            const int64_t i = first + s;
            wait(i);
            const float4 *b = buf[i & 1];
            const int q0 = s * A.segment, qn = (s + 1 < n ? A.segment : nch - q0);
            if (ok)
#pragma unroll 2
                for (int q = tid; q < qn; q += NT) {
                    const float4 v = b[q];
                    const int j0 = 4 * (q0 + q) - h;
                    if (j0 >= 0 && j0 + 3 < V) {
                        m = max_nan(m, max_nan(max_nan(v.x, v.y), max_nan(v.z, v.w)));
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (j0 + c >= 0 && j0 + c < V) m = max_nan(m, comp(v, c));
                    }
                }
            if (n > 2) {                     // the buffer is free for the load after next
                __syncthreads();
                if (tid == 0) issue(i + 2);
            }
        }
        constexpr int kGroup = NT / 32;      // lanes of a group
#pragma unroll
        for (int off = kGroup / 2; off >= 1; off >>= 1)
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (lane % kGroup == 0) sh.red[tid / kGroup] = m;
        if (tid == 0) sh.listed = 0;
        if (__syncthreads_or(!ok)) {
            if (tid == 0) {
                atomicOr(&g_logprob_watchdog, kWatchdogLogprob);
                for (int k = 0; k < 2; ++k)  // let the copies in flight land
                    for (uint32_t p = 0; p < 2; ++p)
                        (void)mbar_wait_bounded(smem_u32(&sh.bar[k]), p);
            }
            return;
        }
        const float wm = sh.red[lane];
        m = wm;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        m = __fadd_rn(m, 0.0f);              // a zero maximum is +0
        const bool finite_m = fabsf(m) <= 0x1.fffffep127f;
        float bound = kInf;
        if (A.top_k > 0 && finite_m) {       // the top_k-th largest of the groups'
            if (warp == 0) {
                int before = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float o = __shfl_sync(0xffffffffu, wm, i);
                    before += o > wm || (o == wm && i < lane);
                }
                if (before == A.top_k - 1) sh.bound = wm;
            }
            __syncthreads();
            bound = sh.bound;
        }
        // 2. e in place, T, the candidates, the chains of S
        float S = 0.0f;
        float4 tb[kSets], tt[kSets];         // T of the current block, and in all
#pragma unroll
        for (int u = 0; u < kSets; ++u) tb[u] = tt[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        auto flush = [&](float4 &t, float4 &b, int from, int to) {
            if (from <= 0 && 0 < to) { t.x = __fadd_rn(t.x, b.x); b.x = 0.0f; }
            if (from <= 1 && 1 < to) { t.y = __fadd_rn(t.y, b.y); b.y = 0.0f; }
            if (from <= 2 && 2 < to) { t.z = __fadd_rn(t.z, b.z); b.z = 0.0f; }
            if (from <= 3 && 3 < to) { t.w = __fadd_rn(t.w, b.w); b.w = 0.0f; }
        };
        auto note = [&](float v, int j) {
            const int at = atomicAdd(&sh.listed, 1);
            if (at < kListed) sh.list[at] = rank_of(v, j);
        };
        auto add_t = [](float &t, float e, float d) {
            if (e != 0.0f) t = __fmaf_rn(e, d, t);
        };
        for (int s = 0; s < n; ++s) {
            const int64_t i = first + (n <= 2 ? s : n + s);
            if (n > 2) wait(i);
            float4 *b = buf[i & 1];
            const int q0 = s * A.segment, own = s + 1 < n ? A.segment : nch - q0;
            // q0 + q = tid mod NT, so a thread's granules meet its own chains of T
            for (int q1 = 0; q1 < own; q1 += kSweep) {
#pragma unroll
                for (int u = 0; u < kSets; ++u) {
                    const int q = q1 + u * NT + tid;
                    if (q >= own) break;
                    const int g = q0 + q, j0 = 4 * g - h;
                    const int set = u;       // (g / NT) mod kSets, as q0 is whole sweeps
                    const float4 v = b[q];
                    // a granule that starts a block holds h elements of the last
                    const bool turn = g >= kTBlock / 4 && g % (kTBlock / 4) < kSweep;
                    const int keep = turn && g % (kTBlock / 4) == 0 ? h : 0;
                    if (turn) flush(tt[set], tb[set], keep, 4);
                    if (finite_m && j0 >= 0 && j0 + 3 < V) {
                        const f32x2 m2 = splat2(m);
                        const f32x2 x01 = pack2(v.x, v.y), x23 = pack2(v.z, v.w);
                        int n0, n1, n2, n3;
                        const f32x2 e01 = exp2_le0_fast(x01, m2, n0, n1);
                        const f32x2 e23 = exp2_le0_fast(x23, m2, n2, n3);
                        float4 e;
                        unpack2(e01, e.x, e.y);
                        unpack2(e23, e.z, e.w);
                        if (min(min(n0, n1), min(n2, n3)) >= -125) {
                            unpack2(fma2(e01, sub2(x01, m2), pack2(tb[set].x, tb[set].y)),
                                    tb[set].x, tb[set].y);
                            unpack2(fma2(e23, sub2(x23, m2), pack2(tb[set].z, tb[set].w)),
                                    tb[set].z, tb[set].w);
                        } else {
                            if (n0 < -125) e.x = det_exp_call(__fsub_rn(v.x, m));
                            if (n1 < -125) e.y = det_exp_call(__fsub_rn(v.y, m));
                            if (n2 < -125) e.z = det_exp_call(__fsub_rn(v.z, m));
                            if (n3 < -125) e.w = det_exp_call(__fsub_rn(v.w, m));
                            add_t(tb[set].x, e.x, __fsub_rn(v.x, m));
                            add_t(tb[set].y, e.y, __fsub_rn(v.y, m));
                            add_t(tb[set].z, e.z, __fsub_rn(v.z, m));
                            add_t(tb[set].w, e.w, __fsub_rn(v.w, m));
                        }
                        b[q] = e;
                        if (fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) >= bound) {
                            if (v.x >= bound) note(v.x, j0);
                            if (v.y >= bound) note(v.y, j0 + 1);
                            if (v.z >= bound) note(v.z, j0 + 2);
                            if (v.w >= bound) note(v.w, j0 + 3);
                        }
                        if (keep) flush(tt[set], tb[set], 0, keep);
                    } else {
                        float e[4], t[4] = {tb[set].x, tb[set].y, tb[set].z, tb[set].w};
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float d = __fsub_rn(comp(v, c), m);
                            e[c] = det_exp_call(d);
                            if (j0 + c >= 0 && j0 + c < V) {
                                add_t(t[c], e[c], d);
                                if (comp(v, c) >= bound) note(comp(v, c), j0 + c);
                            }
                        }
                        tb[set] = make_float4(t[0], t[1], t[2], t[3]);
                        b[q] = make_float4(e[0], e[1], e[2], e[3]);
                        if (keep) flush(tt[set], tb[set], 0, keep);
                    }
                }
            }
            if (tid == 0 && s + 1 < n) {     // the granule shared with the next segment
                const float4 v = b[own];
                b[own] = make_float4(
                    det_exp_call(__fsub_rn(v.x, m)), det_exp_call(__fsub_rn(v.y, m)),
                    det_exp_call(__fsub_rn(v.z, m)), det_exp_call(__fsub_rn(v.w, m)));
            }
            if (s + 1 == n) {
                // T's chains are complete; the sums in fours straddle two threads
                // where h > 0: the first lane's go to the lane before it
#pragma unroll
                for (int u = 0; u < kSets; ++u) flush(tt[u], tb[u], 0, 4);
                if (lane == 0)
#pragma unroll
                    for (int u = 0; u < kSets; ++u) sh.edge[u * kWarps + warp] = tt[u];
            }
            if (__syncthreads_or(!ok)) break;
            if (tid < kXentLanes) {
                const int left = s + 1 < n ? 4 * A.segment : V - 4 * q0;
                const uint32_t at = smem_u32(b);
                S = h == 0   ? xent_smem_chain<0>(at, left, S)
                    : h == 1 ? xent_smem_chain<1>(at, left, S)
                    : h == 2 ? xent_smem_chain<2>(at, left, S)
                             : xent_smem_chain<3>(at, left, S);
            }
            if (s + 1 < n) {
                __syncthreads();
                if (tid == 0) issue(i + 2);
            }
        }
        if (__syncthreads_or(!ok)) {         // the chains are done, or a wait gave up
            if (!ok || tid == 0) atomicOr(&g_logprob_watchdog, ok ? 0u : kWatchdogLogprob);
            if (tid == 0)
                for (int k = 0; k < 2; ++k)
                    for (uint32_t p = 0; p < 2; ++p)
                        (void)mbar_wait_bounded(smem_u32(&sh.bar[k]), p);
            return;
        }
        if (tid == 0) issue(first + (n == 1 ? 2 : n == 2 ? 3 : 2 * n + 1));
        // 3. the folds
        if (tid < kXentLanes) {
            S = warp_butterfly_sum(S);
            if (lane == 0) sh.red[warp] = S;
        }
#pragma unroll
        for (int u = 0; u < kSets; ++u) {
            const int w = u * kWarps + warp;             // 32 of the sums in fours
            float4 nx;
            nx.x = __shfl_down_sync(0xffffffffu, tt[u].x, 1);
            nx.y = __shfl_down_sync(0xffffffffu, tt[u].y, 1);
            nx.z = __shfl_down_sync(0xffffffffu, tt[u].z, 1);
            nx.w = 0.0f;
            if (lane == 31) nx = sh.edge[(w + 1) & 31];
            const float4 c = h == 0   ? group_of<0>(tt[u], nx)
                             : h == 1 ? group_of<1>(tt[u], nx)
                             : h == 2 ? group_of<2>(tt[u], nx)
                                      : group_of<3>(tt[u], nx);
            const float t = warp_butterfly_sum(__fadd_rn(__fadd_rn(__fadd_rn(c.x, c.y), c.z), c.w));
            if (lane == 0) sh.tsum[w] = t;
        }
        const bool rounds = A.top_k > 0 && (!finite_m || sh.listed > kListed);
        if (A.top_k > 0 && !rounds) {
            const int listed = sh.listed;
            for (int c = tid; c < listed; c += NT) {
                const uint64_t r = sh.list[c];
                int better = 0;
                for (int k = 0; k < listed; ++k) better += sh.list[k] > r;
                if (better < A.top_k) sh.top[better] = r;
            }
        }
        __syncthreads();
        if (rounds) top_by_rounds<NT>(x, V, A.top_k, sh);      // ends with a barrier
        if (warp == 0) {
            const float *t = sh.red;
            const float Sum =
                __fadd_rn(__fadd_rn(__fadd_rn(t[0], t[1]), __fadd_rn(t[2], t[3])),
                          __fadd_rn(__fadd_rn(t[4], t[5]), __fadd_rn(t[6], t[7])));
            const float Ts = warp_butterfly_sum(sh.tsum[lane]);
            const float logS = det_log(Sum);
            const float ent = __fsub_rn(logS, __fdiv_rn(Ts, Sum));
            if (lane == 0) {
                const int y = A.tokens[row];
                const bool none = y == -1, wrong = !none && (y < 0 || y >= V);
                A.logp[row] = none    ? 0.0f
                              : wrong ? __uint_as_float(0x7fc00000u)
                                      : __fsub_rn(__fsub_rn(x[y], m), logS);
                A.entropy[row] = ent;
                if (A.stats) A.stats[row] = make_float4(m, __fdiv_rn(1.0f, Sum), logS, ent);
                if (wrong && A.dev_status) atomicOr(reinterpret_cast<int *>(A.dev_status), 1);
            }
            if (lane < A.top_k) {
                const int j = id_of(sh.top[lane]);
                A.top_ids[row * A.top_k + lane] = j;
                A.top_logp[row * A.top_k + lane] = __fsub_rn(__fsub_rn(x[j], m), logS);
            }
        }
        __syncthreads();                     // red, tsum, list and top are used again
    }
}

constexpr int kBwdThreads = 256;
constexpr int kBwdGranules = 4;              // of a thread

template <bool ENT>
__device__ __forceinline__ float grad_of(float x, float e, float hot, const float4 &st, float g,
                                         float gH, bool none) {
    const float p = __fmul_rn(e, st.y);
    float a = none ? 0.0f : __fmul_rn(g, __fsub_rn(hot, p));
    if (ENT) {
        const float w = __fmul_rn(p, __fadd_rn(__fsub_rn(__fsub_rn(x, st.x), st.z), st.w));
        a = __fsub_rn(a, __fmul_rn(gH, p == 0.0f ? 0.0f : w));
    }
    return a;
}

template <bool ENT>
__global__ void __launch_bounds__(kBwdThreads)
    logprob_bwd_kernel(int64_t rows, int V, const float *logits, int64_t ld,
                       const int32_t *__restrict__ tokens, const float4 *__restrict__ stats,
                       const float *__restrict__ dlogp, const float *__restrict__ dentropy,
                       float *dlogits, int64_t ldd) {
    const int tid = threadIdx.x;
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const float *x = logits + row * ld;
        float *dx = dlogits + row * ldd;
        const int h = int((reinterpret_cast<uintptr_t>(x) >> 2) & 3), nch = (V + h + 3) >> 2;
        const bool vec = int((reinterpret_cast<uintptr_t>(dx) >> 2) & 3) == h;
        const int q0 = blockIdx.x * (kBwdThreads * kBwdGranules) + tid;
        float4 v[kBwdGranules];
#pragma unroll
        for (int u = 0; u < kBwdGranules; ++u) {
            const int q = q0 + u * kBwdThreads;
            if (q < nch) v[u] = __ldcs(reinterpret_cast<const float4 *>(x - h) + q);
        }
        const float4 st = stats[row];
        const int y = tokens[row];
        const bool none = y == -1, wrong = !none && (y < 0 || y >= V);
        const float g = wrong ? __uint_as_float(0x7fc00000u) : none ? 0.0f : dlogp[row];
        const float gH = ENT ? dentropy[row] : 0.0f;
        const bool finite_m = fabsf(st.x) <= 0x1.fffffep127f;
#pragma unroll
        for (int u = 0; u < kBwdGranules; ++u) {
            const int q = q0 + u * kBwdThreads, j0 = 4 * q - h;
            if (q >= nch) break;
            float4 e;
            if (finite_m) {
                e = exp4(v[u], st.x);
            } else {
                e = make_float4(
                    det_exp_call(__fsub_rn(v[u].x, st.x)), det_exp_call(__fsub_rn(v[u].y, st.x)),
                    det_exp_call(__fsub_rn(v[u].z, st.x)), det_exp_call(__fsub_rn(v[u].w, st.x)));
            }
            float4 o;
            o.x = grad_of<ENT>(v[u].x, e.x, j0 == y ? 1.0f : 0.0f, st, g, gH, none);
            o.y = grad_of<ENT>(v[u].y, e.y, j0 + 1 == y ? 1.0f : 0.0f, st, g, gH, none);
            o.z = grad_of<ENT>(v[u].z, e.z, j0 + 2 == y ? 1.0f : 0.0f, st, g, gH, none);
            o.w = grad_of<ENT>(v[u].w, e.w, j0 + 3 == y ? 1.0f : 0.0f, st, g, gH, none);
            if (wrong) o.x = o.y = o.z = o.w = g;
            if (vec && j0 >= 0 && j0 + 3 < V) {
                __stcs(reinterpret_cast<float4 *>(dx + j0), o);
            } else {
                if (j0 >= 0 && j0 < V) dx[j0] = o.x;
                if (j0 + 1 >= 0 && j0 + 1 < V) dx[j0 + 1] = o.y;
                if (j0 + 2 >= 0 && j0 + 2 < V) dx[j0 + 2] = o.z;
                if (j0 + 3 >= 0 && j0 + 3 < V) dx[j0 + 3] = o.w;
            }
        }
    }
}

}  // namespace

cudaError_t logprob_watchdog(unsigned int *code, int clear) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_logprob_watchdog, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    if (clear && *code) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_logprob_watchdog, &zero, sizeof(unsigned int));
    }
    return e;
}

cudaError_t launch_logprob(int64_t rows, int64_t V, const float *logits, int64_t ld,
                           const int32_t *tokens, int top_k, float *logp, float *entropy,
                           float *stats, int32_t *top_ids, float *top_logp, int32_t *dev_status,
                           cudaStream_t s) {
    LogprobArgs A = {rows, int(V), logits, ld, tokens, top_k, logp, entropy,
                     reinterpret_cast<float4 *>(stats), top_ids, top_logp, dev_status, 0, 0};
    const int groups = int((V + 3) / 4), most = int((V + 6) / 4);     // most: granules
    A.segment = std::min(most <= kOnChip ? kSegment : kLongSegment, groups);
    A.segments = (groups + A.segment - 1) / A.segment;
    const size_t smem =
        16 * (A.segments == 2 ? size_t(most) + 4 : size_t(2) * (A.segment + 2));
    const int sms = sm_count_current_device();
    // small rows: four CTAs of 256 threads an SM, so a row's barriers overlap
    const bool small = groups <= kSmallRow;
    auto run = [&](auto kern, int threads, int per_sm) {
        const cudaError_t e = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
        kern<<<unsigned(std::min<int64_t>(rows, int64_t(sms) * per_sm)), threads, smem, s>>>(A);
        return cudaGetLastError();
    };
    return small ? run(logprob_kernel<256>, 256, 4) : run(logprob_kernel<1024>, 1024, 1);
}

cudaError_t launch_logprob_bwd(int64_t rows, int64_t V, const float *logits, int64_t ld,
                               const int32_t *tokens, const float *stats, const float *dlogp,
                               const float *dentropy, float *dlogits, int64_t ldd,
                               cudaStream_t s) {
    const int64_t per = kBwdThreads * kBwdGranules, granules = (V + 6) / 4;
    const dim3 grid(unsigned((granules + per - 1) / per), unsigned(std::min<int64_t>(rows, 65535)));
    const auto *st = reinterpret_cast<const float4 *>(stats);
    if (dentropy)
        logprob_bwd_kernel<true><<<grid, kBwdThreads, 0, s>>>(rows, int(V), logits, ld, tokens, st,
                                                              dlogp, dentropy, dlogits, ldd);
    else
        logprob_bwd_kernel<false><<<grid, kBwdThreads, 0, s>>>(rows, int(V), logits, ld, tokens,
                                                               st, dlogp, dentropy, dlogits, ldd);
    return cudaGetLastError();
}

}  // namespace det
