// logprob.cu -- log probabilities of given tokens under rows of logits, with
// entropy and the largest alternatives, and their gradient, for sm_103a.
//
//   m = max x_j,  e_j = exp(x_j - m),  S = the cross-entropy's 256-chain sum,
//   logp = (x_y - m) - log S,  entropy = log S - T / S,
//   T = sum e_j (x_j - m): chain j mod 4096 of each 16384 elements by fmaf from
//   +0, the blocks' chains added left to right from +0, then the tree
//   dx_j = dlogp ([j == y] - p_j) - dentropy p_j ((x_j - m) - log S + entropy)
//
// The forward reads each logit from memory once and writes a few floats a row,
// the gradient reads and writes each element once: HBM bounds both, with the exps
// close behind (about 14 instructions an element).
//
// Forward, rows of more than 4096 logits: one persistent CTA an SM, its warps in
// roles that follow one another down the rows, so that the max of one row, the
// exps of the row before and its sums run at the same time:
//   max    8 warps read a row straight from global memory (it stays in L2): its
//          max and the maxima of 32 groups of threads, up to three rows ahead
//   load   a lane brings the rows a second time, from L2, in segments of 2048
//          granules (row_stage.cuh) through a ring in shared memory
//   exp    16 warps: e in place and T's chains (a chain belongs to the thread that
//          owns its granules), and a list of the elements that may be alternatives
//   chain  4 warps: the 256 chains of S, a segment behind where a group straddles
//   final  a warp folds S and T, ranks the list and writes the row's results
// They meet at mbarriers only, every wait bounded. Staging whole rows and going
// through them phase by phase with all warps measured 2.6 times slower (874 us for
// 8192 x 50257 with 5 alternatives).
// Rows of at most 4096 logits: a warp a row, each chain of T one element.
// The alternatives: with t the top_k-th largest of 32 group maxima, at least
// top_k elements are >= t, and few more; they are listed while the exps are
// formed and ranked by (value, lowest id) with a count of the better ones. A list
// that overflows (many equal logits) or a row without a finite max is done by
// top_k maxima over the row instead. Neither way depends on the order of arrival.
// Gradient: a thread four granules of a row; the exps again from the row's m.
#include <algorithm>
#include <cstddef>

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
constexpr int kSeg = 2 * kSweep;        // granules of a segment
constexpr int kRing = 4;                // segments in shared memory
constexpr int kChainWarps = 4, kExpWarps = 16, kMaxWarps = 8;
constexpr int kChainThreads = kChainWarps * 32, kChains = kXentLanes / kChainThreads;
constexpr int kExpThreads = kExpWarps * 32, kMaxThreads = kMaxWarps * 32;
constexpr int kWarps = kChainWarps + kExpWarps + kMaxWarps + 2;
constexpr int kStreamThreads = kWarps * 32;
constexpr int kSets = kSweep / kExpThreads;  // granules a thread has in a sweep
constexpr int kMaxLoads = 8;            // granules a max thread reads at once
constexpr int kAhead = 3;               // rows whose max may wait for its exps
constexpr int kListed = 512;
constexpr int kSmallVocab = kTChains;   // a warp a row up to here
constexpr int kSmallWarps = 8, kSmallListed = 128;
constexpr unsigned kWatchdogLogprob = 64u;   // det_watchdog_status bit 6
constexpr float kInf = __builtin_inff();
static_assert(kSeg % kXentLanes == 0 && kTBlock % (4 * kSeg) == 0, "whole sweeps");

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
    int ahead;                  // 1: rows are prefetched into L2
};

// What a row's warp 0 lane writes of it, given S, T and the alternatives' ranks
// (lane k < top_k holds the k-th).
__device__ __forceinline__ void write_row(const LogprobArgs &A, int64_t row, const float *x, float m,
                                          float S, float T, uint64_t rank, int lane) {
    const float logS = det_log(S);
    const float ent = __fsub_rn(logS, __fdiv_rn(T, S));
    if (lane == 0) {
        const int y = A.tokens[row];
        const bool none = y == -1, wrong = !none && (y < 0 || y >= A.V);
        A.logp[row] = none    ? 0.0f
                      : wrong ? __uint_as_float(0x7fc00000u)
                              : __fsub_rn(__fsub_rn(x[y], m), logS);
        A.entropy[row] = ent;
        if (A.stats) A.stats[row] = make_float4(m, __fdiv_rn(1.0f, S), logS, ent);
        if (wrong && A.dev_status) atomicOr(reinterpret_cast<int *>(A.dev_status), 1);
    }
    if (lane < A.top_k) {
        const int j = id_of(rank);
        A.top_ids[row * A.top_k + lane] = j;
        A.top_logp[row * A.top_k + lane] = __fsub_rn(__fsub_rn(x[j], m), logS);
    }
}

// The alternatives one at a time, by one warp: each lane holds the best rank of
// its elements (j mod 32) below the last one taken; the winner's elements are
// looked through again by the whole warp. Returns the k-th rank in lane k.
__device__ __noinline__ uint64_t top_by_rounds(const float *x, int V, int top_k, int lane) {
    uint64_t mine = 0, got = 0;
    for (int j = lane; j < V; j += 32) {
        const uint64_t c = rank_of(x[j], j);
        mine = c > mine ? c : mine;
    }
    for (int k = 0; k < top_k; ++k) {
        const uint64_t best = warp_max(mine);
        if (lane == k) got = best;
        const int owner = __ffs(__ballot_sync(0xffffffffu, mine == best)) - 1;
        uint64_t r = 0;
        for (int j = owner + 32 * lane; j < V; j += 1024) {
            const uint64_t c = rank_of(x[j], j);
            if (c < best && c > r) r = c;
        }
        r = warp_max(r);
        if (lane == owner) mine = r;
    }
    return got;
}

// The bound for the list: the top_k-th largest of the lanes' values (group
// maxima), the lower lane first among equals.
__device__ __forceinline__ float list_bound(float v, int top_k, int lane) {
    int before = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float o = __shfl_sync(0xffffffffu, v, i);
        before += o > v || (o == v && i < lane);
    }
    const unsigned at = __ballot_sync(0xffffffffu, before == top_k - 1);
    return __shfl_sync(0xffffffffu, v, __ffs(at) - 1);
}

// The ranks of a list of n candidates in order: the k-th in lane k.
__device__ __forceinline__ uint64_t rank_list(const uint64_t *list, int n, int top_k,
                                              uint64_t *top, int lane) {
    for (int c0 = 0; c0 < n; c0 += 128) {
        uint64_t r[4];
        int better[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = c0 + 32 * i + lane < n ? list[c0 + 32 * i + lane] : 0;
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const uint64_t o = list[k];
#pragma unroll
            for (int i = 0; i < 4; ++i) better[i] += o > r[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r[i] && better[i] < top_k) top[better[i]] = r[i];
    }
    __syncwarp();
    return lane < top_k ? top[lane] : 0;
}

// e = exp(x - m) for the 4 elements of a granule and T's fmaf on their chains,
// for a finite m: exp4's bits. n = rint(d log2 e) sits in the low bits of tm, so
// p 2^n is p's bits plus tm's shifted up. Elements below the fast range (and
// -inf) take the general exp; e == 0 leaves T alone.
__device__ __forceinline__ float4 exp_and_t(float4 v, f32x2 m2, float m, float4 &t) {
    const f32x2 d01 = sub2(pack2(v.x, v.y), m2), d23 = sub2(pack2(v.z, v.w), m2);
    float d0, d1, d2, d3;
    unpack2(d01, d0, d1);
    unpack2(d23, d2, d3);
    const f32x2 magic = splat2(kRoundMagic);
    const f32x2 tm01 = add2(pack2(__fmul_rn(d0, kLog2e), __fmul_rn(d1, kLog2e)), magic);
    const f32x2 tm23 = add2(pack2(__fmul_rn(d2, kLog2e), __fmul_rn(d3, kLog2e)), magic);
    const f32x2 n01 = sub2(tm01, magic), n23 = sub2(tm23, magic);
    const f32x2 hi = splat2(-kLn2Hi), lo = splat2(-kLn2Lo);
    const f32x2 r01 = fma2(n01, lo, fma2(n01, hi, d01)), r23 = fma2(n23, lo, fma2(n23, hi, d23));
    f32x2 p01 = fma2(splat2(kC7), r01, splat2(kC6)), p23 = fma2(splat2(kC7), r23, splat2(kC6));
    p01 = fma2(p01, r01, splat2(kC5)); p23 = fma2(p23, r23, splat2(kC5));
    p01 = fma2(p01, r01, splat2(kC4)); p23 = fma2(p23, r23, splat2(kC4));
    p01 = fma2(p01, r01, splat2(kC3)); p23 = fma2(p23, r23, splat2(kC3));
    p01 = fma2(p01, r01, splat2(kC2)); p23 = fma2(p23, r23, splat2(kC2));
    p01 = fma2(p01, r01, splat2(1.0f)); p23 = fma2(p23, r23, splat2(1.0f));
    p01 = fma2(p01, r01, splat2(1.0f)); p23 = fma2(p23, r23, splat2(1.0f));
    float a0, a1, a2, a3, q0, q1, q2, q3;
    unpack2(tm01, a0, a1);
    unpack2(tm23, a2, a3);
    unpack2(p01, q0, q1);
    unpack2(p23, q2, q3);
    auto scaled = [](float p, float tm) {
        return __int_as_float(__float_as_int(p) + int(__float_as_uint(tm) << 23));
    };
    float4 e = make_float4(scaled(q0, a0), scaled(q1, a1), scaled(q2, a2), scaled(q3, a3));
    constexpr float kFast = kRoundMagic - 125.0f;        // n >= -125
    if (fminf(fminf(a0, a1), fminf(a2, a3)) >= kFast) {
        unpack2(fma2(pack2(e.x, e.y), d01, pack2(t.x, t.y)), t.x, t.y);
        unpack2(fma2(pack2(e.z, e.w), d23, pack2(t.z, t.w)), t.z, t.w);
    } else {
        if (!(a0 >= kFast)) e.x = det_exp_call(d0);
        if (!(a1 >= kFast)) e.y = det_exp_call(d1);
        if (!(a2 >= kFast)) e.z = det_exp_call(d2);
        if (!(a3 >= kFast)) e.w = det_exp_call(d3);
        if (e.x != 0.0f) t.x = __fmaf_rn(e.x, d0, t.x);
        if (e.y != 0.0f) t.y = __fmaf_rn(e.y, d1, t.y);
        if (e.z != 0.0f) t.z = __fmaf_rn(e.z, d2, t.z);
        if (e.w != 0.0f) t.w = __fmaf_rn(e.w, d3, t.w);
    }
    return e;
}

struct alignas(16) RowState {           // of the rows 0 and 1 mod 2 of a CTA
    float T[kTChains];
    uint64_t list[kListed];
    uint64_t top[32];
    float red[kXentLanes / 32];
    int listed;
};
struct RowMax {                         // of the rows 0 .. kAhead - 1 mod kAhead
    float parts[kMaxWarps][32];         // the max threads' own maxima
    float m, bound;
};
struct Stream {
    float4 ring[kRing][kSeg];
    RowState row[2];
    RowMax max[kAhead];
    uint64_t loaded[kRing], exped[kRing], freed[kRing];
    uint64_t parted[kAhead], maxed[kAhead], passed[kAhead], done[2], taken[2];
    int abort;
};

static_assert(sizeof(RowState) % 16 == 0 && offsetof(Stream, row) % 16 == 0 &&
                  offsetof(Stream, max) % 16 == 0 && offsetof(Stream, loaded) % 8 == 0 &&
                  offsetof(RowState, T) == 0 && sizeof(Stream) <= 227 * 1024,
              "16-byte reads of T, 8-byte barriers");

__device__ __forceinline__ void fence_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// The groups of chains l, l + kChainThreads, ... in a staged segment (granules at
// `at`, `next` the address of the granule after it), in ascending order. inner:
// every group is inside the row.
template <int H>
__device__ __forceinline__ void chain_segment(uint32_t at, uint32_t next, int l, int left,
                                              bool inner, float (&s)[kChains]) {
    if (inner) {
#pragma unroll
        for (int i = 0; i < kSeg / kChainThreads; ++i) {
            const int g = l + kChainThreads * i;
            const float4 c0 = lds4(at + 16u * g);
            const float4 c1 =
                H ? lds4(i + 1 < kSeg / kChainThreads || g + 1 < kSeg ? at + 16u * (g + 1) : next)
                  : c0;
            const float4 v = group_of<H>(c0, c1);
            float &c = s[i % kChains];
            c = __fadd_rn(__fadd_rn(__fadd_rn(__fadd_rn(c, v.x), v.y), v.z), v.w);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < kChains; ++k)
        for (int i = k; i < kSeg / kChainThreads; i += kChains) {
            const int g = l + kChainThreads * i;
            for (int j = 4 * g; j < min(left, 4 * g + 4); ++j) {
                const int at_j = j + H;      // past the segment: in the next one
                s[k] = __fadd_rn(s[k], lds1(at_j < 4 * kSeg ? at + 4u * at_j
                                                            : next + 4u * (at_j - 4 * kSeg)));
            }
        }
}

__global__ void __launch_bounds__(kStreamThreads, 1) logprob_stream_kernel(LogprobArgs A) {
    extern __shared__ __align__(128) unsigned char smem_raw[];
    Stream &sh = *reinterpret_cast<Stream *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = A.V;
    auto bar = [](uint64_t &b) { return smem_u32(&b); };
    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(bar(sh.loaded[i]), 1);
            mbar_init(bar(sh.exped[i]), kExpWarps);
            mbar_init(bar(sh.freed[i]), kChainWarps);
        }
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(bar(sh.parted[i]), kMaxWarps);
            mbar_init(bar(sh.maxed[i]), 1);
            mbar_init(bar(sh.passed[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(sh.done[i]), kExpWarps + kChainWarps);
            mbar_init(bar(sh.taken[i]), 1);
            sh.row[i].listed = 0;
        }
        sh.abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    volatile int *abort = &sh.abort;
    // waits of a whole warp; false once any wait of the CTA has given up
    auto wait = [&](uint64_t &b, uint32_t phase) {
        return __all_sync(0xffffffffu, mbar_wait_or_abort(bar(b), phase & 1u, abort)) != 0;
    };
    auto arrive = [&](uint64_t &b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(b));
    };
    auto start_of = [&](int64_t r) { return A.logits + r * A.ld; };
    auto shift_of = [](const float *x) {
        return int((reinterpret_cast<uintptr_t>(x) >> 2) & 3);
    };
    uint32_t k = 0, seg = 0;            // rows and segments done so far
    if (warp < kChainWarps) {
        // ---- the chains of S
        for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x, ++k) {
            const int h = shift_of(start_of(row)), ns = ((V + h + 3) / 4 + kSeg - 1) / kSeg;
            float S[kChains];
#pragma unroll
            for (int c = 0; c < kChains; ++c) S[c] = 0.0f;
            bool ok = true;
            for (int s = 0; s < ns && ok; ++s, ++seg) {
                ok = wait(sh.exped[seg % kRing], seg / kRing);
                if (h && s + 1 < ns && ok)
                    ok = wait(sh.exped[(seg + 1) % kRing], (seg + 1) / kRing);
                if (!ok) break;
                const uint32_t at = smem_u32(sh.ring[seg % kRing]);
                const uint32_t next = smem_u32(sh.ring[(seg + 1) % kRing]);
                const int left = V - 4 * kSeg * s;
                const bool inner = left >= 4 * kSeg;
                if (h == 0) chain_segment<0>(at, next, tid, left, inner, S);
                else if (h == 1) chain_segment<1>(at, next, tid, left, inner, S);
                else if (h == 2) chain_segment<2>(at, next, tid, left, inner, S);
                else chain_segment<3>(at, next, tid, left, inner, S);
                arrive(sh.freed[seg % kRing]);
            }
            if (!ok) break;
#pragma unroll
            for (int c = 0; c < kChains; ++c) {
                const float t = warp_butterfly_sum(S[c]);
                if (lane == 0) sh.row[k & 1].red[c * kChainWarps + warp] = t;
            }
            arrive(sh.done[k & 1]);
        }
    } else if (warp < kChainWarps + kExpWarps) {
        // ---- e in place, T, the list
        const int et = tid - kChainThreads;
        for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x, ++k) {
            const int h = shift_of(start_of(row)), nch = (V + h + 3) / 4;
            const int ns = (nch + kSeg - 1) / kSeg;
            RowState &R = sh.row[k & 1];
            if (!wait(sh.maxed[k % kAhead], k / kAhead)) break;
            if (k >= 2 && !wait(sh.taken[k & 1], k / 2 - 1)) break;
            const float m = sh.max[k % kAhead].m, bound = sh.max[k % kAhead].bound;
            const bool finite_m = fabsf(m) <= 0x1.fffffep127f;
            const f32x2 m2 = splat2(m);
            auto note = [&](float v, int j) {
                const int at = atomicAdd(&R.listed, 1);
                if (at < kListed) R.list[at] = rank_of(v, j);
            };
            float4 tb[kSets], tt[kSets];     // T of the current block, and in all
#pragma unroll
            for (int u = 0; u < kSets; ++u) tb[u] = tt[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            auto flush = [](float4 &t, float4 &b, int from, int to) {
                if (from <= 0 && 0 < to) { t.x = __fadd_rn(t.x, b.x); b.x = 0.0f; }
                if (from <= 1 && 1 < to) { t.y = __fadd_rn(t.y, b.y); b.y = 0.0f; }
                if (from <= 2 && 2 < to) { t.z = __fadd_rn(t.z, b.z); b.z = 0.0f; }
                if (from <= 3 && 3 < to) { t.w = __fadd_rn(t.w, b.w); b.w = 0.0f; }
            };
            bool ok = true;
            for (int s = 0; s < ns; ++s, ++seg) {
                ok = wait(sh.loaded[seg % kRing], seg / kRing);
                if (!ok) break;
                float4 *b = sh.ring[seg % kRing];
                // a block's first granule holds h elements of the block before
                const bool turn = s > 0 && s % (kTBlock / (4 * kSeg)) == 0;
                if (turn)
#pragma unroll
                    for (int u = 0; u < kSets; ++u)
                        flush(tt[u], tb[u], et + u * kExpThreads == 0 ? h : 0, 4);
                const int keep = turn && et == 0 ? h : 0;
                auto listing = [&](float4 v, int q) {
                    if (fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) >= bound) {
                        const int j0 = 4 * (s * kSeg + q) - h;
                        if (v.x >= bound) note(v.x, j0);
                        if (v.y >= bound) note(v.y, j0 + 1);
                        if (v.z >= bound) note(v.z, j0 + 2);
                        if (v.w >= bound) note(v.w, j0 + 3);
                    }
                };
                if (finite_m && s > 0 && 4 * kSeg * (s + 1) - h <= V) {
                    // every element is inside the row
#pragma unroll 1
                    for (int q0 = et; q0 < kSeg; q0 += kSweep) {
#pragma unroll
                        for (int u = 0; u < kSets; ++u) {
                            const int q = q0 + u * kExpThreads;
                            const float4 v = b[q];
                            b[q] = exp_and_t(v, m2, m, tb[u]);
                            listing(v, q);
                        }
                        if (keep && q0 == et) flush(tt[0], tb[0], 0, keep);
                    }
                } else {
                    // the row's ends, or a row without a finite max
#pragma unroll 1
                    for (int q0 = et; q0 < kSeg; q0 += kSweep) {
#pragma unroll
                        for (int u = 0; u < kSets; ++u) {
                            const int q = q0 + u * kExpThreads, j0 = 4 * (s * kSeg + q) - h;
                            if (s * kSeg + q >= nch) break;
                            const float4 v = b[q];
                            if (finite_m && j0 >= 0 && j0 + 3 < V) {
                                b[q] = exp_and_t(v, m2, m, tb[u]);
                                listing(v, q);
                                continue;
                            }
                            float e[4], t[4] = {tb[u].x, tb[u].y, tb[u].z, tb[u].w};
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const float d = __fsub_rn(comp(v, c), m);
                                e[c] = det_exp_call(d);
                                if (j0 + c >= 0 && j0 + c < V) {
                                    if (e[c] != 0.0f) t[c] = __fmaf_rn(e[c], d, t[c]);
                                    if (comp(v, c) >= bound) note(comp(v, c), j0 + c);
                                }
                            }
                            tb[u] = make_float4(t[0], t[1], t[2], t[3]);
                            b[q] = make_float4(e[0], e[1], e[2], e[3]);
                        }
                        if (keep && q0 == et) flush(tt[0], tb[0], 0, keep);
                    }
                }
                arrive(sh.exped[seg % kRing]);
            }
            if (!ok) break;
#pragma unroll
            for (int u = 0; u < kSets; ++u) {
                flush(tt[u], tb[u], 0, 4);
                const int c = 4 * (et + u * kExpThreads) - h;
                R.T[c & (kTChains - 1)] = tt[u].x;
                R.T[(c + 1) & (kTChains - 1)] = tt[u].y;
                R.T[(c + 2) & (kTChains - 1)] = tt[u].z;
                R.T[(c + 3) & (kTChains - 1)] = tt[u].w;
            }
            arrive(sh.done[k & 1]);
        }
    } else if (warp < kChainWarps + kExpWarps + kMaxWarps) {
        // ---- the max, and the 32 groups' (the lanes of the same number)
        const int mw = warp - kChainWarps - kExpWarps, mt = mw * 32 + lane;
        for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x, ++k) {
            RowMax &R = sh.max[k % kAhead];
            if (k >= kAhead && !wait(sh.passed[k % kAhead], k / kAhead - 1)) break;
            const float *x = start_of(row);
            const int h = shift_of(x);
            if (A.ahead && mt == 0 && row + gridDim.x < A.rows) {
                const float *y = start_of(row + gridDim.x);
                prefetch_granules_l2(y - shift_of(y), (V + shift_of(y) + 3) / 4);
            }
            const int lo = h ? 1 : 0, hi = (V + h) / 4;      // granules inside the row
            const float4 *xa = reinterpret_cast<const float4 *>(x - h);
            float m = -kInf;
            for (int q0 = lo + mt; q0 < hi; q0 += kMaxThreads * kMaxLoads) {
                float4 v[kMaxLoads];
#pragma unroll
                for (int u = 0; u < kMaxLoads; ++u)
                    if (q0 + u * kMaxThreads < hi) v[u] = __ldcg(xa + q0 + u * kMaxThreads);
#pragma unroll
                for (int u = 0; u < kMaxLoads; ++u)
                    if (q0 + u * kMaxThreads < hi)
                        m = max_nan(m, max_nan(max_nan(v[u].x, v[u].y), max_nan(v[u].z, v[u].w)));
            }
            // the elements before and after those granules
            const int head = h ? 4 - h : 0, tail = 4 * hi - h;
            if (mt < head) m = max_nan(m, x[mt]);
            if (mt >= 32 && tail + mt - 32 < V) m = max_nan(m, x[tail + mt - 32]);
            R.parts[mw][lane] = m;
            arrive(sh.parted[k % kAhead]);
            if (mw == 0) {
                if (!wait(sh.parted[k % kAhead], k / kAhead)) break;
                float g = R.parts[0][lane];
#pragma unroll
                for (int w = 1; w < kMaxWarps; ++w) g = max_nan(g, R.parts[w][lane]);
                float all = g;
#pragma unroll
                for (int off = 16; off >= 1; off >>= 1)
                    all = max_nan(all, __shfl_xor_sync(0xffffffffu, all, off));
                all = __fadd_rn(all, 0.0f);              // a zero maximum is +0
                const bool list = A.top_k > 0 && fabsf(all) <= 0x1.fffffep127f;
                const float bound = list ? list_bound(g, A.top_k, lane) : kInf;
                if (lane == 0) {
                    R.m = all;
                    R.bound = bound;
                }
                arrive(sh.maxed[k % kAhead]);
            }
        }
    } else if (warp == kWarps - 2) {
        // ---- the loads
        if (lane == 0) {
            bool ok = true;
            for (int64_t row = blockIdx.x; row < A.rows && ok; row += gridDim.x) {
                const float *x = start_of(row);
                const int h = shift_of(x), nch = (V + h + 3) / 4;
                for (int q = 0; q < nch; q += kSeg, ++seg) {
                    const int at = seg % kRing;
                    if (seg >= kRing &&
                        !mbar_wait_or_abort(bar(sh.freed[at]), (seg / kRing - 1) & 1u, abort)) {
                        ok = false;
                        break;
                    }
                    fence_async_shared();    // the exps written there come before the copy
                    load_granules(sh.ring[at] - q, x - h, q, min(nch, q + kSeg), &sh.loaded[at]);
                }
            }
        }
    } else {
        // ---- the results
        for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x, ++k) {
            RowState &R = sh.row[k & 1];
            if (!wait(sh.done[k & 1], k / 2)) break;
            const float *x = start_of(row);
            float T = 0.0f;
#pragma unroll 4
            for (int i = 0; i < 32; ++i) {
                const float4 c = *reinterpret_cast<const float4 *>(&R.T[4 * (32 * i + lane)]);
                const float t =
                    warp_butterfly_sum(__fadd_rn(__fadd_rn(__fadd_rn(c.x, c.y), c.z), c.w));
                if (lane == i) T = t;
            }
            T = warp_butterfly_sum(T);
            const float *t = R.red;
            const float S =
                __fadd_rn(__fadd_rn(__fadd_rn(t[0], t[1]), __fadd_rn(t[2], t[3])),
                          __fadd_rn(__fadd_rn(t[4], t[5]), __fadd_rn(t[6], t[7])));
            const float m = sh.max[k % kAhead].m;
            uint64_t rank = 0;
            if (A.top_k > 0)
                rank = R.listed > kListed || !(fabsf(m) <= 0x1.fffffep127f)
                           ? top_by_rounds(x, V, A.top_k, lane)
                           : rank_list(R.list, R.listed, A.top_k, R.top, lane);
            write_row(A, row, x, m, S, T, rank, lane);
            __syncwarp();
            if (lane == 0) R.listed = 0;
            arrive(sh.taken[k & 1]);
            arrive(sh.passed[k % kAhead]);
        }
    }
    __syncthreads();
    if (sh.abort && warp == kWarps - 2 && lane == 0) {     // let the copies in flight land
        atomicOr(&g_logprob_watchdog, kWatchdogLogprob);
        for (uint32_t i = seg > uint32_t(kRing) ? seg - kRing : 0; i < seg; ++i)
            (void)mbar_wait_bounded(bar(sh.loaded[i % kRing]), (i / kRing) & 1u);
    }
}

// A warp a row of at most 4096 logits, read once a pass (the row stays in L1); a
// lane has the groups lane + 32 w + 256 t, so chain lane + 32 w of S adds its
// groups in ascending t, and T's chains have an element each.
__global__ void __launch_bounds__(kSmallWarps * 32) logprob_small_kernel(LogprobArgs A) {
    __shared__ uint64_t lists[kSmallWarps][kSmallListed], tops[kSmallWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, V = A.V;
    for (int64_t row = blockIdx.x * int64_t(kSmallWarps) + warp; row < A.rows;
         row += gridDim.x * int64_t(kSmallWarps)) {
        const float *x = A.logits + row * A.ld;
        const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0;
        auto group = [&](int g, float fill) {
            const int j = 4 * g;
            if (vec && j + 3 < V) return *reinterpret_cast<const float4 *>(x + j);
            return make_float4(j < V ? x[j] : fill, j + 1 < V ? x[j + 1] : fill,
                               j + 2 < V ? x[j + 2] : fill, j + 3 < V ? x[j + 3] : fill);
        };
        float mine = -kInf;
#pragma unroll 8
        for (int g = lane; 4 * g < V; g += 32) {
            const float4 v = group(g, -kInf);
            mine = max_nan(mine, max_nan(max_nan(v.x, v.y), max_nan(v.z, v.w)));
        }
        float m = mine;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        m = __fadd_rn(m, 0.0f);              // a zero maximum is +0
        const bool finite_m = fabsf(m) <= 0x1.fffffep127f;
        const bool list = A.top_k > 0 && finite_m;
        const float bound = list ? list_bound(mine, A.top_k, lane) : kInf;
        const f32x2 m2 = splat2(m);
        float s[8], T = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s[w] = 0.0f;
        int listed = 0;
        for (int g0 = 0; 4 * g0 < V; g0 += kXentLanes) {
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                if (4 * (g0 + 32 * w) >= V) break;       // uniform across the warp
                const int g = g0 + 32 * w + lane, j = 4 * g;
                const float4 v = group(g, -kInf);
                float4 t = make_float4(0.f, 0.f, 0.f, 0.f), e = t;
                if (finite_m) {
                    e = exp_and_t(v, m2, m, t);          // e = 0 past the row's end
                } else if (j < V) {                      // every e of the row is NaN or 0
                    e.x = det_exp(__fsub_rn(v.x, m));
                    e.y = j + 1 < V ? det_exp(__fsub_rn(v.y, m)) : 0.0f;
                    e.z = j + 2 < V ? det_exp(__fsub_rn(v.z, m)) : 0.0f;
                    e.w = j + 3 < V ? det_exp(__fsub_rn(v.w, m)) : 0.0f;
                    if (e.x != 0.0f) t.x = __fmaf_rn(e.x, __fsub_rn(v.x, m), 0.0f);
                    if (e.y != 0.0f) t.y = __fmaf_rn(e.y, __fsub_rn(v.y, m), 0.0f);
                    if (e.z != 0.0f) t.z = __fmaf_rn(e.z, __fsub_rn(v.z, m), 0.0f);
                    if (e.w != 0.0f) t.w = __fmaf_rn(e.w, __fsub_rn(v.w, m), 0.0f);
                }
                s[w] = __fadd_rn(__fadd_rn(__fadd_rn(__fadd_rn(s[w], e.x), e.y), e.z), e.w);
                // each chain's one block, added to +0
                t.x = __fadd_rn(t.x, 0.0f);
                t.y = __fadd_rn(t.y, 0.0f);
                t.z = __fadd_rn(t.z, 0.0f);
                t.w = __fadd_rn(t.w, 0.0f);
                const float u =
                    warp_butterfly_sum(__fadd_rn(__fadd_rn(__fadd_rn(t.x, t.y), t.z), t.w));
                if (lane == g0 / 32 + w) T = u;
                if (list) {
                    const float best = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
                    if (__any_sync(0xffffffffu, best >= bound && j < V)) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const bool in = comp(v, c) >= bound && j + c < V;
                            const unsigned who = __ballot_sync(0xffffffffu, in);
                            const int at = listed + __popc(who & ((1u << lane) - 1u));
                            if (in && at < kSmallListed)
                                lists[warp][at] = rank_of(comp(v, c), j + c);
                            listed += __popc(who);
                        }
                    }
                }
            }
        }
        T = warp_butterfly_sum(T);
        float f[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) f[w] = warp_butterfly_sum(s[w]);
        const float S = __fadd_rn(__fadd_rn(__fadd_rn(f[0], f[1]), __fadd_rn(f[2], f[3])),
                                  __fadd_rn(__fadd_rn(f[4], f[5]), __fadd_rn(f[6], f[7])));
        uint64_t rank = 0;
        __syncwarp();
        if (A.top_k > 0)
            rank = !list || listed > kSmallListed
                       ? top_by_rounds(x, V, A.top_k, lane)
                       : rank_list(lists[warp], listed, A.top_k, tops[warp], lane);
        write_row(A, row, x, m, S, T, rank, lane);
        __syncwarp();
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
                     reinterpret_cast<float4 *>(stats), top_ids, top_logp, dev_status, 0};
    const int64_t sms = sm_count_current_device();
    if (V <= kSmallVocab) {
        const int64_t blocks = std::min<int64_t>((rows + kSmallWarps - 1) / kSmallWarps, sms * 8);
        logprob_small_kernel<<<unsigned(blocks), kSmallWarps * 32, 0, s>>>(A);
        return cudaGetLastError();
    }
    const int64_t grid = std::min<int64_t>(rows, sms);
    // the rows between max and exps in L2, and the next one asked for where it fits
    A.ahead = 3 * grid * V * 4 <= int64_t(96) << 20;
    const cudaError_t e = cudaFuncSetAttribute(
        logprob_stream_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(Stream)));
    if (e != cudaSuccess) return e;
    logprob_stream_kernel<<<unsigned(grid), kStreamThreads, sizeof(Stream), s>>>(A);
    return cudaGetLastError();
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
