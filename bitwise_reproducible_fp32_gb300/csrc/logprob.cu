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
// roles that follow one another down the rows, so that the max of one row and the
// exps and sums of the row before run at the same time:
//   max    8 warps read a row straight from global memory (it stays in L2): its
//          max and the maxima of 32 groups of threads, ahead of the sums
//   load   a lane brings the rows a second time, from L2, which may drop them then,
//          in segments of 4096 elements through a ring in shared memory
//   sum    8 warps, thread l the profile's chain l: groups of 4 elements two at a
//          time, straight-line, step by step over both: e, the chain of S, T's 16
//          chains of the thread, and a list of the groups that may hold alternatives
//   final  a warp folds the totals, ranks the list and writes the row's results
// Two teams of load, sum and final warps take every other row. They meet at
// mbarriers only, every wait bounded. us for 8192 x 50257 / 16384 x 16000 /
// 2720 x 151936 with 5 alternatives: 544 / 364 / 513 (3.0, 2.9, 3.2 TB/s; longer
// rows outgrow L2 between their readings, which is what bounds them: the second
// reading kept in L2 556 / 363 / 523, the next row prefetched 576 / 364 / 695); one
// team, four groups at a time 576 / 410 / 564; 16 warps of exps handing e to 8
// warps of chains through shared memory 668 / 582 / 501; whole rows staged and
// gone through phase by phase by all warps 874 / 788 / 846. Both roles are busy
// nearly all of the time: the sums by the latency between their steps, the max by
// that of its loads; instructions issue in 48% of the cycles. All 28 warps have the
// same 72 registers, too few for the sums, which spill 172 bytes.
// Few rows of more than 4096 logits: a cluster of 4..16 CTAs a row (below).
// Rows of at most 4096 logits: a warp a row, each chain of T one element (with 5
// alternatives 2048 x 256: 5.5 us, 16384 x 256: 16, 65536 x 1000: 172, of which 38
// are the alternatives'). A row that does not fill its last sweep pays for it: what
// is past its end counts as -inf, and the exps of a thread that has any of it are
// formed again in the general way (65536 x 1024: 124 us; 32768 x 4000: 202, 32768 x
// 4096: 162).
// The alternatives: with t the top_k-th largest of 32 (or 64) group maxima, at least
// top_k elements are >= t, and few more; they are listed while the exps are
// formed and ranked by (value, lowest id) with a count of the better ones. A list
// that overflows or a row without a finite max is done by top_k maxima over the row
// instead, by one warp. Neither way depends on the order of arrival. Lists overflow
// with many equal logits, and where fewer than top_k groups hold a logit above -inf
// (t is -inf then): in rows masked down to a few tokens, and over a cluster of 16 in
// rows of at most 8192 logits, of 8 in rows of at most 6144, whose shares leave groups
// empty (8 x 8000 for 16 alternatives 7.8 us, for 17 30).
// Masks: a -inf among a thread's 8 elements takes all 8 through the general exps. us
// for 5 / 20 alternatives with nothing, half, 99% and all but 10 masked: 8192 x 50257
// 544 / 589, 1913 / 1931, 1505 / 1532, 1347 / 5152; 64 x 50257 15 / 16, 19 / 20,
// 19 / 20, 18 / 151.
// Gradient: a thread four granules of a row; the exps again from the row's m (8192 x
// 50257 with the entropy's 483 us, 6.8 TB/s, the rate of a copy).
#include <cooperative_groups.h>

#include <algorithm>
#include <cstddef>

#include "det_internal.cuh"
#include "det_math.cuh"
#include "row_stage.cuh"

namespace cg = cooperative_groups;

namespace det {

// Set when a bounded wait for a row's segment gave up.
__device__ unsigned int g_logprob_watchdog;

namespace {

constexpr int kTChains = 4096;
constexpr int kTBlock = 16384;          // elements
constexpr int kSeg = kTChains / 4;      // groups of a segment: T's chains once
constexpr int kTeams = 2;               // teams of sum warps, a row each
constexpr int kRing = 3;                // segments of a team in shared memory
constexpr int kSumWarps = kXentLanes / 32, kMaxWarps = 8;
constexpr int kMaxThreads = kMaxWarps * 32;
constexpr int kFirstMax = kTeams * kSumWarps, kFirstLoad = kFirstMax + kMaxWarps;
constexpr int kFirstFinal = kFirstLoad + kTeams, kWarps = kFirstFinal + kTeams;
constexpr int kStreamThreads = kWarps * 32;
constexpr int kSets = kSeg / kXentLanes;     // groups a thread has in a segment
constexpr int kMaxLoads = 8;            // granules a max thread reads at once
// Rows between the start of the max and the results. A team waits on every other
// use of a max slot only; the use between is of a row before the team's last one,
// so it is over by then.
constexpr int kAhead = 3;
constexpr int kRounds = 8;               // alternatives whose bound is found in rounds
constexpr int kFound = 256, kListed = 512;    // granules, elements that may be alternatives
constexpr int kSmallVocab = kTChains;   // a warp a row up to here
constexpr int kSmallWarps = 8, kSmallListed = 128;
constexpr unsigned kWatchdogLogprob = 64u;   // det_watchdog_status bit 6
constexpr float kInf = __builtin_inff();
static_assert(kSets * kSumWarps == 32 && kTBlock % kTChains == 0, "T's tree and blocks");

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

// max / min of three (NaN-propagating where it forms the row's max).
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max4(float4 v) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(v.x), "f"(v.y), "f"(v.z));
    return fmaxf(r, v.w);
}
__device__ __forceinline__ float min4(float a, float b, float c, float d) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return fminf(r, d);
}
__device__ __forceinline__ float more_max(float m, float4 v) {
    return max3_nan(max3_nan(m, v.x, v.y), v.z, v.w);
}

// Eight butterflies 16..1 at once: in each level the two halves of the warp go
// on with different values, so 9 shuffles serve instead of 40; the additions are
// the butterfly's. Returns the total of v[row_of_lane(lane)].
__device__ __forceinline__ float butterfly8(float (&v)[8], int lane) {
#pragma unroll
    for (int half = 4, off = 16; half >= 1; half >>= 1, off >>= 1) {
        const bool up = lane & off;
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float keep = up ? v[i + half] : v[i], send = up ? v[i] : v[i + half];
            v[i] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, send, off));
        }
    }
    float t = __fadd_rn(v[0], __shfl_xor_sync(0xffffffffu, v[0], 2));
    return __fadd_rn(t, __shfl_xor_sync(0xffffffffu, t, 1));
}
// The lane that holds the total of v[w] then (among others).
__device__ __forceinline__ int lane_of_row(int w) {
    return (w & 4) << 2 | (w & 2) << 2 | (w & 1) << 2;
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

// The logit whose rank this is (+0 for -0, which x - m does not tell apart).
__device__ __forceinline__ float logit_of(uint64_t rank) {
    const uint32_t k = uint32_t(rank >> 32);
    if (k == 0xffffffffu) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// A row's token and its logit, asked for before the sums are there.
struct Asked {
    int y;
    float x;
};
__device__ __forceinline__ Asked ask(const LogprobArgs &A, int64_t row, const float *x) {
    Asked a = {A.tokens[row], 0.0f};
    if (a.y >= 0 && a.y < A.V) a.x = x[a.y];
    return a;
}

// What a warp writes of a row, given S, T and the alternatives' ranks (lane
// k < top_k holds the k-th).
__device__ __forceinline__ void write_row(const LogprobArgs &A, int64_t row, Asked a, float m,
                                          float S, float T, uint64_t rank, int lane) {
    const float logS = det_log(S);
    const float ent = __fsub_rn(logS, __fdiv_rn(T, S));
    if (lane == 0) {
        const bool none = a.y == -1, wrong = !none && (a.y < 0 || a.y >= A.V);
        A.logp[row] = none    ? 0.0f
                      : wrong ? __uint_as_float(0x7fc00000u)
                              : __fsub_rn(__fsub_rn(a.x, m), logS);
        A.entropy[row] = ent;
        if (A.stats) A.stats[row] = make_float4(m, __fdiv_rn(1.0f, S), logS, ent);
        if (wrong && A.dev_status) atomicOr(reinterpret_cast<int *>(A.dev_status), 1);
    }
    if (lane < A.top_k) {
        A.top_ids[row * A.top_k + lane] = id_of(rank);
        A.top_logp[row * A.top_k + lane] = __fsub_rn(__fsub_rn(logit_of(rank), m), logS);
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
// maxima), the lower lane first among equals; for few by rounds (5 alternatives of
// 16384 x 256 17 us, by counting 20.5; 20 the same either way).
__device__ __forceinline__ float list_bound(float v, int top_k, int lane) {
    if (top_k <= kRounds) {              // one maximum after the other
        uint32_t key = key_of(v);
        for (int k = 1;; ++k) {
            const uint32_t best = __reduce_max_sync(0xffffffffu, key);
            const int who = __ffs(__ballot_sync(0xffffffffu, key == best)) - 1;
            if (k == top_k) return __shfl_sync(0xffffffffu, v, who);
            if (lane == who) key = 0;
        }
    }
    int before = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float o = __shfl_sync(0xffffffffu, v, i);
        before += o > v || (o == v && i < lane);
    }
    const unsigned at = __ballot_sync(0xffffffffu, before == top_k - 1);
    return __shfl_sync(0xffffffffu, v, __ffs(at) - 1);
}

// The same of 64 groups, two a lane. The best elements fall on groups as they
// come: until 32 groups have one, about 130 have been seen, and now and then more
// than a list holds; until 32 of 64 have one, about 44. So this one serves calls
// for more than kFewAlternatives (8192 x 50257 for 32: 1158 us -> 628).
constexpr int kFewAlternatives = 24;
__device__ __noinline__ float list_bound_64(float v, float w, int top_k, int lane) {
    int v_before = 0, w_before = 0;
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
        const float a = __shfl_sync(0xffffffffu, v, i), b = __shfl_sync(0xffffffffu, w, i);
        v_before += (a > v || (a == v && i < lane)) + (b > v);
        w_before += (a >= w) + (b > w || (b == w && i < lane));
    }
    const unsigned in_v = __ballot_sync(0xffffffffu, v_before == top_k - 1);
    const unsigned in_w = __ballot_sync(0xffffffffu, w_before == top_k - 1);
    const float of_v = __shfl_sync(0xffffffffu, v, in_v ? __ffs(in_v) - 1 : 0);
    const float of_w = __shfl_sync(0xffffffffu, w, in_w ? __ffs(in_w) - 1 : 0);
    return in_v ? of_v : of_w;
}

// The ranks of a list of n candidates in order: the k-th in lane k.
__device__ __forceinline__ uint64_t rank_list(const uint64_t *list, int n, int top_k,
                                              uint64_t *top, int lane) {
    if (n <= 32) {                       // as nearly always: one a lane
        const uint64_t r = lane < n ? list[lane] : 0;
        int better = 0;
        for (int k = 0; k < n; ++k) better += list[k] > r;
        if (r && better < top_k) top[better] = r;
        __syncwarp();
        return lane < top_k ? top[lane] : 0;
    }
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

// e = exp(x - m) for N groups of 4 elements and T's fmaf on their chains, for a
// finite m, without branches and step by step over all of them, so that each
// instruction finds 2N independent ones around it. exp4's bits where the returned
// value, the least n = rint(d log2 e) plus kRoundMagic, is at least kFast; below
// (and at -inf) both are formed again by exp_slow from the old t. n sits in the
// low bits of tm, so p 2^n is p's bits plus tm's shifted up.
constexpr float kFast = kRoundMagic - 125.0f;
template <int N>
__device__ __forceinline__ float exp_and_t(const float4 (&v)[N], f32x2 m2, float4 (&e)[N],
                                           float4 (&t)[N]) {
    f32x2 d[2 * N], tm[2 * N], p[2 * N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        d[2 * i] = sub2(pack2(v[i].x, v[i].y), m2);
        d[2 * i + 1] = sub2(pack2(v[i].z, v[i].w), m2);
    }
    // d log2 e rounded on its own by scalar multiplies: a packed multiply that feeds a
    // packed add rounds as if fused with it, and so does a packed fma with -0
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) {
        float d0, d1;
        unpack2(d[i], d0, d1);
        tm[i] = pack2(__fmul_rn(d0, kLog2e), __fmul_rn(d1, kLog2e));
    }
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) tm[i] = add2(tm[i], splat2(kRoundMagic));
    f32x2 n[2 * N], r[2 * N];
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) n[i] = sub2(tm[i], splat2(kRoundMagic));
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) r[i] = fma2(n[i], splat2(-kLn2Hi), d[i]);
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) r[i] = fma2(n[i], splat2(-kLn2Lo), r[i]);
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) p[i] = fma2(splat2(kC7), r[i], splat2(kC6));
    auto step = [&](float c) {
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) p[i] = fma2(p[i], r[i], splat2(c));
    };
    step(kC5);
    step(kC4);
    step(kC3);
    step(kC2);
    step(1.0f);
    step(1.0f);
    float least = kInf;
    auto scaled = [](float q, float a) {
        return __int_as_float(__float_as_int(q) + int(__float_as_uint(a) << 23));
    };
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float a0, a1, a2, a3, q0, q1, q2, q3;
        unpack2(tm[2 * i], a0, a1);
        unpack2(tm[2 * i + 1], a2, a3);
        unpack2(p[2 * i], q0, q1);
        unpack2(p[2 * i + 1], q2, q3);
        least = fminf(least, min4(a0, a1, a2, a3));
        e[i] = make_float4(scaled(q0, a0), scaled(q1, a1), scaled(q2, a2), scaled(q3, a3));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        unpack2(fma2(pack2(e[i].x, e[i].y), d[2 * i], pack2(t[i].x, t[i].y)), t[i].x, t[i].y);
        unpack2(fma2(pack2(e[i].z, e[i].w), d[2 * i + 1], pack2(t[i].z, t[i].w)), t[i].z, t[i].w);
    }
    return least;
}

// The general form of it, for any m: elements with e == 0 leave T alone. e in
// the first half, the new t in the second.
struct ExpT { float4 e, t; };
__device__ __noinline__ ExpT exp_slow(float4 v, float m, float4 t) {
    float e[4], c[4] = {t.x, t.y, t.z, t.w};
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const float d = __fsub_rn(comp(v, i), m);
        const float x = det_exp(d);
        const float y = x != 0.0f ? __fmaf_rn(x, d, i == 0 ? c[0] : i == 1 ? c[1] : i == 2 ? c[2] : c[3])
                                  : (i == 0 ? c[0] : i == 1 ? c[1] : i == 2 ? c[2] : c[3]);
        if (i == 0) { e[0] = x; c[0] = y; }
        if (i == 1) { e[1] = x; c[1] = y; }
        if (i == 2) { e[2] = x; c[2] = y; }
        if (i == 3) { e[3] = x; c[3] = y; }
    }
    return {make_float4(e[0], e[1], e[2], e[3]), make_float4(c[0], c[1], c[2], c[3])};
}

// One thread: copies granules [q0, q1) of the row whose aligned base is xa into
// the same granules of buf, completing on bar; the row is not read again, so L2
// may drop it first.
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

struct RowState {                       // of the rows 0 and 1 mod 2 of a CTA
    float4 found[kFound];               // the listed groups, and where they start
    int found_at[kFound];
    uint64_t list[kListed], top[32];
    float red[kSumWarps], tsum[32];
    int listed, pad[3];
};
struct RowMax {                         // of the rows 0 .. kAhead - 1 mod kAhead
    float parts[kMaxWarps][32];         // the max threads' own maxima
    float m, bound, pad[2];
};
struct Team {
    float4 ring[kRing][kSeg + 1];       // a segment and the granule after it
    float4 T[kSets][kXentLanes];        // each thread's chains over the blocks so far
    RowState row[2];
    uint64_t loaded[kRing], freed[kRing], done[2], taken[2];
};
struct Stream {
    Team team[kTeams];
    RowMax max[kAhead];
    uint64_t parted[kAhead], maxed[kAhead], passed[kAhead];
    int abort;
};
static_assert(sizeof(RowState) % 16 == 0 && sizeof(RowMax) % 16 == 0 && sizeof(Team) % 16 == 0 &&
                  offsetof(Team, T) % 16 == 0 && offsetof(Team, row) % 16 == 0 &&
                  offsetof(Team, loaded) % 8 == 0 && offsetof(Stream, max) % 16 == 0 &&
                  offsetof(Stream, parted) % 8 == 0 && sizeof(Stream) <= 227 * 1024,
              "16-byte reads, 8-byte barriers");

// A thread's chain of S over one row, its groups l + 256 i of the segments, and its
// chains of T: 4 sums in fours. H: the row's misalignment. wait(segment number)
// and freed(segment number) are the ring's barriers; false when a wait gave up.
struct RowSums { float S, u[kSets]; };
template <int H, class Wait, class Freed>
__device__ __forceinline__ bool sum_row(Team &team, RowState &R, int V, float m, float bound,
                                        uint32_t &seg, Wait wait, Freed freed, RowSums &out) {
    constexpr int kPair = 2;                 // sets taken at once
    const int l = threadIdx.x % kXentLanes, ns = (V + 4 * kSeg - 1) / (4 * kSeg);
    const bool finite_m = fabsf(m) <= 0x1.fffffep127f;
    const f32x2 m2 = splat2(m);
    float S = 0.0f;
    float4 t[kSets];                         // T of the current block
#pragma unroll
    for (int u = 0; u < kSets; ++u) t[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    bool fresh = true;                       // team.T holds nothing of this row
    auto flush = [&](int u) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!fresh) a = team.T[u][l];
        a = make_float4(__fadd_rn(a.x, t[u].x), __fadd_rn(a.y, t[u].y), __fadd_rn(a.z, t[u].z),
                        __fadd_rn(a.w, t[u].w));
        t[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        return a;
    };
    for (int s = 0; s < ns; ++s, ++seg) {
        if (!wait(seg)) return false;
        const uint32_t at = smem_u32(team.ring[seg % kRing]) + 16u * l;
        if (s > 0 && s % (kTBlock / kTChains) == 0) {
#pragma unroll
            for (int u = 0; u < kSets; ++u) team.T[u][l] = flush(u);
            fresh = false;
        }
        const bool tail = 4 * kSeg * (s + 1) > V;
        const int j0 = 4 * (s * kSeg + l);
#pragma unroll
        for (int u0 = 0; u0 < kSets; u0 += kPair) {
            float4 v[kPair], e[kPair], tn[kPair];
            float most = -kInf;
#pragma unroll
            for (int i = 0; i < kPair; ++i) {
                const uint32_t here = at + 16u * kXentLanes * (u0 + i);
                const float4 c0 = lds4(here), c1 = H ? lds4(here + 16u) : c0;
                v[i] = group_of<H>(c0, c1);
                if (tail) {                  // past the row's end: as m, and e = 0 below
                    const int j = j0 + 4 * kXentLanes * (u0 + i);
                    if (j >= V) v[i].x = m;
                    if (j + 1 >= V) v[i].y = m;
                    if (j + 2 >= V) v[i].z = m;
                    if (j + 3 >= V) v[i].w = m;
                }
                most = fmaxf(most, max4(v[i]));
                tn[i] = t[u0 + i];
            }
            const float least = exp_and_t<kPair>(v, m2, e, tn);
            if (!(least >= kFast) || !finite_m) {
#pragma unroll
                for (int i = 0; i < kPair; ++i) {
                    const ExpT x = exp_slow(v[i], m, t[u0 + i]);
                    e[i] = x.e;
                    tn[i] = x.t;
                }
            }
#pragma unroll
            for (int i = 0; i < kPair; ++i) {
                t[u0 + i] = tn[i];
                if (tail) {
                    const int j = j0 + 4 * kXentLanes * (u0 + i);
                    if (j >= V) e[i].x = 0.0f;
                    if (j + 1 >= V) e[i].y = 0.0f;
                    if (j + 2 >= V) e[i].z = 0.0f;
                    if (j + 3 >= V) e[i].w = 0.0f;
                }
                S = __fadd_rn(__fadd_rn(__fadd_rn(__fadd_rn(S, e[i].x), e[i].y), e[i].z), e[i].w);
            }
            if (most >= bound)
#pragma unroll
                for (int i = 0; i < kPair; ++i) {
                    const int j = j0 + 4 * kXentLanes * (u0 + i);
                    if (max4(v[i]) >= bound && j < V) {
                        const int slot = atomicAdd(&R.listed, 1);
                        if (slot < kFound) {
                            R.found[slot] = v[i];
                            R.found_at[slot] = j;
                        }
                    }
                }
        }
        freed(seg);
    }
    out.S = S;
#pragma unroll
    for (int u = 0; u < kSets; ++u) {
        const float4 a = flush(u);
        out.u[u] = __fadd_rn(__fadd_rn(__fadd_rn(a.x, a.y), a.z), a.w);
    }
    return true;
}

__global__ void __launch_bounds__(kStreamThreads, 1) logprob_stream_kernel(LogprobArgs A) {
    extern __shared__ __align__(128) unsigned char smem_raw[];
    Stream &sh = *reinterpret_cast<Stream *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = A.V;
    auto bar = [](uint64_t &b) { return smem_u32(&b); };
    if (tid == 0) {
        for (Team &t : sh.team) {
            for (int i = 0; i < kRing; ++i) {
                mbar_init(bar(t.loaded[i]), 1);
                mbar_init(bar(t.freed[i]), kSumWarps);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(bar(t.done[i]), kSumWarps);
                mbar_init(bar(t.taken[i]), 1);
                t.row[i].listed = 0;
            }
        }
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(bar(sh.parted[i]), kMaxWarps);
            mbar_init(bar(sh.maxed[i]), 1);
            mbar_init(bar(sh.passed[i]), 1);
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
    // a team's rows are every kTeams-th of the CTA's: row number k of them is the
    // CTA's row kTeams * k + the team's number
    const int64_t step = gridDim.x * int64_t(kTeams);
    uint32_t k = 0, seg = 0;            // rows and segments done so far
    if (warp < kFirstMax) {
        // ---- e, S, T, the list
        const int ti = warp / kSumWarps, w8 = warp % kSumWarps;
        Team &team = sh.team[ti];
        auto loaded = [&](uint32_t i) { return wait(team.loaded[i % kRing], i / kRing); };
        auto freed = [&](uint32_t i) { arrive(team.freed[i % kRing]); };
        for (int64_t row = blockIdx.x + ti * int64_t(gridDim.x); row < A.rows; row += step, ++k) {
            RowState &R = team.row[k & 1];
            const uint32_t r = kTeams * k + ti;
            if (!wait(sh.maxed[r % kAhead], r / kAhead)) break;
            if (k >= 2 && !wait(team.taken[k & 1], k / 2 - 1)) break;
            const float m = sh.max[r % kAhead].m, bound = sh.max[r % kAhead].bound;
            RowSums o;
            bool ok;
            switch (shift_of(start_of(row))) {
                case 0: ok = sum_row<0>(team, R, V, m, bound, seg, loaded, freed, o); break;
                case 1: ok = sum_row<1>(team, R, V, m, bound, seg, loaded, freed, o); break;
                case 2: ok = sum_row<2>(team, R, V, m, bound, seg, loaded, freed, o); break;
                default: ok = sum_row<3>(team, R, V, m, bound, seg, loaded, freed, o); break;
            }
            if (!ok) break;
            // the first level of the folds: 32 chains of S, 32 sums in fours of T
            float v[8] = {o.S, o.u[0], o.u[1], o.u[2], o.u[3], 0.0f, 0.0f, 0.0f};
            const float f = butterfly8(v, lane);
            if (lane == lane_of_row(0)) R.red[w8] = f;
#pragma unroll
            for (int u = 0; u < kSets; ++u)
                if (lane == lane_of_row(u + 1)) R.tsum[kSumWarps * u + w8] = f;
            arrive(team.done[k & 1]);
        }
    } else if (warp < kFirstLoad) {
        // ---- the max, and the 32 groups' (the lanes of the same number)
        const int mw = warp - kFirstMax, mt = mw * 32 + lane;
        for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x, ++k) {
            RowMax &R = sh.max[k % kAhead];
            if (k >= kAhead && !wait(sh.passed[k % kAhead], k / kAhead - 1)) break;
            const float *x = start_of(row);
            const int h = shift_of(x);
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
                    if (q0 + u * kMaxThreads < hi) m = more_max(m, v[u]);
            }
            // the elements before and after those granules
            const int head = h ? 4 - h : 0, tail = 4 * hi - h;
            if (mt < head) m = max_nan(m, x[mt]);
            if (mt >= 32 && tail + mt - 32 < V) m = max_nan(m, x[tail + mt - 32]);
            R.parts[mw][lane] = m;
            arrive(sh.parted[k % kAhead]);
            if (mw == 0) {
                if (!wait(sh.parted[k % kAhead], k / kAhead)) break;
                float g0 = R.parts[0][lane], g1 = R.parts[kMaxWarps / 2][lane];
#pragma unroll
                for (int w = 1; w < kMaxWarps / 2; ++w) {
                    g0 = max_nan(g0, R.parts[w][lane]);
                    g1 = max_nan(g1, R.parts[kMaxWarps / 2 + w][lane]);
                }
                float all = max_nan(g0, g1);
#pragma unroll
                for (int off = 16; off >= 1; off >>= 1)
                    all = max_nan(all, __shfl_xor_sync(0xffffffffu, all, off));
                all = __fadd_rn(all, 0.0f);              // a zero maximum is +0
                const bool list = A.top_k > 0 && fabsf(all) <= 0x1.fffffep127f;
                const float bound = !list ? kInf
                                    : A.top_k > kFewAlternatives
                                        ? list_bound_64(g0, g1, A.top_k, lane)
                                        : list_bound(fmaxf(g0, g1), A.top_k, lane);
                if (lane == 0) {
                    R.m = all;
                    R.bound = bound;
                }
                arrive(sh.maxed[k % kAhead]);
            }
        }
    } else if (warp < kFirstFinal) {
        // ---- the loads
        Team &team = sh.team[warp - kFirstLoad];
        if (lane == 0) {
            const uint64_t evict_first = l2_policy_evict_first();
            bool ok = true;
            for (int64_t row = blockIdx.x + (warp - kFirstLoad) * int64_t(gridDim.x);
                 row < A.rows && ok; row += step) {
                const float *x = start_of(row);
                const int h = shift_of(x), nch = (V + h + 3) / 4, groups = (V + 3) / 4;
                for (int q = 0; q < groups; q += kSeg, ++seg) {
                    const int at = seg % kRing;
                    if (seg >= kRing &&
                        !mbar_wait_or_abort(bar(team.freed[at]), (seg / kRing - 1) & 1u, abort)) {
                        ok = false;
                        break;
                    }
                    load_granules_last(team.ring[at] - q, x - h, q, min(nch, q + kSeg + 1),
                                       &team.loaded[at], evict_first);
                }
            }
        }
    } else {
        // ---- the results
        const int ti = warp - kFirstFinal;
        Team &team = sh.team[ti];
        for (int64_t row = blockIdx.x + ti * int64_t(gridDim.x); row < A.rows; row += step, ++k) {
            RowState &R = team.row[k & 1];
            const uint32_t r = kTeams * k + ti;
            const float *x = start_of(row);
            const Asked asked = ask(A, row, x);
            if (!wait(team.done[k & 1], k / 2)) break;
            const float T = warp_butterfly_sum(R.tsum[lane]);
            const float *t = R.red;
            const float S =
                __fadd_rn(__fadd_rn(__fadd_rn(t[0], t[1]), __fadd_rn(t[2], t[3])),
                          __fadd_rn(__fadd_rn(t[4], t[5]), __fadd_rn(t[6], t[7])));
            const float m = sh.max[r % kAhead].m, bound = sh.max[r % kAhead].bound;
            uint64_t rank = 0;
            if (A.top_k > 0) {
                // the elements of the listed groups, then their order
                int n = 0;
                const bool all = R.listed <= kFound && fabsf(m) <= 0x1.fffffep127f;
                for (int c0 = 0; all && c0 < R.listed; c0 += 32) {
                    const bool in = c0 + lane < R.listed;
                    const float4 v = in ? R.found[c0 + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
                    const int j0 = in ? R.found_at[c0 + lane] : 0;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const bool is = in && comp(v, c) >= bound && j0 + c < V;
                        const unsigned who = __ballot_sync(0xffffffffu, is);
                        const int at = n + __popc(who & ((1u << lane) - 1u));
                        if (is && at < kListed) R.list[at] = rank_of(comp(v, c), j0 + c);
                        n += __popc(who);
                    }
                }
                __syncwarp();
                rank = !all || n > kListed ? top_by_rounds(x, V, A.top_k, lane)
                                           : rank_list(R.list, n, A.top_k, R.top, lane);
            }
            write_row(A, row, asked, m, S, T, rank, lane);
            __syncwarp();
            if (lane == 0) R.listed = 0;
            arrive(team.taken[k & 1]);
            arrive(sh.passed[r % kAhead]);
        }
    }
    __syncthreads();
    if (sh.abort && warp >= kFirstLoad && warp < kFirstFinal && lane == 0) {
        // let the copies in flight land
        atomicOr(&g_logprob_watchdog, kWatchdogLogprob);
        Team &team = sh.team[warp - kFirstLoad];
        for (uint32_t i = seg > uint32_t(kRing) ? seg - kRing : 0; i < seg; ++i)
            (void)mbar_wait_bounded(bar(team.loaded[i % kRing]), (i / kRing) & 1u);
    }
}

// A warp a row of at most 4096 logits, 1024 (a sweep) at a time: read once where
// that is the whole row, else once a pass (the row stays in L1). A lane has the
// groups lane + 32 w + 256 t, so chain lane + 32 w of S adds its groups in ascending
// t, and T's chains have an element each.
template <int W, bool ONE>
__global__ void __launch_bounds__(kSmallWarps * 32, W == 2 ? 4 : ONE ? 2 : 3) logprob_small_kernel(LogprobArgs A) {
    __shared__ uint64_t lists[kSmallWarps][kSmallListed], tops[kSmallWarps][32];
    __shared__ int counts[kSmallWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, V = A.V;
    for (int64_t row = blockIdx.x * int64_t(kSmallWarps) + warp; row < A.rows;
         row += gridDim.x * int64_t(kSmallWarps)) {
        const float *x = A.logits + row * A.ld;
        const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0;
        const Asked asked = ask(A, row, x);
        float4 v[W];                         // a sweep's groups; -inf past the row's end
        auto load = [&](int g0) {
            if (vec && 4 * g0 + 128 * W <= V) {
#pragma unroll
                for (int w = 0; w < W; ++w)
                    v[w] = *reinterpret_cast<const float4 *>(x + 4 * (g0 + 32 * w + lane));
                return;
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const int j = 4 * (g0 + 32 * w + lane);
                if (vec && j + 3 < V) {
                    v[w] = *reinterpret_cast<const float4 *>(x + j);
                } else {
                    v[w].x = j < V ? x[j] : -kInf;
                    v[w].y = j + 1 < V ? x[j + 1] : -kInf;
                    v[w].z = j + 2 < V ? x[j + 2] : -kInf;
                    v[w].w = j + 3 < V ? x[j + 3] : -kInf;
                }
            }
        };
        float mine[2] = {-kInf, -kInf};
        for (int g0 = 0; 4 * g0 < V; g0 += kXentLanes) {
            load(g0);
#pragma unroll
            for (int w = 0; w < W; ++w) mine[w % 2] = more_max(mine[w % 2], v[w]);
        }
        float m = max_nan(mine[0], mine[1]);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
            m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        m = __fadd_rn(m, 0.0f);              // a zero maximum is +0
        const bool finite_m = fabsf(m) <= 0x1.fffffep127f;
        const bool list = A.top_k > 0 && finite_m;
        const float bound =
            !list ? kInf
            : A.top_k > kFewAlternatives ? list_bound_64(mine[0], mine[1], A.top_k, lane)
                                         : list_bound(fmaxf(mine[0], mine[1]), A.top_k, lane);
        const f32x2 m2 = splat2(m);
        float s[8], T = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s[w] = 0.0f;
        if (lane == 0) counts[warp] = 0;
        __syncwarp();
        for (int g0 = 0; 4 * g0 < V; g0 += kXentLanes) {
            if (!ONE) load(g0);
            if (list) {
                float best = -kInf;
#pragma unroll
                for (int w = 0; w < W; ++w) best = fmaxf(best, max4(v[w]));
                if (best >= bound)
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const int j = 4 * (g0 + 32 * w + lane);
                        if (max4(v[w]) >= bound)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (comp(v[w], c) >= bound && j + c < V) {
                                    const int at = atomicAdd(&counts[warp], 1);
                                    if (at < kSmallListed)
                                        lists[warp][at] = rank_of(comp(v[w], c), j + c);
                                }
                    }
                __syncwarp();
            }
            float u[8] = {};                 // T's sums in fours
#pragma unroll
            for (int w0 = 0; w0 < W; w0 += 2) {
                float4 es[2], ts[2], vs[2] = {v[w0], v[w0 + 1]};
                ts[0] = ts[1] = es[0] = es[1] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (4 * (g0 + 32 * w0) < V) {
                    const float least = exp_and_t<2>(vs, m2, es, ts);
                    if (!(least >= kFast) || !finite_m)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int j = 4 * (g0 + 32 * (w0 + i) + lane);
                            const ExpT x2 =
                                exp_slow(vs[i], m, make_float4(0.f, 0.f, 0.f, 0.f));
                            es[i] = x2.e;
                            ts[i] = x2.t;
                            if (!finite_m) {     // past the end -inf - m need not be -inf
                                if (j >= V) es[i].x = ts[i].x = 0.0f;
                                if (j + 1 >= V) es[i].y = ts[i].y = 0.0f;
                                if (j + 2 >= V) es[i].z = ts[i].z = 0.0f;
                                if (j + 3 >= V) es[i].w = ts[i].w = 0.0f;
                            }
                        }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                const int w = w0 + i;
                const float4 e = es[i], t = ts[i];
                s[w] = __fadd_rn(__fadd_rn(__fadd_rn(__fadd_rn(s[w], e.x), e.y), e.z), e.w);
                // each chain's one block, added to +0
                u[w] = __fadd_rn(__fadd_rn(__fadd_rn(__fadd_rn(t.x, 0.0f), __fadd_rn(t.y, 0.0f)),
                                           __fadd_rn(t.z, 0.0f)),
                                 __fadd_rn(t.w, 0.0f));
                }
            }
            const float t = __shfl_sync(0xffffffffu, butterfly8(u, lane), lane_of_row(lane & 7));
            if (lane >> 3 == g0 / kXentLanes) T = t;
        }
        T = warp_butterfly_sum(T);
        const float part = butterfly8(s, lane);
        float f[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) f[w] = __shfl_sync(0xffffffffu, part, lane_of_row(w));
        const float S = __fadd_rn(__fadd_rn(__fadd_rn(f[0], f[1]), __fadd_rn(f[2], f[3])),
                                  __fadd_rn(__fadd_rn(f[4], f[5]), __fadd_rn(f[6], f[7])));
        uint64_t rank = 0;
        __syncwarp();
        const int listed = counts[warp];
        if (A.top_k > 0)
            rank = !list || listed > kSmallListed
                       ? top_by_rounds(x, V, A.top_k, lane)
                       : rank_list(lists[warp], listed, A.top_k, tops[warp], lane);
        write_row(A, row, asked, m, S, T, rank, lane);
        __syncwarp();
    }
}

// Few rows: a cluster of C CTAs a row. Of each 1024 logits CTA r has the 1024 / C
// from 1024 r / C on, so its elements make up whole chains of S (j mod 1024 picks
// the chain) and of T (j mod 4096), and only the maxima, the chains' sums and the
// listed alternatives cross the cluster. Latency bounds it: the row's load, three
// meetings of the cluster and the chain of V / 256 additions (8.3 us for one row of
// 50257, 15 for one of 256000).
struct Split {
    float parts[16], groups[32];        // maxima of this CTA, of the row's 32 groups
    float chain[kXentLanes], u[kSeg];   // of the row, in its first CTA: S, T in fours
    float red[8], tsum[32];
    uint64_t list[kListed], top[32];
    int listed, pad[3];
};
static_assert(sizeof(Split) % 16 == 0 && offsetof(Split, list) % 8 == 0, "aligned float4s");

__global__ void __launch_bounds__(kXentLanes, 2) logprob_split_kernel(LogprobArgs A) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Split &sh = *reinterpret_cast<Split *>(smem_raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = A.V;
    const int64_t row = blockIdx.x / C;
    const float *x = A.logits + row * A.ld;
    // stripes of 1024 logits; this CTA's groups of 4 in each, in order
    const int stripes = (V + 4 * kXentLanes - 1) / (4 * kXentLanes), width = kXentLanes / C;
    const int mine = stripes * width;
    float4 *xs = reinterpret_cast<float4 *>(&sh + 1), *es = xs + mine;
    auto element_of = [&](int i) {       // the first of local group i
        return 4 * (i / width * kXentLanes + rank * width + i % width);
    };
    if (tid == 0) sh.listed = 0;
    cluster.barrier_arrive();
    const Asked asked = ask(A, row, x);
    const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0;
    float most = -kInf;
    for (int i0 = tid; i0 < mine; i0 += 4 * kXentLanes) {
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + k * kXentLanes, j = element_of(i);
            if (i >= mine) break;
            if (vec && j + 3 < V) {
                v[k] = *reinterpret_cast<const float4 *>(x + j);
            } else {
                v[k].x = j < V ? x[j] : -kInf;
                v[k].y = j + 1 < V ? x[j + 1] : -kInf;
                v[k].z = j + 2 < V ? x[j + 2] : -kInf;
                v[k].w = j + 3 < V ? x[j + 3] : -kInf;
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + k * kXentLanes;
            if (i >= mine) break;
            xs[i] = v[k];
            most = more_max(most, v[k]);
        }
    }
    // the maxima of 32 groups of 8 C threads of the cluster
    const int team = min(32, 8 * C), teams = kXentLanes / team, per = 8 * C / team;
    for (int off = team / 2; off >= 1; off >>= 1)
        most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, off));
    if (lane % team == 0) sh.parts[tid / team] = most;
    __syncthreads();
    cluster.barrier_wait();
    if (tid < teams / per) {
        float g = sh.parts[tid * per];
        for (int i = 1; i < per; ++i) g = max_nan(g, sh.parts[tid * per + i]);
        for (int r = 0; r < C; ++r)
            *cluster.map_shared_rank(&sh.groups[rank * (teams / per) + tid], r) = g;
    }
    cluster.sync();
    float m = sh.groups[lane];
    const float group = m;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
    m = __fadd_rn(m, 0.0f);              // a zero maximum is +0
    const bool finite_m = fabsf(m) <= 0x1.fffffep127f;
    const bool list = A.top_k > 0 && finite_m;
    const float bound = list ? list_bound(group, A.top_k, lane) : kInf;
    Split &first = *cluster.map_shared_rank(&sh, 0);
    for (int i = tid; i < mine; i += kXentLanes) {
        const float4 v = xs[i];
        const int j = element_of(i);
        float4 e = finite_m ? exp4(v, m) : exp_slow(v, m, make_float4(0.f, 0.f, 0.f, 0.f)).e;
        if (j >= V) e.x = 0.0f;
        if (j + 1 >= V) e.y = 0.0f;
        if (j + 2 >= V) e.z = 0.0f;
        if (j + 3 >= V) e.w = 0.0f;
        es[i] = e;
        if (list && max4(v) >= bound)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (comp(v, c) >= bound && j + c < V) {
                    const int at = atomicAdd(&first.listed, 1);
                    if (at < kListed) first.list[at] = rank_of(comp(v, c), j + c);
                }
    }
    __syncthreads();
    if (tid >= kXentLanes - width) {     // the chains of S
        const int p = tid - (kXentLanes - width);
        float s = 0.0f;
#pragma unroll 4
        for (int i = p; i < mine; i += width) {
            const float4 e = es[i];
            s = __fadd_rn(__fadd_rn(__fadd_rn(__fadd_rn(s, e.x), e.y), e.z), e.w);
        }
        first.chain[rank * width + p] = s;
    }
    for (int f = tid; f < 4 * width; f += kXentLanes) {      // the chains of T, in fours
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int b = f; b < mine; b += 16 * width) {         // the blocks of 16 stripes
            float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = b + 4 * k * width;
                if (i >= mine) break;
                const float4 e = es[i], v = xs[i];
                if (e.x != 0.0f) t.x = __fmaf_rn(e.x, __fsub_rn(v.x, m), t.x);
                if (e.y != 0.0f) t.y = __fmaf_rn(e.y, __fsub_rn(v.y, m), t.y);
                if (e.z != 0.0f) t.z = __fmaf_rn(e.z, __fsub_rn(v.z, m), t.z);
                if (e.w != 0.0f) t.w = __fmaf_rn(e.w, __fsub_rn(v.w, m), t.w);
            }
            a = make_float4(__fadd_rn(a.x, t.x), __fadd_rn(a.y, t.y), __fadd_rn(a.z, t.z),
                            __fadd_rn(a.w, t.w));
        }
        first.u[f / width * kXentLanes + rank * width + f % width] =
            __fadd_rn(__fadd_rn(__fadd_rn(a.x, a.y), a.z), a.w);
    }
    cluster.sync();
    if (rank != 0) return;
    const float s = warp_butterfly_sum(sh.chain[tid]);
    if (lane == 0) sh.red[warp] = s;
#pragma unroll
    for (int q = 0; q < kSets; ++q) {
        const float t = warp_butterfly_sum(sh.u[q * kXentLanes + tid]);
        if (lane == 0) sh.tsum[q * kSumWarps + warp] = t;
    }
    __syncthreads();
    if (warp != 0) return;
    const float T = warp_butterfly_sum(sh.tsum[lane]);
    const float *f = sh.red;
    const float S = __fadd_rn(__fadd_rn(__fadd_rn(f[0], f[1]), __fadd_rn(f[2], f[3])),
                              __fadd_rn(__fadd_rn(f[4], f[5]), __fadd_rn(f[6], f[7])));
    uint64_t got = 0;
    if (A.top_k > 0)
        got = !list || sh.listed > kListed ? top_by_rounds(x, V, A.top_k, lane)
                                           : rank_list(sh.list, sh.listed, A.top_k, sh.top, lane);
    write_row(A, row, asked, m, S, T, got, lane);
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

namespace {
size_t split_bytes(int64_t V, int64_t cluster) {
    const int64_t stripes = (V + 4 * kXentLanes - 1) / (4 * kXentLanes);
    return sizeof(Split) + size_t(stripes * (kXentLanes / cluster) * 2 * int(sizeof(float4)));
}

// The CTAs a row is split over where rows are few; 0: a CTA a row (the stream
// kernel). The most whose clusters run at once, two CTAs an SM; where only that
// many fit an SM's shared memory, 7/8 of it, as not every SM finds a place in a
// cluster then. Rows of more than 65536 logits, whose stream takes long, may also
// take two turns of 16. us, stream / split over 4 / 8 / 16: 1 x 50257 18.5 / 11.8 /
// 8.9 / 8.3; 19 x 50257 19.5 / 12.5 / 10.3 / 9.9; 38: 19.6 / 14.4 / 12.2 / 12.8; 64:
// 20.0 / 14.6 / 19.4 / 20.0; 76: 20.0 / 23.1 / 20.6 / 23.8; 64 x 16000 10.1 / 8.9 / 9.3 /
// 16.4; 38 x 128000 42 / - / - / 24; 1 x 256000 67 / - / - / 15. Over 2 it was no
// faster anywhere.
int split_cluster(int64_t rows, int64_t V, int64_t sms) {
    constexpr int64_t kSmem = 227 * 1024;
    if (V > (int64_t(1) << 20)) return 0;        // no share fits
    for (int c = 16; c >= 4; c /= 2) {
        const int64_t fit = kSmem / int64_t(split_bytes(V, c) + 1024);
        const int64_t two = std::min<int64_t>(fit, 2) * sms;
        if (fit > 0 && rows * c <= (fit > 2 ? two : two * 7 / 8)) return c;
    }
    const int64_t fit = kSmem / int64_t(split_bytes(V, 16) + 1024);
    return V > 65536 && rows * 16 <= 2 * fit * sms ? 16 : 0;
}
}  // namespace

cudaError_t launch_logprob(int64_t rows, int64_t V, const float *logits, int64_t ld,
                           const int32_t *tokens, int top_k, float *logp, float *entropy,
                           float *stats, int32_t *top_ids, float *top_logp, int32_t *dev_status,
                           cudaStream_t s) {
    LogprobArgs A = {rows, int(V), logits, ld, tokens, top_k, logp, entropy,
                     reinterpret_cast<float4 *>(stats), top_ids, top_logp, dev_status};
    const int64_t sms = sm_count_current_device();
    if (V <= kSmallVocab) {
        const int64_t blocks = std::min<int64_t>((rows + kSmallWarps - 1) / kSmallWarps, sms * 8);
        // two groups a lane up to 256 logits: 21 us instead of 33 for 16384 x 256
        if (V <= 256)
            logprob_small_kernel<2, true><<<unsigned(blocks), kSmallWarps * 32, 0, s>>>(A);
        else if (V <= 1024)
            logprob_small_kernel<8, true><<<unsigned(blocks), kSmallWarps * 32, 0, s>>>(A);
        else
            logprob_small_kernel<8, false><<<unsigned(blocks), kSmallWarps * 32, 0, s>>>(A);
        return cudaGetLastError();
    }
    if (const int cluster = split_cluster(rows, V, sms)) {
        const size_t share = split_bytes(V, cluster);
        cudaError_t e = cudaFuncSetAttribute(
            logprob_split_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e == cudaSuccess && cluster > 8)
            e = cudaFuncSetAttribute(logprob_split_kernel,
                                     cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(rows * cluster));
        cfg.blockDim = dim3(kXentLanes);
        cfg.dynamicSmemBytes = share;
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = unsigned(cluster);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, logprob_split_kernel, A);
        return e == cudaSuccess ? cudaGetLastError() : e;
    }
    const int64_t grid = std::min<int64_t>(rows, sms);
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
