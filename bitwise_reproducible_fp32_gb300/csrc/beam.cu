// beam.cu -- the next beams of a beam search from the alternatives of the present
// ones, with the beams' token histories, for sm_103a.
//
//   candidates: each beam's alternatives j, score s_w + logp_j (rounded once); a
//   beam that has ended is one candidate, itself. rank = score * weight(length).
//   The largest ranks are kept, the lowest (beam, id, j) first among equals.
//
// A request has at most 32 x 32 candidates, so latency bounds the selection, and the
// histories' bytes (each read and written once) a call with long answers. A warp
// holds a beam's alternatives, one a lane, as 64-bit keys (the rank's bits in their
// order, then the complement of beam and place of the id in its beam), sorts them
// by a bitonic network of shuffles, and the warps' lists are joined pairwise: the 32
// largest of two sorted lists are max(a_i, b_31-i), five exchanges from sorted. The
// histories of a request are copied by several CTAs, each of which makes the same
// selection again, so nothing waits. Measured on the GPU: 16 requests of 4 beams 8 us; 512
// of 16 beams of 32 alternatives with histories of 2048 tokens 31 us, with one parent a
// request and with four (67 MB are written, much of which stays in L2, and 4 to 16 MB
// read: the selection, before the first of these bytes, is a good part of it).
#include <algorithm>

#include "det_internal.cuh"

namespace det {
namespace {

constexpr int kMaxBeams = 32;
constexpr unsigned kAll = 0xffffffffu;

struct SelectArgs {
    int win, wout, k;
    const float *scores;
    const int32_t *finished, *lens, *hist;
    int64_t ldh;
    const int32_t *ids;
    const float *logp;
    int32_t eos;
    const float *weights;
    int64_t nweights;
    int64_t cols, part;           // history columns, and those of a CTA
    float *scores_out;
    int32_t *finished_out, *lens_out, *hist_out;
    int64_t ldho;
    int32_t *tokens, *parents, *forks, *dev_status;
    int vec;                      // histories by 16 bytes
};

__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t min64(uint64_t a, uint64_t b) { return a < b ? a : b; }

// One exchange of a network that sorts descending: lane keeps the larger of the pair
// (lane, lane ^ step) where `up` says so.
__device__ __forceinline__ uint64_t exchange(uint64_t v, int step, bool larger) {
    const uint64_t o = __shfl_xor_sync(kAll, v, step);
    return larger ? max64(v, o) : min64(v, o);
}
__device__ __forceinline__ uint64_t merge_down(uint64_t v, int lane) {
#pragma unroll
    for (int step = 16; step >= 1; step >>= 1) v = exchange(v, step, (lane & step) == 0);
    return v;
}
__device__ __forceinline__ uint64_t sort_down(uint64_t v, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int step = size / 2; step >= 1; step >>= 1)
            v = exchange(v, step, ((lane & size) == 0) == ((lane & step) == 0));
    return v;
}

__global__ void __launch_bounds__(1024) beam_select_kernel(const SelectArgs A) {
    __shared__ uint64_t lists[kMaxBeams][32];
    __shared__ int32_t place[kMaxBeams][32];      // the alternative at each place
    // of each beam kept: its parent, the history's tokens, the column and the token
    // that is added (column -1: none)
    __shared__ int s_parent[32], s_len[32], s_col[32], s_token[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t req = blockIdx.x, row0 = req * A.win;
    int status = 0;
    auto weigh = [&](float s, int len) {
        if (!A.weights) return s;
        const int64_t at = min(int64_t(max(len, 0)), A.nweights - 1);
        return __fmul_rn(s, A.weights[at]);
    };
    if (warp < A.win) {
        const int64_t row = row0 + warp;
        const float score = A.scores[row];
        const bool done = A.finished && A.finished[row] != 0;
        const int len = A.lens ? A.lens[row] : 0;
        const int n = done ? 1 : A.k;
        bool live = lane < n && score != __uint_as_float(0xff800000u);
        int32_t id = 0;
        float s = score;
        if (live && !done) {
            id = A.ids[row * A.k + lane];
            s = __fadd_rn(score, A.logp[row * A.k + lane]);
        }
        live = live && s != __uint_as_float(0xff800000u);
        float rank = weigh(s, done ? len : int(unsigned(len) + 1u));
        if (live && rank != rank) {
            status = 1;
            live = false;
        }
        // the place of the id in its beam: ids before it, the first of equal ones first
        int at = 0;
        const unsigned uid = unsigned(id) ^ 0x80000000u;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const unsigned o = __shfl_sync(kAll, uid, j);
            at += j < n && (o < uid || (o == uid && j < lane));
        }
        if (lane < n) place[warp][at] = lane;
        const unsigned b = __float_as_uint(__fadd_rn(rank, 0.0f));     // -0 counts as +0
        const unsigned order = b ^ (b >> 31 ? kAll : 0x80000000u);
        uint64_t key = live ? uint64_t(order) << 32 | (kAll - unsigned(warp * 32 + at)) : 0;
        lists[warp][lane] = sort_down(key, lane);
    }
    // the warps' lists, joined pairwise
    for (int n = A.win; n > 1;) {
        const int half = (n + 1) >> 1;
        __syncthreads();
        if (warp + half < n) {
            const uint64_t v = max64(lists[warp][lane], lists[warp + half][31 - lane]);
            lists[warp][lane] = merge_down(v, lane);
        }
        n = half;
    }
    __syncthreads();
    if (warp == 0) {
        const uint64_t key = lists[0][lane];
        int parent = -1, len = 0, token = -1;
        float s = __uint_as_float(0xff800000u);
        bool done = false;
        if (lane < A.wout && key) {
            const unsigned at = kAll - unsigned(key);
            const int w = at >> 5, j = place[w][at & 31];
            const int64_t row = row0 + w;
            parent = w;
            done = A.finished && A.finished[row] != 0;
            s = A.scores[row];
            len = A.lens ? A.lens[row] : 0;
            token = A.eos;
            if (!done) {
                s = __fadd_rn(s, A.logp[row * A.k + j]);
                token = A.ids[row * A.k + j];
                if (A.hist && (len < 0 || len >= A.cols)) status |= 2;
            } else if (A.hist && (len < 0 || len > A.cols)) {
                status |= 2;
            }
        }
        const bool dead = parent < 0;
        const bool ended = dead || done || (A.eos >= 0 && token == A.eos);
        s_parent[lane] = parent;
        s_len[lane] = len;
        s_col[lane] = dead || done || len < 0 ? -1 : len;
        s_token[lane] = token;
        if (lane < A.wout && blockIdx.y == 0) {
            const int64_t out = req * A.wout + lane;
            A.scores_out[out] = s;
            A.tokens[out] = token;
            A.parents[out] = dead ? -1 : int(row0 + parent);
            if (A.forks) A.forks[out] = ended ? -1 : int(row0 + parent);
            if (A.finished_out) A.finished_out[out] = ended;
            if (A.lens_out) A.lens_out[out] = dead ? 0 : done ? len : int(unsigned(len) + 1u);
        }
    }
    if (A.dev_status && blockIdx.y == 0) {
        status = __reduce_or_sync(kAll, unsigned(status));
        if (lane == 0 && status) atomicOr(reinterpret_cast<int *>(A.dev_status), status);
    }
    if (!A.hist) return;
    __syncthreads();
    const int warps = blockDim.x >> 5;
    const int64_t c0 = blockIdx.y * A.part, c1 = min(A.cols, c0 + A.part);
    for (int n = warp; n < A.wout; n += warps) {
        if (s_parent[n] < 0) continue;
        const int32_t *from = A.hist + (row0 + s_parent[n]) * A.ldh;
        int32_t *to = A.hist_out + (req * A.wout + n) * A.ldho;
        const int64_t len = s_len[n], end = min(c1, max(len, int64_t(0)));
        int64_t c = c0;
        if (A.vec) {
            for (; c + 512 <= end; c += 512) {
                int4 v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    v[u] = *reinterpret_cast<const int4 *>(from + c + 128 * u + 4 * lane);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    *reinterpret_cast<int4 *>(to + c + 128 * u + 4 * lane) = v[u];
            }
            for (; c + 128 <= end; c += 128)
                *reinterpret_cast<int4 *>(to + c + 4 * lane) =
                    *reinterpret_cast<const int4 *>(from + c + 4 * lane);
        }
        for (int64_t i = c + lane; i < end; i += 32) to[i] = from[i];
        if (lane == 0 && s_col[n] >= c0 && s_col[n] < c1) to[s_col[n]] = s_token[n];
    }
}

}  // namespace

cudaError_t launch_beam_select(int64_t requests, const det_beams &in, const det_beams &out,
                               int top_k, const int32_t *top_ids, const float *top_logp,
                               int32_t eos, const float *weights, int64_t nweights, int64_t cols,
                               int32_t *tokens, int32_t *parents, int32_t *forks,
                               int32_t *dev_status, cudaStream_t s) {
    SelectArgs A = {int(in.beams), int(out.beams), top_k, in.scores, in.finished, in.lens, in.hist,
                    in.ldh, top_ids, top_logp, eos, weights, nweights, cols, cols, out.scores,
                    out.finished, out.lens, out.hist, out.ldh, tokens, parents, forks, dev_status,
                    0};
    int warps = A.win;
    int64_t parts = 1;
    if (A.hist) {
        auto al16 = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
        A.vec = al16(A.hist) && al16(A.hist_out) && A.ldh % 4 == 0 && A.ldho % 4 == 0;
        warps = std::max(warps, A.wout);
        // 1024 columns and more a CTA, and no more CTAs than about one wave: each makes the
        // selection again (512 requests of 16 beams and 2048 tokens: 33 us in two parts, 31
        // in one)
        const int64_t wave = int64_t(sm_count_current_device()) * 4;
        parts = std::max<int64_t>(1, std::min((cols + 1023) / 1024, wave / requests));
        A.part = std::max<int64_t>(128, ((cols + parts - 1) / parts + 127) / 128 * 128);
        parts = std::max<int64_t>(1, (cols + A.part - 1) / A.part);
    }
    beam_select_kernel<<<dim3(unsigned(requests), unsigned(parts)), unsigned(warps * 32), 0, s>>>(
        A);
    return cudaGetLastError();
}

}  // namespace det
