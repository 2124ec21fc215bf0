// decode_group.cu -- decode attention of small groups that share a prefix (at most 8 query
// rows a key-value head, as beam search with shared pages has), for sm_103a.
//
// The formulas and bits of decode.cu, and its structure: a unit (a group and a
// key-value head) is one cluster of 1..16 CTAs, whose warps stream pieces of keys, then of
// values, through rings of their own. The unit's tokens are the group's shared chunks,
// with all its rows, and after them each request's own, with its rows. Scores, exps and
// partials lie in the workspace, by chunk, which stays in L2. So a step of beam search
// reads its prompts' keys and values once, in one launch: HBM bounds it, and the latency
// of its phases (the shared pages, K, the maxima, S, V, the chunks left to right).
// Measured, 12 heads of 64: 16 groups of 4 requests of 700..1900 tokens and up to 148 of
// their own 60..63 us (157 MB; K and V go by at 4.9 TB/s, 32 us, the phases between take
// about 16, and the units, all on the GPU at once, end with the longest: 1.2 to 1.45 times
// the mean; each request for itself 73 us), of 4500..6000 tokens 129 us (4.3 TB/s; 228). Three CTAs
// an SM with rings of two pieces: two CTAs with three took 72 us and 162; clusters of
// twice the CTAs 77 and 149.
#include <cooperative_groups.h>

#include <algorithm>

#include "decode_shared.cuh"

namespace cg = cooperative_groups;

namespace det {

// Set when a bounded wait for a piece gave up.
__device__ unsigned int g_group_watchdog;

namespace {

constexpr int kMaxCluster = 16;
constexpr int kGroupCtas = 3;             // an SM's
constexpr int kDeep = 8;                  // groups of a chain of S in flight

// A chunk of the unit: `vc` of it, shared ones first, then request after request.
struct Chunk {
    int w;                    // the request, -1: shared
    int t0, tokens;           // its first token, how many
    int64_t slot;             // its first row's 256 scores (and d partials)
};

// NH: rows that registers hold, at least the group's; PER: likewise of a request.
template <int NH, int PER, Loader LOAD>
__global__ void __launch_bounds__(kThreads, kGroupCtas)
    group_kernel(const SharedArgs A, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap, int64_t unit_x, int64_t unit_part) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ uint64_t full[kWarps][kRingPieces];
    __shared__ __align__(16) float rows[NH][256];     // q, the chains of S, then each warp's
                                                      // probabilities of a piece
    __shared__ float red[NH][8], top[kMaxCluster][NH], most_of[kWarps][NH], inv[NH];
    __shared__ int lost[kMaxCluster], found[kMaxCluster], s_bad, s_lost;
    __shared__ int len[kFewRows], raw[kFewRows], own_at[kFewRows + 1];
    static_assert(kWarps * kTile <= 256, "a piece's probabilities of all warps");
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x / C, g = unit / A.kv_heads, kv = unit - g * A.kv_heads;
    const int b0 = g * A.group, W = min(A.group, A.batch - b0), per = A.per_kv, R = W * per;
    const int d = A.d, nsl = (d + 31) / 32;
    float *const X = A.x + unit * unit_x, *const P = A.part + unit * unit_part;
    if (tid < kMaxCluster) found[tid] = 0;
    if (C > 1) cluster.barrier_arrive();  // waited for before the first remote access
    init_bars<LOAD>(&full[0][0]);
    int status = 0;
    if (tid < W) {
        const int n = A.kv_lens[b0 + tid];
        raw[tid] = n;
        len[tid] = n > 0 && n <= A.max_len ? n : 0;
        if (n < 0 || n > A.max_len) status = 1;
    }
    if (tid == 0) {
        s_bad = INT32_MAX;
        s_lost = 0;
    }
    if (lane < NH) most_of[warp][lane] = __uint_as_float(0xff800000u);
    for (int i = tid; i < R * d; i += kThreads) {
        const int h = i / d, w = h / per;
        rows[h][i - h * d] =
            A.q[(b0 + w) * A.ldq + int64_t(kv * per + h - w * per) * d + (i - h * d)];
    }
    __syncthreads();
    auto meet = [&]() {                   // all threads of the unit
        if (C > 1) cluster.sync(); else __syncthreads();
    };

    // ---- the shared chunks: whole ones before the shortest's last token whose pages are
    // the same in all requests
    int lead = 0, live = 0, least = INT32_MAX;
    for (int w = W - 1; w >= 0; --w)
        if (len[w]) {
            lead = w;
            ++live;
            least = min(least, len[w]);
        }
    int shared = live > 1 ? (least - 1) / kKChunk : 0;
    const int32_t *first = A.table + (b0 + lead) * A.ldt;
    const int pages = int((int64_t(shared) * kKChunk + A.page_size - 1) / A.page_size);
    int bad_at = INT32_MAX;
    for (int j = rank * kThreads + tid; j < pages; j += C * kThreads) {
        const int id = first[j];
        bool bad = unsigned(id) >= unsigned(A.num_pages);
#pragma unroll
        for (int w = 0; w < kFewRows; ++w)
            if (w < W && len[w]) bad |= A.table[(b0 + w) * A.ldt + j] != id;
        if (bad) bad_at = min(bad_at, j);
    }
    if (bad_at != INT32_MAX) atomicMin(&s_bad, bad_at);
    __syncthreads();
    bad_at = s_bad;
    if (C > 1) {
        cluster.barrier_wait();
        if (tid < C) *cluster.map_shared_rank(found + rank, tid) = bad_at;
        cluster.sync();
        for (int r = 0; r < C; ++r) bad_at = min(bad_at, found[r]);
    }
    if (bad_at != INT32_MAX) shared = min(shared, int(int64_t(bad_at) * A.page_size / kKChunk));
    if (tid == 0) {
        int at = shared;
        for (int w = 0; w < W; ++w) {
            own_at[w] = at;
            if (len[w]) at += (len[w] + kKChunk - 1) / kKChunk - shared;
        }
        own_at[W] = at;
    }
    __syncthreads();
    const int all = own_at[W], base = all / C, rem = all % C;
    const int c0 = rank * base + min(rank, rem), my = base + (rank < rem);
    auto chunk = [&](int vc) {
        Chunk c;
        if (vc < shared) {
            c = {-1, vc * kKChunk, kKChunk, int64_t(vc) * R};
        } else {
            int w = 0;
            while (vc >= own_at[w + 1]) ++w;
            const int t0 = (shared + vc - own_at[w]) * kKChunk;
            c = {w, t0, min(kKChunk, len[w] - t0), int64_t(shared) * R + int64_t(vc - shared) * per};
        }
        return c;
    };
    // of chunk c of row h (of request w): its scores' slot
    auto slot_of = [&](int c, int h, int w) {
        return c < shared ? int64_t(c) * R + h
                          : int64_t(shared) * R + int64_t(own_at[w] - shared + c - shared) * per +
                                (h - w * per);
    };

    // ---- the warp's pieces: of each chunk of the CTA one tile of 64 tokens (a quarter,
    // another one from chunk to chunk), all slices of keys; then of every fourth
    // (chunk, slice) the values, 64 tokens at a time
    const int jobs = my * nsl;
    Ring<LOAD> ring(A, &kmap, A.k, smem_u32(smem_raw) + warp * kRingBytes, smem_u32(&full[warp][0]));
    auto quarter = [&](int place) { return (warp + place) & 3; };
    int kp = -1, ksl = 0, vj = warp, vt = 0, in_t = 0, in_live = 0;
    Chunk in;
    int lost_mask = 0;
    auto look_up = [&](int t, int n) {
        in_t = in.t0 + t;
        in_live = n;
        const int32_t *p = A.table + (b0 + (in.w < 0 ? lead : in.w)) * A.ldt;
        if (ring.template look_up<true>(p, in_t, in_live)) lost_mask |= 1 << in.w;
    };
    auto next_job = [&]() {               // the first piece of job vj
        if (vj < jobs) {
            in = chunk(c0 + vj / nsl);
            vt = 0;
            look_up(0, min(kTile, in.tokens));
        }
    };
    auto next_tile = [&]() {              // the next tile that has tokens, or the first job
        while (++kp < my) {
            in = chunk(c0 + kp);
            const int t = quarter(kp) * kTile;
            if (t < in.tokens) {
                look_up(t, min(kTile, in.tokens - t));
                return;
            }
        }
        ring.map = &vmap;
        ring.cache = A.v;
        next_job();
    };
    next_tile();
    auto issue = [&]() {
        if (kp < my) {
            ring.fetch(kv, ksl, in_t, in_live);
            if (++ksl == nsl) {
                ksl = 0;
                next_tile();
            }
        } else if (vj < jobs) {
            ring.fetch(kv, vj % nsl, in_t, in_live);
            vt += kTile;
            if (vt < in.tokens) {
                look_up(vt, min(kTile, in.tokens - vt));
            } else {
                vj += kWarps;
                next_job();
            }
        }
        if (LOAD != kTma) cp_commit();
    };
    for (int i = 0; i < kRingPieces - 1; ++i) issue();
    uint32_t kat[8], vat[8];      // 16-byte unit i of row `lane` of a piece; column `lane` of row i
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        kat[i] = lane * 128 + ((i ^ (lane & 7)) << 4);
        vat[i] = i * 128 + (((lane >> 2) ^ i) << 4) + ((lane & 3) << 2);
    }

    // ---- scores
    auto tile = [&](auto held, const Chunk &c, int q4, int row0, int n) {
        constexpr int N = decltype(held)::value;
        float acc[2][N];                  // of tokens lane and lane + 32
#pragma unroll
        for (int h = 0; h < N; ++h) acc[0][h] = acc[1][h] = 0.0f;
        for (int sl = 0; sl < nsl; ++sl) {
            ring.wait();
            if (!ring.stuck) issue();     // into the slot consumed before this one
            const uint32_t piece = ring.piece();
            const int width = min(32, d - 32 * sl);
            const float *q = &rows[row0][32 * sl];
            auto four = [&](int u) {
                const float4 k0 = lds4(piece + kat[u]), k1 = lds4(piece + 4096 + kat[u]);
#pragma unroll
                for (int h = 0; h < N; ++h) {
                    const float4 qv = *reinterpret_cast<const float4 *>(q + h * 256 + 4 * u);
                    acc[0][h] = __fmaf_rn(qv.x, k0.x, acc[0][h]);
                    acc[1][h] = __fmaf_rn(qv.x, k1.x, acc[1][h]);
                    acc[0][h] = __fmaf_rn(qv.y, k0.y, acc[0][h]);
                    acc[1][h] = __fmaf_rn(qv.y, k1.y, acc[1][h]);
                    acc[0][h] = __fmaf_rn(qv.z, k0.z, acc[0][h]);
                    acc[1][h] = __fmaf_rn(qv.z, k1.z, acc[1][h]);
                    acc[0][h] = __fmaf_rn(qv.w, k0.w, acc[0][h]);
                    acc[1][h] = __fmaf_rn(qv.w, k1.w, acc[1][h]);
                }
            };
            if (width == 32) {
#pragma unroll
                for (int u = 0; u < 8; ++u) four(u);
            } else {
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    if (4 * u + 4 <= width) {
                        four(u);
                    } else if (4 * u < width) {
                        for (int j = 4 * u; j < width; ++j) {
                            const float k0 = lds1(piece + kat[u] + 4 * (j & 3));
                            const float k1 = lds1(piece + 4096 + kat[u] + 4 * (j & 3));
#pragma unroll
                            for (int h = 0; h < N; ++h) {
                                acc[0][h] = __fmaf_rn(q[h * 256 + j], k0, acc[0][h]);
                                acc[1][h] = __fmaf_rn(q[h * 256 + j], k1, acc[1][h]);
                            }
                        }
                    }
                }
            }
        }
        const int t = q4 * kTile + lane;
#pragma unroll
        for (int h = 0; h < N; ++h) {
            float m = __uint_as_float(0xff800000u);
            if (h < n) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (t + 32 * k < c.tokens) {
                        const float x = __fmul_rn(acc[k][h], A.scale);
                        X[(c.slot + h) * 256 + t + 32 * k] = x;
                        m = max_nan(m, x);
                    }
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1)
                m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
            if (lane == 0 && h < n) most_of[warp][row0 + h] = max_nan(most_of[warp][row0 + h], m);
        }
    };
    for (int p = 0; p < my; ++p) {
        const Chunk c = chunk(c0 + p);
        const int q4 = quarter(p);
        if (q4 * kTile >= c.tokens) continue;
        if (c.w < 0) tile(std::integral_constant<int, NH>(), c, q4, 0, R);
        else tile(std::integral_constant<int, PER>(), c, q4, c.w * per, per);
    }
    // ---- m over the cluster, and the requests whose pages are out of range
    if (lost_mask) atomicOr(&s_lost, lost_mask);
    __syncthreads();
    if (tid < NH) {
        float t = most_of[0][tid];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) t = max_nan(t, most_of[w][tid]);
        for (int r = 0; r < C; ++r) *cluster.map_shared_rank(&top[rank][tid], r) = t;
    }
    if (tid < C) *cluster.map_shared_rank(&lost[rank], tid) = s_lost;
    meet();

    // ---- e in place of x, and the chains of S: a warp 32 chains of a row, each in
    // ascending order; the sums go to every CTA
    for (int i = warp * C + rank; i < R * 8; i += C * kWarps) {
        const int h = i >> 3, l = (i & 7) * 32 + lane, w = h / per, n = len[w];
        float m = top[0][h];
        for (int r = 1; r < C; ++r) m = max_nan(m, top[r][h]);
        const bool finite = fabsf(m) <= 0x1.fffffep127f;
        float sum = 0.0f;
        for (int t = 4 * l; t < n; t += 1024 * kDeep) {
            float4 *at[kDeep], e[kDeep];
#pragma unroll
            for (int u = 0; u < kDeep; ++u) {
                const int tu = t + 1024 * u;
                if (tu >= n) break;
                at[u] = reinterpret_cast<float4 *>(X + slot_of(tu / kKChunk, h, w) * 256 +
                                                   (tu & (kKChunk - 1)));
                e[u] = __ldcg(at[u]);
            }
#pragma unroll
            for (int u = 0; u < kDeep; ++u) {
                const int tu = t + 1024 * u;
                if (tu >= n) break;
                e[u] = finite ? exp4(e[u], m) : exp4_any(e[u], m);
                *at[u] = e[u];
                sum = __fadd_rn(sum, e[u].x);
                if (tu + 1 < n) sum = __fadd_rn(sum, e[u].y);
                if (tu + 2 < n) sum = __fadd_rn(sum, e[u].z);
                if (tu + 3 < n) sum = __fadd_rn(sum, e[u].w);
            }
        }
        for (int r = 0; r < C; ++r) *cluster.map_shared_rank(&rows[h][l], r) = sum;
    }
    meet();
    for (int i = warp; i < R * 8; i += kWarps) {
        const float s = butterfly32(rows[i >> 3][(i & 7) * 32 + lane]);
        if (lane == 0) red[i >> 3][i & 7] = s;
    }
    __syncthreads();
    if (tid < R) {
        const float *t = red[tid];
        inv[tid] = __fdiv_rn(
            1.0f, __fadd_rn(__fadd_rn(__fadd_rn(t[0], t[1]), __fadd_rn(t[2], t[3])),
                            __fadd_rn(__fadd_rn(t[4], t[5]), __fadd_rn(t[6], t[7]))));
    }
    __syncthreads();

    // ---- P V: exps asked for a piece ahead
    const uint32_t copies = smem_u32(&rows[0][0]) + warp * (NH * kTile * 4);
    float keep[2 * NH];
    auto ask = [&](const Chunk &c, int t) {
        const int n = c.w < 0 ? R : per;
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int at = t + 32 * k + lane;
                keep[2 * h + k] =
                    h < n && at < c.tokens ? __ldcg(X + (c.slot + h) * 256 + at) : 0.0f;
            }
    };
    Chunk next;
    auto job = [&](auto held, const Chunk &c, int j, int row0, int n) {
        constexpr int N = decltype(held)::value;
        float acc[N], w[N];
#pragma unroll
        for (int h = 0; h < N; ++h) {
            acc[h] = 0.0f;
            w[h] = inv[row0 + min(h, n - 1)];
        }
        for (int t = 0; t < c.tokens; t += kTile) {
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 2 * N; ++k)
                sts1(copies + (k * 32 + lane) * 4, __fmul_rn(keep[k], w[k / 2]));
            if (t + kTile < c.tokens) {
                ask(c, t + kTile);
            } else if (j + kWarps < jobs) {
                next = chunk(c0 + (j + kWarps) / nsl);
                ask(next, 0);
            }
            ring.wait();
            if (!ring.stuck) issue();     // into the slot consumed before this one
            const uint32_t piece = ring.piece();
            const int here = c.tokens - t;
            if (here >= kTile) {
#pragma unroll
                for (int r = 0; r < kTile; r += 4) {
                    const uint32_t up = piece + (r & ~7) * 128;
                    const float v0 = lds1(up + vat[r & 7]), v1 = lds1(up + vat[(r & 7) + 1]),
                                v2 = lds1(up + vat[(r & 7) + 2]), v3 = lds1(up + vat[(r & 7) + 3]);
#pragma unroll
                    for (int h = 0; h < N; ++h) {
                        const float4 p = lds4(copies + h * (kTile * 4) + r * 4);
                        acc[h] = __fmaf_rn(p.x, v0, acc[h]);
                        acc[h] = __fmaf_rn(p.y, v1, acc[h]);
                        acc[h] = __fmaf_rn(p.z, v2, acc[h]);
                        acc[h] = __fmaf_rn(p.w, v3, acc[h]);
                    }
                }
            } else {
                for (int r8 = 0; r8 < here; r8 += 8) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (r8 + k < here) {
                            const float v = lds1(piece + r8 * 128 + vat[k]);
#pragma unroll
                            for (int h = 0; h < N; ++h)
                                acc[h] = __fmaf_rn(lds1(copies + h * (kTile * 4) + (r8 + k) * 4), v,
                                                   acc[h]);
                        }
                }
            }
        }
        const int col = j % nsl * 32 + lane;
        if (col < d)
#pragma unroll
            for (int h = 0; h < N; ++h)
                if (h < n) P[(c.slot + h) * d + col] = acc[h];
    };
    if (warp < jobs) {
        next = chunk(c0 + warp / nsl);
        ask(next, 0);
    }
    for (int j = warp; j < jobs; j += kWarps) {
        const Chunk c = next;
        if (c.w < 0) job(std::integral_constant<int, NH>(), c, j, 0, R);
        else job(std::integral_constant<int, PER>(), c, j, c.w * per, per);
    }
    if (ring.stuck && lane == 0)          // tell the unit: its rows are NaN
        for (int r = 0; r < C; ++r) *cluster.map_shared_rank(&found[rank], r) = -1;
    ring.drain(&g_group_watchdog);
    meet();
    int gone = 0;
    bool stuck = false;
    for (int r = 0; r < C; ++r) {
        gone |= lost[r];
        stuck |= found[r] < 0;
    }
    // ---- the chunks left to right
    for (int i = (warp * C + rank) * 32 + lane; i < R * d; i += C * kThreads) {
        const int h = i / d, w = h / per, j = i - h * d;
        const int chunks = (len[w] + kKChunk - 1) / kKChunk;
        float t = 0.0f;
        for (int c = 0; c < chunks; c += 16) {
            float v[16];
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (c + k < chunks) v[k] = __ldcg(P + slot_of(c + k, h, w) * d + j);
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (c + k < chunks) t = c + k == 0 ? v[k] : __fadd_rn(t, v[k]);
        }
        // a request without tokens is 0 whatever happened to the others
        if (raw[w] != 0 && (stuck || gone >> w & 1 || len[w] == 0)) t = __uint_as_float(0x7fc00000u);
        A.out[(b0 + w) * A.ldo + int64_t(kv * per + h - w * per) * d + j] = t;
    }
    if (A.dev_status && rank == 0) {
        if (tid == 0 && gone) status |= 2;
        if (status) atomicOr(reinterpret_cast<int *>(A.dev_status), status);
    }
}

template <int NH, int PER, Loader LOAD>
cudaError_t run_group(const SharedArgs &A, const GroupPlan &p, const CUtensorMap *maps,
                      cudaStream_t s) {
    auto kern = group_kernel<NH, PER, LOAD>;
    const size_t smem = size_t(kWarps) * kRingBytes;
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e == cudaSuccess && p.cluster > 8)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p.units * p.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(p.cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const CUtensorMap none = {};
    e = cudaLaunchKernelEx(&cfg, kern, A, maps ? maps[0] : none, maps ? maps[1] : none,
                           p.chunks * A.rows * 256, p.chunks * A.rows * A.d);
    return e == cudaSuccess ? cudaGetLastError() : e;
}
template <int NH, int PER>
cudaError_t group_of_loader(const SharedArgs &A, const GroupPlan &p, const CUtensorMap *maps,
                            cudaStream_t s) {
    return maps     ? run_group<NH, PER, kTma>(A, p, maps, s)
           : A.wide ? run_group<NH, PER, kCopy16>(A, p, maps, s)
                    : run_group<NH, PER, kCopy4>(A, p, maps, s);
}

}  // namespace

// The cluster: as many CTAs (a power of two) as let all units be on the GPU at once, and
// no more than a request has chunks.
GroupPlan group_plan(int64_t groups, int64_t rows, int64_t kv_heads, int64_t head_dim,
                     int64_t max_len) {
    GroupPlan p;
    p.units = groups * kv_heads;
    p.chunks = (max_len + kKChunk - 1) / kKChunk;
    const int64_t slots = int64_t(sm_count_current_device()) * kGroupCtas;
    int64_t c = 1;
    while (2 * c <= kMaxCluster && 2 * c * p.units <= slots && 2 * c <= p.chunks) c *= 2;
    p.cluster = int(c);
    // shared chunks with all rows and own ones with a request's: no more than all of them
    // with all rows
    p.part = size_t(p.units * p.chunks * rows) * 256 * 4;
    p.bytes = p.part + size_t(p.units * p.chunks * rows * head_dim) * 4;
    return p;
}

cudaError_t launch_group_decode(const SharedArgs &A, const GroupPlan &p, const CUtensorMap *maps,
                                cudaStream_t s) {
    const bool four = A.rows <= 4;
    return A.per_kv == 1   ? four ? group_of_loader<4, 1>(A, p, maps, s)
                                  : group_of_loader<8, 1>(A, p, maps, s)
           : A.per_kv == 2 ? four ? group_of_loader<4, 2>(A, p, maps, s)
                                  : group_of_loader<8, 2>(A, p, maps, s)
                           : group_of_loader<8, 4>(A, p, maps, s);
}

cudaError_t group_decode_watchdog(unsigned int *code, int clear) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_group_watchdog, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    if (clear && *code) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_group_watchdog, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace det
