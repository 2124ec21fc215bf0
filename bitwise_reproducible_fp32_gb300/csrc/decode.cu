// decode.cu -- attention of one new token a request over a paged key-value
// cache, for sm_103a.
//
//   s_j = q K_j (fmaf chain from +0),  x_j = s_j scale,  m = max x_j,
//   e_j = exp(x_j - m),  S = the 256-chain sum of the e_j,  p_j = e_j (1/S),
//   o = sum over 256-token chunks, left to right, of fmaf chains of p_j V_j
//
// the last row of the causal attention over the same tokens, bit for bit.
//
// Each key and value is read once; per element there are one or, with shared
// heads, up to 8 multiply-adds: HBM bounds it. p_j needs S, which needs every
// score, so K goes by first and V after; a unit (a request, a key-value head, up
// to kMaxHeads of the query heads that share it) is one cluster of 1..16 CTAs,
// which keeps the scores in its shared memory between the two, so no second
// launch, no atomics and, but for very long rows, no workspace are needed.
//  - The row is cut at the profile's 256-token chunks; a CTA takes a run of them.
//  - Every warp streams its own pieces of 32 tokens x 32 dimensions through a
//    ring of kStages slots by 16-byte cp.async (4-byte where the strides want it),
//    K pieces first, then V pieces: the ring already fills with V while the
//    CTAs meet for m and S.
//  - Scores: a lane a token, the chain over d from shared memory (rows padded to
//    36 floats: 16-byte reads without bank conflicts), q broadcast.
//  - m and the 256 chains of S cross the cluster through distributed shared
//    memory; a chain adds its groups in ascending order wherever they lie.
//  - P V: a warp a (chunk, 32 dimensions), a lane a dimension, the chain over the
//    chunk's tokens; the chunk partials are joined left to right at the end.
// Rows whose scores and partials do not fit shared memory keep them in the
// workspace, which stays in L2.
#include <cooperative_groups.h>

#include <algorithm>
#include <cstdlib>

#include "det_internal.cuh"
#include "det_math.cuh"

namespace cg = cooperative_groups;

namespace det {
namespace {

#ifndef DEC_W
#define DEC_W 4
#define DEC_ST 4
#define DEC_CTAS 2
#endif
constexpr int kWarps = DEC_W;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = DEC_ST;
constexpr int kRow = 36;                    // floats a piece's row takes
constexpr int kPiece = 32 * kRow;
constexpr int kMaxHeads = 8;
constexpr int kMaxCluster = 16;
constexpr int kPageCache = 1024;            // page ids of a CTA kept on chip
constexpr int kCtasPerSm = DEC_CTAS;
constexpr int kSmemPerCta = (227 / kCtasPerSm - 1) * 1024;

struct DecodeArgs {
    int heads, kv_heads, head_dim;
    const float *q;
    int64_t ldq;
    const float *k, *v;
    int64_t num_pages;
    unsigned page_size;
    int page_shift;           // log2(page_size), or -1
    int64_t page_stride, token_stride, head_stride;
    const int32_t *table;
    int64_t ldt;
    const int32_t *kv_lens;
    float scale;
    float *out;
    int64_t ldo;
    float *workspace;
    int64_t max_len, ws_cta;  // ws_cta: floats of the workspace a CTA has
    int room;                 // floats of shared memory for scores and partials
    int unit_heads, batches;  // query heads a unit takes; units a key-value head
    int32_t *dev_status;
};

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

struct Fixed {                          // the fixed part of a CTA's shared memory
    float ring[kWarps][kStages][kPiece];
    float q[kMaxHeads][256];
    float chain[kMaxHeads][256];
    float red[kMaxHeads][8];
    float top[kMaxCluster][kMaxHeads];  // each CTA's maxima
    int lost[kMaxCluster];
    int pages[kPageCache];
};

static_assert(sizeof(Fixed) % 16 == 0 && int(sizeof(Fixed)) + 4096 <= kSmemPerCta,
              "room for scores beside the fixed part");

// NH: the heads of a unit the registers hold (nh <= NH of them live).
template <int NH, bool VEC>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_kernel(const DecodeArgs A) {
    extern __shared__ float4 smem4[];
    Fixed &F = *reinterpret_cast<Fixed *>(smem4);
    float *room = reinterpret_cast<float *>(smem4) + sizeof(Fixed) / 4;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x / C, b = blockIdx.y;
    const int g = unit / A.batches, d = A.head_dim;
    const int per_kv = A.heads / A.kv_heads, h_in = (unit - g * A.batches) * A.unit_heads;
    const int nh = min(A.unit_heads, per_kv - h_in), h0 = g * per_kv + h_in;
    float *o = A.out + b * A.ldo + int64_t(h0) * d;
    const int n = A.kv_lens[b];
    if (n <= 0 || n > A.max_len) {      // the whole cluster
        const float fill = n == 0 ? 0.0f : __uint_as_float(0x7fc00000u);
        for (int i = rank * kThreads + tid; i < nh * d; i += C * kThreads) o[i] = fill;
        if (n != 0 && rank == 0 && tid == 0 && A.dev_status)
            atomicOr(reinterpret_cast<int *>(A.dev_status), 1);
        return;
    }
    cluster.barrier_arrive();           // waited for before the first remote access
    // this CTA's run of chunks and tokens
    const int nch = (n + kKChunk - 1) / kKChunk, base = nch / C, rem = nch % C;
    auto first_chunk = [&](int r) { return r * base + min(r, rem); };
    const int c0 = first_chunk(rank), my = base + (rank < rem), most = base + (rem > 0);
    const int t0 = c0 * kKChunk, t1 = min(n, t0 + my * kKChunk);
    // scores [head][token], then partials [head][chunk][d], here or in L2
    const int xs_ld = most * kKChunk, part_at = nh * xs_ld;
    const bool on_chip = nh * most * (kKChunk + d) <= A.room;
    float *const ws = on_chip ? nullptr
                              : A.workspace + (int64_t(b) * (gridDim.x / C) + unit) * C * A.ws_cta;
    auto scores_of = [&](int r) {
        return on_chip ? cluster.map_shared_rank(room, r) : ws + r * A.ws_cta;
    };
    float *xs = on_chip ? room : ws + rank * A.ws_cta;

    const int32_t *pages = A.table + b * A.ldt;
    const float *kb = A.k + g * A.head_stride, *vb = A.v + g * A.head_stride;
    auto page_of = [&](int t) {
        return A.page_shift >= 0 ? unsigned(t) >> A.page_shift : unsigned(t) / A.page_size;
    };
    const unsigned pg0 = page_of(t0), pgs = t1 > t0 ? page_of(t1 - 1) - pg0 + 1 : 0;
    const bool cached = pgs <= unsigned(kPageCache);
    int lost = 0;
    for (unsigned i = tid; i < pgs; i += kThreads) {
        int id = pages[pg0 + i];
        if (id < 0 || id >= A.num_pages) {
            lost = 1;
            id = 0;
        }
        if (cached) F.pages[i] = id;
    }
    for (int i = tid; i < nh * d; i += kThreads) {
        const int h = i / d;
        F.q[h][i - h * d] = A.q[b * A.ldq + int64_t(h0) * d + i];
    }
    lost = __syncthreads_or(lost);
    // a token's offset in the cache (a page out of range reads page 0 instead)
    auto offset_of = [&](int t) {
        const unsigned p = page_of(t);
        int id;
        if (cached) {
            id = F.pages[p - pg0];
        } else {
            id = pages[p];
            if (id < 0 || id >= A.num_pages) id = 0;
        }
        return id * A.page_stride + int64_t(unsigned(t) - p * A.page_size) * A.token_stride;
    };

    // ---- the warp's pieces: K tiles warp, warp + kWarps, ... of 32 tokens, all
    // their slices of 32 dimensions; then V jobs warp, warp + kWarps, ... (chunk,
    // slice), 32 tokens at a time
    const int nsl = (d + 31) / 32, tiles = (t1 - t0 + 31) / 32, jobs = my * nsl;
    const uint32_t ring = smem_u32(&F.ring[warp][0][0]);
    int kt = warp, ksl = 0, vj = warp, vt = 0, slot_in = 0;
    int64_t off = 0;
    auto issue = [&](const float *src, int t, int sl, int end) {
        const uint32_t dst = ring + slot_in * (kPiece * 4);
        const int live = min(32, end - t), width = min(32, d - 32 * sl);
        src += 32 * sl;
        if constexpr (VEC) {
            const int col = lane & 7, r0 = lane >> 3;
            const bool in = 4 * col < width;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 4 * i + r0;
                const int64_t at = __shfl_sync(0xffffffffu, off, r);
                if (in && r < live) cp_async<16>(dst + (r * kRow + 4 * col) * 4, src + at + 4 * col);
            }
        } else {
#pragma unroll 8
            for (int r = 0; r < 32; ++r) {
                const int64_t at = __shfl_sync(0xffffffffu, off, r);
                if (lane < width && r < live)
                    cp_async<4>(dst + (r * kRow + lane) * 4, src + at + lane);
            }
        }
    };
    auto issue_next = [&]() {
        if (kt < tiles) {
            const int t = t0 + 32 * kt;
            if (ksl == 0 && t + lane < t1) off = offset_of(t + lane);
            issue(kb, t, ksl, t1);
            if (++ksl == nsl) {
                ksl = 0;
                kt += kWarps;
            }
        } else if (vj < jobs) {
            const int c = vj / nsl, sl = vj - c * nsl;
            const int t = t0 + c * kKChunk + vt, end = min(t1, t0 + (c + 1) * kKChunk);
            if (t + lane < end) off = offset_of(t + lane);
            issue(vb, t, sl, end);
            vt += 32;
            if (t + 32 >= end) {
                vt = 0;
                vj += kWarps;
            }
        }
        cp_commit();
        slot_in = slot_in + 1 == kStages ? 0 : slot_in + 1;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue_next();
    int slot = 0;
    auto next_piece = [&]() {
        cp_wait<kStages - 2>();
        __syncwarp();
        issue_next();               // into the slot consumed before this one
        const float *p = &F.ring[warp][slot][0];
        slot = slot + 1 == kStages ? 0 : slot + 1;
        return p;
    };

    // ---- scores
    float m[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) m[h] = __uint_as_float(0xff800000u);
    for (int tl = warp; tl < tiles; tl += kWarps) {
        float acc[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) acc[h] = 0.0f;
        for (int sl = 0; sl < nsl; ++sl) {
            const float *row = next_piece() + lane * kRow;
            const int width = min(32, d - 32 * sl);
            const float *q = &F.q[0][32 * sl];
            auto four = [&](int c) {
                const float4 kv = *reinterpret_cast<const float4 *>(row + c);
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const float4 qv = *reinterpret_cast<const float4 *>(q + h * 256 + c);
                    acc[h] = __fmaf_rn(qv.x, kv.x, acc[h]);
                    acc[h] = __fmaf_rn(qv.y, kv.y, acc[h]);
                    acc[h] = __fmaf_rn(qv.z, kv.z, acc[h]);
                    acc[h] = __fmaf_rn(qv.w, kv.w, acc[h]);
                }
            };
            if (width == 32) {
#pragma unroll
                for (int c = 0; c < 32; c += 4) four(c);
            } else {
                int c = 0;
                for (; c + 4 <= width; c += 4) four(c);
                for (; c < width; ++c) {
                    const float kv = row[c];
#pragma unroll
                    for (int h = 0; h < NH; ++h) acc[h] = __fmaf_rn(q[h * 256 + c], kv, acc[h]);
                }
            }
        }
        const int t = t0 + 32 * tl + lane;
        if (t < t1) {
#pragma unroll
            for (int h = 0; h < NH; ++h)
                if (h < nh) {
                    const float x = __fmul_rn(acc[h], A.scale);
                    xs[h * xs_ld + (t - t0)] = x;
                    m[h] = max_nan(m[h], x);
                }
        }
    }
    // ---- m over the cluster
#pragma unroll
    for (int h = 0; h < NH; ++h) {
#pragma unroll
        for (int off2 = 16; off2 >= 1; off2 >>= 1)
            m[h] = max_nan(m[h], __shfl_xor_sync(0xffffffffu, m[h], off2));
        if (lane == 0) F.red[h][warp] = m[h];
    }
    __syncthreads();
    cluster.barrier_wait();
    if (tid < NH) {
        float t = F.red[tid][0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) t = max_nan(t, F.red[tid][w]);
        for (int r = 0; r < C; ++r) cluster.map_shared_rank(&F.top[rank][tid], r)[0] = t;
    }
    if (tid < C) cluster.map_shared_rank(&F.lost[rank], tid)[0] = lost;
    cluster.sync();
    for (int r = 0; r < C; ++r) lost |= F.lost[r];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
        m[h] = F.top[0][h];
        for (int r = 1; r < C; ++r) m[h] = max_nan(m[h], F.top[r][h]);
    }
    // ---- e in place (slots past t1 hold anything and are never added)
    const int quads = (t1 - t0 + 3) >> 2;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
        if (h >= nh) break;
        float4 *x4 = reinterpret_cast<float4 *>(xs + h * xs_ld);
        if (fabsf(m[h]) <= 0x1.fffffep127f) {
            for (int i = tid; i < quads; i += kThreads) x4[i] = exp4(x4[i], m[h]);
        } else {
            for (int i = tid; i < quads; i += kThreads) {
                const float4 v = x4[i];
                x4[i] = make_float4(
                    det_exp_call(__fsub_rn(v.x, m[h])), det_exp_call(__fsub_rn(v.y, m[h])),
                    det_exp_call(__fsub_rn(v.z, m[h])), det_exp_call(__fsub_rn(v.w, m[h])));
            }
        }
    }
    cluster.sync();
    // ---- chains of S: (head, chain) over the cluster's threads; the total goes
    // to every CTA
    for (int i = rank * kThreads + tid; i < nh * 256; i += C * kThreads) {
        const int h = i >> 8, l = i & 255;
        float s = 0.0f;
        int r = 0, next = first_chunk(1);
        const float *src = scores_of(0) + h * xs_ld;
        int start = 0;
        for (int t = 4 * l; t < n; t += 1024) {
            while ((t >> 8) >= next) {
                ++r;
                start = next * kKChunk;
                next = first_chunk(r + 1);
                src = scores_of(r) + h * xs_ld;
            }
            const float4 e = *reinterpret_cast<const float4 *>(src + (t - start));
            s = __fadd_rn(s, e.x);
            if (t + 1 < n) s = __fadd_rn(s, e.y);
            if (t + 2 < n) s = __fadd_rn(s, e.z);
            if (t + 3 < n) s = __fadd_rn(s, e.w);
        }
        for (r = 0; r < C; ++r) cluster.map_shared_rank(&F.chain[h][l], r)[0] = s;
    }
    cluster.sync();
    for (int i = warp; i < nh * 8; i += kWarps) {
        const float s = butterfly32(F.chain[i >> 3][(i & 7) * 32 + lane]);
        if (lane == 0) F.red[i >> 3][i & 7] = s;
    }
    __syncthreads();
    // ---- p in place
#pragma unroll
    for (int h = 0; h < NH; ++h) {
        if (h >= nh) break;
        const float *t = F.red[h];
        const float inv = __fdiv_rn(
            1.0f, __fadd_rn(__fadd_rn(__fadd_rn(t[0], t[1]), __fadd_rn(t[2], t[3])),
                            __fadd_rn(__fadd_rn(t[4], t[5]), __fadd_rn(t[6], t[7]))));
        float4 *x4 = reinterpret_cast<float4 *>(xs + h * xs_ld);
        for (int i = tid; i < quads; i += kThreads) {
            const float4 e = x4[i];
            x4[i] = make_float4(__fmul_rn(e.x, inv), __fmul_rn(e.y, inv), __fmul_rn(e.z, inv),
                                __fmul_rn(e.w, inv));
        }
    }
    __syncthreads();
    // ---- P V: chunk partials (registers past the unit's heads repeat its last)
    int head_at[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) head_at[h] = min(h, nh - 1) * xs_ld;
    for (int j = warp; j < jobs; j += kWarps) {
        const int c = j / nsl, sl = j - c * nsl;
        const int end = min(t1 - t0, (c + 1) * kKChunk);
        float acc[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) acc[h] = 0.0f;
        for (int t = c * kKChunk; t < end; t += 32) {
            const float *p = next_piece() + lane;
            const float *pr = xs + t;
            auto four = [&](int r) {
                const float v0 = p[r * kRow], v1 = p[(r + 1) * kRow], v2 = p[(r + 2) * kRow],
                            v3 = p[(r + 3) * kRow];
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const float4 w = *reinterpret_cast<const float4 *>(pr + head_at[h] + r);
                    acc[h] = __fmaf_rn(w.x, v0, acc[h]);
                    acc[h] = __fmaf_rn(w.y, v1, acc[h]);
                    acc[h] = __fmaf_rn(w.z, v2, acc[h]);
                    acc[h] = __fmaf_rn(w.w, v3, acc[h]);
                }
            };
            if (end - t >= 32) {
#pragma unroll
                for (int r = 0; r < 32; r += 4) four(r);
            } else {
                int r = 0;
                for (; r + 4 <= end - t; r += 4) four(r);
                for (; r < end - t; ++r) {
                    const float v = p[r * kRow];
#pragma unroll
                    for (int h = 0; h < NH; ++h)
                        acc[h] = __fmaf_rn(pr[head_at[h] + r], v, acc[h]);
                }
            }
        }
        if (32 * sl + lane < d)
#pragma unroll
            for (int h = 0; h < NH; ++h)
                if (h < nh) xs[part_at + (h * most + c) * d + 32 * sl + lane] = acc[h];
    }
    cp_wait<0>();
    cluster.sync();
    // ---- the chunks left to right
    for (int i = rank * kThreads + tid; i < nh * d; i += C * kThreads) {
        const int h = i / d;
        float t = 0.0f;
        for (int r = 0; r < C; ++r) {
            const float *p = scores_of(r) + part_at + h * most * d + (i - h * d);
            const int chunks = base + (r < rem);
            for (int c = 0; c < chunks; ++c) {
                const float v = p[c * d];
                t = r == 0 && c == 0 ? v : __fadd_rn(t, v);
            }
        }
        o[i] = lost ? __uint_as_float(0x7fc00000u) : t;
    }
    if (lost && rank == 0 && tid == 0 && A.dev_status)
        atomicOr(reinterpret_cast<int *>(A.dev_status), 2);
    cluster.sync();               // the others still read this CTA's shared memory
}

struct DecodePlan {
    int unit_heads, batches, cluster;
    int room;                     // floats of shared memory
    int64_t ws_cta, ws_bytes;
};

DecodePlan decode_plan(int64_t batch, int64_t heads, int64_t kv_heads, int64_t head_dim,
                       int64_t max_len) {
    DecodePlan p;
    const int64_t per_kv = heads / kv_heads;
    p.batches = int((per_kv + kMaxHeads - 1) / kMaxHeads);
    p.unit_heads = int((per_kv + p.batches - 1) / p.batches);
    const int64_t units = std::max<int64_t>(1, batch * kv_heads * p.batches);
    const int64_t chunks = (max_len + kKChunk - 1) / kKChunk;
    const int64_t slots = int64_t(sm_count_current_device()) * kCtasPerSm;
    int c = 1;
    while (c < kMaxCluster && units * c < slots && 2 * c <= chunks) c *= 2;
    const char *ev = getenv("DEC_C");
    if (ev) { c = atoi(ev); while (c > 1 && c > chunks) c /= 2; }
    p.cluster = c;
    const int64_t need = int64_t(p.unit_heads) * ((chunks + c - 1) / c) * (kKChunk + head_dim);
    const int64_t cap = (kSmemPerCta - int64_t(sizeof(Fixed))) / 4;
    p.room = int(std::min(need, cap));
    p.ws_cta = need > cap ? (need + 3) / 4 * 4 : 0;
    p.ws_bytes = p.ws_cta * 4 * units * c;
    return p;
}

}  // namespace

size_t decode_workspace_bytes(int64_t batch, int64_t heads, int64_t kv_heads, int64_t head_dim,
                              int64_t max_len) {
    return size_t(decode_plan(batch, heads, kv_heads, head_dim, max_len).ws_bytes);
}

cudaError_t launch_decode_attention(int64_t batch, int heads, const float *q, int64_t ldq,
                                    const det_kv_cache &c, const int32_t *table,
                                    int64_t max_pages, int64_t ldt, const int32_t *kv_lens,
                                    float scale, float *out, int64_t ldo, float *workspace,
                                    int32_t *dev_status, cudaStream_t s) {
    const int64_t max_len = max_pages * c.page_size;
    const DecodePlan p = decode_plan(batch, heads, c.kv_heads, c.head_dim, max_len);
    DecodeArgs A = {heads, int(c.kv_heads), int(c.head_dim), q, ldq, c.k, c.v, c.num_pages,
                    unsigned(c.page_size), -1, c.page_stride, c.token_stride, c.head_stride,
                    table, ldt, kv_lens, scale, out, ldo, workspace, max_len, p.ws_cta, p.room,
                    p.unit_heads, p.batches, dev_status};
    for (int i = 0; i < 31; ++i)
        if (c.page_size == int64_t(1) << i) A.page_shift = i;
    auto al16 = [](const void *x) { return reinterpret_cast<uintptr_t>(x) % 16 == 0; };
    const bool vec = al16(c.k) && al16(c.v) && c.head_dim % 4 == 0 && c.page_stride % 4 == 0 &&
                     c.token_stride % 4 == 0 && c.head_stride % 4 == 0;
    auto run = [&](auto kern) {
        const size_t smem = sizeof(Fixed) + size_t(p.room) * 4;
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             int(smem));
        if (e == cudaSuccess && p.cluster > 8)
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(p.cluster * A.kv_heads * p.batches), unsigned(batch));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = unsigned(p.cluster);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, kern, A);
        return e == cudaSuccess ? cudaGetLastError() : e;
    };
    const int nh = p.unit_heads;
    if (vec) {
        if (nh == 1) return run(decode_kernel<1, true>);
        if (nh == 2) return run(decode_kernel<2, true>);
        if (nh <= 4) return run(decode_kernel<4, true>);
        return run(decode_kernel<8, true>);
    }
    if (nh == 1) return run(decode_kernel<1, false>);
    if (nh == 2) return run(decode_kernel<2, false>);
    if (nh <= 4) return run(decode_kernel<4, false>);
    return run(decode_kernel<8, false>);
}

}  // namespace det
