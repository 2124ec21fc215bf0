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
//  - Every warp streams its own pieces of 64 tokens x 32 dimensions through a
//    ring of kStages slots, K pieces first, then V pieces: the ring already fills
//    with V while the CTAs meet for m and S. A piece is one or a few TMA boxes (a
//    box a page) where the page size is 8, 16, 32 or a multiple of 64 and every
//    stride a multiple of 16 bytes; else 16- or 4-byte cp.async. Either way its
//    rows are 128 bytes, the 16-byte units of row r swapped by r mod 8, so that
//    reads along rows and along columns meet no bank conflict.
//  - Scores: a lane two tokens, the chains over d from shared memory, q broadcast.
//  - m and the 256 chains of S cross the cluster through distributed shared
//    memory; a chain adds its groups in ascending order wherever they lie.
//  - P V: a warp a (chunk, 32 dimensions), a lane a dimension, the chain over the
//    chunk's tokens; the chunk partials are joined left to right at the end.
// Rows whose scores and partials do not fit shared memory keep them in the
// workspace, which stays in L2; a piece's probabilities are then asked for one
// piece ahead.
// Measured, 12 heads of 64: 64 requests of 700..2048 tokens 93 us (5.8 TB/s of keys
// and values), 256 of 100..512 96 us (5.1 TB/s), one of 32768 50 us (4.0 TB/s); 32
// heads of 128 over 8, 4 of 22853..32768, 178 us (5.1 TB/s): the passes over K and
// over V run at HBM's rate, the rest is 30 us between them and the longest
// request's tail. 32 heads over 4, 32 requests of 2000..4096, 129 us (3.1 TB/s): the
// longest is a third longer than the mean, and the 8 heads' multiply-adds and
// shared-memory reads keep a warp about as long as its pieces' arrival. A unit has at
// most 16 CTAs, so few requests of few key-value heads leave most of the GPU idle: one
// of 32768 tokens takes 107 us over one head of 128 for 8 query heads (33.6 MB, 0.3
// TB/s), 102 over 8 such heads for 32, 40 over one head of 64. Asking L2 for 4 or more
// pieces of V ahead while the CTAs meet ran 1..10% slower.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "decode.cuh"

namespace cg = cooperative_groups;

namespace det {

// Set when a bounded wait for a piece gave up.
__device__ unsigned int g_decode_watchdog;

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTokens = 64;                 // of a piece, 32 dimensions each
constexpr int kPieceBytes = kTokens * 128;
constexpr int kMaxHeads = 8;
constexpr int kMaxCluster = 16;
constexpr int kDeep = 8;                    // groups of a chain of S in flight
constexpr int kPageCache = 512;             // page ids of a CTA kept on chip
constexpr unsigned kWatchdogDecode = 32u;   // det_watchdog_status bit 5
constexpr int kCtasPerSm = 2;
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
    int box;                  // tokens of a TMA box
    int unit_heads, batches;  // query heads a unit takes; units a key-value head
    int stages;               // slots of a warp's ring
    int64_t max_pages;
    int32_t *dev_status;
};

template <int NH>
struct Fixed {                          // a CTA's shared memory after the rings
    uint64_t full[kWarps][4];
    float rows[NH][256];                // q, then the chains of S, then each warp's
                                        // probabilities of a piece (rows in the workspace)
    float red[NH][8];
    float top[kMaxCluster][NH];         // each CTA's maxima
    int lost[kMaxCluster];
    int pages[kPageCache];
};
// Beside it there is room for the scores and partials of short rows.
constexpr int kRingBytes = kWarps * kPieceBytes;      // a stage of all warps
constexpr int kStages = 3;
template <int NH>
constexpr bool kFits = sizeof(Fixed<NH>) % 16 == 0 &&
                       kStages * kRingBytes + int(sizeof(Fixed<NH>)) <= kSmemPerCta;
static_assert(kFits<1> && kFits<2> && kFits<4> && kFits<kMaxHeads>, "shared memory");
static_assert(kWarps * kTokens <= 256, "a piece's probabilities of all warps");

// Where a chunk of the row lies: the place'th of CTA r's run. CTAs r < rem have
// base + 1 chunks, the others base.
struct Walk {
    int r = 0, place, base, rem;
    __device__ __forceinline__ Walk(int chunk, int base_, int rem_)
        : place(chunk), base(base_), rem(rem_) {}
    // of a chunk that exists
    __device__ __forceinline__ void settle() {
        for (int run; place >= (run = base + (r < rem)); ++r) place -= run;
    }
};

// NH: the heads of a unit the registers hold (nh <= NH of them live).
template <int NH, Loader LOAD>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    decode_kernel(const DecodeArgs A, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const int stages = A.stages;                    // 2 or 3
    Fixed<NH> &F = *reinterpret_cast<Fixed<NH> *>(smem_raw + stages * kRingBytes);
    float *room = reinterpret_cast<float *>(&F + 1);
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x / C;
    const int b = blockIdx.y;
    const int g = unit / A.batches, d = A.head_dim;
    const int per_kv = A.heads / A.kv_heads, h_in = (unit - g * A.batches) * A.unit_heads;
    const int nh = min(A.unit_heads, per_kv - h_in), h0 = g * per_kv + h_in;
    float *o = A.out + b * A.ldo + int64_t(h0) * d;
    const int32_t *pages = A.table + b * A.ldt;
    if (LOAD == kTma && tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
        for (int i = 0; i < kWarps * 4; ++i) mbar_init(smem_u32(&F.full[0][i]), 1);
        fence_mbar_init();
    }
    // the length, the query and, for a unit of one CTA, the first page ids are
    // asked for together
    int early[kPageCache / kThreads];
    if (C == 1)
#pragma unroll
        for (int i = 0; i < kPageCache / kThreads; ++i)
            early[i] = tid + i * kThreads < A.max_pages ? pages[tid + i * kThreads] : 0;
    for (int i = tid; i < nh * d; i += kThreads) {
        const int h = i / d;
        F.rows[h][i - h * d] = A.q[b * A.ldq + int64_t(h0) * d + i];
    }
    const int n = A.kv_lens[b];
    if (n <= 0 || n > A.max_len) {      // the whole cluster
        const float fill = n == 0 ? 0.0f : __uint_as_float(0x7fc00000u);
        for (int i = rank * kThreads + tid; i < nh * d; i += C * kThreads) o[i] = fill;
        if (n != 0 && rank == 0 && tid == 0 && A.dev_status)
            atomicOr(reinterpret_cast<int *>(A.dev_status), 1);
        return;
    }
    if (C > 1) cluster.barrier_arrive();    // waited for before the first remote access
    auto meet = [&]() {                 // all threads of the unit
        if (C > 1) cluster.sync(); else __syncthreads();
    };
    // this CTA's run of chunks and tokens
    const int nch = (n + kKChunk - 1) / kKChunk, base = nch / C, rem = nch % C;
    auto first_chunk = [&](int r) { return r * base + min(r, rem); };
    const int c0 = first_chunk(rank), my = base + (rank < rem), most = base + (rem > 0);
    const int t0 = c0 * kKChunk, t1 = min(n, t0 + my * kKChunk);
    // scores [head][token], then partials [head][chunk][d], here or in L2
    const int64_t xs_ld = int64_t(most) * kKChunk, part_at = nh * xs_ld;
    const bool on_chip = int64_t(nh) * most * (kKChunk + d) <= A.room;
    float *const ws = on_chip ? nullptr
                              : A.workspace + (int64_t(b) * (gridDim.x / C) + unit) * C * A.ws_cta;
    auto scores_of = [&](int r) {
        return on_chip ? cluster.map_shared_rank(room, r) : ws + r * A.ws_cta;
    };
    float *xs = on_chip ? room : ws + rank * A.ws_cta;

    const float *kb = A.k + g * A.head_stride, *vb = A.v + g * A.head_stride;
    auto page_of = [&](int t) {
        return A.page_shift >= 0 ? unsigned(t) >> A.page_shift : unsigned(t) / A.page_size;
    };
    const unsigned pg0 = page_of(t0), pgs = t1 > t0 ? page_of(t1 - 1) - pg0 + 1 : 0;
    const bool cached = pgs <= unsigned(kPageCache);
    int lost = 0;
    auto check = [&](unsigned i, int id) {
        if (id < 0 || id >= A.num_pages) {
            lost = 1;
            id = 0;
        }
        if (cached) F.pages[i] = id;
    };
    if (C == 1 && cached) {
#pragma unroll
        for (int i = 0; i < kPageCache / kThreads; ++i)
            if (unsigned(tid + i * kThreads) < pgs) check(tid + i * kThreads, early[i]);
    } else {
        for (unsigned i = tid; i < pgs; i += kThreads) check(i, pages[pg0 + i]);
    }
    lost = __syncthreads_or(lost) ? 1 : 0;
    // a token's page (one out of range reads page 0 instead)
    auto id_of = [&](unsigned p) {
        if (cached) return F.pages[p - pg0];
        const int id = pages[p];
        return id < 0 || id >= A.num_pages ? 0 : id;
    };
    auto offset_of = [&](int t) {
        const unsigned p = page_of(t);
        return id_of(p) * A.page_stride + int64_t(unsigned(t) - p * A.page_size) * A.token_stride;
    };

    // ---- the warp's pieces: K tiles warp, warp + kWarps, ... of 64 tokens, all
    // their slices of 32 dimensions; then V jobs warp, warp + kWarps, ... (chunk,
    // slice), 64 tokens at a time
    const int nsl = (d + 31) / 32, tiles = (t1 - t0 + kTokens - 1) / kTokens, jobs = my * nsl;
    const uint32_t ring = smem_u32(smem_raw) + warp * stages * kPieceBytes, bars = smem_u32(&F.full[warp][0]);
    int kt = warp, ksl = 0, vj = warp, vt = 0, vsl = 0, vend = 0, slot_in = 0;
    int64_t off[2] = {0, 0};
    auto offsets = [&](int t, int end) {      // of the piece's tokens lane, lane + 32
        if (LOAD == kTma) return;
        if (t + lane < end) off[0] = offset_of(t + lane);
        if (t + lane + 32 < end) off[1] = offset_of(t + lane + 32);
    };
    auto issue = [&](const float *src, const CUtensorMap *map, int t, int sl, int end) {
        const uint32_t dst = ring + slot_in * kPieceBytes, bar = bars + 8 * slot_in;
        slot_in = slot_in + 1 == stages ? 0 : slot_in + 1;
        const int live = min(kTokens, end - t);
        if constexpr (LOAD == kTma) {
            const int boxes = (live + A.box - 1) / A.box;
            if (lane == 0) mbar_arrive_expect_tx(bar, boxes * A.box * 128);
            __syncwarp();
            if (lane < boxes) {
                const int at = t + lane * A.box;
                const unsigned p = page_of(at);
                tma_load_4d(dst + lane * A.box * 128, map, 32 * sl, g,
                            int(unsigned(at) - p * A.page_size), id_of(p), bar);
            }
        } else if constexpr (LOAD == kCopy16) {
            const int col = lane & 7, r0 = lane >> 3;
            const bool in = 4 * col < d - 32 * sl;
            src += 32 * sl + 4 * col;
#pragma unroll
            for (int i = 0; i < kTokens / 4; ++i) {
                const int r = 4 * i + r0;
                const int64_t at = __shfl_sync(0xffffffffu, off[i >> 3], r & 31);
                if (in && r < live) cp_async<16>(dst + r * 128 + ((col ^ (r & 7)) << 4), src + at);
            }
        } else {
            const bool in = lane < d - 32 * sl;
            src += 32 * sl + lane;
#pragma unroll 8
            for (int r = 0; r < kTokens; ++r) {
                const int64_t at = __shfl_sync(0xffffffffu, r < 32 ? off[0] : off[1], r & 31);
                if (in && r < live)
                    cp_async<4>(dst + r * 128 + ((((lane >> 2) ^ (r & 7)) << 4) | (lane & 3) << 2),
                                src + at);
            }
        }
    };
    auto issue_next = [&]() {
        if (kt < tiles) {
            const int t = t0 + kTokens * kt;
            if (ksl == 0) offsets(t, t1);
            issue(kb, &kmap, t, ksl, t1);
            if (++ksl == nsl) {
                ksl = 0;
                kt += kWarps;
            }
        } else if (vj < jobs) {
            if (vt >= vend) {               // the next job: its slice and tokens
                const int c = vj / nsl;
                vsl = vj - c * nsl;
                vt = t0 + c * kKChunk;
                vend = min(t1, vt + kKChunk);
            }
            offsets(vt, vend);
            issue(vb, &vmap, vt, vsl, vend);
            vt += kTokens;
            if (vt >= vend) vj += kWarps;
        }
        if (LOAD != kTma) cp_commit();
    };
    for (int i = 0; i < stages - 1; ++i) issue_next();
    int slot = 0;
    uint32_t phase = 0;
    bool stuck = false;           // a wait gave up: the rest wait no more, the ring stops there
    auto turn = [&]() {
        if (++slot == stages) {
            slot = 0;
            phase ^= 1;
        }
    };
    auto next_piece = [&]() {
        if constexpr (LOAD == kTma) {
            if (!stuck) stuck = __any_sync(0xffffffffu, !wait_for_piece(bars, slot, phase, stages));
        } else {
            if (stages == 3) cp_wait<1>(); else cp_wait<0>();
        }
        __syncwarp();
        if (!stuck) issue_next();   // into the slot consumed before this one
        const uint32_t p = ring + slot * kPieceBytes;
        if (!stuck) turn();
        return p;
    };
    // shared-memory offsets in a piece: 16-byte unit c of row `lane`, and column
    // `lane` of rows r = 0..7 mod 8
    uint32_t kat[8], vat[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        kat[i] = lane * 128 + ((i ^ (lane & 7)) << 4);
        vat[i] = i * 128 + (((lane >> 2) ^ i) << 4) + ((lane & 3) << 2);
    }

    // ---- scores
    float m[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) m[h] = __uint_as_float(0xff800000u);
    for (int tl = warp; tl < tiles; tl += kWarps) {
        float acc[2][NH];               // of tokens lane and lane + 32
#pragma unroll
        for (int h = 0; h < NH; ++h) acc[0][h] = acc[1][h] = 0.0f;
        for (int sl = 0; sl < nsl; ++sl) {
            const uint32_t piece = next_piece();
            const int width = min(32, d - 32 * sl);
            const float *q = &F.rows[0][32 * sl];
            auto four = [&](int i) {
                const float4 k0 = lds4(piece + kat[i]), k1 = lds4(piece + 4096 + kat[i]);
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const float4 qv = *reinterpret_cast<const float4 *>(q + h * 256 + 4 * i);
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
                for (int i = 0; i < 8; ++i) four(i);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (4 * i + 4 <= width) {
                        four(i);
                    } else if (4 * i < width) {
                        for (int c = 4 * i; c < width; ++c) {
                            const float k0 = lds1(piece + kat[i] + 4 * (c & 3));
                            const float k1 = lds1(piece + 4096 + kat[i] + 4 * (c & 3));
#pragma unroll
                            for (int h = 0; h < NH; ++h) {
                                acc[0][h] = __fmaf_rn(q[h * 256 + c], k0, acc[0][h]);
                                acc[1][h] = __fmaf_rn(q[h * 256 + c], k1, acc[1][h]);
                            }
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int t = t0 + kTokens * tl + 32 * k + lane;
            if (t < t1) {
#pragma unroll
                for (int h = 0; h < NH; ++h)
                    if (h < nh) {
                        const float x = __fmul_rn(acc[k][h], A.scale);
                        xs[h * xs_ld + (t - t0)] = x;
                        m[h] = max_nan(m[h], x);
                    }
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
    if (C > 1) cluster.barrier_wait();
    if (tid < NH) {
        float t = F.red[tid][0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) t = max_nan(t, F.red[tid][w]);
        for (int r = 0; r < C; ++r) *cluster.map_shared_rank(&F.top[rank][tid], r) = t;
    }
    if (tid < C) *cluster.map_shared_rank(&F.lost[rank], tid) = lost;
    meet();
    for (int r = 0; r < C; ++r) lost |= F.lost[r];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
        m[h] = F.top[0][h];
        for (int r = 1; r < C; ++r) m[h] = max_nan(m[h], F.top[r][h]);
    }
    // ---- e in place of x, and the chains of S: a warp 32 chains of a head, which
    // it walks through the cluster's runs kDeep groups at a time (slots past n
    // hold anything and are not added); the total goes to every CTA
    for (int i = warp * C + rank; i < nh * 8; i += C * kWarps) {
        const int h = i >> 3, l = (i & 7) * 32 + lane;
        float top = m[0];
#pragma unroll
        for (int k = 1; k < NH; ++k) top = h == k ? m[k] : top;
        const bool finite = fabsf(top) <= 0x1.fffffep127f;
        float sum = 0.0f;
        Walk w(l >> 6, base, rem);
        for (int t = 4 * l; t < n; t += 1024 * kDeep) {
            float4 *at[kDeep], e[kDeep];
#pragma unroll
            for (int u = 0; u < kDeep; ++u) {
                if (t + 1024 * u >= n) break;
                w.settle();
                at[u] = reinterpret_cast<float4 *>(scores_of(w.r) + h * xs_ld +
                                                   w.place * kKChunk + (t & 255));
                e[u] = *at[u];
                w.place += 4;
            }
#pragma unroll
            for (int u = 0; u < kDeep; ++u) {
                const int tu = t + 1024 * u;
                if (tu >= n) break;
                const float4 x = e[u];
                e[u] = finite ? exp4(x, top) : exp4_any(x, top);
                *at[u] = e[u];
                sum = __fadd_rn(sum, e[u].x);
                if (tu + 1 < n) sum = __fadd_rn(sum, e[u].y);
                if (tu + 2 < n) sum = __fadd_rn(sum, e[u].z);
                if (tu + 3 < n) sum = __fadd_rn(sum, e[u].w);
            }
        }
        for (int r = 0; r < C; ++r) *cluster.map_shared_rank(&F.rows[h][l], r) = sum;
    }
    meet();
    for (int i = warp; i < nh * 8; i += kWarps) {
        const float s = butterfly32(F.rows[i >> 3][(i & 7) * 32 + lane]);
        if (lane == 0) F.red[i >> 3][i & 7] = s;
    }
    __syncthreads();
    // ---- p in place, or, from the workspace, with each piece
    float inv[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
        const float *t = F.red[min(h, nh - 1)];
        inv[h] = __fdiv_rn(
            1.0f, __fadd_rn(__fadd_rn(__fadd_rn(t[0], t[1]), __fadd_rn(t[2], t[3])),
                            __fadd_rn(__fadd_rn(t[4], t[5]), __fadd_rn(t[6], t[7]))));
        if (on_chip && h < nh) {
            float4 *x4 = reinterpret_cast<float4 *>(xs + h * xs_ld);
            for (int i = tid; i < (t1 - t0 + 3) >> 2; i += kThreads) {
                const float4 e = x4[i];
                x4[i] = make_float4(__fmul_rn(e.x, inv[h]), __fmul_rn(e.y, inv[h]),
                                    __fmul_rn(e.z, inv[h]), __fmul_rn(e.w, inv[h]));
            }
        }
    }
    __syncthreads();
    // ---- P V: chunk partials (registers past the unit's heads repeat its last)
    uint32_t pat[NH];             // shared-memory addresses of the heads' rows
    const uint32_t copies = smem_u32(&F.rows[0][0]) + warp * (NH * kTokens * 4);
#pragma unroll
    for (int h = 0; h < NH; ++h)
        pat[h] = on_chip ? smem_u32(room) + min(h, nh - 1) * int(xs_ld) * 4
                         : copies + h * (kTokens * 4);
    float keep[2 * NH];           // of the next piece, from the workspace
    auto ask = [&](int t, int end) {
#pragma unroll
        for (int i = 0; i < 2 * NH; ++i) {
            const int at = t + 32 * (i & 1) + lane;
            keep[i] = at < end ? xs[min(i >> 1, nh - 1) * xs_ld + at] : 0.0f;
        }
    };
    auto end_of = [&](int c) { return min(t1 - t0, (c + 1) * kKChunk); };
    if (!on_chip && warp < jobs) ask(warp / nsl * kKChunk, end_of(warp / nsl));
    for (int j = warp; j < jobs; j += kWarps) {
        const int c = j / nsl, sl = j - c * nsl;
        const int end = end_of(c);
        float acc[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) acc[h] = 0.0f;
        for (int t = c * kKChunk; t < end; t += kTokens) {
            const uint32_t piece = next_piece();
            if (!on_chip) {
#pragma unroll
                for (int i = 0; i < 2 * NH; ++i)
                    sts1(copies + (i * 32 + lane) * 4, __fmul_rn(keep[i], inv[i / 2]));
                __syncwarp();
                if (t + kTokens < end) {
                    ask(t + kTokens, end);
                } else if (j + kWarps < jobs) {
                    const int next = (j + kWarps) / nsl;
                    ask(next * kKChunk, end_of(next));
                }
            }
            const uint32_t po = on_chip ? t * 4 : 0;
            auto four = [&](int r) {
                const uint32_t up = piece + (r & ~7) * 128;
                const float v0 = lds1(up + vat[r & 7]), v1 = lds1(up + vat[(r & 7) + 1]),
                            v2 = lds1(up + vat[(r & 7) + 2]), v3 = lds1(up + vat[(r & 7) + 3]);
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const float4 w = lds4(pat[h] + po + r * 4);
                    acc[h] = __fmaf_rn(w.x, v0, acc[h]);
                    acc[h] = __fmaf_rn(w.y, v1, acc[h]);
                    acc[h] = __fmaf_rn(w.z, v2, acc[h]);
                    acc[h] = __fmaf_rn(w.w, v3, acc[h]);
                }
            };
            const int live = end - t;
            if (live >= kTokens) {
#pragma unroll
                for (int r = 0; r < kTokens; r += 4) four(r);
            } else {
#pragma unroll 2
                for (int r8 = 0; r8 < kTokens; r8 += 8) {
#pragma unroll
                    for (int r = 0; r < 8; r += 4) {
                        if (r8 + r + 4 <= live) {
                            const uint32_t up = piece + r8 * 128;
                            const float v0 = lds1(up + vat[r]), v1 = lds1(up + vat[r + 1]),
                                        v2 = lds1(up + vat[r + 2]), v3 = lds1(up + vat[r + 3]);
#pragma unroll
                            for (int h = 0; h < NH; ++h) {
                                const float4 w = lds4(pat[h] + po + (r8 + r) * 4);
                                acc[h] = __fmaf_rn(w.x, v0, acc[h]);
                                acc[h] = __fmaf_rn(w.y, v1, acc[h]);
                                acc[h] = __fmaf_rn(w.z, v2, acc[h]);
                                acc[h] = __fmaf_rn(w.w, v3, acc[h]);
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (r8 + r + k < live) {
                                    const float v = lds1(piece + r8 * 128 + vat[r + k]);
#pragma unroll
                                    for (int h = 0; h < NH; ++h)
                                        acc[h] = __fmaf_rn(lds1(pat[h] + po + (r8 + r + k) * 4), v,
                                                           acc[h]);
                                }
                        }
                    }
                }
            }
        }
        if (32 * sl + lane < d)
#pragma unroll
            for (int h = 0; h < NH; ++h)
                if (h < nh) xs[part_at + (int64_t(h) * most + c) * d + 32 * sl + lane] = acc[h];
    }
    if (LOAD != kTma) cp_wait<0>();
    if (LOAD == kTma && stuck) {        // let the copies in flight land, tell the cluster
        for (; slot != slot_in; turn()) (void)mbar_wait_bounded(bars + 8 * slot, phase);
        if (lane == 0) {
            atomicOr(&g_decode_watchdog, kWatchdogDecode);
            for (int r = 0; r < C; ++r) *cluster.map_shared_rank(&F.lost[rank], r) = 2;
        }
    }
    meet();
    for (int r = 0; r < C; ++r) lost |= F.lost[r];
    // ---- the chunks left to right
    for (int i = (warp * C + rank) * 32 + lane; i < nh * d; i += C * kThreads) {
        const int h = i / d;
        float t = 0.0f;
        for (int r = 0; r < C; ++r) {
            const float *p = scores_of(r) + part_at + int64_t(h) * most * d + (i - h * d);
            const int chunks = base + (r < rem);
            for (int cg = 0; cg < chunks; cg += 16) {
                float v[16];
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if (cg + k < chunks) v[k] = p[int64_t(cg + k) * d];
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if (cg + k < chunks) t = r + cg + k == 0 ? v[k] : __fadd_rn(t, v[k]);
            }
        }
        o[i] = lost ? __uint_as_float(0x7fc00000u) : t;
    }
    if ((lost & 1) && rank == 0 && tid == 0 && A.dev_status)
        atomicOr(reinterpret_cast<int *>(A.dev_status), 2);
    if (C > 1) cluster.sync();    // the others still read this CTA's shared memory
}

int register_heads(int nh) { return nh <= 2 ? nh : nh <= 4 ? 4 : kMaxHeads; }

// Shared memory of a CTA before the room.
size_t fixed_bytes(int nh) {
    switch (register_heads(nh)) {
        case 1: return sizeof(Fixed<1>);
        case 2: return sizeof(Fixed<2>);
        case 4: return sizeof(Fixed<4>);
        default: return sizeof(Fixed<kMaxHeads>);
    }
}

struct DecodePlan {
    int unit_heads, batches, cluster, stages;
    int room;                     // floats of shared memory
    int64_t ws_cta, ws_bytes;
};

// The cluster: the largest power of two whose units all fit on the GPU at once
// (and no more CTAs than the longest row has chunks). us on one GB300 with 1 / 2 /
// 4 / 8 / 16 CTAs, 12 heads of 64: 64 requests of 700..2048 tokens 93 / 110 / 132 /
// 237 / 542; 8 of 1024..2048: 30 / 24 / 24 / 37 / 78; one of 32768: 430 / 224 / 110 /
// 67 / 50. 32 heads of 128 over 8: 4 requests of 22853..32768: 907 / 464 / 247 /
// 178 / 256; over 4: 32 of 2000..4096: 189 / 129 / 148 / 176 / 309. Sizes between
// powers of two measured slower than the power below. Two stages where a CTA's run is at most two chunks (three CTAs then fit
// an SM: 256 requests of 100..512 tokens 112 -> 95), three else.
DecodePlan decode_plan(int64_t batch, int64_t heads, int64_t kv_heads, int64_t head_dim,
                       int64_t max_len) {
    DecodePlan p;
    const int64_t per_kv = heads / kv_heads;
    p.batches = int((per_kv + kMaxHeads - 1) / kMaxHeads);
    p.unit_heads = int((per_kv + p.batches - 1) / p.batches);
    const int64_t units = std::max<int64_t>(1, batch * kv_heads * p.batches);
    const int64_t chunks = (max_len + kKChunk - 1) / kKChunk;
    const int64_t slots = int64_t(sm_count_current_device()) * kCtasPerSm;
    int64_t c = 1;
    while (2 * c <= kMaxCluster && 2 * c * units <= slots && 2 * c <= chunks) c *= 2;
    p.cluster = int(c);
    const int64_t run = (chunks + c - 1) / c;         // a CTA's most chunks
    p.stages = run <= 2 ? 2 : kStages;
    const int64_t need = int64_t(p.unit_heads) * run * (kKChunk + head_dim);
    const int64_t cap =
        (kSmemPerCta - p.stages * kRingBytes - int64_t(fixed_bytes(p.unit_heads))) / 4;
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
                    0, p.unit_heads, p.batches, p.stages, max_pages, dev_status};
    for (int i = 0; i < 31; ++i)
        if (c.page_size == int64_t(1) << i) A.page_shift = i;
    auto al16 = [](const void *x) { return reinterpret_cast<uintptr_t>(x) % 16 == 0; };
    const bool vec = al16(c.k) && al16(c.v) && c.page_stride % 4 == 0 &&
                     c.token_stride % 4 == 0 && c.head_stride % 4 == 0;
    Loader load = vec && c.head_dim % 4 == 0 ? kCopy16 : kCopy4;
    CUtensorMap kmap = {}, vmap = {};
    const bool boxes = c.page_size == 8 || c.page_size == 16 || c.page_size == 32 ||
                       c.page_size % kTokens == 0;
    if (vec && boxes) {
        A.box = int(std::min<int64_t>(c.page_size, kTokens));
        const int64_t extent[4] = {c.head_dim, c.kv_heads, c.page_size, c.num_pages};
        const int64_t stride[3] = {c.head_stride, c.token_stride, c.page_stride};
        const uint32_t box[4] = {32, 1, uint32_t(A.box), 1};
        if (make_tensor_map_4d(&kmap, c.k, extent, stride, box) &&
            make_tensor_map_4d(&vmap, c.v, extent, stride, box))
            load = kTma;
    }
    auto run = [&](auto kern) {
        const size_t smem =
            size_t(p.stages) * kRingBytes + fixed_bytes(p.unit_heads) + size_t(p.room) * 4;
        // the most any plan takes: the limit is the kernel's, and another thread's call
        // of another size may come between this line and the launch
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kSmemPerCta);
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
        e = cudaLaunchKernelEx(&cfg, kern, A, kmap, vmap);
        return e == cudaSuccess ? cudaGetLastError() : e;
    };
    auto pick = [&](auto heads_in) {
        constexpr int NH = decltype(heads_in)::value;
        return load == kTma      ? run(decode_kernel<NH, kTma>)
               : load == kCopy16 ? run(decode_kernel<NH, kCopy16>)
                                 : run(decode_kernel<NH, kCopy4>);
    };
    switch (register_heads(p.unit_heads)) {
        case 1: return pick(std::integral_constant<int, 1>());
        case 2: return pick(std::integral_constant<int, 2>());
        case 4: return pick(std::integral_constant<int, 4>());
        default: return pick(std::integral_constant<int, kMaxHeads>());
    }
}

cudaError_t decode_watchdog(unsigned int *code, int clear) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_decode_watchdog, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    if (clear && *code) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_decode_watchdog, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace det
