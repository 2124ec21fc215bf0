// decode_shared.cu -- decode attention of requests that share a prefix in a paged
// cache, its keys and values read once a group, for sm_103a.
//
// The mathematics and every bit are decode.cu's; what changes is that scores and chunk
// partials are formed by units: a group's shared tokens with all its query rows, and
// each request's own tokens with its rows.
//   1. plan: of each group, the 256-token chunks whose pages are the same ids in all
//      its requests; of each request, the chunks of its own;
//   2. scores: for a unit, a key-value head and a chunk, S = Q K^T, kept in the
//      workspace, and the rows' maxima;
//   3. sums: e = exp(x - m) in place, the 256 chains of S over the row, 1 / S;
//   4. partials: for a unit, a key-value head and a chunk, P V;
//   5. join: each row's chunk partials, left to right.
// The profile's chains are of fmaf, so the products run on the CUDA cores: with R
// rows, a key and value (2 x 4 bytes a dimension) take 2 R multiply-adds, and from R of
// about 24 on they, not HBM, bound a unit. Scores lie in octets of 8 tokens, a group's
// rows side by side: [octet][row][8], so a warp's stores of 4 rows x 8 tokens and its
// loads of exps are whole 128-byte lines, and a block of rows is one bulk copy an octet.
// Own tokens with few rows (decode_few.cu) are bound by HBM; their kernels run behind
// those of the shared ones and beside their last waves. Every launch overlaps the end
// of the one before (programmatic dependent launches).
// Measured: 48 requests on a document of 20001..24000 tokens, 32 heads of 128 over 8, 541
// us (32 TFLOP/s; scores 180 us and P V 168, the FMA pipe about 65% busy, sums 48, own
// tokens 45 of which some is hidden, the join 15); 64 requests on 8100..8192 tokens and up
// to 1000 of their own, 12 heads of 64, 140 us (1.8 TB/s, 12 TFLOP/s: seven dependent
// launches of 5 to 35 us).
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "decode_shared.cuh"

namespace cg = cooperative_groups;

#ifdef DET_TEST_SHARED_HOW
// Of the test suite's copies of the library: how groups are read whatever their size
// (det::How), below 0 as the estimate says.
extern "C" __attribute__((visibility("default"))) int det_test_shared_how = -1;
#endif

namespace det {

// Set when a bounded wait for a piece gave up.
__device__ unsigned int g_shared_watchdog;

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanRows = 1024;                    // requests looked through at once
constexpr int kPlanCtas = 8;                       // of a cluster
constexpr size_t kScoreRing = size_t(kWarps) * kRingBytes;
constexpr int kScoreRows = 4;                      // of a thread
constexpr int kScoreCtas = 3;                      // an SM's
constexpr int kPvTokens = 16;                      // of a step of P V
constexpr int kPvGrid = 3;                         // CTAs an SM, where two run: finer shares

// ---------------------------------------------------------------- plan
// A cluster of up to 8 CTAs a group. Every request keeps a token of its own, so a
// chunk is shared where it ends before the shortest's last token. A request whose own
// pages are not all in order has no chunks and no part in the rest. What bounds it is
// the latency of the lengths, then the shared pages, then the own ones: 32 columns of
// the table are a warp's, and where there are few, the requests are dealt out too.
__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedArgs A) {
    __shared__ int s_least, s_lead, s_live, s_bad, who[kPlanRows], found[kPlanCtas];
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int g = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int w0 = rank * (kPlanThreads / 32) + warp, all = C * (kPlanThreads / 32);
    const int b0 = g * A.group, b1 = min(A.batch, b0 + A.group);
    auto in_order = [&](int n) { return n > 0 && n <= A.max_len; };
    if (C > 1) cluster.barrier_arrive();    // waited for before the first remote access
    grid_dependency_wait();
    allow_dependents();
    if (tid == 0) {
        s_least = s_lead = s_bad = INT32_MAX;
        s_live = 0;
    }
    __syncthreads();
    int live = 0, status = 0, least = INT32_MAX, first_live = INT32_MAX;
    for (int b = b0 + tid; b < b1; b += kPlanThreads) {
        const int n = A.kv_lens[b];
        if (!in_order(n)) {
            if (n != 0) status = 1;
            continue;
        }
        least = min(least, n);
        first_live = min(first_live, b);
        ++live;
    }
    if (live) {
        atomicMin(&s_least, least);
        atomicMin(&s_lead, first_live);
        atomicAdd(&s_live, live);
    }
    for (int64_t i = int64_t(b0) * A.heads + rank * kPlanThreads + tid; i < int64_t(b1) * A.heads;
         i += C * kPlanThreads)
        A.top[i] = 0;
    __syncthreads();
    if (C > 1) cluster.barrier_wait();
    int chunks = 0;
    if (s_live > 1) {
        chunks = (s_least - 1) / kKChunk;
        const int64_t ps = A.page_size;
        const int pages = int((int64_t(chunks) * kKChunk + ps - 1) / ps);
        const int32_t *first = A.table + s_lead * A.ldt;
        const int cols = (pages + 31) / 32;
        for (int r0 = b0; r0 < b1; r0 += kPlanRows) {
            const int rows = min(kPlanRows, b1 - r0);
            __syncthreads();
            if (tid < rows) who[tid] = in_order(A.kv_lens[r0 + tid]) ? r0 + tid : s_lead;
            __syncthreads();
            const int parts = cols ? max(1, min(rows, all / cols)) : 0;
            for (int i = w0; i < cols * parts; i += all) {
                const int part = i / cols, j = (i - part * cols) * 32 + lane;
                if (j >= pages) continue;
                const int id = first[j];
                bool bad = id < 0 || id >= A.num_pages;
#pragma unroll 8
                for (int r = part; r < rows; r += parts) bad |= A.table[who[r] * A.ldt + j] != id;
                if (bad) atomicMin(&s_bad, j);
            }
        }
        __syncthreads();
        int bad = s_bad;
        if (C > 1) {
            if (tid < C) *cluster.map_shared_rank(found + rank, tid) = bad;
            cluster.sync();
            for (int r = 0; r < C; ++r) bad = min(bad, found[r]);
        }
        if (bad != INT32_MAX) chunks = min(chunks, int(bad * ps / kKChunk));
    }
    if (rank == 0 && tid == 0) {
        A.chunks[g] = chunks;
        A.lead[g] = s_live ? s_lead : b0;
    }
    // the requests' own pages
    for (int b = b0 + w0; b < b1; b += all) {
        const int n = A.kv_lens[b];
        int own = 0;
        if (in_order(n)) {
            const int32_t *row = A.table + b * A.ldt;
            const int last = page_of(A, n - 1);
            int bad = 0;
            for (int j = int(page_of(A, chunks * kKChunk)) + lane; j <= last; j += 32) {
                const int id = row[j];
                bad |= id < 0 || id >= A.num_pages;
            }
            bad = __any_sync(0xffffffffu, bad);
            own = bad ? 0 : (n + kKChunk - 1) / kKChunk - chunks;
            if (bad) status |= 2;
        }
        if (lane == 0) A.own[b] = own;
    }
    if (A.dev_status) {
        status = __reduce_or_sync(0xffffffffu, unsigned(status));
        if (lane == 0 && status) atomicOr(reinterpret_cast<int *>(A.dev_status), status);
    }
}

// RT consecutive floats of shared memory as pairs.
template <int RT>
__device__ __forceinline__ void load_pairs(const float *p, f32x2 (&v)[RT / 2]) {
#pragma unroll
    for (int i = 0; i < RT / 4; ++i) {
        const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(p + 4 * i);
        v[2 * i] = w.x;
        v[2 * i + 1] = w.y;
    }
}
__device__ __forceinline__ float part_of(const float4 &v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// ---------------------------------------------------------------- scores
// An item: 16 rows, a chunk's 256 tokens; a warp 64 tokens (8 lanes x 8, tokens 8
// apart, so that 16-byte reads along the dimensions of 8 keys meet no bank
// conflict), 4 lanes x RT = 4 rows (4 apart; 8 and 16 rows a lane took as long on large
// cases, 176..185 us for scores of 180, and longer on small ones). A warp's keys come
// through a ring of its own, so warps meet only where the rows change; the query rows
// stay in shared memory, transposed, while they do not.
template <bool OWN, Loader LOAD>
__global__ void __launch_bounds__(kThreads, kScoreCtas)
    shared_scores_kernel(const SharedArgs A, const __grid_constant__ CUtensorMap kmap) {
    constexpr int RT = kScoreRows, R = 4 * RT;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    float *qs = reinterpret_cast<float *>(smem_raw + kScoreRing);
    __shared__ Share share;
    __shared__ int rows[R];           // (b, h) of the row at qs's place
    __shared__ uint64_t full[kWarps][kRingPieces];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tl = lane & 7, rl = lane >> 3;
    const int d = A.d, nsl = (d + 31) / 32, mul = A.kv_heads * A.row_blocks;
    init_bars<LOAD>(&full[0][0]);
    Beside<OWN> beside;
    shares<OWN, 1>(A, mul, blockIdx.x, 1, gridDim.x, &share);
    const int64_t items = share.items;
    if (items <= 0) return;
    Ring<LOAD> ring(A, &kmap, A.k, smem_u32(smem_raw) + warp * kRingBytes, smem_u32(&full[warp][0]));

    // ---- keys
    Item in = share.at;
    int64_t in_items = items;
    int in_sl = 0, in_t0 = 0, in_live = 0, in_kv = 0;
    auto seek = [&]() {               // the warp's tile of the item, or of the next that has one
        while (in_items > 0) {
            const int t0 = first_token<OWN>(in);
            in_t0 = t0 + kTile * warp;
            in_live = min(kTile, tokens_from<OWN>(in, t0) - kTile * warp);
            if (in_live > 0) {
                in_kv = in.run / A.row_blocks;
                ring.look_up(pages_of<OWN>(A, in), in_t0, in_live);
                return;
            }
            advance<OWN>(A, mul, in);
            --in_items;
        }
    };
    seek();
    auto issue = [&]() {
        if (in_items > 0) {
            ring.fetch(in_kv, in_sl, in_t0, in_live);
            if (++in_sl == nsl) {
                in_sl = 0;
                advance<OWN>(A, mul, in);
                --in_items;
                seek();
            }
        }
        if (LOAD != kTma) cp_commit();
    };
    for (int i = 0; i < kRingPieces - 1; ++i) issue();
    Item it = share.at;
    int held_u = -1, held_run = -1;
    for (int64_t i = 0; i < items; ++i) {
        const int kv = it.run / A.row_blocks, r0 = (it.run - kv * A.row_blocks) * R;
        const int g = group_of<OWN>(A, it.u);
        const int t0 = first_token<OWN>(it), live = tokens_from<OWN>(it, t0);
        if (it.u != held_u || it.run != held_run) {         // other rows
            held_u = it.u;
            held_run = it.run;
            __syncthreads();
            // qs's place p has row p / RT + 4 (p mod RT)
            const int p = tid % R, r = r0 + p / RT + 4 * (p % RT);
            const int place = place_of<OWN>(A, it.u, r);
            const int row = r < rows_of<OWN>(A) ? row_at(A, g, kv, place) : -1;
            if (tid < R) rows[p] = row;
            const int b = row / A.heads;
            const float *q = A.q + b * A.ldq + int64_t(row - b * A.heads) * d;
            for (int j = tid / R; j < d; j += kThreads / R) qs[j * R + p] = row >= 0 ? q[j] : 0.0f;
            __syncthreads();
        }
        if (OWN && kTile * warp >= live) {      // the request ends before this warp's tokens
            advance<OWN>(A, mul, it);
            continue;
        }
        f32x2 acc[RT / 2][8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
#pragma unroll
            for (int r = 0; r < RT / 2; ++r) acc[r][c] = 0;
        }
        for (int sl = 0; sl < nsl; ++sl) {
            ring.wait();
            if (!ring.stuck) issue();           // into the slot consumed before this one
            const uint32_t keys = ring.piece() + tl * 128;
            const float *qp = qs + 32 * sl * R + rl * RT;
            auto four = [&](int g4, int live4) {
                float4 k[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) k[c] = lds4(keys + c * 1024 + ((g4 ^ tl) << 4));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    if (kk >= live4) break;
                    const float *p = qp + (4 * g4 + kk) * R;
                    f32x2 a[RT / 2];
                    load_pairs<RT>(p, a);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const f32x2 kc = splat2(part_of(k[c], kk));
#pragma unroll
                        for (int r = 0; r < RT / 2; ++r) acc[r][c] = fma2(a[r], kc, acc[r][c]);
                    }
                }
            };
            const int width = min(32, d - 32 * sl);
            if (width == 32) {
#pragma unroll
                for (int g4 = 0; g4 < 8; ++g4) four(g4, 4);
            } else {
                for (int g4 = 0; 4 * g4 < width; ++g4) four(g4, width - 4 * g4);
            }
        }
        if (ring.stuck) {             // this and the other rows of the share are NaN
            if (lane < R && rows[lane] >= 0) atomicMax(A.top + rows[lane], 0xffffffffu);
        } else {
            const int64_t octet = (int64_t(g) * A.kv_heads + kv) * A.octets + t0 / 8 + 8 * warp;
            float *x = A.x + (octet * A.rows + place_of<OWN>(A, it.u, r0 + rl)) * 8 + tl;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int row = rows[rl * RT + r];
                float most = __uint_as_float(0xff800000u);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    float s, other;
                    unpack2(acc[r / 2][c], s, other);
                    if (r & 1) s = other;
                    const float v = __fmul_rn(s, A.scale);
                    const bool here = !OWN || 64 * warp + 8 * c + tl < live;
                    if (row >= 0 && here) x[c * A.rows * 8 + r * 32] = v;
                    if (here) most = max_nan(most, v);
                }
#pragma unroll
                for (int off = 4; off >= 1; off >>= 1)
                    most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, off));
                if (tl == 0 && row >= 0) atomicMax(A.top + row, max_key(most));
            }
        }
        advance<OWN>(A, mul, it);
    }
    ring.drain(&g_shared_watchdog);
}

// ---------------------------------------------------------------- sums
// A CTA four rows of a group and head: 8 lanes have the two halves of 4 octets of a
// row, so 8 of its 256 chains; a thread a chain, in ascending order.
constexpr int kSumThreads = 1024;
constexpr int kSumRows = 4;
constexpr int kSumDeep = 4;                        // groups of a chain in flight

__global__ void __launch_bounds__(kSumThreads) shared_sums_kernel(const SharedArgs A) {
    __shared__ float chains[kSumRows][256], red[kSumRows][8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 3, place = blockIdx.x * kSumRows + r;
    // the scores written last are still in L2, and are read first
    const int gkv = gridDim.y - 1 - blockIdx.y, g = gkv / A.kv_heads, kv = gkv % A.kv_heads;
    grid_dependency_wait();
    allow_dependents();
    const int row = place < A.rows ? row_at(A, g, kv, place) : -1;
    const int n = row >= 0 ? A.kv_lens[row / A.heads] : 0;
    const float m = row >= 0 ? max_of_key(A.top[row]) : 0.0f;
    const bool finite = fabsf(m) <= 0x1.fffffep127f;
    float *x = A.x + (int64_t(gkv) * A.octets * A.rows + place) * 8;
    for (int l = 8 * warp + (lane & 7); l < 256; l += 8 * (kSumThreads / 32)) {
        float sum = 0.0f;
        for (int t = 4 * l; t < n; t += 1024 * kSumDeep) {
            float4 e[kSumDeep];
#pragma unroll
            for (int u = 0; u < kSumDeep; ++u)
                if (t + 1024 * u < n)
                    e[u] = *reinterpret_cast<const float4 *>(
                        x + (t / 8 + 128 * u) * A.rows * 8 + (t & 4));
#pragma unroll
            for (int u = 0; u < kSumDeep; ++u) {
                const int tu = t + 1024 * u;
                if (tu >= n) break;
                e[u] = finite ? exp4(e[u], m) : exp4_any(e[u], m);
                *reinterpret_cast<float4 *>(x + (t / 8 + 128 * u) * A.rows * 8 + (t & 4)) = e[u];
                sum = __fadd_rn(sum, e[u].x);
                if (tu + 1 < n) sum = __fadd_rn(sum, e[u].y);
                if (tu + 2 < n) sum = __fadd_rn(sum, e[u].z);
                if (tu + 3 < n) sum = __fadd_rn(sum, e[u].w);
            }
        }
        chains[r][l] = sum;
    }
    __syncthreads();
    for (int i = warp; i < kSumRows * 8; i += kSumThreads / 32) {
        const float s = butterfly32(chains[i >> 3][(i & 7) * 32 + lane]);
        if (lane == 0) red[i >> 3][i & 7] = s;
    }
    __syncthreads();
    if (warp == 0 && (lane & 7) == 0 && row >= 0) {
        const float *t = red[r];
        A.inv[row] = __fdiv_rn(
            1.0f, __fadd_rn(__fadd_rn(__fadd_rn(t[0], t[1]), __fadd_rn(t[2], t[3])),
                            __fadd_rn(__fadd_rn(t[4], t[5]), __fadd_rn(t[6], t[7]))));
    }
}

// ---------------------------------------------------------------- partials
// An item: 4 TR rows, 32 DH dimensions, a chunk; it is a warp's alone (4 lanes x TR
// rows, 4 apart; 8 lanes x 4 DH dimensions), which walks the chunk's tokens 16 at a time
// with a ring of its own: values, and exps as they lie (two octets of a block of rows are
// two bulk copies). Accumulators pair dimensions, which come in pairs; an exp is
// multiplied by 1 / S where it is used, once for 4 DH multiply-adds a lane.
template <int TR, int DH>
struct PvWarp {
    static constexpr int kR = 4 * TR;
    static constexpr int kValues = kPvTokens * 128 * DH;
    static constexpr int kStage = kValues + kPvTokens * kR * 4;
    static constexpr int kCtas = TR * DH >= 16 ? 2 : 3;       // an SM's, by registers
    static constexpr int kFit = int((kCtas == 2 ? kMaxSmem : 72 * 1024) / kWarps) / kStage;
    static constexpr int kStages = kFit < 8 ? kFit : 8;
    static constexpr size_t kBytes = size_t(kWarps) * kStages * kStage;
    static_assert(kStage % 1024 == 0 && kStages >= 2, "shared memory");
};

template <int TR, int DH, bool OWN, bool TMA>
__global__ void __launch_bounds__(kThreads, (PvWarp<TR, DH>::kCtas))
    shared_partials_kernel(const SharedArgs A, const __grid_constant__ CUtensorMap vmap) {
    using W = PvWarp<TR, DH>;
    constexpr int R = W::kR, STAGES = W::kStages;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ Share share[kWarps];
    __shared__ uint64_t full[kWarps][STAGES];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, dl = lane & 7, rl = lane >> 3;
    const int d = A.d, mul = A.kv_heads * A.row_blocks * A.dim_tiles;
    if (TMA && tid == 0) {
        for (int i = 0; i < kWarps * STAGES; ++i) mbar_init(smem_u32(&full[0][i]), 1);
        fence_mbar_init();
    }
    Beside<OWN> beside;
    shares<OWN, kWarps>(A, mul, blockIdx.x * kWarps, 1, gridDim.x * kWarps, share);
    const int64_t items = share[warp].items;
    if (items <= 0) return;
    const uint32_t ring = smem_u32(smem_raw) + warp * STAGES * W::kStage;
    // an item's key-value head, first row, and where its first octet's exps are
    auto head_of = [&](const Item &i) { return i.run / (A.row_blocks * A.dim_tiles); };
    auto row_of = [&](const Item &i) { return i.run / A.dim_tiles % A.row_blocks * R; };
    auto exps_of = [&](const Item &i, int t0) {
        const int64_t octet =
            (int64_t(group_of<OWN>(A, i.u)) * A.kv_heads + head_of(i)) * A.octets + t0 / 8;
        return A.x + (octet * A.rows + place_of<OWN>(A, i.u, row_of(i))) * 8;
    };

    // ---- values and exps
    Item in = share[warp].at;
    int64_t in_items = items;
    int in_t = 0, in_live = 0, in_slot = 0, in_id = 0;      // next token of the item, tokens left
    int in_kv = 0, in_dim0 = 0, in_alive = 0;
    const float *in_x = nullptr;
    const int32_t *in_pages = nullptr;
    const int per_half = TMA ? kPvTokens / A.box : 1;       // boxes of 32 dimensions
    auto look_up = [&]() {            // the page of the lane's box of the next step
        if (TMA && in_items > 0 && lane < DH * per_half && lane % per_half * A.box < in_live)
            in_id = in_pages[page_of(A, in_t + lane % per_half * A.box)];
    };
    auto start = [&]() {
        if (in_items <= 0) return;
        in_t = first_token<OWN>(in);
        in_live = tokens_from<OWN>(in, in_t);
        in_kv = head_of(in);
        in_dim0 = in.run % A.dim_tiles * 32 * DH;
        in_alive = min(R, rows_of<OWN>(A) - row_of(in));
        in_x = exps_of(in, in_t);
        in_pages = pages_of<OWN>(A, in);
    };
    start();
    look_up();
    auto issue = [&]() {
        if (in_items > 0) {
            const int kv = in_kv, dim0 = in_dim0, alive = in_alive;
            const uint32_t dst = ring + in_slot * W::kStage, bar = smem_u32(&full[warp][in_slot]);
            const int live = min(kPvTokens, in_live), octets = (live + 7) / 8;
            if constexpr (TMA) {
                const int boxes = (live + A.box - 1) / A.box;
                if (lane == 0)
                    mbar_arrive_expect_tx(bar, boxes * A.box * 128 * DH + octets * alive * 32);
                __syncwarp();
                const int half = lane / per_half, box = lane % per_half;
                if (half < DH && box < boxes) {
                    const int t = in_t + box * A.box;
                    tma_load_4d(dst + half * kPvTokens * 128 + box * A.box * 128, &vmap,
                                dim0 + 32 * half, kv,
                                int(unsigned(t) - page_of(A, t) * A.page_size), in_id, bar);
                } else if (lane >= 30 && lane - 30 < octets) {
                    const int o = lane - 30;
                    bulk_load(dst + W::kValues + o * R * 32, in_x + o * A.rows * 8, alive * 32, bar);
                }
            } else {
                for (int i = lane; i < octets * alive * 2; i += 32) {
                    const int o = i / (alive * 2), unit = i - o * alive * 2;
                    cp_async<16>(dst + W::kValues + o * R * 32 + unit * 16,
                                 in_x + o * A.rows * 8 + unit * 4);
                }
                const int32_t *pages = in_pages;
                const float *src = A.v + kv * A.head_stride + dim0;
                if (A.wide) {
                    for (int r = lane >> 3; r < live; r += 4) {
                        const float *from = src + offset_of(A, pages, in_t + r);
#pragma unroll
                        for (int half = 0; half < DH; ++half)
                            if (dim0 + 32 * half + 4 * dl < d)
                                cp_async<16>(dst + half * kPvTokens * 128 + r * 128 +
                                                 ((dl ^ (r & 7)) << 4),
                                             from + 32 * half + 4 * dl);
                    }
                } else {
                    for (int r = 0; r < live; ++r) {
                        const float *from = src + offset_of(A, pages, in_t + r);
#pragma unroll
                        for (int half = 0; half < DH; ++half)
                            if (dim0 + 32 * half + lane < d)
                                cp_async<4>(dst + half * kPvTokens * 128 + r * 128 +
                                                ((((lane >> 2) ^ (r & 7)) << 4) | (lane & 3) << 2),
                                            from + 32 * half + lane);
                    }
                }
            }
            in_slot = in_slot + 1 == STAGES ? 0 : in_slot + 1;
            in_t += kPvTokens;
            in_live -= kPvTokens;
            in_x += 2 * A.rows * 8;
            if (in_live <= 0) {
                advance<OWN>(A, mul, in);
                --in_items;
                start();
            }
            look_up();
        }
        if (!TMA) cp_commit();
    };
    for (int i = 0; i < STAGES - 1; ++i) issue();

    Item it = share[warp].at;
    int held_u = -1, held_block = -1, slot = 0;
    uint32_t phase = 0;
    bool stuck = false;
    auto step = [&]() {
        if (++slot == STAGES) {
            slot = 0;
            phase ^= 1;
        }
    };
    int mine[TR];                     // the lane's rows (b, h), -1 where there is none
    float inv[TR];
    for (int64_t i = 0; i < items; ++i) {
        if (it.u != held_u || it.run / A.dim_tiles != held_block) {
            held_u = it.u;
            held_block = it.run / A.dim_tiles;
            const int g = group_of<OWN>(A, it.u), kv = head_of(it), r0 = row_of(it);
#pragma unroll
            for (int r = 0; r < TR; ++r) {
                const int at = r0 + 4 * r + rl;
                mine[r] = at < rows_of<OWN>(A) ? row_at(A, g, kv, place_of<OWN>(A, it.u, at)) : -1;
                inv[r] = mine[r] >= 0 ? A.inv[mine[r]] : 0.0f;
            }
        }
        f32x2 acc[TR][2 * DH];
#pragma unroll
        for (int r = 0; r < TR; ++r)
#pragma unroll
            for (int k = 0; k < 2 * DH; ++k) acc[r][k] = 0;
        const int t0 = first_token<OWN>(it), tokens = tokens_from<OWN>(it, t0);
        for (int t1 = 0; t1 < tokens; t1 += kPvTokens) {
            if constexpr (TMA) {
                if (!stuck)
                    stuck = __any_sync(0xffffffffu,
                                       !wait_for_piece(smem_u32(&full[warp][0]), slot, phase, STAGES));
            } else {
                cp_wait<STAGES - 2>();
            }
            __syncwarp();
            if (!stuck) issue();      // into the slot consumed before this one
            const uint32_t vals = ring + slot * W::kStage;
            const uint32_t exps = vals + W::kValues + rl * 32;
            auto four = [&](int t4, int live) {
                float4 e[TR];
#pragma unroll
                for (int r = 0; r < TR; ++r)
                    e[r] = lds4(exps + (t4 >> 3) * R * 32 + r * 128 + (t4 & 4) * 4);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k >= live) break;
                    const int t = t4 + k;
                    const uint32_t at = vals + t * 128 + ((dl ^ (t & 7)) << 4);
                    f32x2 v[2 * DH];
#pragma unroll
                    for (int half = 0; half < DH; ++half) {
                        const float4 u = lds4(at + half * kPvTokens * 128);
                        v[2 * half] = pack2(u.x, u.y);
                        v[2 * half + 1] = pack2(u.z, u.w);
                    }
#pragma unroll
                    for (int r = 0; r < TR; ++r) {
                        const f32x2 w = splat2(__fmul_rn(part_of(e[r], k), inv[r]));
#pragma unroll
                        for (int c = 0; c < 2 * DH; ++c) acc[r][c] = fma2(w, v[c], acc[r][c]);
                    }
                }
            };
            if (!OWN || t1 + kPvTokens <= tokens) {
#pragma unroll
                for (int t = 0; t < kPvTokens; t += 4) four(t, 4);
            } else {
                for (int t = 0; t1 + t < tokens; t += 4) four(t, tokens - t1 - t);
            }
            if (!stuck) step();
        }
        // ---- the partials of the lane's rows and dimensions
        const int dim0 = it.run % A.dim_tiles * 32 * DH + 4 * dl;
#pragma unroll
        for (int r = 0; r < TR; ++r) {
            if (mine[r] < 0) continue;
            float *to = A.part + (mine[r] * A.ldpart + t0 / kKChunk) * d;
#pragma unroll
            for (int half = 0; half < DH; ++half) {
                float4 o;
                unpack2(acc[r][2 * half], o.x, o.y);
                unpack2(acc[r][2 * half + 1], o.z, o.w);
                if (stuck) o.x = o.y = o.z = o.w = __uint_as_float(0x7fc00000u);
                const int at = dim0 + 32 * half;
                if (d % 4 == 0) {
                    if (at < d) *reinterpret_cast<float4 *>(to + at) = o;
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (at + k < d) to[at + k] = part_of(o, k);
                }
            }
        }
        advance<OWN>(A, mul, it);
    }
    if (!TMA) cp_wait<0>();
    if (TMA && stuck) {                   // let the copies in flight land (as Ring::drain)
        for (; slot != in_slot; step()) (void)mbar_wait_bounded(smem_u32(&full[warp][slot]), phase);
        if (lane == 0) atomicOr(&g_shared_watchdog, kWatchdogDecode);
    }
}

// ---------------------------------------------------------------- join
// A thread an element of the output.
constexpr int kJoinDeep = 32;
__global__ void __launch_bounds__(kThreads) shared_join_kernel(const SharedArgs A) {
    const int b = blockIdx.y, i = blockIdx.x * kThreads + threadIdx.x;
    grid_dependency_wait();
    allow_dependents();
    if (i >= A.heads * A.d) return;
    const int n = A.kv_lens[b], h = i / A.d;
    const int chunks = A.own[b] ? (n + kKChunk - 1) / kKChunk : 0;
    const float *p = A.part + (int64_t(b) * A.heads + h) * A.ldpart * A.d + (i - h * A.d);
    float t = chunks || n == 0 ? 0.0f : __uint_as_float(0x7fc00000u);
    for (int c = 0; c < chunks; c += kJoinDeep) {
        float v[kJoinDeep];
#pragma unroll
        for (int k = 0; k < kJoinDeep; ++k)
            if (c + k < chunks) v[k] = p[int64_t(c + k) * A.d];
#pragma unroll
        for (int k = 0; k < kJoinDeep; ++k)
            if (c + k < chunks) t = c + k == 0 ? v[k] : __fadd_rn(t, v[k]);
    }
    A.out[b * A.ldo + i] = t;
}

// ---------------------------------------------------------------- host
constexpr size_t kSliceBytes = size_t(1) << 30;     // scores and partials of a round of heads

// How requests are read: each for itself (decode.cu), in small groups (decode_group.cu) or
// many together (this file), by an estimate of the three with rows as long as the table
// is wide; as they are shorter, only a gain of a tenth, or a quarter for this file's
// longer chain of launches, counts.
//  - each for itself: 18 us and the keys and values of all from L2 at 9 TB/s (with 4 and 8
//    heads of a key-value head 1.5 and 3 times as long for their multiply-adds);
//  - in groups: 34 us and each key and value once, with 200 tokens of its own a request, at
//    5.8 TB/s or 18 GB/s a CTA;
//  - together: 45 us and each once at 4.2 TB/s, or the multiply-adds at 20 TFLOP/s.
// Measured, us, each for itself / in groups: 12 heads of 64, 16 groups of 4 of 700..1900
// tokens 73 / 63, of 4500..6000 228 / 129, of 8 of 1100..1500 138 / 96; 4 groups of 4 of
// 1500 29 / 36; 16 groups of 2 with 4 query heads a key-value head of 6000 240 / 168. Each
// for itself / together: one group of 32 of 1500 50 / 65, of 6000 150 / 75; 4 groups of 4
// with 4 query heads a key-value head of 1500 46 / 68, of 6000 128 / 90.
// Where it is wrong: reading each for itself has at most 16 CTAs a unit too, which the first
// line leaves out (two requests of 32768 tokens with 8 query heads over one head of 128
// take 115 us so, 69 together); together is not weighed for 8 rows and fewer (one group of
// 8, a head of 128, 24000 tokens: 53 / 106 in groups / 58 together); and rows may be much
// shorter than the table is wide (two groups of 8 of 400 tokens, 12 heads of 64, in a table
// of 2^17: 12.5 us each for itself, 51 in groups; 48 of 1200, 32 heads of 128 over 8: 114
// and 170 together).
enum How { kAlone, kInGroups, kTogether };
How how_to_read(int64_t batch, int64_t group, int64_t heads, int64_t kv_heads, int64_t d,
                int64_t max_len) {
#ifdef DET_TEST_SHARED_HOW
    if (det_test_shared_how >= 0 && group >= 2)
        return det_test_shared_how == kInGroups && group * (heads / kv_heads) > kFewRows
                   ? kTogether
                   : How(det_test_shared_how);
#endif
    if (group < 2 || max_len <= 2 * kKChunk) return kAlone;
    const double token = 8.0 * double(kv_heads * d), len = double(max_len);
    const double per_kv = double(heads / kv_heads), groups = double((batch + group - 1) / group);
    const double alone = 18.0 + double(batch) * token * len / 9.0e6 * std::max(1.0, 0.37 * per_kv);
    if (double(group) * per_kv <= kFewRows) {
        const GroupPlan p = group_plan(int64_t(groups), 1, kv_heads, d, max_len);
        const double rate = std::min(5.8e6, 18.0e3 * double(p.units * p.cluster));
        return alone > 1.1 * (34.0 + groups * (len + 200.0 * double(group)) * token / rate)
                   ? kInGroups
                   : kAlone;
    }
    const double shared = 45.0 + std::max(groups * token * len / 4.2e6,
                                          double(batch) * per_kv * token * len / 2.0 / 20.0e6);
    return alone > 1.25 * shared ? kTogether : kAlone;
}

struct SharedPlan {
    How how;
    GroupPlan group;          // in groups; the rest is of this file
    int64_t groups, kv, heads, ldx, ldpart;      // kv, heads: of a round
    size_t top, inv, x, part, bytes;             // offsets in the workspace
};

SharedPlan shared_plan(int64_t batch, int64_t group, int64_t heads, int64_t kv_heads,
                       int64_t head_dim, int64_t max_len) {
    SharedPlan p = {};
    group = std::min(group, batch);
    const int64_t per_kv = heads / kv_heads;
    p.groups = group > 0 ? (batch + group - 1) / group : 0;
    p.how = how_to_read(batch, group, heads, kv_heads, head_dim, max_len);
    if (p.groups * group * heads >= 0x7fffffff / 8) p.how = kAlone;
    if (p.how == kInGroups) {
        p.group = group_plan(p.groups, group * per_kv, kv_heads, head_dim, max_len);
        p.bytes = p.group.bytes;
        return p;
    }
    if (p.how == kAlone) {
        p.bytes = decode_workspace_bytes(batch, heads, kv_heads, head_dim, max_len);
        return p;
    }
    p.ldpart = (max_len + kKChunk - 1) / kKChunk;
    p.ldx = p.ldpart * kKChunk;
    const int64_t rows = p.groups * group * per_kv;       // of a key-value head
    const size_t head = size_t(rows) * (p.ldx + p.ldpart * head_dim) * 4;
    p.kv = std::max<int64_t>(1, std::min<int64_t>(kv_heads, int64_t(kSliceBytes / head)));
    p.heads = p.kv * per_kv;
    auto after = [](size_t at, size_t bytes) { return (at + bytes + 255) / 256 * 256; };
    p.top = after(0, size_t(2 * p.groups + batch) * 4);
    p.inv = after(p.top, size_t(batch) * p.heads * 4);
    p.x = after(p.inv, size_t(batch) * p.heads * 4);
    p.part = after(p.x, size_t(rows) * p.kv * p.ldx * 4);
    p.bytes = after(p.part, size_t(batch) * p.heads * p.ldpart * head_dim * 4);
    return p;
}

template <class K>
cudaError_t run(K kern, int64_t grid, size_t smem, cudaStream_t s, const SharedArgs &A,
                const CUtensorMap &map) {
    // the most any call takes: the limit is the kernel's, and another thread's call may
    // come between this line and the launch
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMaxSmem));
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(unsigned(std::max<int64_t>(1, grid))), dim3(kThreads), smem,
                            s, A, map);
}

cudaError_t run_plan(const SharedArgs &A, int64_t max_pages, cudaStream_t s) {
    // CTAs a group: while a thread looks at many entries and SMs are idle
    int ctas = 1;
    while (ctas < kPlanCtas && A.groups * 2 * ctas <= sm_count_current_device() &&
           A.group * max_pages > int64_t(4) * kPlanThreads * ctas)
        ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(A.groups * ctas));
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, shared_plan_kernel, A);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

// most: the chunks of all units, at most.
template <bool OWN>
cudaError_t scores(SharedArgs A, const CUtensorMap *map, int64_t most, cudaStream_t s) {
    constexpr int R = 4 * kScoreRows;
    const int64_t rows = OWN ? A.per_kv : A.rows;
    A.row_blocks = int((rows + R - 1) / R);
    const int64_t grid = std::min<int64_t>(most * A.kv_heads * A.row_blocks,
                                           int64_t(sm_count_current_device()) * kScoreCtas);
    const size_t smem = kScoreRing + size_t(A.d) * R * 4;
    const CUtensorMap none = {};
    return map      ? run(shared_scores_kernel<OWN, kTma>, grid, smem, s, A, *map)
           : A.wide ? run(shared_scores_kernel<OWN, kCopy16>, grid, smem, s, A, none)
                    : run(shared_scores_kernel<OWN, kCopy4>, grid, smem, s, A, none);
}

template <int TR, int DH, bool OWN>
cudaError_t run_partials(SharedArgs A, const CUtensorMap *map, int64_t rows, int64_t most,
                         cudaStream_t s) {
    using W = PvWarp<TR, DH>;
    A.row_blocks = int((rows + W::kR - 1) / W::kR);
    A.dim_tiles = (A.d + 32 * DH - 1) / (32 * DH);
    const int64_t items = most * A.kv_heads * A.row_blocks * A.dim_tiles;
    const int64_t grid = std::min<int64_t>((items + kWarps - 1) / kWarps,
                                           int64_t(sm_count_current_device()) * kPvGrid);
    const CUtensorMap none = {};
    return map ? run(shared_partials_kernel<TR, DH, OWN, true>, grid, W::kBytes, s, A, *map)
               : run(shared_partials_kernel<TR, DH, OWN, false>, grid, W::kBytes, s, A, none);
}
// The rows and slices a lane takes: an item's time is as 6 + TR DH (measured: 53 cycles a
// token for 4 x 1, 65 for 4 x 2, 100 for 4 x 4, 104 for 8 x 2, 179 for 8 x 4), and a
// scheduler's items come one after the other.
template <bool OWN>
cudaError_t partials(const SharedArgs &A, const CUtensorMap *map, int64_t most, cudaStream_t s) {
    const int64_t rows = OWN ? A.per_kv : A.rows;
    const int64_t tiles = most * A.kv_heads, workers = int64_t(sm_count_current_device()) * kWarps;
    int best = 0;
    int64_t least = INT64_MAX;
    for (int tr = 4; tr <= 8; tr *= 2)
        for (int dh = 1; dh <= 4; dh *= 2) {
            if (dh > 1 && 16 * dh >= A.d) break;      // a half of the slices would be empty
            const int64_t items =
                tiles * ((rows + 4 * tr - 1) / (4 * tr)) * ((A.d + 32 * dh - 1) / (32 * dh));
            const int64_t cost = (items + workers - 1) / workers * (6 + tr * dh);
            if (cost < least) {
                least = cost;
                best = tr * 10 + dh;
            }
        }
    switch (best) {
        case 41: return run_partials<4, 1, OWN>(A, map, rows, most, s);
        case 42: return run_partials<4, 2, OWN>(A, map, rows, most, s);
        case 44: return run_partials<4, 4, OWN>(A, map, rows, most, s);
        case 81: return run_partials<8, 1, OWN>(A, map, rows, most, s);
        case 82: return run_partials<8, 2, OWN>(A, map, rows, most, s);
        default: return run_partials<8, 4, OWN>(A, map, rows, most, s);
    }
}

}  // namespace

size_t shared_decode_workspace_bytes(int64_t batch, int64_t group, int64_t heads,
                                     int64_t kv_heads, int64_t head_dim, int64_t max_len) {
    return shared_plan(batch, group, heads, kv_heads, head_dim, max_len).bytes;
}

cudaError_t launch_shared_decode(int64_t batch, int64_t group, int heads, const float *q,
                                 int64_t ldq, const det_kv_cache &c, const int32_t *table,
                                 int64_t max_pages, int64_t ldt, const int32_t *kv_lens,
                                 float scale, float *out, int64_t ldo, float *workspace,
                                 int32_t *dev_status, cudaStream_t s) {
    const int64_t max_len = max_pages * c.page_size, d = c.head_dim;
    const SharedPlan p = shared_plan(batch, group, heads, c.kv_heads, d, max_len);
    if (p.how == kAlone)
        return launch_decode_attention(batch, heads, q, ldq, c, table, max_pages, ldt, kv_lens,
                                       scale, out, ldo, workspace, dev_status, s);
    char *ws = reinterpret_cast<char *>(workspace);
    SharedArgs A = {};
    A.batch = int(batch);
    A.group = int(std::min(group, batch));
    A.groups = int(p.groups);
    A.per_kv = int(heads / c.kv_heads);
    A.rows = int64_t(A.group) * A.per_kv;
    A.d = int(d);
    A.ldq = ldq;
    A.num_pages = c.num_pages;
    A.page_size = unsigned(c.page_size);
    A.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (c.page_size == int64_t(1) << i) A.page_shift = i;
    A.page_stride = c.page_stride;
    A.token_stride = c.token_stride;
    A.head_stride = c.head_stride;
    A.table = table;
    A.ldt = ldt;
    A.kv_lens = kv_lens;
    A.max_len = max_len;
    A.scale = scale;
    A.chunks = reinterpret_cast<int *>(ws);
    A.lead = A.chunks + p.groups;
    A.own = A.lead + p.groups;
    A.top = reinterpret_cast<unsigned *>(ws + p.top);
    A.inv = reinterpret_cast<float *>(ws + p.inv);
    A.x = reinterpret_cast<float *>(ws + p.x);
    A.octets = p.ldx / 8;
    A.part = reinterpret_cast<float *>(ws + p.part);
    A.ldpart = p.ldpart;
    A.ldo = ldo;
    A.dev_status = dev_status;
    auto al16 = [](const void *x) { return reinterpret_cast<uintptr_t>(x) % 16 == 0; };
    const bool vec = al16(c.k) && al16(c.v) && c.page_stride % 4 == 0 &&
                     c.token_stride % 4 == 0 && c.head_stride % 4 == 0;
    A.wide = vec && d % 4 == 0;
    const bool boxes = c.page_size == 8 || c.page_size == 16 || c.page_size == 32 ||
                       c.page_size % 64 == 0;
    const int kbox = int(std::min<int64_t>(c.page_size, 64));
    const int vbox = int(std::min<int64_t>(c.page_size, kPvTokens));
    if (p.how == kInGroups) {
        A.kv_heads = int(c.kv_heads);
        A.heads = heads;
        A.k = c.k;
        A.v = c.v;
        A.q = q;
        A.out = out;
        A.x = reinterpret_cast<float *>(ws);
        A.part = reinterpret_cast<float *>(ws + p.group.part);
        A.box = kbox;
        CUtensorMap maps[2] = {};
        const int64_t extent[4] = {d, c.kv_heads, c.page_size, c.num_pages};
        const int64_t stride[3] = {c.head_stride, c.token_stride, c.page_stride};
        const uint32_t box[4] = {32, 1, uint32_t(kbox), 1};
        const bool tma = vec && boxes && make_tensor_map_4d(&maps[0], c.k, extent, stride, box) &&
                         make_tensor_map_4d(&maps[1], c.v, extent, stride, box);
        return launch_group_decode(A, p.group, tma ? maps : nullptr, s);
    }
    const bool few = A.per_kv <= kFewRows;        // rows of a request
    const int64_t most = p.groups * p.ldpart, most_own = batch * p.ldpart;
    for (int64_t g0 = 0; g0 < c.kv_heads; g0 += p.kv) {
        A.kv_heads = int(std::min(p.kv, c.kv_heads - g0));
        A.heads = A.kv_heads * A.per_kv;
        A.k = c.k + g0 * c.head_stride;
        A.v = c.v + g0 * c.head_stride;
        A.q = q + g0 * A.per_kv * d;
        A.out = out + g0 * A.per_kv * d;
        CUtensorMap kmap = {}, vmap = {}, vmap_few = {};
        bool tma = false;
        if (vec && boxes) {
            const int64_t extent[4] = {d, A.kv_heads, c.page_size, c.num_pages};
            const int64_t stride[3] = {c.head_stride, c.token_stride, c.page_stride};
            tma = make_tensor_map_4d(&kmap, A.k, extent, stride, {32, 1, uint32_t(kbox), 1}) &&
                  make_tensor_map_4d(&vmap, A.v, extent, stride, {32, 1, uint32_t(vbox), 1}) &&
                  make_tensor_map_4d(&vmap_few, A.v, extent, stride, {32, 1, uint32_t(kbox), 1});
        }
        cudaError_t e = run_plan(A, max_pages, s);
        A.box = kbox;
        const CUtensorMap *map = tma ? &kmap : nullptr;
        if (e == cudaSuccess) e = scores<false>(A, map, most, s);
        if (e == cudaSuccess)
            e = few ? launch_few_scores(A, map, most_own, s) : scores<true>(A, map, most_own, s);
        if (e == cudaSuccess) {
            e = launch_dependent(shared_sums_kernel,
                                 dim3(unsigned((A.rows + kSumRows - 1) / kSumRows),
                                      unsigned(p.groups * A.kv_heads)),
                                 dim3(kSumThreads), 0, s, A);
        }
        A.box = vbox;
        map = tma ? &vmap : nullptr;
        if (e == cudaSuccess) e = partials<false>(A, map, most, s);
        if (e == cudaSuccess && few) {
            A.box = kbox;
            e = launch_few_partials(A, tma ? &vmap_few : nullptr, most_own, s);
        } else if (e == cudaSuccess) {
            e = partials<true>(A, map, most_own, s);
        }
        if (e == cudaSuccess) {
            e = launch_dependent(shared_join_kernel,
                                 dim3(unsigned((A.heads * d + kThreads - 1) / kThreads),
                                      unsigned(batch)),
                                 dim3(kThreads), 0, s, A);
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t shared_decode_watchdog(unsigned int *code, int clear) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_shared_watchdog, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    if (clear && *code) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_shared_watchdog, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace det
