// decode_shared.cu -- decode attention of requests that share a prefix in a paged
// cache, its keys and values read once a group, for sm_103a.
//
// The mathematics and every bit are decode.cu's; what changes is who forms the
// scores and chunk partials of the tokens that a group's requests have in common:
//   1. plan: of each group, the 256-token chunks whose pages are the same ids in all
//      its requests;
//   2. scores: for a group, a key-value head and a chunk, S = Q K^T for all the
//      group's query rows of that head, kept in the workspace, and the rows' maxima;
//   3. decode.cu's kernel for each request's own tokens, which also takes the
//      maximum over both, walks the chains of S through the shared scores (leaving
//      their exps in place) and says 1 / S;
//   4. partials: P V of each shared chunk for all rows of the group;
//   5. join: each row's chunk partials, left to right.
// The profile's chains are of fmaf, so the products run on the CUDA cores: with R
// rows a key and value (2 x 4 bytes a dimension) takes 2 R multiply-adds, and from R of
// about 24 on they, not HBM, bound the shared part. As in the GEMM, shared memory's
// rate sets the register tile: up to 16 rows x 8 tokens (or dimensions) a thread.
#include <algorithm>
#include <type_traits>

#include "decode.cuh"

namespace det {

// Set when a bounded wait for a piece gave up.
__device__ unsigned int g_shared_watchdog;

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kPlanThreads = 1024;
constexpr unsigned kWatchdogDecode = 32u;          // det_watchdog_status bit 5
constexpr int kScoreStage = kKChunk * 128;         // a chunk's tokens x 32 dimensions
constexpr int kScoreStages = 2;
constexpr int kPvTokens = 16;                      // of a step of P V
constexpr int kPvSteps = kKChunk / kPvTokens;
constexpr int kPvStages = 3;

struct SharedArgs {
    int batch, group, groups, heads, kv_heads, per_kv, d;
    const float *q;
    int64_t ldq;
    const float *k, *v;
    int64_t num_pages;
    unsigned page_size;
    int page_shift;           // log2(page_size), or -1
    int64_t page_stride, token_stride, head_stride;
    const int32_t *table;
    int64_t max_pages, ldt;
    const int32_t *kv_lens;
    int64_t max_len;
    float scale;
    int box;                  // tokens of a TMA box
    int row_blocks, dim_tiles;
    int *chunks, *lead;       // of each group: shared chunks, a request in order
    unsigned *top;
    float *x;
    int64_t ldx;
    const float *inv;
    float *part;
    int64_t ldpart;
    float *out;
    int64_t ldo;
};

__device__ __forceinline__ bool in_order(const SharedArgs &A, int n) {
    return n > 0 && n <= A.max_len;
}

// ---------------------------------------------------------------- plan
// A CTA a group. Every request keeps a token of its own, so a chunk is shared where
// it ends before the shortest's last token.
__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const SharedArgs A) {
    __shared__ int s_least, s_lead, s_live, s_bad;
    const int g = blockIdx.x, tid = threadIdx.x;
    const int b0 = g * A.group, b1 = min(A.batch, b0 + A.group);
    if (tid == 0) {
        s_least = s_lead = s_bad = INT32_MAX;
        s_live = 0;
    }
    __syncthreads();
    int live = 0;
    for (int b = b0 + tid; b < b1; b += kPlanThreads) {
        const int n = A.kv_lens[b];
        if (!in_order(A, n)) continue;
        atomicMin(&s_least, n);
        atomicMin(&s_lead, b);
        ++live;
    }
    if (live) atomicAdd(&s_live, live);
    for (int i = b0 * A.heads + tid; i < b1 * A.heads; i += kPlanThreads) A.top[i] = 0;
    __syncthreads();
    int chunks = 0;
    if (s_live > 1) {
        chunks = (s_least - 1) / kKChunk;
        const int64_t ps = A.page_size;
        const int pages = int((int64_t(chunks) * kKChunk + ps - 1) / ps);
        const int32_t *first = A.table + s_lead * A.ldt;
        // 256 pages at a time, the requests dealt out to four
        const int col = tid & 255, part = tid >> 8;
        for (int j0 = 0; j0 < pages; j0 += 256) {
            const int j = j0 + col;
            bool bad = false;
            if (j < pages) {
                const int id = first[j];
                bad = id < 0 || id >= A.num_pages;
#pragma unroll 8
                for (int b = b0 + part; b < b1; b += 4)
                    bad |= A.table[b * A.ldt + j] != id && in_order(A, A.kv_lens[b]);
            }
            if (bad) atomicMin(&s_bad, j);
            if (__syncthreads_or(bad)) break;
        }
        if (s_bad != INT32_MAX) chunks = min(chunks, int(s_bad * ps / kKChunk));
    }
    if (tid == 0) {
        A.chunks[g] = chunks;
        A.lead[g] = s_live ? s_lead : b0;
    }
}

// ---------------------------------------------------------------- work
// The items of a kernel: for each group `mul` runs (of heads and blocks of rows or
// dimensions) of its shared chunks, the chunk fastest.
struct Item {
    int g, run, c, n;         // n: the group's chunks
};

// Every worker's share [lo, hi) of the items is an equal run of them; its first
// item. All threads of the CTA call; worker w < workers of the CTA are numbers first
// .. first + workers - 1 of `all`.
struct Share {
    int64_t lo, hi;
    Item at;
};
template <int WORKERS>
__device__ __forceinline__ void shares(const SharedArgs &A, int mul, int first, int all,
                                       Share *out) {
    __shared__ int64_t warp_sums[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (A.groups + kThreads - 1) / kThreads;
    const int g0 = min(A.groups, tid * per), g1 = min(A.groups, g0 + per);
    int64_t sum = 0;
    for (int g = g0; g < g1; ++g) sum += A.chunks[g];
    int64_t in = sum;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
        const int64_t o = __shfl_up_sync(0xffffffffu, in, off);
        if (lane >= off) in += o;
    }
    if (lane == 31) warp_sums[warp] = in;
    __syncthreads();
    int64_t before = in - sum, total = 0;
    for (int w = 0; w < kWarps; ++w) {
        before += w < warp ? warp_sums[w] : 0;
        total += warp_sums[w];
    }
    total *= mul;
    for (int w = 0; w < WORKERS; ++w) {
        const int64_t lo = total * (first + w) / all, hi = total * (first + w + 1) / all;
        if (tid == 0) {
            out[w].lo = lo;
            out[w].hi = hi;
        }
        if (lo < hi && before * mul <= lo && lo < (before + sum) * mul) {
            int64_t at = before;
            int g = g0;
            while ((at + A.chunks[g]) * mul <= lo) at += A.chunks[g++];
            const int n = A.chunks[g];
            const int64_t i = lo - at * mul;
            out[w].at = {g, int(i / n), int(i % n), n};
        }
    }
    __syncthreads();
}
__device__ __forceinline__ void advance(const SharedArgs &A, int mul, Item &it) {
    if (++it.c < it.n) return;
    it.c = 0;
    if (++it.run < mul) return;
    it.run = 0;
    do {
        ++it.g;
    } while (it.g < A.groups && (it.n = A.chunks[it.g]) == 0);
}

__device__ __forceinline__ unsigned page_of(const SharedArgs &A, int t) {
    return A.page_shift >= 0 ? unsigned(t) >> A.page_shift : unsigned(t) / A.page_size;
}
// A token's offset in the cache (its page is in order: the plan has seen it).
__device__ __forceinline__ int64_t offset_of(const SharedArgs &A, const int32_t *pages, int t) {
    const unsigned p = page_of(A, t);
    return pages[p] * A.page_stride + int64_t(unsigned(t) - p * A.page_size) * A.token_stride;
}
// Row r of a group's rows of key-value head kv: its number b * heads + h, or -1
// where there is none or its request is not in order.
__device__ __forceinline__ int row_of(const SharedArgs &A, int g, int kv, int r) {
    const int m = r / A.per_kv, b = g * A.group + m;
    if (m >= A.group || b >= A.batch || !in_order(A, A.kv_lens[b])) return -1;
    return b * A.heads + kv * A.per_kv + (r - m * A.per_kv);
}

// RT consecutive floats of shared memory as pairs.
template <int RT>
__device__ __forceinline__ void load_pairs(const float *p, f32x2 (&v)[RT / 2]) {
    if constexpr (RT == 2) {
        v[0] = *reinterpret_cast<const f32x2 *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < RT / 4; ++i) {
            const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(p + 4 * i);
            v[2 * i] = w.x;
            v[2 * i + 1] = w.y;
        }
    }
}
__device__ __forceinline__ float part_of(const float4 &v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// ---------------------------------------------------------------- scores
// An item: 4 RT rows, a chunk's 256 tokens; a warp 64 tokens (8 lanes x 8, tokens 8
// apart, so that 16-byte reads along the dimensions of 8 keys meet no bank
// conflict), 4 lanes x RT rows. Keys come 32 dimensions at a time, a stage ahead; the
// query rows stay in shared memory, transposed, while they do not change.
template <int RT, Loader LOAD>
__global__ void __launch_bounds__(kThreads, RT >= 8 ? 2 : 3)
    shared_scores_kernel(const SharedArgs A, const __grid_constant__ CUtensorMap kmap) {
    constexpr int R = 4 * RT;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    float *qs = reinterpret_cast<float *>(smem_raw + kScoreStages * kScoreStage);
    __shared__ Share share;
    __shared__ int rows[R];
    __shared__ uint64_t full[kScoreStages];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tl = lane & 7, rl = lane >> 3;
    const int d = A.d, nsl = (d + 31) / 32, mul = A.kv_heads * A.row_blocks;
    if (LOAD == kTma && tid == 0) {
        for (int i = 0; i < kScoreStages; ++i) mbar_init(smem_u32(full + i), 1);
        fence_mbar_init();
    }
    shares<1>(A, mul, blockIdx.x, gridDim.x, &share);
    const int64_t items = share.hi - share.lo;
    if (items <= 0) return;
    const uint32_t ring = smem_u32(smem_raw);

    // ---- keys
    Item in = share.at;
    int in_sl = 0, in_slot = 0;
    int64_t left = items * nsl;
    const int boxes = LOAD == kTma ? kKChunk / A.box : 1;      // at most 32
    int id = 0;               // warp 0: the page of the lane's box
    auto ask_page = [&]() {
        if (LOAD == kTma && warp == 0 && lane < boxes && in.g < A.groups)
            id = A.table[A.lead[in.g] * A.ldt + page_of(A, in.c * kKChunk + lane * A.box)];
    };
    ask_page();
    auto issue = [&]() {
        if (left > 0) {
            --left;
            const int kv = in.run / A.row_blocks, t0 = in.c * kKChunk;
            const uint32_t dst = ring + in_slot * kScoreStage, bar = smem_u32(full + in_slot);
            if constexpr (LOAD == kTma) {
                if (warp == 0) {
                    if (lane == 0) mbar_arrive_expect_tx(bar, kScoreStage);
                    __syncwarp();
                    if (lane < boxes) {
                        const int t = t0 + lane * A.box;
                        tma_load_4d(dst + lane * A.box * 128, &kmap, 32 * in_sl, kv,
                                    int(unsigned(t) - page_of(A, t) * A.page_size), id, bar);
                    }
                }
            } else {
                const int32_t *pages = A.table + A.lead[in.g] * A.ldt;
                const float *src = A.k + kv * A.head_stride + 32 * in_sl;
                if constexpr (LOAD == kCopy16) {
                    const int col = tid & 7;
                    if (4 * col < d - 32 * in_sl)
                        for (int r = tid >> 3; r < kKChunk; r += kThreads / 8)
                            cp_async<16>(dst + r * 128 + ((col ^ (r & 7)) << 4),
                                         src + offset_of(A, pages, t0 + r) + 4 * col);
                } else {
                    if (lane < d - 32 * in_sl)
                        for (int r = warp; r < kKChunk; r += kWarps)
                            cp_async<4>(dst + r * 128 + ((((lane >> 2) ^ (r & 7)) << 4) |
                                                         (lane & 3) << 2),
                                        src + offset_of(A, pages, t0 + r) + lane);
                }
            }
            in_slot ^= 1;
            if (++in_sl == nsl) {
                in_sl = 0;
                advance(A, mul, in);
                ask_page();
            }
        }
        if (LOAD != kTma) cp_commit();
    };
    issue();
    Item it = share.at;
    int held_g = -1, held_run = -1, slot = 0;
    uint32_t phase = 0;
    bool stuck = false;
    for (int64_t i = 0; i < items; ++i) {
        const int kv = it.run / A.row_blocks, rb = it.run - kv * A.row_blocks;
        if (it.g != held_g || it.run != held_run) {         // other rows
            held_g = it.g;
            held_run = it.run;
            __syncthreads();
            for (int r = tid; r < R; r += kThreads) rows[r] = row_of(A, it.g, kv, rb * R + r);
            const int r = tid % R, m = (rb * R + r) / A.per_kv, b = it.g * A.group + m;
            const bool there = m < A.group && b < A.batch;
            const float *q =
                A.q + b * A.ldq + int64_t(kv * A.per_kv + rb * R + r - m * A.per_kv) * d;
            for (int j = tid / R; j < d; j += kThreads / R) qs[j * R + r] = there ? q[j] : 0.0f;
        }
        f32x2 acc[RT >= 2 ? RT / 2 : 1][8];
        float one[RT == 1 ? 8 : 1];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
#pragma unroll
            for (int r = 0; r < RT / 2; ++r) acc[r][c] = 0;
            if (RT == 1) one[c] = 0.0f;
        }
        for (int sl = 0; sl < nsl; ++sl) {
            if constexpr (LOAD == kTma) {
                if (!stuck) stuck = !mbar_wait_bounded(smem_u32(full + slot), phase);
                stuck = __syncthreads_or(stuck);
                if (stuck) break;
            } else {
                cp_wait<0>();
                __syncthreads();
            }
            issue();              // into the slot consumed before this one
            const uint32_t keys = ring + slot * kScoreStage + (64 * warp + tl) * 128;
            const float *qp = qs + 32 * sl * R + rl * RT;
            auto four = [&](int g4, int live) {
                float4 k[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) k[c] = lds4(keys + c * 1024 + ((g4 ^ tl) << 4));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    if (kk >= live) break;
                    const float *p = qp + (4 * g4 + kk) * R;
                    if constexpr (RT >= 2) {
                        f32x2 a[RT / 2];
                        load_pairs<RT>(p, a);
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const f32x2 kc = splat2(part_of(k[c], kk));
#pragma unroll
                            for (int r = 0; r < RT / 2; ++r) acc[r][c] = fma2(a[r], kc, acc[r][c]);
                        }
                    } else {
                        const float a = *p;
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            one[c] = __fmaf_rn(a, part_of(k[c], kk), one[c]);
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
            slot ^= 1;
            phase ^= slot == 0;
        }
        if (stuck) {              // this and the other rows of the share are NaN
            for (int r = tid; r < R; r += kThreads) {
                const int row = row_of(A, it.g, kv, rb * R + r);
                if (row >= 0) atomicMax(A.top + row, 0xffffffffu);
            }
        } else {
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int row = rows[rl * RT + r];
                float most = __uint_as_float(0xff800000u);
                float *to = A.x + row * A.ldx + it.c * kKChunk + 64 * warp + tl;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    float s, other;
                    if constexpr (RT == 1) {
                        s = one[c];
                    } else {
                        unpack2(acc[r / 2][c], s, other);
                        if (r & 1) s = other;
                    }
                    const float x = __fmul_rn(s, A.scale);
                    if (row >= 0) to[8 * c] = x;
                    most = max_nan(most, x);
                }
#pragma unroll
                for (int off = 4; off >= 1; off >>= 1)
                    most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, off));
                if (tl == 0 && row >= 0) atomicMax(A.top + row, max_key(most));
            }
        }
        advance(A, mul, it);
    }
    if (LOAD == kTma && stuck) {          // let the copies in flight land
        for (int i = 0; i < kScoreStages; ++i) {
            (void)mbar_wait_bounded(smem_u32(full + slot), phase);
            slot ^= 1;
            phase ^= slot == 0;
        }
        if (tid == 0) atomicOr(&g_shared_watchdog, kWatchdogDecode);
    }
}

// ---------------------------------------------------------------- partials
// An item: 4 RT rows, 32 DH dimensions, a chunk; it is a warp's alone (4 lanes x RT
// rows, 8 lanes x 4 DH dimensions), which walks the chunk's tokens 16 at a time:
// values by its own ring, exps loaded a step ahead, multiplied by 1 / S and laid
// down transposed.
template <int RT, int DH>
struct PvWarp {
    static constexpr int kR = 4 * RT;
    static constexpr int kStage = kPvTokens * 128 * DH;
    static constexpr int kBytes = (kPvStages * kStage + kPvTokens * kR * 4 + 1023) / 1024 * 1024;
};

template <int RT, int DH, Loader LOAD>
__global__ void __launch_bounds__(kThreads, RT >= 8 ? 2 : 3)
    shared_partials_kernel(const SharedArgs A, const __grid_constant__ CUtensorMap vmap) {
    using W = PvWarp<RT, DH>;
    constexpr int R = W::kR;
    constexpr int LOADS = R / 8 > 1 ? R / 8 : 1;      // 16-byte loads of exps a lane and step
    constexpr int OWN = R == 64 ? 2 : 1;              // rows whose exps a lane loads
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ Share share[kWarps];
    __shared__ uint64_t full[kWarps][kPvStages];
    __shared__ int rows[kWarps][R];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, dl = lane & 7, rl = lane >> 3;
    const int d = A.d, mul = A.kv_heads * A.row_blocks * A.dim_tiles;
    if (LOAD == kTma && tid == 0) {
        for (int i = 0; i < kWarps * kPvStages; ++i) mbar_init(smem_u32(&full[0][i]), 1);
        fence_mbar_init();
    }
    shares<kWarps>(A, mul, blockIdx.x * kWarps, gridDim.x * kWarps, share);
    const int64_t items = share[warp].hi - share[warp].lo;
    if (items <= 0) return;
    const uint32_t ring = smem_u32(smem_raw) + warp * W::kBytes;
    float *ps = reinterpret_cast<float *>(smem_raw + warp * W::kBytes + kPvStages * W::kStage);

    // ---- values
    Item in = share[warp].at;
    int in_step = 0, in_slot = 0;
    int64_t left = items * kPvSteps;
    const int per_half = LOAD == kTma ? kPvTokens / A.box : 1;       // boxes of 32 dimensions
    int id = 0;
    auto ask_page = [&]() {
        if (LOAD == kTma && lane < DH * per_half && in.g < A.groups)
            id = A.table[A.lead[in.g] * A.ldt +
                         page_of(A, in.c * kKChunk + in_step * kPvTokens + lane % per_half * A.box)];
    };
    ask_page();
    auto issue = [&]() {
        if (left > 0) {
            --left;
            const int kv = in.run / (A.row_blocks * A.dim_tiles), dim0 = in.run % A.dim_tiles * 32 * DH;
            const int t0 = in.c * kKChunk + in_step * kPvTokens;
            const uint32_t dst = ring + in_slot * W::kStage, bar = smem_u32(&full[warp][in_slot]);
            if constexpr (LOAD == kTma) {
                if (lane == 0) mbar_arrive_expect_tx(bar, W::kStage);
                __syncwarp();
                if (lane < DH * per_half) {
                    const int half = lane / per_half, box = lane % per_half, t = t0 + box * A.box;
                    tma_load_4d(dst + half * kPvTokens * 128 + box * A.box * 128, &vmap,
                                dim0 + 32 * half, kv,
                                int(unsigned(t) - page_of(A, t) * A.page_size), id, bar);
                }
            } else {
                const int32_t *pages = A.table + A.lead[in.g] * A.ldt;
                const float *src = A.v + kv * A.head_stride + dim0;
                if constexpr (LOAD == kCopy16) {
                    for (int r = lane >> 3; r < kPvTokens; r += 4) {
                        const float *from = src + offset_of(A, pages, t0 + r);
#pragma unroll
                        for (int half = 0; half < DH; ++half)
                            if (dim0 + 32 * half + 4 * dl < d)
                                cp_async<16>(dst + half * kPvTokens * 128 + r * 128 +
                                                 ((dl ^ (r & 7)) << 4),
                                             from + 32 * half + 4 * dl);
                    }
                } else {
                    for (int r = 0; r < kPvTokens; ++r) {
                        const float *from = src + offset_of(A, pages, t0 + r);
#pragma unroll
                        for (int half = 0; half < DH; ++half)
                            if (dim0 + 32 * half + lane < d)
                                cp_async<4>(dst + half * kPvTokens * 128 + r * 128 +
                                                ((((lane >> 2) ^ (r & 7)) << 4) | (lane & 3) << 2),
                                            from + 32 * half + lane);
                    }
                }
            }
            in_slot = in_slot + 1 == kPvStages ? 0 : in_slot + 1;
            if (++in_step == kPvSteps) {
                in_step = 0;
                advance(A, mul, in);
            }
            ask_page();
        }
        if (LOAD != kTma) cp_commit();
    };
    for (int i = 0; i < kPvStages - 1; ++i) issue();

    // ---- exps: load i of a lane is of row (lane + 32 i) mod R, tokens 4 ((lane + 32 i) / R) on
    const float *from[OWN];
    float inv[OWN];
    float4 e[LOADS];
    const bool loads = R >= 8 || lane < 16;
    auto ask = [&](int t) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            e[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (loads && from[i % OWN])
                e[i] = *reinterpret_cast<const float4 *>(from[i % OWN] + t +
                                                         4 * ((lane + 32 * i) / R));
        }
    };
    Item it = share[warp].at;
    int held_g = -1, held_run = -1, slot = 0;
    uint32_t phase = 0;
    bool stuck = false;
    auto hold = [&]() {           // the item's rows
        if (it.g == held_g && it.run == held_run) return;
        held_g = it.g;
        held_run = it.run;
        const int block = it.run / A.dim_tiles, kv = block / A.row_blocks;
        const int r0 = (block - kv * A.row_blocks) * R;
        __syncwarp();
        for (int r = lane; r < R; r += 32) rows[warp][r] = row_of(A, it.g, kv, r0 + r);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int row = rows[warp][(lane + 32 * i) % R];
            from[i] = row >= 0 ? A.x + row * A.ldx : nullptr;
            inv[i] = row >= 0 ? A.inv[row] : 0.0f;
        }
    };
    hold();
    ask(it.c * kKChunk);
    constexpr bool kRowPairs = RT >= 8;
    for (int64_t i = 0; i < items; ++i) {
        constexpr int N0 = kRowPairs ? RT / 2 : RT, N1 = kRowPairs ? 4 * DH : 2 * DH;
        f32x2 acc[N0][N1];
#pragma unroll
        for (int a = 0; a < N0; ++a)
#pragma unroll
            for (int b = 0; b < N1; ++b) acc[a][b] = 0;
        const Item now = it;
        int mine[RT];             // the rows whose partials the lane has
#pragma unroll
        for (int r = 0; r < RT; ++r) mine[r] = rows[warp][rl * RT + r];
        for (int step = 0; step < kPvSteps; ++step) {
            __syncwarp();
#pragma unroll
            for (int k = 0; k < LOADS; ++k)
                if (loads) {
                    float *to = ps + 4 * ((lane + 32 * k) / R) * R + (lane + 32 * k) % R;
                    const float w = inv[k % OWN];
                    to[0] = __fmul_rn(e[k].x, w);
                    to[R] = __fmul_rn(e[k].y, w);
                    to[2 * R] = __fmul_rn(e[k].z, w);
                    to[3 * R] = __fmul_rn(e[k].w, w);
                }
            if (step + 1 < kPvSteps) {
                ask(it.c * kKChunk + (step + 1) * kPvTokens);
            } else if (i + 1 < items) {
                advance(A, mul, it);
                hold();
                ask(it.c * kKChunk);
            }
            if constexpr (LOAD == kTma) {
                if (!stuck)
                    stuck = __any_sync(0xffffffffu,
                                       !mbar_wait_bounded(smem_u32(&full[warp][slot]), phase));
            } else {
                cp_wait<kPvStages - 2>();
            }
            __syncwarp();
            if (!stuck) issue();      // into the slot consumed before this one
            const uint32_t vals = ring + slot * W::kStage;
#pragma unroll
            for (int t = 0; t < kPvTokens; ++t) {
                const float *p = ps + t * R + rl * RT;
                const uint32_t at = vals + t * 128 + ((dl ^ (t & 7)) << 4);
                if constexpr (kRowPairs) {
                    f32x2 w[RT / 2];
                    load_pairs<RT>(p, w);
#pragma unroll
                    for (int half = 0; half < DH; ++half) {
                        const float4 v = lds4(at + half * kPvTokens * 128);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const f32x2 vk = splat2(part_of(v, k));
#pragma unroll
                            for (int r = 0; r < RT / 2; ++r)
                                acc[r][4 * half + k] = fma2(w[r], vk, acc[r][4 * half + k]);
                        }
                    }
                } else {
                    f32x2 v[2 * DH];
#pragma unroll
                    for (int half = 0; half < DH; ++half) {
                        const float4 u = lds4(at + half * kPvTokens * 128);
                        v[2 * half] = pack2(u.x, u.y);
                        v[2 * half + 1] = pack2(u.z, u.w);
                    }
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const f32x2 w = splat2(p[r]);
#pragma unroll
                        for (int k = 0; k < 2 * DH; ++k) acc[r][k] = fma2(w, v[k], acc[r][k]);
                    }
                }
            }
            if (++slot == kPvStages) {
                slot = 0;
                phase ^= 1;
            }
        }
        // ---- the partials of the lane's rows and dimensions
        const int dim0 = now.run % A.dim_tiles * 32 * DH + 4 * dl;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            if (mine[r] < 0) continue;
            float *to = A.part + (mine[r] * A.ldpart + now.c) * d;
#pragma unroll
            for (int half = 0; half < DH; ++half) {
                float4 o;
                float other;
                if constexpr (kRowPairs) {
                    float o4[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        unpack2(acc[r / 2][4 * half + k], o4[k], other);
                        if (r & 1) o4[k] = other;
                    }
                    o = make_float4(o4[0], o4[1], o4[2], o4[3]);
                } else {
                    unpack2(acc[r][2 * half], o.x, o.y);
                    unpack2(acc[r][2 * half + 1], o.z, o.w);
                }
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
    }
    if (LOAD != kTma) cp_wait<0>();
    if (LOAD == kTma && stuck) {          // let the copies in flight land
        for (int i = 0; i < kPvStages; ++i) {
            (void)mbar_wait_bounded(smem_u32(&full[warp][slot]), phase);
            if (++slot == kPvStages) {
                slot = 0;
                phase ^= 1;
            }
        }
        if (lane == 0) atomicOr(&g_shared_watchdog, kWatchdogDecode);
    }
}

// ---------------------------------------------------------------- join
// A thread an element of the output; rows whose group shares nothing are done.
constexpr int kJoinDeep = 32;
__global__ void __launch_bounds__(kThreads) shared_join_kernel(const SharedArgs A) {
    const int b = blockIdx.y, i = blockIdx.x * kThreads + threadIdx.x;
    const int n = A.kv_lens[b];
    if (i >= A.heads * A.d || A.chunks[b / A.group] == 0 || !in_order(A, n)) return;
    const int h = i / A.d, chunks = (n + kKChunk - 1) / kKChunk;
    const float *p = A.part + (int64_t(b) * A.heads + h) * A.ldpart * A.d + (i - h * A.d);
    float t = 0.0f;
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

struct SharedPlan {
    bool together;            // false: decode.cu alone
    int rt, dh, row_blocks, dim_tiles;
    int64_t groups, kv, heads, ldx, ldpart;      // kv, heads: of a round
    size_t top, inv, x, part, own, bytes;        // offsets in the workspace
};

SharedPlan shared_plan(int64_t batch, int64_t group, int64_t heads, int64_t kv_heads,
                       int64_t head_dim, int64_t max_len) {
    SharedPlan p = {};
    group = std::min(group, batch);
    const int64_t per_kv = heads / kv_heads, rows = group * per_kv;
    p.together = group > 1 && max_len > 2 * kKChunk && rows <= 0x7fffffff / 2 &&
                 batch * heads <= 0x7fffffff / 2;
    if (!p.together) {
        p.bytes = decode_workspace_bytes(batch, heads, kv_heads, head_dim, max_len);
        return p;
    }
    p.groups = (batch + group - 1) / group;
    p.rt = rows <= 4 ? 1 : rows <= 8 ? 2 : rows <= 16 ? 4 : rows <= 32 || head_dim > 192 ? 8 : 16;
    p.dh = head_dim <= 32 ? 1 : 2;
    p.row_blocks = int((rows + 4 * p.rt - 1) / (4 * p.rt));
    p.dim_tiles = int((head_dim + 32 * p.dh - 1) / (32 * p.dh));
    p.ldx = (max_len - 1) / kKChunk * kKChunk;
    p.ldpart = (max_len + kKChunk - 1) / kKChunk;
    const size_t head = size_t(batch) * per_kv * (p.ldx + p.ldpart * head_dim) * 4;
    p.kv = std::max<int64_t>(1, std::min<int64_t>(kv_heads, int64_t(kSliceBytes / head)));
    p.heads = p.kv * per_kv;
    auto after = [](size_t at, size_t bytes) { return (at + bytes + 255) / 256 * 256; };
    p.top = after(0, size_t(p.groups) * 8);
    p.inv = after(p.top, size_t(batch) * p.heads * 4);
    p.x = after(p.inv, size_t(batch) * p.heads * 4);
    p.part = after(p.x, size_t(batch) * p.heads * p.ldx * 4);
    p.own = after(p.part, size_t(batch) * p.heads * p.ldpart * head_dim * 4);
    p.bytes = p.own + decode_workspace_bytes(batch, p.heads, p.kv, head_dim, max_len);
    return p;
}

template <class K, class... Args>
cudaError_t run(K kern, int64_t grid, size_t smem, cudaStream_t s, Args... args) {
    // the most any call takes: the limit is the kernel's, and another thread's call may
    // come between this line and the launch
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 112 * 1024);
    if (e != cudaSuccess) return e;
    kern<<<unsigned(grid), kThreads, smem, s>>>(args...);
    return cudaGetLastError();
}

template <int RT, Loader LOAD>
cudaError_t run_scores(const SharedArgs &A, const CUtensorMap &map, int64_t most, cudaStream_t s) {
    const int64_t grid = std::min<int64_t>(
        most * A.kv_heads * A.row_blocks, int64_t(sm_count_current_device()) * (RT >= 8 ? 2 : 3));
    const size_t smem = kScoreStages * kScoreStage + size_t(A.d) * 4 * RT * 4;
    return run(shared_scores_kernel<RT, LOAD>, grid, smem, s, A, map);
}
template <int RT, int DH, Loader LOAD>
cudaError_t run_partials(const SharedArgs &A, const CUtensorMap &map, int64_t most,
                         cudaStream_t s) {
    const int64_t items = most * A.kv_heads * A.row_blocks * A.dim_tiles;
    const int64_t grid =
        std::min<int64_t>((items + kWarps - 1) / kWarps,
                          int64_t(sm_count_current_device()) * (RT >= 8 ? 2 : 3));
    return run(shared_partials_kernel<RT, DH, LOAD>, grid, size_t(kWarps) * PvWarp<RT, DH>::kBytes,
               s, A, map);
}

template <Loader LOAD>
cudaError_t scores_for(int rt, const SharedArgs &A, const CUtensorMap &map, int64_t most,
                       cudaStream_t s) {
    switch (rt) {
        case 1: return run_scores<1, LOAD>(A, map, most, s);
        case 2: return run_scores<2, LOAD>(A, map, most, s);
        case 4: return run_scores<4, LOAD>(A, map, most, s);
        case 8: return run_scores<8, LOAD>(A, map, most, s);
        default: return run_scores<16, LOAD>(A, map, most, s);
    }
}
template <int DH, Loader LOAD>
cudaError_t partials_for(int rt, const SharedArgs &A, const CUtensorMap &map, int64_t most,
                         cudaStream_t s) {
    switch (rt) {
        case 1: return run_partials<1, DH, LOAD>(A, map, most, s);
        case 2: return run_partials<2, DH, LOAD>(A, map, most, s);
        case 4: return run_partials<4, DH, LOAD>(A, map, most, s);
        case 8: return run_partials<8, DH, LOAD>(A, map, most, s);
        default: return run_partials<16, DH, LOAD>(A, map, most, s);
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
    if (!p.together)
        return launch_decode_attention(batch, heads, q, ldq, c, table, max_pages, ldt, kv_lens,
                                       scale, out, ldo, workspace, dev_status, s);
    char *ws = reinterpret_cast<char *>(workspace);
    SharedArgs A = {};
    A.batch = int(batch);
    A.group = int(std::min(group, batch));
    A.groups = int(p.groups);
    A.per_kv = int(heads / c.kv_heads);
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
    A.max_pages = max_pages;
    A.ldt = ldt;
    A.kv_lens = kv_lens;
    A.max_len = max_len;
    A.scale = scale;
    A.row_blocks = p.row_blocks;
    A.dim_tiles = p.dim_tiles;
    A.chunks = reinterpret_cast<int *>(ws);
    A.lead = A.chunks + p.groups;
    A.top = reinterpret_cast<unsigned *>(ws + p.top);
    A.x = reinterpret_cast<float *>(ws + p.x);
    A.ldx = p.ldx;
    float *inv = reinterpret_cast<float *>(ws + p.inv);
    A.inv = inv;
    A.part = reinterpret_cast<float *>(ws + p.part);
    A.ldpart = p.ldpart;
    A.ldo = ldo;
    auto al16 = [](const void *x) { return reinterpret_cast<uintptr_t>(x) % 16 == 0; };
    const bool vec = al16(c.k) && al16(c.v) && c.page_stride % 4 == 0 &&
                     c.token_stride % 4 == 0 && c.head_stride % 4 == 0;
    const bool boxes = c.page_size == 8 || c.page_size == 16 || c.page_size == 32 ||
                       c.page_size % 64 == 0;
    const int64_t most = p.groups * (p.ldx / kKChunk);       // items of a run, at most
    for (int64_t g0 = 0; g0 < c.kv_heads; g0 += p.kv) {
        det_kv_cache part = c;
        part.kv_heads = std::min(p.kv, c.kv_heads - g0);
        part.k += g0 * c.head_stride;
        part.v += g0 * c.head_stride;
        A.kv_heads = int(part.kv_heads);
        A.heads = A.kv_heads * A.per_kv;
        A.k = part.k;
        A.v = part.v;
        A.q = q + g0 * A.per_kv * d;
        A.out = out + g0 * A.per_kv * d;
        Loader load = vec && d % 4 == 0 ? kCopy16 : kCopy4;
        CUtensorMap kmap = {}, vmap = {};
        const int kbox = int(std::min<int64_t>(c.page_size, 64));
        const int vbox = int(std::min<int64_t>(c.page_size, kPvTokens));
        if (vec && boxes) {
            const int64_t extent[4] = {d, part.kv_heads, c.page_size, c.num_pages};
            const int64_t stride[3] = {c.head_stride, c.token_stride, c.page_stride};
            if (make_tensor_map_4d(&kmap, part.k, extent, stride, {32, 1, uint32_t(kbox), 1}) &&
                make_tensor_map_4d(&vmap, part.v, extent, stride, {32, 1, uint32_t(vbox), 1}))
                load = kTma;
        }
        shared_plan_kernel<<<unsigned(p.groups), kPlanThreads, 0, s>>>(A);
        cudaError_t e = cudaGetLastError();
        A.box = kbox;
        if (e == cudaSuccess)
            e = load == kTma      ? scores_for<kTma>(p.rt, A, kmap, most, s)
                : load == kCopy16 ? scores_for<kCopy16>(p.rt, A, kmap, most, s)
                                  : scores_for<kCopy4>(p.rt, A, kmap, most, s);
        const SharedPrefix sh = {A.chunks, A.group, A.x, A.ldx, A.top, inv, A.part, A.ldpart};
        if (e == cudaSuccess)
            e = launch_decode_attention(batch, A.heads, A.q, ldq, part, table, max_pages, ldt,
                                        kv_lens, scale, A.out, ldo,
                                        reinterpret_cast<float *>(ws + p.own), dev_status, s, &sh);
        A.box = vbox;
        auto pv = [&](auto dh) {
            constexpr int DH = decltype(dh)::value;
            return load == kTma      ? partials_for<DH, kTma>(p.rt, A, vmap, most, s)
                   : load == kCopy16 ? partials_for<DH, kCopy16>(p.rt, A, vmap, most, s)
                                     : partials_for<DH, kCopy4>(p.rt, A, vmap, most, s);
        };
        if (e == cudaSuccess)
            e = p.dh == 1 ? pv(std::integral_constant<int, 1>())
                          : pv(std::integral_constant<int, 2>());
        if (e == cudaSuccess) {
            shared_join_kernel<<<dim3(unsigned((A.heads * d + kThreads - 1) / kThreads),
                                      unsigned(batch)),
                                 kThreads, 0, s>>>(A);
            e = cudaGetLastError();
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
