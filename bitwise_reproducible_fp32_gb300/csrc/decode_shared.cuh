// decode_shared.cuh -- what the kernels of decode attention for requests that share a
// prefix have in common (decode_shared.cu: the plan, and units of many rows;
// decode_few.cu: requests' own tokens with up to 8 rows; decode_group.cu: groups of up to
// 8 rows).
#pragma once

#include "decode.cuh"

namespace det {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kWatchdogDecode = 32u;          // det_watchdog_status bit 5
constexpr size_t kMaxSmem = 112 * 1024;            // of a CTA

struct SharedArgs {
    int batch, group, groups, heads, kv_heads, per_kv, d;
    int64_t rows;             // of a whole group and a key-value head: group * per_kv
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
    int64_t max_len;
    float scale;
    int wide;                 // 16-byte loads of the cache where TMA cannot be used
    int box;                  // tokens of a TMA box
    int row_blocks, dim_tiles;
    int *chunks, *lead;       // of each group: shared chunks, a request in order
    int *own;                 // of each request: its own chunks, 0 if it is not in order
    unsigned *top;            // of each row (b, h): the maximum of its scores, by max_key
    float *inv;               // 1 / S
    float *x;                 // ((group * kv_heads + head) * octets + octet) * rows + row) * 8
    int64_t octets;
    float *part;              // (row * ldpart + chunk) * d
    int64_t ldpart;
    float *out;
    int64_t ldo;
    int32_t *dev_status;
};

namespace {

__device__ __forceinline__ unsigned page_of(const SharedArgs &A, int t) {
    return A.page_shift >= 0 ? unsigned(t) >> A.page_shift : unsigned(t) / A.page_size;
}

// ---------------------------------------------------------------- work
// The items of a kernel: for each unit (a group with the shared chunks, or a request
// with its own chunks, or with tiles of kTile tokens of them) `mul` runs (of heads and
// blocks of rows or dimensions) of its chunks or tiles, these fastest.
enum Cut { kShared, kOwn, kOwnTiles };
template <int CUT>
constexpr bool kIsOwn = CUT != kShared;
template <int CUT>
constexpr bool kInTiles = CUT == kOwnTiles;
constexpr int kTile = 64;
struct Item {
    int u, run, c;
    int n, base, end;         // the unit's chunks or tiles, its first token and its end
};
template <int CUT>
__device__ __forceinline__ int units(const SharedArgs &A) { return kIsOwn<CUT> ? A.batch : A.groups; }
template <int CUT>
__device__ __forceinline__ int chunks_of(const SharedArgs &A, int u) {
    const int n = kIsOwn<CUT> ? A.own[u] : A.chunks[u];
    if (!kInTiles<CUT> || n == 0) return n;
    return (A.kv_lens[u] - A.chunks[u / A.group] * kKChunk + kTile - 1) / kTile;
}
template <int CUT>
__device__ __forceinline__ void enter(const SharedArgs &A, Item &it) {      // its unit
    it.n = chunks_of<CUT>(A, it.u);
    it.base = kIsOwn<CUT> ? A.chunks[it.u / A.group] * kKChunk : 0;
    it.end = kIsOwn<CUT> ? A.kv_lens[it.u] : A.chunks[it.u] * kKChunk;
}
// The item's first token, how many it has, and the table row of its pages.
template <int CUT>
__device__ __forceinline__ int first_token(const Item &it) {
    return it.base + it.c * (kInTiles<CUT> ? kTile : kKChunk);
}
template <int CUT>
__device__ __forceinline__ int tokens_from(const Item &it, int t0) {
    return min(kInTiles<CUT> ? kTile : kKChunk, it.end - t0);
}
template <int CUT>
__device__ __forceinline__ const int32_t *pages_of(const SharedArgs &A, const Item &it) {
    return A.table + (kIsOwn<CUT> ? it.u : A.lead[it.u]) * A.ldt;
}
// Row r of the unit's rows of a key-value head: its place among its group's; the row
// (b, h) of a place, -1 where there is none or its request is not in order.
template <int CUT>
__device__ __forceinline__ int place_of(const SharedArgs &A, int u, int r) {
    return kIsOwn<CUT> ? u % A.group * A.per_kv + r : r;
}
template <int CUT>
__device__ __forceinline__ int group_of(const SharedArgs &A, int u) {
    return kIsOwn<CUT> ? u / A.group : u;
}
template <int CUT>
__device__ __forceinline__ int rows_of(const SharedArgs &A) {
    return kIsOwn<CUT> ? A.per_kv : int(A.rows);
}
__device__ __forceinline__ int row_at(const SharedArgs &A, int g, int kv, int place) {
    const int m = place / A.per_kv, b = g * A.group + m;
    if (m >= A.group || b >= A.batch || A.own[b] == 0) return -1;
    return b * A.heads + kv * A.per_kv + (place - m * A.per_kv);
}

// A worker's share [lo, hi) of the items is a run of them, all as long but for one;
// the longer ones go to the first workers. All threads of the CTA call; the CTA has
// the workers first, first + step, ... of `all`.
struct Share {
    int64_t items;
    Item at;
};
template <int CUT, int WORKERS>
__device__ __forceinline__ void shares(const SharedArgs &A, int mul, int first, int step, int all,
                                       Share *out) {
    __shared__ int64_t warp_sums[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = units<CUT>(A);
    const int per = (n + kThreads - 1) / kThreads;
    const int u0 = min(n, tid * per), u1 = min(n, u0 + per);
    int64_t sum = 0;
    for (int u = u0; u < u1; ++u) sum += chunks_of<CUT>(A, u);
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
    const int64_t base = total / all, rem = total % all;
    for (int w = 0; w < WORKERS; ++w) {
        const int64_t i = first + int64_t(w) * step, lo = i * base + min(i, rem);
        if (tid == 0) out[w].items = base + (i < rem);
        if (base + (i < rem) > 0 && before * mul <= lo && lo < (before + sum) * mul) {
            int64_t at = before;
            int u = u0;
            while ((at + chunks_of<CUT>(A, u)) * mul <= lo) at += chunks_of<CUT>(A, u++);
            const int c = chunks_of<CUT>(A, u);
            const int64_t k = lo - at * mul;
            out[w].at = {u, int(k / c), int(k % c)};
            enter<CUT>(A, out[w].at);
        }
    }
    __syncthreads();
}
template <int CUT>
__device__ __forceinline__ void advance(const SharedArgs &A, int mul, Item &it) {
    if (++it.c < it.n) return;
    it.c = 0;
    if (++it.run < mul) return;
    it.run = 0;
    do {
        ++it.u;
    } while (it.u < units<CUT>(A) && chunks_of<CUT>(A, it.u) == 0);
    if (it.u < units<CUT>(A)) enter<CUT>(A, it);
}

// Scores (and partials) of the shared chunks and of the own ones do not depend on each
// other. So the kernel of the own ones (OWN), launched behind the other one, starts as
// soon as that one's CTAs have all begun (which they do once everything before them is
// complete, so the plan's lists, the exps and 1 / S may be read before the wait) and
// there is room, and waits for it at its end, so that its own end is both's.
template <bool OWN>
struct Beside {
    __device__ __forceinline__ Beside() {
        if (!OWN) grid_dependency_wait();
        allow_dependents();
    }
    __device__ __forceinline__ ~Beside() {
        if (OWN) grid_dependency_wait();
    }
};

// A token's offset in the cache (its page is in order: the plan has seen it).
__device__ __forceinline__ int64_t offset_of(const SharedArgs &A, const int32_t *pages, int t) {
    const unsigned p = page_of(A, t);
    return pages[p] * A.page_stride + int64_t(unsigned(t) - p * A.page_size) * A.token_stride;
}

// ---------------------------------------------------------------- pieces
// kTile tokens x 32 dimensions in shared memory: rows of 128 bytes, their 16-byte units
// swapped by row mod 8.
constexpr int kPieceBytes = kTile * 128;
constexpr int kRingPieces = 2;            // three leave room for two CTAs an SM, not three
constexpr int kRingBytes = kRingPieces * kPieceBytes;

// A warp's ring of pieces.
template <Loader LOAD>
struct Ring {
    const SharedArgs &A;
    const CUtensorMap *map;              // of the keys or values that are fetched
    const float *cache;
    uint32_t slots, bars;
    int slot_in = 0, slot = 0;
    uint32_t phase = 0;
    bool stuck = false;
    int id = 0;                           // of the lane's box
    int64_t off[2];                       // of tokens lane, lane + 32

    __device__ __forceinline__ Ring(const SharedArgs &a, const CUtensorMap *m, const float *c,
                                    uint32_t s, uint32_t b)
        : A(a), map(m), cache(c), slots(s), bars(b) {}
    // where the piece of `live` tokens from t on is; ahead of fetch. CHECK: whether one
    // of the lane's pages is out of range (page 0 stands for it).
    template <bool CHECK = false>
    __device__ __forceinline__ bool look_up(const int32_t *pages, int t, int live) {
        const int lane = threadIdx.x & 31;
        bool bad = false;
        auto page = [&](unsigned p) {
            const int at = pages[p];
            if (!CHECK || unsigned(at) < unsigned(A.num_pages)) return at;
            bad = true;
            return 0;
        };
        if constexpr (LOAD == kTma) {
            if (lane * A.box < live) id = page(page_of(A, t + lane * A.box));
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int at = t + lane + 32 * k;
                if (lane + 32 * k >= live) continue;
                const unsigned p = page_of(A, at);
                off[k] = page(p) * A.page_stride + int64_t(unsigned(at) - p * A.page_size) * A.token_stride;
            }
        }
        return bad;
    }
    __device__ __forceinline__ void fetch(int kv, int sl, int t, int live) {
        const int lane = threadIdx.x & 31;
        const uint32_t dst = slots + slot_in * kPieceBytes;
        if constexpr (LOAD == kTma) {
            const uint32_t bar = bars + 8 * slot_in;
            const int boxes = (live + A.box - 1) / A.box;
            if (lane == 0) mbar_arrive_expect_tx(bar, boxes * A.box * 128);
            __syncwarp();
            if (lane < boxes) {
                const int at = t + lane * A.box;
                tma_load_4d(dst + lane * A.box * 128, map, 32 * sl, kv,
                            int(unsigned(at) - page_of(A, at) * A.page_size), id, bar);
            }
        } else if constexpr (LOAD == kCopy16) {
            const int col = lane & 7, r0 = lane >> 3;
            const bool in = 4 * col < A.d - 32 * sl;
            const float *src = cache + kv * A.head_stride + 32 * sl + 4 * col;
#pragma unroll
            for (int i = 0; i < kTile / 4; ++i) {
                const int r = 4 * i + r0;
                const int64_t at = __shfl_sync(0xffffffffu, off[i >> 3], r & 31);
                if (in && r < live) cp_async<16>(dst + r * 128 + ((col ^ (r & 7)) << 4), src + at);
            }
        } else {
            const bool in = lane < A.d - 32 * sl;
            const float *src = cache + kv * A.head_stride + 32 * sl + lane;
#pragma unroll 8
            for (int r = 0; r < kTile; ++r) {
                const int64_t at = __shfl_sync(0xffffffffu, r < 32 ? off[0] : off[1], r & 31);
                if (in && r < live)
                    cp_async<4>(dst + r * 128 + ((((lane >> 2) ^ (r & 7)) << 4) | (lane & 3) << 2),
                                src + at);
            }
        }
        slot_in = slot_in + 1 == kRingPieces ? 0 : slot_in + 1;
    }
    __device__ __forceinline__ void wait() {
        if constexpr (LOAD == kTma) {
            if (!stuck)
                stuck = __any_sync(0xffffffffu, !wait_for_piece(bars, slot, phase, kRingPieces));
        } else {
            cp_wait<kRingPieces - 2>();
        }
        __syncwarp();
    }
    __device__ __forceinline__ void step() {
        if (++slot == kRingPieces) {
            slot = 0;
            phase ^= 1;
        }
    }
    // the piece that was waited for; once a wait has given up, that one for good
    __device__ __forceinline__ uint32_t piece() {
        const uint32_t p = slots + slot * kPieceBytes;
        if (!stuck) step();
        return p;
    }
    // at the end: the copies in flight land, which are those from the one that a wait
    // gave up on to the last one asked for
    __device__ __forceinline__ void drain(unsigned *watchdog) {
        if constexpr (LOAD != kTma) {
            cp_wait<0>();
        } else if (stuck) {
            for (; slot != slot_in; step()) (void)mbar_wait_bounded(bars + 8 * slot, phase);
            if ((threadIdx.x & 31) == 0) atomicOr(watchdog, kWatchdogDecode);
        }
    }
};

template <Loader LOAD>
__device__ __forceinline__ void init_bars(uint64_t *bars) {
    if (LOAD == kTma && threadIdx.x == 0) {
        for (int i = 0; i < kWarps * kRingPieces; ++i) mbar_init(smem_u32(bars + i), 1);
        fence_mbar_init();
    }
}

}  // namespace

constexpr int kFewRows = 8;

// The requests' own tokens, at most kFewRows rows a key-value head: scores and their
// maxima; partials of the chunks. map: keys or values with boxes of A.box tokens
// (nullptr: TMA cannot be used); most: the chunks of all requests, at most.
cudaError_t launch_few_scores(const SharedArgs &A, const CUtensorMap *map, int64_t most,
                              cudaStream_t s);
cudaError_t launch_few_partials(const SharedArgs &A, const CUtensorMap *map, int64_t most,
                                cudaStream_t s);

// Groups of at most kFewRows rows a key-value head, in one launch. maps: keys and values
// with boxes of A.box tokens.
struct GroupPlan {
    int cluster;
    int64_t units, chunks;        // chunks: of a request, at most
    size_t part, bytes;           // the partials' place in the workspace, and its size
};
GroupPlan group_plan(int64_t groups, int64_t rows, int64_t kv_heads, int64_t head_dim,
                     int64_t max_len);
cudaError_t launch_group_decode(const SharedArgs &A, const GroupPlan &p, const CUtensorMap *maps,
                                cudaStream_t s);

}  // namespace det
