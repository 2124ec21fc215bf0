// fork.cu -- pages of a paged key-value cache that several requests share, for
// sm_103a: rows forked, reordered and freed, the pool compacted, pages copied.
//
// Fork and compaction are integers over the block tables: a step's are kilobytes,
// and what bounds them is latency; large ones read and write each entry once. Each
// is one cluster of up to 16 CTAs, whose shared memory has a bit a page and whose
// barriers part the phases; so one launch serves a small table, and no workspace or
// memory that somebody has to clear is needed. The bits are set by atomic or, so in
// any order. Where all pages' fit, each CTA marks bits of its own, and the cluster
// joins them slice by slice; past that (1.3 million pages) a CTA has a slice of
// them and the others mark it from afar, at about 5 cycles a mark and SM. An entry
// that is the one above it in the table (a shared prefix) is not marked again. What is
// written entry by entry, the new table and the compacted free list, goes to the
// whole GPU in launches of its own where it is large; a warp has kDeep loads in flight.
//
// Measured, us: a step of 16 x 4 rows forked 15 (on the GPU; latency of its phases), 8192
// rows of up to 375 pages 96 (of which the marks and their joining take most), a pool of
// half a million pages compacted 37, of 3000 pages 16.
//
// The copy streams pages through registers, 16 bytes a thread where the layout
// allows; HBM bounds it (each byte read and written once): 4096 pages of 131 KB in 175
// us, 6.1 TB/s, 90% of the measured copy rate. Four loads a thread: with eight, which
// spill, 195 us. A destination that the filters (a bit for each of up to 2^18 residues of
// page ids) do not clear costs a walk over all pairs, a team's each time: none for a
// step's copies, but the time of very many pairs in a larger pool goes by their square
// (111,000 moves of 16 KB in 517,000 pages 13.6 ms, 262,000 in a million 114 ms, for 0.54
// and 1.26 ms of bytes).
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "det_internal.cuh"

namespace cg = cooperative_groups;

namespace det {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBatch = 8192;
constexpr int kPerThread = kMaxBatch / kThreads;
constexpr int kMaxCluster = 16;
constexpr int kSegment = 256;                  // entries of a table row a warp takes at once
constexpr int kDeep = kSegment / 32;
constexpr int64_t kLarge = 1 << 16;            // entries from which the whole GPU writes them
constexpr int kSliceShift = 19;                // most pages of a slice from afar: 2^19
constexpr int64_t kMaxBits = 160 * 1024;       // bytes of the pages' bits
constexpr size_t kMaxSmem = kMaxBits + 2 * kMaxBatch * 4;
static_assert(kMaxSmem <= 226 * 1024 && (1 << kSliceShift) / 8 <= kMaxBits, "shared memory of a CTA");

// Exclusive prefix of v over the CTA's threads (all of them call); *total: the sum.
__device__ __forceinline__ int block_scan(int v, int *warp_sums, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int in = v;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, in, off);
        if (lane >= off) in += o;
    }
    if (lane == 31) warp_sums[warp] = in;
    __syncthreads();
    int w = warp_sums[lane];
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, w, off);
        if (lane >= off) w += o;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
    __syncthreads();      // warp_sums is used again
    return (warp ? before : 0) + in - v;
}

// The pages' bits, cut into slices of `words` words, a CTA's after the other's. Near:
// every CTA has all of them; else its own slice (of 2^shift pages).
struct Marks {
    cg::cluster_group &cluster;
    uint32_t *bits;
    int words, shift;
    bool near;
    __device__ __forceinline__ uint32_t *mine() const {
        return near ? bits + int(cluster.block_rank()) * words : bits;
    }
    template <bool SET>
    __device__ __forceinline__ void mark(int page) const {
        const uint32_t bit = 1u << (page & 31);
        if (near) {
            if (SET) atomicOr(bits + (page >> 5), bit);
            else atomicAnd(bits + (page >> 5), ~bit);
            return;
        }
        uint32_t w;
        asm("mapa.shared::cluster.u32 %0, %1, %2;"
            : "=r"(w)
            : "r"(smem_u32(bits + ((page & ((1 << shift) - 1)) >> 5))), "r"(page >> shift));
        if (SET)
            asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(w), "r"(bit)
                         : "memory");
        else
            asm volatile("red.relaxed.cluster.shared::cluster.and.b32 [%0], %1;" ::"r"(w), "r"(~bit)
                         : "memory");
    }
    // All threads, after a phase of marks: mine() is the whole of them then (SET: a bit
    // that any CTA has set; else one that none has cleared).
    template <bool SET>
    __device__ __forceinline__ void join() const {
        cluster.sync();
        const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
        if (!near || C == 1) return;
        uint4 *own = reinterpret_cast<uint4 *>(mine());
        for (int i = threadIdx.x; i < words / 4; i += kThreads) {
            uint4 v = own[i];
#pragma unroll 5
            for (int r = 1; r < C; ++r) {
                const uint4 o = *cluster.map_shared_rank(own + i, (rank + r) & (C - 1));
                if (SET) v.x |= o.x, v.y |= o.y, v.z |= o.z, v.w |= o.w;
                else v.x &= o.x, v.y &= o.y, v.z &= o.z, v.w &= o.w;
            }
            own[i] = v;
        }
        __syncthreads();
    }
    // All threads, after a join: everybody's bits are the whole ones.
    __device__ __forceinline__ void spread() const {
        const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
        if (!near || C == 1) return;
        cluster.sync();
        for (int i = threadIdx.x; i < words / 4; i += kThreads) {
#pragma unroll 5
            for (int k = 1; k < C; ++k) {
                const int r = (rank + k) & (C - 1);
                uint4 *at = reinterpret_cast<uint4 *>(bits + r * words) + i;
                *at = *cluster.map_shared_rank(at, r);
            }
        }
        cluster.sync();
    }
};

// The table's segments that a warp takes: w, w + all, ...
struct Segments {
    int row, seg, rows, segs, row_step, seg_step;
    __device__ __forceinline__ Segments(int rows_, int64_t max_pages, int w, int all) : rows(rows_) {
        segs = max(1, int((max_pages + kSegment - 1) / kSegment));
        row = w / segs;
        seg = w - row * segs;
        row_step = all / segs;
        seg_step = all - row_step * segs;
    }
    __device__ __forceinline__ bool more() const { return row < rows; }
    __device__ __forceinline__ void next() {
        row += row_step;
        seg += seg_step;
        if (seg >= segs) {
            seg -= segs;
            ++row;
        }
    }
    // the lane's first entry, and how many of the row's n are left from there
    __device__ __forceinline__ int64_t first() const {
        return int64_t(seg) * kSegment + (threadIdx.x & 31);
    }
    __device__ __forceinline__ int left(int64_t n) const {
        return int(max(int64_t(-1), min(n - first(), int64_t(kSegment))));
    }
};

// Every 32nd of n entries from p, and of `above` <= n entries from up; -2 past them.
__device__ __forceinline__ void load_entries(const int32_t *p, int n, const int32_t *up, int above,
                                             int (&id)[kDeep], int (&over)[kDeep]) {
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
        id[k] = 32 * k < n ? p[32 * k] : -2;
        over[k] = 32 * k < above ? up[32 * k] : -2;
    }
}

// The sum of the CTAs' values before this one's, and of all.
__device__ __forceinline__ void add_up(const int *slots, int C, int rank, int *before, int *total) {
    int b = 0, t = 0;
    for (int r = 0; r < C; ++r) {
        b += r < rank ? slots[r] : 0;
        t += slots[r];
    }
    *before = b;
    *total = t;
}
// The warp's set bits as ids, ascending, to `to` on: thread t of the CTA has `run` words
// from word t * run on, and `at` set bits before them. word(w): the bits of word w, whose
// first id is base + 32 w. A word is a warp's step, so stores are of consecutive ids:
// for words with many bits (half a million pages compacted 45 -> 37 us).
template <class Word>
__device__ __forceinline__ void list_bits(int32_t *to, int at, int base, int run, int words, Word word) {
    const int lane = threadIdx.x & 31, w0 = int(threadIdx.x) * run;
    for (int k = 0; k < run; ++k) {
        const uint32_t mine = w0 + k < words ? word(w0 + k) : 0u;
        for (unsigned some = __ballot_sync(0xffffffffu, mine != 0); some; some &= some - 1) {
            const int l = __ffs(int(some)) - 1;
            const uint32_t bits = __shfl_sync(0xffffffffu, mine, l);
            const int from = __shfl_sync(0xffffffffu, at, l);
            const int id = base + (__shfl_sync(0xffffffffu, w0, l) + k) * 32 + lane;
            if (bits >> lane & 1) to[from + __popc(bits & ((1u << lane) - 1))] = id;
        }
        at += __popc(mine);
    }
}

// Every CTA's value to every CTA, and add_up. The cluster meets once; `slots` is not
// reused before it meets again.
__device__ __forceinline__ void exchange(cg::cluster_group &cluster, int *slots, int value,
                                         int *before, int *total) {
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    if (int(threadIdx.x) < C) *cluster.map_shared_rank(slots + rank, threadIdx.x) = value;
    cluster.sync();
    add_up(slots, C, rank, before, total);
}

struct ForkArgs {
    int batch, batch_out;
    int64_t page_size, num_pages;
    const int32_t *lens, *parents, *table;
    int64_t max_pages, ldt;
    int32_t *table_out;
    int64_t ldto;
    int32_t *free_pages;
    int64_t capacity;
    const int32_t *free_count;
    int32_t *lens_out, *free_count_out, *src, *dst, *tokens, *dev_status;
    int words, shift;         // of the pages' bits
    bool near;
    bool apart;               // the new table is written by a launch of its own
};

// The new table: warp w of `all`. row(r, own): the new row's pages, and the page that it
// has in the place of the last one (-1: none).
template <class Row>
__device__ __forceinline__ void fork_rows(const ForkArgs &A, int w, int all, Row row) {
    for (Segments at(A.batch_out, A.max_pages, w, all); at.more(); at.next()) {
        const int r = at.row;
        int own;
        const int64_t pages = row(r, own);
        const int n = at.left(pages);
        if (n <= 0) continue;
        const int32_t *from = A.table + A.parents[r] * A.ldt + at.first();
        int32_t *to = A.table_out + r * A.ldto + at.first();
        const int last = own >= 0 ? int(min(pages - 1 - at.first(), int64_t(kSegment))) : -1;
        int id[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
            if (32 * k < n) id[k] = from[32 * k];
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
            if (32 * k < n) to[32 * k] = 32 * k == last ? own : id[k];
    }
}

__global__ void __launch_bounds__(kThreads) pages_fork_kernel(const ForkArgs A) {
    extern __shared__ __align__(16) uint32_t sm[];
    __shared__ int warp_sums[32], slots[kMaxCluster];
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int held = A.near ? C * A.words : A.words;
    const Marks marks = {cluster, sm, A.words, A.shift, A.near};
    int *first = reinterpret_cast<int *>(sm + held);         // each row's first child
    int *pages = first + A.batch;       // each row's pages; then, of each new row:
    int *fresh = pages;                 // a page of its own, -1: none, -2: refused
    const int64_t ps = A.page_size, room = min(A.max_pages * ps, int64_t(0x7fffffff));
    int status = 0;
    int64_t count = *A.free_count;
    if (count < 0 || count > A.capacity) {
        count = 0;
        status |= 1;
    }
    auto pages_of = [&](int len) {      // of a row that is in order
        return len < 0 || len > room ? int64_t(0) : (len + ps - 1) / ps;
    };
    for (int i = tid; i < held; i += kThreads) sm[i] = 0;
    for (int i = tid; i < A.batch; i += kThreads) {
        const int len = A.lens[i];
        if (len < 0 || len > room) status |= 1;
        first[i] = INT32_MAX;
        pages[i] = int(pages_of(len));
    }
    __syncthreads();
    // the thread's new rows
    const int per = (A.batch_out + kThreads - 1) / kThreads, r0 = tid * per;
    for (int r = tid; r < A.batch_out; r += kThreads) {
        const int p = A.parents[r];
        if (p >= 0 && p < A.batch) atomicMin(first + p, r);
        else if (p != -1) status |= 1;
    }
    __syncthreads();
    int orphan = 0;
    for (int i = tid; i < A.batch; i += kThreads) orphan |= first[i] == INT32_MAX && pages[i] > 0;
    orphan = __syncthreads_or(orphan);
    // of new rows r0.. the partly filled page that each shares with an earlier one, or -1;
    // where a thread has one row it is asked for here, and used in 3
    auto shared_pages = [&](auto rows, int *page) {
        constexpr int N = decltype(rows)::value;
        int len[N];
#pragma unroll
        for (int k = 0; k < N; ++k)
            page[k] = k < per && r0 + k < A.batch_out ? A.parents[r0 + k] : -1;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int p = page[k];
            const bool shares = p >= 0 && p < A.batch && first[p] != r0 + k;
            len[k] = shares ? A.lens[p] : 0;
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int64_t n = pages_of(len[k]);
            page[k] = n > 0 && len[k] % ps != 0 ? A.table[page[k] * A.ldt + n - 1] : -1;
        }
    };
    int early = -1;
    if (per == 1) shared_pages(std::integral_constant<int, 1>(), &early);
    if (!A.near) cluster.sync();        // every CTA's bits are clear
    // 1. the pages of rows that have no child, then without those of rows that have one;
    // an entry that is the one above it is that row's to mark, or kept by it
    auto look = [&](auto orphans) {
        constexpr bool SET = decltype(orphans)::value;
        for (Segments at(A.batch, A.max_pages, rank * kWarps + warp, C * kWarps); at.more(); at.next()) {
            const int b = at.row, n = at.left(pages[b]);
            if ((first[b] == INT32_MAX) != SET || n <= 0) continue;
            const bool over = orphan && b > 0 && (SET || first[b - 1] != INT32_MAX);
            const int32_t *p = A.table + b * A.ldt + at.first();
            int id[kDeep], up[kDeep];
            load_entries(p, n, p - A.ldt, over ? min(n, at.left(pages[b - 1])) : 0, id, up);
#pragma unroll
            for (int k = 0; k < kDeep; ++k) {
                if (32 * k >= n) break;
                if (unsigned(id[k]) >= unsigned(A.num_pages)) status |= 4;
                else if (orphan && up[k] != id[k]) marks.mark<SET>(id[k]);
            }
        }
    };
    look(std::true_type());
    if (orphan) {
        marks.join<true>();
        marks.spread();
    }
    look(std::false_type());
    // 2. the pages that nobody holds any more, ascending, to the end of the free list
    int freed = 0, before;
    if (orphan) {
        marks.join<false>();
        const uint32_t *drop = marks.mine();
        const int run = (A.words + kThreads - 1) / kThreads, w0 = tid * run;
        const int w1 = min(A.words, w0 + run);
        int mine = 0;
        for (int w = w0; w < w1; ++w) mine += __popc(drop[w]);
        int cta, total;
        int at = block_scan(mine, warp_sums, &cta);
        exchange(cluster, slots, cta, &before, &total);
        freed = total;
        if (count + freed > A.capacity) {
            freed = 0;
            status |= 1;
        } else {
            int64_t to = count + before + at;
            for (int w = w0; w < w1; ++w)
                for (uint32_t bits = drop[w]; bits; bits &= bits - 1)
                    A.free_pages[to++] = (rank * A.words + w) * 32 + __ffs(int(bits)) - 1;
        }
    }
    // 3. a page for every child that shares a partly filled one with an earlier child
    allow_dependents();
    int need = 0, last[kPerThread];     // that page, then the page of their own
    unsigned wants = 0;
    if (per == 1) {
#pragma unroll
        for (int k = 0; k < kPerThread; ++k) last[k] = k == 0 ? early : -1;
    } else {
        shared_pages(std::integral_constant<int, kPerThread>(), last);
    }
#pragma unroll
    for (int k = 0; k < kPerThread; ++k)
        if (last[k] >= 0 && last[k] < A.num_pages) {
            wants |= 1u << k;
            ++need;
        }
    int wanted;
    int nth = block_scan(need, warp_sums, &wanted);
    cluster.sync();                     // the free list is whole
    const int64_t have = count + freed;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        last[k] = -1;
        if (wants >> k & 1) {
            const int64_t at = have - 1 - nth++;
            if (at >= 0) {
                last[k] = __ldcg(A.free_pages + at);
            } else {
                status |= 2;
                wants &= ~(1u << k);
                last[k] = -2;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        if (k >= per || r0 + k >= A.batch_out) break;
        int page = last[k];
        if (wants >> k & 1 && (page < 0 || page >= A.num_pages)) {
            status |= 4;
            page = -2;
        }
        fresh[r0 + k] = page;
    }
    __syncthreads();
    for (int r = rank * kThreads + tid; r < A.batch_out; r += C * kThreads) {
        const int p = A.parents[r];
        const bool there = p >= 0 && p < A.batch && fresh[r] != -2;
        const int len = there ? A.lens[p] : 0;
        const int64_t n = there ? pages_of(len) : 0;
        const bool own = n > 0 && fresh[r] >= 0;
        A.lens_out[r] = n > 0 ? len : 0;
        A.src[r] = own ? A.table[p * A.ldt + n - 1] : -1;
        A.dst[r] = own ? fresh[r] : -1;
        A.tokens[r] = own ? int(len % ps) : 0;
    }
    // 4. the new table
    if (!A.apart)
        fork_rows(A, rank * kWarps + warp, C * kWarps, [&](int r, int &own) {
            const int p = A.parents[r];
            own = fresh[r];
            return p >= 0 && p < A.batch && own != -2 ? pages_of(A.lens[p]) : int64_t(0);
        });
    if (rank == 0 && tid == 0)
        *A.free_count_out = int(have - min(int64_t(wanted), have));
    if (A.dev_status) {
        status = __reduce_or_sync(0xffffffffu, unsigned(status));
        if (lane == 0 && status) atomicOr(reinterpret_cast<int *>(A.dev_status), status);
    }
}

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;

__global__ void __launch_bounds__(kRowThreads) pages_fork_rows_kernel(const ForkArgs A) {
    grid_dependency_wait();
    fork_rows(A, blockIdx.x * kRowWarps + (threadIdx.x >> 5), gridDim.x * kRowWarps,
              [&](int r, int &own) {
                  own = __ldcg(A.dst + r);
                  return (__ldcg(A.lens_out + r) + A.page_size - 1) / A.page_size;
              });
}

struct CompactArgs {
    int batch;
    int64_t page_size, num_pages;
    const int32_t *lens, *table;
    int64_t max_pages, ldt;
    int32_t *table_out;
    int64_t ldto;
    int32_t *free_pages, *free_count_out, *src, *dst, *moves, *dev_status;
    int words, shift;         // of the pages' bits
    bool near;
    bool apart;               // the rows and the free list by launches of their own
};

// The new rows: warp w of `all`. Until the free list is written its place holds the
// new ids of the pages past the first `used` ids: exactly as many entries.
__device__ __forceinline__ void compact_rows(const CompactArgs &A, int used, int w, int all) {
    const int64_t ps = A.page_size, room = min(A.max_pages * ps, int64_t(0x7fffffff));
    for (Segments at(A.batch, A.max_pages, w, all); at.more(); at.next()) {
        const int b = at.row, len = A.lens[b];
        const int n = at.left(len < 0 || len > room ? 0 : (len + ps - 1) / ps);
        if (n <= 0) continue;
        const int32_t *from = A.table + b * A.ldt + at.first();
        int32_t *to = A.table_out + b * A.ldto + at.first();
        int id[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) id[k] = 32 * k < n ? from[32 * k] : -1;
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
            if (id[k] >= used && id[k] < A.num_pages) id[k] = __ldcg(A.free_pages + (id[k] - used));
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
            if (32 * k < n) to[32 * k] = id[k];
    }
}
__device__ __forceinline__ void compact_free(const CompactArgs &A, int used, int64_t t, int64_t all) {
    for (int64_t i = t; i < A.num_pages - used; i += all)
        A.free_pages[i] = int(A.num_pages - 1 - i);
}

__global__ void __launch_bounds__(kRowThreads) pages_compact_rows_kernel(const CompactArgs A) {
    grid_dependency_wait();
    allow_dependents();
    compact_rows(A, int(A.num_pages - __ldcg(A.free_count_out)),
                 blockIdx.x * kRowWarps + (threadIdx.x >> 5), gridDim.x * kRowWarps);
}
__global__ void __launch_bounds__(kRowThreads) pages_compact_free_kernel(const CompactArgs A) {
    grid_dependency_wait();
    compact_free(A, int(A.num_pages - __ldcg(A.free_count_out)),
                 int64_t(blockIdx.x) * kRowThreads + threadIdx.x, int64_t(gridDim.x) * kRowThreads);
}

__global__ void __launch_bounds__(kThreads) pages_compact_kernel(const CompactArgs A) {
    extern __shared__ __align__(16) uint32_t sm[];
    __shared__ int warp_sums[32], slots[3][kMaxCluster];
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int words = A.words;
    const Marks marks = {cluster, sm, words, A.shift, A.near};
    const int64_t ps = A.page_size, room = min(A.max_pages * ps, int64_t(0x7fffffff));
    int status = 0;
    auto pages_of = [&](int len) {
        return len < 0 || len > room ? int64_t(0) : (len + ps - 1) / ps;
    };
    for (int i = tid; i < (A.near ? C * words : words); i += kThreads) sm[i] = 0;
    if (A.near) __syncthreads(); else cluster.sync();
    for (Segments at(A.batch, A.max_pages, rank * kWarps + warp, C * kWarps); at.more(); at.next()) {
        const int b = at.row, len = A.lens[b], over = b > 0 ? A.lens[b - 1] : 0;
        if (len < 0 || len > room) status |= 1;
        const int n = at.left(pages_of(len));
        if (n <= 0) continue;
        const int32_t *p = A.table + b * A.ldt + at.first();
        int id[kDeep], up[kDeep];
        load_entries(p, n, p - A.ldt, min(n, at.left(pages_of(over))), id, up);
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            if (32 * k >= n) break;
            if (unsigned(id[k]) >= unsigned(A.num_pages)) status |= 4;
            else if (up[k] != id[k]) marks.mark<true>(id[k]);
        }
    }
    marks.join<true>();
    const uint32_t *held = marks.mine();
    // the pages in use, then those of them past the first `used` ids and the holes before
    const int run = (words + kThreads - 1) / kThreads, w0 = tid * run, w1 = min(words, w0 + run);
    int mine = 0, cta, before, used;
    for (int w = w0; w < w1; ++w) mine += __popc(held[w]);
    block_scan(mine, warp_sums, &cta);
    exchange(cluster, slots[0], cta, &before, &used);
    const int base = rank * words * 32;
    auto moving = [&](int w) {          // of word w: in use at or past `used`
        const int at = base + w * 32;
        const uint32_t past = at >= used ? ~0u : at + 32 <= used ? 0u : ~0u << (used - at);
        return held[w] & past;
    };
    auto holes = [&](int w) {           // free before `used`
        const int at = base + w * 32;
        const uint32_t low = at >= used ? 0u : at + 32 <= used ? ~0u : ~(~0u << (used - at));
        return ~held[w] & low;
    };
    int nm = 0, nh = 0, cm, ch, bm, bh, total, same;
    for (int w = w0; w < w1; ++w) {
        nm += __popc(moving(w));
        nh += __popc(holes(w));
    }
    const int am = block_scan(nm, warp_sums, &cm), ah = block_scan(nh, warp_sums, &ch);
    if (tid < C) {
        *cluster.map_shared_rank(slots[1] + rank, tid) = cm;
        *cluster.map_shared_rank(slots[2] + rank, tid) = ch;
    }
    cluster.sync();
    add_up(slots[1], C, rank, &bm, &total);
    add_up(slots[2], C, rank, &bh, &same);
    list_bits(A.src + bm, am, base, run, words, moving);
    list_bits(A.dst + bh, ah, base, run, words, holes);
    cluster.sync();                     // the lists are whole
    allow_dependents();
    for (int i = rank * kThreads + tid; i < total; i += C * kThreads)
        A.free_pages[__ldcg(A.src + i) - used] = __ldcg(A.dst + i);
    const int64_t spare = A.num_pages - used;
    if (!A.apart) {
        cluster.sync();                 // the moved pages' new ids are there
        compact_rows(A, used, rank * kWarps + warp, C * kWarps);
        cluster.sync();                 // and have been used
        compact_free(A, used, rank * kThreads + tid, C * kThreads);
    }
    if (rank == 0 && tid == 0) {
        *A.free_count_out = int(spare);
        *A.moves = total;
    }
    if (A.dev_status) {
        status = __reduce_or_sync(0xffffffffu, unsigned(status));
        if (lane == 0 && status) atomicOr(reinterpret_cast<int *>(A.dev_status), status);
    }
}

// ---------------------------------------------------------------- copy
constexpr int kCopyThreads = 512;
constexpr int kMostFilter = 18;                     // filters of at most 2^18 bits
constexpr int kUnroll = 4;
constexpr int kCopyCtas = 2;                        // an SM's
constexpr double kStreamBytes = 128.0 * (1 << 20);

struct CopyArgs {
    float *k, *v;
    int64_t num_pages;
    int page_size, kv_heads, head_dim;
    int64_t page_stride, token_stride, head_stride;
    const int32_t *src, *dst, *tokens, *count;
    int pairs;
    int seg_tokens, segs;             // tokens of a piece; pieces of a page
    int filter;                       // bits of a filter, by the pages' low bits
    int32_t *dev_status;
};

// Whether x holds for any thread of the CTA's team'th team of N threads (all of them
// call).
template <int N>
__device__ __forceinline__ bool team_any(bool x, int team) {
    if (N == 32) return __any_sync(0xffffffffu, x);
    unsigned r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(unsigned(x)), "r"(team + 1), "r"(N)
        : "memory");
    return r != 0;
}

// WIDE: floats of a unit (4 or 1). Units of a piece: token, then head, then dim. A team of
// TEAM threads takes a piece, so that small pages go by many at a time (4096 of 512 bytes
// 26 -> 11 us). STREAM: more than L2 holds, so nothing is kept there (4096 pages of 131 KB
// 183 -> 175 us).
template <int WIDE, int TEAM, bool STREAM = false>
__global__ void __launch_bounds__(kCopyThreads, kCopyCtas) kv_copy_kernel(const CopyArgs A) {
    // pages that are a source; a destination; a destination at least twice
    extern __shared__ uint32_t is_src[];
    const int words = A.filter / 32;
    uint32_t *is_dst = is_src + words, *twice = is_dst + words;
    const int tid = threadIdx.x, lane = tid & 31;
    constexpr int teams = kCopyThreads / TEAM;
    const int team = tid / TEAM, at_team = tid % TEAM;
    int n = A.pairs, status = 0;
    if (A.count) {
        const int c = *A.count;
        if (c < 0 || c > n) status |= 1;
        n = min(max(c, 0), n);
    }
    const int64_t pieces = int64_t(n) * A.segs;
    if (int64_t(blockIdx.x) * teams >= pieces && blockIdx.x != 0) return;
    for (int i = tid; i < 3 * words; i += kCopyThreads) is_src[i] = 0;
    __syncthreads();
    // a pair that copies: both pages there, and as many tokens as a page holds
    auto valid = [&](int i, int &s, int &d, int &t) {
        s = A.src[i];
        d = A.dst[i];
        t = A.tokens ? A.tokens[i] : A.page_size;
        if (s < 0 || d < 0) return false;
        if (s >= A.num_pages || d >= A.num_pages || t < 0 || t > A.page_size) {
            status |= 1;
            return false;
        }
        return s != d && t > 0;
    };
#pragma unroll 4
    for (int i = tid; i < n; i += kCopyThreads) {
        int s, d, t;
        if (!valid(i, s, d, t)) continue;
        const unsigned a = unsigned(s) & unsigned(A.filter - 1);
        const unsigned b = unsigned(d) & unsigned(A.filter - 1);
        atomicOr(is_src + (a >> 5), 1u << (a & 31));
        if (atomicOr(is_dst + (b >> 5), 1u << (b & 31)) >> (b & 31) & 1)
            atomicOr(twice + (b >> 5), 1u << (b & 31));
    }
    __syncthreads();
    const int units = A.head_dim / WIDE, row = A.kv_heads * units;
    for (int64_t w = int64_t(blockIdx.x) * teams + team; w < pieces; w += int64_t(gridDim.x) * teams) {
        const int i = int(w / A.segs), seg = int(w - int64_t(i) * A.segs);
        int s, d, t;
        if (!valid(i, s, d, t)) continue;           // the same for the whole team
        const unsigned b = unsigned(d) & unsigned(A.filter - 1);
        const uint32_t bit = 1u << (b & 31);
        if ((is_src[b >> 5] | twice[b >> 5]) & bit) {
            // maybe: look through the pairs
            bool later = false, read = false;
            for (int j = at_team; j < n; j += TEAM) {
                int s2, d2, t2;
                if (!valid(j, s2, d2, t2)) continue;
                read |= s2 == d;
                later |= d2 == d && j > i;
            }
            read = team_any<TEAM>(read, team);
            later = team_any<TEAM>(later, team);
            if (read) status |= 2;
            if (read || later) continue;
        }
        const int t0 = seg * A.seg_tokens, t1 = min(t, t0 + A.seg_tokens);
        const int64_t from = s * A.page_stride, to = d * A.page_stride;
        const int total = max(0, t1 - t0) * row;
        for (int half = 0; half < 2; ++half) {
            float *base = half ? A.v : A.k;
            for (int u0 = at_team; u0 < total; u0 += TEAM * kUnroll) {
                float4 v4[kUnroll];
                int64_t at[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int x = u0 + u * TEAM;
                    if (x >= total) break;
                    const int tok = x / row, rest = x - tok * row, g = rest / units;
                    at[u] = (t0 + tok) * A.token_stride + g * A.head_stride +
                            int64_t(rest - g * units) * WIDE;
                    const float *p = base + from + at[u];
                    if (WIDE == 1) v4[u].x = *p;
                    else if (STREAM) v4[u] = __ldcs(reinterpret_cast<const float4 *>(p));
                    else v4[u] = *reinterpret_cast<const float4 *>(p);
                }
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    if (u0 + u * TEAM >= total) break;
                    float *p = base + to + at[u];
                    if (WIDE == 1) *p = v4[u].x;
                    else if (STREAM) __stcs(reinterpret_cast<float4 *>(p), v4[u]);
                    else *reinterpret_cast<float4 *>(p) = v4[u];
                }
            }
        }
    }
    if (A.dev_status) {
        __syncwarp();
        status = __reduce_or_sync(0xffffffffu, unsigned(status));
        if (lane == 0 && status) atomicOr(reinterpret_cast<int *>(A.dev_status), status);
    }
}

// CTAs of the cluster, so many that a warp has few table segments, and the words of a
// slice of the pages' bits (a multiple of 4).
struct ClusterPlan {
    int ctas, words, shift;
    bool near;
    size_t bytes;             // of the bits, of a CTA
};
ClusterPlan cluster_plan(int64_t rows, int64_t max_pages, int64_t num_pages) {
    ClusterPlan p = {1, 0, 0, true, 0};
    const int64_t work = rows * ((max_pages + kSegment - 1) / kSegment) + num_pages / 4096;
    while (p.ctas < kMaxCluster && p.ctas * kWarps < work) p.ctas *= 2;
    int64_t slice = (num_pages + p.ctas * 128 - 1) / (p.ctas * 128) * 128;
    p.near = slice * p.ctas / 8 <= kMaxBits;
    if (!p.near) {
        while ((int64_t(p.ctas) << kSliceShift) < num_pages) p.ctas *= 2;
        p.shift = 7;
        while ((int64_t(p.ctas) << p.shift) < num_pages) ++p.shift;
        slice = int64_t(1) << p.shift;
    }
    p.words = int(slice / 32);
    p.bytes = size_t(slice) / 8 * (p.near ? p.ctas : 1);
    return p;
}

template <class K, class Args>
cudaError_t run_cluster(K kern, const Args &A, int ctas, size_t smem, cudaStream_t s) {
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMaxSmem));
    if (e == cudaSuccess && ctas > 8)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, A);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

// A warp a segment of a row, at most 8 CTAs an SM.
dim3 rows_grid(int64_t rows, int64_t max_pages) {
    const int64_t warps = rows * ((max_pages + kSegment - 1) / kSegment);
    return dim3(unsigned(std::max<int64_t>(
        1, std::min<int64_t>((warps + kRowWarps - 1) / kRowWarps,
                             int64_t(sm_count_current_device()) * 8))));
}

}  // namespace

cudaError_t launch_pages_fork(int64_t batch, int64_t batch_out, int64_t page_size,
                              int64_t num_pages, const int32_t *lens, const int32_t *parents,
                              const int32_t *table, int64_t max_pages, int64_t ldt,
                              int32_t *table_out, int64_t ldto, int32_t *free_pages,
                              int64_t capacity, const int32_t *free_count, int32_t *lens_out,
                              int32_t *free_count_out, int32_t *src, int32_t *dst,
                              int32_t *tokens, int32_t *dev_status, cudaStream_t s) {
    const ClusterPlan p = cluster_plan(std::max(batch, batch_out), max_pages, num_pages);
    const ForkArgs A = {int(batch), int(batch_out), page_size, num_pages, lens, parents, table,
                        max_pages, ldt, table_out, ldto, free_pages, capacity, free_count, lens_out,
                        free_count_out, src, dst, tokens, dev_status, p.words, p.shift, p.near,
                        batch_out * max_pages >= kLarge};
    const size_t smem = p.bytes + size_t(batch + std::max(batch, batch_out)) * 4;
    const cudaError_t e = run_cluster(pages_fork_kernel, A, p.ctas, smem, s);
    if (e != cudaSuccess || !A.apart) return e;
    return launch_dependent(pages_fork_rows_kernel, rows_grid(batch_out, max_pages),
                            dim3(kRowThreads), 0, s, A);
}

cudaError_t launch_pages_compact(int64_t batch, int64_t page_size, int64_t num_pages,
                                 const int32_t *lens, const int32_t *table, int64_t max_pages,
                                 int64_t ldt, int32_t *table_out, int64_t ldto,
                                 int32_t *free_pages, int32_t *free_count_out, int32_t *src,
                                 int32_t *dst, int32_t *moves, int32_t *dev_status,
                                 cudaStream_t s) {
    const ClusterPlan p = cluster_plan(batch, max_pages, num_pages);
    const CompactArgs A = {int(batch), page_size, num_pages, lens, table, max_pages, ldt, table_out,
                           ldto, free_pages, free_count_out, src, dst, moves, dev_status, p.words,
                           p.shift, p.near, batch * max_pages + num_pages >= kLarge};
    cudaError_t e = run_cluster(pages_compact_kernel, A, p.ctas, p.bytes, s);
    if (e != cudaSuccess || !A.apart) return e;
    e = launch_dependent(pages_compact_rows_kernel, rows_grid(batch, max_pages), dim3(kRowThreads), 0,
                         s, A);
    if (e != cudaSuccess) return e;
    const int64_t grid = std::min<int64_t>((num_pages + kRowThreads - 1) / kRowThreads,
                                           int64_t(sm_count_current_device()) * 8);
    return launch_dependent(pages_compact_free_kernel, dim3(unsigned(std::max<int64_t>(1, grid))),
                            dim3(kRowThreads), 0, s, A);
}

cudaError_t launch_kv_copy(int64_t pairs, const int32_t *src, const int32_t *dst,
                           const int32_t *tokens, const int32_t *count, const det_kv_cache &c,
                           int32_t *dev_status, cudaStream_t s) {
    auto al16 = [](const void *x) { return reinterpret_cast<uintptr_t>(x) % 16 == 0; };
    const bool vec = al16(c.k) && al16(c.v) && c.page_stride % 4 == 0 && c.token_stride % 4 == 0 &&
                     c.head_stride % 4 == 0 && c.head_dim % 4 == 0;
    CopyArgs A = {c.k, c.v, c.num_pages, int(c.page_size), int(c.kv_heads), int(c.head_dim),
                  c.page_stride, c.token_stride, c.head_stride, src, dst, tokens, count, int(pairs),
                  0, 0, 0, dev_status};
    // a piece: tokens whose units all have one round of a CTA's loads, fewer where the
    // pieces would be too few for the GPU, or one; a thread takes up to eight units of it
    const int64_t units = c.kv_heads * c.head_dim / (vec ? 4 : 1);
    const int64_t ctas = int64_t(sm_count_current_device()) * kCopyCtas;
    const int64_t fit = std::min(kCopyThreads * kUnroll / units, pairs * c.page_size / ctas);
    A.seg_tokens = int(std::max<int64_t>(1, std::min(fit, c.page_size)));
    A.segs = int((c.page_size + A.seg_tokens - 1) / A.seg_tokens);
    const int64_t wants = A.seg_tokens * units / 8;
    const int team = wants <= 32 ? 32 : wants <= 128 ? 128 : kCopyThreads;
    const int64_t teams = kCopyThreads / team;
    const int64_t grid = std::min<int64_t>((pairs * A.segs + teams - 1) / teams, ctas);
    A.filter = 1024;
    while (A.filter < (1 << kMostFilter) && A.filter < c.num_pages) A.filter *= 2;
    const size_t smem = size_t(A.filter) / 8 * 3;
    auto run = [&](auto kern) {
        if (smem > 48 * 1024) {           // the most any call takes
            const cudaError_t e = cudaFuncSetAttribute(
                kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (1 << kMostFilter) / 8 * 3);
            if (e != cudaSuccess) return e;
        }
        kern<<<unsigned(grid), kCopyThreads, smem, s>>>(A);
        return cudaGetLastError();
    };
    const bool stream =
        16.0 * double(pairs) * double(c.page_size) * double(c.kv_heads * c.head_dim) > kStreamBytes;
    if (vec)
        return team == 32    ? run(kv_copy_kernel<4, 32>)
               : team == 128 ? run(kv_copy_kernel<4, 128>)
               : stream      ? run(kv_copy_kernel<4, kCopyThreads, true>)
                             : run(kv_copy_kernel<4, kCopyThreads>);
    return team == 32    ? run(kv_copy_kernel<1, 32>)
           : team == 128 ? run(kv_copy_kernel<1, 128>)
                         : run(kv_copy_kernel<1, kCopyThreads>);
}

}  // namespace det
