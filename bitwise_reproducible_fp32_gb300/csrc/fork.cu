// fork.cu -- pages of a paged key-value cache that several requests share, for
// sm_103a: rows forked, reordered and freed, the pool compacted, pages copied.
//
// Fork and compaction are integers over the block tables: a step's are kilobytes,
// and what bounds them is latency; large ones read and write each entry once. Each
// is one cluster of up to 16 CTAs: the pages' marks are bitmaps cut over the
// CTAs' shared memory (distributed, by atomic or, so in any order), which the
// cluster's barriers part into phases. So one launch serves and no workspace or
// memory that somebody has to clear is needed. An entry that is the one above it
// in the table (a shared prefix) is not marked again.
//
// The copy streams pages through registers, 16 bytes a thread where the layout
// allows; HBM bounds it (each byte read and written once).
#include <cooperative_groups.h>

#include <algorithm>

#include "det_internal.cuh"

namespace cg = cooperative_groups;

namespace det {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBatch = 8192;
constexpr int kPerThread = kMaxBatch / kThreads;
constexpr int kMaxCluster = 16;
constexpr int kSegment = 1024;                 // entries of a table row a warp takes at once
constexpr int kSliceShift = 19;                // most pages of a CTA's marks: 2^19
constexpr size_t kMaxSmem = (size_t(1) << kSliceShift) / 8 * 2 + 2 * kMaxBatch * 4;
static_assert(kMaxSmem <= 220 * 1024, "shared memory of a CTA");

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

// The pages' marks: page p's bit is word (p & mask) / 32 of CTA p >> shift.
struct Marks {
    cg::cluster_group &cluster;
    int shift;
    __device__ __forceinline__ void set(uint32_t *own, int page) const {
        uint32_t *w = cluster.map_shared_rank(own, page >> shift);
        const int at = page & ((1 << shift) - 1);
        atomicOr(w + (at >> 5), 1u << (at & 31));
    }
};

// Every CTA's value to every CTA: the sum before this one's, and of all. The
// cluster meets once; `slots` is not reused before it meets again.
__device__ __forceinline__ void exchange(cg::cluster_group &cluster, int *slots, int value,
                                         int *before, int *total) {
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    if (int(threadIdx.x) < C) *cluster.map_shared_rank(slots + rank, threadIdx.x) = value;
    cluster.sync();
    int b = 0, t = 0;
    for (int r = 0; r < C; ++r) {
        b += r < rank ? slots[r] : 0;
        t += slots[r];
    }
    *before = b;
    *total = t;
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
    int shift;
};

__global__ void __launch_bounds__(kThreads) pages_fork_kernel(const ForkArgs A) {
    extern __shared__ uint32_t sm[];
    const int words = 1 << (A.shift - 5);
    uint32_t *keep = sm, *drop = sm + words;      // pages of rows with and without a child
    int *first = reinterpret_cast<int *>(drop + words);      // each row's first child
    int *fresh = first + kMaxBatch;     // each new row: a page of its own, -1: none, -2: refused
    __shared__ int warp_sums[32], slots[kMaxCluster];
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Marks marks = {cluster, A.shift};
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
    for (int i = tid; i < 2 * words; i += kThreads) sm[i] = 0;
    for (int i = tid; i < A.batch; i += kThreads) first[i] = INT32_MAX;
    __syncthreads();
    for (int r = tid; r < A.batch_out; r += kThreads) {
        const int p = A.parents[r];
        if (p >= 0 && p < A.batch) atomicMin(first + p, r);
        else if (p != -1) status |= 1;
    }
    __syncthreads();
    int orphan = 0;
    for (int i = tid; i < A.batch; i += kThreads) {
        const int len = A.lens[i];
        if (len < 0 || len > room) status |= 1;
        orphan |= first[i] == INT32_MAX && pages_of(len) > 0;
    }
    orphan = __syncthreads_or(orphan);
    cluster.sync();                     // every CTA's marks are clear
    // 1. the pages of rows that have no child and those of rows that have one
    const int64_t segs = (A.max_pages + kSegment - 1) / kSegment;
    for (int64_t i = int64_t(rank) * kWarps + warp; i < A.batch * segs; i += C * kWarps) {
        const int b = int(i / segs);
        const int64_t n = pages_of(A.lens[b]), j0 = (i - b * segs) * kSegment;
        if (j0 >= n) continue;
        const bool has = first[b] != INT32_MAX;
        const int64_t above =
            b > 0 && (first[b - 1] != INT32_MAX) == has ? pages_of(A.lens[b - 1]) : 0;
        const int32_t *row = A.table + b * A.ldt;
        for (int64_t j = j0 + lane; j < min(n, j0 + kSegment); j += 32) {
            const int id = row[j];
            if (id < 0 || id >= A.num_pages) status |= 4;
            else if (orphan && !(j < above && row[j - A.ldt] == id)) marks.set(has ? keep : drop, id);
        }
    }
    cluster.sync();
    // 2. the pages that nobody holds any more, ascending, to the end of the free list
    int freed = 0, before;
    if (orphan) {
        const int run = max(1, words / kThreads), w0 = tid * run;
        int mine = 0;
        for (int w = w0; w < min(words, w0 + run); ++w) mine += __popc(drop[w] & ~keep[w]);
        int cta, total;
        int at = block_scan(mine, warp_sums, &cta);
        exchange(cluster, slots, cta, &before, &total);
        freed = total;
        if (count + freed > A.capacity) {
            freed = 0;
            status |= 1;
        } else {
            int64_t to = count + before + at;
            for (int w = w0; w < min(words, w0 + run); ++w)
                for (uint32_t bits = drop[w] & ~keep[w]; bits; bits &= bits - 1)
                    A.free_pages[to++] = (rank << A.shift) + w * 32 + __ffs(int(bits)) - 1;
        }
    }
    // 3. a page for every child that shares a partly filled one with an earlier child
    const int per = (A.batch_out + kThreads - 1) / kThreads, r0 = tid * per;
    int need = 0;
    unsigned wants = 0;
    for (int k = 0; k < per && r0 + k < A.batch_out; ++k) {
        const int r = r0 + k, p = A.parents[r];
        if (p < 0 || p >= A.batch || first[p] == r) continue;
        const int len = A.lens[p];
        const int64_t n = pages_of(len);
        if (n == 0 || len % ps == 0) continue;
        const int id = A.table[p * A.ldt + n - 1];
        if (id < 0 || id >= A.num_pages) continue;
        wants |= 1u << k;
        ++need;
    }
    int wanted;
    int nth = block_scan(need, warp_sums, &wanted);
    cluster.sync();                     // the free list is whole
    const int64_t have = count + freed;
    for (int k = 0; k < per && r0 + k < A.batch_out; ++k) {
        int page = -1;
        if (wants >> k & 1) {
            const int64_t at = have - 1 - nth++;
            page = at >= 0 ? __ldcg(A.free_pages + at) : -2;
            if (at < 0) status |= 2;
            else if (page < 0 || page >= A.num_pages) status |= 4, page = -2;
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
    for (int64_t i = int64_t(rank) * kWarps + warp; i < A.batch_out * segs; i += C * kWarps) {
        const int r = int(i / segs), p = A.parents[r];
        if (p < 0 || p >= A.batch || fresh[r] == -2) continue;
        const int64_t n = pages_of(A.lens[p]), j0 = (i - r * segs) * kSegment;
        const int32_t *from = A.table + p * A.ldt;
        int32_t *to = A.table_out + r * A.ldto;
        for (int64_t j = j0 + lane; j < min(n, j0 + kSegment); j += 32)
            to[j] = j == n - 1 && fresh[r] >= 0 ? fresh[r] : from[j];
    }
    if (rank == 0 && tid == 0)
        *A.free_count_out = int(have - min(int64_t(wanted), have));
    if (A.dev_status) {
        status = __reduce_or_sync(0xffffffffu, unsigned(status));
        if (lane == 0 && status) atomicOr(reinterpret_cast<int *>(A.dev_status), status);
    }
}

struct CompactArgs {
    int batch;
    int64_t page_size, num_pages;
    const int32_t *lens, *table;
    int64_t max_pages, ldt;
    int32_t *table_out;
    int64_t ldto;
    int32_t *free_pages, *free_count_out, *src, *dst, *moves, *dev_status;
    int shift;
};

__global__ void __launch_bounds__(kThreads) pages_compact_kernel(const CompactArgs A) {
    extern __shared__ uint32_t sm[];
    const int words = 1 << (A.shift - 5);
    uint32_t *held = sm;
    __shared__ int warp_sums[32], slots[3][kMaxCluster];
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Marks marks = {cluster, A.shift};
    const int64_t ps = A.page_size, room = min(A.max_pages * ps, int64_t(0x7fffffff));
    int status = 0;
    auto pages_of = [&](int len) {
        return len < 0 || len > room ? int64_t(0) : (len + ps - 1) / ps;
    };
    for (int i = tid; i < words; i += kThreads) held[i] = 0;
    cluster.sync();
    const int64_t segs = (A.max_pages + kSegment - 1) / kSegment;
    for (int64_t i = int64_t(rank) * kWarps + warp; i < A.batch * segs; i += C * kWarps) {
        const int b = int(i / segs), len = A.lens[b];
        if (len < 0 || len > room) status |= 1;
        const int64_t n = pages_of(len), j0 = (i - b * segs) * kSegment;
        if (j0 >= n) continue;
        const int64_t above = b > 0 ? pages_of(A.lens[b - 1]) : 0;
        const int32_t *row = A.table + b * A.ldt;
        for (int64_t j = j0 + lane; j < min(n, j0 + kSegment); j += 32) {
            const int id = row[j];
            if (id < 0 || id >= A.num_pages) status |= 4;
            else if (!(j < above && row[j - A.ldt] == id)) marks.set(held, id);
        }
    }
    cluster.sync();
    // the pages in use, then those of them past the first `used` ids and the holes before
    const int run = max(1, words / kThreads), w0 = tid * run, w1 = min(words, w0 + run);
    int mine = 0, cta, before, used;
    for (int w = w0; w < w1; ++w) mine += __popc(held[w]);
    block_scan(mine, warp_sums, &cta);
    exchange(cluster, slots[0], cta, &before, &used);
    const int base = rank << A.shift;
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
    int am = block_scan(nm, warp_sums, &cm), ah = block_scan(nh, warp_sums, &ch);
    exchange(cluster, slots[1], cm, &bm, &total);
    exchange(cluster, slots[2], ch, &bh, &same);
    for (int w = w0; w < w1; ++w) {
        for (uint32_t bits = moving(w); bits; bits &= bits - 1)
            A.src[bm + am++] = base + w * 32 + __ffs(int(bits)) - 1;
        for (uint32_t bits = holes(w); bits; bits &= bits - 1)
            A.dst[bh + ah++] = base + w * 32 + __ffs(int(bits)) - 1;
    }
    cluster.sync();                     // the lists are whole
    for (int64_t i = int64_t(rank) * kWarps + warp; i < A.batch * segs; i += C * kWarps) {
        const int b = int(i / segs);
        const int64_t n = pages_of(A.lens[b]), j0 = (i - b * segs) * kSegment;
        for (int64_t j = j0 + lane; j < min(n, j0 + kSegment); j += 32) {
            int id = A.table[b * A.ldt + j];
            if (id >= used && id < A.num_pages) {
                int lo = 0, hi = total;         // src[lo] <= id < src[hi]
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (__ldcg(A.src + mid) <= id) lo = mid; else hi = mid;
                }
                id = __ldcg(A.dst + lo);
            }
            A.table_out[b * A.ldto + j] = id;
        }
    }
    const int64_t spare = A.num_pages - used;
    for (int64_t i = int64_t(rank) * kThreads + tid; i < spare; i += C * kThreads)
        A.free_pages[i] = int(A.num_pages - 1 - i);
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
constexpr int kCopyThreads = 256;
constexpr int kFilterWords = 4096;                  // 2^17 pages, by the low bits
constexpr int kUnroll = 8;

struct CopyArgs {
    float *k, *v;
    int64_t num_pages;
    int page_size, kv_heads, head_dim;
    int64_t page_stride, token_stride, head_stride;
    const int32_t *src, *dst, *tokens, *count;
    int pairs;
    int seg_tokens, segs;             // tokens of a CTA's piece; pieces of a page
    int32_t *dev_status;
};

// WIDE: floats of a unit (4 or 1). Units of a piece: token, then head, then dim.
template <int WIDE>
__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const CopyArgs A) {
    // pages that are a source; a destination; a destination at least twice
    __shared__ uint32_t is_src[kFilterWords], is_dst[kFilterWords], twice[kFilterWords];
    const int tid = threadIdx.x;
    int n = A.pairs, status = 0;
    if (A.count) {
        const int c = *A.count;
        if (c < 0 || c > n) status |= 1;
        n = min(max(c, 0), n);
    }
    if (int64_t(blockIdx.x) >= int64_t(n) * A.segs && blockIdx.x != 0) return;
    for (int i = tid; i < kFilterWords; i += kCopyThreads) is_src[i] = is_dst[i] = twice[i] = 0;
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
    for (int i = tid; i < n; i += kCopyThreads) {
        int s, d, t;
        if (!valid(i, s, d, t)) continue;
        const unsigned a = unsigned(s) & (kFilterWords * 32 - 1);
        const unsigned b = unsigned(d) & (kFilterWords * 32 - 1);
        atomicOr(is_src + (a >> 5), 1u << (a & 31));
        if (atomicOr(is_dst + (b >> 5), 1u << (b & 31)) >> (b & 31) & 1)
            atomicOr(twice + (b >> 5), 1u << (b & 31));
    }
    __syncthreads();
    const int units = A.head_dim / WIDE, row = A.kv_heads * units;
    for (int64_t w = blockIdx.x; w < int64_t(n) * A.segs; w += gridDim.x) {
        const int i = int(w / A.segs), seg = int(w - int64_t(i) * A.segs);
        int s, d, t;
        if (!valid(i, s, d, t)) continue;           // the same for all threads
        const unsigned b = unsigned(d) & (kFilterWords * 32 - 1);
        const uint32_t bit = 1u << (b & 31);
        if ((is_src[b >> 5] | twice[b >> 5]) & bit) {
            // maybe: look through the pairs
            int later = 0, read = 0;
            for (int j = tid; j < n; j += kCopyThreads) {
                int s2, d2, t2;
                if (!valid(j, s2, d2, t2)) continue;
                read |= s2 == d;
                later |= d2 == d && j > i;
            }
            read = __syncthreads_or(read);
            later = __syncthreads_or(later);
            if (read) status |= 2;
            if (read || later) continue;
        }
        const int t0 = seg * A.seg_tokens, t1 = min(t, t0 + A.seg_tokens);
        const int64_t from = s * A.page_stride, to = d * A.page_stride;
        const int total = max(0, t1 - t0) * row;
        for (int half = 0; half < 2; ++half) {
            float *base = half ? A.v : A.k;
            for (int u0 = tid; u0 < total; u0 += kCopyThreads * kUnroll) {
                float4 v4[kUnroll];
                int64_t at[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int x = u0 + u * kCopyThreads;
                    if (x >= total) break;
                    const int tok = x / row, rest = x - tok * row, g = rest / units;
                    at[u] = (t0 + tok) * A.token_stride + g * A.head_stride +
                            int64_t(rest - g * units) * WIDE;
                    if (WIDE == 4) v4[u] = *reinterpret_cast<const float4 *>(base + from + at[u]);
                    else v4[u].x = base[from + at[u]];
                }
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    if (u0 + u * kCopyThreads >= total) break;
                    if (WIDE == 4) *reinterpret_cast<float4 *>(base + to + at[u]) = v4[u];
                    else base[to + at[u]] = v4[u].x;
                }
            }
        }
    }
    if (A.dev_status) {
        status = __reduce_or_sync(0xffffffffu, unsigned(status));
        if ((tid & 31) == 0 && status) atomicOr(reinterpret_cast<int *>(A.dev_status), status);
    }
}

// CTAs of the cluster and pages of a CTA's marks (a power of two of at least 32):
// enough CTAs that a warp has few table segments and the marks fit.
struct ClusterPlan {
    int ctas, shift;
};
ClusterPlan cluster_plan(int64_t rows, int64_t max_pages, int64_t num_pages) {
    ClusterPlan p = {1, 5};
    const int64_t work = rows * ((max_pages + 127) / 128) + num_pages / 4096;
    while (p.ctas < kMaxCluster && p.ctas * kWarps < work) p.ctas *= 2;
    while ((int64_t(p.ctas) << kSliceShift) < num_pages) p.ctas *= 2;
    while ((int64_t(p.ctas) << p.shift) < num_pages) ++p.shift;
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
                        free_count_out, src, dst, tokens, dev_status, p.shift};
    const size_t smem = (size_t(1) << p.shift) / 8 * 2 + 2 * kMaxBatch * 4;
    return run_cluster(pages_fork_kernel, A, p.ctas, smem, s);
}

cudaError_t launch_pages_compact(int64_t batch, int64_t page_size, int64_t num_pages,
                                 const int32_t *lens, const int32_t *table, int64_t max_pages,
                                 int64_t ldt, int32_t *table_out, int64_t ldto,
                                 int32_t *free_pages, int32_t *free_count_out, int32_t *src,
                                 int32_t *dst, int32_t *moves, int32_t *dev_status,
                                 cudaStream_t s) {
    const ClusterPlan p = cluster_plan(batch, max_pages, num_pages);
    const CompactArgs A = {int(batch), page_size, num_pages, lens, table, max_pages, ldt, table_out,
                           ldto, free_pages, free_count_out, src, dst, moves, dev_status, p.shift};
    return run_cluster(pages_compact_kernel, A, p.ctas, (size_t(1) << p.shift) / 8, s);
}

cudaError_t launch_kv_copy(int64_t pairs, const int32_t *src, const int32_t *dst,
                           const int32_t *tokens, const int32_t *count, const det_kv_cache &c,
                           int32_t *dev_status, cudaStream_t s) {
    auto al16 = [](const void *x) { return reinterpret_cast<uintptr_t>(x) % 16 == 0; };
    const bool vec = al16(c.k) && al16(c.v) && c.page_stride % 4 == 0 && c.token_stride % 4 == 0 &&
                     c.head_stride % 4 == 0 && c.head_dim % 4 == 0;
    CopyArgs A = {c.k, c.v, c.num_pages, int(c.page_size), int(c.kv_heads), int(c.head_dim),
                  c.page_stride, c.token_stride, c.head_stride, src, dst, tokens, count, int(pairs),
                  0, 0, dev_status};
    // a piece: tokens whose units all have one round of the threads' loads, or one
    const int64_t units = c.kv_heads * c.head_dim / (vec ? 4 : 1);
    const int64_t fit = std::max<int64_t>(1, kCopyThreads * kUnroll / units);
    A.seg_tokens = int(std::min(fit, c.page_size));
    A.segs = int((c.page_size + A.seg_tokens - 1) / A.seg_tokens);
    const int64_t grid = std::min<int64_t>(pairs * A.segs, int64_t(sm_count_current_device()) * 4);
    if (vec) kv_copy_kernel<4><<<unsigned(grid), kCopyThreads, 0, s>>>(A);
    else kv_copy_kernel<1><<<unsigned(grid), kCopyThreads, 0, s>>>(A);
    return cudaGetLastError();
}

}  // namespace det
