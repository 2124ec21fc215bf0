// rotary.cu -- the rotary embedding at positions of the caller's own, and the
// append of new keys and values to a paged cache, for sm_103a.
//
//   y0 = x0 c - x1 s,  y1 = x0 s + x1 c  over the pairs of a head's first rot_dim
//   elements (products rounded, then the difference or sum); the rest passes.
//
// Both stream each element once in and once out, so HBM bounds them. A thread
// owns one unit of a row -- 16 bytes of a head: two interleaved pairs, or four
// pairs of the half layout (two 16-byte pieces) -- and walks the heads of a
// group, kBatch loads in flight, so an angle's sin and cos are formed once a
// group and not once a head; the first batch is on its way while they are. Rows
// with other alignments or odd sizes take units of one pair (or one element where
// nothing turns).
// Measured in a graph, inputs and outputs beyond L2: 8192 rows of 24 heads of 64
// turned in 17.9 us (5.6 TB/s; 14.3 where the calls share an output, which stays in
// L2), in the half layout 22.4 (4.5 TB/s); the backward of 4099 rows of 40 heads of
// 128, half of each turned, 34 us (4.9 TB/s); 8192 rows of 32 + 2 x 8 heads of 128,
// 7/8 of them kept, appended in 70 us (5.0 TB/s).
#include <algorithm>

#include "det_internal.cuh"
#include "det_math.cuh"

namespace det {
namespace {

constexpr int kBatch = 4;         // heads a thread loads before it stores

enum UnitMode { kInterleaved4, kHalf4, kScalar };

struct Angles {
    const uint64_t *turns;        // null: theta
    float theta;
    int rot, half;
};

__device__ __forceinline__ void pair_sincos(const Angles &a, float log_theta, int pos, int i,
                                            float &sn, float &cs) {
    if (a.turns) {
        turns_sincos(uint64_t(pos) * a.turns[i], sn, cs);
    } else {
        const float ex = __fdiv_rn(float(2 * i), float(a.rot));
        const float w = det_exp(__fmul_rn(-ex, log_theta));
        det_sincos(__fmul_rn(float(pos), w), sn, cs);
    }
}

__device__ __forceinline__ void turn(float &x0, float &x1, float sn, float cs) {
    const float y0 = __fsub_rn(__fmul_rn(x0, cs), __fmul_rn(x1, sn));
    x1 = __fadd_rn(__fmul_rn(x0, sn), __fmul_rn(x1, cs));
    x0 = y0;
}
// the transpose, in the backward's spelling: dx0 = y0 c + y1 s, dx1 = y1 c - y0 s
__device__ __forceinline__ void turn_back(float &x0, float &x1, float sn, float cs) {
    const float y0 = __fadd_rn(__fmul_rn(x0, cs), __fmul_rn(x1, sn));
    x1 = __fsub_rn(__fmul_rn(x1, cs), __fmul_rn(x0, sn));
    x0 = y0;
}

// Units of a head: first those that turn, then those that pass through.
template <int MODE>
struct Unit {
    static constexpr int kPairs = MODE == kInterleaved4 ? 2 : MODE == kHalf4 ? 4 : 1;
    static constexpr int kWide = MODE == kScalar ? 1 : 4;       // floats of a passing unit
    float sn[kPairs], cs[kPairs];
    int at0, at1;       // offsets of the pieces in a head (at1: the partner's)
    bool turns;

    __device__ __forceinline__ Unit(const Angles &a, int u, int pos) {
        const int nturn = a.rot / (2 * kPairs);
        turns = u < nturn && pos >= 0;
        if (u >= nturn) {
            at0 = a.rot + (u - nturn) * kWide;
            at1 = -1;
        } else if (MODE == kInterleaved4) {
            at0 = 4 * u;
            at1 = -1;
        } else if (MODE == kHalf4) {
            at0 = 4 * u;
            at1 = a.rot / 2 + 4 * u;
        } else {
            at0 = a.half ? u : 2 * u;
            at1 = a.half ? a.rot / 2 + u : 2 * u + 1;
        }
    }
    __device__ __forceinline__ void angles(const Angles &a, int u, int pos) {
        if (!turns) return;
        const float log_theta = a.turns ? 0.0f : det_log(a.theta);
#pragma unroll
        for (int k = 0; k < kPairs; ++k)
            pair_sincos(a, log_theta, pos, u * kPairs + k, sn[k], cs[k]);
    }
};

struct Piece4 { float4 a, b; };
struct Piece1 { float a, b; };
template <int MODE> struct PieceOf { using type = Piece4; };
template <> struct PieceOf<kScalar> { using type = Piece1; };

template <int MODE>
__device__ __forceinline__ typename PieceOf<MODE>::type load_unit(const float *head,
                                                                  const Unit<MODE> &u) {
    typename PieceOf<MODE>::type p;
    if constexpr (MODE == kScalar) {
        p.a = head[u.at0];
        p.b = u.at1 >= 0 ? head[u.at1] : 0.0f;
    } else {
        p.a = *reinterpret_cast<const float4 *>(head + u.at0);
        if (MODE == kHalf4 && u.at1 >= 0) p.b = *reinterpret_cast<const float4 *>(head + u.at1);
    }
    return p;
}

template <int MODE>
__device__ __forceinline__ void store_unit(float *head, const Unit<MODE> &u,
                                           const typename PieceOf<MODE>::type &p) {
    if constexpr (MODE == kScalar) {
        head[u.at0] = p.a;
        if (u.at1 >= 0) head[u.at1] = p.b;
    } else {
        *reinterpret_cast<float4 *>(head + u.at0) = p.a;
        if (MODE == kHalf4 && u.at1 >= 0) *reinterpret_cast<float4 *>(head + u.at1) = p.b;
    }
}

template <int MODE, bool BACK>
__device__ __forceinline__ void turn_unit(const Unit<MODE> &u, typename PieceOf<MODE>::type &p) {
    auto t = [](float &x0, float &x1, float sn, float cs) {
        BACK ? turn_back(x0, x1, sn, cs) : turn(x0, x1, sn, cs);
    };
    if constexpr (MODE == kInterleaved4) {
        t(p.a.x, p.a.y, u.sn[0], u.cs[0]);
        t(p.a.z, p.a.w, u.sn[1], u.cs[1]);
    } else if constexpr (MODE == kHalf4) {
        t(p.a.x, p.b.x, u.sn[0], u.cs[0]);
        t(p.a.y, p.b.y, u.sn[1], u.cs[1]);
        t(p.a.z, p.b.z, u.sn[2], u.cs[2]);
        t(p.a.w, p.b.w, u.sn[3], u.cs[3]);
    } else {
        t(p.a, p.b, u.sn[0], u.cs[0]);
    }
}

// Thread e of grid.x: unit e mod units of row e / units; grid.y: the group of
// heads. In place, the units that pass through and padding rows have no work.
template <int MODE, bool BACK>
__global__ void __launch_bounds__(256)
    rope_at_kernel(int64_t rows, int heads, int head_dim, const float *x, int64_t ldx,
                   const int32_t *__restrict__ positions, Angles ang, int units, int group,
                   float *out, int64_t ldo) {
    const int64_t e = blockIdx.x * int64_t(blockDim.x) + threadIdx.x;
    const int64_t t = e / units;
    if (t >= rows) return;
    const int pos = positions[t];
    Unit<MODE> u(ang, int(e - t * units), pos);
    if (!u.turns && out == x) return;
    const int h0 = blockIdx.y * group, h1 = min(heads, h0 + group);
    const float *src = x + t * ldx;
    float *dst = out + t * ldo;
    typename PieceOf<MODE>::type p[kBatch];
    auto load = [&](int h) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (h + k < h1) p[k] = load_unit<MODE>(src + int64_t(h + k) * head_dim, u);
    };
    load(h0);
    u.angles(ang, int(e - t * units), pos);
    for (int h = h0; h < h1; h += kBatch) {
        if (h > h0) load(h);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (h + k < h1) {
                if (u.turns) turn_unit<MODE, BACK>(u, p[k]);
                store_unit<MODE>(dst + int64_t(h + k) * head_dim, u, p[k]);
            }
    }
}

struct AppendArgs {
    int64_t rows;
    int heads, kv_heads, head_dim;
    const float *qkv;
    int64_t ldqkv;
    const int64_t *slots;
    const int32_t *positions;     // null: nothing turns
    float *q_out;                 // null: Q is left out
    int64_t ldq;
    float *k, *v;
    int64_t nslots, page_size, page_stride, token_stride, head_stride;
    int32_t *dev_status;
    int units, group, tile;       // tile: rows of a CTA
};

constexpr int kAppendTile = 16;
constexpr int kScan = 8;          // slots a thread has in flight
constexpr int kFilterBits = 4096;

// A CTA takes `tile` rows and a group of the row's heads (Q, then K, then V;
// grid.y), a thread one unit of one row. Where a later row names the same slot,
// the earlier row's K and V are not written, so the cache always holds the last
// one: each CTA with K or V heads looks through the slots after its rows, most of
// which a bit filter of its own slots' low bits passes over at once (comparing
// each with the tile's 16: 63 us instead of 32 for 8192 rows of 36 heads of 64). The
// search grows with the square of the rows: 8192 rows of 1 + 2 x 1 heads of 64 take
// 15.5 us, 65536 252 us, 2^18 3.6 ms, 2^20 55 ms.
// Four CTAs an SM: with more registers for loads over the search, 96 us instead of
// 70 for the 8192 rows above.
template <int MODE>
__global__ void __launch_bounds__(256, 4) kv_append_kernel(AppendArgs A, Angles ang) {
    __shared__ int64_t slot_of[kAppendTile];
    __shared__ int later[kAppendTile], pos_of[kAppendTile];
    __shared__ unsigned filter[kFilterBits / 32];
    const int tid = threadIdx.x;
    const int64_t row0 = int64_t(blockIdx.x) * A.tile;
    const int all = A.heads + 2 * A.kv_heads;
    const int first = A.q_out ? 0 : A.heads;
    const int h0 = first + blockIdx.y * A.group, h1 = min(all, h0 + A.group);
    for (int i = tid; i < kFilterBits / 32; i += blockDim.x) filter[i] = 0;
    __syncthreads();
    if (tid < A.tile) {
        slot_of[tid] = row0 + tid < A.rows ? A.slots[row0 + tid] : -1;
        pos_of[tid] = row0 + tid < A.rows && A.positions ? A.positions[row0 + tid] : 0;
        later[tid] = 0;
        const unsigned b = unsigned(slot_of[tid]) % kFilterBits;
        if (slot_of[tid] >= 0) atomicOr(&filter[b / 32], 1u << b % 32);
        if (blockIdx.y == 0 && slot_of[tid] >= A.nslots && A.dev_status &&
            pos_of[tid] >= 0)
            atomicOr(reinterpret_cast<int *>(A.dev_status), 1);
    }
    __syncthreads();
    if (h1 > A.heads) {
        for (int64_t j0 = row0 + 1 + tid; j0 < A.rows; j0 += kScan * blockDim.x) {
            int64_t s[kScan];
#pragma unroll
            for (int k = 0; k < kScan; ++k) {
                const int64_t j = j0 + k * blockDim.x;
                s[k] = j < A.rows ? A.slots[j] : -1;
            }
#pragma unroll
            for (int k = 0; k < kScan; ++k) {
                const unsigned b = unsigned(s[k]) % kFilterBits;
                if (!(filter[b / 32] >> (b % 32) & 1)) continue;
                const int64_t j = j0 + k * blockDim.x;
                for (int i = 0; i < A.tile; ++i)
                    if (s[k] >= 0 && s[k] == slot_of[i] && j > row0 + i &&
                        (!A.positions || A.positions[j] >= 0))
                        later[i] = 1;
            }
        }
        __syncthreads();
    }
    const int r = tid / A.units, unit = tid - r * A.units;
    const int64_t t = row0 + r;
    const int64_t slot = r < A.tile ? slot_of[r] : -1;
    if (slot < 0 || slot >= A.nslots || pos_of[r] < 0) return;
    const int pos = A.positions ? pos_of[r] : -1;
    Unit<MODE> u(ang, unit, pos);
    const float *src = A.qkv + t * A.ldqkv;
    typename PieceOf<MODE>::type p[kBatch];
    auto load = [&](int h) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (h + k < h1) p[k] = load_unit<MODE>(src + int64_t(h + k) * A.head_dim, u);
    };
    load(h0);
    u.angles(ang, unit, pos);
    const int64_t at = (slot / A.page_size) * A.page_stride + (slot % A.page_size) * A.token_stride;
    const bool keep = !later[r];
    for (int h = h0; h < h1; h += kBatch) {
        if (h > h0) load(h);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int hh = h + k;
            if (hh >= h1) break;
            const int g = hh - A.heads;
            if (u.turns && g < A.kv_heads) turn_unit<MODE, false>(u, p[k]);
            if (g < 0)
                store_unit<MODE>(A.q_out + t * A.ldq + int64_t(hh) * A.head_dim, u, p[k]);
            else if (keep)
                store_unit<MODE>(g < A.kv_heads
                                     ? A.k + at + g * A.head_stride
                                     : A.v + at + (g - A.kv_heads) * A.head_stride,
                                 u, p[k]);
        }
    }
}

bool al16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// 16-byte units where every piece of every head is 16-byte aligned.
UnitMode unit_mode(int head_dim, int rot, int half, bool aligned) {
    if (!aligned || head_dim % 4) return kScalar;
    if (half && rot) return rot % 8 ? kScalar : kHalf4;
    return rot % 4 ? kScalar : kInterleaved4;
}

int units_of(UnitMode m, int head_dim, int rot) {
    const int pairs = m == kInterleaved4 ? 2 : m == kHalf4 ? 4 : 1, wide = m == kScalar ? 1 : 4;
    return rot / (2 * pairs) + (head_dim - rot) / wide;
}

// Heads a thread walks: as many as leave the GPU 2048 threads an SM, in groups of
// whole batches, equal but for the last. The kernels' registers let 1024 (half
// layout, append) or 1280 (interleaved) run at once, so this is about two waves; the
// last one is not full (4099 rows of 40 heads: 1540 CTAs on 608 places; 8192 rows of 24
// heads of 64, interleaved: 1536 on 760). Fewer heads form each angle more often
// (8192 rows of 32 + 16 heads of 128 appended: 16 heads 70 us, 4 heads 85), more
// leave SMs idle (64 rows of 36 heads of 64: 4 heads 5.2 us, 48 heads 9.8) or the
// last group short (4099 rows of 40 heads turned: 12 heads 34 us, 16 heads 37).
int head_group(int64_t threads, int heads) {
    const int64_t full = int64_t(sm_count_current_device()) * 2048;
    const int64_t want = std::max<int64_t>((heads * threads + full - 1) / full, 1);
    const int64_t groups = (heads + want - 1) / want, even = (heads + groups - 1) / groups;
    return int(std::min<int64_t>(heads, (even + kBatch - 1) / kBatch * kBatch));
}

}  // namespace

cudaError_t launch_rope_at(int64_t rows, int heads, int head_dim, const float *x, int64_t ldx,
                           const int32_t *positions, const RotaryArgs &ro, int inverse,
                           float *out, int64_t ldo, cudaStream_t s) {
    const UnitMode m = unit_mode(head_dim, ro.rot, ro.half,
                                 al16(x) && al16(out) && ldx % 4 == 0 && ldo % 4 == 0);
    const int units = units_of(m, head_dim, ro.rot);
    const Angles ang = {ro.turns, ro.theta, ro.rot, ro.half};
    const int group = head_group(rows * units, heads);
    const dim3 grid(unsigned((rows * units + 255) / 256), unsigned((heads + group - 1) / group));
    auto run = [&](auto kern) {
        kern<<<grid, 256, 0, s>>>(rows, heads, head_dim, x, ldx, positions, ang, units, group, out,
                                  ldo);
        return cudaGetLastError();
    };
    if (m == kInterleaved4)
        return inverse ? run(rope_at_kernel<kInterleaved4, true>)
                       : run(rope_at_kernel<kInterleaved4, false>);
    if (m == kHalf4)
        return inverse ? run(rope_at_kernel<kHalf4, true>) : run(rope_at_kernel<kHalf4, false>);
    return inverse ? run(rope_at_kernel<kScalar, true>) : run(rope_at_kernel<kScalar, false>);
}

cudaError_t launch_kv_append(int64_t rows, int heads, const float *qkv, int64_t ldqkv,
                             const int64_t *slots, const int32_t *positions, const RotaryArgs &ro,
                             const det_kv_cache &c, float *q_out, int64_t ldq,
                             int32_t *dev_status, cudaStream_t s) {
    const int head_dim = int(c.head_dim);
    const bool aligned = al16(qkv) && ldqkv % 4 == 0 && al16(c.k) && al16(c.v) &&
                         c.page_stride % 4 == 0 && c.token_stride % 4 == 0 &&
                         c.head_stride % 4 == 0 && (!q_out || (al16(q_out) && ldq % 4 == 0));
    const UnitMode m = unit_mode(head_dim, ro.rot, ro.half, aligned);
    AppendArgs A = {rows, heads, int(c.kv_heads), head_dim, qkv, ldqkv, slots, positions, q_out,
                    ldq, c.k, c.v, c.num_pages * c.page_size, c.page_size, c.page_stride,
                    c.token_stride, c.head_stride, dev_status, 0, 0, 0};
    A.units = units_of(m, head_dim, ro.rot);
    A.tile = std::min(kAppendTile, std::max(1, 256 / A.units));
    const int all = (q_out ? heads : 0) + 2 * A.kv_heads;
    A.group = head_group(rows * A.units, all);
    const Angles ang = {ro.turns, ro.theta, ro.rot, ro.half};
    const dim3 grid(unsigned((rows + A.tile - 1) / A.tile), unsigned((all + A.group - 1) / A.group));
    const unsigned threads = unsigned((A.tile * A.units + 31) / 32 * 32);
    if (m == kInterleaved4)
        kv_append_kernel<kInterleaved4><<<grid, threads, 0, s>>>(A, ang);
    else if (m == kHalf4)
        kv_append_kernel<kHalf4><<<grid, threads, 0, s>>>(A, ang);
    else
        kv_append_kernel<kScalar><<<grid, threads, 0, s>>>(A, ang);
    return cudaGetLastError();
}

}  // namespace det
