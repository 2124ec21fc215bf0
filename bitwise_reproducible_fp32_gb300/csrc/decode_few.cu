// decode_few.cu -- the tokens that a request of decode_shared.cu has to itself, with at
// most 8 query rows a key-value head, for sm_103a.
//
// The same formulas and bits; a key or value takes at most 16 multiply-adds, so HBM
// bounds it. As in decode.cu a warp streams pieces of 64 tokens x 32 dimensions through
// a ring of its own (rows of 128 bytes, their 16-byte units swapped by row mod 8), with
// two tokens a lane for the scores and a dimension a lane for P V. A worker is a warp,
// and its work a run of all units' tiles or chunks, so short requests leave no SM
// idle. Measured: 64 requests with 157..1255 tokens of their own, 12 heads of 64, scores 25
// us and P V 26 (123 MB each, 4.8 TB/s). Neighbouring runs go to one CTA's warps (a call of
// 64 requests on 8192 tokens 157 -> 146 us with the same in P V of the shared ones), and
// rings of two pieces leave room for three CTAs an SM.
#include <algorithm>

#include "decode_shared.cuh"

namespace det {

// Set when a bounded wait for a piece gave up.
__device__ unsigned int g_few_watchdog;

namespace {

constexpr int kFewCtas = 3;               // an SM's, where registers allow

// NH: the rows the registers hold, of which the unit has at most NH.
template <int NH, Loader LOAD>
__global__ void __launch_bounds__(kThreads, 2)
    few_scores_kernel(const SharedArgs A, const __grid_constant__ CUtensorMap kmap) {
    constexpr int CUT = kOwnTiles;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ Share share[kWarps];
    __shared__ uint64_t full[kWarps][kRingPieces];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d = A.d, nsl = (d + 31) / 32, live_rows = rows_of<CUT>(A), ldq = nsl * 32;
    init_bars<LOAD>(&full[0][0]);
    Beside<true> beside;
    shares<CUT, kWarps>(A, A.kv_heads, blockIdx.x * kWarps, 1, gridDim.x * kWarps, share);
    const int64_t items = share[warp].items;
    if (items <= 0) return;
    Ring<LOAD> ring(A, &kmap, A.k, smem_u32(smem_raw) + warp * kRingBytes, smem_u32(&full[warp][0]));
    float *qs = reinterpret_cast<float *>(smem_raw + kWarps * kRingBytes) +
                warp * NH * ldq;

    Item in = share[warp].at;
    int64_t left = items * nsl;
    int in_sl = 0, in_t0 = 0, in_live = 0;
    auto start = [&]() {
        in_t0 = first_token<CUT>(in);
        in_live = tokens_from<CUT>(in, in_t0);
        ring.look_up(pages_of<CUT>(A, in), in_t0, in_live);
    };
    start();
    auto issue = [&]() {
        if (left > 0) {
            ring.fetch(in.run, in_sl, in_t0, in_live);
            if (++in_sl == nsl) {
                in_sl = 0;
                advance<CUT>(A, A.kv_heads, in);
                if (left > 1) start();
            }
            --left;
        }
        if (LOAD != kTma) cp_commit();
    };
    for (int i = 0; i < kRingPieces - 1; ++i) issue();
    uint32_t kat[8];              // 16-byte unit i of row `lane` of a piece
#pragma unroll
    for (int i = 0; i < 8; ++i) kat[i] = lane * 128 + ((i ^ (lane & 7)) << 4);

    Item it = share[warp].at;
    int held_u = -1, held_kv = -1;
    int rows[NH];                 // (b, h), -1 where there is none
    float m[NH];
    auto flush = [&]() {          // the held rows' maxima
        if (held_u < 0) return;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            float t = m[h];
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1)
                t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, off));
            if (lane == 0 && rows[h] >= 0) atomicMax(A.top + rows[h], max_key(t));
        }
    };
    for (int64_t i = 0; i < items; ++i) {
        if (it.u != held_u || it.run != held_kv) {
            flush();
            held_u = it.u;
            held_kv = it.run;
            __syncwarp();
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                m[h] = __uint_as_float(0xff800000u);
                rows[h] = h < live_rows ? row_at(A, group_of<CUT>(A, it.u), it.run,
                                                 place_of<CUT>(A, it.u, h))
                                        : -1;
                if (rows[h] < 0) continue;
                const int b = rows[h] / A.heads;
                const float *q = A.q + b * A.ldq + int64_t(rows[h] - b * A.heads) * d;
                for (int j = lane; j < d; j += 32) qs[h * ldq + j] = q[j];
            }
            __syncwarp();
        }
        const int t0 = first_token<CUT>(it), live = tokens_from<CUT>(it, t0);
        float acc[2][NH];         // of tokens lane and lane + 32
#pragma unroll
        for (int h = 0; h < NH; ++h) acc[0][h] = acc[1][h] = 0.0f;
        for (int sl = 0; sl < nsl; ++sl) {
            ring.wait();
            if (!ring.stuck) issue();         // into the slot consumed before this one
            const uint32_t piece = ring.piece();
            const int width = min(32, d - 32 * sl);
            const float *q = qs + 32 * sl;
            auto four = [&](int u) {
                const float4 k0 = lds4(piece + kat[u]), k1 = lds4(piece + 4096 + kat[u]);
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const float4 qv = *reinterpret_cast<const float4 *>(q + h * ldq + 4 * u);
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
                        for (int c = 4 * u; c < width; ++c) {
                            const float k0 = lds1(piece + kat[u] + 4 * (c & 3));
                            const float k1 = lds1(piece + 4096 + kat[u] + 4 * (c & 3));
#pragma unroll
                            for (int h = 0; h < NH; ++h) {
                                acc[0][h] = __fmaf_rn(q[h * ldq + c], k0, acc[0][h]);
                                acc[1][h] = __fmaf_rn(q[h * ldq + c], k1, acc[1][h]);
                            }
                        }
                    }
                }
            }
        }
        if (ring.stuck) {         // this and the other rows of the share are NaN
#pragma unroll
            for (int h = 0; h < NH; ++h) m[h] = __uint_as_float(0x7fc00000u);
        } else {
            const int g = group_of<CUT>(A, it.u), place = place_of<CUT>(A, it.u, 0);
            const int64_t octet = (int64_t(g) * A.kv_heads + it.run) * A.octets + t0 / 8 + lane / 8;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (32 * k + lane >= live) continue;
                float *x = A.x + ((octet + 4 * k) * A.rows + place) * 8 + (lane & 7);
#pragma unroll
                for (int h = 0; h < NH; ++h)
                    if (rows[h] >= 0) {
                        const float v = __fmul_rn(acc[k][h], A.scale);
                        x[h * 8] = v;
                        m[h] = max_nan(m[h], v);
                    }
            }
        }
        advance<CUT>(A, A.kv_heads, it);
    }
    flush();
    ring.drain(&g_few_watchdog);
}

template <int NH, Loader LOAD>
__global__ void __launch_bounds__(kThreads, 2)
    few_partials_kernel(const SharedArgs A, const __grid_constant__ CUtensorMap vmap) {
    constexpr int CUT = kOwn;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ Share share[kWarps];
    __shared__ uint64_t full[kWarps][kRingPieces];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d = A.d, nsl = (d + 31) / 32, live_rows = rows_of<CUT>(A), mul = A.kv_heads * nsl;
    init_bars<LOAD>(&full[0][0]);
    Beside<true> beside;
    shares<CUT, kWarps>(A, mul, blockIdx.x * kWarps, 1, gridDim.x * kWarps, share);
    const int64_t items = share[warp].items;
    if (items <= 0) return;
    Ring<LOAD> ring(A, &vmap, A.v, smem_u32(smem_raw) + warp * kRingBytes, smem_u32(&full[warp][0]));
    const uint32_t copies = smem_u32(smem_raw) + kWarps * kRingBytes + warp * (NH * kTile * 4);

    Item in = share[warp].at;
    int64_t in_items = items;
    int in_t = 0, in_left = 0;            // next token of the item, tokens left
    int in_kv = 0, in_sl = 0;
    auto look_up = [&]() {
        if (in_items > 0) ring.look_up(pages_of<CUT>(A, in), in_t, min(kTile, in_left));
    };
    auto start = [&]() {
        in_t = first_token<CUT>(in);
        in_left = tokens_from<CUT>(in, in_t);
        in_kv = in.run / nsl;
        in_sl = in.run - in_kv * nsl;
    };
    start();
    look_up();
    auto issue = [&]() {
        if (in_items > 0) {
            ring.fetch(in_kv, in_sl, in_t, min(kTile, in_left));
            in_t += kTile;
            in_left -= kTile;
            if (in_left <= 0) {
                advance<CUT>(A, mul, in);
                if (--in_items > 0) start();
            }
            look_up();
        }
        if (LOAD != kTma) cp_commit();
    };
    for (int i = 0; i < kRingPieces - 1; ++i) issue();
    uint32_t vat[8];              // column `lane` of rows i mod 8 of a piece
#pragma unroll
    for (int i = 0; i < 8; ++i) vat[i] = i * 128 + (((lane >> 2) ^ i) << 4) + ((lane & 3) << 2);

    // ---- exps, asked for a piece ahead
    Item it = share[warp].at;
    float keep[2 * NH], inv[NH];
    int rows[NH];                 // (b, h), -1 where there is none
    const float *from = nullptr;  // of the item's first token, at the lane's place in its octet
    int held_u = -1, held_kv = -1;
    auto hold = [&]() {
        const int kv = it.run / nsl, g = group_of<CUT>(A, it.u), place = place_of<CUT>(A, it.u, 0);
        const int64_t octet = (int64_t(g) * A.kv_heads + kv) * A.octets + first_token<CUT>(it) / 8;
        from = A.x + ((octet + lane / 8) * A.rows + place) * 8 + (lane & 7);
        if (it.u == held_u && kv == held_kv) return;
        held_u = it.u;
        held_kv = kv;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            rows[h] = h < live_rows ? row_at(A, g, kv, place + h) : -1;
            inv[h] = rows[h] >= 0 ? A.inv[rows[h]] : 0.0f;
        }
    };
    auto ask = [&](int t, int tokens) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const int at = t + 32 * k + lane;
                keep[2 * h + k] = rows[h] >= 0 && at < tokens
                                      ? from[int64_t(t / 8 + 4 * k) * A.rows * 8 + h * 8]
                                      : 0.0f;
            }
    };
    auto tokens_of = [&]() { return tokens_from<CUT>(it, first_token<CUT>(it)); };
    hold();
    ask(0, tokens_of());
    for (int64_t i = 0; i < items; ++i) {
        const int sl = it.run % nsl;
        const int t0 = first_token<CUT>(it), tokens = tokens_of();
        float *out = A.part + int64_t(t0 / kKChunk) * d + 32 * sl + lane;
        float acc[NH];
        int mine[NH];             // the rows, before the next item's
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            acc[h] = 0.0f;
            mine[h] = rows[h];
        }
        for (int t = 0; t < tokens; t += kTile) {
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 2 * NH; ++k)
                sts1(copies + (k * 32 + lane) * 4, __fmul_rn(keep[k], inv[k / 2]));
            if (t + kTile < tokens) {
                ask(t + kTile, tokens);
            } else if (i + 1 < items) {
                advance<CUT>(A, mul, it);
                hold();
                ask(0, tokens_of());
            }
            ring.wait();
            if (!ring.stuck) issue();         // into the slot consumed before this one
            const uint32_t piece = ring.piece();
            auto four = [&](int r) {
                const uint32_t up = piece + (r & ~7) * 128;
                const float v0 = lds1(up + vat[r & 7]), v1 = lds1(up + vat[(r & 7) + 1]),
                            v2 = lds1(up + vat[(r & 7) + 2]), v3 = lds1(up + vat[(r & 7) + 3]);
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const float4 w = lds4(copies + h * (kTile * 4) + r * 4);
                    acc[h] = __fmaf_rn(w.x, v0, acc[h]);
                    acc[h] = __fmaf_rn(w.y, v1, acc[h]);
                    acc[h] = __fmaf_rn(w.z, v2, acc[h]);
                    acc[h] = __fmaf_rn(w.w, v3, acc[h]);
                }
            };
            const int live = tokens - t;
            if (live >= kTile) {
#pragma unroll
                for (int r = 0; r < kTile; r += 4) four(r);
            } else {
#pragma unroll 2
                for (int r8 = 0; r8 < kTile; r8 += 8) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (r8 + k < live) {
                            const float v = lds1(piece + r8 * 128 + vat[k]);
#pragma unroll
                            for (int h = 0; h < NH; ++h)
                                acc[h] = __fmaf_rn(lds1(copies + h * (kTile * 4) + (r8 + k) * 4), v,
                                                   acc[h]);
                        }
                }
            }
        }
        if (32 * sl + lane < d)
#pragma unroll
            for (int h = 0; h < NH; ++h)
                if (mine[h] >= 0)
                    out[mine[h] * A.ldpart * d] = ring.stuck ? __uint_as_float(0x7fc00000u) : acc[h];
    }
    ring.drain(&g_few_watchdog);
}

template <class K>
cudaError_t run_few(K kern, int64_t items, size_t row_bytes, const SharedArgs &A,
                    const CUtensorMap *map, cudaStream_t s) {
    // the most any call takes, as another thread's call may come before the launch
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMaxSmem));
    if (e != cudaSuccess) return e;
    const int64_t grid = std::min<int64_t>((items + kWarps - 1) / kWarps,
                                           int64_t(sm_count_current_device()) * kFewCtas);
    const CUtensorMap none = {};
    return launch_dependent(kern, dim3(unsigned(std::max<int64_t>(1, grid))), dim3(kThreads),
                            kWarps * (kRingBytes + row_bytes), s, A,
                            map ? *map : none);
}

template <int NH>
cudaError_t scores_of(const SharedArgs &A, const CUtensorMap *map, int64_t most, cudaStream_t s) {
    const size_t rows = size_t(NH) * ((A.d + 31) / 32 * 32) * 4;
    const int64_t items = most * (kKChunk / kTile) * A.kv_heads;
    return map      ? run_few(few_scores_kernel<NH, kTma>, items, rows, A, map, s)
           : A.wide ? run_few(few_scores_kernel<NH, kCopy16>, items, rows, A, map, s)
                    : run_few(few_scores_kernel<NH, kCopy4>, items, rows, A, map, s);
}
template <int NH>
cudaError_t partials_of(const SharedArgs &A, const CUtensorMap *map, int64_t most, cudaStream_t s) {
    const size_t rows = size_t(NH) * kTile * 4;
    const int64_t items = most * A.kv_heads * ((A.d + 31) / 32);
    return map      ? run_few(few_partials_kernel<NH, kTma>, items, rows, A, map, s)
           : A.wide ? run_few(few_partials_kernel<NH, kCopy16>, items, rows, A, map, s)
                    : run_few(few_partials_kernel<NH, kCopy4>, items, rows, A, map, s);
}

}  // namespace

cudaError_t launch_few_scores(const SharedArgs &A, const CUtensorMap *map, int64_t most,
                              cudaStream_t s) {
    return A.per_kv == 1   ? scores_of<1>(A, map, most, s)
           : A.per_kv == 2 ? scores_of<2>(A, map, most, s)
           : A.per_kv <= 4 ? scores_of<4>(A, map, most, s)
                           : scores_of<kFewRows>(A, map, most, s);
}
cudaError_t launch_few_partials(const SharedArgs &A, const CUtensorMap *map, int64_t most,
                                cudaStream_t s) {
    return A.per_kv == 1   ? partials_of<1>(A, map, most, s)
           : A.per_kv == 2 ? partials_of<2>(A, map, most, s)
           : A.per_kv <= 4 ? partials_of<4>(A, map, most, s)
                           : partials_of<kFewRows>(A, map, most, s);
}

cudaError_t few_decode_watchdog(unsigned int *code, int clear) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_few_watchdog, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    if (clear && *code) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_few_watchdog, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace det
