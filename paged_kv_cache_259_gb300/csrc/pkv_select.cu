// Choice of the cache blocks a decode query attends over, by a cheap score.
//
// update_key_bounds keeps, for every (block, kv head), the smallest and the
// largest value of each key dim over the block's filled slots. For any key of
// the block q.k = sum_d q_d k_d <= sum_d max(q_d lo_d, q_d hi_d), so
//     score(h, j) = max_{g < G} sum_d max(q_gd lo_jd, q_gd hi_jd)
// bounds the logit of every token of block j under every query head of kv head
// h. select_blocks takes the first and last blocks of the sequence and the
// highest-scoring others.
//
// Scores as a matrix product. max(q lo, q hi) = q+ hi + q- lo with q+ = max(q,
// 0), q- = min(q, 0): the score of 16 blocks under 8 heads is one m16n8 tile of
// [lo hi] (16 x 2D) times [q- q+] (2D x 8), on mma.sync (8 columns at most, far
// below the tcgen05 tiles). The kernel streams the bounds once: 2 D values per
// block against the 2 D block_size values of its K and V.
//
// Exact choice. A float32 score carries rounding, and blocks whose scores lie
// within it could change places with the summation order. The choice made is
// that of the exact scores: the float32 scores s' are off by at most E (below),
// so with T the k-th largest s', a block with s' > T + 2E is in, one with s' <
// T - 2E is out, and only if the window between holds more blocks than places
// left are those few scored again in 64 bits and ranked, equal scores by the
// lower index.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cmath>
#include <type_traits>

#include "pkv_internal.cuh"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// min / max that return NaN if either operand is (a NaN key must not vanish)
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, __nv_bfloat16) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __nv_bfloat16) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, __half) {
    uint32_t r;
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, __half) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, float) {
    return __float_as_uint(min_nan(__uint_as_float(a), __uint_as_float(b)));
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, float) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
}

// ------------------------------------------------------------ update_key_bounds
// What 16 bytes of a K tile hold, as registers of comparable values: 4 x f32,
// 4 x bf16x2, or (E4M3, exact in f16) 8 x f16x2.
template <typename KV> struct Cmp;
template <> struct Cmp<float> {
    using T = float;
    static constexpr int kRegs = 4, kElt = 4;
    static constexpr uint32_t kInf = 0x7f800000u, kNegInf = 0xff800000u;
};
template <> struct Cmp<__nv_bfloat16> {
    using T = __nv_bfloat16;
    static constexpr int kRegs = 4, kElt = 2;
    static constexpr uint32_t kInf = 0x7f807f80u, kNegInf = 0xff80ff80u;
};
template <> struct Cmp<uint8_t> {
    using T = __half;
    static constexpr int kRegs = 8, kElt = 1;
    static constexpr uint32_t kInf = 0x7c007c00u, kNegInf = 0xfc00fc00u;
};

template <typename KV>
__device__ __forceinline__ void widen(const uint4& raw, uint32_t (&x)[Cmp<KV>::kRegs]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (std::is_same<KV, uint8_t>::value) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const unsigned short in = (unsigned short)(w[i] >> (16 * j));
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(x[2 * i + j]) : "h"(in));
            }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = w[i];
    }
}

// One warp per (changed block, kv head). A load of the warp covers 4 chunks of
// dims x 8 tokens (512 contiguous bytes of the K tile); the token groups are
// compared in registers, then the 8 token lanes reduce by halves: each step
// exchanges half of the registers, so 7 shuffles (14 for E4M3) leave every lane
// its share of the result, in the order the bounds are stored.
// Bound: HBM bytes of the changed blocks' K; a decode step (one block per
// sequence) is launch latency.
template <typename KV>
__global__ void __launch_bounds__(128, 8) update_key_bounds_kernel(
    const uint4* __restrict__ k_pool, void* __restrict__ bounds, const int32_t* __restrict__ tables,
    const int32_t* __restrict__ lens, const int32_t* __restrict__ first, int max_blocks,
    int num_blocks, int hkv, int d, int bs, int* err) {
    pdl_enter();                                           // launched with launch_pdl
    using C = Cmp<KV>;
    constexpr int R = C::kRegs;
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    int L = lens[b];
    int f = first[b];
    if (L < 0 || L > max_blocks * bs || f < 0) {
        if (blockIdx.x == 0 && threadIdx.x == 0) flag_error(err, kErrOutOfRange);
        L = min(max(L, 0), max_blocks * bs);
        f = max(f, 0);
    }
    if (f >= L) return;
    const int j0 = f / bs, nblk = (L + bs - 1) / bs;
    const long long items = (long long)(nblk - j0) * hkv;
    const int planes = d * C::kElt / 16;                   // 16-byte chunks per token
    const int tl = lane & 7, pl = lane >> 3;               // token and chunk of the load
    for (long long it = blockIdx.x * 4LL + (threadIdx.x >> 5); it < items; it += gridDim.x * 4LL) {
        const int j = j0 + (int)(it / hkv), h = (int)(it % hkv);
        const int id = tables[(size_t)b * max_blocks + j];
        if (id < 0 || id >= num_blocks) {
            if (lane == 0 && h == 0) flag_error(err, kErrOutOfRange);
            continue;
        }
        const int ntok = min(bs, L - j * bs);
        const uint4* tile = k_pool + ((size_t)id * hkv + h) * planes * bs;
        char* out = static_cast<char*>(bounds) +
                    ((size_t)id * hkv + h) * 2 * d * (C::kElt == 4 ? 4 : 2);
        for (int q = 0; q < planes; q += 4) {
            const bool in = q + pl < planes;
            uint32_t x[2 * R];                             // min | max
#pragma unroll
            for (int i = 0; i < R; ++i) x[i] = C::kInf, x[R + i] = C::kNegInf;
            for (int g = 0; g * 8 < ntok; ++g) {
                if (in && g * 8 + tl < ntok) {
                    uint32_t v[R];
                    widen<KV>(tile[(g * planes + q + pl) * 8 + tl], v);
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        x[i] = min2(x[i], v[i], typename C::T{});
                        x[R + i] = max2(x[R + i], v[i], typename C::T{});
                    }
                }
            }
            // step 1 (tokens t, t^4): the lower lane keeps the minima, the upper
            // the maxima; steps 2 and 3 halve what is left
            const bool up = (tl & 4) != 0;
            uint32_t y[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const uint32_t other = __shfl_xor_sync(kFull, up ? x[i] : x[R + i], 4);
                y[i] = up ? max2(x[R + i], other, typename C::T{}) : min2(x[i], other, typename C::T{});
            }
#pragma unroll
            for (int s = 1; s <= 2; ++s) {
                const int keep = R >> s;
                const bool hi = (tl & (4 >> s)) != 0;
#pragma unroll
                for (int i = 0; i < R / 2; ++i)
                    if (i < keep) {
                        const uint32_t other = __shfl_xor_sync(kFull, hi ? y[i] : y[keep + i], 4 >> s);
                        const uint32_t mine = hi ? y[keep + i] : y[i];
                        y[i] = up ? max2(mine, other, typename C::T{}) : min2(mine, other, typename C::T{});
                    }
            }
            if (!in) continue;
            // lane tl holds registers (tl & 3) * R/4 .. of the chunk's minima or maxima
            if constexpr (std::is_same<KV, uint8_t>::value) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&y[i]));
                    const __nv_bfloat162 w = __floats2bfloat162_rn(v.x, v.y);   // exact
                    y[i] = *reinterpret_cast<const uint32_t*>(&w);
                }
                *reinterpret_cast<uint2*>(out + (up ? 2 * d : 0) + (q + pl) * 32 + (tl & 3) * 8) =
                    make_uint2(y[0], y[1]);
            } else {
                *reinterpret_cast<uint32_t*>(out + (up ? d * C::kElt : 0) + (q + pl) * 16 + (tl & 3) * 4) = y[0];
            }
        }
    }
}

// ----------------------------------------------------------------- select_blocks
struct SelectParams {
    int32_t* selected;                 // [B][Hkv][K]
    const void* q;                     // [B][Hq][D]
    const void* bounds;                // [NB][Hkv][2][D]
    const int32_t* tables;
    const int32_t* lens;
    float* scores;                     // [B][Hkv][stride], stride a multiple of 16
    float* tile_max;                   // [B][Hkv][stride / 16]: largest |bound| of 16 blocks
    unsigned long long* exact;         // [B][Hkv][stride]
    int max_blocks, num_blocks, hq, hkv, d, bs, k, first, last;
    int stride, cached;                // cached: scores a row keeps in shared memory
    int* err;
};

// Blocks of sequence b (lengths outside the table clamped; flagged by `flag`).
__device__ __forceinline__ int row_blocks(const SelectParams& p, int b, bool flag) {
    int L = p.lens[b];
    if (L < 0 || L > p.max_blocks * p.bs) {
        if (flag) flag_error(p.err, kErrOutOfRange);
        L = L < 0 ? 0 : p.max_blocks * p.bs;
    }
    return (L + p.bs - 1) / p.bs;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t x) {
    uint32_t r;                                            // |r| = max(|m|, |x|), NaN kept
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x));
    return r;
}

// Scores of 16 blocks per warp. The k order of the product is free as long as
// both operands agree on it, so lane (r, c) loads 16 bytes of blocks r and r+8
// at dims 32i + 8c .. +7 straight into the A fragments of k-steps 2i and 2i+1
// (no shared memory), and the same dims of query head r into the B fragments.
// Four accumulator chains (by i) shorten the dependency and the rounding.
// Bound: HBM bytes of the bounds.
template <int D>
__global__ void __launch_bounds__(128) score_blocks_bf16(const SelectParams p, int tiles_per_warp) {
    pdl_enter();                                           // launched with launch_pdl
    const int h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31;
    const int n = row_blocks(p, b, false);
    if (n <= p.k) return;                                  // every block is selected
    const int lo = p.first, hi = n - p.last;               // blocks with a score: [lo, hi)
    const int tile0 = (blockIdx.x * 4 + (threadIdx.x >> 5)) * tiles_per_warp;
    if (tile0 * 16 >= hi) return;
    const int r = lane >> 2, c = lane & 3, G = p.hq / p.hkv;
    constexpr int I = D / 32;                              // 16-byte chunks a lane holds per bound
    uint32_t qn[I][4], qp[I][4];                           // min(q, 0), max(q, 0)
#pragma unroll
    for (int i = 0; i < I; ++i) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (r < G)
            w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                ((size_t)b * p.hq + h * G + r) * D + 32 * i + 8 * c);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            qn[i][j] = min2(x[j], 0u, __nv_bfloat16{});
            qp[i][j] = max2(x[j], 0u, __nv_bfloat16{});
        }
    }
    const size_t row = (size_t)b * p.hkv + h;
    for (int tile = tile0; tile < tile0 + tiles_per_warp && tile * 16 < hi; ++tile) {
        if (tile * 16 + 15 < lo) continue;
        const int j = tile * 16 + (lane & 15);
        int id = -1;
        if (j >= lo && j < hi) {
            id = p.tables[(size_t)b * p.max_blocks + j];
            if (id < 0 || id >= p.num_blocks) {
                flag_error(p.err, kErrOutOfRange);
                id = -1;
            }
        }
        const int id0 = __shfl_sync(kFull, id, r), id1 = __shfl_sync(kFull, id, r + 8);
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.bounds);
        const uint4* p0 = reinterpret_cast<const uint4*>(src + ((size_t)max(id0, 0) * p.hkv + h) * 2 * D) + c;
        const uint4* p1 = reinterpret_cast<const uint4*>(src + ((size_t)max(id1, 0) * p.hkv + h) * 2 * D) + c;
        uint4 x0[2 * I], x1[2 * I];
#pragma unroll
        for (int i = 0; i < 2 * I; ++i) {
            x0[i] = id0 >= 0 ? __ldg(p0 + 4 * i) : make_uint4(0, 0, 0, 0);
            x1[i] = id1 >= 0 ? __ldg(p1 + 4 * i) : make_uint4(0, 0, 0, 0);
        }
        float acc[4][4];
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[a][e] = 0.f;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 2 * I; ++i) {
            const uint32_t(&qq)[4] = i < I ? qn[i < I ? i : 0] : qp[i < I ? 0 : i - I];
            mma_bf16(acc[i & 3], x0[i].x, x1[i].x, x0[i].y, x1[i].y, qq[0], qq[1]);
            mma_bf16(acc[i & 3], x0[i].z, x1[i].z, x0[i].w, x1[i].w, qq[2], qq[3]);
            m = abs_max2(abs_max2(m, x0[i].x), x0[i].y);
            m = abs_max2(abs_max2(m, x0[i].z), x0[i].w);
            m = abs_max2(abs_max2(m, x1[i].x), x1[i].y);
            m = abs_max2(abs_max2(m, x1[i].z), x1[i].w);
        }
        // heads 2c, 2c+1 of blocks r (s0) and r+8 (s1); columns past G are no heads
        float s0 = -INFINITY, s1 = -INFINITY;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (2 * c + e < G) {
                s0 = max_nan(s0, (acc[0][e] + acc[1][e]) + (acc[2][e] + acc[3][e]));
                s1 = max_nan(s1, (acc[0][2 + e] + acc[1][2 + e]) + (acc[2][2 + e] + acc[3][2 + e]));
            }
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            s0 = max_nan(s0, __shfl_xor_sync(kFull, s0, o));
            s1 = max_nan(s1, __shfl_xor_sync(kFull, s1, o));
        }
        float* out = p.scores + row * p.stride + tile * 16;
        if (c == 0) {
            out[r] = id0 >= 0 ? s0 + 0.f : -INFINITY;      // + 0: no negative zero
            out[r + 8] = id1 >= 0 ? s1 + 0.f : -INFINITY;
        }
        m &= 0x7fff7fffu;
        float mf = max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mf = max_nan(mf, __shfl_xor_sync(kFull, mf, o));
        if (lane == 0) p.tile_max[row * (p.stride / 16) + tile] = mf;
    }
}

// float32 bounds and queries (tensor cores would round them): a warp takes a
// block at a time, lane l the dims l, l + 32, ..., and the heads' sums are
// reduced across the lanes.
template <int D>
__global__ void __launch_bounds__(128) score_blocks_f32(const SelectParams p, int tiles_per_warp) {
    pdl_enter();                                           // launched with launch_pdl
    const int h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31;
    const int n = row_blocks(p, b, false);
    if (n <= p.k) return;
    const int lo = p.first, hi = n - p.last;
    const int tile0 = (blockIdx.x * 4 + (threadIdx.x >> 5)) * tiles_per_warp;
    if (tile0 * 16 >= hi) return;
    constexpr int I = D / 32;
    const int G = p.hq / p.hkv;
    float qv[8][I];
#pragma unroll
    for (int g = 0; g < 8; ++g)
#pragma unroll
        for (int i = 0; i < I; ++i)
            qv[g][i] = g < G ? static_cast<const float*>(p.q)[((size_t)b * p.hq + h * G + g) * D + lane + 32 * i] : 0.f;
    const size_t row = (size_t)b * p.hkv + h;
    for (int tile = tile0; tile < tile0 + tiles_per_warp && tile * 16 < hi; ++tile) {
        if (tile * 16 + 15 < lo) continue;
        float mf = 0.f;
#pragma unroll 4
        for (int jj = 0; jj < 16; ++jj) {
            const int j = tile * 16 + jj;
            if (j < lo || j >= hi) continue;
            const int id = p.tables[(size_t)b * p.max_blocks + j];
            float best = -INFINITY;
            if (id < 0 || id >= p.num_blocks) {
                if (lane == 0) flag_error(p.err, kErrOutOfRange);
            } else {
                const float* src = static_cast<const float*>(p.bounds) + ((size_t)id * p.hkv + h) * 2 * D + lane;
                float l[I], u[I];
#pragma unroll
                for (int i = 0; i < I; ++i) {
                    l[i] = __ldg(src + 32 * i);
                    u[i] = __ldg(src + D + 32 * i);
                    mf = max_nan(mf, max_nan(fabsf(l[i]), fabsf(u[i])));
                }
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    if (g >= G) break;
                    float s = 0.f;
#pragma unroll
                    for (int i = 0; i < I; ++i) {
                        s = fmaf(min_nan(qv[g][i], 0.f), l[i], s);
                        s = fmaf(max_nan(qv[g][i], 0.f), u[i], s);
                    }
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
                    best = max_nan(best, s);
                }
            }
            if (lane == 0) p.scores[row * p.stride + j] = best + 0.f;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mf = max_nan(mf, __shfl_xor_sync(kFull, mf, o));
        if (lane == 0) p.tile_max[row * (p.stride / 16) + tile] = mf;
    }
}

// Values whose unsigned order is the numbers' order.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float((k >> 31) ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ unsigned long long ordered64(double x) {
    const unsigned long long u = __double_as_longlong(x);
    return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}

constexpr int kBins = 2048;            // 11 bits a pass
constexpr int kListMax = 1024;         // candidates ranked in shared memory

// One CTA per (kv head, sequence) over the row's scores: threshold by radix
// passes over the score's range (the range cut into 2,048 bins, then the bin,
// ...; three passes at most), the 64-bit tie break when the rounding window is
// crowded, then the selected blocks' bits written out in ascending order.
// Bound: latency (a row is at most a few hundred KB of scores, from L2).
template <typename T, int NT>
__global__ void __launch_bounds__(NT) select_rows(const SelectParams p) {
    pdl_enter();                                           // launched with launch_pdl
    constexpr int NW = NT / 32;
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const size_t row = (size_t)b * p.hkv + h;
    int32_t* out = p.selected + row * p.k;
    const int n = row_blocks(p, b, h == 0 && tid == 0);
    if (n <= p.k) {                                        // all of them
        for (int i = tid; i < p.k; i += NT) out[i] = i < n ? i : -1;
        return;
    }
    extern __shared__ __align__(16) unsigned char smem[];
    const int words = (n + 31) / 32;
    const int words_max = (p.max_blocks + 31) / 32;
    unsigned long long* list_key = reinterpret_cast<unsigned long long*>(smem);    // [kListMax]
    int* list_id = reinterpret_cast<int*>(list_key + kListMax);                    // [kListMax]
    uint32_t* hist = reinterpret_cast<uint32_t*>(list_id + kListMax);              // [kBins]
    uint32_t* sel = hist + kBins;                                                  // selected blocks
    uint32_t* cand = sel + words_max;                                              // undecided blocks
    float* cache = reinterpret_cast<float*>(cand + words_max);                     // [cached]
    __shared__ uint32_t warp_a[NW], warp_b[NW];
    __shared__ uint32_t sh_bin, sh_left;

    const int lo = p.first, hi = n - p.last;               // scored blocks
    const int nmid = hi - lo, need = p.k - p.first - p.last;   // 0 <= need < nmid
    const float* scores = p.scores + row * p.stride + lo;
    const bool in_smem = nmid <= p.cached;
    for (int i = tid; i < words; i += NT) {
        // the forced blocks' bits: [0, first) and [n - last, n)
        uint32_t bits = 0;
        for (int j = 0; j < 32; ++j) {
            const int blk = 32 * i + j;
            if (blk < lo || (blk >= hi && blk < n)) bits |= 1u << j;
        }
        sel[i] = bits;
        cand[i] = 0;
    }

    auto block_sum = [&](uint32_t a, uint32_t bb, uint32_t* suma, uint32_t* sumb) {
        a = __reduce_add_sync(kFull, a);
        bb = __reduce_add_sync(kFull, bb);
        __syncthreads();                                   // earlier readers of warp_a / warp_b
        if (lane == 0) warp_a[w] = a, warp_b[w] = bb;
        __syncthreads();
        uint32_t x = lane < NW ? warp_a[lane] : 0, y = lane < NW ? warp_b[lane] : 0;
        *suma = __reduce_add_sync(kFull, x);
        *sumb = __reduce_add_sync(kFull, y);
    };
    // exclusive prefix over the threads
    auto block_scan = [&](uint32_t v, uint32_t* total) -> uint32_t {
        uint32_t incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += t;
        }
        __syncthreads();
        if (lane == 31) warp_a[w] = incl;
        __syncthreads();
        uint32_t x = lane < NW ? warp_a[lane] : 0, xi = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(kFull, xi, o);
            if (lane >= o) xi += t;
        }
        *total = __shfl_sync(kFull, xi, 31);
        return __shfl_sync(kFull, xi - x, w) + incl - v;
    };
    const int per = (words + NT - 1) / NT;                 // bitmap words of a thread, in order
    const int w0 = min(words, tid * per), w1 = min(words, w0 + per);

    if (need > 0) {
        // ---- how far a score can be off. A = max_g sum_d |q_gd| times the largest
        // |bound| of the row is at least the sum of the magnitudes of a score's
        // terms. bf16: products exact in float32; four chains of at most four
        // mma.sync, each aligning at most 17 terms to the largest and dropping
        // bits below its 24th (17 x 2^-23 of it) and rounding once, chains adding
        // up to A: 4 x 18 x 2^-23 A < 2^-16 A with the last adds and A's own
        // rounding. float32: at most 2 D / 32 + 5 roundings of 2^-24: < 2^-19 A.
        const int G = p.hq / p.hkv, d = p.d;
        float qsum = 0.f;
        if (w < G) {
            const T* qr = static_cast<const T*>(p.q) + ((size_t)b * p.hq + h * G + w) * d;
            for (int i = lane; i < d; i += 32) qsum += fabsf((float)qr[i]);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) qsum += __shfl_xor_sync(kFull, qsum, o);
        }
        float mx = 0.f;
        const float* tm = p.tile_max + row * (p.stride / 16);
        for (int i = lo / 16 + tid; i * 16 < hi; i += NT) mx = max_nan(mx, tm[i]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(kFull, mx, o));
        if (lane == 0) {
            warp_a[w] = __float_as_uint(qsum);             // 0 for warps past G
            warp_b[w] = __float_as_uint(mx);
        }
        // ---- the row's scores, their range
        uint32_t kmin = 0xffffffffu, kmax = 0;
        for (int i = tid; i < nmid; i += NT) {
            const float s = scores[i];
            if (in_smem) cache[i] = s;
            const uint32_t k = ordered(s);
            kmin = min(kmin, k);
            kmax = max(kmax, k);
        }
        kmin = __reduce_min_sync(kFull, kmin);
        kmax = __reduce_max_sync(kFull, kmax);
        if (lane == 0) list_id[w] = (int)kmin, list_id[32 + w] = (int)kmax;
        __syncthreads();
        const float qs = lane < NW ? __uint_as_float(warp_a[lane]) : 0.f;
        const float ms = lane < NW ? __uint_as_float(warp_b[lane]) : 0.f;
        kmin = __reduce_min_sync(kFull, lane < NW ? (uint32_t)list_id[lane] : 0xffffffffu);
        kmax = __reduce_max_sync(kFull, lane < NW ? (uint32_t)list_id[32 + lane] : 0u);
        float qm = qs, mm = ms;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            qm = max_nan(qm, __shfl_xor_sync(kFull, qm, o));
            mm = max_nan(mm, __shfl_xor_sync(kFull, mm, o));
        }
        const float A = qm * mm;
        // (1e-35: products too small for float32; a zero side makes every score 0)
        const bool zero = qm == 0.f || mm == 0.f;
        const float E = zero ? 0.f : A * (std::is_same<T, float>::value ? 0x1p-19f : 0x1p-16f) + 1e-35f;
        const bool sane = A < 1e37f;                       // false for NaN too
        const float* src = in_smem ? cache : scores;

        uint32_t left = need;                              // places among the undecided blocks
        uint32_t undecided = nmid;
        if (sane) {
            // ---- T: the need-th largest score
            uint32_t base = kmin, range = kmax - kmin;
            uint32_t want = need;
            while (range > 0) {
                const int bits = 32 - __clz(range);
                const int shift = bits > 11 ? bits - 11 : 0;
                for (int i = tid; i < kBins; i += NT) hist[i] = 0;
                __syncthreads();
                for (int i = tid; i < nmid; i += NT) {
                    const uint32_t off = ordered(src[i]) - base;
                    if (ordered(src[i]) >= base && off <= range) atomicAdd(&hist[off >> shift], 1u);
                }
                __syncthreads();
                // the bin that holds the want-th from the top: thread t sums the
                // bins kBins-1 - t*BPT downwards
                constexpr int BPT = kBins / NT;
                uint32_t cnt[BPT], sum = 0;
#pragma unroll
                for (int i = 0; i < BPT; ++i) {
                    cnt[i] = hist[kBins - 1 - (tid * BPT + i)];
                    sum += cnt[i];
                }
                uint32_t total;
                uint32_t above = block_scan(sum, &total);
#pragma unroll
                for (int i = 0; i < BPT; ++i) {
                    if (above < want && want <= above + cnt[i]) {
                        sh_bin = kBins - 1 - (tid * BPT + i);
                        sh_left = want - above;
                    }
                    above += cnt[i];
                }
                __syncthreads();
                base += sh_bin << shift;
                want = sh_left;
                // what is left of the range inside that bin
                const uint32_t top = kmax - base;
                range = shift == 0 ? 0u : min((1u << shift) - 1u, top);
                __syncthreads();                           // sh_bin, hist are rewritten
            }
            const float thr = unordered(base);
            // ---- the window 2E around it (2.02: the rounding of these two sums)
            const float win = 2.02f * E, up = thr + win, dn = thr - win;
            uint32_t in = 0, near = 0;
            for (int i = tid; i < nmid; i += NT) {
                const float s = src[i];
                in += s > up;
                near += s >= dn && s <= up;
            }
            uint32_t n_in, n_near;
            block_sum(in, near, &n_in, &n_near);
            left = need - n_in;
            undecided = n_near;
            for (int i0 = tid - lane; i0 < nmid; i0 += NT) {
                const int i = i0 + lane;
                const float s = i < nmid ? src[i] : 0.f;
                const bool is_in = i < nmid && s > up, is_near = i < nmid && s >= dn && s <= up;
                // block lo + i: bit (lo + i) & 31 of its word; a warp's 32 blocks
                // reach over two words at most
                if (is_in) atomicOr(&sel[(lo + i) >> 5], 1u << ((lo + i) & 31));
                if (is_near) atomicOr(&cand[(lo + i) >> 5], 1u << ((lo + i) & 31));
            }
        } else {
            for (int i = tid; i < nmid; i += NT)
                atomicOr(&cand[(lo + i) >> 5], 1u << ((lo + i) & 31));
        }
        __syncthreads();

        if (undecided > left && !(sane && zero)) {
            // ---- score the undecided blocks in 64 bits (products of two float32 or
            // bf16 values are exact there; one order of summation for all blocks)
            auto exact_key = [&](int blk) -> unsigned long long {   // the whole warp
                const int id = p.tables[(size_t)b * p.max_blocks + blk];
                if (id < 0 || id >= p.num_blocks) return 0ull;      // flagged when it was scored
                const T* bl = static_cast<const T*>(p.bounds) + ((size_t)id * p.hkv + h) * 2 * d;
                double best = -INFINITY;
                bool nan = false;
                for (int g = 0; g < G; ++g) {
                    const T* qr = static_cast<const T*>(p.q) + ((size_t)b * p.hq + h * G + g) * d;
                    double s = 0.0;
                    for (int i = lane; i < d; i += 32) {
                        const double q = (double)(float)qr[i];
                        const double neg = q > 0.0 ? 0.0 : q, pos = q < 0.0 ? 0.0 : q;   // NaN stays
                        s = fma(neg, (double)(float)bl[i], s);
                        s = fma(pos, (double)(float)bl[d + i], s);
                    }
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
                    nan |= s != s;
                    best = s > best ? s : best;
                }
                // a block that no finite score describes comes first
                if (nan || !(fabs(best) < INFINITY)) best = INFINITY;
                return ordered64(best + 0.0);
            };
            uint32_t mine = 0;
            for (int i = w0; i < w1; ++i) mine += __popc(cand[i]);
            uint32_t total;
            uint32_t at = block_scan(mine, &total);
            if (total <= kListMax) {
                for (int i = w0; i < w1; ++i)
                    for (uint32_t m = cand[i]; m; m &= m - 1) list_id[at++] = 32 * i + __ffs(m) - 1;
                __syncthreads();
                for (int i = w; i < (int)total; i += NW) {
                    const unsigned long long k = exact_key(list_id[i]);
                    if (lane == 0) list_key[i] = k;
                }
                __syncthreads();
                for (int i = tid; i < (int)total; i += NT) {
                    const unsigned long long k = list_key[i];
                    uint32_t before = 0;
                    for (int j = 0; j < (int)total; ++j)
                        before += list_key[j] > k || (list_key[j] == k && j < i);
                    if (before < left) atomicOr(&sel[list_id[i] >> 5], 1u << (list_id[i] & 31));
                }
                undecided = left = 0;                      // decided
            } else {
                // a crowd (degenerate scores): keys to the workspace, threshold by
                // bisection of the 64-bit keys
                unsigned long long* key = p.exact + row * p.stride;
                for (int blk = lo + w; blk < hi; blk += NW)
                    if ((cand[blk >> 5] >> (blk & 31)) & 1) {
                        const unsigned long long k = exact_key(blk);
                        if (lane == 0) key[blk] = k;
                    }
                __syncthreads();
                unsigned long long thr = 0;                // largest t with >= left keys >= t
                for (int bit = 63; bit >= 0; --bit) {
                    const unsigned long long t = thr | (1ull << bit);
                    uint32_t c = 0;
                    for (int blk = lo + tid; blk < hi; blk += NT)
                        c += ((cand[blk >> 5] >> (blk & 31)) & 1) && key[blk] >= t;
                    uint32_t all, none;
                    block_sum(c, 0, &all, &none);
                    if (all >= left) thr = t;
                }
                uint32_t c = 0;
                for (int blk = lo + tid; blk < hi; blk += NT) {
                    const uint32_t bit = 1u << (blk & 31);
                    if (!(cand[blk >> 5] & bit)) continue;
                    if (key[blk] > thr) {
                        atomicOr(&sel[blk >> 5], bit);
                        ++c;
                    }
                    if (key[blk] != thr) atomicAnd(&cand[blk >> 5], ~bit);
                }
                uint32_t above, none;
                block_sum(c, 0, &above, &none);
                left -= above;
                undecided = left + 1;                      // equal keys: by index
            }
        }
        __syncthreads();
        if (left > 0) {
            // ---- the `left` lowest-indexed undecided blocks (all of them, or equals)
            uint32_t mine = 0;
            for (int i = w0; i < w1; ++i) mine += __popc(cand[i]);
            uint32_t total;
            uint32_t at = block_scan(mine, &total);
            for (int i = w0; i < w1; ++i) {
                uint32_t m = cand[i], take = 0;
                for (; m && at < left; m &= m - 1, ++at) take |= m & (~m + 1);
                sel[i] |= take;
            }
        }
    }
    __syncthreads();
    // ---- the selected blocks, ascending
    uint32_t mine = 0;
    for (int i = w0; i < w1; ++i) mine += __popc(sel[i]);
    uint32_t total;
    uint32_t at = block_scan(mine, &total);
    for (int i = w0; i < w1; ++i)
        for (uint32_t m = sel[i]; m && at < (uint32_t)p.k; m &= m - 1) out[at++] = 32 * i + __ffs(m) - 1;
}

constexpr size_t kSelectFixed = kListMax * 12 + kBins * 4;
constexpr int kSmemMax = 200 * 1024;
constexpr int kMaxBlocks = 1 << 19;    // 128 KB of bitmaps

inline int padded(int max_blocks) { return (max_blocks + 15) / 16 * 16; }

template <typename T, int NT>
int launch_select(SelectParams p, int num_seqs, cudaStream_t stream) {
    const int words = (p.max_blocks + 31) / 32;
    const size_t fixed = kSelectFixed + (size_t)words * 8;
    // the row's scores in shared memory when they fit (read once from L2, then
    // three to five times)
    p.cached = fixed + (size_t)padded(p.max_blocks) * 4 <= kSmemMax ? padded(p.max_blocks) : 0;
    const size_t smem = fixed + (size_t)p.cached * 4;
    auto kern = select_rows<T, NT>;
    int occ = 0;
    const int st = kernel_setup(reinterpret_cast<const void*>(kern), kSmemMax, NT, &occ);
    if (st != PKV_OK) return st;
    note_launch();
    const cudaError_t e = launch_pdl(kern, dim3(p.hkv, num_seqs), dim3(NT), smem, stream, p);
    return e == cudaSuccess ? PKV_OK : cuda_fail("select_blocks: selection launch", e);
}

template <typename T>
int launch_scores(const SelectParams& p, int num_seqs, cudaStream_t stream) {
    const int tiles = padded(p.max_blocks) / 16;
    // 16-block tiles a warp walks: more once the warps fill the GPU's 16 resident
    // warps per SM several times over
    int per = 1;
    const long long rows = (long long)num_seqs * p.hkv, fill = 64LL * num_sms();
    while (per < 8 && rows * tiles / (2 * per) >= fill) per *= 2;
    dim3 grid((tiles + 4 * per - 1) / (4 * per), p.hkv, num_seqs);
    note_launch();
    cudaError_t e;
    if constexpr (std::is_same<T, float>::value)
        e = p.d == 64 ? launch_pdl(score_blocks_f32<64>, grid, dim3(128), 0, stream, p, per)
                      : launch_pdl(score_blocks_f32<128>, grid, dim3(128), 0, stream, p, per);
    else
        e = p.d == 64 ? launch_pdl(score_blocks_bf16<64>, grid, dim3(128), 0, stream, p, per)
                      : launch_pdl(score_blocks_bf16<128>, grid, dim3(128), 0, stream, p, per);
    return e == cudaSuccess ? PKV_OK : cuda_fail("select_blocks: scoring launch", e);
}

template <typename T>
int select_all(const SelectParams& p, int num_seqs, cudaStream_t stream) {
    if (p.max_blocks > p.k && p.k > p.first + p.last) {
        const int st = launch_scores<T>(p, num_seqs, stream);
        if (st != PKV_OK) return st;
    }
    if (p.max_blocks > 4096) return launch_select<T, 1024>(p, num_seqs, stream);
    return launch_select<T, 256>(p, num_seqs, stream);
}

}  // namespace
}  // namespace pkv

extern "C" {

int update_key_bounds(const void* k_pool, void* key_bounds, const int32_t* block_tables,
                      const int32_t* seq_lens, const int32_t* first_changed, int num_seqs,
                      int max_blocks_per_seq, int num_blocks, int num_kv_heads, int head_dim,
                      int block_size, int max_new_tokens, int kv_dtype, void* stream) {
    using namespace pkv;
    if (num_seqs < 0 || num_seqs > 65535 || max_blocks_per_seq <= 0 || num_blocks <= 0 ||
        num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_new_tokens < 0 ||
        max_blocks_per_seq > 0x7fffffff / block_size)
        return PKV_ERR_INVALID_ARG;
    if (head_dim % 16 != 0 || block_size % 16 != 0) return PKV_ERR_UNSUPPORTED;
    if (kv_dtype != PKV_F32 && kv_dtype != PKV_BF16 && kv_dtype != PKV_E4M3) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!k_pool || !key_bounds || !block_tables || !seq_lens || !first_changed || !aligned16(k_pool) ||
        !aligned16(key_bounds))
        return PKV_ERR_INVALID_ARG;
    int* err = error_word();
    if (!err) return PKV_ERR_CUDA;
    // changed blocks of a sequence (at most one more than the new tokens fill); the
    // kernel strides, so a wrong hint costs time only
    long long blocks = max_new_tokens > 0 ? (max_new_tokens - 1LL + block_size - 1) / block_size + 1
                                          : max_blocks_per_seq;
    if (blocks > max_blocks_per_seq) blocks = max_blocks_per_seq;
    long long gx = (blocks * num_kv_heads + 3) / 4;
    const long long cap = 64LL * num_sms() / num_seqs + 1;  // 4 waves of 16 CTAs per SM
    if (gx > cap) gx = cap;
    auto kern = kv_dtype == PKV_F32    ? update_key_bounds_kernel<float>
                : kv_dtype == PKV_BF16 ? update_key_bounds_kernel<__nv_bfloat16>
                                       : update_key_bounds_kernel<uint8_t>;
    note_launch();
    const cudaError_t e =
        launch_pdl(kern, dim3((unsigned)gx, num_seqs), dim3(128), 0, static_cast<cudaStream_t>(stream),
                   static_cast<const uint4*>(k_pool), key_bounds, block_tables, seq_lens, first_changed,
                   max_blocks_per_seq, num_blocks, num_kv_heads, head_dim, block_size, err);
    return e == cudaSuccess ? PKV_OK : cuda_fail("update_key_bounds: kernel launch", e);
}

size_t select_blocks_workspace_size(int num_seqs, int num_kv_heads, int max_blocks_per_seq) {
    if (num_seqs <= 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0) return 0;
    const size_t rows = (size_t)num_seqs * num_kv_heads, stride = pkv::padded(max_blocks_per_seq);
    return rows * stride * (8 + 4) + rows * (stride / 16) * 4;
}

int select_blocks(int32_t* selected, const void* q, const void* key_bounds,
                  const int32_t* block_tables, const int32_t* seq_lens, int num_seqs,
                  int max_blocks_per_seq, int num_blocks, int num_heads, int num_kv_heads,
                  int head_dim, int block_size, int num_selected, int first_blocks, int last_blocks,
                  int q_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace pkv;
    if (num_seqs < 0 || num_seqs > 65535 || max_blocks_per_seq <= 0 || num_blocks <= 0 ||
        num_heads <= 0 || num_kv_heads <= 0 || num_kv_heads > 65535 || head_dim <= 0 ||
        block_size <= 0 || num_selected <= 0 || first_blocks < 0 || last_blocks < 0 ||
        (long long)first_blocks + last_blocks > num_selected || num_heads % num_kv_heads != 0 ||
        max_blocks_per_seq > 0x7fffffff / block_size)
        return PKV_ERR_INVALID_ARG;
    const int G = num_heads / num_kv_heads;
    if ((head_dim != 64 && head_dim != 128) || G > 8 || max_blocks_per_seq > kMaxBlocks)
        return PKV_ERR_UNSUPPORTED;
    if (q_dtype != PKV_F32 && q_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!selected || !q || !key_bounds || !block_tables || !seq_lens || !aligned16(q) ||
        !aligned16(key_bounds))
        return PKV_ERR_INVALID_ARG;
    const bool scored = max_blocks_per_seq > num_selected && num_selected > first_blocks + last_blocks;
    if (scored && (!workspace || !aligned16(workspace) ||
                   workspace_bytes < select_blocks_workspace_size(num_seqs, num_kv_heads, max_blocks_per_seq)))
        return PKV_ERR_INVALID_ARG;
    SelectParams p{};
    p.selected = selected;
    p.q = q;
    p.bounds = key_bounds;
    p.tables = block_tables;
    p.lens = seq_lens;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.hq = num_heads;
    p.hkv = num_kv_heads;
    p.d = head_dim;
    p.bs = block_size;
    p.k = num_selected;
    p.first = first_blocks;
    p.last = last_blocks;
    p.stride = padded(max_blocks_per_seq);
    const size_t rows = (size_t)num_seqs * num_kv_heads;
    if (scored) {
        p.exact = static_cast<unsigned long long*>(workspace);
        p.scores = reinterpret_cast<float*>(p.exact + rows * p.stride);
        p.tile_max = p.scores + rows * p.stride;
    }
    p.err = error_word();
    if (!p.err) return PKV_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return q_dtype == PKV_F32 ? select_all<float>(p, num_seqs, s)
                              : select_all<__nv_bfloat16>(p, num_seqs, s);
}

}  // extern "C"
