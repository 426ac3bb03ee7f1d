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
// left are those few scored again, as 64-bit whole numbers of 2^-51 of the row's largest
// magnitudes, and ranked, equal scores by the lower index. Where terms had more bits
// than that and scores lie within their roundings of the last place, those blocks'
// scores are compared as whole numbers of 1024 bits. (What the look at the last place
// costs rows that need no more: 4 rows of 63 blocks 4.96 -> 5.2 us, 8 of 8,192 13.5 -> 14.0.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cmath>
#include <type_traits>

#include "pkv_check.cuh"
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
// Bound: HBM bytes of the changed blocks' K (8 sequences of 16384 new tokens, 8 bf16
// heads of 128: 54 us, 0.82 of the copy rate; 2048 new tokens: 9.6, float32 15.7); a
// decode step is a chain of loads (length, table, tile): 64 sequences of 40 heads 3.3 us,
// one sequence 1.9.
template <typename KV>
__global__ void __launch_bounds__(128, 5) update_key_bounds_kernel(
    const uint4* __restrict__ k_pool, void* __restrict__ bounds, const int32_t* __restrict__ tables,
    const int32_t* __restrict__ lens, const int32_t* __restrict__ first, int max_blocks,
    int num_blocks, int hkv, int d, int bs, int* err) {
    pdl_enter();                                           // launched with launch_pdl
    using C = Cmp<KV>;
    constexpr int R = C::kRegs, QB = R == 8 ? 2 : 4;       // chunks of 4 planes read together
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
    const int changed = nblk - j0;
    const int planes = d * C::kElt / 16;                   // 16-byte chunks per token
    const int tl = lane & 7, pl = lane >> 3;               // token and chunk of the load
    // item (changed block i, kv head h), heads fastest; the next one's id is read ahead
    const unsigned heads = (unsigned)hkv, start = blockIdx.x * 4u + (threadIdx.x >> 5), step = gridDim.x * 4u;
    const int step_i = (int)(step / heads), step_h = (int)(step % heads);
    int i = (int)(start / heads), h = (int)(start % heads);
    auto id_at = [&](int x) { return x < changed ? tables[(size_t)b * max_blocks + j0 + x] : -1; };
    int id_next = id_at(i);
    while (i < changed) {
        const int id = id_next, j = j0 + i, hc = h;
        i += step_i;
        h += step_h;
        if (h >= hkv) h -= hkv, ++i;
        id_next = id_at(i);
        if (id < 0 || id >= num_blocks) {
            if (lane == 0 && hc == 0) flag_error(err, kErrOutOfRange);
            continue;
        }
        const int ntok = min(bs, L - j * bs);
        const uint4* tile = k_pool + ((size_t)id * hkv + hc) * planes * bs;
        char* out = static_cast<char*>(bounds) +
                    ((size_t)id * hkv + hc) * 2 * d * (C::kElt == 4 ? 4 : 2);
        for (int q0 = 0; q0 < planes; q0 += 4 * QB) {
            uint32_t x[QB][2 * R];                         // min | max
#pragma unroll
            for (int u = 0; u < QB; ++u)
#pragma unroll
                for (int i = 0; i < R; ++i) x[u][i] = C::kInf, x[u][R + i] = C::kNegInf;
            for (int g0 = 0; g0 * 8 < ntok; g0 += 2) {
                uint4 raw[2][QB];                          // read together
                bool ok[2][QB];
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int u = 0; u < QB; ++u) {
                        const int plane = q0 + 4 * u + pl;
                        ok[g][u] = plane < planes && (g0 + g) * 8 + tl < ntok;
                        if (ok[g][u]) raw[g][u] = tile[((g0 + g) * planes + plane) * 8 + tl];
                    }
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int u = 0; u < QB; ++u)
                        if (ok[g][u]) {
                            uint32_t v[R];
                            widen<KV>(raw[g][u], v);
#pragma unroll
                            for (int i = 0; i < R; ++i) {
                                x[u][i] = min2(x[u][i], v[i], typename C::T{});
                                x[u][R + i] = max2(x[u][R + i], v[i], typename C::T{});
                            }
                        }
            }
            // step 1 (tokens t, t^4): the lower lane keeps the minima, the upper
            // the maxima; steps 2 and 3 halve what is left
            const bool up = (tl & 4) != 0;
#pragma unroll
            for (int u = 0; u < QB; ++u) {
                uint32_t y[R];
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const uint32_t other = __shfl_xor_sync(kFull, up ? x[u][i] : x[u][R + i], 4);
                    y[i] = up ? max2(x[u][R + i], other, typename C::T{}) : min2(x[u][i], other, typename C::T{});
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
                const int plane = q0 + 4 * u + pl;
                if (plane >= planes) continue;
                // lane tl holds registers (tl & 3) * R/4 .. of the chunk's minima or maxima
                if constexpr (std::is_same<KV, uint8_t>::value) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&y[i]));
                        const __nv_bfloat162 z = __floats2bfloat162_rn(v.x, v.y);   // exact
                        y[i] = *reinterpret_cast<const uint32_t*>(&z);
                    }
                    *reinterpret_cast<uint2*>(out + (up ? 2 * d : 0) + plane * 32 + (tl & 3) * 8) =
                        make_uint2(y[0], y[1]);
                } else {
                    *reinterpret_cast<uint32_t*>(out + (up ? d * C::kElt : 0) + plane * 16 + (tl & 3) * 4) = y[0];
                }
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
    int stride, scored;                // scored: behind a scoring launch of the same call
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

// Scores of 16 blocks of a kv head per warp and stage. A CTA takes `side` neighbouring
// kv heads of (4 / side) x 16 blocks at a time, so a block's rows of those heads are
// one contiguous copy (side * 4 D bytes) into a stage of a shared-memory ring, two
// stages deep (66 KB of copies in flight per CTA, three CTAs an SM); rows lie 16 bytes
// apart from a multiple of 128 so that the operand reads (ldmatrix) meet no bank
// twice. Four accumulator chains shorten the dependency and the rounding.
// Bound: HBM bytes of the bounds (32 ragged sequences of up to 2048 blocks, 8 heads: 139 MB
// in about 25 us, 0.82 of the copy rate); a short stream, its ramp (33 MB in 7.5).
constexpr int kScoreStages = 2;
constexpr int kStageRows = 64;         // rows of 16-bit [2][D], of all warps

template <int D>
struct ScoreSmem {
    static constexpr int kRow = 4 * D;                     // bytes of one head's bounds
    static constexpr int kStage = kStageRows * (kRow + 16);
    static constexpr int kBytes = kScoreStages * kStage;
};

template <int D>
__global__ void __launch_bounds__(128) score_blocks_bf16(const SelectParams p, int per, int side) {
    pdl_enter();                                           // launched with launch_pdl
    using S = ScoreSmem<D>;
    constexpr int KS = D / 16;                             // k-steps of one bound
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(8) uint64_t bars[kScoreStages];
    __shared__ int ids[kScoreStages][kStageRows];
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, b = blockIdx.z;
    const int r = lane >> 2, c = lane & 3, G = p.hq / p.hkv;
    const int h0 = blockIdx.y * side, h = h0 + w % side;   // the CTA's first kv head, this warp's
    const int blocks = kStageRows / side;                  // blocks of a stage
    const int pitch = side * S::kRow + 16;
    const int first = blockIdx.x * per;                    // stages first .. first + per - 1 of the row
    // the table and the query are read beside the length: entries past it are in the
    // table, and unused
    auto table_at = [&](int stage) {
        const int j = stage * blocks + tid;
        return tid < blocks && j < p.max_blocks ? p.tables[(size_t)b * p.max_blocks + j] : -1;
    };
    int next[kScoreStages];
#pragma unroll
    for (int s = 0; s < kScoreStages; ++s) next[s] = s < per ? table_at(first + s) : -1;
    uint32_t qn[KS][2], qp[KS][2];                         // min(q, 0), max(q, 0)
    {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                              ((size_t)b * p.hq + h * G + r) * D);
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) qp[i][j] = r < G ? __ldg(q + 8 * i + 4 * j + c) : 0u;
    }
    const int n = row_blocks(p, b, false);
    if (n <= p.k) return;                                  // every block is selected
    const int lo = p.first, hi = n - p.last;               // blocks with a score: [lo, hi)
    const int count = min(per, (hi + blocks - 1) / blocks - first);
    if (count <= 0) return;
    if (tid < kScoreStages) mbar_init(smem_addr(&bars[tid]), 2);
    fence_mbar_init();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            qn[i][j] = min2(qp[i][j], 0u, __nv_bfloat16{});
            qp[i][j] = max2(qp[i][j], 0u, __nv_bfloat16{});
        }
    const char* src = static_cast<const char*>(p.bounds) + (size_t)h0 * S::kRow;
    const size_t block_bytes = (size_t)p.hkv * S::kRow;
    // warps 0 and 1, a lane a block: its rows into slot s
    auto issue = [&](int stage, int s, int id) {
        if (w >= 2) return;
        const int j = stage * blocks + tid;
        if (tid >= blocks || j < lo || j >= hi) {
            id = -1;
        } else if (id < 0 || id >= p.num_blocks) {
            flag_error(p.err, kErrOutOfRange);
            id = -1;
        }
        ids[s][tid] = id;
        const unsigned live = __ballot_sync(kFull, id >= 0);
        const uint32_t bar = smem_addr(&bars[s]);
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(live) * side * S::kRow);
        __syncwarp();
        if (id >= 0)
            bulk_g2s(smem_addr(smem + s * S::kStage + tid * pitch), src + id * block_bytes, side * S::kRow, bar,
                     l2_evict_first());
    };
#pragma unroll
    for (int s = 0; s < kScoreStages; ++s)
        if (s < count) issue(first + s, s, next[s]);
    int id_next = count > kScoreStages ? table_at(first + kScoreStages) : -1;
    const size_t row = (size_t)b * p.hkv + h;
    const int tile0 = (w / side) * 16;                     // this warp's blocks within a stage
    int s = 0;
    uint32_t phase = 0;
    for (int k = 0; k < count; ++k) {
        const bool ok = mbar_wait_bounded(smem_addr(&bars[s]), phase, p.err);
        if (__syncthreads_or(!ok)) {
            // gave up: record it, let the copies in flight land, leave
            if (tid == 0) flag_error(p.err, kErrTimeout);
            for (int kk = k; kk < min(count, k + kScoreStages); ++kk) {
                (void)mbar_wait_bounded(smem_addr(&bars[s]), phase, nullptr);
                if (++s == kScoreStages) s = 0, phase ^= 1;
            }
            return;
        }
        const uint32_t base = smem_addr(smem + s * S::kStage + tile0 * pitch + (w % side) * S::kRow) +
                              (lane & 15) * pitch + (lane >> 4) * 16;
        const bool ok0 = ids[s][tile0 + r] >= 0, ok1 = ids[s][tile0 + r + 8] >= 0;
        float acc[4][4];
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[a][e] = 0.f;
        uint32_t m0 = 0, m1 = 0;                           // largest |bound| of blocks r and r+8
#pragma unroll
        for (int i = 0; i < 2 * KS; ++i) {
            uint32_t a0, a1, a2, a3;                       // rows r, r+8; dims 16i + 2c, + 8
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                         : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3)
                         : "r"(base + i * 32)
                         : "memory");
            const uint32_t(&q)[2] = i < KS ? qn[i < KS ? i : 0] : qp[i < KS ? 0 : i - KS];
            mma_bf16(acc[i & 3], a0, a1, a2, a3, q[0], q[1]);
            m0 = abs_max2(abs_max2(m0, a0), a2);
            m1 = abs_max2(abs_max2(m1, a1), a3);
        }
        __syncthreads();                                   // the slot is free
        if (k + kScoreStages < count) {
            fence_proxy_async_smem();
            issue(first + k + kScoreStages, s, id_next);
            id_next = k + 1 + kScoreStages < count ? table_at(first + k + 1 + kScoreStages) : -1;
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
        const int j0 = (first + k) * blocks + tile0;
        float* out = p.scores + row * p.stride + j0;
        if (c == 0 && j0 < p.stride) {
            out[r] = ok0 ? s0 + 0.f : -INFINITY;           // + 0: no negative zero
            out[r + 8] = ok1 ? s1 + 0.f : -INFINITY;
        }
        // bf16 magnitudes order as their bits, NaN on top
        m0 = ok0 ? m0 & 0x7fff7fffu : 0u;
        m1 = ok1 ? m1 & 0x7fff7fffu : 0u;
        const uint32_t mm = __reduce_max_sync(kFull, max(max(m0 & 0xffffu, m0 >> 16), max(m1 & 0xffffu, m1 >> 16)));
        if (lane == 0 && j0 < p.stride) p.tile_max[row * (p.stride / 16) + j0 / 16] = __uint_as_float(mm << 16);
        if (++s == kScoreStages) {
            s = 0;
            phase ^= 1;
        }
    }
}

// float32 bounds and queries (tensor cores would round them): a warp takes eight blocks
// at a time, lane l the dims l, l + 32, ..., and the eight sums of a head are reduced
// across the lanes together, ending with one block to four lanes. Two warps share a tile
// of 16. (4 heads, 8 rows of 4,096 blocks of 128 dims: 25.6 us with one block at a time and a
// reduction a head, 14.6 so; 256 rows of 2,048: 91 and 68.)
template <int D>
__global__ void __launch_bounds__(128) score_blocks_f32(const SelectParams p, int tiles_per_pair) {
    pdl_enter();                                           // launched with launch_pdl
    const int h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31;
    const int n = row_blocks(p, b, false);
    if (n <= p.k) return;
    const int lo = p.first, hi = n - p.last;
    const int w = threadIdx.x >> 5, half = w & 1, tile0 = blockIdx.x * 2 * tiles_per_pair;
    if (tile0 * 16 >= hi) return;
    constexpr int I = D / 32;
    const int G = p.hq / p.hkv;
    __shared__ float qn[8][D], qp[8][D];                   // min(q, 0), max(q, 0)
    __shared__ float top[2][4];                            // the warps' largest |bound|
    for (int i = threadIdx.x; i < G * D; i += 128) {
        const float q = static_cast<const float*>(p.q)[((size_t)b * p.hq + h * G) * D + i];
        qn[i / D][i % D] = min_nan(q, 0.f);
        qp[i / D][i % D] = max_nan(q, 0.f);
    }
    __syncthreads();
    const size_t row = (size_t)b * p.hkv + h;
    for (int it = 0; it < tiles_per_pair; ++it) {
        const int tile = tile0 + 2 * it + (w >> 1);
        const int jl = tile * 16 + 8 * half + (lane & 7);
        int ids = jl >= lo && jl < hi ? p.tables[(size_t)b * p.max_blocks + jl] : -1;
        if (jl >= lo && jl < hi && (ids < 0 || ids >= p.num_blocks)) {
            flag_error(p.err, kErrOutOfRange);
            ids = -1;
        }
        float mf = 0.f;
        if (__any_sync(kFull, ids >= 0)) {
            float l[8][I], u[8][I];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int id = __shfl_sync(kFull, ids, k);
                const float* src = static_cast<const float*>(p.bounds) + ((size_t)max(id, 0) * p.hkv + h) * 2 * D + lane;
#pragma unroll
                for (int i = 0; i < I; ++i) {
                    l[k][i] = id >= 0 ? __ldg(src + 32 * i) : 0.f;
                    u[k][i] = id >= 0 ? __ldg(src + D + 32 * i) : 0.f;
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int i = 0; i < I; ++i) mf = max_nan(mf, max_nan(fabsf(l[k][i]), fabsf(u[k][i])));
            float best = -INFINITY;                        // of block lane / 4
#pragma unroll 1
            for (int g = 0; g < G; ++g) {
                float s[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) s[k] = 0.f;
#pragma unroll
                for (int i = 0; i < I; ++i) {
                    const float n = qn[g][lane + 32 * i], q = qp[g][lane + 32 * i];
#pragma unroll
                    for (int k = 0; k < 8; ++k) s[k] = fmaf(q, u[k][i], fmaf(n, l[k][i], s[k]));
                }
                // eight sums over the lanes at once: each step hands half of them over
#pragma unroll
                for (int o = 16, m = 4; m >= 1; o >>= 1, m >>= 1)
#pragma unroll
                    for (int k = 0; k < m; ++k) {
                        const float mine = lane & o ? s[k + m] : s[k], other = lane & o ? s[k] : s[k + m];
                        s[k] = mine + __shfl_xor_sync(kFull, other, o);
                    }
                s[0] += __shfl_xor_sync(kFull, s[0], 2);
                s[0] += __shfl_xor_sync(kFull, s[0], 1);
                best = max_nan(best, s[0]);
            }
            const int j = tile * 16 + 8 * half + (lane >> 2), id = __shfl_sync(kFull, ids, lane >> 2);
            if ((lane & 3) == 0 && j >= lo && j < hi) p.scores[row * p.stride + j] = id >= 0 ? best + 0.f : -INFINITY;
        } else if (lane < 8 && jl >= lo && jl < hi) {
            p.scores[row * p.stride + jl] = -INFINITY;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mf = max_nan(mf, __shfl_xor_sync(kFull, mf, o));
        if (lane == 0) top[it & 1][w] = mf;
        __syncthreads();
        if (half == 0 && lane == 0 && tile * 16 < hi)
            p.tile_max[row * (p.stride / 16) + tile] = max_nan(top[it & 1][w], top[it & 1][w + 1]);
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

// 2^(127 - e) for the biased exponent e of a finite float: brings it into [1, 2)
// (below 1 if it is subnormal).
__device__ __forceinline__ float unit_scale(float x) {
    const int e = max((int)(__float_as_uint(x) >> 23), 1);
    return __uint_as_float(e < 254 ? (uint32_t)(254 - e) << 23 : 0x00400000u);
}

// What a term leaves of itself in three exact float32 sums: x is cut at 2^-19, the
// rest at 2^-35, the rest of that at 2^-51 (adding and subtracting 1.5 x 2^23 units
// rounds to the unit). With sums of magnitudes below 4 every sum is a whole number
// of its unit below 2^24, so it is exact in any order. Returns what is left.
__device__ __forceinline__ float add_exact(float (&s)[3], float x) {
    const float a = __fadd_rn(__fadd_rn(x, 24.f), -24.f);
    s[0] = __fadd_rn(s[0], a);
    x = __fadd_rn(x, -a);
    const float b = __fadd_rn(__fadd_rn(x, 0x1.8p-12f), -0x1.8p-12f);
    s[1] = __fadd_rn(s[1], b);
    x = __fadd_rn(x, -b);
    const float c = __fadd_rn(__fadd_rn(x, 0x1.8p-28f), -0x1.8p-28f);
    s[2] = __fadd_rn(s[2], c);
    return __fadd_rn(x, -c);
}

// The score of a block (row `id_row` of the bounds) under the heads of `heads` (rows
// of `qs`, float32 in shared memory) in 64 bits, as an ordered key above 0 (the
// whole warp). The query times scale_q and the bounds times scale_b make a score's
// magnitudes sum to less than 4; its terms, exact products (float32 inputs: with
// the rest of the product), are summed exactly down to 2^-51; MORE: *vague is set where one has
// bits below that. (In float64, at two multiply-adds a clock per SM, a block with 8 heads
// took 3 us. Looking for lower bits costs a choice of 64 blocks 0.3 us, float32 0.8, so it
// is left until keys lie too close to tell without.)
template <typename T, bool MORE>
__device__ __forceinline__ unsigned long long exact_key(const T* bounds, size_t id_row, int d, const float* qs,
                                                        unsigned heads, int lane, float scale_q, float scale_b,
                                                        int* vague) {
    const T* bl = bounds + id_row * 2 * d + lane;
    float lo[4], hi[4];                                     // d is 64 or 128
    bool more = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float l = 32 * i < d ? (float)bl[32 * i] : 0.f, u = 32 * i < d ? (float)bl[d + 32 * i] : 0.f;
        lo[i] = l * scale_b;
        hi[i] = u * scale_b;
        if constexpr (MORE) more |= (lo[i] == 0.f && l != 0.f) || (hi[i] == 0.f && u != 0.f);
    }
    unsigned long long best = 0;
    for (; heads; heads &= heads - 1) {
        const int g = __ffs(heads) - 1;
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (32 * i >= d) break;
            const float q = qs[g * d + lane + 32 * i], u = q * scale_q;
            const float x = u < 0.f ? lo[i] : hi[i];
            const float t = __fmul_rn(u, x);
            float rest = add_exact(s, t);
            if constexpr (std::is_same<T, float>::value) rest = fabsf(rest) + fabsf(add_exact(s, __fmaf_rn(u, x, -t)));
            // what float32's range cuts off leaves something, unless it leaves nothing at all
            if constexpr (MORE) more |= rest != 0.f || (t == 0.f && q != 0.f && x != 0.f);
        }
        const long long i0 = __reduce_add_sync(kFull, (int)(s[0] * 0x1p19f));
        const long long i1 = __reduce_add_sync(kFull, (int)(s[1] * 0x1p35f));
        const long long i2 = __reduce_add_sync(kFull, (int)(s[2] * 0x1p51f));
        const long long sum = i0 * (1ll << 32) + i1 * (1ll << 16) + i2;
        best = max(best, (unsigned long long)sum ^ (1ull << 63));
    }
    if constexpr (MORE)
        if (__any_sync(kFull, more) && lane == 0) *vague = 1;
    return best;
}

// How far a key of terms with lower bits can be off: half a unit a term (float32: two terms
// a product), and one for what float32's range cut off.
template <typename T>
__device__ __forceinline__ unsigned long long key_error(int d) {
    return (std::is_same<T, float>::value ? d : d / 2) + 1;
}

// Whether a block's score is not finite, in rows with values that are not: some head's
// is NaN or +infinity, or none is finite. Heads of finite queries are finite on all other
// blocks. In float64, whose range no sum of these products leaves.
template <typename T>
__device__ __noinline__ bool score_not_finite(const T* bounds, size_t id_row, int d, const float* qs, int heads, int lane) {
    const T* bl = bounds + id_row * 2 * d;
    bool top = false, some = false;
    for (int g = 0; g < heads; ++g) {
        double s = 0.0;
        for (int i = lane; i < d; i += 32) {
            const double q = (double)qs[g * d + i];
            const double neg = q > 0.0 ? 0.0 : q, pos = q < 0.0 ? 0.0 : q;   // NaN stays
            s = fma(neg, (double)(float)bl[i], s);
            s = fma(pos, (double)(float)bl[d + i], s);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
        top |= !(s < INFINITY);
        some |= fabs(s) < INFINITY;
    }
    return top || !some;
}

// m 2^(e) for a finite float, m below 2^24
__device__ __forceinline__ void take_apart(float x, uint32_t& m, int& e) {
    const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
    const int field = (int)(u >> 23);
    m = (u & 0x7fffffu) | (field ? 0x800000u : 0u);
    e = max(field, 1) - 150;
}

// A finite block's score with every bit: a whole number of 2^-320 in two's complement,
// lane l of the warp holding bits 32 l .. 32 l + 31 (the top one biased, so that the
// lanes' words compare as unsigned from the highest down). A product of two floats is
// below 2^48 times 2^-298 to 2^208, so a sum fits with room to spare.
template <typename T>
__device__ __forceinline__ uint32_t score_word(const T* bounds, size_t id_row, int d, const float* qs, unsigned heads,
                                               int lane) {
    const T* bl = bounds + id_row * 2 * d;
    uint32_t best = 0;                                     // below every number
#pragma unroll 1
    for (; heads; heads &= heads - 1) {
        const float* qr = qs + (__ffs(heads) - 1) * d;
        long long sum = 0;                                 // of the terms' words here: 128 of them
#pragma unroll 1
        for (int i = lane; i < d; i += 32) {
            const float q = qr[i], x = (float)bl[q < 0.f ? i : d + i];
            uint32_t mq, mx;
            int eq, ex;
            take_apart(q, mq, eq);
            take_apart(x, mx, ex);
            const unsigned long long m = (unsigned long long)mq * mx;
            const int at = (eq + ex + 320) | ((__float_as_uint(q) ^ __float_as_uint(x)) & 0x80000000u ? 1 << 16 : 0);
#pragma unroll 8
            for (int j = 0; j < 32; ++j) {
                const unsigned long long mj = __shfl_sync(kFull, m, j);
                const int a = __shfl_sync(kFull, at, j), k = lane - ((a & 0xffff) >> 5), bit = a & 31;
                uint32_t word = 0;
                if (k == 0) word = (uint32_t)(mj << bit);
                if (k == 1) word = (uint32_t)(mj >> (32 - bit));
                if (k == 2 && bit > 0) word = (uint32_t)(mj >> (64 - bit));
                sum += a >> 16 ? -(long long)word : (long long)word;
            }
        }
        uint32_t word = 0;
        long long carry = 0;
#pragma unroll 1
        for (int j = 0; j < 32; ++j) {
            const long long v = __shfl_sync(kFull, sum, j) + carry;
            if (lane == j) word = (uint32_t)v;
            carry = v >> 32;
        }
        if (lane == 31) word ^= 0x80000000u;
        if (__ballot_sync(kFull, word > best) > __ballot_sync(kFull, word < best)) best = word;
    }
    return best;
}

// The `left` blocks of the highest scores among those of `cand`, equal ones by the lower
// index, into `sel` (bitmaps; the whole CTA). Each round compares every candidate with one
// of them, exactly, and keeps those above or those below it; the round's one lies in the
// middle of the candidates by index first, then at changing places. `mark`: a word per
// block for the comparisons' results. Rare, and out of the way of the code that is not.
template <typename T, int NT>
__device__ __forceinline__ void settle(const T* bounds, const int32_t* table, int hkv, int h, int d, const float* qs,
                                    unsigned heads, int lo, int hi, int left, unsigned char* sel, unsigned char* cand,
                                    unsigned long long* mark) {
    constexpr int NW = NT / 32;
    __shared__ uint32_t pivot[32], part[NW];
    __shared__ int where;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, c0 = lo / 8, c1 = (hi + 7) / 8;
    auto total = [&](uint32_t v) -> int {
        v = __reduce_add_sync(kFull, v);
        __syncthreads();
        if (lane == 0) part[w] = v;
        __syncthreads();
        return (int)__reduce_add_sync(kFull, lane < NW ? part[lane] : 0u);
    };
    // exclusive prefix over the threads
    auto under = [&](uint32_t v) -> int {
        uint32_t incl = v;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += t;
        }
        __syncthreads();
        if (lane == 31) part[w] = incl;
        __syncthreads();
        return (int)(__reduce_add_sync(kFull, lane < w ? part[lane] : 0u) + incl - v);
    };
    const int per = (c1 - c0 + NT - 1) / NT;               // bytes of the bitmaps a thread owns, in order
    const int b0 = min(c1, c0 + tid * per), b1 = min(c1, b0 + per);
    for (uint32_t round = 0; left > 0; ++round) {
        __syncthreads();
        uint32_t mine = 0;
        for (int c = b0; c < b1; ++c) mine += __popc(cand[c]);
        const int count = total(mine);
        if (count <= left) {
            for (int c = b0; c < b1; ++c) sel[c] |= cand[c];
            break;
        }
        // the candidate to compare with
        const int rank = (int)(((unsigned long long)(round * 0x9e3779b9u + 0x80000000u) * (uint32_t)count) >> 32);
        int at = under(mine);
        for (int c = b0; c < b1; ++c)
            for (uint32_t m = cand[c]; m; m &= m - 1, ++at)
                if (at == rank) where = 8 * c + __ffs(m) - 1;
        __syncthreads();
        // blocks of the same bounds (mark 1) need no score
        const size_t pivot_row = (size_t)table[where] * hkv + h;
        bool differ = false;
        for (int blk = 8 * c0 + w; blk < 8 * c1; blk += NW)
            if ((cand[blk >> 3] >> (blk & 7)) & 1) {
                const T *x = bounds + pivot_row * 2 * d, *y = bounds + ((size_t)table[blk] * hkv + h) * 2 * d;
                bool same = true;
                for (int i = lane; i < 2 * d; i += 32) same &= (float)x[i] == (float)y[i];
                same = __all_sync(kFull, same);
                differ |= !same;
                if (lane == 0) mark[blk] = same ? 1 : 3;
            }
        if (__syncthreads_or(differ) && w == 0) pivot[lane] = score_word(bounds, pivot_row, d, qs, heads, lane);
        __syncthreads();
        for (int blk = 8 * c0 + w; blk < 8 * c1; blk += NW)
            if (((cand[blk >> 3] >> (blk & 7)) & 1) && mark[blk] == 3) {
                const uint32_t x = score_word(bounds, (size_t)table[blk] * hkv + h, d, qs, heads, lane), y = pivot[lane];
                const unsigned up = __ballot_sync(kFull, x > y), dn = __ballot_sync(kFull, x < y);
                __syncwarp();
                if (lane == 0) mark[blk] = up > dn ? 2 : up < dn ? 0 : 1;
            }
        __syncthreads();
        uint32_t more = 0, same = 0;
        for (int c = b0; c < b1; ++c)
            for (uint32_t m = cand[c]; m; m &= m - 1) {
                const int r = (int)mark[8 * c + __ffs(m) - 1];
                more += r == 2;
                same += r == 1;
            }
        const int above = total(more), equal = total(same);
        int rest = left - above, first = under(same);      // places for the equal ones; how many lie before
        for (int c = b0; c < b1; ++c) {
            uint32_t in = 0, keep = 0;
            for (uint32_t m = cand[c]; m; m &= m - 1) {
                const uint32_t bit = m & -m;
                const int r = (int)mark[8 * c + __ffs(m) - 1];
                if (above >= left) keep |= r == 2 ? bit : 0u;
                else if (r == 2 || (r == 1 && first++ < rest)) in |= bit;
                else if (r == 0) keep |= bit;
            }
            sel[c] |= in;
            cand[c] = above + equal >= left && above < left ? 0 : keep;
        }
        if (above < left) left = max(0, rest - equal);
    }
    __syncthreads();
}

constexpr int kBins = 1024;
constexpr int kListMax = 512;         // blocks ranked in shared memory
constexpr int kMaxRounds = 8;         // to a lower bound of the last place's score

// Scores of a row's blocks by one CTA, into shared memory (`out`, and the tiles'
// largest |bound|): 16 blocks per warp at a time, read straight into the operand
// fragments. The k order of the product is free as long as both operands agree on it,
// so lane (r, c) loads 16 bytes of blocks r and r+8 at dims 32i + 8c .. +7 into the A
// fragments of k-steps 2i and 2i+1, and the same dims of query head r into the B
// fragments. Four accumulator chains, as above.
template <int D, int NW>
__device__ __forceinline__ void score_row(const SelectParams& p, int b, int h, int lo, int hi, float* out,
                                          float* tile_max) {
    constexpr int I = D / 32;                              // 16-byte chunks a lane holds per bound
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3, G = p.hq / p.hkv;
    auto table_at = [&](int tile) {
        const int j = tile * 16 + (lane & 15);
        return j >= lo && j < hi ? p.tables[(size_t)b * p.max_blocks + j] : -1;
    };
    int id_next = table_at(w);
    uint32_t qn[I][4], qp[I][4];                           // min(q, 0), max(q, 0)
#pragma unroll
    for (int i = 0; i < I; ++i) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < G)
            x = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                     ((size_t)b * p.hq + h * G + r) * D + 32 * i + 8 * c));
        const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            qn[i][j] = min2(v[j], 0u, __nv_bfloat16{});
            qp[i][j] = max2(v[j], 0u, __nv_bfloat16{});
        }
    }
    const uint4* base = reinterpret_cast<const uint4*>(p.bounds) + (size_t)h * (D / 4) + c;
    const size_t pitch = (size_t)p.hkv * (D / 4);          // 16-byte units of a block
#pragma unroll 1
    for (int tile = w; tile * 16 < hi; tile += NW) {
        int id = id_next;
        id_next = table_at(tile + NW);
        const int j = tile * 16 + (lane & 15);
        if (j >= lo && j < hi && (id < 0 || id >= p.num_blocks)) {
            flag_error(p.err, kErrOutOfRange);
            id = -1;
        }
        const int id0 = __shfl_sync(kFull, id, r), id1 = __shfl_sync(kFull, id, r + 8);
        const uint4 *p0 = base + max(id0, 0) * pitch, *p1 = base + max(id1, 0) * pitch;
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
            const uint32_t(&q)[4] = i < I ? qn[i < I ? i : 0] : qp[i < I ? 0 : i - I];
            mma_bf16(acc[i & 3], x0[i].x, x1[i].x, x0[i].y, x1[i].y, q[0], q[1]);
            mma_bf16(acc[i & 3], x0[i].z, x1[i].z, x0[i].w, x1[i].w, q[2], q[3]);
            m = abs_max2(abs_max2(m, x0[i].x), x0[i].y);
            m = abs_max2(abs_max2(m, x0[i].z), x0[i].w);
            m = abs_max2(abs_max2(m, x1[i].x), x1[i].y);
            m = abs_max2(abs_max2(m, x1[i].z), x1[i].w);
        }
        float s0 = -INFINITY, s1 = -INFINITY;              // heads 2c, 2c+1 of blocks r and r+8
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
        if (c == 0) {
            out[tile * 16 + r] = id0 >= 0 ? s0 + 0.f : -INFINITY;
            out[tile * 16 + r + 8] = id1 >= 0 ? s1 + 0.f : -INFINITY;
        }
        m &= 0x7fff7fffu;
        const uint32_t mm = __reduce_max_sync(kFull, max(m & 0xffffu, m >> 16));
        if (lane == 0) tile_max[tile] = __uint_as_float(mm << 16);
    }
}

// One CTA per (kv head, sequence) over the row's scores (FD: which it computes itself,
// head_dim FD). A thread owns chunks of 8 blocks (KEEP: one chunk, in registers). The
// score range is cut into 1,024 equal bins; the bin of the last place and its
// neighbours within the rounding window hold the few blocks that are undecided (the
// range is cut again when they are too many), which are ranked among themselves: by
// their float32 scores, those within the window of the last place by their 64-bit scores
// if there are more of them than places, and what those cannot tell by every bit. A bin of a score is a monotone function
// of it, so bins decide soundly whatever the rounding of their edges.
// Rows of no more blocks than threads have one to a thread.
// Bound: latency and, with 32 warps, issue: about 14,000 clocks of dependent steps for
// 8,192 blocks, of which loads 2,000, bins and their scan 3,500, scores in 64 bits 3,000, the
// look at the last place 900, writing 1,000; a row's scores are at most a few hundred KB,
// from L2.
template <typename T, int NT, bool KEEP, int FD = 0>
__global__ void __launch_bounds__(NT) select_rows(const SelectParams p) {
    constexpr int NW = NT / 32;
    // Launched behind this call's scoring kernel: lengths, tables and queries were
    // written before that launch began, its scores only when it has completed.
    if (p.scored) launch_dependents();
    else pdl_enter();
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const size_t row = (size_t)b * p.hkv + h;
    int32_t* out = p.selected + row * p.k;
    const int n = row_blocks(p, b, h == 0 && tid == 0);
    if (n <= p.k) {                                        // all of them
        if (p.scored) wait_prerequisites();
        for (int i = tid; i < p.k; i += NT) out[i] = i < n ? i : -1;
        return;
    }
    extern __shared__ __align__(16) unsigned char smem[];
    const int words_max = (p.max_blocks + 31) / 32;
    unsigned long long* list_key = reinterpret_cast<unsigned long long*>(smem);    // [kListMax]
    float* list_s = reinterpret_cast<float*>(list_key + kListMax);                 // [kListMax]
    int* list_id = reinterpret_cast<int*>(list_s + kListMax);                      // [kListMax]
    int* list_row = list_id + kListMax;                                            // [kListMax]
    float* qf = reinterpret_cast<float*>(list_row + kListMax);                     // [8][128]
    uint32_t* hist = reinterpret_cast<uint32_t*>(qf + 8 * 128);                    // [kBins]
    uint32_t* sel = hist + kBins;                                                  // selected blocks
    uint32_t* cand = sel + (words_max + 3) / 4 * 4;                                // a crowd
    float* own_scores = reinterpret_cast<float*>(cand + (words_max + 3) / 4 * 4);  // FD: [blocks, padded to 16]
    float* own_max = own_scores + (p.max_blocks + 15) / 16 * 16;                   // FD: [tiles]
    unsigned char* sel8 = reinterpret_cast<unsigned char*>(sel);
    unsigned char* cand8 = reinterpret_cast<unsigned char*>(cand);
    __shared__ uint32_t sh_a[NW], sh_b[NW], sh_c[NW], sh_q[NW], sh_m[NW];
    __shared__ int sh_bin, sh_cnt, sh_likely, sh_vague, sh_win[2];
    __shared__ float sh_thr;
    __shared__ unsigned long long sh_key[2];

    const int lo = p.first, hi = n - p.last;               // scored blocks
    const int need = p.k - p.first - p.last;               // 0 <= need < hi - lo
    const int chunks = (n + 7) / 8;
    // a chunk's blocks below n, and those of them that are scored
    auto below = [](int c, int end) -> uint32_t {
        const int m = end - 8 * c;
        return m >= 8 ? 0xffu : m <= 0 ? 0u : (1u << m) - 1u;
    };
    auto scored_of = [&](int c) { return below(c, hi) & ~below(c, lo); };
    auto forced_of = [&](int c) { return below(c, n) & ~scored_of(c); };
    // exclusive prefix over the threads, and the total
    auto block_scan = [&](uint32_t v, uint32_t* total) -> uint32_t {
        uint32_t incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += t;
        }
        __syncthreads();                                   // earlier readers of sh_a
        if (lane == 31) sh_a[w] = incl;
        __syncthreads();
        const uint32_t x = lane < NW ? sh_a[lane] : 0;
        const uint32_t under = __reduce_add_sync(kFull, lane < w ? x : 0u);
        *total = __reduce_add_sync(kFull, x);
        return under + incl - v;
    };

    if (need > 0) {
        // ---- how far a score can be off. A = max_g sum_d |q_gd| times the largest
        // |bound| of the row is at least the sum of the magnitudes of a score's
        // terms. bf16: products exact in float32; four chains of at most four
        // mma.sync, each aligning at most 17 terms to the largest and dropping
        // bits below its 24th (17 x 2^-23 of it) and rounding once, chains adding
        // up to A: D / 32 x 18 x 2^-23 A, and 3 x 2^-23 A for the last adds, A's own
        // rounding and the window's. float32: at most 2 D / 32 + 6 roundings of 2^-24.
        const int G = p.hq / p.hkv, d = p.d;
        float qsum = 0.f;
        if (w < G) {
            const T* qr = static_cast<const T*>(p.q) + ((size_t)b * p.hq + h * G + w) * d;
            for (int i = lane; i < d; i += 32) {
                const float q = (float)qr[i];
                qf[w * d + i] = q;
                qsum += fabsf(q);
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) qsum += __shfl_xor_sync(kFull, qsum, o);
        }
        for (int i = tid; i < kBins; i += NT) hist[i] = 0;
        for (int c = tid; c < chunks; c += NT) sel8[c] = (unsigned char)forced_of(c);
        if (tid == 0) sh_cnt = 0, sh_likely = 0, sh_vague = 0, sh_win[0] = 0, sh_win[1] = 0;
        if (p.scored) wait_prerequisites();
        if constexpr (FD > 0) {
            score_row<FD, NW>(p, b, h, lo, hi, own_scores, own_max);
            __syncthreads();
        }

        const T* bounds = static_cast<const T*>(p.bounds);
        const float* scores = FD > 0 ? own_scores : p.scores + row * p.stride;   // 64-byte aligned rows
        const float* tm = FD > 0 ? own_max : p.tile_max + row * (p.stride / 16);
        // a chunk's scores, -inf for blocks that have none
        auto load_chunk = [&](int c, float (&s)[8]) {
            const float4 x = *reinterpret_cast<const float4*>(scores + 8 * c);
            const float4 y = *reinterpret_cast<const float4*>(scores + 8 * c + 4);
            s[0] = x.x, s[1] = x.y, s[2] = x.z, s[3] = x.w;
            s[4] = y.x, s[5] = y.y, s[6] = y.z, s[7] = y.w;
            const uint32_t m = scored_of(c);
            if (m != 0xffu) {
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = (m >> j) & 1 ? s[j] : -INFINITY;
            }
        };
        float kept[8];
        // f(chunk, its scores) for every chunk of this thread
        auto for_chunks = [&](auto f) {
            if constexpr (KEEP) {
                if (tid < chunks) f(tid, kept);
            } else {
                for (int c = tid; c < chunks; c += NT) {
                    float s[8];
                    load_chunk(c, s);
                    f(c, s);
                }
            }
        };
        uint32_t mx = 0;                                   // |bounds|: their bits' order, NaN on top
        for (int i = lo / 16 + tid; i * 16 < hi; i += NT) mx = max(mx, __float_as_uint(tm[i]));
        float smin = INFINITY, smax = -INFINITY;
        bool single = FD > 0 || hi - lo <= NT;             // a thread has one block to look at, at most
        float s1 = -INFINITY;
        int blk1 = lo + tid;
        if (single) {
            if (blk1 < hi) s1 = scores[blk1];
            smax = s1;
            smin = s1 == -INFINITY ? INFINITY : s1;
        } else {
            if (KEEP && tid < chunks) load_chunk(tid, kept);
            for_chunks([&](int, const float (&s)[8]) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    smin = fminf(smin, s[j] == -INFINITY ? INFINITY : s[j]);
                    smax = fmaxf(smax, s[j]);
                }
            });
        }
        const uint32_t kmin = __reduce_min_sync(kFull, ordered(smin));
        const uint32_t kmax = __reduce_max_sync(kFull, ordered(smax));
        // Scores read again in every phase (KEEP false): a score that at least `need` are
        // not below -- the lowest of the warps' r-th largest thread maxima, r warps' worth
        // being need or more -- leaves few to look at (1 x 16,384 blocks: 24.6 us without,
        // 21.9 so; where a thread keeps its scores it gained nothing).
        uint32_t kth = 0xffffffffu;
        const int r = KEEP ? 0 : (need + NW - 1) / NW;
        if (!KEEP && r <= kMaxRounds) {                    // a warp without r scores gives -inf: no bound
            uint32_t v = ordered(smax);
#pragma unroll 1
            for (int i = 0;; ++i) {
                kth = __reduce_max_sync(kFull, v);
                if (i == r - 1) break;
                if (lane == __ffs(__ballot_sync(kFull, v == kth)) - 1) v = 0;
            }
        }
        mx = __reduce_max_sync(kFull, mx);
        const uint32_t qx = __reduce_max_sync(kFull, __float_as_uint(qsum));
        if (lane == 0) sh_a[w] = kmin, sh_b[w] = kmax, sh_c[w] = kth, sh_q[w] = qx, sh_m[w] = mx;
        __syncthreads();
        float rlo = unordered(__reduce_min_sync(kFull, lane < NW ? sh_a[lane] : 0xffffffffu));
        float rhi = unordered(__reduce_max_sync(kFull, lane < NW ? sh_b[lane] : 0u));
        if (!KEEP) kth = __reduce_min_sync(kFull, lane < NW ? sh_c[lane] : 0xffffffffu);
        const float qm = __uint_as_float(__reduce_max_sync(kFull, lane < NW ? sh_q[lane] : 0u));
        const float mm = __uint_as_float(__reduce_max_sync(kFull, lane < NW ? sh_m[lane] : 0u));
        const float A = qm * mm;
        // 1e-35: products too small for float32
        const float E = A * (std::is_same<T, float>::value ? (float)(2 * (d / 32) + 6) * 0x1p-24f
                                                           : (float)(d / 32 * 18 + 3) * 0x1p-23f) + 1e-35f;
        const float win = 2.02f * E;                       // 2E, and the rounding of what it is added to
        const bool sane = A < 1e37f;                       // false for NaN too
        const bool finite = qm < INFINITY && mm < INFINITY;
        float scale_q = unit_scale(qm), scale_b = unit_scale(mm);   // for exact_key
        unsigned heads = (1u << G) - 1;                    // whose scores are finite

        // what could still be undecided lies within the window of that score
        const bool bounded = !KEEP && !single && r <= kMaxRounds && kth > ordered(-INFINITY);
        if (bounded) rlo = fmaxf(rlo, unordered(kth) - win);

        bool crowd = false;                                // the undecided blocks are in `cand`
        bool all = !sane;                                  // and are all that have a score
        int left = need;                                   // places among the undecided blocks
        if (sane && (qm == 0.f || mm == 0.f)) {
            // every score is zero: the lowest blocks, of those with a good id
            bool bad = single && blk1 < hi && s1 == -INFINITY;
            if (!single)
                for_chunks([&](int c, const float (&s)[8]) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) bad |= ((scored_of(c) >> j) & 1) && s[j] == -INFINITY;
                });
            all = __syncthreads_or(bad);
            if (!all)
                for_chunks([&](int c, const float (&)[8]) {
                    sel8[c] = (unsigned char)(forced_of(c) | (below(c, lo + need) & ~below(c, lo)));
                });
        } else if (sane) {
            // ---- bins over [rlo, rhi]; scores above it are in, scores below out
            int bin0 = 0, bin1 = 0;                        // undecided bins
            float inv = 0.f;
            auto bin_of = [&](float s) -> int {            // -1: below the range
                if (s > rhi) return kBins - 1;
                return s < rlo ? -1 : min(kBins - 2, (int)((s - rlo) * inv));
            };
            if (bounded) {
                // the few scores not below it, one to a thread (their places: the list's)
                float* some_s = reinterpret_cast<float*>(list_key);
                int* some_id = reinterpret_cast<int*>(list_s);
                static_assert(NT <= 2 * kListMax, "room for a score and a block per thread");
                for (int c0 = 0; c0 < chunks; c0 += NT) {
                    float s[8];
                    const int c = c0 + tid;
                    if (c < chunks) load_chunk(c, s);
                    uint32_t who[8];
                    int total = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        who[j] = __ballot_sync(kFull, c < chunks && s[j] >= rlo);
                        total += __popc(who[j]);
                    }
                    if (total == 0) continue;
                    int at = 0;
                    if (lane == 0) at = atomicAdd(&sh_likely, total);
                    at = __shfl_sync(kFull, at, 0);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int to = at + __popc(who[j] & ((1u << lane) - 1u));
                        if (((who[j] >> lane) & 1) && to < NT) {
                            some_s[to] = s[j];
                            some_id[to] = 8 * c + j;
                        }
                        at += __popc(who[j]);
                    }
                }
                __syncthreads();
                const int likely = sh_likely;
                if (likely <= NT) {
                    single = true;
                    s1 = tid < likely ? some_s[tid] : -INFINITY;
                    blk1 = tid < likely ? some_id[tid] : 0;
                }
                // the next sync comes before the list is written
            }
            int bins[8], bin_1 = -1;                       // KEEP: of the scores this thread holds
            // read ahead of its use in the list
            const int row1 = single && s1 != -INFINITY ? p.tables[(size_t)b * p.max_blocks + blk1] : -1;
            for (int round = 0;; ++round) {
                const float width = (rhi - rlo) * (1.f / (kBins - 2));
                inv = width > 1e-30f && width < 1e30f ? 1.f / width : 0.f;
                if (single) {
                    bin_1 = s1 == -INFINITY ? -1 : bin_of(s1);
                    if (bin_1 >= 0) atomicAdd(&hist[bin_1], 1u);
                } else {
                    for_chunks([&](int, const float (&s)[8]) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int bin = bin_of(s[j]);
                            if (KEEP) bins[j] = bin;
                            if (bin >= 0) atomicAdd(&hist[bin], 1u);
                        }
                    });
                }
                __syncthreads();
                // the bin of the last place: thread t sums bins from the top down
                constexpr int BPT = kBins / NT;
                uint32_t cnt[BPT], sum = 0;
#pragma unroll
                for (int i = 0; i < BPT; ++i) {
                    cnt[i] = hist[kBins - 1 - (tid * BPT + i)];
                    sum += cnt[i];
                }
                const float reach = win * inv;             // the window in bins
                const int span = reach < (float)kBins ? (int)reach + 2 : kBins;
                uint32_t total;
                uint32_t above = block_scan(sum, &total);
                if ((int)total < need) {                   // blocks with a bad id must fill up
                    all = true;
                    break;
                }
#pragma unroll
                for (int i = 0; i < BPT; ++i) {
                    if (above < (uint32_t)need && (uint32_t)need <= above + cnt[i]) {
                        // this thread: the bin, what lies above its window, what in it
                        const int bin = kBins - 1 - (tid * BPT + i);
                        int over = above, in = cnt[i];
                        for (int x = bin + 1; x <= min(kBins - 2, bin + span); ++x) over -= hist[x], in += hist[x];
                        for (int x = max(0, bin - span); x < bin; ++x) in += hist[x];
                        sh_bin = bin;
                        sh_win[0] = over;
                        sh_win[1] = in;
                    }
                    above += cnt[i];
                }
                __syncthreads();
                const int bin = sh_bin;
                bin0 = max(0, bin - span);
                bin1 = min(kBins - 2, bin + span);
                left = need - sh_win[0];
                crowd = sh_win[1] > kListMax;
                if (!crowd || round == 3 || inv == 0.f || bin1 - bin0 > kBins / 4) break;
                // too many to rank: cut the undecided bins (and one more on each side) again
                const float a = rlo + (float)(bin0 - 1) * width, z = rlo + (float)(bin1 + 2) * width;
                rlo = fmaxf(rlo, a);
                rhi = fminf(rhi, z);
                __syncthreads();                           // hist, sh_bin, sh_win are read
                for (int i = tid; i < kBins; i += NT) hist[i] = 0;
                __syncthreads();
            }
            if (!all && single) {
                if (crowd) {
                    for (int c = tid; c < chunks; c += NT) cand8[c] = 0;
                    __syncthreads();
                }
                if (bin_1 > bin1) {
                    atomicOr(&sel[blk1 >> 5], 1u << (blk1 & 31));
                } else if (bin_1 >= bin0) {                // bin0 >= 0
                    if (crowd) {
                        atomicOr(&cand[blk1 >> 5], 1u << (blk1 & 31));
                    } else {
                        const int at = atomicAdd(&sh_cnt, 1);
                        list_s[at] = s1;
                        list_key[at] = 0;
                        list_row[at] = row1;               // a good id
                        list_id[at] = blk1;
                    }
                }
            } else if (!all) {
                for_chunks([&](int c, const float (&s)[8]) {
                    uint32_t in = forced_of(c), un = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int bin = KEEP ? bins[j] : bin_of(s[j]);
                        in |= bin > bin1 ? 1u << j : 0u;
                        un |= bin >= bin0 && bin <= bin1 ? 1u << j : 0u;
                    }
                    sel8[c] = (unsigned char)in;
                    if (crowd) {
                        cand8[c] = (unsigned char)un;
                    } else if (un) {
                        int at = atomicAdd(&sh_cnt, __popc(un));
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if ((un >> j) & 1) {
                                list_s[at] = s[j];
                                list_key[at] = 0;
                                list_row[at] = p.tables[(size_t)b * p.max_blocks + 8 * c + j];   // a good id
                                list_id[at++] = 8 * c + j;
                            }
                    }
                });
            }
        }
        if (all) {
            for_chunks([&](int c, const float (&)[8]) {
                sel8[c] = (unsigned char)forced_of(c);
                cand8[c] = (unsigned char)scored_of(c);
            });
            crowd = true;
            left = need;
        }
        __syncthreads();
        int open = 0;                                      // places among `cand` that keys cannot tell
        const int32_t* table = p.tables + (size_t)b * p.max_blocks;
        const int listed = sh_cnt;
        if (listed > 0) {
            // ---- the list: `left` of its blocks are selected
            float up = INFINITY, dn = -INFINITY;           // undecided: dn <= score <= up
            int certain = 0;
            bool crowded = listed > left;
            // Only those within the window of T, the left-th largest, are scored again; bf16:
            // all of them where that is a block a warp, the ranking costing as much (1 x
            // 8,192 blocks: 15.2 us, 15.6 with the ranking; float32, whose window seldom
            // holds two, 1 x 4,096 blocks: 27.4 and 25.9)
            if (listed > (std::is_same<T, float>::value ? 4 : NW) && crowded) {
                for (int i = w; i < listed; i += NW) {
                    const float s = list_s[i];
                    const int id = list_id[i];
                    int before = 0;
                    for (int j0 = 0; j0 < listed; j0 += 32) {
                        const int j = min(j0 + lane, listed - 1);
                        const float o = list_s[j];
                        before += __popc(__ballot_sync(
                            kFull, j0 + lane < listed && (o > s || (o == s && list_id[j] < id))));
                    }
                    if (before == left - 1 && lane == 0) sh_thr = s;
                }
                if (tid == 0) sh_win[0] = sh_win[1] = 0;
                __syncthreads();
                up = sh_thr + win;
                dn = sh_thr - win;
                for (int i = tid; i < listed; i += NT) {
                    const float s = list_s[i];
                    if (s > up) atomicAdd(&sh_win[0], 1);
                    else if (s >= dn) atomicAdd(&sh_win[1], 1);
                }
                __syncthreads();
                certain = sh_win[0];
                crowded = certain + sh_win[1] > left;      // more than places
            }
            if (crowded) {
                // a warp takes a block and as few heads as there are warps for
                int bits = 0;
                while ((2 << bits) <= G && (2 << bits) * listed <= NW) ++bits;
                const int some = (G + (1 << bits) - 1) >> bits;
                for (int i = w; i < listed << bits; i += NW) {
                    const int e = i >> bits, g0 = (i & ((1 << bits) - 1)) * some;
                    const float s = list_s[e];
                    // an id that is not good has a score only if the scoring kernel gave up
                    if (s <= up && s >= dn && g0 < G && (unsigned)list_row[e] < (unsigned)p.num_blocks) {
                        const unsigned mine = heads & (((1u << some) - 1) << g0);
                        const unsigned long long k = exact_key<T, false>(bounds, (size_t)list_row[e] * p.hkv + h, d, qf,
                                                                         mine, lane, scale_q, scale_b, nullptr);
                        if (lane == 0) atomicMax(&list_key[e], k);
                    }
                }
                __syncthreads();
            }
            // a warp ranks a block, a lane compares it with one other at a time
            for (int i = w; i < listed; i += NW) {
                const float s = list_s[i];
                const int id = list_id[i];
                bool take = s >= dn;
                if (crowded && take && s <= up) {
                    const unsigned long long k = list_key[i];
                    int before = certain;
                    for (int j0 = 0; j0 < listed; j0 += 32) {
                        const int j = min(j0 + lane, listed - 1);
                        const float o = list_s[j];
                        const unsigned long long x = list_key[j];
                        const bool ahead = j0 + lane < listed && o <= up && o >= dn &&
                                           (x > k || (x == k && list_id[j] < id));
                        before += __popc(__ballot_sync(kFull, ahead));
                    }
                    take = before < left;
                    if (lane == 0 && before == left - 1) sh_key[0] = k;
                    if (lane == 0 && before == left) sh_key[1] = k;
                }
                if (take && lane == 0) atomicOr(&sel[id >> 5], 1u << (id & 31));
            }
            if (crowded) {
                __syncthreads();
                // ---- the last place's key and the first one's behind it: within the keys' errors?
                const unsigned long long last = sh_key[0], reach = 2 * key_error<T>(d);
                if (last - sh_key[1] <= reach && sh_key[1] != 0) {
                    auto near = [&](int i) {
                        const unsigned long long k = list_key[i];
                        return list_s[i] <= up && list_s[i] >= dn && k + reach >= last && k <= last + reach;
                    };
                    if (tid == 0) sh_cnt = 0;
                    for (int c = tid; c < chunks; c += NT) cand8[c] = 0;
                    for (int i = w; i < listed; i += NW)
                        if (near(i))
                            exact_key<T, true>(bounds, (size_t)list_row[i] * p.hkv + h, d, qf, heads, lane, scale_q, scale_b,
                                               &sh_vague);
                    __syncthreads();
                    if (sh_vague) {                        // (keys without lower bits are the scores)
                        for (int i = tid; i < listed; i += NT)
                            if (near(i)) {
                                const int id = list_id[i];
                                const uint32_t bit = 1u << (id & 31);
                                if (atomicAnd(&sel[id >> 5], ~bit) & bit) atomicAdd(&sh_cnt, 1);
                                atomicOr(&cand[id >> 5], bit);
                            }
                        __syncthreads();
                        open = sh_cnt;                     // the places they had
                    }
                }
            }
        } else if (crowd) {
            // ---- a crowd (many equal scores, or none finite): 64-bit keys to the
            // workspace, their threshold by bisection, equal keys by index
            unsigned long long* key = p.exact + row * p.stride;
            auto is_cand = [&](int blk) { return (cand8[blk >> 3] >> (blk & 7)) & 1; };
            auto block_count = [&](uint32_t c) -> int {
                c = __reduce_add_sync(kFull, c);
                __syncthreads();
                if (lane == 0) sh_a[w] = c;
                __syncthreads();
                return (int)__reduce_add_sync(kFull, lane < NW ? sh_a[lane] : 0u);
            };
            if (!finite) {
                // ---- blocks whose score is not finite come first; the others are scaled by the
                // largest of their bounds and of the finite heads' queries (times d: no sum
                // of them passes float32's range)
                if (tid == 0) sh_win[0] = sh_win[1] = 0, sh_cnt = 0;
                __syncthreads();
                if (w < G) {
                    uint32_t top = 0;
                    for (int i = lane; i < d; i += 32) top = max(top, __float_as_uint(qf[w * d + i]) & 0x7fffffffu);
                    top = __reduce_max_sync(kFull, top);
                    if (lane == 0 && top < 0x7f800000u) atomicOr(&sh_cnt, 1 << w), atomicMax(&sh_win[0], (int)top);
                }
                for (int blk = lo + w; blk < hi; blk += NW)
                    if (is_cand(blk)) {
                        const int id = table[blk];
                        if (id < 0 || id >= p.num_blocks) continue;
                        const size_t id_row = (size_t)id * p.hkv + h;
                        const bool first = score_not_finite(bounds, id_row, d, qf, G, lane);
                        if (lane == 0) key[blk] = first ? ~0ull : 0ull;
                        if (first) continue;
                        uint32_t top = 0;
                        for (int i = lane; i < 2 * d; i += 32)
                            top = max(top, __float_as_uint((float)bounds[id_row * 2 * d + i]) & 0x7fffffffu);
                        top = __reduce_max_sync(kFull, top);
                        if (lane == 0) atomicMax(&sh_win[1], (int)top);
                    }
                __syncthreads();
                heads = (unsigned)sh_cnt;
                scale_q = unit_scale(__int_as_float(sh_win[0])) * 0x1p-7f;
                scale_b = unit_scale(__int_as_float(sh_win[1]));
            }
            for (int blk = lo + w; blk < hi; blk += NW)
                if (is_cand(blk)) {
                    const int id = table[blk];
                    unsigned long long k = 0;              // a bad id (flagged when it was scored)
                    if (id >= 0 && id < p.num_blocks) {
                        if (!finite && key[blk] != 0) continue;
                        k = exact_key<T, true>(bounds, (size_t)id * p.hkv + h, d, qf, heads, lane, scale_q, scale_b,
                                               &sh_vague);
                    }
                    __syncwarp();
                    if (lane == 0) key[blk] = k;
                }
            __syncthreads();
            unsigned long long thr = 0;                    // the left-th largest key
            for (int bit = 63; bit >= 0; --bit) {
                const unsigned long long t = thr | (1ull << bit);
                uint32_t c = 0;
                for (int blk = lo + tid; blk < hi; blk += NT) c += is_cand(blk) && key[blk] >= t;
                if (block_count(c) >= left) thr = t;
            }
            if (sh_vague && thr != 0 && thr != ~0ull) {
                // more within the keys' errors of the last place than places?
                const unsigned long long reach = 2 * key_error<T>(d);
                uint32_t over = 0, near = 0;
                for (int blk = lo + tid; blk < hi; blk += NT)
                    if (is_cand(blk)) over += key[blk] > thr + reach, near += key[blk] >= thr - reach && key[blk] <= thr + reach;
                const int above = block_count(over);
                if (above + block_count(near) > left) {
                    open = left - above;
                    for (int ch = tid; ch < chunks; ch += NT) {
                        uint32_t in = 0, keep = 0;
                        for (uint32_t m = cand8[ch]; m; m &= m - 1) {
                            const unsigned long long k = key[8 * ch + __ffs(m) - 1];
                            if (k > thr + reach) in |= m & -m;
                            else if (k >= thr - reach) keep |= m & -m;
                        }
                        sel8[ch] |= (unsigned char)in;
                        cand8[ch] = (unsigned char)keep;
                    }
                }
            }
            uint32_t c = 0;
            for (int blk = lo + tid; blk < hi && open == 0; blk += NT)
                if (is_cand(blk) && key[blk] > thr) {
                    atomicOr(&sel[blk >> 5], 1u << (blk & 31));
                    ++c;
                }
            int places = open ? 0 : left - block_count(c);
            for (int base = 0; base < chunks && places > 0; base += NT) {
                const int ch = base + tid;
                uint32_t eq = 0;
                if (ch < chunks)
                    for (uint32_t m = cand8[ch]; m; m &= m - 1) {
                        const int j = __ffs(m) - 1;
                        if (key[8 * ch + j] == thr) eq |= 1u << j;
                    }
                uint32_t total;
                int at = (int)block_scan(__popc(eq), &total);
                for (; eq && at < places; eq &= eq - 1, ++at) {
                    const int blk = 8 * ch + __ffs(eq) - 1;
                    atomicOr(&sel[blk >> 5], 1u << (blk & 31));
                }
                places -= min(places, (int)total);
            }
        }
        if (open > 0)
            settle<T, NT>(bounds, table, p.hkv, h, d, qf, heads, lo, hi, open, sel8, cand8, p.exact + row * p.stride);
    } else {
        for (int c = tid; c < chunks; c += NT) sel8[c] = (unsigned char)forced_of(c);
    }
    __syncthreads();
    // ---- the selected blocks, ascending
    uint32_t done = 0;
    for (int base = 0; base < chunks; base += NT) {
        const int c = base + tid;
        uint32_t m = c < chunks ? sel8[c] : 0, total;
        uint32_t at = done + block_scan(__popc(m), &total);
        for (; m && at < (uint32_t)p.k; m &= m - 1) out[at++] = 8 * c + __ffs(m) - 1;
        done += total;
    }
}

constexpr size_t kSelectFixed = kListMax * 20 + 8 * 128 * 4 + kBins * 4;
constexpr int kMaxBlocks = 1 << 19;    // 128 KB of bitmaps

inline int padded(int max_blocks) { return (max_blocks + 15) / 16 * 16; }

template <typename T, int NT, bool KEEP, int FD = 0>
int launch_select(const SelectParams& p, int num_seqs, cudaStream_t stream) {
    auto bytes = [](int blocks) {
        const int words = ((blocks + 31) / 32 + 3) / 4 * 4;
        return (int)kSelectFixed + words * 8 + (FD > 0 ? padded(blocks) / 16 * 68 : 0);
    };
    auto kern = select_rows<T, NT, KEEP, FD>;
    int occ = 0;
    const int st = kernel_setup(reinterpret_cast<const void*>(kern), bytes(KEEP ? NT * 8 : kMaxBlocks), NT, &occ);
    if (st != PKV_OK) return st;
    note_launch();
    const cudaError_t e = launch_pdl(kern, dim3(p.hkv, num_seqs), dim3(NT), bytes(p.max_blocks), stream, p);
    return e == cudaSuccess ? PKV_OK : cuda_fail("select_blocks: selection launch", e);
}

template <int D>
int launch_scores_bf16(const SelectParams& p, int num_seqs, cudaStream_t stream) {
    auto kern = score_blocks_bf16<D>;
    constexpr int kSmem = ScoreSmem<D>::kBytes;
    int occ = 0;
    const int st = kernel_setup(reinterpret_cast<const void*>(kern), kSmem, 128, &occ);
    if (st != PKV_OK) return st;
    // kv heads side by side in a CTA: the power of two up to 4 that divides them
    const int side = p.hkv % 4 == 0 ? 4 : p.hkv % 2 == 0 ? 2 : 1;
    const int blocks = kStageRows / side, stages = (p.max_blocks + blocks - 1) / blocks;
    // stages a CTA walks: the GPU's share of one wave, at most 6 (rows are ragged; 32
    // sequences of up to 2048 blocks: 35.4 us with 8, which left a ragged second wave, 32.2
    // with 6, 32.6 with 4; 1 of 32768: 42, 38, 39; 40 kv heads: 134, 134, 138. Sharing the
    // stages there are evenly among the CTAs of one wave: 33.0, 44, 140, as each has to
    // read the lengths before it knows its first block)
    const long long all = (long long)num_seqs * (p.hkv / side) * stages;
    const long long slots = (long long)num_sms() * (occ > 0 ? occ : 1);
    const int per = (int)(all <= slots ? 1 : all >= 6 * slots ? 6 : (all + slots - 1) / slots);
    note_launch();
    const cudaError_t e = launch_pdl(kern, dim3((stages + per - 1) / per, p.hkv / side, num_seqs), dim3(128), kSmem,
                                     stream, p, per, side);
    return e == cudaSuccess ? PKV_OK : cuda_fail("select_blocks: scoring launch", e);
}

int launch_scores_f32(const SelectParams& p, int num_seqs, cudaStream_t stream) {
    const int tiles = padded(p.max_blocks) / 16;
    // 16-block tiles two warps walk: more once the warps fill the GPU
    int per = 1;
    const long long rows = (long long)num_seqs * p.hkv, fill = 20LL * num_sms();
    while (per < 16 && rows * tiles / (2 * per) >= fill) per *= 2;
    dim3 grid((tiles + 2 * per - 1) / (2 * per), p.hkv, num_seqs);
    note_launch();
    const cudaError_t e = p.d == 64 ? launch_pdl(score_blocks_f32<64>, grid, dim3(128), 0, stream, p, per)
                                    : launch_pdl(score_blocks_f32<128>, grid, dim3(128), 0, stream, p, per);
    return e == cudaSuccess ? PKV_OK : cuda_fail("select_blocks: scoring launch", e);
}

template <typename T>
int launch_scores(const SelectParams& p, int num_seqs, cudaStream_t stream) {
    if constexpr (std::is_same<T, float>::value) return launch_scores_f32(p, num_seqs, stream);
    else return p.d == 64 ? launch_scores_bf16<64>(p, num_seqs, stream) : launch_scores_bf16<128>(p, num_seqs, stream);
}

// Rows of at most this many blocks are scored by the CTA that selects from them: a tile
// of 16 blocks a warp. 4 sequences of 63 blocks: 6.6 us in one launch against 7.5 in
// two; 1 of 256: 9.3 against 8.1; 64 of 256: 25 against 17.
constexpr int kFuseBlocks = 128;      // at most a block a thread (256)

template <typename T>
int select_all(const SelectParams& p, int num_seqs, cudaStream_t stream) {
    if constexpr (!std::is_same<T, float>::value) {
        if (p.scored && p.max_blocks <= kFuseBlocks) {
            SelectParams f = p;
            f.scored = 0;
            return p.d == 64 ? launch_select<T, 256, true, 64>(f, num_seqs, stream)
                             : launch_select<T, 256, true, 128>(f, num_seqs, stream);
        }
    }
    if (p.scored) {
        const int st = launch_scores<T>(p, num_seqs, stream);
        if (st != PKV_OK) return st;
    }
    // a thread keeps 8 scores; CTAs of 256 where rows are short (64 sequences of 512
    // blocks: 23 us, 28 with 512 threads) or too many for one wave of 512 (512 rows of 2048:
    // 55 us, 60 with 512; 256 rows: 33 and 32), of 512 up to 4096 blocks
    const bool many = (long long)num_seqs * p.hkv > 2 * num_sms();
    if (p.max_blocks <= (many ? 2048 : 1024)) return launch_select<T, 256, true>(p, num_seqs, stream);
    if (p.max_blocks <= 4096) return launch_select<T, 512, true>(p, num_seqs, stream);
    if (p.max_blocks <= 8192) return launch_select<T, 1024, true>(p, num_seqs, stream);
    return launch_select<T, 1024, false>(p, num_seqs, stream);
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
    if (checking()) return PKV_OK;
    int* err = error_word();
    if (!err) return PKV_ERR_CUDA;
    // changed blocks of a sequence (at most one more than the new tokens fill); the
    // kernel strides, so a wrong hint costs time only
    long long blocks = max_new_tokens > 0 ? (max_new_tokens - 1LL + block_size - 1) / block_size + 1
                                          : max_blocks_per_seq;
    if (blocks > max_blocks_per_seq) blocks = max_blocks_per_seq;
    long long gx = (blocks * num_kv_heads + 3) / 4;
    // six waves of 5 CTAs an SM (8 sequences of 1024 changed bf16 blocks: 54 us, 58 with
    // twice as many CTAs, 60 with a third)
    const long long cap = 30LL * num_sms() / num_seqs + 1;
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
    if (checking()) return PKV_OK;
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
    p.scored = scored;
    const size_t rows = (size_t)num_seqs * num_kv_heads;
    if (scored) {
        p.exact = static_cast<unsigned long long*>(workspace);
        p.scores = reinterpret_cast<float*>(p.exact + rows * p.stride);
        p.tile_max = p.scores + rows * p.stride;
    }
    p.err = error_word();
    if (!p.err) return PKV_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    try {
        return q_dtype == PKV_F32 ? select_all<float>(p, num_seqs, s)
                                  : select_all<__nv_bfloat16>(p, num_seqs, s);
    } catch (...) {                                         // the per-kernel records' host memory
        return cuda_fail("select_blocks: host memory", cudaErrorMemoryAllocation);
    }
}

}  // extern "C"
