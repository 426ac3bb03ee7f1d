// Decode attention over selected blocks: paged_attention_decode_sparse.
//
// The mathematics is the decode kernel's (online softmax over a sequence's cached
// tokens, tile by tile) over the tokens of the blocks that a list names for each row
// (sequence, kv head). What differs is the walk and the merge. A thread-block cluster
// takes some rows, lays their listed blocks end to end and gives every warp of its CTAs
// an equal run of them: a warp streams its run through a ring of its own, across the
// borders of rows, and keeps no state but the current row's. A row that lies within one
// warp's run is written at once; the parts of the others meet in shared memory and are
// merged at the end (a warp has at most two: the row its run begins in and the one it
// ends in): first a CTA's, then the cluster's, or, where the cluster has one row, by
// every warp pushing its part to the CTAs that merge it. So one launch does it without
// a workspace, few rows are spread over many warps, and many rows make one wave of equal
// shares, whatever their lengths, where a CTA a row left a ragged second wave.
// Bound: HBM bytes of the selected tiles when there are many rows (1280 rows of 64 bf16
// blocks 94.3 us, 0.96 of the copy rate; 512 rows of 128 E4M3 blocks, 4 heads, 49.3, 0.77:
// the stream itself is at the copy rate, 5 us lie before it and 7 in the merges); a chain of
// loads (length, list, table, tile, partner's partials) when there are few (8 rows of 128
// blocks 6.3 us on the GPU).
#pragma once

#include "pkv_decode_impl.cuh"

namespace pkv {
namespace sparse {

using decode::kFull;
using decode::kLog2e;

struct Params {
    void* out;
    const void* q;
    const char* k_pool;
    const char* v_pool;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* selected;           // [B][Hkv][K] logical blocks, ascending, -1 padded
    int* err;
    int max_blocks, num_blocks, num_heads, num_kv_heads, k;
    int num_rows;                      // (sequence, kv head), kv heads fastest
    int cluster_rows;                  // rows of a cluster, at most kMaxRows
    int stages;                        // of a warp's ring
    int push;                          // a cluster's one row is merged by pushes (below)
    float qscale, v_scale;
};

struct Args {
    Params p;
    int num_seqs, head_dim, block_size;
    float scale, k_scale, v_scale;
    cudaStream_t stream;
};

constexpr int kNumWarps = 4;           // of a CTA; twice as many when there are few rows
constexpr int kMaxCluster = 8;         // the portable size
constexpr int kMaxRows = 32;           // rows of a cluster: one per lane
constexpr int kMaxStages = 8;          // of a warp's ring
constexpr int kSmemSm = 227 * 1024;    // shared memory of an SM for CTAs, 1 KB of each reserved

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// orders nothing: for partners that only have to stay
__device__ __forceinline__ void cluster_sync_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// The address of a shared-memory location in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float cluster_ld(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// 16 or 8 bytes into the shared memory of the cluster's CTA that `addr` lies in, counted
// by the mbarrier `bar` of that CTA.
__device__ __forceinline__ void push4(uint32_t addr, float4 v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void push2(uint32_t addr, float x, float y, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(addr), "f"(x),
                 "f"(y), "r"(bar)
                 : "memory");
}
// mbar_wait_bounded for what the cluster's other CTAs push
__device__ __forceinline__ bool pushed_wait_bounded(uint32_t bar, const int* err) {
    const unsigned long long t0 = global_ns();
    while (true) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0, %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(20000u)
            : "memory");
        if (done) return true;
        if (global_ns() - t0 > kWaitLimitNs) return false;
        if (err && (*reinterpret_cast<const volatile int*>(err) & kErrTimeout)) return false;
    }
}

// Shared memory: mbarriers | tokens per stage | row borders and lengths per warp |
// first parts | (CUDA-core math) the warps' query rows and scratch | rings, for a CTA
// of `nw` warps with rings of `stages`, both chosen at launch. A warp's last part goes
// into its own ring, which is drained by then, a CTA's parts into the second halves of
// warp 0's and 1's. Behind the rings, where a cluster has one row: what is pushed here,
// an mbarrier and a slot per warp of the cluster.
template <class Math, int D, int BS, int G>
struct Smem {
    static constexpr bool kSimt = Math::kWarpSmemFloats > 0;
    static constexpr int kStage = 2 * Math::Lay::kTile;    // bytes of a K and a V tile
    static constexpr int kPartFloats = G * (D + 4);        // m [G], l [G], (pad), o [G][D]
    static constexpr int kO = 4 * G;                       // of o within a part
    __host__ __device__ static constexpr int tok_off(int nw) { return nw * kMaxStages * 8; }
    __host__ __device__ static constexpr int row_off(int nw) { return tok_off(nw) + nw * kMaxStages * 4; }
    __host__ __device__ static constexpr int part_off(int nw) {
        return (row_off(nw) + nw * (2 * kMaxRows + 1) * 4 + 15) / 16 * 16;
    }
    __host__ __device__ static constexpr int q_off(int nw) { return part_off(nw) + nw * kPartFloats * 4; }
    __host__ __device__ static constexpr int warp_off(int nw) { return q_off(nw) + (kSimt ? nw * G * D * 4 : 0); }
    __host__ __device__ static constexpr int ring_off(int nw) {
        return (warp_off(nw) + nw * Math::kWarpSmemFloats * 4 + 127) / 128 * 128;
    }
    // a warp's part and a CTA's part fit in a ring
    static constexpr int kMinStages = (2 * kPartFloats * 4 + kStage - 1) / kStage;
    // stages of a warp's ring within `bytes` of shared memory per CTA
    static constexpr int stages(int nw, int bytes) {
        const int n = (bytes - ring_off(nw)) / (nw * kStage);
        return n < kMinStages ? kMinStages : n > kMaxStages ? kMaxStages : n;
    }
    static constexpr int kQuads = G * D / 4;               // 16-byte pieces of a part's o
    static constexpr int recv_bytes(int nw) { return 16 + nw * (kQuads + 8) * 16; }
    static constexpr int bytes(int nw, int stages) { return ring_off(nw) + nw * stages * kStage; }
    static_assert(kStage % 32 == 0, "halves of a ring are 16-byte aligned");
    static_assert(kMinStages <= kMaxStages && bytes(kNumWarps, kMinStages) <= kSmemSm, "shared memory per CTA");
    // eight warps a CTA where their rings fit (not: float32, 8 heads, 32-token blocks)
    static constexpr bool kWide = bytes(2 * kNumWarps, kMinStages) + recv_bytes(2 * kNumWarps) <= kSmemSm;
};

// A 16 x 8 product on the tensor cores: c += a b
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A maximum that is NaN if an operand is: a NaN logit has to reach its whole row,
// whichever warp sees it.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// What logits are taken relative to: their maximum; 0 where all so far are -infinity, so
// that their weights are 0 and not the NaN of -infinity less -infinity.
__device__ __forceinline__ float softmax_base(float m) { return m == -INFINITY ? 0.f : m; }

// Two weights as 16-bit numbers, and what that rounding left of each as two more: hi + lo
// is a weight up to 2^-16 of itself in bf16 (2^-8 twice), in f16 up to 2^-22 (2^-11 twice)
// and half of f16's smallest step, 2^-25. Both go through the product, so the output is
// that of float32 weights but for its own rounding, and their sum, of float32 weights, is
// theirs. (A second product a tile: 64 sequences x 128 blocks of 128 dims, E4M3 46.0 us
// without and 46.0 with it, 8 heads a kv head 48.3 and 50.0; bf16 83 and 84.5; 64 dims in
// E4M3 blocks of 32 tokens 44.1 and 47.7; 1 sequence 6.0 and 6.25. What is left over in the
// columns of absent heads instead, for up to 4: 46.8, -, 85.5, 46.8, 6.15.)
template <bool F16>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        hi = *reinterpret_cast<const uint32_t*>(&h);
        lo = decode::pack_f16(x - f.x, y - f.y);
    } else {
        hi = decode::pack_bf16(x, y);
        lo = decode::pack_bf16(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
    }
}

// 2^x, results below the normal range flushed: such weights vanish in their sum
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a tile's logits (in units of log2 e) are also given to, as runs of consecutive tokens
// of one head: nothing here; decode with token weights keeps them.
struct NoSink {
    __device__ __forceinline__ void put(int, int, float, float) const {}
    __device__ __forceinline__ void put(int, int, float, float, float, float) const {}
    __device__ __forceinline__ void put(int, int, float) const {}
};

// Tensor-core math for up to 8 query heads a kv head, bf16 and E4M3 caches. Scores as
// in the decode kernel (query heads are the rows of A, half of them zero): lane 4r + c
// holds the scores of head r, tokens 2c + e of two groups of 8, which is how the B
// operand of a product over tokens wants them. So O^T = V^T P: 16 dims are the rows
// of A (the same words that the decode kernel loads as two B operands), the heads its
// 8 columns, and a product carries 16 dims instead of 8. Lane 4r + c holds dims r and
// r + 8 of heads 2c, 2c + 1. One softmax step a tile of 16 or 32 tokens. (64 sequences
// x 128 E4M3 blocks of 8 kv heads: 55.7 us with the decode kernel's math, 47.5 so; bf16:
// 87 and 84; one sequence of 512 blocks: 13.9 and 12.2; all with one product a tile for the
// weights, where there are two now. The issue slots bound E4M3: 47% in use before, on 12
// warps an SM, 29% now.)
template <typename KV, int D, int BS, int G>
struct HeadsMath {
    using Lay = decode::Layout<KV, D, BS>;
    static constexpr bool F8 = std::is_same<KV, uint8_t>::value;
    static constexpr int KS = D / 16, MT = D / 16, SUB = BS / 16;
    static constexpr int kWarpSmemFloats = 0;
    // weights are 2^kLift times themselves, and so are their sums: E4M3 caches take them in
    // f16, whose smallest step is then 2^-38 of the largest weight instead of 2^-24
    static constexpr float kLift = F8 ? 14.f : 0.f;
    static_assert(G >= 1 && G <= 8 && BS % 16 == 0 && D % 32 == 0, "mma shape");

    struct State {
        uint32_t qa[KS][2];                                // A fragments of Q (a0, a2)
        float o[MT][4];
        float m, l;                                        // of head r, l this lane's tokens'
        float qscale;                                      // E4M3: what head r's scores are times
    };

    // The values of unwritten slots (ntok and up) may be anything: zero, in place.
    __device__ __forceinline__ static void clear_tail(unsigned char* vt, int ntok, int lane) {
        constexpr int X = Lay::kX, E = Lay::kElt;
#pragma unroll 1
        for (int t = ntok / X; t < BS / X; ++t) {
            const int keep = max(0, ntok - t * X) * E * 8;  // bits of the 16 bytes
#pragma unroll 1
            for (int d = lane; d < D; d += 32) {
                uint32_t* w = reinterpret_cast<uint32_t*>(vt + Lay::v_off(d, t));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int bits = keep - 32 * i;
                    if (bits < 32) w[i] = bits > 0 ? w[i] & ((1u << bits) - 1u) : 0u;
                }
            }
        }
        __syncwarp();
    }

    template <class Sink = NoSink>
    __device__ __forceinline__ static void tile(State& st, const unsigned char* kt, const unsigned char* vt, int ntok,
                                                int lane, float qscale, const Sink& sink = Sink()) {
        const int c = lane & 3, mi = lane >> 3, rr = lane & 7;
        const float by = F8 ? st.qscale : qscale;
        const uint32_t kbase = smem_addr(kt), vbase = smem_addr(vt);
        float x[SUB][2][2], mx = -INFINITY;                // scores of head r
#pragma unroll
        for (int h = 0; h < SUB; ++h) {
            // even and odd k-steps apart: shorter chains
            float s[2][2][4];
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i >> 3][(i >> 2) & 1][i & 3] = 0.f;
            uint32_t k8[4];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t b[2][2];
                if constexpr (F8) {
                    // byte pairs: a row is a token's 16 dims, lane (r, c) gets bytes 4c .. 4c+3
                    if ((ks & 1) == 0)
                        decode::ldsm_x4(kbase + Lay::k_off(ks + (mi >> 1), 16 * h + 4 * (rr >> 1) + 2 * (mi & 1) + (rr & 1)),
                                        k8[0], k8[1], k8[2], k8[3]);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t w = k8[(ks & 1) * 2 + u];
                        b[u][0] = decode::e4m3x2_to_f16x2(w);
                        b[u][1] = decode::e4m3x2_to_f16x2(w >> 16);
                    }
                } else {
                    decode::ldsm_x4(kbase + Lay::k_off(2 * ks + (mi & 1), 16 * h + 8 * (mi >> 1) + rr), b[0][0], b[0][1],
                                    b[1][0], b[1][1]);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) mma<F8>(s[ks & 1][u], st.qa[ks][0], 0u, st.qa[ks][1], 0u, b[u][0], b[u][1]);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) x[h][u][e] = (s[0][u][e] + s[1][u][e]) * by;
        }
        if (ntok < BS) {
#pragma unroll
            for (int i = 0; i < SUB * 4; ++i) {
                const int h = i >> 2, u = (i >> 1) & 1, e = i & 1;
                const int tok = F8 ? 16 * h + 4 * c + 2 * u + e : 16 * h + 8 * u + 2 * c + e;
                if (tok >= ntok) x[h][u][e] = -INFINITY;
            }
        }
#pragma unroll
        for (int h = 0; h < SUB; ++h) {
            if constexpr (F8) {
                sink.put(lane >> 2, 16 * h + 4 * c, x[h][0][0], x[h][0][1], x[h][1][0], x[h][1][1]);
            } else {
                sink.put(lane >> 2, 16 * h + 2 * c, x[h][0][0], x[h][0][1]);
                sink.put(lane >> 2, 16 * h + 8 + 2 * c, x[h][1][0], x[h][1][1]);
            }
        }
#pragma unroll
        for (int i = 0; i < SUB * 4; ++i) mx = max_nan(mx, x[i >> 2][(i >> 1) & 1][i & 1]);
        // ---- online softmax, once a tile
        mx = max_nan(mx, __shfl_xor_sync(kFull, mx, 1));
        mx = max_nan(mx, __shfl_xor_sync(kFull, mx, 2));
        const float m_new = max_nan(st.m, mx), base = softmax_base(m_new), alpha = ex2(st.m - base);
        float psum = 0.f;
#pragma unroll
        for (int h = 0; h < SUB; ++h)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[h][u][e] = ex2(x[h][u][e] - base + kLift);
                    psum += x[h][u][e];
                }
        st.l = st.l * alpha + psum;
        st.m = m_new;
        if (!__all_sync(kFull, alpha == 1.f)) {            // a running max moved
            const float a0 = __shfl_sync(kFull, alpha, 8 * c), a1 = __shfl_sync(kFull, alpha, 8 * c + 4);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                st.o[i][0] *= a0;
                st.o[i][1] *= a1;
                st.o[i][2] *= a0;
                st.o[i][3] *= a1;
            }
        }
#pragma unroll
        for (int h = 0; h < SUB; ++h) {
            uint32_t p0, p1, r0, r1;
            split_pair<F8>(x[h][0][0], x[h][0][1], p0, r0);
            split_pair<F8>(x[h][1][0], x[h][1][1], p1, r1);
            uint32_t v8[4];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uint32_t a[2][2];                          // dims 16 i + 8 y + r, tokens' words z
                if constexpr (F8) {
                    // byte pairs: a row is a dim's 16 tokens, lane (r, c) gets tokens 4c .. 4c+3
                    if ((i & 1) == 0)
                        decode::ldsm_x4(vbase + Lay::v_off(16 * i + 8 * mi + rr, h), v8[0], v8[1], v8[2], v8[3]);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t v = v8[(i & 1) * 2 + y];
                        a[y][0] = decode::e4m3x2_to_f16x2(v);
                        a[y][1] = decode::e4m3x2_to_f16x2(v >> 16);
                    }
                } else {
                    decode::ldsm_x4(vbase + Lay::v_off(16 * i + 8 * (mi >> 1) + rr, 2 * h + (mi & 1)), a[0][0], a[0][1],
                                    a[1][0], a[1][1]);
                }
                mma<F8>(st.o[i], a[0][0], a[1][0], a[0][1], a[1][1], p0, p1);
                mma<F8>(st.o[i], a[0][0], a[1][0], a[0][1], a[1][1], r0, r1);
            }
        }
    }

    // f(head, dim, value) of what this lane holds
    template <typename F>
    __device__ __forceinline__ static void each(const State& st, int lane, F f) {
        const int r = lane >> 2, c = lane & 3;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (2 * c + e < G) {
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    f(2 * c + e, 16 * i + r, st.o[i][e]);
                    f(2 * c + e, 16 * i + 8 + r, st.o[i][2 + e]);
                }
            }
    }
    __device__ __forceinline__ static float sum(const State& st) {
        float l = st.l;
        l += __shfl_xor_sync(kFull, l, 1);
        return l + __shfl_xor_sync(kFull, l, 2);
    }
    // this warp's part of a row
    __device__ __forceinline__ static void finish(State& st, float* pm, float* pl, float* po, int, int lane, bool dead) {
        const float l = sum(st);
        const int r = lane >> 2;
        if (r < G && (lane & 3) == 0) {
            pm[r] = dead ? -INFINITY : st.m;
            pl[r] = dead ? 0.f : l;
        }
        each(st, lane, [&](int g, int d, float v) { po[g * D + d] = dead ? 0.f : v; });
    }
};

// 2^n, -126 <= n <= 127
__device__ __forceinline__ float pow2(int n) { return __uint_as_float((uint32_t)(n + 127) << 23); }

// The query rows of one (sequence, kv head) into a warp's state. Tensor-core math:
// straight into the operand fragments; CUDA-core
// math: through the warp's shared-memory rows, scaled.
// E4M3 caches multiply in f16: a head's query is brought to f16's upper range by the power
// of two that takes its largest element into [2^14, 2^15), exactly but for elements below
// 2^-28 of that (f16 keeps 2^-24, half a step of it 2^-39 of the largest), and its scores
// are scaled back.
template <class Math, typename QT, int D, int G>
__device__ __forceinline__ void begin_row(typename Math::State& st, const QT* q, float qscale, float* qs, int lane) {
    if constexpr (Math::kWarpSmemFloats > 0) {
        __syncwarp();
        for (int i = lane; i < G * D; i += 32) qs[i] = decode::to_f(q[i]) * qscale;
        __syncwarp();
        Math::init(st, qs, lane);
    } else {
        const int r = lane >> 2, c = lane & 3;
        const bool live = r < G;
        if constexpr (Math::F8) {
            uint2 x[Math::KS];
            uint32_t top = 0;                              // largest magnitude: bf16 bits order as numbers
#pragma unroll
            for (int s = 0; s < Math::KS; ++s) {
                x[s] = live ? __ldg(reinterpret_cast<const uint2*>(q + r * D + 16 * s + 4 * c)) : make_uint2(0, 0);
                top = __vmaxu2(top, __vmaxu2(x[s].x & 0x7fff7fffu, x[s].y & 0x7fff7fffu));
            }
            top = __vmaxu2(top, __shfl_xor_sync(kFull, top, 1));
            top = __vmaxu2(top, __shfl_xor_sync(kFull, top, 2));
            // infinite and NaN elements stay so under any scale; 2^106 is enough for zeros and subnormals
            const int e = min((int)(max(top & 0xffffu, top >> 16) >> 7), 254) - 127, up = min(14 - e, 106);
            const float by = pow2(up);
            st.qscale = qscale * pow2(-up);
#pragma unroll
            for (int s = 0; s < Math::KS; ++s) {
                st.qa[s][0] = decode::pack_f16(__uint_as_float(x[s].x << 16) * by, __uint_as_float(x[s].x & 0xffff0000u) * by);
                st.qa[s][1] = decode::pack_f16(__uint_as_float(x[s].y << 16) * by, __uint_as_float(x[s].y & 0xffff0000u) * by);
            }
        } else {
#pragma unroll
            for (int s = 0; s < Math::KS; ++s) {
                st.qa[s][0] = live ? __ldg(reinterpret_cast<const uint32_t*>(q + r * D + 16 * s + 2 * c)) : 0u;
                st.qa[s][1] = live ? __ldg(reinterpret_cast<const uint32_t*>(q + r * D + 16 * s + 8 + 2 * c)) : 0u;
            }
        }
#pragma unroll
        for (int i = 0; i < 4 * Math::MT; ++i) st.o[i >> 2][i & 3] = 0.f;
        st.m = -INFINITY;
        st.l = 0.f;
    }
}

// A row that one warp has seen whole, to the output.
template <class Math, typename QT, int D, int G>
__device__ __forceinline__ void write_row(typename Math::State& st, QT* out, float v_scale, int lane) {
    if constexpr (Math::kWarpSmemFloats > 0) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float l = st.l[g];
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
            const float inv = l > 0.f ? v_scale / l : 0.f;
#pragma unroll
            for (int k = 0; k < Math::DPL; ++k) decode::store_out(out + g * D + lane + 32 * k, st.acc[g][k] * inv);
        }
    } else {
        const float l = Math::sum(st), inv = l > 0.f ? v_scale / l : 0.f;
        const int c = lane & 3;
        const float inv0 = __shfl_sync(kFull, inv, 8 * c), inv1 = __shfl_sync(kFull, inv, 8 * c + 4);
        Math::each(st, lane, [&](int g, int d, float v) { decode::store_out(out + g * D + d, v * ((g & 1) ? inv1 : inv0)); });
    }
}

// PAIR = 2: a pipeline stage holds two list entries of BS / 2 tokens side by side
// (see the decode kernel); BS is then the stage's token count.
// 168 registers: three CTAs of 4 warps an SM.
template <class Math, typename QT, int D, int BS, int G, int PAIR>
__global__ void __maxnreg__(168) sparse_decode_kernel(const Params p) {
    using S = Smem<Math, D, BS, G>;
    constexpr int TILE = Math::Lay::kTile;
    constexpr int PBS = BS / PAIR, PTILE = TILE / PAIR;
    static_assert(PAIR == 1 || PAIR == 2, "entries per stage");
    pdl_enter();                                           // launched with programmatic serialisation
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int NW = blockDim.x >> 5, ST = p.stages, warp_ring = ST * S::kStage;
    unsigned char* const rings = smem + S::ring_off(NW);
    unsigned char* const ring = rings + w * warp_ring;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem) + w * kMaxStages;
    int32_t* stage_tok = reinterpret_cast<int32_t*>(smem + S::tok_off(NW)) + w * kMaxStages;
    int32_t* border = reinterpret_cast<int32_t*>(smem + S::row_off(NW)) + w * (2 * kMaxRows + 1);
    int32_t* length = border + kMaxRows + 1;
    float* part0 = reinterpret_cast<float*>(smem + S::part_off(NW));
    float* qs = reinterpret_cast<float*>(smem + S::q_off(NW)) + w * G * D;
    float* pb = reinterpret_cast<float*>(smem + S::warp_off(NW)) + w * Math::kWarpSmemFloats;

    // ---- the cluster's rows: stages (every warp works them out for itself)
    const int rank = (int)cluster_rank(), csize = (int)cluster_size();
    const int row0 = (int)(blockIdx.x / csize) * p.cluster_rows;
    const int nrows = min(p.cluster_rows, p.num_rows - row0);
    int L = 0;
    if (lane < nrows) {
        const int b = (row0 + lane) / p.num_kv_heads;
        L = p.seq_lens[b];
        if (L < 0 || L > p.max_blocks * PBS) {              // length the table cannot hold
            flag_error(p.err, kErrOutOfRange);
            L = L < 0 ? 0 : p.max_blocks * PBS;
        }
    }
    // distinct entries below the row's blocks: no more than there are blocks
    const int entries = min(p.k, (L + PBS - 1) / PBS);
    int end = (entries + PAIR - 1) / PAIR;                  // inclusive scan
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, end, o);
        if (lane >= o) end += x;
    }
    const int total = __shfl_sync(kFull, end, 31);
    if (lane == 0) border[0] = 0;
    border[lane + 1] = end;                                 // rows past nrows: empty
    length[lane] = L;
    // ---- this warp's run of them
    const int share = (total + csize * NW - 1) / (csize * NW);
    const int begin = min(total, (rank * NW + w) * share), stop = min(total, begin + share);
    const int nk = stop - begin;

    if (lane < ST) mbar_init(smem_addr(&bars[lane]), 1);
    fence_mbar_init();
    __syncwarp();
    const uint64_t pol = l2_evict_first();
    // the tile of entry e of row r (-1: none) and its tokens; j, before: the entry and
    // the one in front of it
    auto tile_of = [&](int r, int e, int j, int before, int* ntok) -> int {
        *ntok = 0;
        const int len = length[r], nblk = (len + PBS - 1) / PBS;
        if (e >= min(p.k, nblk) || j < 0) return -1;        // past the list, padding
        // past the sequence, repeated or out of order, or behind padding
        if (j >= nblk || j <= before || (e > 0 && before < 0)) {
            flag_error(p.err, kErrOutOfRange);
            return -1;
        }
        const unsigned b = (unsigned)(row0 + r) / (unsigned)p.num_kv_heads;
        const int id = p.block_tables[(size_t)b * p.max_blocks + j];
        if (id < 0 || id >= p.num_blocks) {
            flag_error(p.err, kErrOutOfRange);
            return -1;
        }
        *ntok = min(PBS, len - j * PBS);
        return id * p.num_kv_heads + (row0 + r - (int)b * p.num_kv_heads);
    };
    // 32 stages per warp-wide read: tiles and tokens
    int id_a = -1, id_b = -1, tok_a = 0, tok_b = 0, chunk = -1;
    auto issue = [&](int kk, int s) {                       // stage kk into slot s: the whole converged warp
        if ((kk >> 5) != chunk) {
            chunk = kk >> 5;
            const int at = begin + (chunk << 5) + lane;
            id_a = id_b = -1;
            tok_a = tok_b = 0;
            if (at < stop) {
                int r = 0;
                while (border[r + 1] <= at) ++r;
                const int e = (at - border[r]) * PAIR;
                const int32_t* list = p.selected + (size_t)(row0 + r) * p.k + e;
                const int before = e > 0 ? list[-1] : -1, j0 = list[0], j1 = PAIR == 2 && e + 1 < p.k ? list[1] : -1;
                id_a = tile_of(r, e, j0, before, &tok_a);
                if constexpr (PAIR == 2) {
                    id_b = tile_of(r, e + 1, j1, j0, &tok_b);
                    if (id_a < 0) {                         // a lone second entry moves up
                        id_a = id_b;
                        tok_a = tok_b;
                        id_b = -1;
                        tok_b = 0;
                    }
                }
            }
            __syncwarp();
        }
        const uint32_t bar = smem_addr(&bars[s]);
        const int ia = __shfl_sync(kFull, id_a, kk & 31), ta = __shfl_sync(kFull, tok_a, kk & 31);
        const int ib = PAIR == 2 ? __shfl_sync(kFull, id_b, kk & 31) : -1;
        const int tb = PAIR == 2 ? __shfl_sync(kFull, tok_b, kk & 31) : 0;
        if (lane == 0) stage_tok[s] = ta + tb;
        __syncwarp();
        if (ia >= 0) {
            const uint32_t dst = smem_addr(ring + (size_t)s * 2 * TILE);
            const size_t off = (size_t)ia * PTILE;
            mbar_arrive_expect_tx_elect(bar, (ib >= 0 ? 4 : 2) * PTILE);
            bulk_g2s_elect(dst, p.k_pool + off, PTILE, bar, pol);
            bulk_g2s_elect(dst + TILE, p.v_pool + off, PTILE, bar, pol);
            if (ib >= 0) {
                const size_t off2 = (size_t)ib * PTILE;
                bulk_g2s_elect(dst + PTILE, p.k_pool + off2, PTILE, bar, pol);
                bulk_g2s_elect(dst + TILE + PTILE, p.v_pool + off2, PTILE, bar, pol);
            }
        } else {
            mbar_arrive_elect(bar);
        }
    };
    for (int kk = 0; kk < nk && kk < ST; ++kk) issue(kk, kk);
    // ---- one row: every CTA will merge a slice of it, the same quads of every warp's part
    if (p.push) {
        if (tid == 0) {
            const uint32_t recv = smem_addr(rings + NW * warp_ring);
            mbar_init(recv, 1);
            fence_mbar_init();                             // releases it to the cluster
            const int active = share > 0 ? (total + share - 1) / share : 0;
            if (active > 1) mbar_arrive_expect_tx(recv, active * (S::kQuads / csize * 16 + max(1, G / csize) * 8));
        }
        __syncwarp();
        cluster_arrive_relaxed();                          // the others may push from here on
    }

    typename Math::State st;
    int row = -1, row_end = begin;                          // the current row ends before stage row_end
    // the current row's result: whole, or this warp's part of it
    auto finish_row = [&](bool dead) {
        if (row < 0) return;
        const bool first_here = border[row] >= begin, last_here = border[row + 1] <= stop;
        if (first_here && last_here) {
            if (!dead)
                write_row<Math, QT, D, G>(st, static_cast<QT*>(p.out) + (size_t)(row0 + row) * G * D, p.v_scale, lane);
        } else {
            float* part = first_here ? reinterpret_cast<float*>(ring) : part0 + w * S::kPartFloats;
            Math::finish(st, part, part + G, part + S::kO, 0, lane, dead);
        }
    };
    bool aborted = false;
    int k = 0, s = 0;                                       // stage, its slot
    uint32_t phase = 0;                                     // how often the ring has gone round, mod 2
    for (; k < nk; ++k) {
        if (begin + k >= row_end) {                         // the next row
            finish_row(false);
            do ++row;
            while (border[row + 1] <= begin + k);
            row_end = border[row + 1];
            begin_row<Math, QT, D, G>(st, static_cast<const QT*>(p.q) + (size_t)(row0 + row) * G * D, p.qscale, qs, lane);
        }
        const bool ok = mbar_wait_bounded(smem_addr(&bars[s]), phase, p.err);
        if (__any_sync(kFull, !ok)) {
            aborted = true;
            break;
        }
        const int ntok = stage_tok[s];
        if (ntok > 0) {
            unsigned char* kt = ring + (size_t)s * 2 * TILE;
            if constexpr (Math::kWarpSmemFloats > 0) {
                Math::tile(st, kt, kt + TILE, ntok, lane, qs, pb);
            } else {
                if (ntok < BS) Math::clear_tail(kt + TILE, ntok, lane);
                Math::tile(st, kt, kt + TILE, ntok, lane, p.qscale);
            }
        }
        __syncwarp();
        if (k + ST < nk) {
            fence_proxy_async_smem();
            issue(k + ST, s);
        }
        if (++s == ST) {
            s = 0;
            phase ^= 1;
        }
    }
    if (aborted) {
        // as in the decode kernel: record it and let the copies in flight land; the
        // parts that the partners will read are marked empty
        if (lane == 0) flag_error(p.err, kErrTimeout);
        for (int kk = k; kk < min(nk, k + ST); ++kk) {
            (void)mbar_wait_bounded(smem_addr(&bars[s]), phase, nullptr);
            if (++s == ST) {
                s = 0;
                phase ^= 1;
            }
        }
        for (int i = lane; i < 2 * G; i += 32) {              // m, l
            reinterpret_cast<float*>(ring)[i] = i < G ? -INFINITY : 0.f;
            part0[w * S::kPartFloats + i] = i < G ? -INFINITY : 0.f;
        }
        __syncwarp();
    }
    finish_row(aborted);

    constexpr int kQuads = S::kQuads;                       // a thread's share: four elements
    QT* const out = static_cast<QT*>(p.out) + (size_t)row0 * G * D;
    auto store4 = [&](int r, int i, float4 v, float by) {
        QT* dst = out + (size_t)r * G * D + 4 * i;
        if constexpr (std::is_same<QT, float>::value)
            *reinterpret_cast<float4*>(dst) = make_float4(v.x * by, v.y * by, v.z * by, v.w * by);
        else
            *reinterpret_cast<uint2*>(dst) = make_uint2(decode::pack_bf16(v.x * by, v.y * by), decode::pack_bf16(v.z * by, v.w * by));
    };
    auto add4 = [](float4& v, float e, float4 o) {
        v.x += e * o.x;
        v.y += e * o.y;
        v.z += e * o.z;
        v.w += e * o.w;
    };
    // ---- one row: every warp pushes each CTA its slice of its part, one trip through
    // the cluster instead of two barriers around a read (1 sequence, 8 rows of 128 blocks:
    // 0.7 us less than with the barriers, of 7.1; 16 blocks: 0.8 of 5.8)
    if (p.push) {
        __syncwarp();
        cluster_wait();                                    // every CTA's mbarrier is up
        const int active = share > 0 ? (total + share - 1) / share : 0;   // warps with a run
        if (active <= 1) {                                 // written by its warp, or nothing listed
            if (active == 0)
                for (int i = rank * NW * 32 + tid; i < kQuads; i += csize * NW * 32)
                    store4(0, i, make_float4(0.f, 0.f, 0.f, 0.f), 0.f);
            return;
        }
        // all of these are powers of two
        const int cbits = __ffs(csize) - 1, slice = kQuads >> cbits, sbits = __ffs(slice) - 1;
        const int heads = max(1, G >> cbits);              // whose m, l a slice needs
        const int slot_bytes = (slice + (heads + 1) / 2) * 16;
        const uint32_t recv = smem_addr(rings + NW * warp_ring);
        if (nk > 0) {
            const float* part = begin == 0 ? reinterpret_cast<const float*>(ring) : part0 + w * S::kPartFloats;
            const uint32_t slot = recv + 16 + (rank * NW + w) * slot_bytes;
            __syncwarp();
            const int hbits = __ffs(heads) - 1, hy = lane >> hbits, hx = lane & (heads - 1), hg = ((hy * G) >> cbits) + hx;
            if (hy < csize)
                push2(cluster_map(slot + slice * 16 + hx * 8, hy), part[hg], part[G + hg], cluster_map(recv, hy));
#pragma unroll 1
            for (int i = lane; i < kQuads; i += 32)
                push4(cluster_map(slot + (i & (slice - 1)) * 16, i >> sbits),
                      *reinterpret_cast<const float4*>(part + S::kO + 4 * i), cluster_map(recv, i >> sbits));
        }
        if (__syncthreads_or(!pushed_wait_bounded(recv, p.err))) {
            // the partners may still push: leave after they have, and after it has landed
            if (tid == 0) flag_error(p.err, kErrTimeout);
            cluster_sync_relaxed();
            (void)pushed_wait_bounded(recv, nullptr);
            return;
        }
        // J lanes a quad, each over every J-th warp's part
        const int jbits = max(0, min(5, __ffs(NW) + 4 - sbits)), J = 1 << jbits, quad = tid >> jbits, x0 = tid & (J - 1);
        const int q = min(quad, slice - 1), i = rank * slice + q, g = 4 * i / D - ((rank * G) >> cbits);
        const unsigned char* const at = rings + NW * warp_ring + 16;
        auto ml_of = [&](int x) { return *reinterpret_cast<const float2*>(at + x * slot_bytes + slice * 16 + g * 8); };
        float M = -INFINITY, sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int x = x0; x < active; x += J) M = max_nan(M, ml_of(x).x);
#pragma unroll 1
        for (int o = 1; o < J; o <<= 1) M = max_nan(M, __shfl_xor_sync(kFull, M, o));
        M = softmax_base(M);                               // nothing but empty parts
#pragma unroll 4
        for (int x = x0; x < active; x += J) {
            const float2 ml = ml_of(x);
            const float e = ex2(ml.x - M);
            sum += e * ml.y;
            add4(v, e, *reinterpret_cast<const float4*>(at + x * slot_bytes + q * 16));
        }
#pragma unroll 1
        for (int o = 1; o < J; o <<= 1) {
            sum += __shfl_xor_sync(kFull, sum, o);
            v.x += __shfl_xor_sync(kFull, v.x, o);
            v.y += __shfl_xor_sync(kFull, v.y, o);
            v.z += __shfl_xor_sync(kFull, v.z, o);
            v.w += __shfl_xor_sync(kFull, v.w, o);
        }
        if (quad < slice && x0 == 0) store4(0, i, v, sum > 0.f ? p.v_scale / sum : 0.f);
        return;
    }

    // ---- the rows that several warps of this CTA share: to the output, or (a row
    // that reaches into other CTAs of the cluster) to the CTA's part of it. Rolled
    // loops: this runs once, and fetching straight-line code costs more than it saves.
    __syncthreads();
    const int cta_run = NW * share, cta_begin = min(total, rank * cta_run), cta_stop = min(total, cta_begin + cta_run);
    float* const cta_part = reinterpret_cast<float*>(rings + warp_ring / 2);
    const int cta_part1 = warp_ring / 4;                    // floats from the first to the last
    if (cta_begin < cta_stop) {
        int r = 0;
        while (border[r + 1] <= cta_begin) ++r;
#pragma unroll 1
        for (; border[r] < cta_stop; ++r) {
            const int a = border[r], z = border[r + 1];
            if (a == z) continue;
            const int x0 = max(a - cta_begin, 0) / share, x1 = (min(z, cta_stop) - 1 - cta_begin) / share;
            const bool whole = a >= cta_begin && z <= cta_stop;
            if (whole && x0 == x1) continue;                // written by its warp
            float* const to = cta_part + (a < cta_begin ? 0 : cta_part1);
            // warp x's part: its first where the row began before its run, else its last
            auto part_of = [&](int x) -> const float* {
                return a < cta_begin + x * share ? part0 + x * S::kPartFloats
                                                 : reinterpret_cast<const float*>(rings + x * warp_ring);
            };
#pragma unroll 1
            for (int i = tid; i < kQuads; i += NW * 32) {
                const int g = 4 * i / D;
                float M = -INFINITY, sum = 0.f;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int x = x0; x <= x1; ++x) M = max_nan(M, part_of(x)[g]);
                if (M != -INFINITY) {
#pragma unroll 4
                    for (int x = x0; x <= x1; ++x) {
                        const float* part = part_of(x);
                        const float e = exp2f(part[g] - M);
                        sum += e * part[G + g];
                        add4(v, e, *reinterpret_cast<const float4*>(part + S::kO + 4 * i));
                    }
                }
                if (whole) {
                    store4(r, i, v, sum > 0.f ? p.v_scale / sum : 0.f);
                } else {
                    *reinterpret_cast<float4*>(to + S::kO + 4 * i) = v;
                    if (4 * i % D == 0) {
                        to[g] = M;
                        to[G + g] = sum;
                    }
                }
            }
        }
    }
#pragma unroll 1
    for (int r = rank; r < nrows; r += csize)               // rows with nothing listed
        if (border[r] == border[r + 1])
            for (int i = tid; i < kQuads; i += NW * 32) store4(r, i, make_float4(0.f, 0.f, 0.f, 0.f), 0.f);
    if (csize == 1) return;
    // ---- the rows that several CTAs share (at most the first and the last of this
    // one's): each CTA takes a slice of a row's elements
    cluster_sync();
    if (cta_begin < cta_stop) {
        int r = 0;
        while (border[r + 1] <= cta_begin) ++r;
#pragma unroll 1
        for (; border[r] < cta_stop; ++r) {
            const int a = border[r], z = border[r + 1];
            if (a >= cta_begin && z <= cta_stop) continue;
            const int y0 = a / cta_run, n = (z - 1) / cta_run - y0 + 1;      // its CTAs
            const int slice = (kQuads + n - 1) / n, from = (rank - y0) * slice;
            auto part_of = [&](int y) {
                return cluster_map(smem_addr(cta_part + (a < (y0 + y) * cta_run ? 0 : cta_part1)), y0 + y);
            };
#pragma unroll 1
            for (int i = from + tid; i < min(kQuads, from + slice); i += NW * 32) {
                const int g = 4 * i / D;
                // every CTA's part read at once: one trip through the cluster
                float m[kMaxCluster], l[kMaxCluster], M = -INFINITY, sum = 0.f;
                float4 o[kMaxCluster], v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int y = 0; y < kMaxCluster; ++y) {
                    const uint32_t at = part_of(min(y, n - 1));
                    m[y] = cluster_ld(at + g * 4);
                    l[y] = cluster_ld(at + (G + g) * 4);
                    o[y] = cluster_ld4(at + (S::kO + 4 * i) * 4);
                }
#pragma unroll
                for (int y = 0; y < kMaxCluster; ++y) M = max_nan(M, m[y]);
                if (M != -INFINITY) {
#pragma unroll
                    for (int y = 0; y < kMaxCluster; ++y) {
                        if (y < n) {
                            const float e = exp2f(m[y] - M);
                            sum += e * l[y];
                            add4(v, e, o[y]);
                        }
                    }
                }
                store4(r, i, v, sum > 0.f ? p.v_scale / sum : 0.f);
            }
        }
    }
    cluster_sync_relaxed();                                 // partners are done reading
}

// Clusters of `size` CTAs that fit on the current device at once (cached).
int resident_clusters(const void* kern, int smem, int threads, int size, int* out);

template <class Math, typename QT, int D, int BS, int G, int PAIR>
int launch(const Args& a) {
    using S = Smem<Math, D, BS, G>;
    auto kern = sparse_decode_kernel<Math, QT, D, BS, G, PAIR>;
    const void* fn = reinterpret_cast<const void*>(kern);
    // three CTAs an SM where their rings fit; alone on its SM a CTA gets a deep ring
    constexpr int kStages3 = S::stages(kNumWarps, kSmemSm / 3 - 1024);
    constexpr int kWideWarps = S::kWide ? 2 * kNumWarps : kNumWarps;
    constexpr int kRecv = S::recv_bytes(kWideWarps);
    constexpr int kStages1 = S::stages(kWideWarps, kSmemSm - kRecv);
    constexpr int kSmem1 = S::bytes(kWideWarps, kStages1) + kRecv, kSmem3 = S::bytes(kNumWarps, kStages3);
    constexpr int kMost = kSmem1 > kSmem3 ? kSmem1 : kSmem3;
    static_assert(kMost <= kSmemSm, "shared memory per CTA");
    int occ = 0;
    int st = kernel_setup(fn, kMost, kNumWarps * 32, &occ);
    if (st != PKV_OK) return st;
    const int stages = ((a.p.k < a.p.max_blocks ? a.p.k : a.p.max_blocks) + PAIR - 1) / PAIR;
    const long long rows = (long long)a.num_seqs * a.p.num_kv_heads;
    int size = 1, per = 1, warps = kNumWarps, depth = kStages3, smem = kSmem3;
    if (2 * rows <= num_sms()) {
        // few rows: each to as many warps as have a stage, one CTA an SM
        warps = kWideWarps;
        depth = kStages1;
        smem = kSmem1;
        for (int s = kMaxCluster; s > 1; s /= 2) {
            if (s * rows > num_sms() || s * warps > stages) continue;
            int fit = 0;
            st = resident_clusters(fn, smem, warps * 32, s, &fit);
            if (st != PKV_OK) return st;
            if (fit >= rows) {
                size = s;
                break;
            }
        }
    } else {
        // a CTA a row, in waves; or one wave of clusters that share their rows evenly,
        // where that leaves the fullest CTA a fifth less (512 rows of 128 E4M3 blocks,
        // on 456 places: 67 us in waves of whole rows, 56 us by fours)
        int fit = 0;
        st = resident_clusters(fn, smem, warps * 32, 1, &fit);
        if (st != PKV_OK) return st;
        double best = 0.8 * (double)((rows + fit - 1) / fit);
        for (int s = 2; s <= kMaxCluster; s *= 2) {
            st = resident_clusters(fn, smem, warps * 32, s, &fit);
            if (st != PKV_OK) return st;
            const long long r = fit > 0 ? (rows + fit - 1) / fit : kMaxRows + 1;
            if (r > kMaxRows || r * stages < 2LL * s * warps) continue;
            const double load = (double)r / s;
            if (load < best) {
                best = load;
                size = s;
                per = (int)r;
            }
        }
    }
    const long long ctas = (rows + per - 1) / per * size;
    Params p = a.p;
    p.num_rows = (int)rows;
    p.cluster_rows = per;
    p.stages = depth;
    p.push = 2 * rows <= num_sms() && size > 1;
    p.qscale = a.scale * a.k_scale * kLog2e;
    p.v_scale = a.v_scale;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    note_launch();
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    return e == cudaSuccess ? PKV_OK : cuda_fail("sparse decode: kernel launch", e);
}

// CUDA-core math: the decode's with a logit's products in four sums (by the place in the
// 16-byte chunk) instead of one chain of D / 2 or D, and with infinite and NaN logits as
// above. Of float32 caches with 128 dims and 32-token blocks the outputs' error against 64
// bits falls from 1.1e-6 to half of that.
template <typename QT, typename KV, int D, int BS, int G>
struct SimtSums : decode::SimtMath<QT, KV, D, BS, G> {
    using Base = decode::SimtMath<QT, KV, D, BS, G>;
    using typename Base::Lay;
    using typename Base::State;
    using Base::CPP;
    using Base::CR;
    using Base::DPL;
    using Base::PASSES;
    using Base::X;

    template <class Sink = NoSink>
    __device__ __forceinline__ static void tile(State& st, const unsigned char* kt, const unsigned char* vt,
                                                int ntok, int lane, const float* qs, float* pb,
                                                const Sink& sink = Sink()) {
        const int t = lane % BS, cp = lane / BS;
        float s4[G][4];
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int x = 0; x < 4; ++x) s4[g][x] = 0.f;
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int j = i * CPP + cp;
            float kf[X];
            decode::unpack(*reinterpret_cast<const uint4*>(kt + Lay::k_off(j, t)), kf);
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int x = 0; x < X; ++x) {
                    const float qv = Base::kQRegs ? st.qr[Base::kQRegs ? i * X + x : 0] : qs[g * D + j * X + x];
                    s4[g][x & 3] = fmaf(qv, kf[x], s4[g][x & 3]);
                }
        }
        float alpha[G];
        bool moved = false;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float s = (s4[g][0] + s4[g][1]) + (s4[g][2] + s4[g][3]);
            if constexpr (CPP == 2) s += __shfl_xor_sync(kFull, s, 16);
            if (t >= ntok) s = -INFINITY;
            if (cp == 0) sink.put(g, t, s);
            float mx = s;
#pragma unroll
            for (int o = BS / 2; o >= 1; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(kFull, mx, o));
            const float m_new = max_nan(st.m[g], mx), base = softmax_base(m_new);
            alpha[g] = exp2f(st.m[g] - base);
            const float pv = exp2f(s - base);
            st.m[g] = m_new;
            st.l[g] = st.l[g] * alpha[g] + (cp == 0 ? pv : 0.f);
            if (cp == 0) pb[g * BS + t] = pv;
            moved |= alpha[g] != 1.f;
        }
        __syncwarp();
        if (__any_sync(kFull, moved)) {                    // running max moved
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int k = 0; k < DPL; ++k) st.acc[g][k] *= alpha[g];
        }
#pragma unroll
        for (int ch = 0; ch < CR; ++ch) {
            if (ch * X >= ntok) break;
#pragma unroll
            for (int k = 0; k < DPL; ++k) {
                float vf[X];
                decode::unpack(*reinterpret_cast<const uint4*>(vt + Lay::v_off(lane + 32 * k, ch)), vf);
#pragma unroll
                for (int x = 0; x < X; ++x)
                    if (ch * X + x >= ntok) vf[x] = 0.f;   // unwritten slots
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int x = 0; x < X; x += 4) {
                        const float4 pp = *reinterpret_cast<const float4*>(pb + g * BS + ch * X + x);
                        st.acc[g][k] = fmaf(pp.x, vf[x], st.acc[g][k]);
                        st.acc[g][k] = fmaf(pp.y, vf[x + 1], st.acc[g][k]);
                        st.acc[g][k] = fmaf(pp.z, vf[x + 2], st.acc[g][k]);
                        st.acc[g][k] = fmaf(pp.w, vf[x + 3], st.acc[g][k]);
                    }
            }
        }
        __syncwarp();
    }
};

// float32 caches on CUDA cores, as in the decode; bf16 caches on the tensor cores for 2, 4,
// 8 query heads a kv head, on CUDA cores for one, whose weights then stay float32 (1280
// rows of 64 blocks: 94.5 us, 0.96 of the copy rate; 91.8 on the tensor cores with weights
// of one bf16 number); E4M3 caches on the tensor cores, for one head too (512 rows of 128
// blocks: 56.0 us on CUDA cores, 45.5 so); their tiles of 16 tokens two a stage.
template <typename QT, typename KV, int D, int BS, int G>
int launch_heads(const Args& a) {
    if constexpr (std::is_same<KV, float>::value || (G == 1 && !std::is_same<KV, uint8_t>::value))
        return launch<SimtSums<QT, KV, D, BS, G>, QT, D, BS, G, 1>(a);
    else if constexpr (BS == 16 && std::is_same<KV, uint8_t>::value)
        return launch<HeadsMath<KV, D, 2 * BS, G>, QT, D, 2 * BS, G, 2>(a);
    else return launch<HeadsMath<KV, D, BS, G>, QT, D, BS, G, 1>(a);
}

template <typename QT, typename KV, int D, int BS>
int dispatch_group(const Args& a) {
    switch (a.p.num_heads / a.p.num_kv_heads) {
        case 1: return launch_heads<QT, KV, D, BS, 1>(a);
        case 2: return launch_heads<QT, KV, D, BS, 2>(a);
        case 4: return launch_heads<QT, KV, D, BS, 4>(a);
        case 8: return launch_heads<QT, KV, D, BS, 8>(a);
        default: return PKV_ERR_UNSUPPORTED;
    }
}

template <typename QT, typename KV>
int dispatch(const Args& a) {
    if (a.head_dim == 64 && a.block_size == 16) return dispatch_group<QT, KV, 64, 16>(a);
    if (a.head_dim == 64 && a.block_size == 32) return dispatch_group<QT, KV, 64, 32>(a);
    if (a.head_dim == 128 && a.block_size == 16) return dispatch_group<QT, KV, 128, 16>(a);
    if (a.head_dim == 128 && a.block_size == 32) return dispatch_group<QT, KV, 128, 32>(a);
    return PKV_ERR_UNSUPPORTED;
}

}  // namespace sparse
}  // namespace pkv
