// weigh_prefill_tokens: the attention weight that every cached token gets from the last
// queries of a prefill chunk, on the fifth-generation tensor cores (tcgen05).
//
// Mathematics. With the rows r = (query, head of the kv head's group) and s[r][t] their
// logits in units of log2 e, a token's gain is sum_r 2^(s[r][t] - M_r), M_r = max_t s[r][t] +
// log2(sum_t 2^(s[r][t] - max)). M_r needs every token of the row, the gain every row of the
// token: two passes over the products Q K^T, none over V, and no logit leaves the chip (a
// stored one would cost more bytes than the key it comes from).
//
// First pass (stats): A = 128 query rows, B = 128 keys, so a thread owns a row (a lane of
// tensor memory) and its maximum and sum run along the thread's own columns. Second pass
// (gain): the operands change places, A = 128 keys, B = 128 rows: a thread owns a token, and
// the sum over the rows again runs along its own columns. Both operands lie in shared memory
// in the same K-major core matrices (the cache's own tiles; the rows, which the first pass
// also writes to the workspace so), so the second pass only exchanges two descriptors, and
// neither pass reduces across threads.
//
// Work split. Stats: a CTA holds a row tile and streams a run of the key tiles (several CTAs a
// row tile where there are few). Gain: with one row tile a kv head (a short window) a CTA
// holds it and streams key tiles; with more, it holds a key tile and streams the row tiles
// that see it. Warps 0-3: one thread a lane of tensor memory; warp 4 issues the products, warp
// 5 the copies; two buffers for the streamed operand and for the products, so the tensor
// cores work on the next tile while the exponentials of this one are taken. Two CTAs an SM.
#include <cmath>

#include <cuda_bf16.h>

#include "pkv_check.cuh"
#include "pkv_internal.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace weigh {

constexpr int kTile = 128;             // rows, keys of a tile
constexpr int kThreads = 320;
constexpr int kMmaWarp = 8, kLoadWarp = 9;               // warps 0-3, 4-7: a lane of tensor memory a thread
constexpr uint32_t kTmemCols = 256;    // two products
constexpr uint32_t kIdesc = tc::idesc_bf16_f32(kTile, kTile);
constexpr int kTargetCtas = 608;       // of the stats pass: two waves of two CTAs an SM
constexpr int kMaxGroup = 128;

struct Params {
    float* weights;
    const int32_t* rows;
    const __nv_bfloat16* q;
    const __nv_bfloat16* k_pool;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* query_start;
    unsigned char* q_tiles;            // [items][row_tiles] tiles of 128 rows, core matrices
    float2* stats;                     // [items][row_tiles][splits][128] maximum, sum
    int* err;
    int num_seqs, max_query_len, window, max_blocks, num_blocks, num_rows, max_tokens;
    int num_heads, num_kv_heads, G, row_tiles, splits, key_tiles, per;
    float scale_log2, decay;           // the scale's magnitude,
    uint32_t q_sign;                   // and what turns its sign on pairs of query elements
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Two float32 numbers an instruction
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
        "r"(bytes), "r"(bar)
        : "memory");
}
// The four warps of a warpgroup; both of them
__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }
__device__ __forceinline__ void groups_sync() { asm volatile("bar.sync 3, 256;" ::: "memory"); }

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
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float cluster_ld(const float* p, uint32_t rank) {
    uint32_t a;
    float v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// One sequence's chunk, or w == 0: nothing to do
struct Chunk {
    int L, C, w, q_first;              // q_first: row of q of the first query that counts
    __device__ __forceinline__ Chunk(const Params& p, int b, int bs, bool flag) {
        L = p.seq_lens[b];
        const int q0 = p.query_start[b], q1 = p.query_start[b + 1], T = p.query_start[p.num_seqs];
        C = q1 - q0;
        w = p.window > 0 && p.window < C ? p.window : C;
        if (C < 0 || C > L || L > p.max_blocks * bs || q0 < 0 || q1 > T || C > p.max_query_len) {
            if (flag && C != 0) flag_error(p.err, kErrOutOfRange);
            w = 0;
        }
        q_first = q1 - w;
    }
};

enum : int { kBarHeld = 0, kBarFull = 1, kBarDone = 3, kBarRead = 5, kBarDrain = 7, kNumBars };

// The pipeline both passes share: tile i of the stream, i < n, goes through buffer i % 2.
// `load(i, dst, bar)`: the loading warp arms `bar` and sends tile i's copies. `use(i, taddr)`:
// the lanes' warps read their products and return; held_is_a: the held tile is A.
template <int D>
struct Pipe {
    static constexpr int kTileBytes = kTile * D * 2, kGroup = D / 8 * 128;   // 8 rows
    static constexpr int kSmem = 3 * kTileBytes;                             // held | streamed x 2

    uint32_t sbase, bar0, tmem;
    const int* err;

    __device__ __forceinline__ uint32_t bar(int i) const { return bar0 + 8u * (uint32_t)i; }
    __device__ __forceinline__ static void init(uint32_t bar0) {             // one thread
        auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
        mbar_init(bar(kBarHeld), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kBarFull + i), 1);
            mbar_init(bar(kBarDone + i), 1);
            mbar_init(bar(kBarRead + i), 128);
        }
        mbar_init(bar(kBarDrain), 1);
        fence_mbar_init();
    }
    template <class Load>
    __device__ __forceinline__ void run_load(int n, int lane, bool held, Load load) const {
        int sent = 0;
        bool ok = true;
        for (int i = 0; i < n && ok; ++i) {
            if (i >= 2) ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarDone + (i & 1)), ((i - 2) >> 1) & 1, err));
            if (!ok) break;
            load(i, sbase + (1 + (i & 1)) * kTileBytes, bar(kBarFull + (i & 1)));
            sent = i + 1;
        }
        // every copy lands before the CTA may exit
        for (int i = max(0, sent - 2); i < sent; ++i) (void)mbar_wait_bounded(bar(kBarFull + (i & 1)), (i >> 1) & 1, nullptr);
        if (held) (void)mbar_wait_bounded(bar(kBarHeld), 0, nullptr);
    }
    __device__ __forceinline__ void run_mma(int n, int lane, bool held, bool held_is_a) const {
        bool ok = true;
        auto wait = [&](int b, int parity) { ok = __all_sync(0xffffffffu, ok && mbar_wait_bounded(bar(b), parity, err)); };
        if (held) wait(kBarHeld, 0);
        constexpr uint32_t hi = tc::desc_hi(kGroup);
        const uint32_t h_lo = tc::desc_lo(sbase, 128);
        for (int i = 0; i < n && ok; ++i) {
            const int s = i & 1;
            wait(kBarFull + s, (i >> 1) & 1);
            if (i >= 2) wait(kBarRead + s, ((i - 2) >> 1) & 1);
            if (!ok) break;
            tc::fence_after_sync();
            const uint32_t s_lo = tc::desc_lo(sbase + (1 + s) * kTileBytes, 128);
            const uint32_t a = held_is_a ? h_lo : s_lo, b = held_is_a ? s_lo : h_lo;
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                tc::mma_ss2_elect(tmem + s * kTile, a + k * 16, hi, b + k * 16, hi, kIdesc, k > 0);
            tc::commit_elect(bar(kBarDone + s));
        }
        if (!ok && lane == 0) flag_error(const_cast<int*>(err), kErrTimeout);
        tc::commit_elect(bar(kBarDrain));                  // all of them complete before tensor memory goes
        (void)mbar_wait_bounded(bar(kBarDrain), 0, nullptr);
        __syncwarp();
    }
    // Products of stream tile i, 32 columns at a time: use(column, values). False: a wait gave up.
    template <class Use>
    __device__ __forceinline__ bool take(int i, int warp, Use use) const {
        const int s = i & 1;
        const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarDone + s), (i >> 1) & 1, err));
        if (!ok) return false;
        tc::fence_after_sync();
        const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + s * kTile;
        uint32_t v[2][32];
        tc::ld32(at, v[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            tc::wait_ld();
            if (c < 3) tc::ld32(at + 32 * (c + 1), v[(c + 1) & 1]);
            else {
                tc::fence_before_sync();
                mbar_arrive(bar(kBarRead + s));
            }
            use(32 * c, v[c & 1]);
        }
        return true;
    }
};

// Key tile j of a sequence into shared memory; blocks that are not in the pool are read from
// block 0 (what comes of them is left out by those who use them).
template <int D, int BS>
__device__ __forceinline__ void load_keys(const Params& p, int b, int hk, int L, int j, int lane, uint32_t dst, uint32_t bar) {
    constexpr int kBlocks = kTile / BS, kBytes = BS * D * 2;
    const int first = j * kBlocks, n = min(kBlocks, (L + BS - 1) / BS - first);
    int id = 0;
    if (lane < n) {
        id = p.block_tables[(size_t)b * p.max_blocks + first + lane];
        if (id < 0 || id >= p.num_blocks) {
            flag_error(p.err, kErrOutOfRange);
            id = 0;
        }
    }
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(n * kBytes));
    __syncwarp();
    if (lane < n)
        bulk_load(dst + lane * kBytes, p.k_pool + ((size_t)id * p.num_kv_heads + hk) * (BS * D), kBytes, bar);
}

template <int D, int BS>
__global__ void __launch_bounds__(kThreads, 2) weigh_stats_kernel(const Params p) {
    pdl_enter();
    using P = Pipe<D>;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(8) uint64_t bars[kNumBars];
    __shared__ uint32_t tmem_slot;
    __shared__ float2 other[kTile];                        // the second warpgroup's statistics
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = blockIdx.x, rt = blockIdx.y, item = blockIdx.z, b = item / p.num_kv_heads, hk = item - b * p.num_kv_heads;
    const Chunk ch(p, b, BS, tid == 0);
    const int r0 = rt * kTile, nr = ch.w * p.G;
    if (r0 >= nr) return;                                  // the whole CTA
    const int p_min = ch.L - ch.w + r0 / p.G, p_max = ch.L - ch.w + (min(nr, r0 + kTile) - 1) / p.G;
    const int tiles = p_max / kTile + 1, per = (tiles + p.splits - 1) / p.splits;
    const int k0 = split * per, n = min(tiles, k0 + per) - k0;
    if (n <= 0) return;
    // blocks that are not in the pool: rare, so the lanes look them up themselves then
    constexpr int kBlocks = kTile / BS;
    const int32_t* const table = p.block_tables + (size_t)b * p.max_blocks;
    bool bad = false;
    for (int i = k0 * kBlocks + tid; i < min((k0 + n) * kBlocks, p_max / BS + 1); i += kThreads)
        bad |= table[i] < 0 || table[i] >= p.num_blocks;
    P pipe;
    pipe.sbase = smem_addr(smem);
    pipe.bar0 = smem_addr(bars);
    pipe.err = p.err;
    if (tid == 0) P::init(pipe.bar0);
    if (warp == kMmaWarp) {
        tc::alloc(smem_addr(&tmem_slot), kTmemCols);
        tc::relinquish_alloc_permit();
    }
    if (warp < 8) {                                        // half a row: to shared memory and the workspace
        const int r = r0 + (tid & 127), c0 = (tid >> 7) * (D / 16);
        const bool valid = r < nr;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + ((size_t)(ch.q_first + (valid ? r / p.G : 0)) * p.num_heads + hk * p.G + (valid ? r % p.G : 0)) * D);
        const int at = ((tid & 127) >> 3) * P::kGroup + (tid & 7) * 16;
        unsigned char* const to = p.q_tiles + ((size_t)item * p.row_tiles + rt) * P::kTileBytes + at;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const int c = c0 + i;
            uint4 v = valid ? src[c] : make_uint4(0, 0, 0, 0);
            v = make_uint4(v.x ^ p.q_sign, v.y ^ p.q_sign, v.z ^ p.q_sign, v.w ^ p.q_sign);
            *reinterpret_cast<uint4*>(smem + at + c * 128) = v;
            if (split == 0) *reinterpret_cast<uint4*>(to + c * 128) = v;
        }
        fence_proxy_async_smem();                          // to the tensor cores, behind the barrier
    }
    tc::fence_before_sync();
    const bool any_bad = __syncthreads_or(bad);
    tc::fence_after_sync();
    pipe.tmem = tmem_slot;
    if (warp == kLoadWarp) {
        pipe.run_load(n, lane, false, [&](int i, uint32_t dst, uint32_t bar) {
            load_keys<D, BS>(p, b, hk, p_max + 1, k0 + i, lane, dst, bar);
        });
    } else if (warp == kMmaWarp) {
        pipe.run_mma(n, lane, false, true);
    } else {
        const int group = warp >> 2, me = tid & 127;
        const int r = r0 + me, pr = ch.L - ch.w + min(r, nr - 1) / p.G;
        const uint64_t sc2 = f2(p.scale_log2, p.scale_log2);
        float m = -INFINITY, l = 0.f;                      // of the raw products; the scale is not negative
        bool ok = true;
        for (int i = group; i < n && ok; i += 2) {         // the groups take turns
            const int key0 = (k0 + i) * kTile;
            const bool masked = any_bad || key0 + kTile - 1 > p_min;
            ok = pipe.take(i, warp, [&](int c0, uint32_t (&v)[32]) {
                if (masked) {
                    constexpr uint32_t kNone = 0xff800000u;   // -infinity
#pragma unroll
                    for (int c = 0; c < 32; ++c) v[c] = key0 + c0 + c <= pr ? v[c] : kNone;
                    if (any_bad)
                        for (int s = 0; s < 32 / BS; ++s) {
                            const int blk = (key0 + c0) / BS + s;
                            const int id = blk <= p_max / BS ? table[blk] : 0;
                            if (id < 0 || id >= p.num_blocks)
#pragma unroll
                                for (int c = 0; c < 32; ++c) v[c] = c / BS == s ? kNone : v[c];
                        }
                }
                float m4[4] = {m, m, m, m};
#pragma unroll
                for (int c = 0; c < 32; c += 2)
                    m4[(c >> 1) & 3] = max_nan(m4[(c >> 1) & 3], __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
                const float mx = max_nan(max_nan(m4[0], m4[1], m4[2]), m4[3]);
                const float base = mx == -INFINITY ? 0.f : mx * p.scale_log2;
                const uint64_t nb2 = f2(-base, -base);
                uint64_t s2[2] = {0ull, 0ull};
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    float a, b;
                    f2_split(fma2(f2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), sc2, nb2), a, b);
                    s2[(c >> 1) & 1] = add2(s2[(c >> 1) & 1], f2(ex2(a), ex2(b)));
                }
                float a, b, c, d;
                f2_split(s2[0], a, b);
                f2_split(s2[1], c, d);
                l = fmaf(l, ex2(fmaf(m, p.scale_log2, -base)), (a + b) + (c + d));
                m = mx;
            });
        }
        if (!ok) flag_error(p.err, kErrTimeout);
        m = m == -INFINITY ? m : m * p.scale_log2;
        if (group == 1) other[me] = make_float2(m, l);
        groups_sync();
        if (group == 0) {
            const float2 o = other[me];
            const float mx = max_nan(m, o.x), base = mx == -INFINITY ? 0.f : mx;
            p.stats[(((size_t)item * p.row_tiles + rt) * p.splits + split) * kTile + me] =
                make_float2(mx, l * ex2(m - base) + o.y * ex2(o.x - base));
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::dealloc(pipe.tmem, kTmemCols);
    }
}

// kStreamKeys: one row tile, held, and p.per key tiles; else a key tile, held, and the row
// tiles that see it, every csize-th for each CTA of a cluster, whose gains meet in its first.
template <int D, int BS, bool kStreamKeys>
__global__ void __launch_bounds__(kThreads, 2) weigh_gain_kernel(const Params p) {
    pdl_enter();
    using P = Pipe<D>;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(8) uint64_t bars[kNumBars];
    __shared__ uint32_t tmem_slot;
    __shared__ __align__(16) float base[2][kTile];         // M_r of the row tile a warpgroup works on
    __shared__ float part[2][kTile];                       // gains of the second group, of the CTA
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = kStreamKeys ? 0 : (int)cluster_rank(), csize = kStreamKeys ? 1 : (int)cluster_size();
    // the items that the first pass read last come first: their keys may still be in L2
    const int item = gridDim.y - 1 - blockIdx.y, b = item / p.num_kv_heads, hk = item - b * p.num_kv_heads;
    const Chunk ch(p, b, BS, false);
    if (ch.w == 0) return;                                 // the whole cluster
    const int tiles = (ch.L + kTile - 1) / kTile, nr = ch.w * p.G, row_tiles = (nr + kTile - 1) / kTile;
    const int kt0 = kStreamKeys ? blockIdx.x * p.per : blockIdx.x / csize;
    if (kt0 >= tiles) return;
    const int first_pos = ch.L - ch.w;                     // of the first query that counts
    const int rt0 = kStreamKeys ? 0 : max(0, kt0 * kTile - first_pos) * p.G / kTile + rank;
    const int n = kStreamKeys ? min(p.per, tiles - kt0) : max(0, (row_tiles - rt0 + csize - 1) / csize);
    int to = b;
    bool lost = false;
    if (p.rows) {
        to = p.rows[b];
        lost = to < 0 || to >= p.num_rows;
        for (int i = tid; i < b; i += kThreads) lost |= p.rows[i] == to;
    }
    P pipe;
    pipe.sbase = smem_addr(smem);
    pipe.bar0 = smem_addr(bars);
    pipe.err = p.err;
    if (tid == 0) P::init(pipe.bar0);
    if (__syncthreads_or(lost)) {
        if (tid == 0) flag_error(p.err, kErrOutOfRange);
        return;
    }
    if (warp == kMmaWarp) {
        tc::alloc(smem_addr(&tmem_slot), kTmemCols);
        tc::relinquish_alloc_permit();
    }
    const unsigned char* const q_tiles = p.q_tiles + (size_t)item * p.row_tiles * P::kTileBytes;
    auto load_rows = [&](int rt, uint32_t dst, uint32_t bar) {
        if (lane == 0) {
            mbar_arrive_expect_tx(bar, P::kTileBytes);
            bulk_load(dst, q_tiles + (size_t)rt * P::kTileBytes, P::kTileBytes, bar);
        }
        __syncwarp();
    };
    if (warp == kLoadWarp) {
        if (kStreamKeys) load_rows(0, pipe.sbase, pipe.bar(kBarHeld));
        else load_keys<D, BS>(p, b, hk, ch.L, kt0, lane, pipe.sbase, pipe.bar(kBarHeld));
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    pipe.tmem = tmem_slot;
    if (warp == kLoadWarp) {
        pipe.run_load(n, lane, true, [&](int i, uint32_t dst, uint32_t bar) {
            if (kStreamKeys) load_keys<D, BS>(p, b, hk, ch.L, kt0 + i, lane, dst, bar);
            else load_rows(rt0 + i * csize, dst, bar);
        });
    } else if (warp == kMmaWarp) {
        pipe.run_mma(n, lane, true, !kStreamKeys);
    } else {
        const int group = warp >> 2, me = tid & 127;
        // Row me of tile rt: its first statistics, and M: +infinity (no gain) for rows that are not
        // there or that see no token
        auto stats_at = [&](int rt) { return p.stats + ((size_t)item * p.row_tiles + rt) * p.splits * kTile + me; };
        auto first_of = [&](int rt) {
            return rt < row_tiles && rt * kTile + me < nr ? stats_at(rt)[0] : make_float2(-INFINITY, 0.f);
        };
        auto base_of = [&](int rt, float2 first) {
            float m = first.x, l = first.y;
            if (p.splits > 1 && rt * kTile + me < nr) {
                const int last = first_pos + (min(nr, (rt + 1) * kTile) - 1) / p.G;
                const int tiles_r = last / kTile + 1, per = (tiles_r + p.splits - 1) / p.splits, splits = (tiles_r + per - 1) / per;
                const float2* at = stats_at(rt);
#pragma unroll 8
                for (int s = 1; s < splits; ++s) m = max_nan(m, at[s * kTile].x);
                l = 0.f;
                const float by = m == -INFINITY ? 0.f : m;
#pragma unroll 8
                for (int s = 0; s < splits; ++s) l += ex2(at[s * kTile].x - by) * at[s * kTile].y;
            }
            return m == -INFINITY ? INFINITY : m + log2f(l);
        };
        const int32_t* const table = p.block_tables + (size_t)b * p.max_blocks;
        float* const out = p.weights + ((size_t)to * p.num_kv_heads + hk) * p.max_tokens;
        auto write = [&](int t, float gain) {              // a token of its own for every thread
            if (t >= ch.L) return;
            const int id = table[t / BS];
            if (id < 0 || id >= p.num_blocks) gain = 0.f;
            out[t] = t < ch.L - ch.C ? fmaf(p.decay, out[t], gain) : gain;
        };
        const uint64_t sc2 = f2(p.scale_log2, p.scale_log2);
        float total = 0.f;
        bool ok = true;
        float2 first = first_of(rt0 + (kStreamKeys ? 0 : group * csize));
        if (kStreamKeys) {
            base[group][me] = base_of(0, first);
            group_sync(group);
        }
        const float* const bs = base[group];
        for (int i = group; i < n; i += 2) {               // to the end: a group's warps meet in group_sync
            const int kt = kStreamKeys ? kt0 + i : kt0, rt = kStreamKeys ? 0 : rt0 + i * csize, t = kt * kTile + me;
            if (!kStreamKeys) {
                const float mine = base_of(rt, first);
                group_sync(group);                         // the last tile's are read
                base[group][me] = mine;
                group_sync(group);
                first = first_of(rt + 2 * csize);
            }
            // token t is seen by the rows from column `from` of this tile on; past the last row a
            // product may be a NaN (zeros times an infinite key)
            const int from = max(0, t - first_pos) * p.G - rt * kTile, until = nr - rt * kTile;
            const bool masked = kt * kTile + kTile - 1 > first_pos + rt * kTile / p.G || until < kTile;
            uint64_t g2[2] = {0ull, 0ull};
            ok = ok && pipe.take(i, warp, [&](int c0, uint32_t (&v)[32]) {
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    const float4 m = *reinterpret_cast<const float4*>(bs + c0 + c);
                    float x[4];
                    f2_split(fma2(f2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), sc2, f2(-m.x, -m.y)), x[0], x[1]);
                    f2_split(fma2(f2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])), sc2, f2(-m.z, -m.w)), x[2], x[3]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = ex2(x[j]);
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[j] = c0 + c + j >= from && c0 + c + j < until ? x[j] : 0.f;
                    }
                    g2[0] = add2(g2[0], f2(x[0], x[1]));
                    g2[1] = add2(g2[1], f2(x[2], x[3]));
                }
            });
            float x, y, z, w;
            f2_split(g2[0], x, y);
            f2_split(g2[1], z, w);
            const float gain = (x + y) + (z + w);
            if (kStreamKeys) {
                if (ok) write(t, gain);
            } else {
                total += gain;
            }
        }
        if (!ok) flag_error(p.err, kErrTimeout);
        if (!kStreamKeys) {
            if (group == 1) part[0][me] = total;
            groups_sync();
            if (group == 0) {
                total += part[0][me];
                if (csize == 1) write(kt0 * kTile + me, total);
                else part[1][me] = total;
            }
        }
    }
    if (!kStreamKeys && csize > 1) {
        __syncwarp();
        cluster_sync();
        if (rank == 0 && tid < kTile && kt0 * kTile + tid < ch.L) {
            const int t = kt0 * kTile + tid, id = p.block_tables[(size_t)b * p.max_blocks + t / BS];
            float gain = 0.f;
            for (int r = 0; r < csize; ++r) gain += cluster_ld(&part[1][tid], r);
            if (id < 0 || id >= p.num_blocks) gain = 0.f;
            float* const at = p.weights + ((size_t)to * p.num_kv_heads + hk) * p.max_tokens + t;
            *at = t < ch.L - ch.C ? fmaf(p.decay, *at, gain) : gain;
        }
        __syncwarp();
        cluster_sync();                                    // the others' shared memory is read
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::dealloc(pipe.tmem, kTmemCols);
    }
}

// Row tiles and splits of the stats pass
struct Shape {
    long long items, row_tiles, splits;
    Shape(int num_seqs, int num_kv_heads, int G, int max_query_len, int window) {
        const long long w = window > 0 && window < max_query_len ? window : max_query_len;
        items = (long long)num_seqs * num_kv_heads;
        row_tiles = (w * G + kTile - 1) / kTile;
        const long long ctas = items * row_tiles;
        splits = ctas > 0 ? kTargetCtas / ctas : 1;
        if (splits < 1) splits = 1;
    }
};

template <int D, int BS>
int launch(Params p, cudaStream_t stream) {
    using P = Pipe<D>;
    auto stats = weigh_stats_kernel<D, BS>;
    auto gain = p.row_tiles == 1 ? weigh_gain_kernel<D, BS, true> : weigh_gain_kernel<D, BS, false>;
    int occ = 0;
    int st = kernel_setup(reinterpret_cast<const void*>(stats), P::kSmem, kThreads, &occ);
    if (st != PKV_OK) return st;
    st = kernel_setup(reinterpret_cast<const void*>(gain), P::kSmem, kThreads, &occ);
    if (st != PKV_OK) return st;
    const int items = p.num_seqs * p.num_kv_heads;
    note_launch();
    cudaError_t e = launch_pdl(stats, dim3((unsigned)p.splits, (unsigned)p.row_tiles, (unsigned)items), dim3(kThreads),
                               P::kSmem, stream, p);
    if (e != cudaSuccess) return cuda_fail("weigh_prefill_tokens: statistics launch", e);
    // key tiles a CTA streams: enough CTAs for two waves, no more than 16
    p.per = 1;
    if (p.row_tiles == 1) {
        const long long all = (long long)items * p.key_tiles;
        p.per = (int)(all / kTargetCtas);
        p.per = p.per < 1 ? 1 : p.per > 16 ? 16 : p.per;
    }
    // CTAs that share a key tile's rows: a few row tiles each, seven waves or so
    const long long key_ctas = ((long long)p.key_tiles + p.per - 1) / p.per;
    int size = 1;
    if (p.row_tiles > 1)
        while (size < 8 && key_ctas * items * size < 2048 && p.row_tiles / size > 4) size *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(key_ctas * size), (unsigned)items);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = P::kSmem;
    cfg.stream = stream;
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
    e = cudaLaunchKernelEx(&cfg, gain, p);
    return e == cudaSuccess ? PKV_OK : cuda_fail("weigh_prefill_tokens: weights launch", e);
}

}  // namespace weigh
}  // namespace pkv

extern "C" size_t weigh_prefill_workspace_size(int num_seqs, int num_heads, int max_query_len, int window) {
    using namespace pkv::weigh;
    if (num_seqs <= 0 || num_heads <= 0 || max_query_len <= 0 || window < 0) return 0;
    // at most (sequences x heads) x (queries + 127) rows: 256 bytes and one pair of statistics
    // each, and the pairs of the splits
    const long long w = window > 0 && window < max_query_len ? window : max_query_len;
    const size_t rows = (size_t)num_seqs * num_heads * (size_t)(w + kTile - 1);
    return rows * (256 + 8) + (size_t)kTargetCtas * kTile * 8;
}

extern "C" int weigh_prefill_tokens(float* token_weights, const int32_t* weight_rows, const void* q, const void* k_pool,
                                    const int32_t* block_tables, const int32_t* seq_lens, const int32_t* query_start,
                                    int num_seqs, int max_query_len, int window, int max_blocks_per_seq,
                                    int num_blocks, int num_rows, int max_tokens, int num_heads, int num_kv_heads,
                                    int head_dim, int block_size, float scale, float decay, int q_dtype, int kv_dtype,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    using namespace pkv;
    if (num_seqs < 0 || num_seqs > 65535 || max_query_len < 0 || window < 0 || max_blocks_per_seq <= 0 ||
        num_blocks <= 0 || num_rows <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_kv_heads > 65535 ||
        head_dim <= 0 || block_size <= 0 || !std::isfinite(scale) || !(decay >= 0.f) || !(decay <= 1.f) ||
        max_blocks_per_seq > (0x7fffffff - weigh::kTile) / block_size)
        return PKV_ERR_INVALID_ARG;
    if (num_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    if (max_tokens < max_blocks_per_seq * block_size || max_tokens % 4 != 0 || (!weight_rows && num_rows < num_seqs))
        return PKV_ERR_INVALID_ARG;
    const int G = num_heads / num_kv_heads;
    if (q_dtype != PKV_BF16 || kv_dtype != PKV_BF16 || (head_dim != 64 && head_dim != 128) ||
        (block_size != 16 && block_size != 32) || G > weigh::kMaxGroup)
        return PKV_ERR_UNSUPPORTED;
    const weigh::Shape shape(num_seqs, num_kv_heads, G, max_query_len, window);
    // the launches' grids; rows and positions times a group in 32 bits
    if (shape.items > 65535 || shape.row_tiles > 65535 ||
        (long long)max_blocks_per_seq * block_size > 0x7fffffffLL / weigh::kMaxGroup)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || max_query_len == 0) return PKV_OK;
    if (!token_weights || !q || !k_pool || !block_tables || !seq_lens || !query_start || !workspace)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(token_weights) || !aligned16(q) || !aligned16(k_pool) || !aligned16(workspace) ||
        workspace_bytes < weigh_prefill_workspace_size(num_seqs, num_heads, max_query_len, window))
        return PKV_ERR_INVALID_ARG;
    if (checking()) return PKV_OK;
    weigh::Params p{};
    p.weights = token_weights;
    p.rows = weight_rows;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_pool = static_cast<const __nv_bfloat16*>(k_pool);
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.query_start = query_start;
    p.num_seqs = num_seqs;
    p.max_query_len = max_query_len;
    p.window = window;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.num_rows = num_rows;
    p.max_tokens = max_tokens;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.G = G;
    p.row_tiles = (int)shape.row_tiles;
    p.splits = (int)shape.splits;
    p.key_tiles = (max_blocks_per_seq * block_size + weigh::kTile - 1) / weigh::kTile;
    // never 0: hidden logits are -infinity times it
    p.scale_log2 = scale == 0.f ? 1.17549435e-38f : std::fabs(scale) * 1.4426950408889634f;
    p.q_sign = scale < 0.f ? 0x80008000u : 0u;
    p.decay = decay;
    p.q_tiles = static_cast<unsigned char*>(workspace);
    p.stats = reinterpret_cast<float2*>(p.q_tiles + (size_t)(shape.items * shape.row_tiles) * weigh::kTile * head_dim * 2);
    p.err = error_word();
    if (!p.err) return PKV_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    try {
        if (head_dim == 64) return block_size == 16 ? weigh::launch<64, 16>(p, s) : weigh::launch<64, 32>(p, s);
        return block_size == 16 ? weigh::launch<128, 16>(p, s) : weigh::launch<128, 32>(p, s);
    } catch (...) {                                         // the per-kernel records' host memory
        return cuda_fail("weigh_prefill_tokens: host memory", cudaErrorMemoryAllocation);
    }
}
