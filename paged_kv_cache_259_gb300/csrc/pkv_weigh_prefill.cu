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
constexpr int kThreads = 192;
constexpr int kMmaWarp = 4, kLoadWarp = 5;
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
    float scale_log2, decay;
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
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
        "r"(bytes), "r"(bar)
        : "memory");
}
// The four warps that own tensor memory's lanes
__device__ __forceinline__ void lanes_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

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
        const uint32_t at = tmem + ((uint32_t)(warp * 32) << 16) + s * kTile;
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
    if (warp < 4) {                                        // row r0 + tid: to shared memory and the workspace
        const int r = r0 + tid;
        const bool valid = r < nr;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + ((size_t)(ch.q_first + (valid ? r / p.G : 0)) * p.num_heads + hk * p.G + (valid ? r % p.G : 0)) * D);
        const int at = (tid >> 3) * P::kGroup + (tid & 7) * 16;
        unsigned char* const to = p.q_tiles + ((size_t)item * p.row_tiles + rt) * P::kTileBytes + at;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            const uint4 v = valid ? src[c] : make_uint4(0, 0, 0, 0);
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
        const int r = r0 + tid, pr = ch.L - ch.w + min(r, nr - 1) / p.G;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int i = 0; i < n && ok; ++i) {
            const int key0 = (k0 + i) * kTile;
            const bool masked = any_bad || key0 + kTile - 1 > p_min;
            ok = pipe.take(i, warp, [&](int c0, const uint32_t (&v)[32]) {
                float x[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) x[c] = __uint_as_float(v[c]) * p.scale_log2;
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) x[c] = key0 + c0 + c <= pr ? x[c] : -INFINITY;
                    if (any_bad)
                        for (int s = 0; s < 32 / BS; ++s) {
                            const int blk = (key0 + c0) / BS + s;
                            const int id = blk <= p_max / BS ? table[blk] : 0;
                            if (id < 0 || id >= p.num_blocks)
#pragma unroll
                                for (int c = 0; c < 32; ++c) x[c] = c / BS == s ? -INFINITY : x[c];
                        }
                }
                float mx = m;
#pragma unroll
                for (int c = 0; c < 32; ++c) mx = max_nan(mx, x[c]);
                const float base = mx == -INFINITY ? 0.f : mx;
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < 32; ++c) sum += ex2(x[c] - base);
                l = fmaf(l, ex2(m - base), sum);
                m = mx;
            });
        }
        if (!ok) flag_error(p.err, kErrTimeout);
        p.stats[(((size_t)item * p.row_tiles + rt) * p.splits + split) * kTile + tid] = make_float2(m, l);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::dealloc(pipe.tmem, kTmemCols);
    }
}

// kStreamKeys: one row tile, held, and p.per key tiles; else a key tile, held, and the row
// tiles that see it.
template <int D, int BS, bool kStreamKeys>
__global__ void __launch_bounds__(kThreads, 2) weigh_gain_kernel(const Params p) {
    pdl_enter();
    using P = Pipe<D>;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(8) uint64_t bars[kNumBars];
    __shared__ uint32_t tmem_slot;
    __shared__ __align__(16) float base[2][kTile];         // M_r of a row tile
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the items that the first pass read last come first: their keys may still be in L2
    const int item = gridDim.y - 1 - blockIdx.y, b = item / p.num_kv_heads, hk = item - b * p.num_kv_heads;
    const Chunk ch(p, b, BS, false);
    if (ch.w == 0) return;                                 // the whole CTA
    const int tiles = (ch.L + kTile - 1) / kTile, nr = ch.w * p.G, row_tiles = (nr + kTile - 1) / kTile;
    const int kt0 = kStreamKeys ? blockIdx.x * p.per : blockIdx.x;
    if (kt0 >= tiles) return;
    const int first_pos = ch.L - ch.w;                     // of the first query that counts
    const int rt0 = kStreamKeys ? 0 : max(0, kt0 * kTile - first_pos) * p.G / kTile;
    const int n = kStreamKeys ? min(p.per, tiles - kt0) : row_tiles - rt0;
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
            else load_rows(rt0 + i, dst, bar);
        });
    } else if (warp == kMmaWarp) {
        pipe.run_mma(n, lane, true, !kStreamKeys);
    } else {
        // M of row tid of a tile: +infinity (no gain) for rows that are not there or have no weight
        auto row_base = [&](int rt) {
            if (rt * kTile + tid >= nr) return INFINITY;
            const int last = first_pos + (min(nr, (rt + 1) * kTile) - 1) / p.G;
            const int tiles_r = last / kTile + 1, per = (tiles_r + p.splits - 1) / p.splits, splits = (tiles_r + per - 1) / per;
            const float2* at = p.stats + ((size_t)item * p.row_tiles + rt) * p.splits * kTile + tid;
            float m = -INFINITY, l = 0.f;
            for (int s = 0; s < splits; ++s) m = max_nan(m, at[s * kTile].x);
            if (m == -INFINITY) return INFINITY;
            for (int s = 0; s < splits; ++s) l += ex2(at[s * kTile].x - m) * at[s * kTile].y;
            return m + log2f(l);
        };
        const int32_t* const table = p.block_tables + (size_t)b * p.max_blocks;
        float* const out = p.weights + ((size_t)to * p.num_kv_heads + hk) * p.max_tokens;
        auto write = [&](int t, float gain) {              // a token of its own for every thread
            if (t >= ch.L) return;
            const int id = table[t / BS];
            if (id < 0 || id >= p.num_blocks) gain = 0.f;
            out[t] = t < ch.L - ch.C ? fmaf(p.decay, out[t], gain) : gain;
        };
        float total = 0.f;
        bool ok = true;
        if (kStreamKeys) {
            base[0][tid] = row_base(0);
            lanes_sync();
        }
        for (int i = 0; i < n; ++i) {                      // to the end: all four warps meet in lanes_sync
            const int kt = kStreamKeys ? kt0 + i : kt0, rt = kStreamKeys ? 0 : rt0 + i, t = kt * kTile + tid;
            const float* const bs = base[kStreamKeys ? 0 : i & 1];
            if (!kStreamKeys) {
                base[i & 1][tid] = row_base(rt);
                lanes_sync();                              // the other buffer is read before the next one
            }
            // token t is seen by the rows from column `from` of this tile on; past the last row a
            // product may be a NaN (zeros times an infinite key)
            const int from = max(0, t - first_pos) * p.G - rt * kTile, until = nr - rt * kTile;
            const bool masked = kt * kTile + kTile - 1 > first_pos + rt * kTile / p.G || until < kTile;
            float g4[4] = {0.f, 0.f, 0.f, 0.f};
            ok = ok && pipe.take(i, warp, [&](int c0, const uint32_t (&v)[32]) {
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    const float4 m = *reinterpret_cast<const float4*>(bs + c0 + c);
                    float x[4] = {ex2(fmaf(__uint_as_float(v[c]), p.scale_log2, -m.x)),
                                  ex2(fmaf(__uint_as_float(v[c + 1]), p.scale_log2, -m.y)),
                                  ex2(fmaf(__uint_as_float(v[c + 2]), p.scale_log2, -m.z)),
                                  ex2(fmaf(__uint_as_float(v[c + 3]), p.scale_log2, -m.w))};
                    if (masked) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[j] = c0 + c + j >= from && c0 + c + j < until ? x[j] : 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) g4[j] += x[j];
                }
            });
            const float gain = (g4[0] + g4[1]) + (g4[2] + g4[3]);
            if (kStreamKeys) {
                if (ok) write(t, gain);
            } else {
                total += gain;
            }
        }
        if (!kStreamKeys && ok) write(kt0 * kTile + tid, total);
        if (!ok) flag_error(p.err, kErrTimeout);
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
    note_launch();
    e = launch_pdl(gain, dim3((unsigned)((p.key_tiles + p.per - 1) / p.per), (unsigned)items), dim3(kThreads), P::kSmem,
                   stream, p);
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
    p.scale_log2 = scale * 1.4426950408889634f;
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
