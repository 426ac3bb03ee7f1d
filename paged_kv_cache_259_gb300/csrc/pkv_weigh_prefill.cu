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
// in the same K-major core matrices (the cache's own tiles, the rows copied into such), so the
// second pass only exchanges two descriptors, and neither pass reduces across threads.
//
// Work split. One CTA an SM, which takes units of work one after another, the copies of the
// next one on their way while this one's products and exponentials run. A unit holds H tiles
// and streams others past them: stats, H row tiles and a run of their key tiles; gain, with one
// row tile a kv head (a short window), the row tile and a run of key tiles, else two key tiles
// and a run of the row tiles that see them. H is 2 wherever there are two to hold: what is
// streamed comes from L2 at 6.5 TB/s, which bounds a unit that holds one. Warps 0-15: four groups
// with a thread a lane of tensor memory, which holds four products. With two held tiles two groups
// share each product, half of its columns each; else the groups take every fourth tile of the
// stream, its halves one after the other. Warp 16 issues the products, 17 copies keys, 18 rows, 19
// picks the units and joins the groups' results of each. Row runs of the same key tiles leave their
// gains in the workspace; the last of them adds all up, in order.
//
// Bound. 4 chunks of up to 2048 queries (32 bf16 heads, 4 kv heads of 128, up to 4096 tokens): 225 us
// for two products of 101 GFLOP, 0.47 of the measured rate of a large library product. With two groups
// instead of four it took 233, and of those 215 with an eighth of the products' work, 203 with a
// sixteenth of the exponentials, 231 with an eighth of the copies, 131 with all three (warps waiting for
// one another, units changing): not one resource, but two chains of like length, of products of 128 x
// 128 from shared memory (590 cycles each) and of exponentials (1700 for a group's half of them). The
// last 32 queries of 4 prompts of up to 32768: 82 us, of which K, read twice, is 55 at the copy rate
// (once would do if the rows' statistics came from the prefill, which has them), and three launches.
// Small chunks: 12 to 19 us, the launches and a chain of loads in each. Units are made by the tables' width:
// of 8 x 4096 tokens the last 32 of 512 queries take 39.7 us, 49.2 in tables of 131072 tokens (all of
// them 279 and 253). Measured and not kept: two groups with
// halves read ahead (255 us); one exponential in four by a polynomial (255); four held tiles (273 to 295:
// a unit's change weighs more); the next unit's held tiles in places that the stream leaves (220, but 1
// to 2 us more wherever units are few).
#include <cmath>

#include <cuda_bf16.h>

#include "pkv_check.cuh"
#include "pkv_internal.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace weigh {

constexpr int kTile = 128;             // rows, keys of a tile
constexpr int kBufs = 4;               // products (128 columns of tensor memory) and streamed tiles in flight
constexpr int kGroups = 4;             // of 128 threads
constexpr int kMmaWarp = 16, kKeyWarp = 17, kRowWarp = 18, kPickWarp = 19;
constexpr int kThreads = 20 * 32;
constexpr int kHalf = kTile / 2;       // columns of a product that a thread has at a time
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kIdesc = tc::idesc_bf16_f32(kTile, kTile);
constexpr int kExt = kTile * 32;       // bytes of the 16 dims that carry -M_r / scale behind a row tile
// Units of the stats pass: eight on each of 152 SMs (4 chunks of 2048: 231 us; 1824 237, 3648 267). A
// constant, as the workspace's size, which is told without a device, goes by it
constexpr int kTargetUnits = 1216;
constexpr int kMaxGroup = 128;
constexpr int kRing = 4;               // units picked ahead

enum Pass : int { kStats, kGainRows, kGainKeys };          // kGainRows: the row tiles stream

struct Params {
    float* weights;
    const int32_t* rows;
    const __nv_bfloat16* q;
    const __nv_bfloat16* k_pool;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* query_start;
    unsigned char* q_tiles;            // [items][row_tiles] tiles of 128 rows and their 16 more dims, core matrices
    float2* stats;                     // [items][row_tiles][splits][128] maximum, sum
    int* next;                         // the gain pass's next unit,
    int* arrived;                      // and the row runs of each pair of key tiles that are through
    float* parts;                      // their gains [pairs][row_parts][2][128]
    int* err;
    int num_seqs, max_query_len, window, max_blocks, num_blocks, num_rows, max_tokens;
    int num_heads, num_kv_heads, G, row_tiles, splits, per;   // per: key tiles of a unit's stream
    int key_pairs, row_parts;          // of a sequence, at most; row runs of a pair
    uint32_t g_magic;                  // floor(2^32 / G) + 1: r / G for r < 2^32 / G
    float scale_log2, decay;           // the scale's magnitude,
    uint32_t sign;                     // and what turns the sign of two query elements
    int no_scale;                      // a scale of 0: rows of zeros instead
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// Memory to shared memory, completing on `bar`, by a whole converged warp, one lane of it: the
// operands stay warp-uniform (lanes that send a copy each go one after another, 120 cycles each).
__device__ __forceinline__ void bulk_load_elect(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}
// Shared memory to memory (one lane); all of this thread's have been read, have been written
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;" ::"l"(dst), "r"(src),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// A copy of 16 bytes (none: zeros) in the background
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool some) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(some ? 16 : 0) : "memory");
}

// -M_r of row `me` of a tile, in units of the products, as three bf16 numbers (24 bits) in the first of
// the 16 dims behind it, whose partners in the keys' tile are 1: the products come out less M_r, and
// the second pass neither reads nor subtracts it (128 shared-memory reads a tile and thread group
// less: 160 us against 116 for 4 chunks of 2048). -infinity (no gain): a row that is not there or
// sees no token.
__device__ __forceinline__ void write_base(unsigned char* ext, int me, float m, float l, bool there, float scale_log2) {
    const float x = !there || m == -INFINITY ? -INFINITY : -(m + log2f(l)) / scale_log2;
    const __nv_bfloat16 a = __float2bfloat16_rn(x);
    float rest = x - __bfloat162float(a);
    if (!(fabsf(x) < INFINITY)) rest = 0.f;                // infinite and NaN: one number says it
    const __nv_bfloat16 b = __float2bfloat16_rn(rest), c = __float2bfloat16_rn(rest - __bfloat162float(b));
    const uint32_t ab = (uint32_t)__bfloat16_as_ushort(a) | ((uint32_t)__bfloat16_as_ushort(b) << 16);
    uint4* const at = reinterpret_cast<uint4*>(ext + (me >> 3) * 256 + (me & 7) * 16);
    at[0] = make_uint4(ab, (uint32_t)__bfloat16_as_ushort(c), 0u, 0u);
    at[8] = make_uint4(0u, 0u, 0u, 0u);
}

// One unit: `n` stream tiles from `first` on, past the held tiles from `held` on; -1: no more
struct Unit {
    int n, first, held, item, b, hk, split, bad;           // bad: some block of the keys is not in the pool
    int L, C, w, q_first, nr, to, splits;                  // splits: units that share the held tiles
};

// Barriers. Every waiter is at most one phase behind: a phase's successor needs the waiter's
// own next step.
enum : int {
    kBarHeldFull = 0,                  // [2] the held tiles of a unit are there (H = 1: units in turn)
    kBarHeldFree = 2,                  // [2] their products are done
    kBarFull = 4,                      // [4] a streamed tile is there
    kBarFree = 8,                      // [4] its products are done
    kBarDone = 12,                     // [4] a product is done
    kBarRead = 16,                     // [4] and is read (its groups' warps)
    kBarPart = 20,                     // a unit's results are there (16 warps)
    kBarPartFree = 21,                 // they are joined
    kBarUnit = 24,                     // [kRing] a unit is picked
    kBarUnitFree = 28,                 // [kRing] everybody has seen it (19 warps)
    kBarDrain = 32,
    kNumBars
};

template <int D>
struct Shared {
    static constexpr int kTileBytes = kTile * D * 2, kGroupBytes = D / 8 * 128;   // 8 rows
    static constexpr int kSlot = kTileBytes + kExt;                               // of a row tile; a key tile takes less
    static constexpr int kHeld = 0, kStream = 2 * kSlot;
    static constexpr int kOnes = kStream + kBufs * kSlot;                         // the keys' 16 more dims
    static constexpr int kPart = kOnes + kExt;                                    // [kGroups][128] of 8 bytes
    static constexpr int kUnits = kPart + kGroups * kTile * 8;
    static constexpr int kBars = kUnits + (kRing * (int)sizeof(Unit) + 15) / 16 * 16;
    static constexpr int kBytes = kBars + kNumBars * 8;
    static_assert(kBytes <= 227 * 1024, "shared memory per CTA");
};

// One sequence's chunk; w == 0: nothing to do
struct Chunk {
    int L = 0, C = 0, w = 0, q_first = 0;                  // q_first: row of q of the first query that counts
    __device__ __forceinline__ void read(const Params& p, int b, int bs) {
        L = p.seq_lens[b];
        const int q0 = p.query_start[b], q1 = p.query_start[b + 1], T = p.query_start[p.num_seqs];
        C = q1 - q0;
        w = p.window > 0 && p.window < C ? p.window : C;
        if (C < 0 || C > L || L > p.max_blocks * bs || q0 < 0 || q1 > T || C > p.max_query_len) {
            if (C != 0) flag_error(p.err, kErrOutOfRange);
            w = 0;
        }
        q_first = q1 - w;
    }
};

template <Pass PASS, int H, int D, int BS>
__global__ void __launch_bounds__(kThreads, 1) weigh_kernel(const Params p) {
    using S = Shared<D>;
    static_assert(H == 1 || H == 2, "held tiles");
    constexpr int kBlocks = kTile / BS, kTurn = kBufs / H;      // products of a held tile
    constexpr int kShare = kGroups / H;                         // groups that share a held tile
    // place and use of what unit u holds: two places in turn, or one of two tiles
    auto held_at = [](int u) { return H == 1 ? u & 1 : 0; };
    auto held_use = [](int u) { return H == 1 ? u >> 1 : u; };
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ uint32_t tmem_slot;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_addr(smem), bar0 = sbase + S::kBars;
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    auto wait = [&](int i, int parity) { return __all_sync(0xffffffffu, mbar_wait_bounded(bar(i), parity & 1, p.err)) != 0; };
    auto row_div = [&](int r) { return p.G == 1 ? r : (int)__umulhi((uint32_t)r, p.g_magic); };
    Unit* const units = reinterpret_cast<Unit*>(smem + S::kUnits);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kBarHeldFull + i), 1);
            mbar_init(bar(kBarHeldFree + i), 1);
        }
        mbar_init(bar(kBarPart), kGroups * 4);
        mbar_init(bar(kBarPartFree), 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(kBarFull + i), 1);
            mbar_init(bar(kBarFree + i), 1);
            mbar_init(bar(kBarDone + i), 1);
            mbar_init(bar(kBarRead + i), 4 * H);
            mbar_init(bar(kBarUnit + i), 1);
            mbar_init(bar(kBarUnitFree + i), kPickWarp);
        }
        mbar_init(bar(kBarDrain), 1);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tc::alloc(smem_addr(&tmem_slot), kTmemCols);
        tc::relinquish_alloc_permit();
    }
    if (PASS != kStats && tid < kTile) {
        uint4* const at = reinterpret_cast<uint4*>(smem + S::kOnes + (tid >> 3) * 256 + (tid & 7) * 16);
        at[0] = make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u);
        at[8] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_slot;
    // Up to here nothing of the device's memory. Tensor memory held while earlier launches may still run
    // keeps none of them from theirs: beside these registers no CTA that takes some fits (launch_pdl)
    pdl_enter();
    if (PASS == kStats && tid == 0 && blockIdx.x == 0) *p.next = 0;
    if (PASS == kStats && p.row_parts > 1)
        for (int i = blockIdx.x * kThreads + tid; i < p.num_seqs * p.num_kv_heads * p.key_pairs; i += gridDim.x * kThreads)
            p.arrived[i] = 0;

    // Before a copying warp leaves: what it sent has landed (after a wait that gave up, too)
    auto land = [&](int full, int parts, int sent) {
        for (int i = max(0, sent - parts); i < sent; ++i)
            (void)mbar_wait_bounded(bar(full + i % parts), (uint32_t)(i / parts) & 1u, nullptr);
    };

    // The u-th unit of this CTA (every warp but the picking one); false: no more, or a wait gave up
    Unit unit;
    auto next_unit = [&](int u) {
        if (!wait(kBarUnit + u % kRing, u / kRing)) return false;
        unit = units[u % kRing];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarUnitFree + u % kRing));
        return unit.n >= 0;
    };

    if (warp == kPickWarp) {
        // ------------------------------------------------------------ units
        // 32 sequences at a time, one a lane: how many units each has, and where they begin
        int b0 = 0, mine = 0, begin = 0, seen = 0;         // seen: units of the sequences before b0
        Chunk ch;
        int tiles = 0, row_tiles = 0, splits = 1, total = 0;
        auto load = [&] {
            ch = Chunk();
            mine = 0;
            const int b = b0 + lane;
            if (b < p.num_seqs) {
                ch.read(p, b, BS);
                tiles = (ch.L + kTile - 1) / kTile;
                row_tiles = (ch.w * p.G + kTile - 1) / kTile;
                if (ch.w > 0) {
                    if (PASS == kStats) {
                        splits = min(p.splits, (tiles + p.per - 1) / p.per);
                        mine = p.num_kv_heads * ((row_tiles + H - 1) / H) * splits;
                    } else if (PASS == kGainRows) {
                        mine = p.num_kv_heads * ((tiles + H - 1) / H) * p.row_parts;
                    } else {
                        mine = p.num_kv_heads * ((tiles + p.per - 1) / p.per);
                    }
                }
            }
            begin = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, begin, o);
                if (lane >= o) begin += x;
            }
            total = __shfl_sync(0xffffffffu, begin, 31);
            begin -= mine;
        };
        load();
        int to = -1, to_of = -1;                           // the weight row of sequence to_of
        bool ok = true, more = true;
        int at = blockIdx.x, picked = 0;
        auto pick = [&] {                                  // the next unit, or that there is none
          for (;;) {
            if (PASS != kStats) {
                if (lane == 0) at = atomicAdd(p.next, 1);
                at = __shfl_sync(0xffffffffu, at, 0);
            }
            while (at >= seen + total && b0 + 32 < p.num_seqs) {
                seen += total;
                b0 += 32;
                load();
            }
            Unit x;
            x.n = -1;
            more = at < seen + total;
            if (more) {
                const int k = PASS == kGainKeys ? seen + total - 1 - at : at - seen;
                const int src = __ffs(__ballot_sync(0xffffffffu, k >= begin && k < begin + mine)) - 1;
                auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, src); };
                const int local = k - of(begin);
                x.b = b0 + src;
                x.L = of(ch.L), x.C = of(ch.C), x.w = of(ch.w), x.q_first = of(ch.q_first);
                x.nr = x.w * p.G;
                const int nt = of(tiles), nrt = of(row_tiles), ns = of(splits), first_pos = x.L - x.w;
                x.split = 0;
                x.splits = 1;
                if (PASS == kStats) {                      // row tiles' neighbours share their keys: they go side by side
                    const int held = (nrt + H - 1) / H, rest = local / held;
                    x.held = (held - 1 - (local - rest * held)) * H;
                    x.hk = rest / ns;
                    x.split = rest - x.hk * ns;
                    const int seen_tiles = (first_pos + (min(x.nr, (x.held + H) * kTile) - 1) / p.G) / kTile + 1;
                    const int per = (seen_tiles + ns - 1) / ns;
                    x.first = x.split * per;
                    x.n = min(seen_tiles, x.first + per) - x.first;
                } else if (PASS == kGainRows) {            // the tiles that most rows see first
                    const int rest = local / p.row_parts;
                    x.split = local - rest * p.row_parts;
                    x.held = rest / p.num_kv_heads * H;
                    x.hk = rest % p.num_kv_heads;
                    x.first = max(0, x.held * kTile - first_pos) * p.G / kTile;
                    const int all = nrt - x.first, per = (all + p.row_parts - 1) / p.row_parts;
                    x.splits = (all + per - 1) / per;
                    x.first += x.split * per;
                    x.n = min(nrt, x.first + per) - x.first;
                } else {
                    const int run = local / p.num_kv_heads;
                    x.hk = local - run * p.num_kv_heads;
                    x.held = 0;
                    x.first = run * p.per;
                    x.n = min(p.per, nt - x.first);
                }
                x.item = x.b * p.num_kv_heads + x.hk;
                // blocks of its keys that are not in the pool
                const int kt = PASS == kGainRows ? x.held : x.first, kn = PASS == kGainRows ? H : x.n;
                const int32_t* const table = p.block_tables + (size_t)x.b * p.max_blocks;
                bool bad = false;
                for (int i = kt * kBlocks + lane; i < min((kt + kn) * kBlocks, (x.L + BS - 1) / BS); i += 32)
                    bad |= table[i] < 0 || table[i] >= p.num_blocks;
                x.bad = __any_sync(0xffffffffu, bad);
                x.to = x.b;
                if (PASS != kStats && p.rows) {            // good, and no earlier sequence's
                    if (to_of != x.b) {
                        to_of = x.b;
                        to = p.rows[x.b];
                        bool lost = to < 0 || to >= p.num_rows;
                        for (int i = lane; i < x.b; i += 32) lost |= p.rows[i] == to;
                        if (__any_sync(0xffffffffu, lost)) {
                            if (lane == 0) flag_error(p.err, kErrOutOfRange);
                            to = -1;
                        }
                    }
                    x.to = to;
                }
                if (PASS == kStats) at += gridDim.x;
                if (x.n <= 0 || (PASS != kStats && x.to < 0)) continue;
            }
            if (picked >= kRing) ok = wait(kBarUnitFree + picked % kRing, picked / kRing - 1);
            if (!ok) return;
            if (lane == 0) {
                units[picked % kRing] = x;
                mbar_arrive(bar(kBarUnit + picked % kRing));
            }
            __syncwarp();
            ++picked;
            return;
          }
        };
        if (PASS == kGainKeys) {
            while (ok && more) pick();
        } else {
            while (ok && more && picked < kRing - 1) pick();
        }
        // ------------------------------------------------------------ a unit's results
        for (int u = 0; PASS != kGainKeys && ok && u < picked; ++u) {
            unit = units[u % kRing];                       // this warp's own
            if (unit.n < 0 || !wait(kBarPart, u)) break;
            const unsigned char* const part = smem + S::kPart;
            if constexpr (PASS == kStats) {
#pragma unroll
                for (int k = 0; k < 4 * H; ++k) {
                    const int me = lane + 32 * (k & 3), h = k >> 2, rt = unit.held + h;
                    float2 x[kShare];
                    float m = -INFINITY, l = 0.f;
#pragma unroll
                    for (int g = 0; g < kShare; ++g) x[g] = reinterpret_cast<const float2*>(part)[(h * kShare + g) * kTile + me];
#pragma unroll
                    for (int g = 0; g < kShare; ++g) m = max_nan(m, x[g].x);
                    const float by = m == -INFINITY ? 0.f : m;
#pragma unroll
                    for (int g = 0; g < kShare; ++g) l += ex2(x[g].x - by) * x[g].y;
                    if (rt * kTile >= unit.nr) continue;
                    const size_t tile = (size_t)unit.item * p.row_tiles + rt;
                    if (p.splits > 1) p.stats[(tile * p.splits + unit.split) * kTile + me] = make_float2(m, l);
                    else write_base(p.q_tiles + tile * S::kSlot + S::kTileBytes, me, m, l, rt * kTile + me < unit.nr, p.scale_log2);
                }
            } else {
                float gain[4 * H];
#pragma unroll
                for (int k = 0; k < 4 * H; ++k) {
                    gain[k] = 0.f;
#pragma unroll
                    for (int g = 0; g < kShare; ++g)
                        gain[k] += reinterpret_cast<const float*>(part)[((k >> 2) * kShare + g) * kTile + lane + 32 * (k & 3)];
                }
                bool write = true;
                if (unit.splits > 1) {                     // one of several row runs: the last adds them up
                    const int pair = unit.item * p.key_pairs + unit.held / H;
                    float* const all = p.parts + (size_t)pair * p.row_parts * H * kTile + lane;
#pragma unroll
                    for (int k = 0; k < 4 * H; ++k) all[(unit.split * H * 4 + k) * 32] = gain[k];
                    __threadfence();
                    __syncwarp();
                    int before = 0;
                    if (lane == 0) before = atomicAdd(&p.arrived[pair], 1);
                    write = __shfl_sync(0xffffffffu, before, 0) == unit.splits - 1;
                    if (write) {
                        __threadfence();
#pragma unroll
                        for (int k = 0; k < 4 * H; ++k) {
                            gain[k] = 0.f;
                            for (int x = 0; x < unit.splits; ++x) gain[k] += __ldcg(&all[(x * H * 4 + k) * 32]);
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < 4 * H; ++k) {
                    const int t = unit.held * kTile + lane + 32 * k;
                    if (write && t < unit.L) {
                        const int id = unit.bad ? p.block_tables[(size_t)unit.b * p.max_blocks + t / BS] : 0;
                        float* const at = p.weights + ((size_t)unit.to * p.num_kv_heads + unit.hk) * p.max_tokens + t;
                        const float g = id < 0 || id >= p.num_blocks ? 0.f : gain[k];
                        *at = t < unit.L - unit.C ? fmaf(p.decay, *at, g) : g;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarPartFree));
            if (more) pick();
        }
    } else if (warp == kKeyWarp) {
        // ------------------------------------------------------------ keys
        // Block ids, 32 a lane each, the next 32 read ahead. Blocks that are not in the pool are
        // read from block 0 (what comes of them is left out by those who use them).
        long long ids = 0, next_ids = 0;                   // as places in the pool
        int first_block = 0, window = 0;
        auto read_ids = [&](int k) -> long long {
            const int blk = first_block + 32 * k + lane;
            if (blk >= (unit.L + BS - 1) / BS) return 0;
            int id = p.block_tables[(size_t)unit.b * p.max_blocks + blk];
            if (id < 0 || id >= p.num_blocks) {
                flag_error(p.err, kErrOutOfRange);
                id = 0;
            }
            return ((long long)id * p.num_kv_heads + unit.hk) * (BS * D);
        };
        auto begin_ids = [&](int tile) {
            first_block = tile * kBlocks;
            window = 0;
            ids = read_ids(0);
            next_ids = read_ids(1);
        };
        auto blocks_left = [&](int j) { return (unit.L + BS - 1) / BS - first_block - j * kBlocks; };
        auto load_keys = [&](int j, uint32_t dst, uint32_t full) {   // the j-th tile from there; `full` is armed
            if (j * kBlocks / 32 != window) {
                ++window;
                ids = next_ids;
                next_ids = read_ids(window + 1);
            }
            const int n = blocks_left(j);
            if (n >= kBlocks) {
#pragma unroll
                for (int k = 0; k < kBlocks; ++k)
                    bulk_load_elect(dst + k * BS * D * 2, p.k_pool + __shfl_sync(0xffffffffu, ids, j * kBlocks % 32 + k), BS * D * 2, full);
            } else {
#pragma unroll 1
                for (int k = 0; k < n; ++k)
                    bulk_load_elect(dst + k * BS * D * 2, p.k_pool + __shfl_sync(0xffffffffu, ids, j * kBlocks % 32 + k), BS * D * 2, full);
            }
        };
        int it = 0, sent = 0;
        for (int u = 0; next_unit(u); ++u) {
            begin_ids(PASS == kGainRows ? unit.held : unit.first);
            if (PASS == kGainRows) {
                const int full = bar(kBarHeldFull + held_at(u));
                if (held_use(u) > 0 && !wait(kBarHeldFree + held_at(u), held_use(u) - 1)) break;
                const int there = min(H, (unit.L + kTile - 1) / kTile - unit.held);
                mbar_arrive_expect_tx_elect(full, (uint32_t)(min(there * kBlocks, blocks_left(0)) * BS * D * 2));
                for (int h = 0; h < there; ++h) load_keys(h, sbase + S::kHeld + (held_at(u) + h) * S::kSlot, full);
                sent = u + 1;
            } else {
                bool ok = true;
                for (int j = 0; j < unit.n && ok; ++j, ++it) {
                    const int s = it & 3;
                    if (it >= 4) ok = wait(kBarFree + s, (it >> 2) - 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx_elect(bar(kBarFull + s), (uint32_t)(min(kBlocks, blocks_left(j)) * BS * D * 2));
                    load_keys(j, sbase + S::kStream + s * S::kSlot, bar(kBarFull + s));
                    sent = it + 1;
                }
                if (!ok) break;
            }
        }
        land(PASS == kGainRows ? kBarHeldFull : kBarFull, PASS == kGainRows ? 3 - H : 4, sent);
    } else if (warp == kRowWarp) {
        // ------------------------------------------------------------ rows
        // Row tile rt in core matrices: 8 rows x 4 pieces of 16 bytes an instruction; zeros past the last
        auto send_rows = [&](int rt, uint32_t dst) {
            const __nv_bfloat16* const q = p.q + ((size_t)unit.q_first * p.num_heads + unit.hk * p.G) * D + (lane >> 3) * 8;
            const uint32_t to = dst + (lane >> 3) * 128 + (lane & 7) * 16;
#pragma unroll 4
            for (int g = 0; g < kTile / 8; ++g) {
                const int r = rt * kTile + g * 8 + (lane & 7);
                const bool some = r < unit.nr && !p.no_scale;
                const int rr = some ? r : 0;
                const __nv_bfloat16* src = q + ((size_t)row_div(rr) * (p.num_heads - p.G) + rr) * D;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) copy16(to + g * S::kGroupBytes + c * 512, src + c * 32, some);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        auto tile_of = [&](int rt) { return p.q_tiles + ((size_t)unit.item * p.row_tiles + rt) * S::kSlot; };
        auto load_rows = [&](int rt, uint32_t dst, uint32_t full) {
            mbar_arrive_expect_tx_elect(full, S::kSlot);
            bulk_load_elect(dst, tile_of(rt), S::kSlot, full);
        };
        int it = 0, sent = 0;
        for (int u = 0; next_unit(u); ++u) {
            const uint32_t held = sbase + S::kHeld + held_at(u) * S::kSlot, held_full = bar(kBarHeldFull + held_at(u));
            if (PASS != kGainRows && held_use(u) > 0 && !wait(kBarHeldFree + held_at(u), held_use(u) - 1)) break;
            if (PASS == kStats) {
                bulk_stores_read();                        // of the unit that had the place
                __syncwarp();
#pragma unroll
                for (int h = 0; h < H; ++h) send_rows(unit.held + h, held + h * S::kSlot);
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                __syncwarp();
                if (p.sign)                                // a negative scale: the rows turn it
                    for (int i = lane; i < H * S::kSlot / 16; i += 32) {
                        uint4* const at = reinterpret_cast<uint4*>(smem + (held - sbase)) + i;
                        const uint4 v = *at;
                        *at = make_uint4(v.x ^ p.sign, v.y ^ p.sign, v.z ^ p.sign, v.w ^ p.sign);
                    }
                fence_proxy_async_smem();                  // to the tensor cores and the copy below
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(held_full);
                    if (unit.split == 0)                   // for the second pass
                        for (int h = 0; h < min(H, (unit.nr + kTile - 1) / kTile - unit.held); ++h)
                            bulk_store(tile_of(unit.held + h), held + h * S::kSlot, S::kTileBytes);
                }
                __syncwarp();
                continue;
            }
            if (PASS == kGainKeys) {
                load_rows(0, held, held_full);
                sent = u + 1;
                continue;
            }
            bool ok = true;
            for (int j = 0; j < unit.n && ok; ++j, ++it) {
                if (it >= 4) ok = wait(kBarFree + (it & 3), (it >> 2) - 1);
                if (!ok) break;
                load_rows(unit.first + j, sbase + S::kStream + (it & 3) * S::kSlot, bar(kBarFull + (it & 3)));
                sent = it + 1;
            }
            if (!ok) break;
        }
        bulk_stores_done();
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (PASS != kStats) land(PASS == kGainKeys ? kBarHeldFull : kBarFull, PASS == kGainKeys ? 2 : 4, sent);
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ products
        constexpr uint32_t hi = tc::desc_hi(S::kGroupBytes), hi_ext = tc::desc_hi(256);
        const uint32_t ones = tc::desc_lo(sbase + S::kOnes, 128);
        bool ok = true;
        int it = 0;
        for (int u = 0; ok && next_unit(u); ++u) {
            ok = wait(kBarHeldFull + held_at(u), held_use(u));
            if (!ok) break;
            const uint32_t h_lo = tc::desc_lo(sbase + S::kHeld + held_at(u) * S::kSlot, 128);
            for (int j = 0; j < unit.n && ok; ++j, ++it) {
                const int s = it & 3;
                ok = wait(kBarFull + s, it >> 2);
                const uint32_t s_lo = tc::desc_lo(sbase + S::kStream + s * S::kSlot, 128);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const int g = h * kTurn + it % kTurn;
                    if (ok && it >= kTurn) ok = wait(kBarRead + g, it / kTurn - 1);
                    if (!ok) break;
                    tc::fence_after_sync();
                    const uint32_t held = h_lo + h * (S::kSlot / 16);
                    const uint32_t a = PASS == kGainKeys ? s_lo : held, b = PASS == kGainKeys ? held : s_lo;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        tc::mma_ss2_elect(tmem + g * kTile, a + k * 16, hi, b + k * 16, hi, kIdesc, k > 0);
                    if (PASS != kStats) {                  // less M_r
                        const uint32_t row = (PASS == kGainKeys ? held : s_lo) + S::kTileBytes / 16;
                        tc::mma_ss2_elect(tmem + g * kTile, ones, hi_ext, row, hi_ext, kIdesc, 1);
                    }
                    tc::commit_elect(bar(kBarDone + g));
                }
                if (ok) tc::commit_elect(bar(kBarFree + s));
            }
            tc::commit_elect(bar(kBarHeldFree + held_at(u)));
        }
        tc::commit_elect(bar(kBarDrain));                  // all of them complete before tensor memory goes
        (void)mbar_wait_bounded(bar(kBarDrain), 0, nullptr);
        __syncwarp();
    } else {
        // ------------------------------------------------------------ exponentials
        const int group = warp >> 2, me = tid & 127;
        const uint64_t sc2 = f2(p.scale_log2, p.scale_log2);
        // A product's columns, half of them at a time: two held tiles have two groups each, one for each
        // half; of one the groups take every fourth product, both halves
        const int mine = H == 2 ? group >> 1 : 0, half0 = H == 2 ? group & 1 : 0, half1 = H == 2 ? half0 : 1;
        uint32_t v[kHalf];
        auto take = [&](int i, int half) {                 // of the product of stream tile i
            const int buf = (H == 2 ? mine * kTurn : 0) + i % kTurn;
            if (half == half0) {
                if (!wait(kBarDone + buf, i / kTurn)) return false;
                tc::fence_after_sync();
            }
            const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + buf * kTile + half * kHalf;
#pragma unroll
            for (int c = 0; c < 2; ++c) tc::ld32(at + 32 * c, reinterpret_cast<uint32_t(&)[32]>(v[32 * c]));
            tc::wait_ld();
            if (half == half1) {
                tc::fence_before_sync();
                __syncwarp();
                mbar_arrive_elect(bar(kBarRead + buf));
            }
            return true;
        };
        bool ok = true;
        int it = 0;                                        // of the unit's first tile
        for (int u = 0; ok && next_unit(u); it += unit.n, ++u) {
            const int first_pos = unit.L - unit.w, skip = H == 2 ? 0 : (group - it) & (kGroups - 1), held = unit.held + mine;
            constexpr int kStep = H == 2 ? 1 : kGroups;
            if constexpr (PASS == kStats) {
                const int r0 = held * kTile, r = min(r0 + me, unit.nr - 1), pr = first_pos + row_div(r);
                const int p_min = first_pos + row_div(min(r0, unit.nr - 1));
                float m = -INFINITY, l = 0.f;              // of the products; the scale is not negative
                for (int j = skip; j < unit.n && ok; j += kStep)
#pragma unroll 1
                    for (int half = half0; half <= half1; ++half) {
                        const int key0 = (unit.first + j) * kTile + half * kHalf;
                        const bool masked = unit.bad || key0 + kHalf - 1 > p_min;
                        ok = take(it + j, half);
                        if (!ok) break;
                        if (masked) {
                            constexpr uint32_t kNone = 0xff800000u;   // -infinity
#pragma unroll
                            for (int c = 0; c < kHalf; ++c) v[c] = key0 + c <= pr ? v[c] : kNone;
                            if (unit.bad)
                                for (int s = 0; s < kHalf / BS; ++s) {
                                    const int blk = key0 / BS + s;
                                    const int id = blk < (unit.L + BS - 1) / BS ? p.block_tables[(size_t)unit.b * p.max_blocks + blk] : 0;
                                    if (id < 0 || id >= p.num_blocks)
#pragma unroll
                                        for (int c = 0; c < kHalf; ++c) v[c] = c / BS == s ? kNone : v[c];
                                }
                        }
                        float m4[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) m4[c] = max_nan(m, __uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1]));
#pragma unroll
                        for (int c = 4; c < kHalf / 2; ++c)
                            m4[c & 3] = max_nan(m4[c & 3], __uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1]));
                        const float mx = max_nan(max_nan(m4[0], m4[1], m4[2]), m4[3]);
                        const float by = mx == -INFINITY ? 0.f : mx * p.scale_log2;
                        const uint64_t nb2 = f2(-by, -by);
                        uint64_t s2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                        for (int c = 0; c < kHalf; c += 2) {
                            float a, b;
                            f2_split(fma2(f2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), sc2, nb2), a, b);
                            s2[(c >> 1) & 3] = add2(s2[(c >> 1) & 3], f2(ex2(a), ex2(b)));
                        }
                        float a, b;
                        f2_split(add2(add2(s2[0], s2[1]), add2(s2[2], s2[3])), a, b);
                        l = fmaf(l, ex2(fmaf(m, p.scale_log2, -by)), a + b);
                        m = mx;
                    }
                if (ok && u > 0) ok = wait(kBarPartFree, u - 1);
                if (!ok) break;
                reinterpret_cast<float2*>(smem + S::kPart)[group * kTile + me] =
                    make_float2(m == -INFINITY ? m : m * p.scale_log2, l);
            } else {
                constexpr bool kRows = PASS == kGainRows;
                float total = 0.f;                         // of the unit; else of the product
                for (int j = skip; j < unit.n && ok; j += kStep) {
                    const int kt = kRows ? held : unit.first + j, rt = kRows ? unit.first + j : 0, t = kt * kTile + me;
#pragma unroll 1
                    for (int half = half0; half <= half1; ++half) {
                        // token t is seen by the rows from column `from` of this half on; past the last
                        // row a product may be a NaN (zeros times an infinite key)
                        const int first_row = rt * kTile + half * kHalf;
                        const int from = max(0, t - first_pos) * p.G - first_row, until = unit.nr - first_row;
                        const bool masked = kt * kTile + kTile - 1 > first_pos + row_div(first_row) || until < kHalf;
                        ok = take(it + j, half);
                        if (!ok) break;
                        if (masked) {
#pragma unroll
                            for (int c = 0; c < kHalf; ++c) v[c] = c >= from && c < until ? v[c] : 0xff800000u;
                        }
                        uint64_t g2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                        for (int c = 0; c < kHalf; c += 2) {
                            if (!kRows && c % 32 == 0 && c >= until) break;   // no more rows
                            float a, b;
                            f2_split(mul2(f2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), sc2), a, b);
                            g2[(c >> 1) & 3] = add2(g2[(c >> 1) & 3], f2(ex2(a), ex2(b)));
                        }
                        float a, b;
                        f2_split(add2(add2(g2[0], g2[1]), add2(g2[2], g2[3])), a, b);
                        total += a + b;
                    }
                    if (!kRows && ok) {
                        if (t < unit.L) {                  // a token of its own for every thread
                            if (unit.bad) {
                                const int id = p.block_tables[(size_t)unit.b * p.max_blocks + t / BS];
                                if (id < 0 || id >= p.num_blocks) total = 0.f;
                            }
                            float* const at = p.weights + ((size_t)unit.to * p.num_kv_heads + unit.hk) * p.max_tokens + t;
                            *at = t < unit.L - unit.C ? fmaf(p.decay, *at, total) : total;
                        }
                        total = 0.f;
                    }
                }
                if (kRows) {
                    if (ok && u > 0) ok = wait(kBarPartFree, u - 1);
                    if (!ok) break;
                    reinterpret_cast<float*>(smem + S::kPart)[group * kTile + me] = total;
                }
            }
            __syncwarp();
            if (ok) mbar_arrive_elect(bar(kBarPart));
        }
        if (!ok && lane == 0) flag_error(p.err, kErrTimeout);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::dealloc(tmem, kTmemCols);
    }
}

// The splits' statistics of a row to its M_r, eight reads of a thread in flight. More than eight
// splits (dozens of a prompt's last rows, hundreds of one long sequence) are shared by four threads
// a row: the last 32 rows of 4 prompts of 32768, 59 splits, take 88 us with four and 92 with one. A
// chunk has many rows and few splits: 4 of 2048 take 236 us with four and 232 with one.
constexpr int kMergeParts = 4;
__global__ void __launch_bounds__(kTile * kMergeParts) weigh_merge_kernel(const Params p, int block_size, int tile_bytes) {
    pdl_enter();
    const int rt = blockIdx.x, item = blockIdx.y, me = threadIdx.x % kTile, part = threadIdx.x / kTile, num_parts = blockDim.x / kTile;
    Chunk ch;
    ch.read(p, item / p.num_kv_heads, block_size);
    const int nr = ch.w * p.G;
    if (rt * kTile >= nr) return;
    // as the first pass split them: the tiles that it held together
    const int last_tile = p.row_tiles == 1 ? rt : rt | 1;
    const int seen_tiles = (ch.L - ch.w + (min(nr, (last_tile + 1) * kTile) - 1) / p.G) / kTile + 1;
    const int tiles = (ch.L + kTile - 1) / kTile, ns = min(p.splits, (tiles + p.per - 1) / p.per);
    const int per = (seen_tiles + ns - 1) / ns, splits = (seen_tiles + per - 1) / per;
    const size_t tile = (size_t)item * p.row_tiles + rt;
    const float2* const at = p.stats + tile * p.splits * kTile + me;
    __shared__ float2 parts[kMergeParts][kTile];
    float m = -INFINITY, l = 0.f;
    for (int s0 = part; s0 < splits; s0 += 8 * num_parts) {
        float2 x[8];
        float mx = m;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int s = s0 + k * num_parts;
            x[k] = s < splits ? at[(size_t)s * kTile] : make_float2(-INFINITY, 0.f);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) mx = max_nan(mx, x[k].x);
        const float by = mx == -INFINITY ? 0.f : mx;
        l *= ex2(m - by);
#pragma unroll
        for (int k = 0; k < 8; ++k) l += ex2(x[k].x - by) * x[k].y;
        m = mx;
    }
    if (num_parts > 1) {
        parts[part][me] = make_float2(m, l);
        __syncthreads();
        if (part > 0) return;
        for (int k = 1; k < num_parts; ++k) m = max_nan(m, parts[k][me].x);
        const float by = m == -INFINITY ? 0.f : m;
        l = 0.f;
        for (int k = 0; k < num_parts; ++k) l += ex2(parts[k][me].x - by) * parts[k][me].y;
    }
    write_base(p.q_tiles + tile * (tile_bytes + kExt) + tile_bytes, me, m, l, rt * kTile + me < nr, p.scale_log2);
}

// Tiles, and units of both passes: about kTargetUnits each
struct Shape {
    long long items, row_tiles, key_tiles, per, splits, key_pairs, row_parts;
    Shape(int num_seqs, int num_kv_heads, int G, int max_query_len, int window, int max_blocks, int block_size) {
        const long long w = window > 0 && window < max_query_len ? window : max_query_len;
        items = (long long)num_seqs * num_kv_heads;
        row_tiles = (w * G + kTile - 1) / kTile;
        key_tiles = ((long long)max_blocks * block_size + kTile - 1) / kTile;
        const long long held = row_tiles > 1 ? items * ((row_tiles + 1) / 2) : items;
        per = (held * key_tiles + kTargetUnits - 1) / kTargetUnits;
        if (per < 4) per = 4;
        splits = (key_tiles + per - 1) / per;
        const long long most = kTargetUnits / (held > 0 ? held : 1) + 1;
        if (splits > most) splits = most;                  // what the workspace holds
        if (splits < 1) splits = 1;
        key_pairs = (key_tiles + 1) / 2;
        const long long pairs = items * key_pairs;
        row_parts = pairs > 0 && pairs < kTargetUnits ? (kTargetUnits + pairs - 1) / pairs : 1;
        if (row_parts > (row_tiles + 3) / 4) row_parts = (row_tiles + 3) / 4;   // four row tiles or so at least
        if (row_parts < 1) row_parts = 1;
    }
    // of the workspace: the next unit, the row runs' arrivals and gains, whatever the shape (pairs
    // that have row runs are below kTargetUnits, and all their runs below twice that)
    static constexpr size_t kCounters = 128 + (size_t)kTargetUnits * 4, kParts = 2 * (size_t)kTargetUnits * 2 * kTile * 4;
};

template <int D, int BS>
int launch(const Params& p, cudaStream_t stream) {
    using S = Shared<D>;
    auto stats = p.row_tiles == 1 ? weigh_kernel<kStats, 1, D, BS> : weigh_kernel<kStats, 2, D, BS>;
    auto gain = p.row_tiles == 1 ? weigh_kernel<kGainKeys, 1, D, BS> : weigh_kernel<kGainRows, 2, D, BS>;
    int occ = 0;
    int st = kernel_setup(reinterpret_cast<const void*>(stats), S::kBytes, kThreads, &occ);
    if (st != PKV_OK) return st;
    st = kernel_setup(reinterpret_cast<const void*>(gain), S::kBytes, kThreads, &occ);
    if (st != PKV_OK) return st;
    // no more CTAs than there can be units
    const long long all = (long long)p.num_seqs * p.num_kv_heads * p.row_tiles * p.splits;
    const int sms = num_sms();
    note_launch();
    cudaError_t e = launch_pdl(stats, dim3((unsigned)(all < sms ? all : sms)), dim3(kThreads), S::kBytes, stream, p);
    if (e != cudaSuccess) return cuda_fail("weigh_prefill_tokens: statistics launch", e);
    if (p.splits > 1) {
        note_launch();
        e = launch_pdl(weigh_merge_kernel, dim3((unsigned)p.row_tiles, (unsigned)(p.num_seqs * p.num_kv_heads)),
                       dim3(p.splits > 8 ? kTile * kMergeParts : kTile), 0, stream, p, BS, S::kTileBytes);
        if (e != cudaSuccess) return cuda_fail("weigh_prefill_tokens: merge launch", e);
    }
    note_launch();
    e = launch_pdl(gain, dim3((unsigned)sms), dim3(kThreads), S::kBytes, stream, p);
    return e == cudaSuccess ? PKV_OK : cuda_fail("weigh_prefill_tokens: weights launch", e);
}

}  // namespace weigh
}  // namespace pkv

extern "C" size_t weigh_prefill_workspace_size(int num_seqs, int num_heads, int max_query_len, int window) {
    using namespace pkv::weigh;
    if (num_seqs <= 0 || num_heads <= 0 || max_query_len <= 0 || window < 0) return 0;
    // at most (sequences x heads) x (queries + 127) rows, 288 bytes and a pair of statistics each,
    // and the pairs of the splits; what Shape counts
    const long long w = window > 0 && window < max_query_len ? window : max_query_len;
    const size_t rows = (size_t)num_seqs * num_heads * (size_t)(w + kTile - 1);
    return Shape::kCounters + Shape::kParts + rows * (256 + 32 + 8) + 2 * (size_t)kTargetUnits * kTile * 8;
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
        (block_size != 16 && block_size != 32) || G > weigh::kMaxGroup ||
        (scale != 0.f && std::fabs(scale) < 0x1p-100f))        // M_r / scale has to be a number
        return PKV_ERR_UNSUPPORTED;
    const weigh::Shape shape(num_seqs, num_kv_heads, G, max_query_len, window, max_blocks_per_seq, block_size);
    // units, rows and positions times a group in 32 bits
    if (shape.items > 65535 || shape.row_tiles > 65535 || shape.items * shape.row_tiles * shape.splits > 0x3fffffff ||
        shape.items * shape.key_tiles > 0x3fffffff ||
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
    p.per = (int)shape.per;
    p.g_magic = (uint32_t)(0x100000000ull / (unsigned)G) + 1u;
    p.scale_log2 = scale == 0.f ? 1.f : std::fabs(scale) * 1.4426950408889634f;
    p.no_scale = scale == 0.f;
    p.sign = scale < 0.f ? 0x80008000u : 0u;
    p.decay = decay;
    p.key_pairs = (int)shape.key_pairs;
    p.row_parts = (int)shape.row_parts;
    p.next = static_cast<int*>(workspace);
    p.arrived = p.next + 32;
    p.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + weigh::Shape::kCounters);
    p.q_tiles = reinterpret_cast<unsigned char*>(p.parts) + weigh::Shape::kParts;
    const size_t row_count = (size_t)(shape.items * shape.row_tiles) * weigh::kTile;
    p.stats = reinterpret_cast<float2*>(p.q_tiles + row_count * (head_dim * 2 + 32));
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
