// Decode attention with token weights: paged_attention_decode_weighed.
//
// Mathematics. The output is the decode's (online softmax, tile by tile). The weight of a
// token is its softmax probability, which needs the row's final maximum and sum: only known
// after the last tile. So the logits, 4 bytes a (query head, token) beside the 2 D elements
// of K and V that the token costs anyway, are kept, and a second kernel turns them into
// probabilities, adds up the heads of a kv head and updates the weights: no second read of K.
//
// First kernel: a CTA takes a partition (a run of a (sequence, kv head)'s tiles), its warps
// every fourth tile of it through a ring of their own, with the sparse decode's tile math; the
// warps' parts (maximum, sum, unnormalised output) meet in shared memory and go to the
// workspace, or to the output where the row has one partition. Second kernel: a CTA merges the
// partitions' maxima and sums of its row, which gives each head's maximum and sum, and updates
// 1024 or 2048 tokens' weights; the outputs of a row in several partitions are merged by its first
// CTA, or by one a head.
// Bound: HBM bytes for many tokens (32 sequences of up to 8192, 40 bf16 heads of 128: 415 us,
// 0.99 of the copy rate); of E4M3 no unit (64 of up to 4096, 4 heads a kv head: 61.1, 0.67): three
// warps a scheduler, each a chain of fragments, products and exponentials, issue on 0.42 of the cycles,
// tensor pipe 0.26, HBM 0.65. Float32 heads of 64: arithmetic of the CUDA cores beside HBM (16 x 8192:
// one head a kv head 45 us, four 53, floor 40). Few tokens: two launches and their chains of loads
// (1 x 4096: 8.5 us).
// Many short partitions rather than whole rows: 4096 CTAs 415 us, 2048 434, 1024 449 (E4M3: 60.2,
// 60.8, 65.7); 4 tiles a partition instead of 8 make 1 x 4096 12.2 us, 16 no difference.
#pragma once

#include <type_traits>

#include "pkv_sparse_impl.cuh"

namespace pkv {
namespace weighed {

using decode::kFull;
using decode::kLog2e;
using sparse::begin_row;
using sparse::ex2;
using sparse::max_nan;
using sparse::softmax_base;

constexpr int kWarps = 4;
constexpr int kMaxStages = 8;          // of a warp's ring
constexpr int kPartStages = 8;         // tiles of a partition, at least
// Partitions of a row, at most, and of few rows so many that they make kWave CTAs, three on each of 152
// SMs: merging them is the row's last step. 1 x 65536 (8 heads a kv head) 54 us, 78 with 512 partitions a
// row; 2 x 16384 without groups 23.4 and 30.1; 16 x 8192 (4 heads) 48.9 with 12 a row, 52.0 with 32, 51.6
// with 16, 55.7 with 8. Heads of 64, of which an SM holds four CTAs, gain nothing from a fourth more: with
// 608 1 x 65536 takes 33.0 us (31.0 with 456; E4M3 21.2 and 23.0), 4 x 8192 12.9 (14.1), 2 x 16384 16.2 (16.4).
constexpr int kRowParts = 12, kWave = 456;
constexpr int kMaxCtas = 4096;         // partitions are made until there are so many

struct Params {
    void* out;
    float* weights;                    // [rows][Hkv][max_tokens]
    const int32_t* rows;
    const void* q;
    const char* k_pool;
    const char* v_pool;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    float* logits;                     // [B][Hq][pitch], in units of log2 e
    float* part_ml;                    // [B * Hkv][parts][2][G]
    float* part_o;                     // [B * Hkv][parts][G][D]
    int* err;
    int max_blocks, num_blocks, num_rows, max_tokens, num_kv_heads;
    int pitch, parts, part_stages;     // partitions of a row, at most; tiles of one, at least
    int merge_ctas;                    // of a row, in the second kernel: one, or one a head; 0: rows have one partition
    float qscale, v_scale, decay, lift;
};

struct Args {
    Params p;
    int num_seqs, num_heads, head_dim, block_size;
    float scale, k_scale;
    void* workspace;
    cudaStream_t stream;
};

// Tokens of logits a head has room for: whole tiles of up to 32
inline int logits_pitch(int max_blocks, int block_size) { return (max_blocks * block_size + 31) / 32 * 32; }

// Shared memory: mbarriers | tiles' tokens | (CUDA-core math) query rows, scratch | rings.
// The warps' parts go where the rings were.
template <class Math, int D, int BS, int G>
struct Smem {
    // CTAs of an SM: four where heads of 64 leave registers for them, else three (16 sequences of 8192, 4
    // heads a kv head, with three and with four: bf16 of 64 34.4 and 31.0 us, E4M3 28.3 and 25.4; of 128
    // 51.2 and 52.6, 38.0 and 37.4, a batch of 64 60.2 and 63.1; float32 of 64, 8 heads, 101 and 107)
    static constexpr int kCtas = D == 64 && Math::Lay::kTile / (D * BS) < 4 ? 4 : 3;
    static constexpr int kRegisters = 65536 / (kCtas * kWarps * 32) / 8 * 8;
    static constexpr bool kSimt = Math::kWarpSmemFloats > 0;
    static constexpr int kStage = 2 * Math::Lay::kTile;
    static constexpr int kPartFloats = G * (D + 4);        // m [G], l [G], (pad), o [G][D]
    static constexpr int kO = 4 * G;
    static constexpr int kTok = kWarps * kMaxStages * 8;
    static constexpr int kQ = kTok + kWarps * kMaxStages * 4;
    static constexpr int kScratch = kQ + (kSimt ? kWarps * G * D * 4 : 0);
    static constexpr int kRing = (kScratch + kWarps * Math::kWarpSmemFloats * 4 + 127) / 128 * 128;
    static constexpr int kMinStages = (kPartFloats * 4 + kStage - 1) / kStage;   // a part fits
    static constexpr int kFit = (sparse::kSmemSm / kCtas - 1024 - kRing) / (kWarps * kStage);
    static constexpr int kStages = kFit < kMinStages ? kMinStages : kFit > kMaxStages ? kMaxStages : kFit;
    static constexpr int kBytes = kRing + kWarps * kStages * kStage;
    static_assert(kBytes <= sparse::kSmemSm, "shared memory per CTA");
};

// Tiles of a row's partitions: its own length tells, as the tables may be much wider (1 x 4096 in tables of
// 131072 tokens 9.6 us; 35 with the width's partitions)
__device__ __forceinline__ int part_stages(const Params& p, int stages) {
    return max(p.part_stages, (stages + p.parts - 1) / p.parts);
}

// Keeps a tile's logits: at[head][token], tokens below `limit`
struct Keep {
    float* at;
    int pitch, heads, limit;
    __device__ __forceinline__ void put(int g, int t, float a, float b) const {
        if (g < heads && t < limit) *reinterpret_cast<float2*>(at + (size_t)g * pitch + t) = make_float2(a, b);
    }
    __device__ __forceinline__ void put(int g, int t, float a, float b, float c, float d) const {
        if (g < heads && t < limit) *reinterpret_cast<float4*>(at + (size_t)g * pitch + t) = make_float4(a, b, c, d);
    }
    __device__ __forceinline__ void put(int g, int t, float a) const {
        if (t < limit) at[(size_t)g * pitch + t] = a;
    }
};

// PAIR = 2: a stage holds two blocks of BS / 2 tokens side by side; BS is then the stage's. HALVES = 2:
// it holds one half of a block (its K and its V are whole runs of the block's).
template <class Math, typename QT, int D, int BS, int G, int PAIR, int HALVES>
__global__ void __maxnreg__((Smem<Math, D, BS, G>::kRegisters)) weighed_decode_kernel(const Params p) {
    using S = Smem<Math, D, BS, G>;
    constexpr int TILE = Math::Lay::kTile, PBS = BS / PAIR, PTILE = TILE / PAIR, ST = S::kStages;
    static_assert(PAIR == 1 || HALVES == 1, "one or the other");
    pdl_enter();
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    unsigned char* const ring = smem + S::kRing + w * ST * S::kStage;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem) + w * kMaxStages;
    int32_t* stage_tok = reinterpret_cast<int32_t*>(smem + S::kTok) + w * kMaxStages;
    float* qs = reinterpret_cast<float*>(smem + S::kQ) + w * G * D;
    float* pb = reinterpret_cast<float*>(smem + S::kScratch) + w * Math::kWarpSmemFloats;
    const int row = blockIdx.x / p.parts, part = blockIdx.x - row * p.parts;
    const int b = row / p.num_kv_heads, hk = row - b * p.num_kv_heads;
    int L = p.seq_lens[b];
    if (L < 0 || L > p.max_blocks * (PBS * HALVES)) {
        if (tid == 0) flag_error(p.err, kErrOutOfRange);
        L = L < 0 ? 0 : p.max_blocks * (PBS * HALVES);
    }
    const int stages = (L + BS - 1) / BS, per = part_stages(p, stages);
    const int s0 = part * per, s1 = min(stages, s0 + per);
    if (s0 >= s1 && part > 0) return;                      // the first partition writes a row without tokens
    const int nk = max(0, (s1 - s0 - w + kWarps - 1) / kWarps);    // this warp's tiles: s0 + w, + kWarps, ...

    if (lane < ST) mbar_init(smem_addr(&bars[lane]), 1);
    fence_mbar_init();
    __syncwarp();
    const uint64_t pol = l2_evict_first();
    const int32_t* const table = p.block_tables + (size_t)b * p.max_blocks;
    // the tile of the sequence's block (half block) j (-1: none)
    auto tile_of = [&](int j) -> int {
        if (j * PBS >= L) return -1;
        const int id = table[j / HALVES];
        if (id < 0 || id >= p.num_blocks) {
            flag_error(p.err, kErrOutOfRange);
            return -1;
        }
        return (id * p.num_kv_heads + hk) * HALVES + j % HALVES;
    };
    int id_a = -1, id_b = -1, chunk = -1;
    auto issue = [&](int kk, int s) {                      // this warp's tile kk into slot s
        if ((kk >> 5) != chunk) {
            chunk = kk >> 5;
            const int j = (s0 + w + kWarps * ((chunk << 5) + lane)) * PAIR;
            const bool mine = (chunk << 5) + lane < nk;
            id_a = mine ? tile_of(j) : -1;
            id_b = mine && PAIR == 2 ? tile_of(j + 1) : -1;
            __syncwarp();
        }
        const uint32_t bar = smem_addr(&bars[s]);
        int ia = __shfl_sync(kFull, id_a, kk & 31), ib = PAIR == 2 ? __shfl_sync(kFull, id_b, kk & 31) : -1;
        const int left = L - (s0 + w + kWarps * kk) * BS;  // tokens from this tile on
        int tok = (ia >= 0 ? min(PBS, left) : 0) + (ib >= 0 ? min(PBS, left - PBS) : 0), alone = 0;
        if (PAIR == 2 && ia < 0 && ib >= 0) {              // the second block alone moves up
            ia = ib;
            ib = -1;
            alone = 1 << 16;
        }
        if (lane == 0) stage_tok[s] = tok | alone;
        __syncwarp();
        if (ia >= 0) {
            const uint32_t dst = smem_addr(ring + (size_t)s * S::kStage);
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

    float* const logits = p.logits + (size_t)row * G * p.pitch;
    typename Math::State st;
    begin_row<Math, QT, D, G>(st, static_cast<const QT*>(p.q) + (size_t)row * G * D, p.qscale, qs, lane);
    bool aborted = false;
    int k = 0, s = 0;
    uint32_t phase = 0;
    for (; k < nk; ++k) {
        const bool ok = mbar_wait_bounded(smem_addr(&bars[s]), phase, p.err);
        if (__any_sync(kFull, !ok)) {
            aborted = true;
            break;
        }
        const int word = stage_tok[s], ntok = word & 0xffff, first = (s0 + w + kWarps * k) * BS;
        const int have = min(BS, L - first), shift = word >> 16 ? PBS : 0;
        if (ntok < have)                                   // blocks that are not there
            for (int i = lane; i < G * have; i += 32) {
                const int g = i / have, t = i - g * have;
                if (shift ? t < PBS : t >= ntok) logits[(size_t)g * p.pitch + first + t] = -INFINITY;
            }
        if (ntok > 0) {
            unsigned char* kt = ring + (size_t)s * S::kStage;
            const Keep keep{logits + first + shift, p.pitch, G, shift ? PBS : BS};
            if constexpr (S::kSimt) {
                Math::tile(st, kt, kt + TILE, ntok, lane, qs, pb, keep);
            } else {
                if (ntok < BS) Math::clear_tail(kt + TILE, ntok, lane);
                Math::tile(st, kt, kt + TILE, ntok, lane, p.qscale, keep);
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
    if (aborted) {                                         // record it and let the copies in flight land
        if (lane == 0) flag_error(p.err, kErrTimeout);
        for (int kk = k; kk < min(nk, k + ST); ++kk) {
            (void)mbar_wait_bounded(smem_addr(&bars[s]), phase, nullptr);
            if (++s == ST) {
                s = 0;
                phase ^= 1;
            }
        }
    }
    // ---- the warps' parts to one
    __syncwarp();
    float* const part_w = reinterpret_cast<float*>(ring);
    Math::finish(st, part_w, part_w + G, part_w + S::kO, 0, lane, aborted);
    __syncthreads();
    auto part_of = [&](int x) { return reinterpret_cast<const float*>(smem + S::kRing + x * ST * S::kStage); };
    float* const ml = p.part_ml + ((size_t)row * p.parts + part) * 2 * G;
    for (int i = tid; i < G * D / 4; i += kWarps * 32) {
        const int g = 4 * i / D;
        float M = -INFINITY, sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < kWarps; ++x) M = max_nan(M, part_of(x)[g]);
        const float base = softmax_base(M);
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
            const float* from = part_of(x);
            const float e = ex2(from[g] - base);
            const float4 o = *reinterpret_cast<const float4*>(from + S::kO + 4 * i);
            sum += e * from[G + g];
            v.x += e * o.x;
            v.y += e * o.y;
            v.z += e * o.z;
            v.w += e * o.w;
        }
        if (4 * i % D == 0) {
            ml[g] = M;
            ml[G + g] = sum;
        }
        if (p.parts > 1) {
            *reinterpret_cast<float4*>(p.part_o + (((size_t)row * p.parts + part) * G) * D + 4 * i) = v;
        } else {
            const float by = sum > 0.f ? p.v_scale / sum : 0.f;
            QT* dst = static_cast<QT*>(p.out) + (size_t)row * G * D + 4 * i;
            decode::store_out(dst, v.x * by);
            decode::store_out(dst + 1, v.y * by);
            decode::store_out(dst + 2, v.z * by);
            decode::store_out(dst + 3, v.w * by);
        }
    }
}

constexpr int kFinishThreads = 256;
// Pieces of four tokens a thread: what a CTA reads for its row is shared by more of them (both
// kernels, 32 sequences of up to 8192 tokens and 40 heads: 420.6 us with one, 415.0 with two; 64 of up
// to 4096, E4M3: 60.7 and 60.2). Eight heads' logits leave no registers for two.
template <int G> struct Finish {
    static constexpr int kPieces = G <= 4 ? 2 : 1, kTokens = 4 * kPieces * kFinishThreads;
};

template <typename QT, int D, int G>
__global__ void __launch_bounds__(kFinishThreads) weighed_finish_kernel(const Params p, int stage_tokens, int max_len) {
    __shared__ float head_m[G], head_inv[G];               // of each head: maximum, 1 / sum
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int row = blockIdx.y, b = row / p.num_kv_heads, hk = row - b * p.num_kv_heads;
    // Read before the first kernel is through: lengths, rows and weights, which it does not write
    // (and it began behind everything that did). 1 sequence of 4096 tokens: 1.2 us of 9.1.
    const int L = min(max(p.seq_lens[b], 0), max_len);     // flagged by the first kernel
    const bool merges = (int)blockIdx.x < p.merge_ctas;    // the first CTAs of a row in several partitions
    const int t0 = ((int)blockIdx.x - p.merge_ctas) * Finish<G>::kTokens, t = t0 + 4 * tid;
    if (!merges && t0 >= L) {                              // the whole CTA
        if (blockIdx.x == 0) pdl_enter();                  // some CTA waits: what waits for this kernel waits for the first
        return;
    }
    int to = b;
    bool bad = false;
    if (!merges && p.rows) {                               // good, and no earlier sequence's
        to = p.rows[b];
        bad = to < 0 || to >= p.num_rows;
        for (int i = tid; i < b; i += kFinishThreads) bad |= p.rows[i] == to;
    }
    constexpr int N = Finish<G>::kPieces, kStep = 4 * kFinishThreads;
    float4 x[N][G], before[N];
    float* const at = p.weights + ((size_t)to * p.num_kv_heads + hk) * p.max_tokens + t;
#pragma unroll
    for (int n = 0; n < N; ++n)
        if (!merges && t + n * kStep < L && !(to < 0 || to >= p.num_rows))
            before[n] = *reinterpret_cast<const float4*>(at + n * kStep);
    pdl_enter();
    const int stages = (L + stage_tokens - 1) / stage_tokens;
    const int per = part_stages(p, stages), parts = max(1, (stages + per - 1) / per);
    const float* const ml = p.part_ml + (size_t)row * p.parts * 2 * G;
#pragma unroll
    for (int n = 0; n < N; ++n)
        if (!merges && t + n * kStep < L)
#pragma unroll
            for (int g = 0; g < G; ++g)
                x[n][g] = *reinterpret_cast<const float4*>(p.logits + ((size_t)row * G + g) * p.pitch + t + n * kStep);
    if (w < G) {
        float M = -INFINITY, sum = 0.f;
        for (int i = lane; i < parts; i += 32) M = max_nan(M, ml[i * 2 * G + w]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) M = max_nan(M, __shfl_xor_sync(kFull, M, o));
        const float base = softmax_base(M);
        for (int i = lane; i < parts; i += 32) sum += ex2(ml[i * 2 * G + w] - base) * ml[i * 2 * G + G + w];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        if (lane == 0) {
            head_m[w] = base;
            head_inv[w] = M == -INFINITY ? 0.f : 1.f / sum;   // a NaN sum stays one
        }
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) flag_error(p.err, kErrOutOfRange);
        return;
    }
    if (!merges) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int tn = t + n * kStep;
            if (tn >= L) return;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float m = head_m[g], by = head_inv[g] * p.lift;
                sum[0] += ex2(x[n][g].x - m) * by;
                sum[1] += ex2(x[n][g].y - m) * by;
                sum[2] += ex2(x[n][g].z - m) * by;
                sum[3] += ex2(x[n][g].w - m) * by;
            }
            float* const to_n = at + n * kStep;
            const float old[4] = {before[n].x, before[n].y, before[n].z, before[n].w};
            if (tn + 4 < L) {                              // four older ones
                *reinterpret_cast<float4*>(to_n) = make_float4(fmaf(p.decay, old[0], sum[0]), fmaf(p.decay, old[1], sum[1]),
                                                               fmaf(p.decay, old[2], sum[2]), fmaf(p.decay, old[3], sum[3]));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (tn + j < L) to_n[j] = tn + j < L - 1 ? fmaf(p.decay, old[j], sum[j]) : sum[j];
            }
        }
        return;
    }
    // ---- the partitions' outputs: J threads a piece of four dims, over every J-th partition each
    __shared__ float4 sums[kFinishThreads];
    auto merge = [&](auto heads_of_this, int first_head) {
        constexpr int kQuads = decltype(heads_of_this)::value * (D / 4), J = kFinishThreads / kQuads;
        const int i = first_head * (D / 4) + tid % kQuads, g = 4 * i / D;
        const float4* const o = reinterpret_cast<const float4*>(p.part_o) + (size_t)row * p.parts * G * (D / 4) + i;
        const float m = head_m[g];
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int k = tid / kQuads; k < parts; k += J) {
            const float e = ex2(ml[k * 2 * G + g] - m);
            const float4 a = o[(size_t)k * G * (D / 4)];
            v.x += e * a.x;
            v.y += e * a.y;
            v.z += e * a.z;
            v.w += e * a.w;
        }
        if constexpr (J > 1) {
            sums[tid] = v;
            __syncthreads();
            if (tid >= kQuads) return;
#pragma unroll
            for (int j = 1; j < J; ++j) {
                const float4 a = sums[tid + j * kQuads];
                v.x += a.x;
                v.y += a.y;
                v.z += a.z;
                v.w += a.w;
            }
        }
        const float by = head_inv[g] * p.v_scale;
        QT* const dst = static_cast<QT*>(p.out) + (size_t)row * G * D + 4 * i;
        decode::store_out(dst, v.x * by);
        decode::store_out(dst + 1, v.y * by);
        decode::store_out(dst + 2, v.z * by);
        decode::store_out(dst + 3, v.w * by);
    };
    if (G > 1 && p.merge_ctas > 1) merge(std::integral_constant<int, 1>(), (int)blockIdx.x);
    else merge(std::integral_constant<int, G>(), 0);
}

template <class Math, typename QT, int D, int BS, int G, int PAIR, int HALVES = 1>
int launch(const Args& a) {
    using S = Smem<Math, D, BS, G>;
    constexpr int BLOCK = BS / PAIR * HALVES;
    auto kern = weighed_decode_kernel<Math, QT, D, BS, G, PAIR, HALVES>;
    int occ = 0;
    const int st = kernel_setup(reinterpret_cast<const void*>(kern), S::kBytes, kWarps * 32, &occ);
    if (st != PKV_OK) return st;
    Params p = a.p;
    const long long rows = (long long)a.num_seqs * p.num_kv_heads;
    const int stages = (p.max_blocks * BLOCK + BS - 1) / BS;
    long long parts = (kMaxCtas + rows - 1) / rows;
    const long long cap = kRowParts > kWave / rows ? kRowParts : kWave / rows;
    if (parts > cap) parts = cap;
    const int most = stages / kPartStages;
    if (parts > most) parts = most;
    if (parts < 1) parts = 1;
    p.parts = (int)parts;
    // rows enough for kMaxCtas: longer ones do (64 sequences of up to 4096, E4M3: 61.2 us, 63.5 with 8 tiles)
    p.part_stages = rows * parts >= kMaxCtas ? 2 * kPartStages : kPartStages;
    // a CTA a head while those are few (1 x 65536, 8 heads, 512 partitions: 78 us, one a row 97), else their
    // number tells (64 sequences of up to 4096, E4M3, 4 heads: 65.8 and 60.2)
    p.merge_ctas = p.parts == 1 ? 0 : rows * G <= 2 * num_sms() ? G : 1;
    p.qscale = a.scale * a.k_scale * kLog2e;
    p.lift = 1.f;
    if constexpr (!S::kSimt) p.lift = Math::kLift == 0.f ? 1.f : 16384.f;
    p.logits = static_cast<float*>(a.workspace);
    p.part_o = p.logits + (size_t)rows * G * p.pitch;
    p.part_ml = p.part_o + (size_t)rows * p.parts * G * D;
    if (rows * p.parts > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
    note_launch();
    cudaError_t e = launch_pdl(kern, dim3((unsigned)(rows * p.parts)), dim3(kWarps * 32), S::kBytes, a.stream, p);
    if (e != cudaSuccess) return cuda_fail("weighed decode: kernel launch", e);
    note_launch();
    const dim3 grid((unsigned)((p.max_blocks * BLOCK + Finish<G>::kTokens - 1) / Finish<G>::kTokens + p.merge_ctas), (unsigned)rows);
    e = launch_pdl(weighed_finish_kernel<QT, D, G>, grid, dim3(kFinishThreads), 0, a.stream, p, (int)BS,
                   p.max_blocks * BLOCK);
    return e == cudaSuccess ? PKV_OK : cuda_fail("weighed decode: weights launch", e);
}

// as the sparse decode chooses (pkv_sparse_impl.cuh); blocks of 32 float32 tokens of 128 dims, of which the
// ring has room for one a warp, by halves (16 sequences of 8192 tokens, 8 kv heads of one query
// head: 96.5 us whole, 80.8 by halves; of 4: 142 and 99.8)
template <typename QT, typename KV, int D, int BS, int G>
int launch_heads(const Args& a) {
    if constexpr (std::is_same<KV, float>::value && D == 128 && BS == 32)
        return launch<sparse::SimtSums<QT, KV, D, BS / 2, G>, QT, D, BS / 2, G, 1, 2>(a);
    else if constexpr (std::is_same<KV, float>::value || (G == 1 && !std::is_same<KV, uint8_t>::value))
        return launch<sparse::SimtSums<QT, KV, D, BS, G>, QT, D, BS, G, 1>(a);
    else if constexpr (BS == 16 && std::is_same<KV, uint8_t>::value)
        return launch<sparse::HeadsMath<KV, D, 2 * BS, G>, QT, D, 2 * BS, G, 2>(a);
    else return launch<sparse::HeadsMath<KV, D, BS, G>, QT, D, BS, G, 1>(a);
}

template <typename QT, typename KV, int D, int BS>
int dispatch_group(const Args& a) {
    switch (a.num_heads / a.p.num_kv_heads) {
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

}  // namespace weighed
}  // namespace pkv
