// Cache eviction: select_tokens (the tokens of the highest accumulated weight, exactly) and
// keep_tokens (their move to the front of fresh blocks).
//
// select_tokens. A row is one (sequence, kv head): up to hundreds of thousands of float32
// weights, of which the R = num_kept - first - last largest between the always-kept ends are
// wanted, ties to the lower token. The weights become 32-bit keys that order as unsigned
// numbers, are read once into registers (of one CTA, or of a cluster's, a contiguous slice
// each), and the R-th largest is found by narrowing the range of keys that it lies in: from the
// smallest and largest key there are, 2048 bins over the range are counted, summed over the
// cluster through distributed shared memory, and the bin that holds the R-th is the next range
// (at most three times; once or twice where weights differ, as the bins begin where the weights
// do: a fixed first digit left a tenth of the keys in one bin). The taken keys are those above
// the threshold and the first few equal to it; prefix sums over threads, warps and CTAs give
// each its place in the list, which so comes out ascending. Bound, few rows: the chain of passes and
// barriers, not the reads (4 bytes a token); many: instructions, 72 for 32 keys, which an SM with three
// or four rows issues on 0.63 of its cycles, the busiest on 0.80 (the bins' additions are 1.8% of them and
// take 6% of the shared memory's cycles). Rows of 8192: 64 of them 6.1 us, 152 7.0, 304 8.4, 512 12.5 (14.0
// where lengths differ; the bytes 3.1); 8 rows of 131072, in clusters, 19 us.
//
// keep_tokens. K: 16-byte pieces, one per (token, X dims), to their new place: eight
// neighbouring threads write a whole 128-byte core matrix. V is stored transposed: 16 bytes are X
// tokens of one dim, so a thread reads such a piece of each group that its X tokens come from and
// puts their bytes together. Source and target blocks are disjoint, so nothing waits. The weights
// move within their row: kept[i] >= i, so one CTA a row that reads a chunk of the list's weights,
// waits for all its threads, and writes them, overwrites nothing that a later chunk reads. Bound:
// HBM bytes, of K in sectors of 32 that two tokens share: 4096 of 8192 random tokens of 64
// sequences (bf16, 8 heads of 128) move 2.2 GB in 410 us, 5.3 TB/s; with the neighbours' halves of
// the sectors 2.9 GB, 7.2 TB/s. CTAs of their own for K and V took 480 us where one took 430.
#include <cuda_runtime.h>

#include <type_traits>

#include "pkv_check.cuh"
#include "pkv_internal.cuh"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// The weight row of sequence b: -1 (flagged) where it is out of range, or where an earlier
// sequence has it and `unique` asks for that. The whole CTA calls it.
__device__ __forceinline__ int weight_row(const int32_t* rows, int b, int num_rows, bool unique, int* err) {
    if (!rows) return b;                                   // the host has checked num_rows
    const int row = rows[b];
    bool bad = row < 0 || row >= num_rows;
    if (unique) {
        bool again = false;
        for (int i = threadIdx.x; i < b; i += blockDim.x) again |= rows[i] == row;
        bad |= __syncthreads_or(again) != 0;
    }
    if (bad && threadIdx.x == 0) flag_error(err, kErrOutOfRange);
    return bad ? -1 : row;
}

// ------------------------------------------------------------------ select_tokens
constexpr int kBins = 2048, kPasses = 3;                   // 11 bits a pass, of 32
constexpr int kMaxCluster = 8;                             // the portable size

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
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ uint2 cluster_ld2(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}

// A weight as an unsigned number of the same order; -0 as 0; what is not finite above the rest.
// Below all of them the key of no token, above them that of a token which is always kept.
constexpr uint32_t kNoKey = 0u, kNotFinite = 0xfffffffeu, kAlways = 0xffffffffu;
__device__ __forceinline__ uint32_t key_of(float w) {
    const uint32_t x = __float_as_uint(w + 0.f);
    const uint32_t key = x ^ ((uint32_t)((int)x >> 31) | 0x80000000u);
    return fabsf(w) <= 3.402823466e38f ? key : kNotFinite;
}
// One more in bin d >> shift, where d <= span: a predicated instruction, no branch
__device__ __forceinline__ void count_key(uint32_t bins, uint32_t d, uint32_t span, int shift) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.le.u32 p, %0, %1;\n\t@p red.shared.add.u32 [%2], 1;\n\t}" ::"r"(d), "r"(span),
                 "r"(bins + (d >> shift) * 4u)
                 : "memory");
}

struct SelectParams {
    int32_t* kept;
    const float* weights;
    const int32_t* rows;
    const int32_t* seq_lens;
    int* err;
    int num_kv_heads, num_rows, max_tokens, k, first, last;
    int least, most;                   // rows of more tokens than `least`, of at most `most`: the others are another launch's
};

// A CTA's slice of a row: NT threads, V pieces of 4 tokens each in registers (piece j of thread i
// at token 4 (j NT + i)); kLong: slices may be longer, further rounds are read from memory in
// every pass.
template <int NT, int V, bool kLong>
__global__ void __launch_bounds__(NT, 1024 / NT) select_tokens_kernel(const SelectParams p) {
    pdl_enter();
    constexpr int kWarps = NT / 32, kRound = NT * 4 * V, kPairs = kBins / 2 / NT;
    static_assert(kBins % (2 * NT) == 0, "bins a thread");
    __shared__ __align__(16) uint32_t hist[kPasses][kBins];
    __shared__ uint32_t warp_sum[kWarps], warp_min[kWarps], warp_max[kWarps];
    __shared__ uint32_t found[3];                          // digit, keys above it, keys of it
    __shared__ uint32_t run[V * kWarps];                   // taken in each piece of each warp; then before it
    __shared__ __align__(8) uint32_t cta_range[2], cta_taken[2], round_taken;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank(), csize = (int)cluster_size();
    const int item = (int)(blockIdx.x / csize), b = item / p.num_kv_heads, h = item - b * p.num_kv_heads;
    int n = p.seq_lens[b];
    if (n < 0 || n > p.max_tokens) {
        if (tid == 0) flag_error(p.err, kErrOutOfRange);
        n = n < 0 ? 0 : p.max_tokens;
    }
    if (n <= p.least || n > p.most) return;                // the whole cluster
    const int row = weight_row(p.rows, b, p.num_rows, false, p.err);
    if (row < 0) n = 0;
    int32_t* const out = p.kept + (size_t)item * p.k;
    if (n <= p.k) {                                        // the whole cluster
        for (int i = rank * NT + tid; i < p.k; i += csize * NT) out[i] = i < n ? i : -1;
        return;
    }
    // a row that one CTA holds is its own: no trips through the cluster
    const bool alone = csize == 1 || n <= kRound;
    if (alone && rank > 0) return;
    const int slice = alone ? n : ((n + csize - 1) / csize + 3) & ~3;
    const int begin = min(n, rank * slice), count = min(n, begin + slice) - begin;
    const float* const src = p.weights + ((size_t)row * p.num_kv_heads + h) * p.max_tokens + begin;
    // the tokens between the ends
    const int lo = max(0, p.first - begin), hi = min(count, n - p.last - begin);
    uint32_t key[V][4];
    auto load = [&](int round) {
        float4 v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {                      // a piece may pass n, not the row's end
            const int i = round * kRound + 4 * (j * NT + tid);
            v[j] = i < count ? *reinterpret_cast<const float4*>(src + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = round * kRound + 4 * (j * NT + tid);
            const float f[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) key[j][e] = key_of(f[e]);
            if (i < lo || i + 3 >= hi) {                   // an end of the sequence
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (i + e < lo || i + e >= hi) key[j][e] = i + e < count ? kAlways : kNoKey;
            }
        }
    };
    const int rounds = kLong ? (count + kRound - 1) / kRound : 1;
    auto each_round = [&](auto f) {                        // f(round) with its keys in registers
        for (int r = 0; r < rounds; ++r) {
            if (kLong && rounds > 1) load(r);
            f(r);
        }
    };
    auto sync = [&] {
        if (alone) __syncthreads();
        else cluster_sync();
    };
    if (!kLong || rounds <= 1) load(0);
    for (int i = tid; i < kPasses * kBins / 4; i += NT) reinterpret_cast<uint4*>(&hist[0][0])[i] = make_uint4(0, 0, 0, 0);
    uint32_t need = (uint32_t)(p.k - p.first - p.last);    // still to be found at or below the range
    uint32_t threshold = kNotFinite;                       // taken: keys above it, `need` equal ones
    if (need > 0) {
        // ---- the range of the keys: the first digit then tells apart what is there
        uint32_t mn = 0xffffffffu, mx = 0;
        each_round([&](int) {
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    mn = min(mn, key[j][e] - 1u);          // no key, always: they wrap to the other end
                    mx = max(mx, key[j][e] + 1u);
                }
        });
        mn = __reduce_min_sync(kFull, mn);
        mx = __reduce_max_sync(kFull, mx);
        if (lane == 0) {
            warp_min[w] = mn;
            warp_max[w] = mx;
        }
        __syncthreads();
        mn = __reduce_min_sync(kFull, warp_min[lane % kWarps]);
        mx = __reduce_max_sync(kFull, warp_max[lane % kWarps]);
        if (!alone) {
            if (tid == 0) {
                cta_range[0] = mn;
                cta_range[1] = mx;
            }
            cluster_sync();
            const uint2 r = lane < csize ? cluster_ld2(cluster_addr(cta_range, lane)) : make_uint2(0xffffffffu, 0u);
            mn = __reduce_min_sync(kFull, r.x);
            mx = __reduce_max_sync(kFull, r.y);
        }
        mx -= 1u;
        uint32_t base = mn + 1u, span = mx - base;         // keys base .. base + span hold the wanted one
        for (int pass = 0;; ++pass) {
            const int shift = max(0, 21 - __clz(span | 1u));
            uint32_t* const bins = hist[pass];
            const uint32_t at = smem_addr(bins);
            each_round([&](int) {
#pragma unroll
                for (int j = 0; j < V; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) count_key(at, key[j][e] - base, span, shift);
            });
            sync();
            // this thread's bins, two and two from the top down, and how many are above them
            uint2 c[kPairs];
            uint32_t sum = 0;
            const int top = kBins - 2 - 2 * kPairs * tid;
#pragma unroll
            for (int q = 0; q < kPairs; ++q) {
                if (alone) {
                    c[q] = *reinterpret_cast<const uint2*>(&bins[top - 2 * q]);
                } else {
                    uint2 x[kMaxCluster];
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r)
                        x[r] = r < csize ? cluster_ld2(cluster_addr(&bins[top - 2 * q], r)) : make_uint2(0, 0);
                    c[q] = make_uint2(0, 0);
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r) {
                        c[q].x += x[r].x;
                        c[q].y += x[r].y;
                    }
                }
                sum += c[q].x + c[q].y;
            }
            uint32_t before = sum;                         // inclusive scan over the block
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(kFull, before, o);
                if (lane >= o) before += x;
            }
            if (lane == 31) warp_sum[w] = before;
            __syncthreads();
            const uint32_t others = lane < w ? warp_sum[lane] : 0u;
            before += __reduce_add_sync(kFull, others) - sum;
            if (before < need && need <= before + sum) {   // one thread
#pragma unroll
                for (int q = 0; q < kPairs; ++q) {
                    const uint32_t two[2] = {c[q].y, c[q].x};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (before < need && need <= before + two[j]) {
                            found[0] = (uint32_t)(top - 2 * q + 1 - j);
                            found[1] = before;
                            found[2] = two[j];
                        }
                        before += two[j];
                    }
                }
            }
            __syncthreads();
            base += found[0] << shift;
            need -= found[1];
            if (need == found[2]) {                        // every key of the digit
                threshold = base - 1u;
                need = 0;
                break;
            }
            if (shift == 0) {
                threshold = base;
                break;
            }
            span = min((1u << shift) - 1u, mx - base);     // no further than the keys go
        }
    }
    // ---- the places. Taken: the ends, keys above the threshold, the first `need` equal ones
    // (counts of both in one word, equal ones in the upper half)
    auto counts = [&](int j, int e) { return (key[j][e] > threshold ? 1u : 0u) + (key[j][e] == threshold ? 0x10000u : 0u); };
    uint32_t before[V];
    auto count_round = [&] {                               // -> before[], run[]: taken before a piece
#pragma unroll
        for (int j = 0; j < V; ++j) {
            uint32_t mine = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) mine += counts(j, e);
            uint32_t x = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(kFull, x, o);
                if (lane >= o) x += y;
            }
            before[j] = x - mine;
            if (lane == 31) run[j * kWarps + w] = x;
        }
        __syncthreads();
        if (w == 0) {
            constexpr int kEach = (V * kWarps + 31) / 32;
            uint32_t r[kEach], sum = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int at = lane * kEach + i;
                r[i] = at < V * kWarps ? run[at] : 0u;
                sum += r[i];
            }
            uint32_t x = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(kFull, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) round_taken = x;
            x -= sum;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int at = lane * kEach + i;
                if (at < V * kWarps) run[at] = x;
                x += r[i];
            }
        }
        __syncthreads();
    };
    uint32_t gt = 0, eq = 0;                               // taken before this CTA's current round
    if (!alone) {
        uint32_t all_gt = 0, all_eq = 0;
        each_round([&](int) {
            count_round();
            all_gt += round_taken & 0xffffu;
            all_eq += round_taken >> 16;
            if (kLong) __syncthreads();
        });
        if (tid == 0) {
            cta_taken[0] = all_gt;
            cta_taken[1] = all_eq;
        }
        cluster_sync();
        const uint2 x = lane < rank ? cluster_ld2(cluster_addr(cta_taken, lane)) : make_uint2(0u, 0u);
        gt = __reduce_add_sync(kFull, x.x);
        eq = __reduce_add_sync(kFull, x.y);
        cluster_sync();                                    // nobody leaves while others read
    }
    each_round([&](int r) {
        if (alone || (kLong && rounds > 1)) count_round();
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t at = before[j] + run[j * kWarps + w];
            uint32_t g = gt + (at & 0xffffu), q = eq + (at >> 16);
            const int i = begin + r * kRound + 4 * (j * NT + tid);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool above = key[j][e] > threshold, equal = key[j][e] == threshold;
                if (above || (equal && q < need)) out[g + min(q, need)] = i + e;
                g += above;
                q += equal;
            }
        }
        if (kLong) {
            gt += round_taken & 0xffffu;
            eq += round_taken >> 16;
            __syncthreads();                               // run[] is read
        }
    });
}

using SelectKernel = void (*)(SelectParams);
constexpr int kShortRow = 8192;        // what a CTA of 256 threads holds

int launch_select(SelectKernel kern, const SelectParams& p, long long clusters, int size, int threads, void* stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * size));
    cfg.blockDim = dim3(threads);
    cfg.stream = static_cast<cudaStream_t>(stream);
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
    return e == cudaSuccess ? PKV_OK : cuda_fail("select_tokens: kernel launch", e);
}

// -------------------------------------------------------------------- keep_tokens
constexpr int kKeepThreads = 256, kKeepTokens = 64;        // of a CTA
constexpr int kWeightChunk = 8;                            // weights of a thread at a time

struct KeepParams {
    const int32_t* kept;
    float* weights;
    const int32_t* rows;
    char* k_pool;
    char* v_pool;
    const int32_t* tables;
    const int32_t* kept_tables;
    const int32_t* seq_lens;
    int* err;
    int k, max_blocks, max_kept_blocks, num_blocks, num_rows, max_tokens, num_kv_heads, d, bs;
    int chunks;                        // of kKeepTokens tokens
    int weight_ctas;                   // the first ones of the launch
};

// Entry i of a list: the token, -1: padding, -2: an entry that is skipped
__device__ __forceinline__ int kept_token(const int32_t* list, int i, int n) {
    const int t = list[i];
    if (t == -1) return -1;
    const int before = i > 0 ? list[i - 1] : -1;
    return t < 0 || t >= n || t <= before || t < i || (i > 0 && before < 0) ? -2 : t;
}

__device__ void keep_weights(const KeepParams& p, int item) {
    const int b = item / p.num_kv_heads, h = item - b * p.num_kv_heads;
    const int row = weight_row(p.rows, b, p.num_rows, true, p.err);
    if (row < 0) return;
    const int n = min(p.seq_lens[b], p.max_blocks * p.bs);     // the row holds as many
    float* const at = p.weights + ((size_t)row * p.num_kv_heads + h) * p.max_tokens;
    const int32_t* const list = p.kept + (size_t)item * p.k;
    const int most = min(p.k, n);
    for (int i0 = 0; i0 < most; i0 += kWeightChunk * kKeepThreads) {
        float v[kWeightChunk];
        int t[kWeightChunk];
#pragma unroll
        for (int j = 0; j < kWeightChunk; ++j) {
            const int i = i0 + j * kKeepThreads + (int)threadIdx.x;
            t[j] = i < most ? kept_token(list, i, n) : -1;
        }
#pragma unroll
        for (int j = 0; j < kWeightChunk; ++j)
            if (t[j] >= 0) v[j] = at[t[j]];
        __syncthreads();                                   // the chunk is read
#pragma unroll
        for (int j = 0; j < kWeightChunk; ++j)
            if (t[j] >= 0) at[i0 + j * kKeepThreads + threadIdx.x] = v[j];
        __syncthreads();
    }
}

// What a piece of 16 bytes gives to a word: bytes of its lower and of its upper half
struct __align__(16) Piece {
    uint32_t lo, lo_mask, hi, hi_mask;
};

template <int ES>                                          // bytes of an element
__global__ void __launch_bounds__(kKeepThreads) keep_tokens_kernel(const KeepParams p) {
    pdl_enter();
    constexpr int X = 16 / ES;
    // V's elements are read one by one, not the pieces that they lie in: a row of 4 tokens saves few
    // reads (16 sequences of 16384, D 64: 198 us and 205 us; bf16 135 and 123, E4M3 137 and 93)
    constexpr bool kElements = ES == 4;
    if ((int)blockIdx.x < p.weight_ctas) {
        keep_weights(p, blockIdx.x);
        return;
    }
    // of each token: its first 16-byte piece of K; -1: skipped
    __shared__ long long src_k[kKeepTokens], dst_k[kKeepTokens];
    // of each row of X tokens of V: the groups of X tokens (their pieces of 16 bytes of the first dim)
    // that it comes from, and what each of them gives to each word of a piece; kElements: its tokens'
    // elements of the first dim
    constexpr int kRows = kKeepTokens / X;
    __shared__ long long dst_v[kRows], src_v[kRows][X];
    __shared__ int num_src[kRows];
    __shared__ uint32_t has[kRows];                        // bit e: token e is there
    __shared__ Piece give[kElements ? 1 : kRows][X][4];
    const long long unit = (long long)blockIdx.x - p.weight_ctas;
    const int item = (int)(unit / p.chunks), b = item / p.num_kv_heads, h = item - b * p.num_kv_heads;
    const int i0 = (int)(unit - (long long)item * p.chunks) * kKeepTokens;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    if constexpr (!kElements) {
        static_assert(kRows * X * 4 == kKeepThreads, "an entry a thread");
        (&give[0][0][0])[tid] = Piece{0, 0, 0, 0};
        __syncthreads();
    }
    if (tid < kKeepTokens) {                               // whole warps
        const long long tile = (long long)p.d * p.bs * ES;
        long long sk = -1, dk = -1, sv = -1;
        const int i = i0 + tid, row = tid / X, e = tid % X;
        int at = 0;                                        // of the token in its group, in bytes
        if (i < p.k) {
            int n = p.seq_lens[b];
            if (n < 0 || n > p.max_blocks * p.bs) {
                flag_error(p.err, kErrOutOfRange);
                n = n < 0 ? 0 : p.max_blocks * p.bs;
            }
            const int t = kept_token(p.kept + (size_t)item * p.k, i, n);
            if (t >= 0) {
                const int sb = t / p.bs, s = t - sb * p.bs, ob = i / p.bs, o = i - ob * p.bs;
                const int from = p.tables[(size_t)b * p.max_blocks + sb];
                const int to = p.kept_tables[(size_t)b * p.max_kept_blocks + ob];
                if (from >= 0 && from < p.num_blocks && to >= 0 && to < p.num_blocks) {
                    const long long st = ((long long)from * p.num_kv_heads + h) * tile;
                    const long long ot = ((long long)to * p.num_kv_heads + h) * tile;
                    sk = st + (long long)(s >> 3) * p.d * 8 * ES + (s & 7) * 16;
                    dk = ot + (long long)(o >> 3) * p.d * 8 * ES + (o & 7) * 16;
                    sv = st + (long long)(s / X) * p.d * 16;
                    at = s % X * ES;
                    dst_v[row] = ot + (long long)(o / X) * p.d * 16;   // the row's tokens agree
                } else {
                    flag_error(p.err, kErrOutOfRange);
                }
            } else if (t == -2) {
                flag_error(p.err, kErrOutOfRange);
            }
        }
        src_k[tid] = sk;
        dst_k[tid] = dk;
        const int shift = lane & ~(X - 1);
        constexpr uint32_t kAll = (1u << X) - 1u;
        const uint32_t there = __ballot_sync(kFull, sv >= 0) >> shift;
        if (e == 0) has[row] = there & kAll;
        if constexpr (kElements) {
            src_v[row][e] = sv + at;
        } else {
            const long long before = __shfl_up_sync(kFull, sv, 1);
            const bool next = sv >= 0 && (e == 0 || before != sv); // the first of its group
            const uint32_t firsts = __ballot_sync(kFull, next) >> shift;
            const int r = __popc(firsts & ((2u << e) - 1u)) - 1;
            if (next) src_v[row][r] = sv;
            if (e == 0) num_src[row] = __popc(firsts & kAll);
            if (sv >= 0) {
                Piece& g = give[row][r][e * ES / 4];
#pragma unroll
                for (int k = 0; k < ES; ++k) {
                    const int to = (e * ES + k) & 3;
                    atomicOr(at < 8 ? &g.lo : &g.hi, (uint32_t)((at & 7) + k) << (4 * to));
                    atomicOr(at < 8 ? &g.lo_mask : &g.hi_mask, 0xffu << (8 * to));
                }
            }
        }
    }
    __syncthreads();
    // ---- K: a warp's 8 tokens, 4 pieces of each at a time
    const int planes = p.d / X;
    {
        const int j = 8 * w + (lane & 7);
        if (src_k[j] >= 0) {
            const char* from = p.k_pool + src_k[j] + (lane >> 3) * 128;
            char* to = p.k_pool + dst_k[j] + (lane >> 3) * 128;
            for (int c = lane >> 3; c < planes; c += 16, from += 16 * 128, to += 16 * 128) {
                uint4 v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (c + 4 * u < planes) v[u] = *reinterpret_cast<const uint4*>(from + 4 * u * 128);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (c + 4 * u < planes) *reinterpret_cast<uint4*>(to + 4 * u * 128) = v[u];
            }
        }
    }
    // ---- V: rows of X tokens of one dim (chunks begin at multiples of X, blocks hold whole ones). A
    // piece of 16 bytes of each group that the row comes from is read once, and its bytes put in place:
    // two or three reads for 16 tokens when half of them stay, where elements take 16.
    // A warp takes rows of 32 dims; the rows of X tokens are shared by kSame warps, or it takes several
    using E = typename std::conditional<ES == 4, uint32_t, typename std::conditional<ES == 2, uint16_t, uint8_t>::type>::type;
    constexpr int kWarps = kKeepThreads / 32, kSame = kRows < kWarps ? kWarps / kRows : 1;
    constexpr int kU = 2, kJ = 2;                          // dims and groups in flight
    for (int row = w / kSame; row < kRows; row += kWarps / kSame) {
        const uint32_t mine = has[row];
        if (mine == 0) continue;
        const int groups = kElements ? 0 : num_src[row];
        for (int d0 = (w % kSame) * 32 * kU + lane; d0 < p.d; d0 += kSame * 32 * kU) {
            uint32_t word[kU][4] = {};
            if constexpr (kElements) {
#pragma unroll
                for (int u = 0; u < kU; ++u)
#pragma unroll
                    for (int e = 0; e < X; ++e)
                        if ((mine >> e & 1u) && d0 + 32 * u < p.d)
                            word[u][e] = *reinterpret_cast<const uint32_t*>(p.v_pool + src_v[row][e] + (d0 + 32 * u) * 16);
            }
            for (int j0 = 0; !kElements && j0 < groups; j0 += kJ) {
                uint4 v[kJ][kU];
#pragma unroll
                for (int j = 0; j < kJ; ++j)
#pragma unroll
                    for (int u = 0; u < kU; ++u)
                        if (j0 + j < groups && d0 + 32 * u < p.d)
                            v[j][u] = *reinterpret_cast<const uint4*>(p.v_pool + src_v[row][j0 + j] + (d0 + 32 * u) * 16);
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    if (j0 + j >= groups) break;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const Piece g = give[row][j0 + j][q];
#pragma unroll
                        for (int u = 0; u < kU; ++u) {
                            word[u][q] |= __byte_perm(v[j][u].x, v[j][u].y, g.lo) & g.lo_mask;
                            word[u][q] |= __byte_perm(v[j][u].z, v[j][u].w, g.hi) & g.hi_mask;
                        }
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int d = d0 + 32 * u;
                if (d >= p.d) break;
                char* const to = p.v_pool + dst_v[row] + d * 16;
                if (mine == (1u << X) - 1u) {
                    *reinterpret_cast<uint4*>(to) = make_uint4(word[u][0], word[u][1], word[u][2], word[u][3]);
                } else {                                   // the others keep what they have
#pragma unroll
                    for (int e = 0; e < X; ++e)
                        if (mine >> e & 1u) reinterpret_cast<E*>(to)[e] = (E)(word[u][e * ES / 4] >> (8 * (e * ES & 3)));
                }
            }
        }
    }
}

}  // namespace
}  // namespace pkv

extern "C" {

int select_tokens(int32_t* kept, const float* token_weights, const int32_t* weight_rows, const int32_t* seq_lens,
                  int num_seqs, int num_kv_heads, int num_rows, int max_tokens, int num_kept, int first_tokens,
                  int last_tokens, void* stream) {
    using namespace pkv;
    if (num_seqs < 0 || num_seqs > 65535 || num_kv_heads <= 0 || num_kv_heads > 65535 || num_rows <= 0 ||
        max_tokens <= 0 || num_kept <= 0 || first_tokens < 0 || last_tokens < 0 || first_tokens > num_kept ||
        last_tokens > num_kept - first_tokens || max_tokens % 4 != 0)
        return PKV_ERR_INVALID_ARG;
    if (!weight_rows && num_rows < num_seqs) return PKV_ERR_INVALID_ARG;
    const long long items = (long long)num_seqs * num_kv_heads;
    if (items > 0x7fffffffLL / kMaxCluster || max_tokens > (1 << 30)) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!kept || !token_weights || !seq_lens || !aligned16(token_weights)) return PKV_ERR_INVALID_ARG;
    if (checking()) return PKV_OK;
    SelectParams p{};
    p.kept = kept;
    p.weights = token_weights;
    p.rows = weight_rows;
    p.seq_lens = seq_lens;
    p.err = error_word();
    if (!p.err) return PKV_ERR_CUDA;
    p.num_kv_heads = num_kv_heads;
    p.num_rows = num_rows;
    p.max_tokens = max_tokens;
    p.k = num_kept;
    p.first = first_tokens;
    p.last = last_tokens;
    // the smallest CTA that holds a row in its registers, then clusters of up to 8 of the largest: a
    // trip through the cluster costs about 1 us, and there are six (128 rows of 30000 tokens take
    // 13.7 us as CTAs of 32768 and 31 us as 2 of 16384; 8 of 65536, 18 us and 20 us)
    SelectKernel kern;
    int size = 1, threads = 256;
    if (max_tokens <= 1024) kern = select_tokens_kernel<256, 1, false>;
    else if (max_tokens <= 2048) kern = select_tokens_kernel<256, 2, false>;
    else if (max_tokens <= 4096) kern = select_tokens_kernel<256, 4, false>;
    else if (max_tokens <= kShortRow) kern = select_tokens_kernel<256, 8, false>;
    else if (max_tokens <= 16384) kern = select_tokens_kernel<512, 8, false>, threads = 512;
    else {
        threads = 1024;
        while (size < kMaxCluster && 32768LL * size < max_tokens) size *= 2;
        kern = 32768LL * size >= max_tokens ? select_tokens_kernel<1024, 8, false> : select_tokens_kernel<1024, 8, true>;
    }
    // More rows than one wave of such CTAs holds, which may all be short: short ones have a launch of
    // their own, in CTAs of which an SM holds four (512 rows of 4096 tokens in rows of 131072: 24 us and
    // 92 us; all of 30000: 97 us and 95 us. Clusters that walk over rows: 15 us, but rows of 100000 took
    // 449 us where one row a cluster takes 245)
    p.least = -1;
    p.most = max_tokens;
    const long long wave = (long long)num_sms() * (1024 / threads) / size;
    if (max_tokens > kShortRow && items > wave) {
        p.most = kShortRow;
        const int st = launch_select(select_tokens_kernel<256, 8, false>, p, items, 1, 256, stream);
        if (st != PKV_OK) return st;
        p.least = kShortRow;
        p.most = max_tokens;
    }
    return launch_select(kern, p, items, size, threads, stream);
}

int keep_tokens(const int32_t* kept, float* token_weights, const int32_t* weight_rows, void* k_pool, void* v_pool,
                const int32_t* block_tables, const int32_t* kept_tables, const int32_t* seq_lens, int num_seqs,
                int num_kept, int max_blocks_per_seq, int max_kept_blocks, int num_blocks, int num_rows,
                int max_tokens, int num_kv_heads, int head_dim, int block_size, int kv_dtype, void* stream) {
    using namespace pkv;
    if (num_seqs < 0 || num_seqs > 65535 || num_kept <= 0 || max_blocks_per_seq <= 0 || max_kept_blocks <= 0 ||
        num_blocks <= 0 || num_kv_heads <= 0 || num_kv_heads > 65535 || head_dim <= 0 || block_size <= 0 ||
        max_blocks_per_seq > 0x7fffffff / block_size || max_kept_blocks > 0x7fffffff / block_size ||
        num_kept > max_kept_blocks * block_size)
        return PKV_ERR_INVALID_ARG;
    if (token_weights && (num_rows <= 0 || max_tokens < max_blocks_per_seq * block_size || max_tokens % 4 != 0 ||
                          (!weight_rows && num_rows < num_seqs) || !aligned16(token_weights)))
        return PKV_ERR_INVALID_ARG;
    if (head_dim % 16 != 0 || head_dim > 512 || block_size % 16 != 0 ||
        (kv_dtype != PKV_F32 && kv_dtype != PKV_BF16 && kv_dtype != PKV_E4M3))
        return PKV_ERR_UNSUPPORTED;
    KeepParams p{};
    const long long items = (long long)num_seqs * num_kv_heads;
    p.chunks = (int)((num_kept + (long long)kKeepTokens - 1) / kKeepTokens);
    const long long ctas = items * p.chunks + (token_weights ? items : 0);
    if (ctas > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!kept || !k_pool || !v_pool || !block_tables || !kept_tables || !seq_lens || !aligned16(k_pool) ||
        !aligned16(v_pool))
        return PKV_ERR_INVALID_ARG;
    if (checking()) return PKV_OK;
    p.kept = kept;
    p.weights = token_weights;
    p.rows = weight_rows;
    p.k_pool = static_cast<char*>(k_pool);
    p.v_pool = static_cast<char*>(v_pool);
    p.tables = block_tables;
    p.kept_tables = kept_tables;
    p.seq_lens = seq_lens;
    p.err = error_word();
    if (!p.err) return PKV_ERR_CUDA;
    p.k = num_kept;
    p.max_blocks = max_blocks_per_seq;
    p.max_kept_blocks = max_kept_blocks;
    p.num_blocks = num_blocks;
    p.num_rows = num_rows;
    p.max_tokens = max_tokens;
    p.num_kv_heads = num_kv_heads;
    p.d = head_dim;
    p.bs = block_size;
    p.weight_ctas = token_weights ? (int)items : 0;
    auto kern = kv_dtype == PKV_F32 ? keep_tokens_kernel<4> : kv_dtype == PKV_BF16 ? keep_tokens_kernel<2> : keep_tokens_kernel<1>;
    note_launch();
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)ctas), dim3(kKeepThreads), 0, static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? PKV_OK : cuda_fail("keep_tokens: kernel launch", e);
}

}  // extern "C"
