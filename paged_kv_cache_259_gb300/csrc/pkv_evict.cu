// Cache eviction: select_tokens (the tokens of the highest accumulated weight, exactly) and
// keep_tokens (their move to the front of fresh blocks).
//
// select_tokens. A row is one (sequence, kv head): up to hundreds of thousands of float32
// weights, of which the R = num_kept - first - last largest between the always-kept ends are
// wanted, ties to the lower token. The weights become 32-bit keys that order as unsigned
// numbers, are read once into the shared memory of a cluster of CTAs (a contiguous slice
// each), and the R-th largest is found digit by digit (11, 11 and 10 bits): every CTA
// counts its keys' digits, the counts are summed over the cluster through distributed shared
// memory, and the digit in which the R-th falls narrows the keys of the next pass. The taken
// keys are those above the threshold and the first few equal to it; every warp counts both in
// its run of the slice, and prefix sums over warps and CTAs give each its places in the list,
// which so comes out ascending. Bound: the reads (4 bytes a token) for many rows, the chain of
// passes and cluster barriers for few.
//
// keep_tokens. K: 16-byte pieces, one per (token, X dims), to their new place: eight
// neighbouring threads write a whole 128-byte core matrix. V is stored transposed: a thread
// gathers the X tokens of one dim and writes them as one 16-byte row. Source and target blocks
// are disjoint, so nothing waits. The weights move within their row: kept[i] >= i, so one CTA
// a row that reads a chunk of the list's weights, waits for all its threads, and writes them,
// overwrites nothing that a later chunk reads. Bound: HBM bytes.
#include <cuda_runtime.h>

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
constexpr int kSelWarps = 16, kSelThreads = kSelWarps * 32;
constexpr int kBins = 2048, kPasses = 3;
constexpr int kMaxCached = 45056;      // keys of a CTA's slice in shared memory (176 KB)
constexpr int kMaxCluster = 8;         // the portable size

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
// a word of the cluster's CTA `rank`, at this CTA's address of it
__device__ __forceinline__ uint32_t cluster_ld(const void* p, uint32_t rank) {
    uint32_t a, v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// A weight as an unsigned number of the same order; -0 as 0; what is not finite on top.
__device__ __forceinline__ uint32_t key_of(float w) {
    uint32_t x = __float_as_uint(w + 0.f);
    if ((x & 0x7f800000u) == 0x7f800000u) return 0xffffffffu;
    return x & 0x80000000u ? ~x : x | 0x80000000u;
}

struct SelectParams {
    int32_t* kept;
    const float* weights;
    const int32_t* rows;
    const int32_t* seq_lens;
    int* err;
    int num_kv_heads, num_rows, max_tokens, k, first, last;
    int cached;                        // keys that a CTA's shared memory holds
};

__global__ void __launch_bounds__(kSelThreads) select_tokens_kernel(const SelectParams p) {
    pdl_enter();
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ uint32_t hist[kPasses][kBins];
    __shared__ uint32_t warp_sum[kSelWarps];
    __shared__ uint32_t found[2];                          // digit, keys above it
    __shared__ uint32_t taken[kSelWarps][2], cta_taken[2]; // above the threshold, equal to it
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank(), csize = (int)cluster_size();
    const int item = (int)(blockIdx.x / csize), b = item / p.num_kv_heads, h = item - b * p.num_kv_heads;
    int n = p.seq_lens[b];
    if (n < 0 || n > p.max_tokens) {
        if (tid == 0) flag_error(p.err, kErrOutOfRange);
        n = n < 0 ? 0 : p.max_tokens;
    }
    const int row = weight_row(p.rows, b, p.num_rows, false, p.err);
    if (row < 0) n = 0;
    int32_t* const out = p.kept + (size_t)item * p.k;
    if (n <= p.k) {                                        // the whole cluster
        for (int i = rank * kSelThreads + tid; i < p.k; i += csize * kSelThreads) out[i] = i < n ? i : -1;
        return;
    }
    const float* const src = p.weights + ((size_t)row * p.num_kv_heads + h) * p.max_tokens;
    // this CTA's slice, a multiple of 4 tokens
    const int slice = ((n + csize - 1) / csize + 3) & ~3;
    const int begin = min(n, rank * slice), count = min(n, begin + slice) - begin;
    const int cached = min(count, p.cached);
    for (int i = tid; i < kPasses * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
    for (int i = 4 * tid; i < cached; i += 4 * kSelThreads) {   // the last piece may pass n, not the row
        const float4 v = *reinterpret_cast<const float4*>(src + begin + i);
        *reinterpret_cast<uint4*>(keys + i) = make_uint4(key_of(v.x), key_of(v.y), key_of(v.z), key_of(v.w));
    }
    auto key = [&](int i) { return i < cached ? keys[i] : key_of(src[begin + i]); };
    // ---- the R-th largest of the tokens between the ends
    const int lo = max(0, p.first - begin), hi = min(count, n - p.last - begin);
    uint32_t need = (uint32_t)(p.k - p.first - p.last);    // still to be found at or below `prefix`
    uint32_t threshold = 0xffffffffu;                      // taken: keys above it, `need` equal ones
    __syncthreads();
    if (need > 0) {
        uint32_t prefix = 0;
        for (int pass = 0; pass < kPasses; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
            const uint32_t mask = (1u << bits) - 1u;
            for (int i = lo + tid; i < hi; i += kSelThreads) {
                const uint32_t x = key(i);
                if (pass == 0 || (x >> (shift + bits)) == prefix) atomicAdd(&hist[pass][(x >> shift) & mask], 1u);
            }
            if (csize > 1) cluster_sync();
            else __syncthreads();
            // bins 4 tid .. 4 tid + 3 counted from the top
            uint32_t c[4], sum = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int bin = kBins - 1 - (4 * tid + j);
                c[j] = 0;
                for (int r = 0; r < csize; ++r) c[j] += csize > 1 ? cluster_ld(&hist[pass][bin], r) : hist[pass][bin];
                sum += c[j];
            }
            uint32_t before = sum;                         // inclusive scan over the block
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(kFull, before, o);
                if (lane >= o) before += x;
            }
            if (lane == 31) warp_sum[w] = before;
            __syncthreads();
            for (int i = 0; i < w; ++i) before += warp_sum[i];
            before -= sum;
            if (before < need && need <= before + sum) {   // one thread
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (before < need && need <= before + c[j]) {
                        found[0] = (uint32_t)(kBins - 1 - (4 * tid + j));
                        found[1] = before;
                    }
                    before += c[j];
                }
            }
            __syncthreads();
            prefix = pass == 0 ? found[0] : (prefix << bits) | found[0];
            need -= found[1];
        }
        threshold = prefix;
    }
    // ---- the places: this warp's run of the slice
    const int run = ((count + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int from = min(count, w * run), to = min(count, from + run);
    const bool none = p.k == p.first + p.last;
    auto above = [&](int i, uint32_t x) { return i < lo || i >= hi || (!none && x > threshold); };
    uint32_t gt = 0, eq = 0;
    for (int i = from + lane; i - lane < to; i += 32) {
        const bool in = i < to;
        const uint32_t x = in ? key(i) : 0u;
        const bool a = in && above(i, x);
        gt += __popc(__ballot_sync(kFull, a));
        eq += __popc(__ballot_sync(kFull, in && !a && !none && x == threshold));
    }
    if (lane == 0) {
        taken[w][0] = gt;
        taken[w][1] = eq;
    }
    __syncthreads();
    if (tid < 2) {
        uint32_t s = 0;
        for (int i = 0; i < kSelWarps; ++i) {
            const uint32_t x = taken[i][tid];
            taken[i][tid] = s;
            s += x;
        }
        cta_taken[tid] = s;
    }
    if (csize > 1) cluster_sync();
    else __syncthreads();
    uint32_t base_gt = taken[w][0], base_eq = taken[w][1];
    for (int r = 0; r < rank; ++r) {
        base_gt += cluster_ld(&cta_taken[0], r);
        base_eq += cluster_ld(&cta_taken[1], r);
    }
    if (csize > 1) cluster_sync();                         // nobody leaves while others read
    const uint32_t below = (1u << lane) - 1u;
    for (int i = from + lane; i - lane < to; i += 32) {
        const bool in = i < to;
        const uint32_t x = in ? key(i) : 0u;
        const bool a = in && above(i, x), e = in && !a && !none && x == threshold;
        const uint32_t ga = __ballot_sync(kFull, a), ge = __ballot_sync(kFull, e);
        const uint32_t ea = base_eq + __popc(ge & below);
        if (a || (e && ea < need)) out[base_gt + __popc(ga & below) + min(ea, need)] = begin + i;
        base_gt += __popc(ga);
        base_eq += __popc(ge);
    }
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
    int items;                         // (sequence, kv head)
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

template <int ES>                                          // bytes of an element
__global__ void __launch_bounds__(kKeepThreads) keep_tokens_kernel(const KeepParams p) {
    pdl_enter();
    constexpr int X = 16 / ES;
    if ((int)blockIdx.x < p.weight_ctas) {
        keep_weights(p, blockIdx.x);
        return;
    }
    __shared__ long long src_tile[kKeepTokens], dst_tile[kKeepTokens];   // bytes; -1: skipped
    __shared__ int src_slot[kKeepTokens], dst_slot[kKeepTokens];
    const long long unit = (long long)blockIdx.x - p.weight_ctas;
    const int item = (int)(unit / p.chunks), b = item / p.num_kv_heads, h = item - b * p.num_kv_heads;
    const int i0 = (int)(unit - (long long)item * p.chunks) * kKeepTokens;
    const int tid = threadIdx.x;
    const long long tile = (long long)p.d * p.bs * ES;
    if (tid < kKeepTokens) {
        long long s = -1, o = -1;
        int ss = 0, os = 0;
        const int i = i0 + tid;
        if (i < p.k) {
            int n = p.seq_lens[b];
            if (n < 0 || n > p.max_blocks * p.bs) {
                flag_error(p.err, kErrOutOfRange);
                n = n < 0 ? 0 : p.max_blocks * p.bs;
            }
            const int t = kept_token(p.kept + (size_t)item * p.k, i, n);
            if (t >= 0) {
                const int from = p.tables[(size_t)b * p.max_blocks + t / p.bs];
                const int to = p.kept_tables[(size_t)b * p.max_kept_blocks + i / p.bs];
                if (from >= 0 && from < p.num_blocks && to >= 0 && to < p.num_blocks) {
                    s = ((long long)from * p.num_kv_heads + h) * tile;
                    o = ((long long)to * p.num_kv_heads + h) * tile;
                    ss = t % p.bs;
                    os = i % p.bs;
                } else {
                    flag_error(p.err, kErrOutOfRange);
                }
            } else if (t == -2) {
                flag_error(p.err, kErrOutOfRange);
            }
        }
        src_tile[tid] = s;
        dst_tile[tid] = o;
        src_slot[tid] = ss;
        dst_slot[tid] = os;
    }
    __syncthreads();
    // ---- K: pieces of 16 bytes
    const int planes = p.d / X;
    for (int x = tid; x < kKeepTokens * planes; x += kKeepThreads) {
        const int c = (x >> 3) % planes, j = (x & 7) + 8 * (x / (8 * planes));
        if (src_tile[j] < 0) continue;
        const int s = src_slot[j], o = dst_slot[j];
        const uint4 v = *reinterpret_cast<const uint4*>(p.k_pool + src_tile[j] + ((s >> 3) * planes + c) * 128 + (s & 7) * 16);
        *reinterpret_cast<uint4*>(p.k_pool + dst_tile[j] + ((o >> 3) * planes + c) * 128 + (o & 7) * 16) = v;
    }
    // ---- V: rows of X tokens of one dim (chunks begin at multiples of X, blocks hold whole ones)
    for (int x = tid; x < kKeepTokens / X * p.d; x += kKeepThreads) {
        const int d = x % p.d, j0 = x / p.d * X;
        uint32_t word[4] = {0, 0, 0, 0};
        bool all = true;
        long long last = -1;
        uint4 r = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < X; ++e) {
            const int j = j0 + e;
            if (src_tile[j] < 0) {                         // the same for all dims
                all = false;
                continue;
            }
            const int s = src_slot[j];
            const long long at = src_tile[j] + ((long long)(s / X) * (p.d / 8) * 8 + d) * 16;
            if (at != last) r = *reinterpret_cast<const uint4*>(p.v_pool + at);
            last = at;
            const int byte = s % X * ES;
            const uint32_t two = byte & 8 ? (byte & 4 ? r.w : r.z) : (byte & 4 ? r.y : r.x);
            uint32_t v = two >> (8 * (byte & 3));
            if constexpr (ES < 4) v &= (1u << (8 * (ES & 3))) - 1u;
            word[e * ES / 4] |= v << (8 * (e * ES & 3));
        }
        // the first token of the row that goes somewhere: they share its target row
#pragma unroll
        for (int e = 0; e < X; ++e) {
            const int j = j0 + e;
            if (dst_tile[j] < 0) continue;
            char* const to = p.v_pool + dst_tile[j] + ((long long)(dst_slot[j] / X) * (p.d / 8) * 8 + d) * 16;
            if (all) {
                *reinterpret_cast<uint4*>(to) = make_uint4(word[0], word[1], word[2], word[3]);
                break;
            }
            const uint32_t v = word[e * ES / 4] >> (8 * (e * ES & 3));
            if constexpr (ES == 4) reinterpret_cast<uint32_t*>(to)[e] = v;
            else if constexpr (ES == 2) reinterpret_cast<uint16_t*>(to)[e] = (uint16_t)v;
            else reinterpret_cast<uint8_t*>(to)[e] = (uint8_t)v;
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
    int size = 1;
    while (size < kMaxCluster && max_tokens / size > 4096 && items * size < 2LL * num_sms()) size *= 2;
    while (size < kMaxCluster && max_tokens / size > kMaxCached) size *= 2;
    const int slice = ((max_tokens + size - 1) / size + 3) & ~3;
    p.cached = slice < kMaxCached ? slice : kMaxCached;
    const void* kern = reinterpret_cast<const void*>(&select_tokens_kernel);
    try {
        int occ = 0;
        const int st = kernel_setup(kern, kMaxCached * 4, kSelThreads, &occ);
        if (st != PKV_OK) return st;
    } catch (...) {
        return cuda_fail("select_tokens: host memory", cudaErrorMemoryAllocation);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * size));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = (size_t)p.cached * 4;
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, select_tokens_kernel, p);
    return e == cudaSuccess ? PKV_OK : cuda_fail("select_tokens: kernel launch", e);
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
    p.items = (int)items;
    p.weight_ctas = token_weights ? (int)items : 0;
    auto kern = kv_dtype == PKV_F32 ? keep_tokens_kernel<4> : kv_dtype == PKV_BF16 ? keep_tokens_kernel<2> : keep_tokens_kernel<1>;
    note_launch();
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)ctas), dim3(kKeepThreads), 0, static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? PKV_OK : cuda_fail("keep_tokens: kernel launch", e);
}

}  // extern "C"
