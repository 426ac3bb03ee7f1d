// Decode attention over selected blocks: paged_attention_decode_sparse.
//
// The mathematics is the decode kernel's (online softmax over a sequence's
// cached tokens, tile by tile) over the tokens of the blocks that a list names
// for each (sequence, kv head), and the tile math is that kernel's (SimtMath,
// MmaMath). What differs is the walk and the merge:
//   - an entry of the list is a logical block, so a tile's address takes two
//     dependent reads (list, block table); a warp makes them for 32 entries at
//     once, before its first copy;
//   - a list is short (tens to hundreds of blocks), so a row is split over the
//     CTAs of one thread-block cluster and its partial results are merged
//     through distributed shared memory: one launch, no workspace. The split is
//     taken from the row's own number of entries, so short rows stay balanced.
// Bound: HBM bytes of the selected tiles when there are many rows; a chain of
// loads (length, list, table, tile, partner's partials) when there are few.
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
    float qscale, v_scale;
};

struct Args {
    Params p;
    int num_seqs, head_dim, block_size;
    float scale, k_scale, v_scale;
    cudaStream_t stream;
};

constexpr int kNumWarps = 4;
constexpr int kMaxParts = 8;           // the portable cluster size

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
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

// CTA (part, kv head, sequence); the parts of a row are one cluster. PAIR = 2:
// a pipeline stage holds two list entries of BS / 2 tokens side by side (see the
// decode kernel); BS is then the stage's token count.
template <class Math, typename QT, int D, int BS, int G, int NW, int PAIR>
__global__ void __launch_bounds__(NW * 32, 3) sparse_decode_kernel(const Params p) {
    using P = decode::Pipe<Math, D, BS, G, NW>;
    constexpr int TILE = P::kTile, ST = P::kStages;
    constexpr int PBS = BS / PAIR, PTILE = TILE / PAIR;
    static_assert(PAIR == 1 || PAIR == 2, "entries per stage");
    pdl_enter();                                           // launched with programmatic serialisation
    extern __shared__ __align__(128) unsigned char smem[];
    unsigned char* ring = smem;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + P::kBarOff);
    int32_t* stage_tok = reinterpret_cast<int32_t*>(smem + P::kIdOff);   // tokens of the stage
    float* qs = reinterpret_cast<float*>(smem + P::kQOff);
    float* wsm = reinterpret_cast<float*>(smem + P::kWarpOff);

    const int part = blockIdx.x, parts = gridDim.x, hk = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    int L = p.seq_lens[b];
    if (L < 0 || L > p.max_blocks * PBS) {                  // length the table cannot hold
        if (part == 0 && hk == 0 && tid == 0) flag_error(p.err, kErrOutOfRange);
        L = L < 0 ? 0 : p.max_blocks * PBS;
    }
    const int nblk = (L + PBS - 1) / PBS;
    // distinct entries below nblk: no more than nblk of them
    const int total = min(p.k, nblk);
    const int stages = (total + PAIR - 1) / PAIR;
    const int per = (stages + parts - 1) / parts;
    const int first = part * per;                           // first stage of this CTA
    const int count = max(0, min(per, stages - first));
    const int32_t* list = p.selected + ((size_t)b * p.num_kv_heads + hk) * p.k;

    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < ST; ++s) mbar_init(smem_addr(&bars[w * ST + s]), 1);
        fence_mbar_init();
    }
    __syncwarp();
    const int nk = count > w ? (count - w + NW - 1) / NW : 0;   // this warp's stages
    const uint64_t pol = l2_evict_first();

    // the block id of list entry e (-1: none) and its tokens
    auto block_of = [&](int e, int* ntok) -> int {
        *ntok = 0;
        if (e >= total) return -1;
        const int j = list[e], before = e > 0 ? list[e - 1] : -1;
        if (j < 0) return -1;                               // padding
        // past the sequence, repeated or out of order, or behind padding
        if (j >= nblk || j <= before || (e > 0 && before < 0)) {
            flag_error(p.err, kErrOutOfRange);
            return -1;
        }
        const int id = p.block_tables[(size_t)b * p.max_blocks + j];
        if (id < 0 || id >= p.num_blocks) {
            flag_error(p.err, kErrOutOfRange);
            return -1;
        }
        *ntok = min(PBS, L - j * PBS);
        return id;
    };
    // 32 stages per warp-wide read
    int id_a = -1, id_b = -1, tok_a = 0, tok_b = 0, chunk = -1;
    auto issue = [&](int kk) {                              // the whole converged warp
        if ((kk >> 5) != chunk) {
            chunk = kk >> 5;
            const int mine = (chunk << 5) + lane;
            id_a = id_b = -1;
            tok_a = tok_b = 0;
            if (mine < nk) {
                const int e = (first + w + mine * NW) * PAIR;
                id_a = block_of(e, &tok_a);
                if constexpr (PAIR == 2) {
                    id_b = block_of(e + 1, &tok_b);
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
        const int s = kk % ST;
        const uint32_t bar = smem_addr(&bars[w * ST + s]);
        const int ia = __shfl_sync(kFull, id_a, kk & 31), ta = __shfl_sync(kFull, tok_a, kk & 31);
        const int ib = PAIR == 2 ? __shfl_sync(kFull, id_b, kk & 31) : -1;
        const int tb = PAIR == 2 ? __shfl_sync(kFull, tok_b, kk & 31) : 0;
        if (lane == 0) stage_tok[w * ST + s] = ta + tb;
        __syncwarp();
        if (ia >= 0) {
            const uint32_t dst = smem_addr(ring + (size_t)((w * ST + s) * 2) * TILE);
            const size_t off = ((size_t)ia * p.num_kv_heads + hk) * PTILE;
            mbar_arrive_expect_tx_elect(bar, (ib >= 0 ? 4 : 2) * PTILE);
            bulk_g2s_elect(dst, p.k_pool + off, PTILE, bar, pol);
            bulk_g2s_elect(dst + TILE, p.v_pool + off, PTILE, bar, pol);
            if (ib >= 0) {
                const size_t off2 = ((size_t)ib * p.num_kv_heads + hk) * PTILE;
                bulk_g2s_elect(dst + PTILE, p.k_pool + off2, PTILE, bar, pol);
                bulk_g2s_elect(dst + TILE + PTILE, p.v_pool + off2, PTILE, bar, pol);
            }
        } else {
            mbar_arrive_elect(bar);
        }
    };
    for (int kk = 0; kk < nk && kk < ST; ++kk) issue(kk);

    for (int i = tid; i < G * D; i += NW * 32) {            // query rows of this CTA
        const float qv = decode::to_f(static_cast<const QT*>(p.q)[((size_t)b * p.num_heads + hk * G) * D + i]);
        qs[i] = Math::kPrescaledQ ? qv * p.qscale : qv;
    }
    __syncthreads();
    typename Math::State st;
    Math::init(st, qs, lane);
    float* pb = wsm + w * Math::kWarpSmemFloats;

    bool aborted = false;
    int k = 0;
    for (; k < nk; ++k) {
        const int s = k % ST;
        const bool ok = mbar_wait_bounded(smem_addr(&bars[w * ST + s]), (k / ST) & 1, p.err);
        if (__any_sync(kFull, !ok)) {
            aborted = true;
            break;
        }
        const int ntok = stage_tok[w * ST + s];
        if (ntok > 0) {
            const unsigned char* kt = ring + (size_t)((w * ST + s) * 2) * TILE;
            if constexpr (Math::kWarpSmemFloats > 0)
                Math::tile(st, kt, kt + TILE, ntok, lane, qs, pb);
            else
                Math::template tile<false>(st, kt, kt + TILE, ntok, lane, p.qscale, qs, pb, -1);
        }
        __syncwarp();
        if (k + ST < nk) {
            fence_proxy_async_smem();
            issue(k + ST);
        }
    }
    if (aborted) {
        // as in the decode kernel: record it and let the copies in flight land
        if (lane == 0) flag_error(p.err, kErrTimeout);
        const int last = min(nk, k + ST);
        for (int kk = k; kk < last; ++kk)
            (void)mbar_wait_bounded(smem_addr(&bars[w * ST + (kk % ST)]), (kk / ST) & 1, nullptr);
    }

    __syncthreads();                                        // every warp is done with its ring
    float* cm = reinterpret_cast<float*>(ring);             // [NW][G]
    float* cl = cm + NW * G;                                // [NW][G]
    float* cacc = cl + NW * G;                              // [NW][G][D]
    float* pm = cacc + NW * G * D;                          // [G]     this part's maxima,
    float* pl = pm + G;                                     // [G]     sums
    float* po = pl + G;                                     // [G][D]  and weighted sums
    static_assert((NW * G * (D + 2) + G * (D + 2)) * 4 <= P::kRingBytes, "merge area");
    Math::finish(st, cm, cl, cacc, w, lane, aborted);
    __syncthreads();
    // ---- merge the warps, then (through the cluster) the parts
    QT* out = static_cast<QT*>(p.out) + ((size_t)b * p.num_heads + hk * G) * D;
    for (int idx = tid; idx < G * D; idx += NW * 32) {
        const int g = idx / D, dd = idx % D;
        float M = -INFINITY;
#pragma unroll
        for (int ww = 0; ww < NW; ++ww) M = fmaxf(M, cm[ww * G + g]);
        float S = 0.f, O = 0.f;
        if (M != -INFINITY) {
#pragma unroll
            for (int ww = 0; ww < NW; ++ww) {
                const float e = exp2f(cm[ww * G + g] - M);
                S += e * cl[ww * G + g];
                O += e * cacc[(ww * G + g) * D + dd];
            }
        }
        if (parts == 1) {
            decode::store_out(out + idx, (S > 0.f ? O / S : 0.f) * p.v_scale);
        } else {
            po[idx] = O;
            if (dd == 0) {
                pm[g] = M;
                pl[g] = S;
            }
        }
    }
    if (parts == 1) return;
    cluster_sync();
    const int share = (G * D + parts - 1) / parts;
    const int i1 = min(G * D, (part + 1) * share);
    for (int idx = part * share + tid; idx < i1; idx += NW * 32) {
        const int g = idx / D;
        float m[kMaxParts], M = -INFINITY;
#pragma unroll
        for (int r = 0; r < kMaxParts; ++r) {
            m[r] = r < parts ? cluster_ld(cluster_map(smem_addr(pm + g), r)) : -INFINITY;
            M = fmaxf(M, m[r]);
        }
        float S = 0.f, O = 0.f;
        if (M != -INFINITY) {
#pragma unroll
            for (int r = 0; r < kMaxParts; ++r)
                if (r < parts) {
                    const float e = exp2f(m[r] - M);
                    S += e * cluster_ld(cluster_map(smem_addr(pl + g), r));
                    O += e * cluster_ld(cluster_map(smem_addr(po + idx), r));
                }
        }
        decode::store_out(out + idx, (S > 0.f ? O / S : 0.f) * p.v_scale);
    }
    cluster_sync();                                         // partners are done reading
}

template <class Math, typename QT, int D, int BS, int G, int PAIR>
int launch(const Args& a) {
    using P = decode::Pipe<Math, D, BS, G, kNumWarps>;
    auto kern = sparse_decode_kernel<Math, QT, D, BS, G, kNumWarps, PAIR>;
    int occ = 0;
    const int st = kernel_setup(reinterpret_cast<const void*>(kern), P::kSmem, kNumWarps * 32, &occ);
    if (st != PKV_OK) return st;
    // parts of a row: doubled until the CTAs make two waves, each part keeping a
    // stage per warp
    const int stages = ((a.p.k < a.p.max_blocks ? a.p.k : a.p.max_blocks) + PAIR - 1) / PAIR;
    const long long rows = (long long)a.num_seqs * a.p.num_kv_heads;
    const long long wave = (long long)num_sms() * (occ > 0 ? occ : 1);
    int parts = 1;
    while (parts < kMaxParts && rows * parts < 2 * wave && 2 * parts * kNumWarps <= stages) parts *= 2;
    Params p = a.p;
    p.qscale = a.scale * a.k_scale * kLog2e;
    p.v_scale = a.v_scale;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(parts, p.num_kv_heads, a.num_seqs);
    cfg.blockDim = dim3(kNumWarps * 32);
    cfg.dynamicSmemBytes = P::kSmem;
    cfg.stream = a.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = parts;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    note_launch();
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    return e == cudaSuccess ? PKV_OK : cuda_fail("sparse decode: kernel launch", e);
}

template <class Math, typename QT, typename KV, int D, int BS, int G>
int launch_variant(const Args& a) {
    if constexpr (Math::kPairStages)
        return launch<decode::MmaMath<KV, D, 2 * BS, G>, QT, D, 2 * BS, G, 2>(a);
    else
        return launch<Math, QT, D, BS, G, 1>(a);
}

// As the decode: float32 caches on CUDA cores, bf16 / E4M3 caches on CUDA cores
// for one query head per kv head and on the tensor cores for 2, 4, 8.
template <typename QT, typename KV, int D, int BS>
int dispatch_group(const Args& a) {
    constexpr bool simt_only = std::is_same<KV, float>::value;
    switch (a.p.num_heads / a.p.num_kv_heads) {
        case 1: return launch_variant<decode::SimtMath<QT, KV, D, BS, 1>, QT, KV, D, BS, 1>(a);
        case 2:
            if constexpr (simt_only) return launch_variant<decode::SimtMath<QT, KV, D, BS, 2>, QT, KV, D, BS, 2>(a);
            else return launch_variant<decode::MmaMath<KV, D, BS, 2>, QT, KV, D, BS, 2>(a);
        case 4:
            if constexpr (simt_only) return launch_variant<decode::SimtMath<QT, KV, D, BS, 4>, QT, KV, D, BS, 4>(a);
            else return launch_variant<decode::MmaMath<KV, D, BS, 4>, QT, KV, D, BS, 4>(a);
        case 8:
            if constexpr (simt_only) return launch_variant<decode::SimtMath<QT, KV, D, BS, 8>, QT, KV, D, BS, 8>(a);
            else return launch_variant<decode::MmaMath<KV, D, BS, 8>, QT, KV, D, BS, 8>(a);
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
