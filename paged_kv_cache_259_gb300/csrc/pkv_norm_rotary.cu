// norm_rotary_and_cache: the rotated append of models that normalise their query and key
// heads. Every head x of q and k becomes
//     y = x * rsqrt(mean(x^2) + eps) * w
// and is then turned and written as rotary_and_cache does; v goes into its slot as it is.
//
// Mathematics. One read of a head gives both its sum of squares and the values to scale, so
// the norm costs no byte next to the append. The sum, the root, both products and the
// rotation are float32, and there is one rounding, to the type of q_out or of the cache: a
// norm written out in between would round to 16 bits (2^-9 of the value) first.
//
// Work split. A lane holds the 16 dims of rotary_and_cache (the two chunks of 8 that turn
// together); the lanes of a row (8 for 128 dims) are neighbours, so the sum of squares is
// log2 of them shuffles. A warp takes 32 / lanes tokens and walks over some of the heads with
// one set of cosines, sines and (if shared by the heads) weights in registers, a batch of
// heads read while the one before it turns. V goes through rotary_and_cache's own path.
#include "pkv_rotary_impl.cuh"

namespace pkv {
namespace {

using namespace rotary;

struct NormParams {
    RotaryParams r;
    const void* q_weight;
    const void* k_weight;
    int q_weight_step, k_weight_step;  // elements from a head's weights to the next's; 0: shared
    int weights_f32;                   // else of q's type
    float eps, inv_d;
    int lanes_log2;                    // of a row
    long long v_warps;                 // the first ones of the launch
};

template <typename ST>
__device__ __forceinline__ void load_weights(const void* w, int f32, long long at, float (&f)[8]) {
    if (f32) {
        load8(static_cast<const float*>(w) + at, f);
    } else {
        Raw8<ST> r;
        r.load(static_cast<const ST*>(w) + at);
        r.floats(f);
    }
}

// Heads h .. h_end-1 of q (KEYS false) or k of the tokens of group tg
template <typename ST, typename CT, bool INTERLEAVED, bool KEYS>
__device__ __forceinline__ void norm_heads(const NormParams& n, long long tg, int h, int h_end) {
    constexpr int HB = Batching<ST>::kHeads;
    const RotaryParams& p = n.r;
    const int lane = threadIdx.x & 31, lanes = 1 << n.lanes_log2, u = lane & (lanes - 1);
    const long long t = (tg << (5 - n.lanes_log2)) + (lane >> n.lanes_log2);
    const int d = p.d, half = p.rot >> 1;
    const bool has = t < p.num_tokens && 16 * u < d;       // a row to read
    const bool turns = 16 * u < p.rot;
    int da, db;                                            // the unit's two chunks of 8 dims
    if (INTERLEAVED || !turns) {
        da = 16 * u;
        db = da + 8;
    } else {
        da = 8 * u;
        db = half + 8 * u;
    }
    Token token;
    if (has) token.read(p, t);
    const ST* src = (KEYS ? static_cast<const ST*>(p.k) + t * p.k_stride
                          : static_cast<const ST*>(p.q) + t * p.q_stride) + (long long)h * d;
    struct Batch {
        Raw8<ST> a[HB], b[HB];
    };
    auto read = [&](Batch& x, int left) {                  // the next batch, `left` heads at most
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            x.a[i].clear();
            x.b[i].clear();
            if (has && i < left) {
                x.a[i].load(src + i * d + da);
                x.b[i].load(src + i * d + db);
            }
        }
        src += HB * d;
    };
    int left = h_end - h;
    Batch now, next;
    read(now, left);
    const void* const weight = KEYS ? n.k_weight : n.q_weight;
    const int step = KEYS ? n.k_weight_step : n.q_weight_step;
    float wa[8], wb[8];
    if (has) {
        load_weights<ST>(weight, n.weights_f32, (long long)h * step + da, wa);
        load_weights<ST>(weight, n.weights_f32, (long long)h * step + db, wb);
    }
    token.check(p);
    const bool live = token.slot >= 0;
    float cs[8], sn[8];
    if (live && turns) load_turns(p, token, u, cs, sn);
    const long long tile_elems = (long long)d * p.bs;
    const long long blk = live ? token.slot / p.bs : 0;
    const int off = live ? (int)(token.slot - blk * p.bs) : 0;
    CT* tile = static_cast<CT*>(p.k_pool) + (blk * p.hkv + h) * tile_elems;
    ST* dst = static_cast<ST*>(p.q_out) + t * p.q_out_stride + (long long)h * d;
    auto turn = [&](const Batch& batch) {
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            if (i >= left) break;                          // the whole warp
            float x[8], y[8];
            batch.a[i].floats(x);
            batch.b[i].floats(y);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], fmaf(y[j], y[j], sum));
            for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (!live) continue;
            const float by = rsqrtf(fmaf(sum, n.inv_d, n.eps));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = x[j] * by * wa[j];
                y[j] = y[j] * by * wb[j];
            }
            if (step && i + 1 < left) {                    // the next head's own weights
                load_weights<ST>(weight, n.weights_f32, (long long)(h + i + 1) * step + da, wa);
                load_weights<ST>(weight, n.weights_f32, (long long)(h + i + 1) * step + db, wb);
            }
            if (turns) turn16<INTERLEAVED>(x, y, cs, sn);
            if constexpr (KEYS) {
                store_k8(tile + i * tile_elems, d, da, off, x, p.k_scale);
                store_k8(tile + i * tile_elems, d, db, off, y, p.k_scale);
            } else {
                store8(dst + i * d + da, x);
                store8(dst + i * d + db, y);
            }
        }
        left -= HB;
        h += HB;
        if constexpr (KEYS) tile += HB * tile_elems;
        else dst += HB * d;
    };
#pragma unroll 1
    while (left > 0) {
        read(next, left - HB);
        turn(now);
        now = next;
    }
}

template <typename ST, typename CT, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 5) norm_rotary_and_cache_kernel(const NormParams n) {
    pdl_enter();                                           // launched with launch_pdl
    __shared__ __align__(16) unsigned char turn[kThreads / 32][Turn<CT>::kWarp];
    const RotaryParams& p = n.r;
    long long warp = blockIdx.x * (long long)(kThreads / 32) + (threadIdx.x >> 5);
    if (warp < n.v_warps) {                                // columns fastest, then heads, then tokens
        const int cg = (int)(warp % p.cols);
        const long long rest = warp / p.cols;
        const int h = (int)(rest % p.kv_chunks) * p.kv_step;
        write_v_heads<ST, CT>(p, rest / p.kv_chunks, cg, h, min(p.hkv, h + p.kv_step), turn[threadIdx.x >> 5]);
        return;
    }
    warp -= n.v_warps;
    const int chunks = p.chunks;                           // of k, then q
    const int chunk = (int)(warp % chunks);
    const long long tg = warp / chunks;
    if ((tg << (5 - n.lanes_log2)) >= p.num_tokens) return;    // the whole warp
    if (chunk < p.kv_chunks) {
        const int h = chunk * p.kv_step;
        norm_heads<ST, CT, INTERLEAVED, true>(n, tg, h, min(p.hkv, h + p.kv_step));
    } else {
        const int h = (chunk - p.kv_chunks) * p.q_step;
        norm_heads<ST, CT, INTERLEAVED, false>(n, tg, h, min(p.hq, h + p.q_step));
    }
}

template <typename ST, typename CT>
cudaError_t launch_norm(NormParams n, bool interleaved, cudaStream_t stream) {
    RotaryParams& p = n.r;
    p.cols = (p.d + 63) / 64;
    n.lanes_log2 = 0;
    while ((16 << n.lanes_log2) < p.d) ++n.lanes_log2;
    const int per = 32 >> n.lanes_log2;                    // tokens of a warp
    const long long groups = ((long long)p.num_tokens + per - 1) / per;
    // heads a warp walks, as in rotary_and_cache: one while the warps are few, then up to 8
    // of q and 4 of k or v
    auto step_of = [&](int heads, int limit) {
        const long long s = groups * (p.hq + 2 * p.hkv) / (32LL * num_sms());
        const int most = s < 1 ? 1 : s > limit ? limit : (int)s;
        const int chunks = (heads + most - 1) / most;
        return (heads + chunks - 1) / chunks;              // even shares
    };
    p.q_step = step_of(p.hq, 8);
    p.kv_step = step_of(p.hkv, 4);
    p.kv_chunks = (p.hkv + p.kv_step - 1) / p.kv_step;
    p.chunks = p.kv_chunks + (p.hq + p.q_step - 1) / p.q_step;
    n.v_warps = ((long long)p.num_tokens + 7) / 8 * p.cols * p.kv_chunks;
    const long long warps = n.v_warps + groups * p.chunks, blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    note_launch();
    auto kern = interleaved ? norm_rotary_and_cache_kernel<ST, CT, true> : norm_rotary_and_cache_kernel<ST, CT, false>;
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(kThreads), 0, stream, n);
}

}  // namespace
}  // namespace pkv

extern "C" int norm_rotary_and_cache(
    void* q_out, const void* q, const void* k, const void* v, const void* q_weight, const void* k_weight,
    void* k_pool, void* v_pool, const int64_t* slot_mapping, const int32_t* positions, const float* cos_sin,
    const int32_t* sections, int num_axes, int64_t q_out_stride, int64_t q_stride, int64_t k_stride,
    int64_t v_stride, int64_t q_weight_stride, int64_t k_weight_stride, int num_tokens, int num_heads,
    int num_kv_heads, int head_dim, int rotary_dim, int interleaved, int block_size, int num_blocks,
    int num_positions, int src_dtype, int cache_dtype, int weight_dtype, float eps, float k_scale, float v_scale,
    void* stream) {
    using namespace pkv;
    NormParams n{};
    if (!std::isfinite(eps) || eps < 0.f) return PKV_ERR_INVALID_ARG;
    bool done;
    const int st = rotary_params(n.r, &done, q_out, q, k, v, k_pool, v_pool, slot_mapping, positions, cos_sin,
                                 sections, num_axes, q_out_stride, q_stride, k_stride, v_stride, num_tokens,
                                 num_heads, num_kv_heads, head_dim, rotary_dim, block_size, num_blocks,
                                 num_positions, src_dtype, cache_dtype, k_scale, v_scale);
    if (st != PKV_OK) return st;
    if (head_dim > 512 || (weight_dtype != src_dtype && weight_dtype != PKV_F32)) return PKV_ERR_UNSUPPORTED;
    const int elt = weight_dtype == PKV_F32 ? 4 : 2;
    for (const int64_t s : {q_weight_stride, k_weight_stride})
        if (s != 0 && (s < head_dim || s > 0x7fffffff || s * elt % 16)) return PKV_ERR_INVALID_ARG;
    if (done) return PKV_OK;
    if (!q_weight || !k_weight || !aligned16(q_weight) || !aligned16(k_weight)) return PKV_ERR_INVALID_ARG;
    if (checking()) return PKV_OK;
    n.r.err = error_word();
    if (!n.r.err) return PKV_ERR_CUDA;
    n.q_weight = q_weight;
    n.k_weight = k_weight;
    n.q_weight_step = (int)q_weight_stride;
    n.k_weight_step = (int)k_weight_stride;
    n.weights_f32 = weight_dtype == PKV_F32;
    n.eps = eps;
    n.inv_d = 1.f / (float)head_dim;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool fp8 = cache_dtype == PKV_E4M3;
    cudaError_t e;
    if (src_dtype == PKV_F32)
        e = fp8 ? launch_norm<float, uint8_t>(n, interleaved != 0, s) : launch_norm<float, float>(n, interleaved != 0, s);
    else
        e = fp8 ? launch_norm<__nv_bfloat16, uint8_t>(n, interleaved != 0, s)
                : launch_norm<__nv_bfloat16, __nv_bfloat16>(n, interleaved != 0, s);
    return e == cudaSuccess ? PKV_OK : cuda_fail("norm_rotary_and_cache: kernel launch", e);
}
