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
// Work split. A lane holds 16 dims: the two chunks of 8 that turn together, or, where neighbours
// turn, two as far apart (so that the lanes' 16 bytes lie side by side either way); the lanes of a
// row (8 for 128 dims) are neighbours, so the sum of squares is log2 of them shuffles. A warp takes
// 32 / lanes tokens and walks over some of the heads with one set of cosines, sines and (if shared by
// the heads) weights in registers, the next heads on their way through asynchronous copies: a lane's
// own 32 bytes of each, which cost no registers and wait for no other lane. V goes through
// rotary_and_cache's own path.
// Bound: HBM bytes for many tokens (8192 tokens of 32 + 2 x 8 bf16 heads of 128, three axes,
// weights of each head: 41 us, 0.73 of the copy rate; the issue slots are half in use), a launch
// and a chain of loads for few (64 tokens 3.6 us). Of the 41 us the heads' own weights cost 5 (36.3 with
// shared ones); pairs side by side take 43.5, and 48.8 with a lane's two chunks next to each other.
// Into an E4M3 cache 45.0 us (shared weights 41.6), 0.61: issue slots, of which the codes take more (0.57
// of all cycles, 0.53 into bf16). Float32 87.7 (83.7), 0.68: twice the shared-memory pieces, on which
// and on whose copies its warps wait (issue on 0.23 of all cycles).
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

// Two float32 numbers an instruction: half the heads' arithmetic. The products' sums are fused
// (a rounding less than rotary_and_cache's, whose bits are given).
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 split(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
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

// 16 bytes from memory to shared memory, in the background
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_sent() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {            // all but the last N groups have landed
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Heads a warp has on their way, and the CTAs of an SM the registers are shared by (8192 bf16
// tokens: 41.0 us; with 4 heads 41.5; 6 or 8 CTAs 43 and 47; registers for two batches of two
// heads instead of the ring 44.4, of one 43.5).
template <typename ST> struct Ring {
    static constexpr int kDepth = 3, kCtas = sizeof(ST) == 4 ? 6 : 7;
    static constexpr int kHead = 32 * 16 * (int)sizeof(ST), kWarp = kDepth * kHead;   // bytes: 16 dims a lane
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

// Cosines and sines of the pairs i0 .. i0+3 at the token's positions
__device__ __forceinline__ void load_four_turns(const RotaryParams& p, const Token& token, int i0, float* cs, float* sn) {
    const int half = p.rot >> 1;
    int a = 0;
    while (i0 >= p.section_end[a]) ++a;
    auto row_of = [&](int axis) {
        int x = token.pos[0];
#pragma unroll
        for (int k = 1; k < kMaxAxes; ++k) x = axis == k ? token.pos[k] : x;
        return p.cos_sin + (long long)x * p.rot;
    };
    if (i0 + 3 < p.section_end[a]) {                       // one axis for all 4 pairs
        const float4 c = *reinterpret_cast<const float4*>(row_of(a) + i0), s = *reinterpret_cast<const float4*>(row_of(a) + i0 + half);
        cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
        sn[0] = s.x, sn[1] = s.y, sn[2] = s.z, sn[3] = s.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            while (i0 + j >= p.section_end[a]) ++a;
            const float* row = row_of(a) + i0 + j;
            cs[j] = row[0];
            sn[j] = row[half];
        }
    }
}

// Heads h .. h_end-1 of q (KEYS false) or k of the tokens of group tg. Every lane copies its own
// dims of the heads ahead to its own places of `ring`, so nothing but its own copies has to land.
template <typename ST, typename CT, bool INTERLEAVED, bool KEYS>
__device__ __forceinline__ void norm_heads(const NormParams& n, long long tg, int h, int h_end, unsigned char* ring) {
    constexpr int DEP = Ring<ST>::kDepth, HEAD = Ring<ST>::kHead, PIECES = sizeof(ST) == 4 ? 2 : 1;   // of 8 dims
    const RotaryParams& p = n.r;
    const int lane = threadIdx.x & 31, lanes = 1 << n.lanes_log2, u = lane & (lanes - 1);
    const long long t = (tg << (5 - n.lanes_log2)) + (lane >> n.lanes_log2);
    const int d = p.d, half = p.rot >> 1;
    const bool has = t < p.num_tokens && 16 * u < d;       // a row to read
    const bool turns = 16 * u < p.rot;
    int da, db;                                            // the unit's two chunks of 8 dims
    if (!turns) {
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
    const int heads = h_end - h;
    unsigned char* const mine = ring + lane * 16;
    auto send = [&](int i, int slot) {                     // head i of these, if there is one
        if (has && i < heads) {
            const uint32_t to = smem_addr(mine) + slot * HEAD;
            const ST* from = src + (long long)i * d;
#pragma unroll
            for (int k = 0; k < PIECES; ++k) {
                copy16(to + k * 512, from + da + k * 4);
                copy16(to + (PIECES + k) * 512, from + db + k * 4);
            }
        }
        copies_sent();
    };
#pragma unroll
    for (int i = 0; i < DEP; ++i) send(i, i);
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
    if (live && turns) {
        if constexpr (INTERLEAVED) {
            load_four_turns(p, token, 4 * u, cs, sn);
            load_four_turns(p, token, half / 2 + 4 * u, cs + 4, sn + 4);
        } else {
            load_turns(p, token, u, cs, sn);
        }
    }
    const long long tile_elems = (long long)d * p.bs;
    const long long blk = live ? token.slot / p.bs : 0;
    const int off = live ? (int)(token.slot - blk * p.bs) : 0;
    CT* tile = static_cast<CT*>(p.k_pool) + (blk * p.hkv + h) * tile_elems;
    ST* dst = static_cast<ST*>(p.q_out) + t * p.q_out_stride + (long long)h * d;
    int slot = 0;
#pragma unroll 1
    for (int i = 0; i < heads; ++i) {
        copies_wait<DEP - 1>();
        float x[8], y[8];
        if constexpr (PIECES == 2) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float4 a = *reinterpret_cast<const float4*>(mine + slot * HEAD + k * 512);
                const float4 b = *reinterpret_cast<const float4*>(mine + slot * HEAD + (2 + k) * 512);
                x[4 * k] = a.x, x[4 * k + 1] = a.y, x[4 * k + 2] = a.z, x[4 * k + 3] = a.w;
                y[4 * k] = b.x, y[4 * k + 1] = b.y, y[4 * k + 2] = b.z, y[4 * k + 3] = b.w;
            }
        } else {
            Raw8<ST> a, b;
            a.load(reinterpret_cast<const ST*>(mine + slot * HEAD));
            b.load(reinterpret_cast<const ST*>(mine + slot * HEAD + 512));
            a.floats(x);
            b.floats(y);
        }
        uint64_t s2 = 0ull;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const uint64_t a = f2(x[j], x[j + 1]), b = f2(y[j], y[j + 1]);
            s2 = fma2(a, a, fma2(b, b, s2));
        }
        float sum = has ? split(s2).x + split(s2).y : 0.f;
        for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        send(i + DEP, slot);                               // the place has been read
        if (++slot == DEP) slot = 0;
        if (live) {
            const float by = rsqrtf(fmaf(sum, n.inv_d, n.eps));
            const uint64_t by2 = f2(by, by);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                uint64_t a = mul2(mul2(f2(x[j], x[j + 1]), by2), f2(wa[j], wa[j + 1]));
                uint64_t b = mul2(mul2(f2(y[j], y[j + 1]), by2), f2(wb[j], wb[j + 1]));
                if (!INTERLEAVED && turns) {
                    const uint64_t c = f2(cs[j], cs[j + 1]), t = f2(sn[j], sn[j + 1]), m = f2(-sn[j], -sn[j + 1]);
                    const uint64_t r = fma2(a, c, mul2(b, m));
                    b = fma2(b, c, mul2(a, t));
                    a = r;
                }
                x[j] = split(a).x, x[j + 1] = split(a).y;
                y[j] = split(b).x, y[j + 1] = split(b).y;
            }
            if (step && i + 1 < heads) {                   // the next head's own weights
                load_weights<ST>(weight, n.weights_f32, (long long)(h + i + 1) * step + da, wa);
                load_weights<ST>(weight, n.weights_f32, (long long)(h + i + 1) * step + db, wb);
            }
            if (INTERLEAVED && turns) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x0 = x[2 * j], y0 = y[2 * j];
                    x[2 * j] = fmaf(x0, cs[j], -(x[2 * j + 1] * sn[j]));
                    x[2 * j + 1] = fmaf(x[2 * j + 1], cs[j], x0 * sn[j]);
                    y[2 * j] = fmaf(y0, cs[4 + j], -(y[2 * j + 1] * sn[4 + j]));
                    y[2 * j + 1] = fmaf(y[2 * j + 1], cs[4 + j], y0 * sn[4 + j]);
                }
            }
            if constexpr (KEYS) {
                store_k8(tile, d, da, off, x, p.k_scale);
                store_k8(tile, d, db, off, y, p.k_scale);
            } else {
                store8(dst + da, x);
                store8(dst + db, y);
            }
        }
        if constexpr (KEYS) tile += tile_elems;
        else dst += d;
    }
    copies_wait<0>();
}

template <typename ST, typename CT, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, Ring<ST>::kCtas) norm_rotary_and_cache_kernel(const NormParams n) {
    pdl_enter();                                           // launched with launch_pdl
    constexpr int kBytes = Turn<CT>::kWarp > Ring<ST>::kWarp ? Turn<CT>::kWarp : Ring<ST>::kWarp;
    __shared__ __align__(16) unsigned char scratch[kThreads / 32][kBytes];   // of v's or of the other heads' warps
    unsigned char* const mine = scratch[threadIdx.x >> 5];
    const RotaryParams& p = n.r;
    long long warp = blockIdx.x * (long long)(kThreads / 32) + (threadIdx.x >> 5);
    if (warp < n.v_warps) {                                // columns fastest, then heads, then tokens
        const int cg = (int)(warp % p.cols);
        const long long rest = warp / p.cols;
        const int h = (int)(rest % p.kv_chunks) * p.kv_step;
        write_v_heads<ST, CT>(p, rest / p.kv_chunks, cg, h, min(p.hkv, h + p.kv_step), mine);
        return;
    }
    warp -= n.v_warps;
    const int chunks = p.chunks;                           // of k, then q
    const int chunk = (int)(warp % chunks);
    const long long tg = warp / chunks;
    if ((tg << (5 - n.lanes_log2)) >= p.num_tokens) return;    // the whole warp
    if (chunk < p.kv_chunks) {
        const int h = chunk * p.kv_step;
        norm_heads<ST, CT, INTERLEAVED, true>(n, tg, h, min(p.hkv, h + p.kv_step), mine);
    } else {
        const int h = (chunk - p.kv_chunks) * p.q_step;
        norm_heads<ST, CT, INTERLEAVED, false>(n, tg, h, min(p.hq, h + p.q_step), mine);
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
