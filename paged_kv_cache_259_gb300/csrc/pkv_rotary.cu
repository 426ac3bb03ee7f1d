// rotary_and_cache: the rotated append. Every new token's q and k heads are
// turned by the token's positions, q goes to q_out, k and v into the token's
// pool slot (the position rotation folded into reshape_and_cache, so k is read
// and written once).
//
// Mathematics. Pair i < R/2 of a head (dims i and i + R/2, or 2i and 2i + 1)
// turns by the angle of position p = positions[axis(i)][t] and frequency i,
// whose cosine and sine the caller's table holds:
//     x1' = x1 cos - x2 sin,   x2' = x2 cos + x1 sin,
// every product and sum rounded to float32 on its own (no fused multiply-add),
// so a result does not depend on how the compiler contracts the expression; then
// one rounding to the query's or the cache's type. The table is an input: an
// angle of a far position needs 64 bits (1e6 rad has an ulp of 0.06 in float32),
// which the table is built in once and the step then never pays for.
//
// Bound: HBM bytes for many tokens (8192 tokens of 32 + 2 x 8 bf16 heads of 128, three
// axes: 34.7 us, 0.85 of the copy rate), a launch and a chain of loads for few (64 tokens
// 2.9 us; 1071 tokens into an E4M3 cache 8.4).
//
// Work split. A warp takes a few tokens and walks over some of the heads with one
// set of cosines and sines in registers, a batch of heads at a time, the first batch
// read before the slot, the positions and the table rows have arrived. For q and k a
// lane holds two chunks of 8 dims that turn together; a K chunk is 16 bytes of the
// block's tile, next to the same chunk of the neighbouring tokens. V is stored
// transposed ([dim][token]): each warp turns its 8 x 64 elements through shared
// memory. No store needs the slots to be consecutive or aligned: each token goes by
// its own slot.
#include "pkv_rotary_impl.cuh"

namespace pkv {
namespace {

using namespace rotary;

// Heads h .. h_end-1 of q (KEYS false) or k: 8 tokens x 4 units of 16 dims, lane
// 4r + c token r, unit c, so a load covers 64 contiguous bytes of 8 rows (bf16). A
// batch of heads is read while the one before it turns.
template <typename ST, typename CT, bool INTERLEAVED, bool KEYS>
__device__ __forceinline__ void rotate_heads(const RotaryParams& p, long long tg, int cg, int h, int h_end) {
    constexpr int HB = Batching<ST>::kHeads;
    const int lane = threadIdx.x & 31, u = cg * 4 + (lane & 3);
    const long long t = tg * 8 + (lane >> 2);
    const int d = p.d, half = p.rot >> 1;
    const bool has = t < p.num_tokens && 16 * u < d;       // a row to read
    const bool turns = 16 * u < p.rot;
    // the unit's two chunks of 8 dims
    int da, db;
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
        for (int i = 0; i < HB; ++i)
            if (has && i < left) {
                x.a[i].load(src + i * d + da);
                x.b[i].load(src + i * d + db);
            }
        src += HB * d;
    };
    int left = h_end - h;
    Batch now, next;
    read(now, left);
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
            if (!live || i >= left) continue;
            float x[8], y[8];
            batch.a[i].floats(x);
            batch.b[i].floats(y);
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
__global__ void __launch_bounds__(kThreads, Batching<ST>::kCtas) rotary_and_cache_kernel(const RotaryParams p) {
    pdl_enter();                                           // launched with launch_pdl
    __shared__ __align__(16) unsigned char turn[kThreads / 32][Turn<CT>::kWarp];
    const long long warp = blockIdx.x * (long long)(kThreads / 32) + (threadIdx.x >> 5);
    // columns fastest, then heads (v, k, q), then tokens: neighbouring warps share rows
    const int cg = (int)(warp % p.cols);
    const long long rest = warp / p.cols;
    int chunk = (int)(rest % p.chunks);
    const long long tg = rest / p.chunks;
    if (tg * 8 >= p.num_tokens) return;                    // the whole warp
    if (chunk < 2 * p.kv_chunks) {
        const bool keys = chunk >= p.kv_chunks;
        const int h = (keys ? chunk - p.kv_chunks : chunk) * p.kv_step, h_end = min(p.hkv, h + p.kv_step);
        if (keys) rotate_heads<ST, CT, INTERLEAVED, true>(p, tg, cg, h, h_end);
        else write_v_heads<ST, CT>(p, tg, cg, h, h_end, turn[threadIdx.x >> 5]);
        return;
    }
    const int h = (chunk - 2 * p.kv_chunks) * p.q_step;
    rotate_heads<ST, CT, INTERLEAVED, false>(p, tg, cg, h, min(p.hq, h + p.q_step));
}

template <typename ST, typename CT>
cudaError_t launch_rotary(RotaryParams p, bool interleaved, cudaStream_t stream) {
    p.cols = (p.d + 63) / 64;
    const long long items = ((long long)p.num_tokens + 7) / 8 * p.cols;
    // heads a warp walks: one while the warps are fewer than 32 an SM, then more, up to
    // 8 of q and 4 of k or v (the slots, positions and table rows are read once for
    // all of them): 8192 tokens took 50 us with one, 39 us with 4 and 2, 35 us with 8
    // and 4, 38 us with 16 and 4
    auto step_of = [&](int heads, int limit) {
        const long long s = items * (p.hq + 2 * p.hkv) / (32LL * num_sms());
        const int most = s < 1 ? 1 : s > limit ? limit : (int)s;
        const int chunks = (heads + most - 1) / most;
        return (heads + chunks - 1) / chunks;              // even shares
    };
    p.q_step = step_of(p.hq, 8);
    p.kv_step = step_of(p.hkv, 4);
    p.kv_chunks = (p.hkv + p.kv_step - 1) / p.kv_step;
    p.chunks = 2 * p.kv_chunks + (p.hq + p.q_step - 1) / p.q_step;
    const long long blocks = (items * p.chunks + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    note_launch();
    auto kern = interleaved ? rotary_and_cache_kernel<ST, CT, true> : rotary_and_cache_kernel<ST, CT, false>;
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(kThreads), 0, stream, p);
}

}  // namespace

namespace rotary {
int rotary_params(RotaryParams& p, bool* done, void* q_out, const void* q, const void* k, const void* v, void* k_pool,
                  void* v_pool, const int64_t* slot_mapping, const int32_t* positions, const float* cos_sin,
                  const int32_t* sections, int num_axes, int64_t q_out_stride, int64_t q_stride, int64_t k_stride,
                  int64_t v_stride, int num_tokens, int num_heads, int num_kv_heads, int head_dim, int rotary_dim,
                  int block_size, int num_blocks, int num_positions, int src_dtype, int cache_dtype, float k_scale,
                  float v_scale) {
    *done = false;
    if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        num_blocks <= 0 || num_positions <= 0 || rotary_dim <= 0 || rotary_dim > head_dim ||
        num_heads % num_kv_heads != 0 || num_axes < 1 || !sections)
        return PKV_ERR_INVALID_ARG;
    if (head_dim % 16 != 0 || rotary_dim % 16 != 0 || block_size % 16 != 0 || num_axes > kMaxAxes ||
        head_dim > 1024 || num_heads > 65535)
        return PKV_ERR_UNSUPPORTED;
    long long pairs = 0;
    for (int a = 0; a < num_axes; ++a) {
        if (sections[a] < 0 || sections[a] > rotary_dim / 2) return PKV_ERR_INVALID_ARG;
        pairs += sections[a];
        p.section_end[a] = (int)pairs;
    }
    if (pairs != rotary_dim / 2) return PKV_ERR_INVALID_ARG;
    const size_t elt = src_dtype == PKV_F32 ? 4 : 2;
    const int64_t q_row = (int64_t)num_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
    if (q_out_stride < q_row || q_stride < q_row || k_stride < kv_row || v_stride < kv_row ||
        (q_out_stride * elt) % 16 || (q_stride * elt) % 16 || (k_stride * elt) % 16 ||
        (v_stride * elt) % 16)
        return PKV_ERR_INVALID_ARG;
    if (q_out && q_out == q && q_out_stride != q_stride) return PKV_ERR_INVALID_ARG;
    const bool fp8 = cache_dtype == PKV_E4M3;
    if (fp8) {
        if (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
            return PKV_ERR_INVALID_ARG;
    } else if (k_scale != 1.f || v_scale != 1.f) {
        return PKV_ERR_INVALID_ARG;
    }
    if (!((src_dtype == PKV_F32 || src_dtype == PKV_BF16) && (fp8 || cache_dtype == src_dtype)))
        return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) {
        *done = true;
        return PKV_OK;
    }
    if (!q_out || !q || !k || !v || !k_pool || !v_pool || !slot_mapping || !positions || !cos_sin)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(q_out) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(k_pool) ||
        !aligned16(v_pool) || !aligned16(cos_sin))
        return PKV_ERR_INVALID_ARG;
    p.q_out = q_out;
    p.q = q;
    p.k = k;
    p.v = v;
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.slots = slot_mapping;
    p.positions = positions;
    p.cos_sin = cos_sin;
    p.q_out_stride = q_out_stride;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.num_tokens = num_tokens;
    p.hq = num_heads;
    p.hkv = num_kv_heads;
    p.d = head_dim;
    p.rot = rotary_dim;
    p.bs = block_size;
    p.num_blocks = num_blocks;
    p.num_positions = num_positions;
    p.axes = num_axes;
    auto scale_of = [](float s) { return Scale{s, s > 0x1p-100f && s < 0x1p100f ? 1.f / s : 0.f}; };
    p.k_scale = scale_of(k_scale);
    p.v_scale = scale_of(v_scale);
    return PKV_OK;
}
}  // namespace rotary
}  // namespace pkv

extern "C" {

int rotary_and_cache(void* q_out, const void* q, const void* k, const void* v, void* k_pool,
                     void* v_pool, const int64_t* slot_mapping, const int32_t* positions,
                     const float* cos_sin, const int32_t* sections, int num_axes,
                     int64_t q_out_stride, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                     int num_tokens, int num_heads, int num_kv_heads, int head_dim, int rotary_dim,
                     int interleaved, int block_size, int num_blocks, int num_positions,
                     int src_dtype, int cache_dtype, float k_scale, float v_scale, void* stream) {
    using namespace pkv;
    RotaryParams p{};
    bool done;
    const int st = rotary_params(p, &done, q_out, q, k, v, k_pool, v_pool, slot_mapping, positions, cos_sin, sections,
                                 num_axes, q_out_stride, q_stride, k_stride, v_stride, num_tokens, num_heads,
                                 num_kv_heads, head_dim, rotary_dim, block_size, num_blocks, num_positions, src_dtype,
                                 cache_dtype, k_scale, v_scale);
    if (st != PKV_OK || done) return st;
    const bool fp8 = cache_dtype == PKV_E4M3;
    if (checking()) return PKV_OK;
    p.err = error_word();
    if (!p.err) return PKV_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (src_dtype == PKV_F32)
        e = fp8 ? launch_rotary<float, uint8_t>(p, interleaved != 0, s)
                : launch_rotary<float, float>(p, interleaved != 0, s);
    else
        e = fp8 ? launch_rotary<__nv_bfloat16, uint8_t>(p, interleaved != 0, s)
                : launch_rotary<__nv_bfloat16, __nv_bfloat16>(p, interleaved != 0, s);
    return e == cudaSuccess ? PKV_OK : cuda_fail("rotary_and_cache: kernel launch", e);
}

}  // extern "C"
