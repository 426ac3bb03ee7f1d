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
// Bound: HBM bytes for many tokens, launch and load latency for few.
//
// Work split. A warp takes 8 tokens x 4 units of 16 dims and walks over `heads`
// heads with one set of cosines and sines in registers: lane 4r + c holds
// token r, unit c, so a load covers 64 contiguous bytes of a row (bf16), and a
// K store 8 tokens x 16 bytes, one 128-byte core matrix when the tokens' slots
// follow one another. V is stored transposed ([dim][token]); movmatrix turns
// each 8 x 8 of 16-bit values in registers, after which a lane holds two
// neighbouring tokens of one dim and a quad stores a dim's 8 tokens. No store
// needs the slots to be consecutive or aligned: each token goes by its own slot.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cmath>
#include <type_traits>

#include "pkv_internal.cuh"

namespace pkv {
namespace {

constexpr int kMaxAxes = 4;
constexpr int kThreads = 256;

struct RotaryParams {
    void* q_out;
    const void* q;
    const void* k;
    const void* v;
    void* k_pool;
    void* v_pool;
    const int64_t* slots;
    const int32_t* positions;          // [axes][T]
    const float* cos_sin;              // [P][2][R/2]
    long long q_out_stride, q_stride, k_stride, v_stride;   // elements between tokens
    int num_tokens, hq, hkv, d, rot, bs, num_blocks, num_positions;
    int axes, section_end[kMaxAxes];   // pairs of axis a: section_end[a-1] .. section_end[a]-1
    int head_step, head_chunks, col_groups;
    float k_scale, v_scale;
    int* err;
};

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// 8 consecutive elements <-> floats
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]),
                                              bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}
// E4M3 codes of two values: IEEE divide by the scale, nearest even, saturating
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi, float scale) {
    float2 f;
    f.x = __fdiv_rn(lo, scale);
    f.y = __fdiv_rn(hi, scale);
    return __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
}

// 8 dims d0 .. d0+7 (d0 a multiple of 8) of slot `off` of a K tile.
// CT = uint8_t: cache bytes are E4M3 codes.
template <typename CT>
__device__ __forceinline__ void store_k8(CT* tile, int d, int d0, int off, const float (&f)[8],
                                         float scale) {
    if constexpr (std::is_same<CT, uint8_t>::value) {
        const uint32_t lo = e4m3_pair(f[0], f[1], scale) | (e4m3_pair(f[2], f[3], scale) << 16);
        const uint32_t hi = e4m3_pair(f[4], f[5], scale) | (e4m3_pair(f[6], f[7], scale) << 16);
        *reinterpret_cast<uint2*>(tile + ((off >> 3) * (d / 16) + (d0 >> 4)) * 128 +
                                  (off & 7) * 16 + (d0 & 8)) = make_uint2(lo, hi);
    } else if constexpr (std::is_same<CT, float>::value) {
        float* p = tile + ((off >> 3) * (d / 4) + (d0 >> 2)) * 32 + (off & 7) * 4;
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(p + 32) = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        store8(tile + ((off >> 3) * (d / 8) + (d0 >> 3)) * 64 + (off & 7) * 8, f);
    }
}

// The value of a V element as the 16-bit halves that movmatrix moves.
template <typename CT>
__device__ __forceinline__ void v_halves(float a, float b, float scale, uint32_t& lo, uint32_t& hi) {
    if constexpr (std::is_same<CT, uint8_t>::value) {
        const uint32_t two = e4m3_pair(a, b, scale);         // one code in each half
        lo = (two & 0xffu) | ((two & 0xff00u) << 8);
        hi = 0;
    } else if constexpr (std::is_same<CT, float>::value) {
        const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
        lo = __byte_perm(x, y, 0x5410);
        hi = __byte_perm(x, y, 0x7632);
    } else {
        lo = bf16_pair(a, b);
        hi = 0;
    }
}

template <typename ST, typename CT, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_and_cache_kernel(const RotaryParams p) {
    pdl_enter();                                           // launched with launch_pdl
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const long long warp = blockIdx.x * (long long)(kThreads / 32) + (threadIdx.x >> 5);
    // column groups fastest, then heads, then tokens: neighbouring warps share rows
    const int cg = (int)(warp % p.col_groups);
    const long long rest = warp / p.col_groups;
    const int hc = (int)(rest % p.head_chunks);
    const long long tg = rest / p.head_chunks;
    if (tg * 8 >= p.num_tokens) return;                    // the whole warp
    const long long t = tg * 8 + r;
    const int d = p.d, half = p.rot >> 1;
    const int u = cg * 4 + c;                              // this lane's unit of 16 dims
    const bool in_row = 16 * u < d;

    // ---- the token: its slot and its positions; a bad one is skipped whole
    long long slot = -1;
    if (t < p.num_tokens) {
        slot = p.slots[t];
        bool bad = slot >= (long long)p.num_blocks * p.bs;
#pragma unroll
        for (int a = 0; a < kMaxAxes; ++a)
            if (a < p.axes && slot >= 0) {
                const int pos = p.positions[(long long)a * p.num_tokens + t];
                bad |= pos < 0 || pos >= p.num_positions;
            }
        if (bad) {
            flag_error(p.err, kErrOutOfRange);
            slot = -1;
        }
    }
    const bool live = slot >= 0 && in_row;
    const long long blk = slot >= 0 ? slot / p.bs : 0;
    const int off = slot >= 0 ? (int)(slot - blk * p.bs) : 0;
    const long long tile_elems = (long long)d * p.bs;

    const int h_end = min(p.hq + 2 * p.hkv, (hc + 1) * p.head_step);
    int h = hc * p.head_step;

    // ---- q and k heads
    if (h < p.hq + p.hkv) {
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
        float cs[8], sn[8];
        if (live && turns) {
            const int i0 = 8 * u;
            int a = 0;
            while (i0 >= p.section_end[a]) ++a;
            if (i0 + 7 < p.section_end[a]) {               // one axis for all 8 pairs
                const long long pos = p.positions[(long long)a * p.num_tokens + t];
                const float* row = p.cos_sin + pos * p.rot + i0;
                load8(row, cs);
                load8(row + half, sn);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    while (i0 + j >= p.section_end[a]) ++a;
                    const long long pos = p.positions[(long long)a * p.num_tokens + t];
                    cs[j] = p.cos_sin[pos * p.rot + i0 + j];
                    sn[j] = p.cos_sin[pos * p.rot + half + i0 + j];
                }
            }
        }
        const int rot_end = min(h_end, p.hq + p.hkv);
#pragma unroll 2
        for (; h < rot_end; ++h) {
            const bool is_k = h >= p.hq;
            const ST* src = is_k ? static_cast<const ST*>(p.k) + t * p.k_stride + (long long)(h - p.hq) * d
                                 : static_cast<const ST*>(p.q) + t * p.q_stride + (long long)h * d;
            if (!live) continue;
            float x[8], y[8];
            load8(src + da, x);
            load8(src + db, y);
            if (turns) {
                if constexpr (INTERLEAVED) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x0 = x[2 * j], x1 = x[2 * j + 1], y0 = y[2 * j], y1 = y[2 * j + 1];
                        x[2 * j] = __fsub_rn(__fmul_rn(x0, cs[j]), __fmul_rn(x1, sn[j]));
                        x[2 * j + 1] = __fadd_rn(__fmul_rn(x1, cs[j]), __fmul_rn(x0, sn[j]));
                        y[2 * j] = __fsub_rn(__fmul_rn(y0, cs[4 + j]), __fmul_rn(y1, sn[4 + j]));
                        y[2 * j + 1] = __fadd_rn(__fmul_rn(y1, cs[4 + j]), __fmul_rn(y0, sn[4 + j]));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float x0 = x[j], y0 = y[j];
                        x[j] = __fsub_rn(__fmul_rn(x0, cs[j]), __fmul_rn(y0, sn[j]));
                        y[j] = __fadd_rn(__fmul_rn(y0, cs[j]), __fmul_rn(x0, sn[j]));
                    }
                }
            }
            if (is_k) {
                CT* tile = static_cast<CT*>(p.k_pool) + (blk * p.hkv + (h - p.hq)) * tile_elems;
                store_k8(tile, d, da, off, x, p.k_scale);
                store_k8(tile, d, db, off, y, p.k_scale);
            } else {
                ST* dst = static_cast<ST*>(p.q_out) + t * p.q_out_stride + (long long)h * d;
                store8(dst + da, x);
                store8(dst + db, y);
            }
        }
    }

    __syncwarp();                                          // movmatrix wants the whole warp
    // ---- v heads: after the turn this lane holds tokens 2c, 2c+1 of dims
    //      16 (4 cg + r/2) + 2w + (r & 1)
    if (h < h_end) {
        constexpr int X = 16 / sizeof(CT);
        const long long s0 = __shfl_sync(0xffffffffu, slot, 8 * c);
        const long long s1 = __shfl_sync(0xffffffffu, slot, 8 * c + 4);
        const int dim0 = 16 * (4 * cg + (r >> 1)) + (r & 1);
        const bool dim_ok = dim0 < d;
        const bool ok0 = s0 >= 0 && dim_ok, ok1 = s1 >= 0 && dim_ok;
        const bool both = ok0 && s1 == s0 + 1 && (s0 & 1) == 0;      // one block: block sizes are even
        auto column = [&](long long s) {                   // element of the slot's column, head 0, dim 0
            const long long b = s / p.bs;
            const int o = (int)(s - b * p.bs);
            return b * p.hkv * tile_elems + (long long)(o / X) * d * X + o % X;
        };
        const long long col0 = ok0 ? column(s0) : 0, col1 = ok1 && !both ? column(s1) : 0;
        for (; h < h_end; ++h) {
            const int hv = h - p.hq - p.hkv;
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = 0.f;
            if (live) {
                const ST* src = static_cast<const ST*>(p.v) + t * p.v_stride + (long long)hv * d + 16 * u;
                float a[8], b[8];
                load8(src, a);
                load8(src + 8, b);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = a[i], x[8 + i] = b[i];
            }
            CT* pool = static_cast<CT*>(p.v_pool) + hv * tile_elems;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                uint32_t lo, hi;
                v_halves<CT>(x[2 * w], x[2 * w + 1], p.v_scale, lo, hi);
                lo = movmatrix(lo);
                const int dim = dim0 + 2 * w;
                const int row = (dim >> 3) * 8 * X + (dim & 7) * X;
                if constexpr (std::is_same<CT, float>::value) {
                    hi = movmatrix(hi);
                    const uint32_t v0 = __byte_perm(lo, hi, 0x5410), v1 = __byte_perm(lo, hi, 0x7632);
                    if (both) {
                        *reinterpret_cast<uint2*>(pool + col0 + row) = make_uint2(v0, v1);
                    } else {
                        if (ok0) pool[col0 + row] = __uint_as_float(v0);
                        if (ok1) pool[col1 + row] = __uint_as_float(v1);
                    }
                } else if constexpr (std::is_same<CT, uint8_t>::value) {
                    if (both) {
                        *reinterpret_cast<uint16_t*>(pool + col0 + row) =
                            (uint16_t)((lo & 0xffu) | (lo >> 8));
                    } else {
                        if (ok0) pool[col0 + row] = (uint8_t)lo;
                        if (ok1) pool[col1 + row] = (uint8_t)(lo >> 16);
                    }
                } else {
                    if (both) {
                        *reinterpret_cast<uint32_t*>(pool + col0 + row) = lo;
                    } else {
                        uint16_t* q16 = reinterpret_cast<uint16_t*>(pool);
                        if (ok0) q16[col0 + row] = (uint16_t)lo;
                        if (ok1) q16[col1 + row] = (uint16_t)(lo >> 16);
                    }
                }
            }
        }
    }
}

template <typename ST, typename CT>
cudaError_t launch_rotary(RotaryParams p, bool interleaved, cudaStream_t stream) {
    const int heads = p.hq + 2 * p.hkv;
    p.col_groups = (p.d + 63) / 64;
    const long long groups = (p.num_tokens + 7) / 8;
    // heads a warp walks: one while the warps are few, up to 4 when they fill the GPU
    int step = 1;
    const long long fill = 64LL * num_sms();
    while (step < 4 && groups * p.col_groups * ((heads + 2 * step - 1) / (2 * step)) >= fill) step *= 2;
    p.head_step = step;
    p.head_chunks = (heads + step - 1) / step;
    const long long warps = groups * p.col_groups * p.head_chunks;
    const long long blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    note_launch();
    auto kern = interleaved ? rotary_and_cache_kernel<ST, CT, true> : rotary_and_cache_kernel<ST, CT, false>;
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(kThreads), 0, stream, p);
}

}  // namespace
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
    if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        num_blocks <= 0 || num_positions <= 0 || rotary_dim <= 0 || rotary_dim > head_dim ||
        num_heads % num_kv_heads != 0 || num_axes < 1 || !sections)
        return PKV_ERR_INVALID_ARG;
    if (head_dim % 16 != 0 || rotary_dim % 16 != 0 || block_size % 16 != 0 || num_axes > kMaxAxes ||
        head_dim > 1024 || num_heads > 65535)
        return PKV_ERR_UNSUPPORTED;
    RotaryParams p{};
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
    const bool fp8 = cache_dtype == PKV_E4M3;
    if (fp8) {
        if (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
            return PKV_ERR_INVALID_ARG;
    } else if (k_scale != 1.f || v_scale != 1.f) {
        return PKV_ERR_INVALID_ARG;
    }
    if (!((src_dtype == PKV_F32 || src_dtype == PKV_BF16) && (fp8 || cache_dtype == src_dtype)))
        return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
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
    p.k_scale = k_scale;
    p.v_scale = v_scale;
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
