// What the rotated appends share (rotary_and_cache, norm_rotary_and_cache): the launch's
// parameters, rows as loaded, the E4M3 codes, the stores into the pools' tiles, a token's
// slot and positions, and the V half, which both write alike.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cmath>
#include <type_traits>

#include "pkv_check.cuh"
#include "pkv_internal.cuh"

namespace pkv {
namespace rotary {

constexpr int kMaxAxes = 4;
constexpr int kThreads = 128;
// Heads a warp reads at a time, and the CTAs of an SM the registers are shared by.
// float32 rows take twice the registers: 34 us for 4096 tokens of 32 + 2 x 8 heads
// of 128 dims, against 46 us with the 16-bit choice; bf16, 8192 tokens: 35 us
// against 38 us the other way round.
template <typename ST> struct Batching {
    static constexpr int kHeads = 2, kCtas = 6;
};
template <> struct Batching<float> {
    static constexpr int kHeads = 1, kCtas = 8;
};

// A cache's scale: what E4M3 codes are x / value of. `inv`: 1 / value, or 0 where that
// is not a normal number.
struct Scale {
    float value, inv;
};

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
    // a warp's share: q_step q heads, or kv_step k or v heads (kv_chunks of each), of
    // one of `cols` groups of 64 columns; chunks: of all heads together
    int q_step, kv_step, kv_chunks, chunks, cols;
    Scale k_scale, v_scale;
    int* err;
};

// 8 consecutive elements as loaded, and as floats
template <typename T> struct Raw8;
template <> struct Raw8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const uint4*>(p);
        b = *reinterpret_cast<const uint4*>(p + 4);
    }
    __device__ __forceinline__ void clear() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void floats(float (&f)[8]) const {
        f[0] = __uint_as_float(a.x), f[1] = __uint_as_float(a.y);
        f[2] = __uint_as_float(a.z), f[3] = __uint_as_float(a.w);
        f[4] = __uint_as_float(b.x), f[5] = __uint_as_float(b.y);
        f[6] = __uint_as_float(b.z), f[7] = __uint_as_float(b.w);
    }
};
template <> struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void clear() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void floats(float (&f)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    Raw8<float> r;
    r.load(p);
    r.floats(f);
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
// x / scale to where its E4M3 code is that of the IEEE quotient. x * (1 / scale) is
// off by at most 2^-23 of itself (two roundings), less than 3 of the float32's last
// places; the code changes at the midpoints of 3-bit mantissas (the lower 20 bits
// 0x80000) and, below 2^-6, at the odd multiples of 2^-10. Only a product next to
// one of those is divided.
static __device__ __noinline__ float divide(float x, float y) { return __fdiv_rn(x, y); }   // rare: kept out of the way
__device__ __forceinline__ float e4m3_quotient(float x, const Scale& s) {
    float q = x * s.inv;
    const uint32_t near = (__float_as_uint(q) & 0xfffffu) - 0x7fffcu;
    const bool small = fabsf(q) < 0x1p-6f;
    if (near <= 8u || small || s.inv == 0.f) {
        const float y = q * 512.f;                         // steps of the subnormal codes
        if (!small || s.inv == 0.f || fabsf(y - rintf(y)) > 0.5f - 0x1p-19f) q = divide(x, s.value);
    }
    return q;
}
// E4M3 codes of two values over the scale: nearest even, saturating
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi, const Scale& s) {
    return __nv_cvt_float2_to_fp8x2(make_float2(e4m3_quotient(lo, s), e4m3_quotient(hi, s)), __NV_SATFINITE,
                                    __NV_E4M3);
}

// 8 dims d0 .. d0+7 (d0 a multiple of 8) of slot `off` of a K tile.
// CT = uint8_t: cache bytes are E4M3 codes.
template <typename CT>
__device__ __forceinline__ void store_k8(CT* tile, int d, int d0, int off, const float (&f)[8],
                                         const Scale& scale) {
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

// The token's slot and positions, checked once the first rows are on their way: a
// bad one is flagged and the token skipped whole (slot -1).
struct Token {
    long long slot = -1;
    int pos[kMaxAxes];

    __device__ __forceinline__ void read(const RotaryParams& p, long long t) {
        slot = p.slots[t];
#pragma unroll
        for (int a = 0; a < kMaxAxes; ++a)
            if (a < p.axes) pos[a] = p.positions[(long long)a * p.num_tokens + t];
    }
    __device__ __forceinline__ void check(const RotaryParams& p) {
        if (slot < 0) return;
        bool bad = slot >= (long long)p.num_blocks * p.bs;
#pragma unroll
        for (int a = 0; a < kMaxAxes; ++a)
            if (a < p.axes) bad |= pos[a] < 0 || pos[a] >= p.num_positions;
        if (bad) {
            flag_error(p.err, kErrOutOfRange);
            slot = -1;
        }
    }
};

// Cosines and sines of the pairs 8u .. 8u+7 at the token's positions
__device__ __forceinline__ void load_turns(const RotaryParams& p, const Token& token, int u, float (&cs)[8],
                                           float (&sn)[8]) {
    const int i0 = 8 * u, half = p.rot >> 1;
    int a = 0;
    while (i0 >= p.section_end[a]) ++a;
    auto row_of = [&](int axis) {
        int x = token.pos[0];
#pragma unroll
        for (int k = 1; k < kMaxAxes; ++k) x = axis == k ? token.pos[k] : x;
        return p.cos_sin + (long long)x * p.rot;
    };
    if (i0 + 7 < p.section_end[a]) {                       // one axis for all 8 pairs
        const float* row = row_of(a) + i0;
        load8(row, cs);
        load8(row + half, sn);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            while (i0 + j >= p.section_end[a]) ++a;
            const float* row = row_of(a) + i0 + j;
            cs[j] = row[0];
            sn[j] = row[half];
        }
    }
}

// A unit's two chunks of 8 dims, turned
template <bool INTERLEAVED>
__device__ __forceinline__ void turn16(float (&x)[8], float (&y)[8], const float (&cs)[8], const float (&sn)[8]) {
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

// What a V row element is while it is turned: 16 bits (a bf16, or an E4M3 code) or
// 32 (float32).
template <typename CT>
struct Turn {
    static constexpr int kBytes = sizeof(CT) == 4 ? 4 : 2;
    static constexpr int kPitch = 64 * kBytes + 16;        // bytes of a token's 64 dims, off the banks
    static constexpr int kWarp = 8 * kPitch;               // of a warp's 8 tokens
};

// 8 elements into a row of the turning buffer
template <typename CT>
__device__ __forceinline__ void put8(unsigned char* dst, const float (&f)[8], const Scale& scale) {
    if constexpr (sizeof(CT) == 4) {
        store8(reinterpret_cast<float*>(dst), f);
    } else if constexpr (sizeof(CT) == 2) {
        store8(reinterpret_cast<__nv_bfloat16*>(dst), f);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t two = e4m3_pair(f[2 * i], f[2 * i + 1], scale);
            w[i] = (two & 0xffu) | ((two & 0xff00u) << 8);
        }
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// v heads: 8 tokens x 64 dims, turned through shared memory (ldmatrix.trans): lane
// 4r + c then holds tokens 2c, 2c+1 of dim 8j + r for j = 0 .. 7, and a store of the
// warp is 8 dims x 8 tokens, one 128-byte core matrix of a bf16 tile. Slots that
// follow one another from an odd one leave every pair astride two words: two stores.
template <typename ST, typename CT>
__device__ __forceinline__ void write_v_heads(const RotaryParams& p, long long tg, int cg, int h, int h_end,
                                              unsigned char* buf) {
    constexpr int HB = Batching<ST>::kHeads, X = 16 / sizeof(CT);
    using TN = Turn<CT>;
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const long long t = tg * 8 + r;
    const int d = p.d, u = cg * 4 + c;
    const bool has = t < p.num_tokens && 16 * u < d;
    const long long tile_elems = (long long)d * p.bs, pitch = (long long)d * X;
    Token token;
    if (t < p.num_tokens) token.read(p, t);
    const ST* src = static_cast<const ST*>(p.v) + t * p.v_stride + (long long)h * d + 16 * u;
    struct Batch {
        Raw8<ST> a[HB], b[HB];
    };
    auto read = [&](Batch& x, int left) {
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            x.a[i].clear();
            x.b[i].clear();
            if (has && i < left) {
                x.a[i].load(src + i * d);
                x.b[i].load(src + i * d + 8);
            }
        }
        src += HB * d;
    };
    int left = h_end - h;
    Batch now, next;
    read(now, left);
    token.check(p);
    __syncwarp();
    const long long slot = token.slot, blk = slot >= 0 ? slot / p.bs : 0;
    const int off = slot >= 0 ? (int)(slot - blk * p.bs) : 0;
    // this token's column of its block's tile (dim 0, head 0), -1: none
    const long long column = slot >= 0 ? blk * p.hkv * tile_elems + (long long)(off / X) * pitch + off % X : -1;
    const int groups = min(8, d / 8 - 8 * cg);             // of 8 dims
    const long long row0 = (long long)h * tile_elems + cg * 64 * X + r * X;   // group j: 8 X j further
    const long long c0 = __shfl_sync(0xffffffffu, column, 8 * c), c1 = __shfl_sync(0xffffffffu, column, 8 * c + 4);
    const long long s_even = __shfl_sync(0xffffffffu, slot, 8 * c), s_odd = __shfl_sync(0xffffffffu, slot, 8 * c + 4);
    const bool ok0 = c0 >= 0, ok1 = c1 >= 0;
    const bool both = ok0 && s_odd == s_even + 1 && (s_even & 1) == 0;   // one block: block sizes are even
    CT* d0 = static_cast<CT*>(p.v_pool) + (ok0 ? c0 : 0) + row0;
    CT* d1 = static_cast<CT*>(p.v_pool) + (ok1 ? c1 : 0) + row0;
    unsigned char* const mine = buf + r * TN::kPitch + c * 16 * TN::kBytes;
    auto write = [&](const Batch& batch) {
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            if (i >= left) break;                          // the whole warp
            float f[8];
            batch.a[i].floats(f);
            put8<CT>(mine, f, p.v_scale);
            batch.b[i].floats(f);
            put8<CT>(mine + 8 * TN::kBytes, f, p.v_scale);
            __syncwarp();
            uint32_t lo[8], hi[8];                         // tokens 2c, 2c+1 (float32: one each)
            if constexpr (sizeof(CT) == 4) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    lo[j] = *reinterpret_cast<const uint32_t*>(buf + 2 * c * TN::kPitch + (8 * j + r) * 4);
                    hi[j] = *reinterpret_cast<const uint32_t*>(buf + (2 * c + 1) * TN::kPitch + (8 * j + r) * 4);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(lo[4 * k]), "=r"(lo[4 * k + 1]), "=r"(lo[4 * k + 2]), "=r"(lo[4 * k + 3])
                                 : "r"(smem_addr(buf + (lane & 7) * TN::kPitch + (4 * k + (lane >> 3)) * 16))
                                 : "memory");
            }
            __syncwarp();
            if constexpr (sizeof(CT) == 1) {
#pragma unroll
                for (int j = 0; j < 8; ++j) lo[j] = (lo[j] & 0xffu) | ((lo[j] >> 8) & 0xff00u);
            }
            const long long head = (long long)i * tile_elems;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j >= groups) break;
                const int row = 8 * X * j;
                if constexpr (sizeof(CT) == 4) {
                    if (both) {
                        *reinterpret_cast<uint2*>(d0 + head + row) = make_uint2(lo[j], hi[j]);
                    } else {
                        if (ok0) d0[head + row] = __uint_as_float(lo[j]);
                        if (ok1) d1[head + row] = __uint_as_float(hi[j]);
                    }
                } else if constexpr (sizeof(CT) == 1) {
                    if (both) {
                        *reinterpret_cast<uint16_t*>(d0 + head + row) = (uint16_t)lo[j];
                    } else {
                        if (ok0) d0[head + row] = (uint8_t)lo[j];
                        if (ok1) d1[head + row] = (uint8_t)(lo[j] >> 8);
                    }
                } else {
                    if (both) {
                        *reinterpret_cast<uint32_t*>(d0 + head + row) = lo[j];
                    } else {
                        if (ok0) reinterpret_cast<uint16_t*>(d0 + head)[row] = (uint16_t)lo[j];
                        if (ok1) reinterpret_cast<uint16_t*>(d1 + head)[row] = (uint16_t)(lo[j] >> 16);
                    }
                }
            }
        }
        left -= HB;
        d0 += HB * tile_elems;
        d1 += HB * tile_elems;
    };
#pragma unroll 1
    while (left > 0) {
        read(next, left - HB);
        write(now);
        now = next;
    }
}

// The checks of a rotated append's arguments, and its parameters (all but the launch's own and
// `err`). *done: nothing to do, the call returns at once.
int rotary_params(RotaryParams& p, bool* done, void* q_out, const void* q, const void* k, const void* v, void* k_pool,
                  void* v_pool, const int64_t* slot_mapping, const int32_t* positions, const float* cos_sin,
                  const int32_t* sections, int num_axes, int64_t q_out_stride, int64_t q_stride, int64_t k_stride,
                  int64_t v_stride, int num_tokens, int num_heads, int num_kv_heads, int head_dim, int rotary_dim,
                  int block_size, int num_blocks, int num_positions, int src_dtype, int cache_dtype, float k_scale,
                  float v_scale);

}  // namespace rotary
}  // namespace pkv
