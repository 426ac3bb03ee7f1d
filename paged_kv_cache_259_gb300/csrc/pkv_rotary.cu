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
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cmath>
#include <type_traits>

#include "pkv_check.cuh"
#include "pkv_internal.cuh"

namespace pkv {
namespace {

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
__device__ __noinline__ float divide(float x, float y) { return __fdiv_rn(x, y); }   // rare: kept out of the way
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
    if (live && turns) {
        const int i0 = 8 * u;
        int a = 0;
        while (i0 >= p.section_end[a]) ++a;
        auto row_of = [&](int axis) {
            int x = token.pos[0];
#pragma unroll
            for (int k = 1; k < kMaxAxes; ++k) x = axis == k ? token.pos[k] : x;
            return p.cos_sin + (long long)x * p.rot;
        };
        if (i0 + 7 < p.section_end[a]) {                   // one axis for all 8 pairs
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
    auto scale_of = [](float s) { return Scale{s, s > 0x1p-100f && s < 0x1p100f ? 1.f / s : 0.f}; };
    p.k_scale = scale_of(k_scale);
    p.v_scale = scale_of(v_scale);
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
