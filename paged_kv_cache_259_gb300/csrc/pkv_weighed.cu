// C ABI entry point of decode attention with token weights: argument checks and dispatch.
#include <cmath>

#include "pkv_check.cuh"
#include "pkv_weighed_impl.cuh"

namespace pkv {
namespace weighed {
int dispatch_f32(const Args& a);
int dispatch_bf16(const Args& a);
int dispatch_e4m3(const Args& a);
}  // namespace weighed
}  // namespace pkv

extern "C" size_t weighed_decode_workspace_size(int num_seqs, int num_heads, int head_dim, int block_size,
                                                int max_blocks_per_seq) {
    using namespace pkv::weighed;
    if (num_seqs <= 0 || num_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 ||
        max_blocks_per_seq > (0x7fffffff - 31) / block_size)
        return 0;
    // logits; at most kMaxCtas + (sequences x kv heads) partitions of at most 8 heads each
    const size_t heads = (size_t)num_seqs * num_heads;
    return 4 * (heads * logits_pitch(max_blocks_per_seq, block_size) + (8 * (size_t)kMaxCtas + heads) * (head_dim + 2));
}

extern "C" int paged_attention_decode_weighed(
    void* out, float* token_weights, const int32_t* weight_rows, const void* q, const void* k_pool,
    const void* v_pool, const int32_t* block_tables, const int32_t* seq_lens, int num_seqs, int max_blocks_per_seq,
    int num_blocks, int num_rows, int max_tokens, int num_heads, int num_kv_heads, int head_dim, int block_size,
    float scale, float decay, int q_dtype, int kv_dtype, float k_scale, float v_scale, void* workspace,
    size_t workspace_bytes, void* stream) {
    using namespace pkv;
    if (num_seqs < 0 || num_seqs > 65535 || max_blocks_per_seq <= 0 || num_blocks <= 0 || num_rows <= 0 ||
        num_heads <= 0 || num_kv_heads <= 0 || num_kv_heads > 65535 || head_dim <= 0 || block_size <= 0 ||
        max_blocks_per_seq > (0x7fffffff - 31) / block_size)
        return PKV_ERR_INVALID_ARG;
    if (num_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    if (max_tokens < max_blocks_per_seq * block_size || max_tokens % 4 != 0 || (!weight_rows && num_rows < num_seqs))
        return PKV_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !std::isfinite(k_scale) || !std::isfinite(v_scale) || !(k_scale > 0.f) ||
        !(v_scale > 0.f) || !(decay >= 0.f) || !(decay <= 1.f))
        return PKV_ERR_INVALID_ARG;
    if (kv_dtype != PKV_E4M3 && (k_scale != 1.f || v_scale != 1.f)) return PKV_ERR_INVALID_ARG;
    const int G = num_heads / num_kv_heads;
    if ((head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32) ||
        (G != 1 && G != 2 && G != 4 && G != 8))
        return PKV_ERR_UNSUPPORTED;
    const bool f32 = q_dtype == PKV_F32 && kv_dtype == PKV_F32;
    const bool bf16 = q_dtype == PKV_BF16 && kv_dtype == PKV_BF16;
    const bool e4m3 = q_dtype == PKV_BF16 && kv_dtype == PKV_E4M3;
    if (!f32 && !bf16 && !e4m3) return PKV_ERR_UNSUPPORTED;
    if ((long long)num_seqs * num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;   // the grid's y
    if (num_seqs == 0) return PKV_OK;
    if (!out || !token_weights || !q || !k_pool || !v_pool || !block_tables || !seq_lens || !workspace)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(q) || !aligned16(out) || !aligned16(token_weights) ||
        !aligned16(workspace) ||
        workspace_bytes < weighed_decode_workspace_size(num_seqs, num_heads, head_dim, block_size, max_blocks_per_seq))
        return PKV_ERR_INVALID_ARG;
    if (checking()) return PKV_OK;
    weighed::Args a{};
    a.p.out = out;
    a.p.weights = token_weights;
    a.p.rows = weight_rows;
    a.p.q = q;
    a.p.k_pool = static_cast<const char*>(k_pool);
    a.p.v_pool = static_cast<const char*>(v_pool);
    a.p.block_tables = block_tables;
    a.p.seq_lens = seq_lens;
    a.p.max_blocks = max_blocks_per_seq;
    a.p.num_blocks = num_blocks;
    a.p.num_rows = num_rows;
    a.p.max_tokens = max_tokens;
    a.p.num_kv_heads = num_kv_heads;
    a.p.pitch = weighed::logits_pitch(max_blocks_per_seq, block_size);
    a.p.v_scale = v_scale;
    a.p.decay = decay;
    a.num_seqs = num_seqs;
    a.num_heads = num_heads;
    a.head_dim = head_dim;
    a.block_size = block_size;
    a.scale = scale;
    a.k_scale = k_scale;
    a.workspace = workspace;
    a.stream = static_cast<cudaStream_t>(stream);
    a.p.err = error_word();
    if (!a.p.err) return PKV_ERR_CUDA;
    try {
        if (f32) return weighed::dispatch_f32(a);
        return bf16 ? weighed::dispatch_bf16(a) : weighed::dispatch_e4m3(a);
    } catch (...) {                                         // the per-kernel records' host memory
        return cuda_fail("weighed decode: host memory", cudaErrorMemoryAllocation);
    }
}
