// C ABI entry point of sparse decode attention: argument checks and dispatch.
#include <cmath>
#include <map>
#include <mutex>
#include <tuple>

#include "pkv_check.cuh"
#include "pkv_sparse_impl.cuh"

namespace pkv {
namespace sparse {
int dispatch_f32(const Args& a);
int dispatch_bf16(const Args& a);
int dispatch_e4m3(const Args& a);

int resident_clusters(const void* kern, int smem, int threads, int size, int* out) {
    static std::mutex mu;
    // (device, kernel, shared memory, threads, size) -> clusters
    static std::map<std::tuple<int, const void*, int, int, int>, int> known;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail("sparse decode: current device", e);
    std::lock_guard<std::mutex> lock(mu);
    auto it = known.find({dev, kern, smem, threads, size});
    if (it == known.end()) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(size);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = size;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        if (e != cudaSuccess) return cuda_fail("sparse decode: cluster occupancy", e);
        it = known.insert({{dev, kern, smem, threads, size}, n}).first;
    }
    *out = it->second;
    return PKV_OK;
}
}  // namespace sparse
}  // namespace pkv

extern "C" int paged_attention_decode_sparse(
    void* out, const void* q, const void* k_pool, const void* v_pool, const int32_t* block_tables,
    const int32_t* seq_lens, const int32_t* selected, int num_seqs, int max_blocks_per_seq,
    int num_blocks, int num_selected, int num_heads, int num_kv_heads, int head_dim, int block_size,
    float scale, int q_dtype, int kv_dtype, float k_scale, float v_scale, void* stream) {
    using namespace pkv;
    if (num_seqs < 0 || num_seqs > 65535 || max_blocks_per_seq <= 0 || num_blocks <= 0 ||
        num_selected <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_kv_heads > 65535 ||
        head_dim <= 0 || block_size <= 0 || max_blocks_per_seq > 0x7fffffff / block_size)
        return PKV_ERR_INVALID_ARG;
    if (num_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !std::isfinite(k_scale) || !std::isfinite(v_scale) ||
        !(k_scale > 0.f) || !(v_scale > 0.f))
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
    if (num_seqs == 0) return PKV_OK;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !seq_lens || !selected)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(q) || !aligned16(out))
        return PKV_ERR_INVALID_ARG;
    if (checking()) return PKV_OK;
    sparse::Args a{};
    a.p.out = out;
    a.p.q = q;
    a.p.k_pool = static_cast<const char*>(k_pool);
    a.p.v_pool = static_cast<const char*>(v_pool);
    a.p.block_tables = block_tables;
    a.p.seq_lens = seq_lens;
    a.p.selected = selected;
    a.p.max_blocks = max_blocks_per_seq;
    a.p.num_blocks = num_blocks;
    a.p.num_heads = num_heads;
    a.p.num_kv_heads = num_kv_heads;
    a.p.k = num_selected;
    a.num_seqs = num_seqs;
    a.head_dim = head_dim;
    a.block_size = block_size;
    a.scale = scale;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.stream = static_cast<cudaStream_t>(stream);
    a.p.err = error_word();
    if (!a.p.err) return PKV_ERR_CUDA;
    try {
        if (f32) return sparse::dispatch_f32(a);
        return bf16 ? sparse::dispatch_bf16(a) : sparse::dispatch_e4m3(a);
    } catch (...) {                                         // the per-kernel records' host memory
        return cuda_fail("sparse decode: host memory", cudaErrorMemoryAllocation);
    }
}
