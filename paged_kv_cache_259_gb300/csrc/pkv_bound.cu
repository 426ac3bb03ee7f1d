// pkv_bound_call, pkv_bound_check: the calls with packed arguments. The number of arguments and their
// types come from the entry points' own declarations.
#include <cstring>
#include <utility>

#include "pkv_check.cuh"
#include "pkv_internal.cuh"

namespace pkv {
namespace {

template <typename T>
T unpack_arg(uint64_t slot) {
    if constexpr (std::is_pointer<T>::value) {
        return reinterpret_cast<T>(static_cast<uintptr_t>(slot));
    } else if constexpr (std::is_same<T, float>::value) {
        const uint32_t bits = static_cast<uint32_t>(slot);
        float f;
        std::memcpy(&f, &bits, sizeof(f));
        return f;
    } else {
        return static_cast<T>(slot);
    }
}

template <typename... A, size_t... I>
int invoke(int (*fn)(A...), const uint64_t* args, void* stream, std::index_sequence<I...>) {
    // the last argument is the stream
    const uint64_t all[sizeof...(A)] = {(I + 1 < sizeof...(A) ? args[I + 1 < sizeof...(A) ? I : 0]
                                                             : (uint64_t) reinterpret_cast<uintptr_t>(stream))...};
    return fn(unpack_arg<A>(all[I])...);
}

template <typename... A>
int call_packed(int (*fn)(A...), const uint64_t* args, int num_args, void* stream) {
    if (num_args != (int)sizeof...(A) - 1) return PKV_ERR_INVALID_ARG;
    return invoke(fn, args, stream, std::index_sequence_for<A...>{});
}

thread_local bool g_checking = false;

// paged_prefill_step finds every argument error of the attention, then of its own
// writes, before it launches anything. Asked for a token without keys it ends there with
// one status, for more pairs than it takes with another: both mean the attention's
// arguments are good, and any error of theirs comes back from both.
int check_prefill(void* out, const void* q, const void* k_pool, const void* v_pool, const int32_t* block_tables,
                  const int32_t* seq_lens, const int32_t* query_start, int num_seqs, int max_query_len,
                  int max_blocks_per_seq, int num_blocks, int num_heads, int num_kv_heads, int head_dim,
                  int block_size, float scale, int q_dtype, int kv_dtype, void* stream) {
    const int64_t pair[2] = {0, 0};
    if (num_seqs == 0 || max_query_len == 0) k_pool = v_pool = pair;   // nothing to attend: not looked at
    auto ask = [&](int num_pairs, int num_tokens) {
        return paged_prefill_step(pair, num_pairs, nullptr, nullptr, nullptr, num_tokens, out, q,
                                  const_cast<void*>(k_pool), const_cast<void*>(v_pool), block_tables, seq_lens,
                                  query_start, num_seqs, max_query_len, max_blocks_per_seq, num_blocks, num_heads,
                                  num_kv_heads, head_dim, block_size, scale, q_dtype, kv_dtype, stream);
    };
    const int no_keys = ask(0, 1), many_pairs = ask((1 << 30) + 1, 0);
    return no_keys == PKV_ERR_INVALID_ARG && many_pairs == PKV_ERR_UNSUPPORTED ? PKV_OK : no_keys;
}

}  // namespace

bool checking() { return g_checking; }

}  // namespace pkv

extern "C" int pkv_bound_check(int call, const uint64_t* args, int num_args) {
    pkv::g_checking = true;
    const int st = pkv_bound_call(call, args, num_args, nullptr);
    pkv::g_checking = false;
    return st;
}

extern "C" int pkv_bound_call(int call, const uint64_t* args, int num_args, void* stream) {
    using namespace pkv;
    if (!args) return PKV_ERR_INVALID_ARG;
    switch (call) {
        case PKV_CALL_ROTARY_AND_CACHE: return call_packed(&rotary_and_cache, args, num_args, stream);
        case PKV_CALL_UPDATE_KEY_BOUNDS: return call_packed(&update_key_bounds, args, num_args, stream);
        case PKV_CALL_SELECT_BLOCKS: return call_packed(&select_blocks, args, num_args, stream);
        case PKV_CALL_DECODE_SPARSE: return call_packed(&paged_attention_decode_sparse, args, num_args, stream);
        case PKV_CALL_PREFILL:
            return call_packed(checking() ? &check_prefill : &paged_attention_prefill, args, num_args, stream);
        case PKV_CALL_NORM_ROTARY_AND_CACHE: return call_packed(&norm_rotary_and_cache, args, num_args, stream);
        case PKV_CALL_DECODE_WEIGHED: return call_packed(&paged_attention_decode_weighed, args, num_args, stream);
        case PKV_CALL_WEIGH_PREFILL: return call_packed(&weigh_prefill_tokens, args, num_args, stream);
        case PKV_CALL_SELECT_TOKENS: return call_packed(&select_tokens, args, num_args, stream);
        case PKV_CALL_KEEP_TOKENS: return call_packed(&keep_tokens, args, num_args, stream);
        default: return PKV_ERR_INVALID_ARG;
    }
}
