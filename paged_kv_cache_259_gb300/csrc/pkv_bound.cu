// pkv_bound_call: the calls with packed arguments. The number of arguments and their
// types come from the entry points' own declarations.
#include <cstring>
#include <utility>

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

}  // namespace
}  // namespace pkv

extern "C" int pkv_bound_call(int call, const uint64_t* args, int num_args, void* stream) {
    using namespace pkv;
    if (!args) return PKV_ERR_INVALID_ARG;
    switch (call) {
        case PKV_CALL_ROTARY_AND_CACHE: return call_packed(&rotary_and_cache, args, num_args, stream);
        case PKV_CALL_UPDATE_KEY_BOUNDS: return call_packed(&update_key_bounds, args, num_args, stream);
        case PKV_CALL_SELECT_BLOCKS: return call_packed(&select_blocks, args, num_args, stream);
        case PKV_CALL_DECODE_SPARSE: return call_packed(&paged_attention_decode_sparse, args, num_args, stream);
        default: return PKV_ERR_INVALID_ARG;
    }
}
