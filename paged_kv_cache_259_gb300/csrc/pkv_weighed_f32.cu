// Decode with token weights instantiated for one (query dtype, cache dtype) pair; one
// translation unit per pair so the library builds in parallel.
#include "pkv_weighed_impl.cuh"

namespace pkv {
namespace weighed {
int dispatch_f32(const Args& a) { return dispatch<float, float>(a); }
}  // namespace weighed
}  // namespace pkv
