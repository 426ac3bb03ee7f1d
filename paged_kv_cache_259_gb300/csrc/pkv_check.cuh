// Argument checks without the call (pkv_bound_check).
#pragma once

namespace pkv {

// True while pkv_bound_check runs a call on this thread: the call returns PKV_OK where
// its argument checks end, before any CUDA call.
bool checking();

}  // namespace pkv
