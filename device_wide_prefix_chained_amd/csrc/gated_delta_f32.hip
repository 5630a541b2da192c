// gated_delta_f32.hip -- the gated delta rule over packed sequences of f32.
#include <hip/hip_runtime.h>

#include "delta_walk.hpp"

namespace dwps {
template ps_status delta_forward<float>(void *, size_t *, const ps_delta_input *, void *, float *, float *, hipStream_t);
}
