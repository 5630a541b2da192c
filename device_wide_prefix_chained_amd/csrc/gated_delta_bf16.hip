// gated_delta_bf16.hip -- the gated delta rule over packed sequences of bf16.
#include <hip/hip_runtime.h>

#include "delta_walk.hpp"

namespace dwps {
template ps_status delta_forward<bf16_t>(void *, size_t *, const ps_delta_input *, void *, float *, float *, hipStream_t);
}
