// gated_delta_bwd_f16.hip -- gradients of the gated delta rule over packed
// sequences of f16.
#include <hip/hip_runtime.h>

#include "delta_back.hpp"

namespace dwps {
template ps_status delta_backward<f16_t>(void *, size_t *, const ps_delta_input *, const void *, const float *, const float *,
                                      const ps_delta_grads *, hipStream_t);
}
