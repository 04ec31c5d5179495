// What the files of the C ABI share: the public headers, the launch
// status and the norms' argument checks.
#pragma once

#include "../../include/moe_fp4.h"
#include "../../include/moe_fp8_block.h"
#include "../../include/moe_mx4.h"

namespace moe {

// Records a launch's result for moe_last_hip_error (0 on success).
moe_status_t hip_status(hipError_t e);

// The checks of moe_norm_before and moe_norm_after, for the callers that
// enqueue other work first.
moe_status_t check_norm_before(const void* x, int32_t x_type, const void* w, int32_t w_type, int32_t T, int32_t H,
                               float eps, const uint16_t* z, const uint8_t* q, const uint8_t* s, int32_t quant);
moe_status_t check_norm_after(const void* y, int32_t y_type, const void* residual, int32_t residual_type,
                              const void* w_post, const void* w_next, int32_t w_type, const float* gate,
                              int64_t gate_t, int64_t gate_h, float eps, int32_t T, int32_t H, const void* out,
                              const uint16_t* z, const uint8_t* q, const uint8_t* s, int32_t quant);

}  // namespace moe
