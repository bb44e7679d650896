// sqllm_rows.h -- the quantiser to 8-bit integers, for the calls that round
// their activations inside (defined in sqllm_norm.hip beside the norm, whose
// rows it shares).
#ifndef SQLLM_ROWS_H
#define SQLLM_ROWS_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

namespace sqllm {

// Arguments as checked by sqllm_int8_quantize.
hipError_t launch_int8_quantize(const uint16_t *x, int64_t rows, int64_t cols, int64_t ldx, int8_t *q, float *scale,
                                hipStream_t stream);

} // namespace sqllm

#endif
