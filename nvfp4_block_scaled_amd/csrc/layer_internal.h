// layer_internal.h -- host-side launch functions of a decoder layer's other
// operators: the norm that encodes its output (mx_norm.hip).  Apart from
// nvfp4_internal.h, as kv_internal.h is.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

struct MxNorm {
  const void *x, *residual, *weight;  // residual and weight may be null
  void *sum, *normed;                 // may be null
  uint8_t *codes, *scales;
  int64_t rows, k;                    // k % 32 == 0
  double eps;
  bool packed;                        // codes and scales in the operand layout of mx_codec.hip
};
// bits: 4 (mxfp4) or 8 (mxfp8); fewer than 2^31 - 64 rows, k below 2^31
hipError_t launch_mx_norm(const MxNorm& n, int dt, int bits, hipStream_t s);

}  // namespace nvfp4
