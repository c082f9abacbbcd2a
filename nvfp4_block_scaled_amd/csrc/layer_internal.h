// layer_internal.h -- host-side launch functions of a decoder layer's other
// operators: the norm that encodes its output (mx_norm.hip) and the rotation on
// the way into the cache (kv_rotate.hip).  Apart from nvfp4_internal.h, as
// kv_internal.h is.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv_internal.h"

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

struct KvRotate {
  const void *k, *v, *q;  // q may be null with query_heads 0
  void* q_out;            // [tokens, query_heads, dim]
  int64_t tokens;         // below 2^26
  int64_t k_token, k_head, v_token, v_head, q_token, q_head;  // strides in elements
  const int64_t* slots;
  const int32_t* positions;
  const float* table;     // [table_rows, rotary]: rotary / 2 cosines, then the sines
  int64_t table_rows;
  int rotary, interleaved, query_heads;
  int turns;              // set by the launch: heads of a wave's run, and the division by pieces of a head
  KvDiv piece_div;
};
hipError_t launch_kv_rotate(const KvCache& c, KvRotate a, int dt, hipStream_t s);

}  // namespace nvfp4
