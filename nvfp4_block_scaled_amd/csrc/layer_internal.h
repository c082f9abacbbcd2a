// layer_internal.h -- host-side launch functions of a decoder layer's other
// operators: the norm that encodes its output (mx_norm.hip), the rotation on the
// way into the cache (kv_rotate.hip) and the expert layer (moe.hip).  Apart from nvfp4_internal.h, as
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
// A launch has fewer than 2^24 workgroups of 256 threads, and 2^22 of the 1024 that
// take a row of more than kMxNormLong values; packed rows are rounded up to 256.
constexpr int kMxNormLong = 16384;
// bits: 4 (mxfp4) or 8 (mxfp8); fewer than 2^22 rows (packed ones of more than
// kMxNormLong values: at most 2^22 - 256), k at most 2^30
hipError_t launch_mx_norm(const MxNorm& n, int dt, int bits, hipStream_t s);

struct KvRotate {
  const void *k, *v, *q;  // q may be null with query_heads 0
  void* q_out;            // [tokens, query_heads, dim]
  int64_t tokens;         // at most 2^26 - 4
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

constexpr int kMoeMaxTokens = 64, kMoeMaxTopK = 32, kMoeMaxExperts = 1024;
constexpr int kMoeMaxPairs = kMoeMaxTokens * kMoeMaxTopK;
struct MoeLayer {
  const void *x, *router;  // [tokens, k], [experts, k]; router null: idx and weights are given
  int32_t* expert_idx;     // [tokens, top_k], with their weights
  float* expert_weights;
  const uint8_t *up_codes, *up_scales;      // [experts, 2 f, k]: gate rows, then up rows
  const uint8_t *down_codes, *down_scales;  // [experts, k, f]
  const float *up_global, *down_global;     // [experts] or null
  void* out;                                // [tokens, k]
  int tokens, top_k, experts, k, f, normalize;  // k and f multiples of 16, below 2^20
  // in the workspace, set by the launch
  double* logits;        // [tokens, experts]
  int* x_exponent;       // [tokens]: x_pieces times 2^this is x; null: float16 x is used as it lies
  uint32_t* h_top;       // [tokens * top_k]: bits of the largest |h|
  uint16_t* x_pieces;    // float16 [pieces][tokens, k]
  float* hidden;         // [tokens * top_k, f]
};
size_t moe_workspace(int64_t tokens, int64_t top_k, int64_t experts, int64_t k, int64_t f, int dt);
hipError_t launch_moe(MoeLayer a, int dt, void* workspace, hipStream_t s);

}  // namespace nvfp4
