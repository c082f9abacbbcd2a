// kv_internal.h -- host-side launch functions of the key/value cache's kernels
// (kv_cache.hip, kv_attention.hip) and the structs they take.  Apart from
// nvfp4_internal.h, which the other kernels include: bench.py's measured
// figures hold for the sources and headers that they were measured on.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

// The cache's layout is described in kv_device.h.
struct KvDiv {  // divisor and the constants of its division (kv_div)
  uint32_t d, mul, shift;
};
KvDiv kv_make_div(uint32_t d);
struct KvCache {
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  const float *global_k, *global_v;
  int pages, page_size, heads, dim;  // dim % 16 == 0, dim <= kKvMaxDim; pages * page_size < 2^31
  KvDiv page_div;
};
constexpr int kKvMaxDim = 256;
constexpr int kKvMaxKeys = INT32_MAX - 4095;  // of a context
// tokens * dim / 8 < 2^31 - 4096; strides in elements; fewer than 2^24 workgroups (check_kv_tokens)
hipError_t launch_kv_write(const KvCache& c, const void* k, const void* v, int dt, int64_t tokens,
                           int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head,
                           const int64_t* slots, hipStream_t s);
hipError_t launch_kv_read(const KvCache& c, const int64_t* slots, int64_t tokens, void* k, void* v, int dt,
                          hipStream_t s);
struct KvAttention {
  const void* q;
  int64_t q_token, q_head;      // strides in elements
  const int32_t* page_table;    // [seqs, table_stride]
  const int32_t* context_lens;  // [seqs]
  const int32_t* query_starts;  // [seqs + 1], or null: one query a sequence
  void* out;                    // [tokens, query_heads, dim]
  float* lse;                   // [tokens, query_heads] or null
  float scale;
  int seqs, query_heads, groups, max_queries, max_keys, causal, window;
  KvDiv group_div;              // by groups
  int64_t table_stride, tokens;
};
size_t kv_attention_workspace(const KvCache& c, const KvAttention& a);
hipError_t launch_kv_attention(const KvCache& c, const KvAttention& a, int dt, void* workspace, hipStream_t s);

}  // namespace nvfp4
