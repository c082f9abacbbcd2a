// kv_attention.hip -- attention over an NVFP4 cache: the instances of
// kv_attention.h for queries at consecutive positions, and the workspace.
#include "kv_attention.h"

namespace nvfp4 {

size_t kv_attention_workspace(const KvCache& c, const KvAttention& a) {
  const size_t one = kv_plan(c, a, 1).bytes, two = kv_plan(c, a, 2).bytes;
  return one > two ? one : two;
}

hipError_t launch_kv_attention(const KvCache& c, const KvAttention& a, int dt, void* workspace, hipStream_t s) {
  return launch_attention<false>(c, a, dt, workspace, s);
}

}  // namespace nvfp4
