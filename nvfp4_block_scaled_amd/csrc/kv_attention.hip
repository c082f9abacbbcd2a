// kv_attention.hip -- attention over an NVFP4 cache: the instances of
// kv_attention.h for queries at consecutive positions, and the workspace.
#include "kv_attention.h"

namespace nvfp4 {

size_t kv_attention_workspace(const KvCache& c, const KvAttention& a) { return attention_workspace<false>(c, a); }

hipError_t launch_kv_attention(const KvCache& c, const KvAttention& a, int dt, void* workspace, hipStream_t s) {
  return launch_attention<false>(c, a, dt, workspace, s);
}

}  // namespace nvfp4
