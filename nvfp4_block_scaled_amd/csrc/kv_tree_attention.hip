// kv_tree_attention.hip -- attention of drafted tokens that form a tree: the
// instances of kv_attention.h whose masks are given bit by bit.
#include "kv_attention.h"

namespace nvfp4 {

size_t kv_tree_attention_workspace(const KvCache& c, const KvAttention& a) { return attention_workspace<true>(c, a); }

hipError_t launch_kv_tree_attention(const KvCache& c, const KvAttention& a, int dt, void* workspace, hipStream_t s) {
  return launch_attention<true>(c, a, dt, workspace, s);
}

}  // namespace nvfp4
