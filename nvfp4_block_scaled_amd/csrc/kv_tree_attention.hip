// kv_tree_attention.hip -- attention of drafted tokens that form a tree: the
// instances of kv_attention.h whose masks are given bit by bit.
#include "kv_attention.h"

namespace nvfp4 {

// The kernels of trees count units in 32 bits, up to one more a workgroup than
// there are: these are bounded here, those of few rows with the sizes that both
// attention calls take.  (In 64 bits they would cost the runs' scalar registers, for
// calls that take tens of seconds.)
bool kv_tree_attention_fits(const KvCache& c, const KvAttention& a) {
  const int64_t rows = (int64_t)a.max_queries * a.groups;
  if (rows <= kFewRows) return true;
  const int64_t tiles = (int64_t)a.seqs * c.heads * ((rows + kManyRows - 1) / kManyRows);  // below 2^54
  return tiles <= ((int64_t)1 << 30) / (kv_most_keys(a) / kManyStep + 1);
}

size_t kv_tree_attention_workspace(const KvCache& c, const KvAttention& a) { return attention_workspace<true>(c, a); }

hipError_t launch_kv_tree_attention(const KvCache& c, const KvAttention& a, int dt, void* workspace, hipStream_t s) {
  return launch_attention<true>(c, a, dt, workspace, s);
}

}  // namespace nvfp4
