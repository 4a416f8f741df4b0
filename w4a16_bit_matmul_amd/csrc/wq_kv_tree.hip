// Attention over the INT4 KV cache for the nodes of a draft tree (gfx950).
//
// A sequence's n queries are the nodes of a tree whose keys and values are its
// last n cached tokens.  Node i sees the tokens before them and of the nodes those
// whose bit of its mask is set, its ancestors and itself as a rule:
//   out_i = sum_t p_t v_t / sum_t p_t over t < len - n and over nodes j with bit j.
// All but the last n tokens are seen by every row, so this is the walk of
// wq_kv_walk.h (and for many rows the kernel of wq_kv_chunk.h) with another mask:
// where a tile of 32 or 64 tokens reaches the nodes, each row's lanes read the
// window of its mask that falls on the tile, one or two 64-bit words from the
// cache, in place of a comparison of token numbers.
#include <stdio.h>

#include "wq_kv_chunk.h"
#include "wq_kv_walk.h"

namespace wq {

int describe_kv_tree(int B, int Hq, int Hkv, int D, int page, int64_t max_context, int64_t max_queries, char* buf,
                     size_t len) {
  const int n = describe_kv_attn(B, Hq, Hkv, D, page, max_context, max_queries, buf, len);
  if (n >= 0 && (size_t)n < len) snprintf(buf + n, len - n, ", tree masks");
  return n;
}

hipError_t launch_kv_tree(const KvAttnArgs& a, hipStream_t stream) {
  const KvPlan p = plan_kv(a.B, a.Hq, a.Hkv, a.D, a.max_context, a.max_queries);
  if (!p.chunk) return launch_walk<true>(a, p, stream);
  return a.D == 64 ? launch_one<64, true>(a, p.grid, p.rtiles, stream) : launch_one<128, true>(a, p.grid, p.rtiles, stream);
}

}  // namespace wq
