// Attention over the INT4 KV cache (gfx950): the walk of wq_kv_walk.h where a
// sequence's queries are its last tokens, one after another.
#include "wq_kv_walk.h"

namespace wq {

size_t kv_attn_workspace_bytes(int B, int Hq, int Hkv, int D, int64_t max_context, int64_t max_queries) {
  const KvPlan p = plan_kv(B, Hq, Hkv, D, max_context, max_queries, false);
  return walk_workspace_bytes(p, D);
}

int describe_kv_attn(int B, int Hq, int Hkv, int D, int page, int64_t max_context, int64_t max_queries, char* buf,
                     size_t len) {
  const KvPlan p = plan_kv(B, Hq, Hkv, D, max_context, max_queries, false);
  if (p.chunk)
    return snprintf(buf, len, "kv_chunk_kernel<D=%d, HP=%d, RT=%d> grid=%lld block=%d whole units", D, p.HP,
                    p.RT, (long long)p.grid, 64 * kChunkWaves);
  return describe_walk(p, D, page, buf, len);
}

hipError_t launch_kv_attn(const KvAttnArgs& a, hipStream_t stream) {
  const KvPlan p = plan_kv(a.B, a.Hq, a.Hkv, a.D, a.max_context, a.max_queries, false);
  return p.chunk ? launch_kv_chunk(a, p.grid, p.rtiles, stream) : launch_walk<false>(a, p, stream);
}

}  // namespace wq
