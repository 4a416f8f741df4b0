// Attention over the INT4 KV cache for many query rows (gfx950): the kernel of
// wq_kv_chunk.h where a sequence's queries are its last tokens, one after another.
#include "wq_kv_chunk.h"

namespace wq {

hipError_t launch_kv_chunk(const KvAttnArgs& a, int64_t grid, int rtiles, hipStream_t stream) {
  return a.D == 64 ? launch_one<64, false>(a, grid, rtiles, stream) : launch_one<128, false>(a, grid, rtiles, stream);
}

}  // namespace wq
