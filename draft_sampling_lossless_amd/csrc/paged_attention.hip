// Paged attention over all of a request's keys, or those up to each row's own place.
#include "paged.hpp"

namespace dspark {

size_t paged_attention_workspace_bytes(int T, int B, int max_q, int nh, int nkv, int hd) {
  (void)T;
  return shape_of(B, max_q, nh, nkv, hd).bytes;
}

hipError_t launch_paged_attention(const PagedArgs& a, int hd, void* workspace, hipStream_t stream) {
  return launch_seen<kBlock>(a, hd, workspace, stream);
}

}  // namespace dspark
