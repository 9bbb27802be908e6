// Paged attention over all of a request's keys, or those up to each row's own place.
#include "paged.hpp"

namespace dspark {

size_t paged_attention_workspace_bytes(int T, int B, int max_q, int nh, int nkv, int hd) {
  (void)T;
  // (a tree's call has shapes of its own, by the keys that there may be)
  return std::max({shape_of<kBlock>(B, max_q, nh, nkv, hd, 0).bytes, shape_of<kTree>(B, max_q, nh, nkv, hd, 0).bytes,
                   shape_of<kTree>(B, max_q, nh, nkv, hd, (int64_t)1 << 40).bytes});
}

hipError_t launch_paged_attention(const PagedArgs& a, int hd, void* workspace, hipStream_t stream) {
  return launch_seen<kBlock>(a, hd, workspace, stream);
}

}  // namespace dspark
