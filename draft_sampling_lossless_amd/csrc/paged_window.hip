// Paged attention under a window with sinks: of the keys that paged_attention.hip's rows see,
// the last `window` up to the row's own place, and the first `sinks`.
#include "paged.hpp"

namespace dspark {

hipError_t launch_paged_window(const PagedArgs& a, int hd, void* workspace, hipStream_t stream) {
  return launch_seen<kRecent>(a, hd, workspace, stream);
}

}  // namespace dspark
