// Paged attention of drafted trees: a node sees the context before the tree and the nodes that
// its mask names.
#include "paged.hpp"

namespace dspark {

hipError_t launch_tree_attention(const PagedArgs& a, int hd, void* workspace, hipStream_t stream) {
  return launch_seen<kTree>(a, hd, workspace, stream);
}

}  // namespace dspark
