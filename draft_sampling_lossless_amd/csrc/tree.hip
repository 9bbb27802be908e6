// A drafted tree's parents to masks and positions.
//
//   m_j = {j} + m_{parent j},   position_j = context + |m_j| - 1
//
// One workgroup per request, one thread per node.  Every node holds the set it has gathered and
// the ancestor to gather from next; a round joins both with that ancestor's, so that ancestors
// 1, 2, 4, .. up are reached and log2(depth) rounds do.  24 bytes a node: a launch's time, 2.6 us
// for one tree of 25 nodes, 5.7 for 512 trees of up to 128.
#include "attention.hpp"
#include "kernels.hpp"

namespace dspark {

namespace {

constexpr int kNodes = 128;

__global__ __launch_bounds__(kNodes) void tree_mask_rows(TreeArgs a) {
  __shared__ uint4 sets[kNodes];
  __shared__ int ups[kNodes];
  const int b = blockIdx.x, j = threadIdx.x;
  const int q0 = clampi(a.cu_q[b], 0, a.T), n = clampi(a.cu_q[b + 1], q0, a.T) - q0;
  const bool ok = j < min(n, a.max_q);
  int up = ok ? a.parent[q0 + j] : -1;
  if (up >= j) up = -1;                           // (a parent that does not come before its child: a root)
  uint4 set = make_uint4(0, 0, 0, 0);
  (j < 64 ? j < 32 ? set.x : set.y : j < 96 ? set.z : set.w) = 1u << (j & 31);
  while (true) {
    sets[j] = set;
    ups[j] = up;
    if (!__syncthreads_or(up >= 0)) break;
    if (up >= 0) {
      const uint4 s = sets[up];
      set = make_uint4(set.x | s.x, set.y | s.y, set.z | s.z, set.w | s.w);
      up = ups[up];
    }
    __syncthreads();
  }
  if (!ok) return;
  reinterpret_cast<uint4*>(a.mask)[q0 + j] = set;
  if (a.positions) a.positions[q0 + j] = a.kv_len[b] - n + __popc(set.x) + __popc(set.y) + __popc(set.z) + __popc(set.w) - 1;
}

}  // namespace

hipError_t launch_tree_mask(const TreeArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(tree_mask_rows, dim3(a.B), dim3(a.max_q <= 64 ? 64 : kNodes), 0, stream, a);
  return hipGetLastError();
}

}  // namespace dspark
