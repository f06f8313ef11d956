// What the two tree attention kernels (decode_tree.cu, decode_tree_tc.cu) share.
#pragma once

#include "rswa_device.cuh"

namespace rswa {

// Live nodes of sequence b; a count outside 0..nodes is flagged and clamped.
__device__ __forceinline__ int live_nodes(const int32_t* counts, int b, int nodes,
                                          int32_t* err) {
  if (!counts) return nodes;
  const int c = counts[b];
  if (c < 0 || c > nodes) flag_error(err, kErrBadTree);
  return min(max(c, 0), nodes);
}

}  // namespace rswa
