// The edge's backward with a LayerNorm on either side (block_edge_bwd.h).

#include "block_edge_bwd.h"

namespace tpmlp {

hipError_t launch_edge_bwd_layer(const EdgeBwdArgs& a, int64_t blocks, int y_type, int r_type, bool full, hipStream_t s) {
  return edge::launch_types<true>(a, blocks, y_type, r_type, full, s);
}

}  // namespace tpmlp
