#include "attn_tree_fp8_rows.cuh"

namespace attn {
namespace tree {
cudaError_t launch_rows_d64(const Params& p, int cols, int grid, cudaStream_t stream) {
  return launch_rows<64>(p, cols, grid, stream);
}
}  // namespace tree
}  // namespace attn
