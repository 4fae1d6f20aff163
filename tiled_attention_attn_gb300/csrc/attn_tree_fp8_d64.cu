#include "attn_tree_fp8_kernel.cuh"

namespace attn {
namespace tree {
cudaError_t launch_d64(const Params& p, int cols, int grid, cudaStream_t stream) { return pick<64>(p, cols, grid, stream); }
}  // namespace tree
}  // namespace attn
