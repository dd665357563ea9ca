// The tcgen05 kernel of pbs_tree_attn (tree_tc.cu): row tiles of 128 or 256.
#pragma once

#include "tree.cuh"

namespace pbs {

cudaError_t launch_tree_tc(const CUtensorMap &mk, const CUtensorMap &mv, const tree::TreeArgs &a,
                           int d, int rows, bool bf16, int grid, cudaStream_t st);

}  // namespace pbs
