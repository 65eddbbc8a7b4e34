// block_gemm_grouped_n.hip -- compiled kernels of the block-scaled product: groups of rows with a weight matrix each, B stored K x N.
#include "bst_block_instances.hpp"

namespace bst {

static const BlockGemmInstance kList[] = {BST_BLOCK_GEMM_TILES(false, true)};

BlockGemmList block_gemm_grouped_n() {
  return BlockGemmList{kList, (int)(sizeof(kList) / sizeof(kList[0]))};
}

}  // namespace bst
