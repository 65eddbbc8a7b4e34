// block_gemm_grouped_t.hip -- compiled kernels of the block-scaled product: groups of rows with a weight matrix each, B stored N x K.
#include "bst_block_instances.hpp"

namespace bst {

static const BlockGemmInstance kList[] = {BST_BLOCK_GEMM_TILES(true, true)};

BlockGemmList block_gemm_grouped_t() {
  return BlockGemmList{kList, (int)(sizeof(kList) / sizeof(kList[0]))};
}

}  // namespace bst
