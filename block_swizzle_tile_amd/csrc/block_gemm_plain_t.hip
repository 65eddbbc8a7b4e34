// block_gemm_plain_t.hip -- compiled kernels of the block-scaled product: one problem, B stored N x K.
#include "bst_block_instances.hpp"

namespace bst {

static const BlockGemmInstance kList[] = {BST_BLOCK_GEMM_TILES(true, false)};

BlockGemmList block_gemm_plain_t() {
  return BlockGemmList{kList, (int)(sizeof(kList) / sizeof(kList[0]))};
}

}  // namespace bst
