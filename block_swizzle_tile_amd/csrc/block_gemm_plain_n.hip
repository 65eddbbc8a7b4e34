// block_gemm_plain_n.hip -- compiled kernels of the block-scaled product: one problem, B stored K x N.
#include "bst_block_instances.hpp"

namespace bst {

static const BlockGemmInstance kList[] = {BST_BLOCK_GEMM_TILES(false, false)};

BlockGemmList block_gemm_plain_n() {
  return BlockGemmList{kList, (int)(sizeof(kList) / sizeof(kList[0]))};
}

}  // namespace bst
