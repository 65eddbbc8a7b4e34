// block_grad.hip -- compiled kernels of the weight gradient from 8-bit activations.
#include "bst_block_instances.hpp"

namespace bst {

static const BlockGradInstance kList[] = {
    BST_BLOCK_GRAD(128, 128, 2, 2, DY_BF16), BST_BLOCK_GRAD(256, 256, 2, 4, DY_BF16),
    BST_BLOCK_GRAD(128, 128, 2, 2, DY_F16),  BST_BLOCK_GRAD(256, 256, 2, 4, DY_F16),
    BST_BLOCK_GRAD(128, 128, 2, 2, DY_F32),  BST_BLOCK_GRAD(256, 256, 2, 4, DY_F32),
};

BlockGradList block_grad_list() {
  return BlockGradList{kList, (int)(sizeof(kList) / sizeof(kList[0]))};
}

}  // namespace bst
