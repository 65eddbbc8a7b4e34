// bst_block_instances.hpp -- tables of the compiled block-scaled kernels.
// block_gemm_*.hip and block_grad.hip instantiate them; block.hip picks one
// per call.
#pragma once

#include <hip/hip_runtime.h>

#include "bst_block_gemm.hpp"
#include "bst_block_grad.hpp"
#include "bst_block_rows.hpp"

namespace bst {

struct BlockGemmInstance {
  int bm, bn;
  int mode;  // BlockMode
  hipError_t (*launch)(uint32_t grid, hipStream_t, const BlockGemmArgs&);
};
struct BlockGemmList {
  const BlockGemmInstance* begin;
  int count;
};
BlockGemmList block_gemm_plain_t();
BlockGemmList block_gemm_plain_n();
BlockGemmList block_gemm_grouped_t();
BlockGemmList block_gemm_grouped_n();

struct BlockGradInstance {
  int bk, bn, dy;
  hipError_t (*launch)(uint32_t grid, hipStream_t, const BlockGradArgs&);
};
struct BlockGradList {
  const BlockGradInstance* begin;
  int count;
};
BlockGradList block_grad_list();

template <int BM, int BN, int WM, int WN, int ST, bool TB, int MODE, bool GR>
hipError_t launch_block_gemm(uint32_t grid, hipStream_t st, const BlockGemmArgs& a) {
  hipLaunchKernelGGL((block_gemm_kernel<BM, BN, WM, WN, ST, TB, MODE, GR>), dim3(grid),
                     dim3(64 * WM * WN), 0, st, a);
  return hipGetLastError();
}

template <int BK, int BN, int WM, int WN, int DY>
hipError_t launch_block_grad(uint32_t grid, hipStream_t st, const BlockGradArgs& a) {
  hipLaunchKernelGGL((block_grad_kernel<BK, BN, WM, WN, DY>), dim3(grid), dim3(64 * WM * WN), 0,
                     st, a);
  return hipGetLastError();
}

#define BST_BLOCK_GEMM(BM, BN, WM, WN, ST, TB, MODE, GR)                \
  BlockGemmInstance {                                                   \
    BM, BN, MODE, &launch_block_gemm<BM, BN, WM, WN, ST, TB, MODE, GR> \
  }
#define BST_BLOCK_GEMM_TILE(BM, BN, WM, WN, ST, TB, GR)     \
  BST_BLOCK_GEMM(BM, BN, WM, WN, ST, TB, MODE_E8M0, GR),    \
      BST_BLOCK_GEMM(BM, BN, WM, WN, ST, TB, MODE_F32, GR), \
      BST_BLOCK_GEMM(BM, BN, WM, WN, ST, TB, MODE_EXACT, GR)
// Eight waves on 64x128 and 128x128, though four of twice the columns would read
// a quarter less from LDS: 2 x 4 against 2 x 2 waves, K x N weights, E8M0,
// 1024 x 2048 x 4096 on 64x128 17.4 / 19.8 us, with fp32 scales 22.6 / 25.2, fp32
// out 33.2 / 36.0; on 128x128 22.0 / 23.5, 25.1 / 31.0, 43.7 / 51.4 (2048 x 4096 x
// 4096, E8M0: 52.8 both).
#define BST_BLOCK_GEMM_TILES(TB, GR)                                                          \
  BST_BLOCK_GEMM_TILE(32, 128, 1, 4, 4, TB, GR), BST_BLOCK_GEMM_TILE(64, 128, 2, 4, 4, TB, GR), \
      BST_BLOCK_GEMM_TILE(128, 128, 2, 4, 4, TB, GR), \
      BST_BLOCK_GEMM(256, 256, 2, 4, 2, TB, MODE_E8M0, GR), BST_BLOCK_GEMM(256, 256, 2, 4, 2, TB, MODE_F32, GR)

#define BST_BLOCK_GRAD(BK, BN, WM, WN, DY) \
  BlockGradInstance { BK, BN, DY, &launch_block_grad<BK, BN, WM, WN, DY> }

}  // namespace bst
