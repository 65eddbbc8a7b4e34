// bst_block_quant.hpp -- 8-bit codes and E8M0 scales of a matrix, and back.
//
// Both directions are one pass over memory.  A thread holds 8 consecutive
// values (16 bytes of bf16 / fp16, 8 bytes of codes), so 16 lanes hold a block
// of 128 and the block's largest magnitude is four lane exchanges away.
#pragma once

#include "bst_block.hpp"

namespace bst {

enum XKind { X_F16 = 1, X_BF16 = 2, X_F32 = 7 };

struct BlockQuantArgs {
  const uint8_t* X;  // quant: input; dequant: unused
  uint8_t* Xo;       // dequant: output
  uint8_t* Q;
  uint8_t* S;        // scales (read or written)
  int64_t ldx, ldq, lds;
  uint32_t M, K, kb;   // kb: blocks per row
  uint32_t blocks;     // M * kb: runs of 128 in the rows, whatever shares a scale
  uint32_t xvec, qvec;  // rows of X / Q start on whole vectors
  uint32_t s_f32, block_rows;
  FastDiv by_kb;
};

// 8 values as fp32 bits; past `live` they are zero.
template <int XK>
__device__ __forceinline__ void load8(float (&v)[8], const uint8_t* p, uint32_t live, bool vec) {
  if (vec && live >= 8u) {
    if constexpr (XK == X_F32) {
      const f32x4_t a = ((const f32x4_t*)p)[0], b = ((const f32x4_t*)p)[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = a[e];
        v[4 + e] = b[e];
      }
    } else {
      const u32x4_t w = *(const u32x4_t*)p;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t h = (w[e / 2] >> (16 * (e & 1))) & 0xffffu;
        v[e] = XK == X_BF16 ? __builtin_bit_cast(float, h << 16)
                            : (float)__builtin_bit_cast(_Float16, (uint16_t)h);
      }
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (uint32_t)e < live ? out_value(p + e * (XK == X_F32 ? 4 : 2), XK) : 0.0f;
}

// The largest finite magnitude's bits (monotonic as integers) of 8 values.
__device__ __forceinline__ uint32_t top8(const float (&v)[8]) {
  uint32_t t = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v[e]) & 0x7fffffffu;
    t = max(t, u < 0x7f800000u ? u : 0u);
  }
  return t;
}

// The scale byte: the smallest e >= 0 with top <= 448 2^(e - 127); 448 =
// 1.75 * 2^8, so the exponent is top's less 8, and one more where top's
// significand is above 1.75.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e > 0 ? (uint32_t)e : 0u;
}

// Codes of 8 values at scale byte e: x * 2^(127 - e) is exact (or far below
// the smallest code), and at most 448, so the conversion's only rounding is
// the code's own; what is not finite becomes NaN.
__device__ __forceinline__ u32x2_t codes8(const float (&v)[8], uint32_t e) {
  const float inv = __builtin_bit_cast(float, (254u - e) << 23);
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu;
    s[i] = u < 0x7f800000u ? v[i] * inv : __builtin_bit_cast(float, 0x7fc00000u);
  }
  u32x2_t o;
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(s[4 * d], s[4 * d + 1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(s[4 * d + 2], s[4 * d + 3], w, true);
    o[d] = (uint32_t)w;
  }
  return o;
}

__device__ __forceinline__ void put_codes(uint8_t* q, const u32x2_t& o, uint32_t live, bool vec) {
  if (vec && live >= 8u) {
    *(u32x2_t*)q = o;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if ((uint32_t)e < live) q[e] = (uint8_t)(o[e / 4] >> (8 * (e & 3)));
}

// Blocks of 1 x 128: 16 blocks per workgroup and step, one step in flight per
// thread.  More steps in flight were slower (16384 x 8192 bf16: 79 us at one,
// 80 at two, 95 at four): the eight waves per SIMD that fit hide the latency,
// and their loads stay near each other in memory.
template <int XK>
__global__ void __launch_bounds__(256) quant_rows_kernel(BlockQuantArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int ES = XK == X_F32 ? 4 : 2;
  const uint32_t sub = threadIdx.x & 15u, step = gridDim.x * 16u;
  // step < 2^20 and blocks < 2^31: b stays in 32 bits
  for (uint32_t b = blockIdx.x * 16u + (threadIdx.x >> 4); b < a.blocks; b += step) {
    const uint32_t row = a.by_kb.div(b), kb = b - row * a.kb;
    const uint32_t k = kb * 128u + sub * 8u;
    float v[8] = {};
    if (k < a.K) load8<XK>(v, a.X + ((int64_t)row * a.ldx + k) * ES, a.K - k, a.xvec != 0);
    uint32_t top = top8(v);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d, 16));
    const uint32_t e = scale_byte(top);
    if (k < a.K) put_codes(a.Q + (int64_t)row * a.ldq + k, codes8(v, e), a.K - k, a.qvec != 0);
    if (sub == 0) a.S[(int64_t)row * a.lds + kb] = (uint8_t)e;
  }
#endif
}

// Blocks of 128 x 128: one workgroup each, the block in registers.
template <int XK>
__global__ void __launch_bounds__(256) quant_square_kernel(BlockQuantArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int ES = XK == X_F32 ? 4 : 2;
  __shared__ uint32_t tops[4];
  const uint32_t rb = a.by_kb.div(blockIdx.x), kb = blockIdx.x - rb * a.kb;
  const uint32_t k = kb * 128u + (threadIdx.x & 15u) * 8u;
  const uint32_t r0 = rb * 128u + (threadIdx.x >> 4);
  float v[8][8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t r = r0 + 16u * i;
    if (r < a.M && k < a.K)
      load8<XK>(v[i], a.X + ((int64_t)r * a.ldx + k) * ES, a.K - k, a.xvec != 0);
    else
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, top8(v[i]));
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
  if ((threadIdx.x & 63u) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  const uint32_t e = scale_byte(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t r = r0 + 16u * i;
    if (r < a.M && k < a.K)
      put_codes(a.Q + (int64_t)r * a.ldq + k, codes8(v[i], e), a.K - k, a.qvec != 0);
  }
  if (threadIdx.x == 0) a.S[(int64_t)rb * a.lds + kb] = (uint8_t)e;
#endif
}

// Codes back to values: 16 blocks of 1 x 128 per workgroup and step.
template <int XK>
__global__ void __launch_bounds__(256) dequant_kernel(BlockQuantArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int ES = XK == X_F32 ? 4 : 2;
  constexpr float LARGEST = XK == X_F32 ? 3.4028234663852886e38f
                            : XK == X_BF16 ? 3.3895313892515355e38f : 65504.0f;
  const uint32_t sub = threadIdx.x & 15u, step = gridDim.x * 16u;
  for (uint32_t b = blockIdx.x * 16u + (threadIdx.x >> 4); b < a.blocks; b += step) {
    const uint32_t row = a.by_kb.div(b), kb = b - row * a.kb;
    const uint32_t k = kb * 128u + sub * 8u;
    if (k >= a.K) continue;
    const uint32_t live = a.K - k;
    const uint8_t* p = a.Q + (int64_t)row * a.ldq + k;
    u32x2_t q = {0u, 0u};
    if (a.qvec && live >= 8u) {
      q = *(const u32x2_t*)p;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if ((uint32_t)e < live) q[e / 4] |= (uint32_t)p[e] << (8 * (e & 3));
    }
    const int64_t at = (int64_t)(a.block_rows == 1 ? row : row / 128u) * a.lds + kb;
    const float f = a.s_f32 ? ((const float*)a.S)[at] : e8m0_value(a.S[at]);
    const bool finite = __builtin_fabsf(f) < __builtin_inff();
    float v[8];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      typedef float f2 __attribute__((ext_vector_type(2)));
      const f2 c = (d & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8((int)q[d / 2], true)
                           : __builtin_amdgcn_cvt_pk_f32_fp8((int)q[d / 2], false);
      v[2 * d] = c[0] * f;
      v[2 * d + 1] = c[1] * f;
    }
    // a finite code never becomes infinite (NaN passes: it fails both comparisons)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (finite && v[e] > LARGEST) v[e] = LARGEST;
      if (finite && v[e] < -LARGEST) v[e] = -LARGEST;
    }
    put_run<8>(a.Xo + ((int64_t)row * a.ldx + k) * ES, nullptr, v, live, a.xvec != 0 && live >= 8u,
               XK);
  }
#endif
}

}  // namespace bst
