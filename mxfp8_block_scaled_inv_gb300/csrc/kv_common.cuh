// Arithmetic shared by the KV-insert kernels (BF16 / E4M3 cache and 4-bit
// cache): BF16 packing of 8 values and the forward rotation of one
// rotate-half pair of 8-value chunks.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "quant_common.cuh"

namespace mxq {

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&r);
}

__device__ __forceinline__ uint4 to_bf16x8(const float (&y)[8]) {
  return make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
}

// Forward rotation of one rotate-half pair of chunks (x0 in the lower half,
// x1 in the upper) with the cos/sin entries j..j+7 of position p: one
// rounding per value, as the oracle.
__device__ __forceinline__ void rope_pair(const uint4& va, const uint4& vb, const uint4& cw,
                                          const uint4& sw, float (&y0)[8], float (&y1)[8]) {
  float x0[8], x1[8], c8[8], s8[8];
  unpack8(va, x0);
  unpack8(vb, x1);
  unpack8(cw, c8);
  unpack8(sw, s8);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    y0[e] = __fsub_rn(__fmul_rn(x0[e], c8[e]), __fmul_rn(x1[e], s8[e]));
    y1[e] = __fadd_rn(__fmul_rn(x1[e], c8[e]), __fmul_rn(x0[e], s8[e]));
  }
}

}  // namespace mxq
