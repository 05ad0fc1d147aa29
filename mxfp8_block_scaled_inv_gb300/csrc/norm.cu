// Residual addition, root-mean-square norm and group-128 E4M3 / E8M0
// quantisation of its result in one pass.  Layouts and rules are stated in
// include/mxq.h.
//
// Mathematics, per row:  s = bf16(x + r)  (s = x without a residual),
//   y_i = bf16(s_i * w_i / sqrt(sum s^2 / D + eps)),
// the sum of squares in fp32 over the *stored* s, so that the result follows
// from residual_out alone; the codes are those of the BF16 y, so that a caller
// of the codes and one of y (quantised later, or by another kernel) see the
// same numbers.
//
// Bound by memory: every byte is moved once.  A thread holds its 16-byte chunks
// of s as packed BF16 between the two uses, and chunk c belongs to thread
// c mod (threads of the row), so that 16 neighbouring lanes hold one scale
// group and every access of a warp is contiguous.  Measured with a residual, y
// and codes, 8192 rows: of 4096 columns 45.4 us, 6.65 TB/s (0.98 of a plain copy's
// rate), of 512 columns 7.6 us (0.74: every CTA runs once, so nothing hides its start
// and end); one row of 4096 columns 2.4 us, which is its launch, one trip to memory
// and the sum over the CTA.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_common.cuh"
#include "mxq.h"
#include "mxq_internal.h"
#include "mxq_ptx.cuh"
#include "quant_common.cuh"

namespace mxq {
namespace {

struct NormArgs {
  const uint4* x;
  const uint4* res;  // NULL: no residual
  uint4* res_out;
  const uint4* w;    // NULL: ones
  uint4* y;          // NULL: not stored
  uint2* q;          // NULL: no codes
  uint8_t* sc;
  int64_t T;
  int chunks, KG;
  float inv_d, eps;
};

__device__ __forceinline__ uint4 add8(const uint4& a, const uint4& b) {
  float p[8], q[8];
  unpack8(a, p);
  unpack8(b, q);
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e] = __fadd_rn(p[e], q[e]);
  return to_bf16x8(p);
}

// THREADS: threads of one row (32: one warp of a CTA of eight rows).  CPT:
// 16-byte chunks of a thread.
template <int THREADS, int CPT>
__global__ void __launch_bounds__(THREADS == 32 ? 256 : THREADS) add_rms_norm_kernel(
    const NormArgs a) {
  constexpr int kWarps = THREADS / 32;
  __shared__ float part[kWarps > 1 ? kWarps : 1];
  ptx::griddep_launch_dependents();
  const int tid = THREADS == 32 ? (int)(threadIdx.x & 31) : (int)threadIdx.x;
  const int lane = tid & 31;
  const int64_t row = THREADS == 32 ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  ptx::griddep_wait();
  if (THREADS == 32 && row >= a.T) return;
  const size_t base = (size_t)row * (size_t)a.chunks;
  uint4 s[CPT];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = i * THREADS + tid;
    s[i] = make_uint4(0, 0, 0, 0);
    // Plain loads: an output may be this very buffer.
    if (c < a.chunks) s[i] = a.x[base + c];
  }
  if (a.res != nullptr) {
    uint4 r[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = i * THREADS + tid;
      r[i] = make_uint4(0, 0, 0, 0);
      if (c < a.chunks) r[i] = a.res[base + c];
    }
#pragma unroll
    for (int i = 0; i < CPT; ++i) s[i] = add8(s[i], r[i]);
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    float v[8];
    unpack8(s[i], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(v[e], v[e], sum);
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  if constexpr (kWarps > 1) {
    if (lane == 0) part[tid >> 5] = sum;
    __syncthreads();
    sum = lane < kWarps ? part[lane] : 0.0f;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  }
  const float inv = rsqrtf(fmaf(sum, a.inv_d, a.eps));
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = i * THREADS + tid;
    if (i * THREADS + (tid & ~31) >= a.chunks) break;  // nothing left for this warp
    const bool in = c < a.chunks;
    float v[8], w[8];
    unpack8(s[i], v);
    if (a.w != nullptr) {
      unpack8(in ? __ldg(a.w + c) : make_uint4(0, 0, 0, 0), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * inv * w[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * inv;
    }
    const uint4 y = to_bf16x8(v);
    if (in && a.res_out != nullptr) a.res_out[base + c] = s[i];
    if (in && a.y != nullptr) a.y[base + c] = y;
    if (a.q != nullptr) {
      unpack8(y, v);
      uint32_t sb;
      const float amax = half_warp_amax(v);
      const uint2 codes = encode8(v, amax, &sb);
      if (in) {
        a.q[base + c] = codes;
        if ((lane & 15) == 0) a.sc[(size_t)row * a.KG + (c >> 4)] = (uint8_t)sb;
      }
    }
  }
}

template <int THREADS, int CPT>
cudaError_t launch_rows(const NormArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(THREADS == 32 ? ceil_div(a.T, 8) : a.T), 1, 1);
  cfg.blockDim = dim3(THREADS == 32 ? 256 : THREADS, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, add_rms_norm_kernel<THREADS, CPT>, a);
}

}  // namespace

cudaError_t launch_add_rms_norm(const void* x, const void* res, void* res_out, const void* w,
                                int64_t T, int D, float eps, void* y, uint8_t* q, uint8_t* sc,
                                cudaStream_t s) {
  NormArgs a = {};
  a.x = static_cast<const uint4*>(x);
  a.res = static_cast<const uint4*>(res);
  a.res_out = static_cast<uint4*>(res_out);
  a.w = static_cast<const uint4*>(w);
  a.y = static_cast<uint4*>(y);
  a.q = reinterpret_cast<uint2*>(q);
  a.sc = sc;
  a.T = T;
  a.chunks = D / 8;
  a.KG = (int)ceil_div(D, kGroup);
  a.inv_d = 1.0f / (float)D;
  a.eps = eps;
  // Rows of up to 512 columns take one warp (no barrier, eight rows to a CTA), longer
  // ones a CTA.  8192 rows and one row, us, this split and the next best:
  //   512 columns   warp 7.8, 2.1       64 threads x 1 chunk 9.2, 1.9
  //   1024          128 x 1 11.7, 2.0   warp 13.2, 2.1 (64 rows: 2.1 and 3.4)
  //   2048          256 x 1 24.3, 2.0   128 x 2 23.9, 2.4 (2048 rows: 7.3 and 7.7)
  //   4096          256 x 2 45.5, 2.5   512 x 1 47.0, 2.5
  //   8192          512 x 2 88.9        1024 x 1 103, 256 x 4 89.1 (64 rows: 3.1, 3.1, 3.4)
  //   16384         512 x 4 174         1024 x 2 213
  if (a.chunks <= 32) return launch_rows<32, 1>(a, s);
  if (a.chunks <= 64) return launch_rows<32, 2>(a, s);
  if (a.chunks <= 128) return launch_rows<128, 1>(a, s);
  if (a.chunks <= 256) return launch_rows<256, 1>(a, s);
  if (a.chunks <= 512) return launch_rows<256, 2>(a, s);
  if (a.chunks <= 1024) return launch_rows<512, 2>(a, s);
  if (a.chunks <= 2048) return launch_rows<512, 4>(a, s);
  return launch_rows<1024, 8>(a, s);
}

}  // namespace mxq
