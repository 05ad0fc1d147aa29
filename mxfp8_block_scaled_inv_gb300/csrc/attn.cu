// Attention over the paged KV cache (mxq_attn): sliding window, first keys
// that stay visible, causal within the new tokens.  Keys and values are the
// same cache row, shared by all query heads.
//
//   s_j = sm_scale * (q . k_j),  out = sum_j exp(s_j - lse) k_j,
//   lse = log(sum_j exp(s_j)) over the visible keys j.
//
// Simple form: one CTA per (token, head); warp w takes the keys w, w + 4, ...
// with a running maximum and sum, lane l the elements 2l, 2l+1 of every 64;
// the four warps' states are joined in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "mxq.h"
#include "mxq_internal.h"
#include "quant_common.cuh"

namespace mxq {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxD = 512;

__device__ __forceinline__ float2 e2m1x2_to_f32(uint8_t b) {
  uint32_t h;
  asm("{\n.reg .b8 x;\n cvt.u8.u32 x, %1;\n cvt.rn.f16x2.e2m1x2 %0, x;\n}\n" : "=r"(h) : "r"((uint32_t)b));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

template <int DT>
__global__ void __launch_bounds__(kWarps * 32) attn_simple_kernel(const AttnArgs a) {
  __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][kMaxD];
  const int64_t r = blockIdx.x;
  const int64_t t = r / a.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nc = a.D >> 6;
  // The sequence of this token: the last b with q_start[b] <= t.
  int b = (int)t, i = 0, n = 1;
  if (a.q_start != nullptr) {
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.q_start[mid] <= t) lo = mid; else hi = mid;
    }
    b = lo;
    n = a.q_start[b + 1] - a.q_start[b];
    i = (int)(t - a.q_start[b]);
    if (i < 0 || i >= n) return;
  }
  const int cap = a.max_pages * a.page_size;
  const int len = min(max(a.seq_lens[b], 0), cap);
  if (a.err_flag != nullptr && threadIdx.x == 0 && len != a.seq_lens[b])
    atomicOr(a.err_flag, MXQ_DEVERR_LENGTH);
  const int p = len - n + i;
  const int lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
  const int ns = min(a.sinks, lo);  // sinks before the window
  const int total = p < 0 ? 0 : ns + (p - lo + 1);
  const float ks = DT == MXQ_CACHE_E4M3 ? *a.kv_scale : 1.0f;
  float2 q[8], o[8];
  const uint32_t* qp = static_cast<const uint32_t*>(a.q) + r * (a.D >> 1) + lane;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    o[c] = make_float2(0.f, 0.f);
    q[c] = make_float2(0.f, 0.f);
    if (c < nc) {
      const uint32_t w = qp[c * 32];
      q[c] = make_float2(bf16_lo(w), bf16_hi(w));
    }
  }
  float m = -INFINITY, l = 0.f;
  for (int k = warp; k < total; k += kWarps) {
    const int j = k < ns ? k : lo + (k - ns);
    const int page = a.block_table[(int64_t)b * a.max_pages + j / a.page_size];
    const int64_t slot = (int64_t)page * a.page_size + j % a.page_size;
    if (page < 0 || slot >= a.num_slots) {
      if (a.err_flag != nullptr && lane == 0) atomicOr(a.err_flag, MXQ_DEVERR_SLOT);
      continue;
    }
    float2 kv[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      kv[c] = make_float2(0.f, 0.f);
      if (c >= nc) continue;
      if (DT == MXQ_CACHE_BF16) {
        const uint32_t w =
            static_cast<const uint32_t*>(a.cache)[slot * (a.D >> 1) + c * 32 + lane];
        kv[c] = make_float2(bf16_lo(w), bf16_hi(w));
      } else if (DT == MXQ_CACHE_E4M3) {
        const __nv_fp8x2_storage_t w =
            static_cast<const uint16_t*>(a.cache)[slot * (a.D >> 1) + c * 32 + lane];
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(w, __NV_E4M3);
        kv[c] = __half22float2(__half2(h));
        kv[c].x *= ks;
        kv[c].y *= ks;
      } else {
        const uint8_t w = static_cast<const uint8_t*>(a.cache)[slot * (a.D >> 1) + c * 32 + lane];
        const uint32_t sb = a.cache_sf[slot * (a.D >> 5) + c * 2 + (lane >> 4)];
        const float s = sb == 255u ? NAN : sb == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(sb << 23);
        kv[c] = e2m1x2_to_f32(w);
        kv[c].x *= s;
        kv[c].y *= s;
      }
    }
    float d = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) d += q[c].x * kv[c].x + q[c].y * kv[c].y;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
    d *= a.sm_scale;
    if (!(fabsf(d) <= 3.4e38f)) d = NAN;  // a non-finite key row (or query): the row is NaN
    const float mn = fmaxf(m, d);
    const float f = m == -INFINITY ? 0.f : __expf(m - mn);
    const float e = __expf(d - mn);
    m = mn;
    l = l * f + e;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      o[c].x = o[c].x * f + e * kv[c].x;
      o[c].y = o[c].y * f + e * kv[c].y;
    }
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int c = 0; c < 8; ++c)
    if (c < nc) *reinterpret_cast<float2*>(&sm_o[warp][c * 64 + lane * 2]) = o[c];
  __syncthreads();
  float mm = -INFINITY, ll = 0.f;
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w]);
  float f[kWarps];
  for (int w = 0; w < kWarps; ++w) {
    f[w] = sm_m[w] == -INFINITY ? 0.f : __expf(sm_m[w] - mm);
    ll += f[w] * sm_l[w];
  }
  const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : NAN);
  for (int d = threadIdx.x; d < a.D; d += kWarps * 32) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) v += f[w] * sm_o[w][d];
    static_cast<__nv_bfloat16*>(a.out)[r * a.D + d] = __float2bfloat16_rn(v * inv);
  }
  if (a.lse != nullptr && threadIdx.x == 0) a.lse[r] = ll == 0.f ? -INFINITY : mm + logf(ll);
}

}  // namespace

size_t attn_workspace_bytes(const AttnArgs&) { return 0; }

cudaError_t launch_attn(const AttnArgs& a, void*, int, cudaStream_t s, const char**) {
  const unsigned grid = (unsigned)(a.T * a.H);
  if (a.dtype == MXQ_CACHE_BF16)
    attn_simple_kernel<MXQ_CACHE_BF16><<<grid, kWarps * 32, 0, s>>>(a);
  else if (a.dtype == MXQ_CACHE_E4M3)
    attn_simple_kernel<MXQ_CACHE_E4M3><<<grid, kWarps * 32, 0, s>>>(a);
  else
    attn_simple_kernel<MXQ_CACHE_E2M1><<<grid, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace mxq
