// The 4-bit KV cache: insertion of rotated KV rows as E2M1 codes with one
// E8M0 scale per 32 values (the OCP MXFP4 block format), and the gather of
// cache rows back to BF16.  Layouts and rules are stated in include/mxq.h.
//
// Mathematics.  Per block of 32 values y with amax = max |y|:
//   e = smallest integer with amax <= 6 * 2^e, clamped to [-127, 127]
//       (amax == 0 gives -127); scale byte e + 127,
//   code = E2M1 round-to-nearest-even, saturating, of y * 2^-e,
// y being the fp32 rotated value (one rounding: both products are exact).
//
// Both kernels are bound by memory.  The insertion's KV item is one 16-byte
// chunk of 8 values; the four lanes of a 32-value block find its amax with
// two shuffles.  A chunk inside the rotated slice reads its rotate-half
// partner chunk too and keeps its own half of the pair: 64 of 512 values are
// read twice (from L1), and no lane waits for another's arithmetic.  The query
// goes the ways of the 8- and 16-bit insertion, large ones out of place through
// its streaming kernel.  Measured with a gather of the same rows behind it: 8192
// tokens, 64 heads of 512, query out of place 180 us = 6.1 TB/s, 0.91 of a copy's
// rate, of which the rows take 8.7 us and the gather 6.9 us; 64 tokens 7.4 us and
// 3.6 us, launch-bound.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kv_common.cuh"
#include "mxq.h"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 8;

struct Kv4Args {
  const uint4* q;
  uint4* q_out;
  const uint4* kv;
  uint8_t* cache;
  uint8_t* cache_sf;
  const int64_t* pos;
  const int64_t* slot;
  const uint16_t* cos_tab;
  const uint16_t* sin_tab;
  int32_t* err_flag;
  int64_t cs_ld, max_pos, num_slots;
  uint32_t kv_items, q_items;
  uint32_t ik;      // chunks per KV row
  uint32_t iq, pq;  // items per query row; of them outside the slice
  int H, Dq, Dk, R;
};

// Eight values times `inv` -> eight E2M1 codes (the first value in the low
// nibble), round to nearest even, saturating at +-6.
__device__ __forceinline__ uint32_t e2m1x8(const float (&y)[8], float inv) {
  uint32_t r;
  asm("{\n.reg .b8 a, b, c, d;\n"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      "mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(y[0] * inv), "f"(y[1] * inv), "f"(y[2] * inv), "f"(y[3] * inv), "f"(y[4] * inv),
        "f"(y[5] * inv), "f"(y[6] * inv), "f"(y[7] * inv));
  return r;
}

// One KV chunk; all 32 lanes call it together (`live` false: past the end).
__device__ __forceinline__ void kv_chunk(const Kv4Args& a, uint32_t it, bool live) {
  const uint32_t t = live ? it / a.ik : 0;
  const int c = live ? (int)(it - t * a.ik) : 0;
  const uint4* src = a.kv + (size_t)t * a.ik;
  int64_t p = 0;
  bool bad = false;
  if (a.R > 0) {
    p = __ldg(a.pos + t);
    bad = p < 0 || p >= a.max_pos;
  }
  const int64_t sl = __ldg(a.slot + t);
  const bool over = sl >= a.num_slots;
  if (live && c == 0 && a.err_flag != nullptr && (bad || over))
    atomicOr(a.err_flag, (bad ? MXQ_DEVERR_POSITION : 0) | (over ? MXQ_DEVERR_SLOT : 0));
  float y[8];
  const int first = (a.Dk - a.R) / 8, half = a.R / 16;
  if (c < first || bad) {
    unpack8(__ldg(src + c), y);
  } else {
    const bool lower = c < first + half;
    const int j = (c - first - (lower ? 0 : half)) * 8;  // entry of the half
    const uint4 cw = __ldg(reinterpret_cast<const uint4*>(a.cos_tab + p * a.cs_ld + j));
    const uint4 sw = __ldg(reinterpret_cast<const uint4*>(a.sin_tab + p * a.cs_ld + j));
    float y0[8], y1[8];
    rope_pair(__ldg(src + (lower ? c : c - half)), __ldg(src + (lower ? c + half : c)), cw, sw, y0,
              y1);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = lower ? y0[e] : y1[e];
  }
  float m = 0.0f;
  bool nan = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    m = fmaxf(m, fabsf(y[e]));
    nan |= !(fabsf(y[e]) <= 3.4028234e38f);
  }
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  nan |= __shfl_xor_sync(0xffffffffu, (int)nan, 1) != 0;
  nan |= __shfl_xor_sync(0xffffffffu, (int)nan, 2) != 0;
  if (!live || sl < 0 || over || bad) return;
  // amax = (1+f) * 2^E and 6 = 1.5 * 2^2: e = E - 2 + (f > 0.5); a zero or
  // subnormal amax clamps to e = -127.
  const uint32_t mb = __float_as_uint(m);
  const int bexp = (int)(mb >> 23);
  int ex = bexp == 0 ? -127 : max(bexp - 127 - 2 + ((mb & 0x7FFFFFu) > 0x400000u ? 1 : 0), -127);
  const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);  // 2^-e, -e in [-125, 127]
  const uint32_t codes = e2m1x8(y, inv);
  uint8_t* row = a.cache + (size_t)sl * (size_t)(a.Dk / 2);
  *reinterpret_cast<uint32_t*>(row + (size_t)c * 4) = codes;
  if ((c & 3) == 0)
    a.cache_sf[(size_t)sl * (size_t)(a.Dk / 32) + (c >> 2)] = nan ? 0xFF : (uint8_t)(ex + 127);
}

// One query item: a chunk outside the slice (out of place only) or one
// rotate-half pair of chunks.
__device__ __forceinline__ void q_item(const Kv4Args& a, uint32_t it) {
  const uint32_t row = it / a.iq;
  const uint32_t i = it - row * a.iq;
  const uint4* src = a.q + (size_t)row * (a.Dq >> 3);
  uint4* dst = a.q_out + (size_t)row * (a.Dq >> 3);
  if (i < a.pq) {
    dst[i] = src[i];
    return;
  }
  const int64_t p = __ldg(a.pos + row / (uint32_t)a.H);
  const int c0 = (a.Dq - a.R) / 8 + (int)(i - a.pq);
  const int c1 = c0 + a.R / 16;
  float y0[8], y1[8];
  if (p < 0 || p >= a.max_pos) {  // invalid position: the slice is written as zeros
#pragma unroll
    for (int e = 0; e < 8; ++e) y0[e] = y1[e] = 0.0f;
  } else {
    const int j = (int)(i - a.pq) * 8;
    const uint4 va = src[c0];  // plain loads: the query may be rotated in place
    const uint4 vb = src[c1];
    const uint4 cw = __ldg(reinterpret_cast<const uint4*>(a.cos_tab + p * a.cs_ld + j));
    const uint4 sw = __ldg(reinterpret_cast<const uint4*>(a.sin_tab + p * a.cs_ld + j));
    rope_pair(va, vb, cw, sw, y0, y1);
  }
  dst[c0] = to_bf16x8(y0);
  dst[c1] = to_bf16x8(y1);
}

__global__ void __launch_bounds__(kThreads, kBlocksPerSm) rope_kv4_insert_kernel(const Kv4Args a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t stride = gridDim.x * kThreads;
  const uint32_t first = blockIdx.x * kThreads + threadIdx.x;
  const uint32_t kv_end = (a.kv_items + 31u) & ~31u;  // whole warps: the lanes shuffle
  for (uint32_t it = first; it < kv_end; it += stride) kv_chunk(a, it, it < a.kv_items);
  for (uint32_t it = first; it < a.q_items; it += stride) q_item(a, it);
}

// The value of an E2M1 code (its low four bits).
__device__ __forceinline__ float e2m1_value(uint32_t code) {
  // Magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6: two significand bits at exponent
  // field EE; twice the value is the integer 0, 1, 2, 3, 4, 6, 8, 12.
  const uint32_t m = code & 7u;
  const uint32_t twice = m < 2u ? m : (2u | (m & 1u)) << ((m >> 1) - 1u);
  const float v = 0.5f * (float)twice;
  return (code & 8u) ? -v : v;
}

// Chunks of 8 codes with their scale byte -> 8 BF16 values, which hold every
// magnitude 0.5..6 times 2^(sb-127) exactly, except that the largest exponents
// overflow to infinity; byte 0xFF gives NaN.
__global__ void __launch_bounds__(kThreads) kv4_gather_kernel(const uint8_t* cache,
                                                              const uint8_t* cache_sf,
                                                              const int64_t* slots, uint4* out,
                                                              uint32_t items, uint32_t per_row,
                                                              int64_t num_slots, int32_t* err_flag) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t stride = gridDim.x * kThreads;
  for (uint32_t it = blockIdx.x * kThreads + threadIdx.x; it < items; it += stride) {
    const uint32_t r = it / per_row, c = it - r * per_row;  // chunk c of 8 values
    const int64_t sl = __ldg(slots + r);
    uint4 o = make_uint4(0, 0, 0, 0);
    if (sl >= 0 && sl < num_slots) {
      const uint32_t w =
          *reinterpret_cast<const uint32_t*>(cache + ((size_t)sl * per_row + c) * 4);
      const uint32_t sb = cache_sf[(size_t)sl * (per_row / 4) + (c >> 2)];
      // 2^(sb-127) as fp32 (2^-127 is subnormal), NaN for 0xFF.
      const float s = sb == 255u ? __uint_as_float(0x7FFFFFFFu)
                                 : sb == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(sb << 23);
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = e2m1_value(w >> (4 * e)) * s;
      o = to_bf16x8(y);
    } else if (sl >= num_slots && c == 0 && err_flag != nullptr) {
      atomicOr(err_flag, MXQ_DEVERR_SLOT);
    }
    out[it] = o;
  }
}

template <typename K, typename... Args>
cudaError_t launch_pdl(K kern, int64_t blocks, int64_t cap, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < cap ? blocks : cap), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  // Programmatic dependent launch: the grid may be scheduled while the
  // preceding kernel finishes; it waits for it before reading anything.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

cudaError_t launch_rope_kv4_insert(const void* q, void* q_out, int64_t T, int H, int Dq,
                                   const void* kv, int Dk, const int64_t* pos, const void* cos,
                                   const void* sin, int64_t cs_ld, int64_t max_pos, int R,
                                   const int64_t* slot, uint8_t* cache, uint8_t* cache_sf,
                                   int64_t num_slots, int32_t* err_flag, int num_sms,
                                   cudaStream_t s) {
  Kv4Args a = {};
  a.q = static_cast<const uint4*>(q);
  a.q_out = static_cast<uint4*>(q_out);
  a.kv = static_cast<const uint4*>(kv);
  a.cache = cache;
  a.cache_sf = cache_sf;
  a.pos = pos;
  a.slot = slot;
  a.cos_tab = static_cast<const uint16_t*>(cos);
  a.sin_tab = static_cast<const uint16_t*>(sin);
  a.err_flag = err_flag;
  a.cs_ld = cs_ld;
  a.max_pos = max_pos;
  a.num_slots = num_slots;
  a.H = H;
  a.Dq = Dq;
  a.Dk = Dk;
  a.R = R;
  a.ik = (uint32_t)(Dk / 8);
  a.kv_items = (uint32_t)T * a.ik;
  if (rope_q_streams(q, q_out, T, H, Dq)) {
    // A large query out of place: the streaming copy of the other insertion.
    cudaError_t e = launch_rope_kv_insert(q, q_out, T, H, Dq, nullptr, Dk, pos, cos, sin, cs_ld,
                                          max_pos, R, nullptr, nullptr, 0, 0, nullptr, nullptr,
                                          num_sms, s);
    if (e != cudaSuccess) return e;
  } else if (H > 0) {
    a.pq = q != q_out ? (uint32_t)((Dq - R) / 8) : 0u;
    a.iq = a.pq + (uint32_t)(R / 16);
    a.q_items = (uint32_t)(T * H) * a.iq;
  }
  const uint32_t most = a.kv_items > a.q_items ? a.kv_items : a.q_items;
  return launch_pdl(rope_kv4_insert_kernel, ceil_div(most, kThreads), (int64_t)num_sms * kBlocksPerSm,
                    s, a);
}

cudaError_t launch_kv4_gather(const uint8_t* cache, const uint8_t* cache_sf, const int64_t* slots,
                              int64_t n, int Dk, int64_t num_slots, void* out, int32_t* err_flag,
                              int num_sms, cudaStream_t s) {
  const uint32_t per_row = (uint32_t)(Dk / 8);
  const uint32_t items = (uint32_t)n * per_row;
  return launch_pdl(kv4_gather_kernel, ceil_div(items, kThreads), (int64_t)num_sms * kBlocksPerSm, s,
                    cache, cache_sf, slots, static_cast<uint4*>(out), items, per_row, num_slots,
                    err_flag);
}

}  // namespace mxq
