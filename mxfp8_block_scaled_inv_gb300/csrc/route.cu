// Routing of tokens to experts: scores, balance bias, groups, top-k, weights.
// Rules are stated in include/mxq.h.
//
// Mathematics, per token over experts e:  p_e = score(l_e),  c_e = p_e + b_e;
// a group's value is the sum of its one or two largest c; of the groups the
// `keep` largest stay; the experts are the k largest c of those, ties going to
// the lowest index; w_j = scale * p_j (/ (sum p + 1e-20)).
//
// A warp takes a token; lane i holds the experts [i * PER, (i + 1) * PER), so
// that lane order is index order and the lowest lane of a tie is the lowest
// index.  Each pick is one warp-wide integer maximum over order-preserving
// keys, one ballot, and a new maximum in the lane that lost an expert.
//
// What is chosen is defined by 64-bit scores: fp32 scores order two experts
// wrongly where they differ by less than their rounding.  So the fp32 pass
// also looks one pick past the last, and where two neighbouring picks (or the
// last kept group and the next) are nearer than the rounding bounds below, and
// not equal in logit and bias, the row is done again with 64-bit scores.
// Without a bias the experts are ordered by their logits, which is exact.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mxq.h"
#include "mxq_internal.h"
#include "mxq_ptx.cuh"

namespace mxq {
namespace {

constexpr int kWarps = 4;
constexpr uint32_t kAll = 0xffffffffu;

struct RouteArgs {
  const void* logits;
  const float* bias;  // NULL: none
  int32_t* ids;
  float* weights;
  int64_t T;
  int E, k, scoring, groups, keep, group_top, renorm, per_group;
  float scale;
};

// Order-preserving 32-bit key of a finite fp32 value; never 0.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 becomes 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// score(l); for the softmax mx is the row's maximum and z the sum of
// exp(l - mx).
__device__ __forceinline__ float score_of(int scoring, float l, float mx, float z) {
  if (scoring == MXQ_SCORE_SOFTMAX) return expf(l - mx) / z;
  if (scoring == MXQ_SCORE_SIGMOID) return 1.0f / (1.0f + expf(-l));
  return sqrtf(fmaxf(l, 0.0f) + log1pf(expf(-fabsf(l))));
}
__device__ __forceinline__ double score_of(int scoring, double l, double mx, double z) {
  if (scoring == MXQ_SCORE_SOFTMAX) return exp(l - mx) / z;
  if (scoring == MXQ_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
  return sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
}

template <typename R>
__device__ __forceinline__ R warp_max(R v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    const R o = __shfl_xor_sync(kAll, v, m);
    v = o > v ? o : v;
  }
  return v;
}
template <typename R>
__device__ __forceinline__ R warp_sum(R v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(kAll, v, m);
  return v;
}

// A value that compares below every candidate.
template <typename R>
__device__ __forceinline__ R lowest();
template <>
__device__ __forceinline__ float lowest<float>() { return -INFINITY; }
template <>
__device__ __forceinline__ double lowest<double>() { return -(double)INFINITY; }

// The lowest lane that holds the largest `v`; -1 if every lane holds lowest().
__device__ __forceinline__ int best_lane(float v, float* top) {
  const uint32_t key = v == -INFINITY ? 0u : key_of(v);
  const uint32_t m = __reduce_max_sync(kAll, key);
  *top = m == 0u ? -INFINITY : value_of(m);
  return m == 0u ? -1 : __ffs(__ballot_sync(kAll, key == m)) - 1;
}
__device__ __forceinline__ int best_lane(double v, double* top) {
  const double m = warp_max(v);
  *top = m;
  return m == -(double)INFINITY ? -1 : __ffs(__ballot_sync(kAll, v == m)) - 1;
}

// One row with scores of type R.  `l`: the lane's logits, `open`: bit i set
// where expert i of the lane may be chosen, b: its biases.  Lane j < k returns
// the j-th expert (-1: none) and its score.  True where fp32 cannot tell.
template <int PER, typename R>
__device__ bool route_row(const RouteArgs& a, const float (&l)[PER], const float (&b)[PER],
                          uint32_t open, uint32_t summed, int lane, int* expert, R* score) {
  const bool grouped = a.keep < a.groups;
  const bool biased = a.bias != nullptr;
  R mx = (R)0, z = (R)1;
  if (a.scoring == MXQ_SCORE_SOFTMAX) {
    R m = lowest<R>();
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if ((summed >> i) & 1u) m = (R)l[i] > m ? (R)l[i] : m;
    mx = warp_max(m);
    R s = (R)0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if ((summed >> i) & 1u) s += exp((R)l[i] - mx);
    z = warp_sum(s);
  }
  // What orders the experts; without a bias the logits do.
  R c[PER];
  R pmax = (R)0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    c[i] = lowest<R>();
    if ((open >> i) & 1u) {
      if (biased || grouped) {
        const R p = score_of(a.scoring, (R)l[i], mx, z);
        pmax = p > pmax ? p : pmax;
        c[i] = p + (R)b[i];
      } else {
        c[i] = (R)l[i];
      }
    }
  }
  // Bounds on the error of an fp32 difference: the scores' relative errors
  // (exp, sums of up to 1024 terms, a quotient: below 2e-6 each), and the
  // rounding of the sums with the bias.
  const R slack = sizeof(R) == 4 && (biased || grouped) ? (R)4e-6f * warp_max(pmax) : (R)0;
  bool unsure = false;
  if (grouped) {
    // The two best of each group; lane g keeps group g's value.
    R mine = lowest<R>();
    for (int g = 0; g < a.groups; ++g) {
      R a1 = lowest<R>(), a2 = lowest<R>();
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = lane * PER + i - g * a.per_group;
        if (e >= 0 && e < a.per_group) {
          const R v = c[i];
          if (v > a1) {
            a2 = a1;
            a1 = v;
          } else if (v > a2) {
            a2 = v;
          }
        }
      }
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) {
        const R o1 = __shfl_xor_sync(kAll, a1, m), o2 = __shfl_xor_sync(kAll, a2, m);
        const R lo = o1 < a1 ? o1 : a1, hi2 = o2 > a2 ? o2 : a2;
        a1 = o1 > a1 ? o1 : a1;
        a2 = lo > hi2 ? lo : hi2;
      }
      const R v = a.group_top == 2 && a2 != lowest<R>() ? a1 + a2 : a1;
      if (lane == g) mine = v;
    }
    uint32_t kept = 0;
    R last = (R)0, top;
    for (int j = 0; j < a.keep; ++j) {
      const int w = best_lane(mine, &top);
      if (w < 0) break;
      last = top;
      kept |= 1u << w;
      if (lane == w) mine = lowest<R>();
    }
    if (sizeof(R) == 4) {
      const int w = best_lane(mine, &top);
      if (w >= 0 && !(last - top > (R)2 * slack + (R)1e-6f * (fabs(last) + fabs(top)))) unsure = true;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (!((kept >> ((lane * PER + i) / a.per_group)) & 1u)) c[i] = lowest<R>();
    if (!biased) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (c[i] != lowest<R>()) c[i] = (R)l[i];
    }
  }
  int eid = -1;
  R prev = (R)0;
  float prev_l = 0.0f, prev_b = 0.0f, my_l = 0.0f;
  R best = lowest<R>();
#pragma unroll
  for (int i = 0; i < PER; ++i) best = c[i] > best ? c[i] : best;
  const int picks = a.k + (sizeof(R) == 4 && biased ? 1 : 0);
  for (int j = 0; j < picks; ++j) {
    R top;
    const int w = best_lane(best, &top);
    if (w < 0) break;
    int e = 0;
    float wl = 0.0f, wb = 0.0f;
    if (lane == w) {
      R next = lowest<R>();
      bool found = false;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (!found && c[i] == top) {
          found = true;
          e = lane * PER + i;
          wl = l[i];
          wb = b[i];
          c[i] = lowest<R>();
        }
        next = c[i] > next ? c[i] : next;
      }
      best = next;
    }
    e = __shfl_sync(kAll, e, w);
    wl = __shfl_sync(kAll, wl, w);
    if (sizeof(R) == 4 && biased) {
      wb = __shfl_sync(kAll, wb, w);
      if (j > 0 && !(prev - top > slack + (R)2.5e-7f * (fabs(prev) + fabs(top))) &&
          !(wl == prev_l && wb == prev_b))
        unsure = true;
      prev = top;
      prev_l = wl;
      prev_b = wb;
    }
    if (lane == j && j < a.k) {
      eid = e;
      my_l = wl;
    }
  }
  *expert = eid;
  *score = eid >= 0 ? score_of(a.scoring, (R)my_l, mx, z) : (R)0;
  return unsure;
}

template <int PER, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteArgs a) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  float l[PER], b[PER];
  uint32_t open = 0, summed = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane * PER + i;
    l[i] = -INFINITY;
    b[i] = 0.0f;
    if (e < a.E) {
      const size_t at = (size_t)t * (size_t)a.E + (size_t)e;
      l[i] = BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[at])
                  : static_cast<const float*>(a.logits)[at];
      if (a.bias != nullptr) b[i] = a.bias[e];
    }
    if (l[i] > -INFINITY) {  // neither -infinity nor NaN
      l[i] = fminf(l[i], 3.4028234e38f);
      summed |= 1u << i;
      if (b[i] > -INFINITY) {
        b[i] = fminf(b[i], 1e30f);
        open |= 1u << i;
      }
    }
  }
  int e;
  float p;
  if (route_row<PER, float>(a, l, b, open, summed, lane, &e, &p)) {
    double pd;
    route_row<PER, double>(a, l, b, open, summed, lane, &e, &pd);
    p = (float)pd;
  }
  if (a.renorm) p = p / (warp_sum(p) + 1e-20f);
  if (lane < a.k) {
    a.ids[t * a.k + lane] = e;
    a.weights[t * a.k + lane] = e >= 0 ? p * a.scale : 0.0f;
  }
}

template <int PER>
cudaError_t launch_per(const RouteArgs& a, bool bf16, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ceil_div(a.T, kWarps), 1, 1);
  cfg.blockDim = dim3(kWarps * 32, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, route_kernel<PER, true>, a)
              : cudaLaunchKernelEx(&cfg, route_kernel<PER, false>, a);
}

}  // namespace

cudaError_t launch_route(const void* logits, bool bf16, int64_t T, int E, const float* bias, int k,
                         int scoring, int groups, int keep, int group_top, int renorm, float scale,
                         int32_t* ids, float* weights, cudaStream_t s) {
  RouteArgs a = {};
  a.logits = logits;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.T = T;
  a.E = E;
  a.k = k;
  a.scoring = scoring;
  a.groups = groups;
  a.keep = keep;
  a.group_top = group_top;
  a.renorm = renorm;
  a.per_group = E / groups;
  a.scale = scale;
  if (E <= 32) return launch_per<1>(a, bf16, s);
  if (E <= 64) return launch_per<2>(a, bf16, s);
  if (E <= 128) return launch_per<4>(a, bf16, s);
  if (E <= 256) return launch_per<8>(a, bf16, s);
  if (E <= 512) return launch_per<16>(a, bf16, s);
  return launch_per<32>(a, bf16, s);
}

}  // namespace mxq
