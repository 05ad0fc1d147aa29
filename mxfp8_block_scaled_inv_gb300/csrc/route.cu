// Routing of tokens to experts: scores, balance bias, groups, top-k, weights.
// Rules are stated in include/mxq.h.
//
// Mathematics, per token over experts e:  p_e = score(l_e),  c_e = p_e + b_e;
// a group's value is the sum of its one or two largest c; of the groups the
// `keep` largest stay; the experts are the k largest c of those, ties going to
// the lowest index; w_j = scale * p_j (/ (sum p + 1e-20)).
//
// A warp takes a token; lane i holds up to PER neighbouring experts, so that lane
// order is index order, the lowest lane of a tie holds the lowest index, and
// groups (a power of two of them) are runs of lanes, whose two best are found by a
// butterfly over the run.  A lane's order-preserving keys are sorted by a network.
// Each pick is one warp-wide integer maximum of the lanes' first keys, one ballot,
// and a step on in the lane that lost an expert; lane j keeps pick j and computes
// its weight.
//
// What is chosen is defined by 64-bit scores: fp32 scores order two experts
// wrongly where they differ by less than their rounding.  So one pick more than
// asked for is made, and where two neighbouring picks, or the last one and an expert
// that is left, are nearer than the rounding bounds below, and not equal in logit and
// bias, picking goes on to the next clear gap and the lanes order their picks by 64-bit
// values, one for each lane.  Groups whose values lie that near to the edge between those kept and
// those left are ordered by the 64-bit sums of their best.  Where this does not
// settle it (no gap within 32 picks, a group with more than its best that near
// together, groups that do not lie on whole lanes) the row is done again in 64 bits
// altogether.  The device has next to no 64-bit units: such a row takes 30 to 40 us,
// as long as thousands of others.  Without a bias the experts are ordered by their
// logits, which is exact.
//
// Bound by what one warp does in a row: 1030 instructions for a row of 256 experts with
// bias and groups (sigmoids 7 % of the time, groups 18, nine picks 20), one behind the
// other where picks and ranks go by shuffles; some 57 % of the issue slots are used on cold
// caches, with the 32 warps of an SM that 64 registers leave.  8192 rows 14.5 us (1.3 us of
// memory), without groups 10.5, without bias and groups 9.0; BF16 logits whose scores tie
// 10.0; one row 3.0 us, of which launch and one trip to memory are 2.  What goes to whole
// rows in 64 bits shows: 8192 rows of BF16 logits around 10 with equal biases, some of
// which have more than 32 sigmoids next to 1, 140 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mxq.h"
#include "mxq_internal.h"
#include "mxq_ptx.cuh"
#include "quant_common.cuh"

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
  int E, k, scoring, groups, keep, group_top, renorm, per_group, vec, bias_vec, lanes;
  // Lane i holds up to `count` experts from run (i >> run_log) * run_len on, at
  // (i mod 2^run_log) * count in the run: a run is a group, or the whole row.
  int run_log, run_len, count;
  float scale;
  __device__ __forceinline__ int base(int lane) const {
    return (lane >> run_log) * run_len + (lane & ((1 << run_log) - 1)) * count;
  }
};

// Order-preserving 32-bit key of an fp32 value that is no NaN; that of -infinity,
// kNone, and what lies below stand for an expert that is not to be chosen.
constexpr uint32_t kNone = 0x007fffffu;
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 becomes 0
  return u ^ (0x80000000u | (uint32_t)((int32_t)u >> 31));
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// score(l); for the softmax mx is the row's maximum and z the sum of
// exp(l - mx), in fp32 its reciprocal.
__device__ __forceinline__ float score_of(int scoring, float l, float mx, float inv_z) {
  if (scoring == MXQ_SCORE_SOFTMAX) return expf(l - mx) * inv_z;
  if (scoring == MXQ_SCORE_SIGMOID) return __fdividef(1.0f, 1.0f + expf(-l));
  // Below -16 the score is exp(l / 2) to 2^-25 of itself, which fp32 holds down to l = -174;
  // exp(l) is subnormal from -87 on.
  const float e = expf(l < -16.0f ? 0.5f * l : -fabsf(l));
  return l < -16.0f ? e : sqrtf(fmaxf(l, 0.0f) + log1pf(e));
}
__device__ __noinline__ double score_of(int scoring, double l, double mx, double z) {
  if (scoring == MXQ_SCORE_SOFTMAX) return exp(l - mx) / z;
  if (scoring == MXQ_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
  return sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
}


__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t t, int e, bool bf16) {
  const size_t at = (size_t)t * (size_t)a.E + (size_t)e;
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[at])
              : static_cast<const float*>(a.logits)[at];
}
// Masked logits (-infinity, NaN) read -infinity, +infinity the largest number.
__device__ __forceinline__ float clean_logit(float l) {
  return fminf(fmaxf(l, -INFINITY), 3.4028234e38f);
}
__device__ __forceinline__ float clean_bias(float b) {
  return fminf(fmaxf(b, -INFINITY), 1e30f);
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

// The two largest of two pairs, each in order.
template <typename R>
__device__ __forceinline__ void merge2(R& a1, R& a2, R b1, R b2) {
  const R lo = b1 < a1 ? b1 : a1, hi2 = b2 > a2 ? b2 : a2;
  a1 = b1 > a1 ? b1 : a1;
  a2 = lo > hi2 ? lo : hi2;
}

// The value of a group of two that may be chosen: a sum past fp32's range (the lowest
// biases) is not that of a group with none, and its bounds leave it to 64 bits.
__device__ __forceinline__ float sum2(float a1, float a2) { return fmaxf(a1 + a2, -3.4028234e38f); }

// Order-preserving 64-bit key of a finite value, never 0, and back: comparisons of
// doubles run on the few 64-bit units, those of integers do not.
typedef unsigned long long Key64;
__device__ __forceinline__ Key64 key64_of(double v) {
  const Key64 u = (Key64)__double_as_longlong(v + 0.0);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ double value64_of(Key64 k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & ~(1ull << 63)) : ~k));
}

// A whole row with 64-bit scores: lane j < k returns the j-th expert (-1: none) and
// its score.  Lane i holds the experts i, i + 32, ...
__device__ __noinline__ void route_row_64(const RouteArgs& a, int64_t t, bool bf16, int lane,
                                          int* expert, float* score) {
  const int rounds = (a.E + 31) / 32;
  double mx = 0.0, z = 1.0;
  if (a.scoring == MXQ_SCORE_SOFTMAX) {
    float m = -INFINITY;
    for (int e = lane; e < a.E; e += 32) m = fmaxf(m, clean_logit(load_logit(a, t, e, bf16)));
    mx = (double)warp_max(m);
    double s = 0.0;
    for (int i = 0; i < rounds; ++i) {
      const int e = i * 32 + lane;
      const float l = e < a.E ? clean_logit(load_logit(a, t, e, bf16)) : -INFINITY;
      if (l > -INFINITY) s += score_of(a.scoring, (double)l, mx, 1.0);
    }
    z = warp_sum(s);
  }
  Key64 c[kMaxExperts / 32];  // 0: not to be chosen
  for (int i = 0; i < rounds; ++i) {
    const int e = i * 32 + lane;
    c[i] = 0;
    if (e < a.E) {
      const float l = clean_logit(load_logit(a, t, e, bf16));
      const float b = a.bias != nullptr ? clean_bias(a.bias[e]) : 0.0f;
      if (l > -INFINITY && b > -INFINITY)
        c[i] = key64_of(score_of(a.scoring, (double)l, mx, z) + (double)b);
    }
  }
  if (a.keep < a.groups) {
    Key64 mine = 0;  // lane g: the value of group g
    for (int g = 0; g < a.groups; ++g) {
      Key64 a1 = 0, a2 = 0;
      for (int i = 0; i < rounds; ++i) {
        const int at = i * 32 + lane - g * a.per_group;
        if (at >= 0 && at < a.per_group) merge2(a1, a2, c[i], (Key64)0);
      }
      for (int m = 16; m > 0; m >>= 1) {
        const Key64 o1 = __shfl_xor_sync(kAll, a1, m), o2 = __shfl_xor_sync(kAll, a2, m);
        merge2(a1, a2, o1, o2);
      }
      if (lane == g)
        mine = a.group_top == 2 && a2 != 0 ? key64_of(value64_of(a1) + value64_of(a2)) : a1;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const Key64 v = __shfl_sync(kAll, mine, g);
      rank += v > mine || (v == mine && g < lane) ? 1 : 0;
    }
    const uint32_t kept = __ballot_sync(kAll, lane < a.groups && rank < a.keep);
    for (int i = 0; i < rounds; ++i) {
      const int e = i * 32 + lane;
      if (e < a.E && !((kept >> (e / a.per_group)) & 1u)) c[i] = 0;
    }
  }
  if (a.bias == nullptr) {
    for (int i = 0; i < rounds; ++i)
      if (c[i] != 0) c[i] = key_of(clean_logit(load_logit(a, t, i * 32 + lane, bf16)));
  }
  *expert = -1;
  *score = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    Key64 best = 0;
    int at = 0;
    for (int i = 0; i < rounds; ++i)
      if (c[i] > best) {
        best = c[i];
        at = i;
      }
    const Key64 top = warp_max(best);
    if (top == 0) break;
    // The lowest index among the lanes that hold it.
    const int e = (int)__reduce_min_sync(kAll, best == top ? (uint32_t)(at * 32 + lane) : 0xffffffffu);
    if (lane == (e & 31)) c[e >> 5] = 0;
    if (lane == j) *expert = e;
  }
  if (*expert >= 0)
    *score = (float)score_of(a.scoring, (double)clean_logit(load_logit(a, t, *expert, bf16)), mx, z);
}

// Odd-even merge sort, largest first: passes of compare-exchanges at distance K
// inside blocks of 2 P.
template <int PER, int P, int K>
__device__ __forceinline__ void sort_pass(uint32_t (&v)[PER]) {
#pragma unroll
  for (int x = 0; x + K < PER; ++x) {
    if (x >= K % P && (x - K % P) % (2 * K) < K && x / (2 * P) == (x + K) / (2 * P)) {
      const uint32_t hi = max(v[x], v[x + K]), lo = min(v[x], v[x + K]);
      v[x] = hi;
      v[x + K] = lo;
    }
  }
  if constexpr (K > 1)
    sort_pass<PER, P, K / 2>(v);
  else if constexpr (2 * P < PER)
    sort_pass<PER, 2 * P, 2 * P>(v);
}

// The rare parts that follow read the row again instead of taking the caller's
// arrays, which stay in registers that way.

// A softmax row's sum of exponentials in 64 bits; lane i holds `per` experts.
__device__ __noinline__ double row_sum_64(const RouteArgs& a, int64_t t, bool bf16, int lane, int per,
                                          float mx) {
  double s = 0.0;
  for (int e = lane * per; e < min(lane * per + per, a.E); ++e) {
    const float l = clean_logit(load_logit(a, t, e, bf16));
    if (l > -INFINITY) s += score_of(MXQ_SCORE_SOFTMAX, (double)l, (double)mx, 1.0);
  }
  return warp_sum(s);
}

// Which groups stay where the bounds lo <= value <= hi of those kept and those left
// overlap: the groups that reach between `low`, the least bound of one kept, and
// `high`, the largest of one left, are ordered by the 64-bit sums of their n best (those
// with an fp32 value of `least` and more), the others stay where they are.  g: the lane's
// group; false in *sure where a group has more than its n best that near to each other.
__device__ __noinline__ bool keep_group_64(const RouteArgs& a, int64_t t, bool bf16, int lane, int per, int n_mine,
                                           float mx, float inv_z, int g, bool any, float lo, float hi,
                                           float low, float high, float least, int n, bool* sure) {
  const bool close = any && hi >= low && lo <= high, clear = any && lo > high;
  const double z = a.scoring == MXQ_SCORE_SOFTMAX && a.bias != nullptr
                       ? row_sum_64(a, t, bf16, lane, per, mx) : 1.0;
  double sum = 0.0;
  int found = 0;
  for (int i = 0; i < per; ++i) {
    const int e = a.base(lane) + i;
    float l = -INFINITY, b = 0.0f;
    if (close && i < n_mine) {
      l = clean_logit(load_logit(a, t, e, bf16));
      if (a.bias != nullptr) b = clean_bias(a.bias[e]);
    }
    const bool counts = l > -INFINITY && b > -INFINITY && score_of(a.scoring, l, mx, inv_z) + b >= least;
    if (__any_sync(kAll, counts)) {
      const double s = score_of(a.scoring, (double)l, (double)mx, z) + (double)b;
      if (counts) {
        sum += s;
        ++found;
      }
    }
  }
  for (int m = 1; m < a.lanes; m <<= 1) {
    sum += __shfl_xor_sync(kAll, sum, m);
    found += __shfl_xor_sync(kAll, found, m);
  }
  *sure = !__any_sync(kAll, close && found != n);
  const Key64 mine = close ? key64_of(sum) : 0;
  int rank = 0;
  for (int q = 0; q < a.groups; ++q) {
    const Key64 o = __shfl_sync(kAll, mine, q * a.lanes);
    rank += o > mine || (o == mine && q < g) ? 1 : 0;
  }
  const int above = __popc(__ballot_sync(kAll, clear)) / a.lanes;
  return clear || (close && rank < a.keep - above);
}

// Whether 64 bits have to order two fp32 values of c, the larger one first.
__device__ __forceinline__ bool too_near(float hi, float lo, float slack) {
  return !(hi - lo > slack + 1.2e-7f * (fabsf(hi) + fabsf(lo)));
}

// (The bound on registers is what the common path needs; the rare parts, whose calls
// would otherwise set it, keep more of theirs in memory.)
// EVEN: lane i begins at expert i * PER.
template <int PER, bool BF16, bool EVEN>
__global__ void __launch_bounds__(kWarps * 32, PER <= 8 ? 8 : PER <= 16 ? 6 : 4) route_kernel(const RouteArgs a) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const bool biased = a.bias != nullptr, grouped = a.keep < a.groups;
  const int e0 = EVEN ? lane * PER : a.base(lane);
  // The lane's experts: what is left of its run.
  const int n = EVEN ? min(PER, a.E - e0)
                     : min(a.count, a.run_len - (lane & ((1 << a.run_log) - 1)) * a.count);
  float l[PER];
  if (PER % 4 == 0 && a.vec && n == PER) {
    const size_t at = (size_t)t * (size_t)a.E + (size_t)e0;
    if constexpr (BF16) {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.logits) + at;
      if constexpr (PER % 8 == 0) {
#pragma unroll
        for (int i = 0; i < PER; i += 8) {
          float v[8];
          unpack8(*reinterpret_cast<const uint4*>(src + i), v);
#pragma unroll
          for (int q = 0; q < 8; ++q) l[i + q] = v[q];
        }
      } else if constexpr (PER % 4 == 0) {
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
          const uint2 v = *reinterpret_cast<const uint2*>(src + i);
          l[i] = bf16_lo(v.x);
          l[i + 1] = bf16_hi(v.x);
          l[i + 2] = bf16_lo(v.y);
          l[i + 3] = bf16_hi(v.y);
        }
      }
    } else if constexpr (PER % 4 == 0) {
      const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + at);
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        const float4 v = src[i / 4];
        l[i] = v.x;
        l[i + 1] = v.y;
        l[i + 2] = v.z;
        l[i + 3] = v.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = i < n ? load_logit(a, t, e0 + i, BF16) : -INFINITY;
  }
  float b[PER];
  if (PER % 4 == 0 && biased && a.bias_vec && n == PER) {
#pragma unroll
    for (int i = 0; i + 4 <= PER; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(a.bias + e0 + i));
      b[i] = v.x;
      b[i + 1] = v.y;
      b[i + 2] = v.z;
      b[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) b[i] = biased && i < n ? __ldg(a.bias + e0 + i) : 0.0f;
  }
  // The row's largest logit bounds the scores; the softmax needs it anyway.
  float mx = -INFINITY, inv_z = 1.0f, pmax = 1.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) l[i] = clean_logit(l[i]);
  if (a.scoring != MXQ_SCORE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < PER; ++i) mx = fmaxf(mx, l[i]);
    const uint32_t top = __reduce_max_sync(kAll, mx == -INFINITY ? 0u : key_of(mx));
    mx = top == 0u ? 0.0f : value_of(top);
    if (a.scoring == MXQ_SCORE_SOFTMAX) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) s += expf(l[i] - mx);
      inv_z = 1.0f / warp_sum(s);
      pmax = inv_z;
    } else {
      pmax = score_of(a.scoring, mx, 0.0f, 1.0f);
    }
  }
  // Bounds on the error of an fp32 difference of two scores, relative to the
  // largest: exp 2 ulp, log1p 1 ulp, reciprocal 1 ulp, sums of up to 37 roundings.
  const float slack = pmax * (a.scoring == MXQ_SCORE_SIGMOID   ? 1e-6f
                              : a.scoring == MXQ_SCORE_SOFTMAX ? 6e-6f
                                                               : 2.5e-6f);
  bool whole = false;  // the row needs 64 bits altogether
  // Order of the lane's experts.
  uint32_t key[PER];
  const bool spread = grouped && a.lanes == 0;  // groups begin or end inside a lane
  float c[PER];
  if (biased || spread) {
    // (One loop for each score: a choice inside it is made once for each value.)
    if (a.scoring == MXQ_SCORE_SIGMOID) {
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] = score_of(MXQ_SCORE_SIGMOID, l[i], mx, inv_z);
    } else if (a.scoring == MXQ_SCORE_SOFTMAX) {
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] = score_of(MXQ_SCORE_SOFTMAX, l[i], mx, inv_z);
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] = score_of(MXQ_SCORE_SQRTSOFTPLUS, l[i], mx, inv_z);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = l[i] > -INFINITY ? c[i] + clean_bias(b[i]) : -INFINITY;
  }
  if (biased) {
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = key_of(c[i]);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = key_of(l[i]);
  }
  // Which groups stay: v is the value of group g, a1 and a2 its best, `step` the lanes
  // of a group.  True where lane's group stays.
  auto group_kept = [&](float v, int g, float a1, float a2, int step) {
    int rank = 0;  // the lanes of a group share the comparisons
    for (int i = 0; i < a.groups; i += step) {
      const int q = i + (lane & (step - 1));
      const float o = __shfl_sync(kAll, v, (q * step) & 31);
      rank += q < a.groups && (o > v || (o == v && q < g)) ? 1 : 0;
    }
    for (int m = 1; m < step; m <<= 1) rank += __shfl_xor_sync(kAll, rank, m);
    bool kept = rank < a.keep;
    // Two scores' share of the value's error, and the roundings of its terms (a score
    // and a bias each, which may cancel) and of their sum.
    const bool any = g < a.groups && v > -INFINITY, two = a.group_top == 2 && a2 > -INFINITY;
    const float err = slack + 2.5e-7f * (fabsf(a1) + (two ? fabsf(a2) : 0.0f));
    const uint32_t low = __reduce_min_sync(kAll, kept && g < a.groups ? (any ? key_of(v - err) : 0u) : 0xffffffffu);
    const uint32_t high = __reduce_max_sync(kAll, !kept && any ? key_of(v + err) : 0u);
    if (low != 0u && low <= high) {
      bool sure = false;  // (groups that do not lie on lanes: the whole row)
      if (a.lanes > 0) {
        const float last = two ? a2 : a1;
        kept = keep_group_64(a, t, BF16, lane, PER, n, mx, inv_z, g, any, v - err, v + err, value_of(low),
                             value_of(high), last - (2.0f * slack + 5e-7f * fabsf(last)), two ? 2 : 1, &sure);
      }
      whole = !sure;
    }
    return kept;
  };
  if (spread) {
    float v = -INFINITY, v1 = -INFINITY, v2 = -INFINITY;
    for (int q = 0; q < a.groups; ++q) {
      float a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int at = e0 + i - q * a.per_group;
        if (at >= 0 && at < a.per_group) {
          a2 = fmaxf(a2, fminf(a1, c[i]));
          a1 = fmaxf(a1, c[i]);
        }
      }
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) {
        const float o1 = __shfl_xor_sync(kAll, a1, m), o2 = __shfl_xor_sync(kAll, a2, m);
        merge2(a1, a2, o1, o2);
      }
      if (lane == q) {
        v = a.group_top == 2 && a2 > -INFINITY ? sum2(a1, a2) : a1;
        v1 = a1;
        v2 = a2;
      }
    }
    const uint32_t mask =
        __ballot_sync(kAll, group_kept(v, lane, v1, v2, 1) && lane < a.groups);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (!((mask >> (min(e0 + i, a.E - 1) / a.per_group)) & 1u)) key[i] = 0u;
  }
  // Each lane's keys in order, so that a pick is their head; which expert the
  // key belongs to is looked up for all picks at once afterwards.
  uint32_t head[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) head[i] = key[i];
  if constexpr (PER > 1) sort_pass<PER, 1, 1>(head);
  if (grouped && !spread) {
    // A group is a run of 2^n lanes, whose two best are among theirs.
    auto value = [&](uint32_t k) {
      if (k <= kNone) return -INFINITY;
      return biased ? value_of(k) : score_of(a.scoring, value_of(k), mx, inv_z);
    };
    float a1 = value(head[0]), a2 = PER > 1 ? value(head[PER > 1 ? 1 : 0]) : -INFINITY;
    for (int m = 1; m < a.lanes; m <<= 1) {
      const float o1 = __shfl_xor_sync(kAll, a1, m), o2 = __shfl_xor_sync(kAll, a2, m);
      merge2(a1, a2, o1, o2);
    }
    const float v = a.group_top == 2 && a2 > -INFINITY ? sum2(a1, a2) : a1;
    if (!group_kept(v, lane >> a.run_log, a1, a2, a.lanes)) head[0] = 0u;  // hides the others
  }
  int expert = -1, picks = 0;
  uint32_t my_key = 0u, my_from = 0u;  // this lane's pick, and the bit of the lane that holds it
  float cj = 0.0f;
  // Takes the next expert into lane `picks`; false where none is left.
  auto pick = [&]() {
    const uint32_t top = __reduce_max_sync(kAll, head[0]);
    if (top <= kNone) return false;
    const uint32_t at = __ballot_sync(kAll, head[0] == top), first = at & (0u - at);
    if (first == 1u << lane) {
#pragma unroll
      for (int i = 0; i + 1 < PER; ++i) head[i] = head[i + 1];
      head[PER - 1] = 0u;
    }
    if (lane == picks) {
      my_key = top;
      my_from = first;
    }
    ++picks;
    return true;
  };
  auto look_up = [&]() {
    const int my_lane = my_from != 0u ? __ffs(my_from) - 1 : 0;
    cj = my_key != 0u ? value_of(my_key) : 0.0f;
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      m |= (__shfl_sync(kAll, key[i], my_lane) == my_key ? 1u : 0u) << i;
    // Equal keys of one lane are picked one behind the other.
    const uint32_t prev = __shfl_up_sync(kAll, my_key, 1);
    const uint32_t prev_from = __shfl_up_sync(kAll, my_from, 1);
    const bool again = lane > 0 && prev == my_key && prev_from == my_from && my_key != 0u;
    const uint32_t run = __ballot_sync(kAll, again);
    if (again) {
      // Length of the run of `again` that ends here.
      const int skip = __clz(~(run << (31 - lane)));
      for (int i = 0; i < skip; ++i) m &= m - 1u;
    }
    expert = my_key != 0u ? (EVEN ? my_lane * PER : a.base(my_lane)) + __ffs(m) - 1 : -1;
  };
  const int want = biased ? a.k + 1 : a.k;
  while (picks < want && picks < 32 && pick()) {
  }
  look_up();
  int place = lane;  // of this lane's pick in the output
  float lj = 0.0f, bj = 0.0f;
  auto near = [&](float hi, float lo) { return too_near(hi, lo, slack); };
  // Whether the last pick is too near to the best expert that is left.
  auto near_rest = [&]() {
    const uint32_t rest = __reduce_max_sync(kAll, head[0]);
    return rest > kNone && near(__shfl_sync(kAll, cj, picks - 1), value_of(rest));
  };
  if (biased && !whole) {
    // Lane j > 0: whether picks j - 1 and j are too near to call.
    auto near_prev = [&]() {
      const float pc = __shfl_up_sync(kAll, cj, 1);
      return lane > 0 && lane < picks && near(pc, cj);
    };
    auto fetch = [&]() {
      if (expert >= 0) {
        lj = clean_logit(load_logit(a, t, expert, BF16));
        bj = clean_bias(a.bias[expert]);
      }
    };
    // Whether an expert that is left is near the last pick without being the same in
    // logit and bias.  (Among the lane's keys up to the last pick's only picks that are the
    // same as that one are not left.)
    auto other_near_rest = [&]() {
      const uint32_t last = __shfl_sync(kAll, my_key, picks - 1);
      const float ll = __shfl_sync(kAll, lj, picks - 1), lb = __shfl_sync(kAll, bj, picks - 1);
      bool other = false;
      uint32_t same = 0u;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (key[i] == last)
          same |= 1u << i;
        else if (key[i] > kNone && key[i] < last)
          other |= near(value_of(last), value_of(key[i]));
      }
      if (head[0] <= kNone) {  // nothing of this lane is left, or its group is out
        other = false;
        same = 0u;
      }
      for (; same != 0u; same &= same - 1u) {
        const int e = e0 + __ffs(same) - 1;
        other |= clean_logit(load_logit(a, t, e, BF16)) != ll || clean_bias(a.bias[e]) != lb;
      }
      return __any_sync(kAll, other) != 0;
    };
    const uint32_t near_picks = __ballot_sync(kAll, near_prev());
    // No room for a pick behind the k-th, and what is left may be as large.
    const bool full = picks == a.k && picks == 32 && near_rest();
    if (near_picks != 0u || full) {
      fetch();
      // Equal logits and biases are ties that indices settle, among the picks and
      // beyond the last one.
      const float pl = __shfl_up_sync(kAll, lj, 1), pb = __shfl_up_sync(kAll, bj, 1);
      const bool last_near = full || (picks > a.k && ((near_picks >> (picks - 1)) & 1u) && near_rest());
      if (__any_sync(kAll, ((near_picks >> lane) & 1u) && !(pl == lj && pb == bj)) ||
          (last_near && other_near_rest())) {
        // On to the first clear gap behind the k-th pick.
        while (picks > a.k && picks < 32 && __shfl_sync(kAll, (int)near_prev(), picks - 1) && pick()) {
          look_up();
        }
        if ((picks == a.k || __shfl_sync(kAll, (int)near_prev(), picks - 1)) && near_rest()) {
          whole = true;
        } else {
          fetch();
          const double z = a.scoring == MXQ_SCORE_SOFTMAX ? row_sum_64(a, t, BF16, lane, PER, mx) : 1.0;
          const Key64 c =
              expert >= 0 ? key64_of(score_of(a.scoring, (double)lj, (double)mx, z) + (double)bj) : 0;
          int rank = 0;
          for (int j = 0; j < picks; ++j) {
            const Key64 o = __shfl_sync(kAll, c, j);
            const int oe = __shfl_sync(kAll, expert, j);
            rank += o > c || (o == c && oe < expert) ? 1 : 0;
          }
          place = expert >= 0 ? rank : 32;
        }
      }
    }
  }
  float p = 0.0f;
  if (whole) {
    route_row_64(a, t, BF16, lane, &expert, &p);
    place = lane;
  } else if (expert >= 0) {
    const float l1 = clean_logit(load_logit(a, t, expert, BF16));
    p = score_of(a.scoring, l1, mx, inv_z);
    if (a.scoring == MXQ_SCORE_SOFTMAX) {
      // exp(l - mx) = exp(d) (1 + lack), lack being what the rounding of d took away: up to
      // 2^-18 at differences of 64 and more.  (The choice does without: the bounds above
      // go by the row's largest score, beside which such ones are nothing.)
      const float d = l1 - mx, back = d - l1, lack = (l1 - (d - back)) - (mx + back);
      p = p > 0.0f ? fmaf(p, lack, p) : 0.0f;
    }
  }
  if (place >= a.k) p = 0.0f;
  if (a.renorm) p = p / (warp_sum(p) + 1e-20f);
  if (lane < a.k && expert < 0) place = lane;  // behind the last expert
  if (place < a.k) {
    a.ids[t * a.k + place] = expert;
    a.weights[t * a.k + place] = expert >= 0 ? p * a.scale : 0.0f;
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
  if (a.count == PER && (a.run_log == 5 || a.run_len == PER << a.run_log))
    return bf16 ? cudaLaunchKernelEx(&cfg, route_kernel<PER, true, true>, a)
                : cudaLaunchKernelEx(&cfg, route_kernel<PER, false, true>, a);
  return bf16 ? cudaLaunchKernelEx(&cfg, route_kernel<PER, true, false>, a)
              : cudaLaunchKernelEx(&cfg, route_kernel<PER, false, false>, a);
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
  // Groups that are a power of two of them get equal runs of lanes; others are found
  // by a search of all lanes for each (8192 x 160 in 8 groups 31 us, with runs 14.5).
  // Room for 12 experts beside 8 and 16: 8192 x 384 17.5 us, and 24.2 with 16.
  const bool select = keep < groups, runs = select && (groups & (groups - 1)) == 0;
  a.run_log = 5;
  while (runs && (32 >> a.run_log) < groups) --a.run_log;
  a.run_len = runs ? a.per_group : E;
  a.lanes = runs ? 1 << a.run_log : 0;
  const int need = (int)ceil_div(a.run_len, 1 << a.run_log);
  const int per = need <= 2 ? need : need <= 4 ? 4 : need <= 8 ? 8 : need <= 12 ? 12 : need <= 16 ? 16 : 32;
  // A lane takes all it has room for where a group ends with a lane (vector loads), else
  // an even share.
  a.count = a.run_len % per == 0 || !runs ? per : need;
  // Loads of four and eight logits and four biases (a bias may begin at any element).
  a.vec = E % 8 == 0 && a.count == per && a.run_len % 4 == 0 && (a.run_len % 8 == 0 || !bf16);
  a.bias_vec = a.vec && (reinterpret_cast<uintptr_t>(bias) & 15u) == 0;
  if (per == 1) return launch_per<1>(a, bf16, s);
  if (per == 2) return launch_per<2>(a, bf16, s);
  if (per == 4) return launch_per<4>(a, bf16, s);
  if (per == 8) return launch_per<8>(a, bf16, s);
  if (per == 12) return launch_per<12>(a, bf16, s);
  if (per == 16) return launch_per<16>(a, bf16, s);
  return launch_per<32>(a, bf16, s);
}

}  // namespace mxq
