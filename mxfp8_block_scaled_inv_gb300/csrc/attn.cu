// Attention over the paged KV cache (mxq_attn): sliding window, first keys
// that stay visible, causal within the new tokens.  Keys and values are the
// same cache row, shared by all query heads.
//
//   s_j = sm_scale * (q . k_j),  out = sum_j exp(s_j - lse) k_j,
//   lse = log(sum_j exp(s_j)) over the visible keys j.
//
// A tile is up to NR rows (token-major, heads within a token) of one
// sequence.  Its visible keys are walked in blocks of 128, made of units of
// 16 consecutive keys (units never straddle a page): first the units of the
// sinks, then those of the window.  Both products run on the tensor cores with the
// keys, respectively the columns, on the M axis, so that the matrix
// instructions run at full width whatever the number of heads:
//
//   S^T [128 keys x NR]  = K [128 x D]  Q^T        (A = the block's rows)
//   O^T [D x NR]        += K^T [D x 128] P^T       (A = the same shared-memory
//                                                   rows, read transposed)
//
// so a cache row is fetched once for both products and for all rows of the
// tile.  P = 2^(x + negm), x = s * log2(e): negm is minus a running maximum
// per row that is only moved when some score passes it by more than 2^8, so
// that most blocks need neither a cross-lane maximum nor a rescale of O.
// Row sums are kept per thread (one key each) in FP32 and joined at the end.
//
// Warps: 0-7 softmax and epilogue (a lane is a key, then a column; the two
// groups of four own half of the tile's rows each and never wait for one
// another), 8 issues the matrix instructions, 9 the TMA copies of BF16 rows, 10
// decodes the work items, 12-15 fetch Q and the cache rows that are widened to
// 16 bits, into the 128-byte-swizzled layout.
//
// E4M3 rows are widened to FP16 (exact), with the query scaled per row by a
// power of two into FP16's range (exact for all values within 2^24 of the
// row's largest) and P shifted by 2^6; BF16 and E2M1 rows and their P are
// BF16 (E2M1 times its scale is exact in BF16).  P's rounding (2^-9 in BF16)
// is of the order of the output's own.
//
// When there are fewer tiles than SMs the keys of a tile are split over
// several CTAs, whose FP32 partial sums a second kernel joins in a fixed order.
//
// Every wait is bounded in wall time; on expiry the kernel sets a watchdog
// bit, stops, waits for the matrix instructions in flight, frees TMEM and
// returns.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "mxq.h"
#include "mxq_internal.h"
#include "mxq_ptx.cuh"
#include "quant_common.cuh"

namespace mxq {

// The driver's tensor-map encoder (bmm.cu), NULL where the driver lacks it.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace {

constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint32_t kHintNs = 20;
constexpr uint32_t kWdAttn = 64;  // watchdog bit of this kernel

constexpr int kKeys = 128;           // keys of a block (M of the first product)
constexpr int kUnit = 16;            // keys of a unit
constexpr int kUnits = kKeys / kUnit;
constexpr int kChunkBytes = kKeys * 128;   // 128 keys x 64 columns of 16 bits
constexpr int kStageBytes = 2 * kChunkBytes;
constexpr int kSoftWarps = 8, kMmaWarp = 8, kTmaWarp = 9, kItemWarp = 10, kUnitWarp = 11,
              kLoadWarp0 = 12, kLoadWarps = 4;
constexpr int kThreads = (kLoadWarp0 + kLoadWarps) * 32;
// Registers per thread: 128 at launch; softmax 168, the issuing warps 40, the
// loading warps 136.  Nothing spills: with 227 KB of shared memory in use the
// L1 cache is too small for local memory.
constexpr int kRegsSoft = 168, kRegsIssue = 40, kRegsLoad = 136;
static_assert(256 * kRegsSoft + 128 * kRegsIssue + 128 * kRegsLoad <= kThreads * 128, "register pool");
constexpr int kLoadThreads = kLoadWarps * 32;
constexpr int kMaxStages = 6;
constexpr uint32_t kTmemCols = 512, kTmemS = 256;
constexpr float kNoKey = 1e30f;      // negm of a row that has seen no key
constexpr float kSlack = 8.0f;       // log2 of how far a score may pass the maximum
constexpr float kLog2e = 1.4426950408889634f;

struct KernelArgs {
  AttnArgs a;
  float* part;      // split form: [tiles][splits][NR][D] partial sums
  float2* part_ml;  // [tiles][splits][NR] (maximum, sum)
  uint32_t* watchdog;
  int tiles, splits, stages, items;
};

__host__ __device__ constexpr int q_bytes(int NR, int D) { return NR * D * 2; }

// What one work item (a tile and a share of its key blocks) covers.
struct alignas(16) Item {
  int b, r0, nrows, pos0;  // sequence, first row in it, rows, position of its first new token
  int p0, p1;              // positions of the tile's first and last row
  int u_lo, ns;            // first unit of the window, units of the sinks
  int units, blk0, blk1;   // units in all; this item's blocks of 8
  int tile, split, pad;
  int64_t qrow;            // first row of the tile in [T*H]
};
static_assert(sizeof(Item) == 64, "four 16-byte words");
constexpr int kItems = 4;  // items handed out ahead
constexpr int kSlots = 4;  // blocks whose units are looked up ahead

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], s_full[2], p_full, pv_done, q_full[4], q_empty, drain;
  uint64_t item_full[kItems], item_empty[kItems], slot_full[kSlots], slot_empty[kSlots];
  uint32_t tmem;
  int abort;
  alignas(16) Item items[kItems];
  int slots[kSlots][kUnits];  // cache row of each unit's first key, -1: none
  float crow[3][64];
  float negm[64];
  float scale[64];  // the rescale factors of a block; in the epilogue 1 / sum
  uint8_t rowt[64];  // a row's token, counted from the tile's first
  float red[2][4][32];
};

// The weights P are held as two 16-bit parts, hi + lo: for NR <= 32 side by
// side in one 128-byte row per key, for NR = 64 in two such buffers.
constexpr int p_bytes(int NR) { return NR == 64 ? 2 * kKeys * 128 : kKeys * 128; }
constexpr int kSmemBudget = 232448;
__host__ __device__ constexpr int smem_fixed(int NR, int D) {
  return p_bytes(NR) + q_bytes(NR, D) + (int)sizeof(Shared);
}
inline int stages_for(int NR, int D) {
  const int n = (kSmemBudget - smem_fixed(NR, D)) / kStageBytes;
  return n < kMaxStages ? n : kMaxStages;
}
static_assert(smem_fixed(64, 512) + 4 * kStageBytes <= kSmemBudget, "a block of the widest rows fits");

__device__ __forceinline__ int seq_start(const AttnArgs& a, int b) {
  return a.q_start != nullptr ? __ldg(a.q_start + b) : b;
}

// Called by whole warps.
template <int NR>
__device__ __forceinline__ Item get_item(const KernelArgs& k, int item) {
  const AttnArgs& a = k.a;
  Item it;
  it.split = item / k.tiles;
  // Later tiles of a chunk see more keys: they go first.
  it.tile = k.tiles - 1 - (item - it.split * k.tiles);
  // Tiles are numbered so that sequence b begins at floor(start_b * H / NR) + b:
  // each has at least as many numbers as tiles, without a prefix sum.
  const int lane = threadIdx.x & 31;
  int b = 0;
  if (a.q_start == nullptr && NR >= 1) {
    // start_b = b: the number of b's whose first tile is at or before this one.
    const int64_t t = it.tile;
    b = (int)min((int64_t)a.B - 1, t * NR / (a.H + NR));
    while (b + 1 < a.B && ((int64_t)(b + 1) * a.H) / NR + b + 1 <= t) ++b;
    while (b > 0 && ((int64_t)b * a.H) / NR + b > t) --b;
  } else {
    for (int base = 0; base < a.B; base += 32) {
      const int i = base + lane;
      const bool before =
          i < a.B && ((int64_t)max(__ldg(a.q_start + min(i, a.B - 1)), 0) * a.H) / NR + i <= it.tile;
      const int c = __popc(__ballot_sync(0xffffffffu, before));
      if (c == 0) break;
      b = base + c - 1;
      if (c < 32) break;
    }
  }
  it.b = b;
  const int start = max(seq_start(a, b), 0);
  const int end = (int)min((int64_t)seq_start(a, b + 1), a.T);
  const int n = max(end - start, 0);
  const int cap = a.max_pages * a.page_size;
  const int said = __ldg(a.seq_lens + b), len = min(max(said, 0), cap);
  const int64_t r0 = ((int64_t)it.tile - b - ((int64_t)start * a.H) / NR) * NR;
  const int64_t rows = (int64_t)n * a.H;
  it.pos0 = len - n;
  it.pad = said != len;
  it.nrows = r0 >= 0 && r0 < rows ? (int)min((int64_t)NR, rows - r0) : 0;
  it.r0 = (int)r0;
  it.qrow = (int64_t)start * a.H + r0;
  it.units = it.ns = it.u_lo = it.blk0 = it.blk1 = 0;
  it.p0 = it.p1 = -1;
  if (it.nrows > 0) {
    it.p0 = it.pos0 + it.r0 / a.H;
    it.p1 = it.pos0 + (it.r0 + it.nrows - 1) / a.H;
    if (it.p1 >= 0) {
      const int lo = a.window > 0 ? max(0, it.p0 - a.window + 1) : 0;
      it.u_lo = lo / kUnit;
      const int sink_end = a.window > 0 ? min(a.sinks, lo) : 0;
      it.ns = min((sink_end + kUnit - 1) / kUnit, it.u_lo);
      it.units = it.ns + it.p1 / kUnit + 1 - it.u_lo;
      const int nb = (it.units + kUnits - 1) / kUnits;
      const int per = (nb + k.splits - 1) / k.splits;
      it.blk0 = min(nb, it.split * per);
      it.blk1 = min(nb, it.blk0 + per);
    }
  }
  return it;
}

// First key of unit x of the item.
template <typename I>
__device__ __forceinline__ int unit_key(const I& it, int x) {
  return (x < it.ns ? x : it.u_lo + (x - it.ns)) * kUnit;
}

// ------------------------------------------------------------- instructions
// D[tmem] (+)= A B^T with 16-bit operands.  The descriptors come as their low
// words (address, leading offset) and constant high words, so that stepping
// through a tile is one 32-bit addition each: a single thread issues all of
// the CTA's products, 64 to 96 in a block, and 64-bit descriptor arithmetic
// in front of each took as long as the product (80 cycles).
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                        uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 a, b;\n"
      "mov.b64 a, {%1, %2};\nmov.b64 b, {%3, %4};\n"
      "setp.ne.b32 p, %6, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Low and high words of a descriptor with 128-byte swizzle: address and
// leading offset; stride offset 1024 (eight 128-byte rows).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (ptx::kSwizzle128B << 29);

// Instruction descriptor of kind::f16: FP32 accumulation, both operands BF16
// (1) or FP16 (0), M = 128, N, and whether A and B are stored with M / N
// running fastest.
__host__ __device__ constexpr uint32_t idesc_f16(bool bf16, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[N]) {
  static_assert(N == 8 || N == 16 || N == 32, "");
  if constexpr (N == 8) ptx::tmem_ld_32x32b_x8(addr, r);
  if constexpr (N == 16) ptx::tmem_ld_32x32b_x16(addr, r);
  if constexpr (N == 32) ptx::tmem_ld_32x32b_x32(addr, r);
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Barrier of `count` threads that also tells whether any of them passed true.
__device__ __forceinline__ bool named_any(uint32_t id, uint32_t count, bool v) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 q, %3, 0;\n"
      "barrier.cta.red.or.pred p, %1, %2, q;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(count), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Maximum that is NaN if either operand is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// Maximum (or sum) over the 32 lanes of N values each, by halving exchanges:
// lane c < N ends with value c.  31 shuffles for 32 values.
template <int N, bool MAX>
__device__ __forceinline__ float lanes_reduce(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    if (off >= N) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float o = __shfl_xor_sync(0xffffffffu, v[i], off);
        v[i] = MAX ? fmaxf(v[i], o) : v[i] + o;
      }
    } else {
#pragma unroll
      for (int i = 0; i < off; ++i) {
        const bool up = lane & off;
        const float o = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + off], off);
        const float mine = up ? v[i + off] : v[i];
        v[i] = MAX ? fmaxf(mine, o) : mine + o;
      }
    }
  }
  return v[0];
}
// 16 lanes x N columns of TMEM: per 8 columns, registers 0-1 hold lane t / 4,
// columns 2 (t % 4) and + 1; registers 2-3 the same of lane t / 4 + 8.
template <int N>
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t addr, uint32_t (&r)[N / 2]) {
  static_assert(N == 8 || N == 16 || N == 32, "");
  if constexpr (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
  if constexpr (N == 16)
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
  if constexpr (N == 32)
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
// Two 8 x 8 matrices of 16-bit values, transposed on the way to shared memory.
__device__ __forceinline__ void stmatrix_x2_trans(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b)
               : "memory");
}
__device__ __forceinline__ float out_of(bool has, uint32_t v) { return has ? __uint_as_float(v) : 0.0f; }
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack16(bool bf16, float lo, float hi) {
  uint32_t r;
  if (bf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// What is left of two values after pack16, packed the same way.
__device__ __forceinline__ uint32_t pack16_rest(bool bf16, float lo, float hi, uint32_t w) {
  if (bf16) return pack16(true, lo - bf16_lo(w), hi - bf16_hi(w));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pack16(false, lo - f.x, hi - f.y);
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(ptx::smem_u32(dst)),
      "l"(m), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

// --------------------------------------------------------------- widening
// 16 E4M3 codes -> 16 FP16 values (exact).
__device__ __forceinline__ void widen_e4m3(const uint4& v, uint4& lo, uint4& hi) {
  uint32_t o[8];
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(o[2 * i]) : "h"((uint16_t)(w[i] & 0xFFFFu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(o[2 * i + 1]) : "h"((uint16_t)(w[i] >> 16)));
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// Table of the eight magnitudes times 2^(sb - 127) as BF16, split into low and
// high bytes for byte selection: BF16 holds each exactly (infinity past its
// range, NaN for sb = 255).
struct E2m1Table {
  uint32_t lo0, lo1, hi0, hi1;
};
__device__ __forceinline__ E2m1Table e2m1_table(uint32_t sb) {
  // 2^(sb-127) as BF16; sb = 0 is the subnormal 2^-127.
  const uint32_t s1 = sb == 255u ? 0x7FFFu : sb == 0u ? 0x0040u : sb << 7;
  const uint32_t s = s1 | (s1 << 16);
  uint32_t t01, t23, t45, t67;  // (0, .5), (1, 1.5), (2, 3), (4, 6)
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(t01) : "r"(s), "r"(0x3F000000u));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(t23) : "r"(s), "r"(0x3FC03F80u));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(t45) : "r"(s), "r"(0x40404000u));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(t67) : "r"(s), "r"(0x40C04080u));
  E2m1Table t;
  t.lo0 = __byte_perm(t01, t23, 0x6420);
  t.lo1 = __byte_perm(t45, t67, 0x6420);
  t.hi0 = __byte_perm(t01, t23, 0x7531);
  t.hi1 = __byte_perm(t45, t67, 0x7531);
  return t;
}
// Four codes (the low 16 bits of w) -> four BF16 values.
__device__ __forceinline__ uint2 widen_e2m1x4(uint32_t w, const E2m1Table& t) {
  const uint32_t sel = w & 0x7777u;
  const uint32_t lo = __byte_perm(t.lo0, t.lo1, sel);
  uint32_t hi = __byte_perm(t.hi0, t.hi1, sel);
  // The code's sign bit is the selector's replicate-the-top-bit flag: 0x80
  // becomes 0xFF for a negative code, whose lowest bit is then the sign.
  uint32_t sg;
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(sg) : "r"(0x80808080u), "r"(w));
  hi |= (sg << 7) & 0x80808080u;
  return make_uint2(__byte_perm(lo, hi, 0x5140), __byte_perm(lo, hi, 0x7362));
}

// Cache rows that a loading thread handles in every block.
template <int DT>
constexpr int kRowsPerThread = DT == MXQ_CACHE_E4M3 ? 8 : 4;

// ------------------------------------------------------------------ kernel
template <int NR, int DT>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap tm_kv, const KernelArgs k) {
  constexpr bool BF = DT != MXQ_CACHE_E4M3;  // operand type: BF16, else FP16
  constexpr int NC = NR / 2;                 // rows of a softmax group
  constexpr int NV = NR == 64 ? 64 : 2 * NR; // N of the second product
  constexpr float kShift = BF ? 0.0f : 6.0f;
  extern __shared__ __align__(1024) uint8_t base[];
  const AttnArgs& a = k.a;
  const int D = a.D, nch = D >> 6, np = (nch + 1) >> 1;
  uint8_t* sm_stage = base;
  uint8_t* sm_p = sm_stage + (size_t)k.stages * kStageBytes;
  uint8_t* sm_q = sm_p + p_bytes(NR);
  Shared& sh = *reinterpret_cast<Shared*>(sm_q + q_bytes(NR, D));
  volatile int* abort_flag = &sh.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    sh.abort = 0;
    for (int s = 0; s < k.stages; ++s) {
      ptx::mbar_init(&sh.full[s], DT == MXQ_CACHE_BF16 ? 1 : kLoadThreads);
      ptx::mbar_init(&sh.empty[s], 1);
    }
    ptx::mbar_init(&sh.s_full[0], 1);
    ptx::mbar_init(&sh.s_full[1], 1);
    ptx::mbar_init(&sh.p_full, kSoftWarps * 32);
    ptx::mbar_init(&sh.pv_done, 1);
    for (int s = 0; s < 4; ++s) ptx::mbar_init(&sh.q_full[s], kLoadThreads);
    ptx::mbar_init(&sh.q_empty, 1);
    ptx::mbar_init(&sh.drain, 1);
    for (int i = 0; i < kItems; ++i) {
      ptx::mbar_init(&sh.item_full[i], 1);
      // Readers: the softmax, loading, issuing and unit warps, and the TMA warp.
      ptx::mbar_init(&sh.item_empty[i], kSoftWarps + kLoadWarps + 2 + (DT == MXQ_CACHE_BF16 ? 1 : 0));
    }
    for (int i = 0; i < kSlots; ++i) {
      ptx::mbar_init(&sh.slot_full[i], 1);
      ptx::mbar_init(&sh.slot_empty[i], kSoftWarps + (DT == MXQ_CACHE_BF16 ? 1 : kLoadWarps));
    }
    ptx::fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&sh.tmem, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();

  // A bounded wait; false once it or any other wait of the CTA gave up.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (*abort_flag) return false;
    if (ptx::mbar_wait_hint(bar, parity, kWaitNs, kHintNs)) return true;
    *abort_flag = 1;
    atomicOr(k.watchdog, kWdAttn);
    return false;
  };

  // The same for a whole warp: its lanes agree on the outcome.
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait(bar, parity));
  };
  // Non-blocking test, agreed on by the warp.
  auto ready = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __any_sync(0xffffffffu, ptx::mbar_test(bar, parity));
  };
  // The i-th item of this CTA, from the item warp; false after the last (or
  // after an abort).
  auto read_item = [&](uint32_t i, Item& it) -> bool {
    if (!wait_warp(&sh.item_full[i % kItems], (i / kItems) & 1u)) return false;
    const int4* src = reinterpret_cast<const int4*>(&sh.items[i % kItems]);
    int4* dst = reinterpret_cast<int4*>(&it);
#pragma unroll
    for (int w = 0; w < 4; ++w) dst[w] = src[w];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&sh.item_empty[i % kItems]);
    return it.b >= 0;
  };

  if (warp >= kLoadWarp0) {
    // ------------------------------------- the query, and rows to be widened
    regs_up<kRegsLoad>();
    const int lt = tid - kLoadWarp0 * 32, lw = lt >> 5;
    const float kvs = DT == MXQ_CACHE_E4M3 ? __ldg(a.kv_scale) : 1.0f;
    int nq = 0;                // items with blocks so far
    [[maybe_unused]] uint32_t nb = 0;  // blocks so far
    [[maybe_unused]] uint32_t st = 0, stp = 0;  // stage and its phase
    bool ok = true;
    Item it;
    for (uint32_t ni = 0; ok && read_item(ni, it); ++ni) {
      if (it.blk0 >= it.blk1) continue;
      // Q rows, one per warp and step; rows past the tile's are zeros.
      if (nq > 0 && !(ok = wait_warp(&sh.q_empty, (uint32_t)(nq - 1) & 1u))) break;
      for (int r0 = lw; r0 < NR; r0 += 4 * kLoadWarps) {
        uint4 v[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            v[i][c] = make_uint4(0, 0, 0, 0);
            const int pc = c * 32 + lane, r = r0 + i * kLoadWarps;
            if (pc < nch * 8 && r < it.nrows)
              v[i][c] = __ldg(reinterpret_cast<const uint4*>(a.q) + (it.qrow + r) * (nch * 8) + pc);
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + i * kLoadWarps;
          if constexpr (!BF) {
            // Largest magnitude of the row -> the power of two that brings it
            // to [2^10, 2^11).
            uint32_t mx = 0;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t w[4] = {v[i][c].x, v[i][c].y, v[i][c].z, v[i][c].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                mx = max(mx, w[e] & 0x7FFFu);
                mx = max(mx, (w[e] >> 16) & 0x7FFFu);
              }
            }
            mx = __reduce_max_sync(0xffffffffu, mx);
            const int ex = (int)(mx >> 7);
            int sft = ex == 255 || mx == 0 ? 0 : 137 - ex;
            sft = min(sft, 120);
            const float f = __uint_as_float((uint32_t)(127 + sft) << 23);
            if (lane == 0) {
              const float inv = __uint_as_float((uint32_t)(127 - sft) << 23);
              sh.crow[nq % 3][r] = r < it.nrows ? a.sm_scale * kLog2e * kvs * inv : 0.0f;
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float y[8];
              unpack8(v[i][c], y);
              v[i][c] = make_uint4(pack16(false, y[0] * f, y[1] * f), pack16(false, y[2] * f, y[3] * f),
                                   pack16(false, y[4] * f, y[5] * f), pack16(false, y[6] * f, y[7] * f));
            }
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int pc = c * 32 + lane;
            if (pc < nch * 8)
              *reinterpret_cast<uint4*>(sm_q + (pc >> 3) * (NR * 128) + r * 128 + (((pc & 7) ^ (r & 7)) << 4)) = v[i][c];
          }
        }
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(&sh.q_full[nq & 3]);
      ++nq;

      if constexpr (DT != MXQ_CACHE_BF16) {
        constexpr int RPT = kRowsPerThread<DT>;          // cache rows of this thread per block
        constexpr int TPR = kLoadThreads * RPT / kKeys;  // threads per row: 8, 4
        constexpr int KSTEP = kKeys / RPT;               // key step between its rows: 16, 32
        constexpr int PIECE_COLS = 128 / TPR;            // columns of a 16-byte piece: 16, 32
        const int key0 = lt / TPR, piece = lt % TPR;
        const uint32_t row_bytes = DT == MXQ_CACHE_E4M3 ? (uint32_t)D : (uint32_t)D / 2;
        // Rows key0 + i * KSTEP of a block (unit i * KSTEP / 16 + key0 / 16).
        const uint8_t* row[RPT];
        const uint8_t* sf[RPT];
        auto open_block = [&]() -> bool {
          if (!wait_warp(&sh.slot_full[nb % kSlots], (nb / kSlots) & 1u)) return false;
          const int* su = sh.slots[nb % kSlots] + (key0 >> 4);
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            const int u = su[i * (KSTEP / 16)];
            const int64_t slot = (int64_t)u + (key0 & 15);
            const bool in = u >= 0 && slot < a.num_slots;
            row[i] = in ? static_cast<const uint8_t*>(a.cache) + slot * row_bytes + piece * 16 : nullptr;
            if (DT == MXQ_CACHE_E2M1) sf[i] = a.cache_sf + (in ? slot : 0) * (D >> 5) + piece;
          }
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sh.slot_empty[nb % kSlots]);
          ++nb;
          return true;
        };
        // The 16-byte pieces of one pair of chunks (and their scale bytes).
        auto fetch = [&](int pr, uint4 (&v)[RPT], uint32_t (&sb)[RPT]) {
          const bool in = pr * 128 + piece * PIECE_COLS < D;  // an odd last chunk: half a pair
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            sb[i] = 0;
            if (in && row[i] != nullptr) {
              v[i] = __ldg(reinterpret_cast<const uint4*>(row[i] + pr * (TPR * 16)));
              if (DT == MXQ_CACHE_E2M1) sb[i] = __ldg(sf[i] + pr * 4);
            }
          }
        };
        auto store = [&](const uint4 (&v)[RPT], const uint32_t (&sb)[RPT]) {
          uint8_t* dst = sm_stage + st * kStageBytes;
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            const int key = key0 + i * KSTEP;
            uint8_t* d = dst + key * 128;
            const int sw = key & 7;
            if constexpr (DT == MXQ_CACHE_E4M3) {
              uint4 lo, hi;
              widen_e4m3(v[i], lo, hi);
              // The two chunks store their halves in opposite order, so that
              // eight lanes always cover eight different 16-byte columns.
              const int ch = piece >> 2, c0 = (piece & 3) * 2;
              d += ch * kChunkBytes;
              *reinterpret_cast<uint4*>(d + (((c0 + ch) ^ sw) << 4)) = ch ? hi : lo;
              *reinterpret_cast<uint4*>(d + (((c0 + 1 - ch) ^ sw) << 4)) = ch ? lo : hi;
            } else {
              const E2m1Table t = e2m1_table(sb[i]);
              const int ch = piece >> 1, c0 = (piece & 1) * 4;
              d += ch * kChunkBytes;
              const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                // Column e ^ (2 * chunk): the same conflict rule as above.
                const uint32_t we = ch ? w[e ^ 2] : w[e];
                const uint2 x = widen_e2m1x4(we, t), y = widen_e2m1x4(we >> 16, t);
                *reinterpret_cast<uint4*>(d + (((c0 + (ch ? e ^ 2 : e)) ^ sw) << 4)) =
                    make_uint4(x.x, x.y, y.x, y.y);
              }
            }
          }
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(&sh.full[st]);
          if (++st == (uint32_t)k.stages) {
            st = 0;
            stp ^= 1u;
          }
        };
        // The next pair is fetched before the current one is stored.
        uint4 v[2][RPT];
        uint32_t sb[2][RPT];
        int left = it.blk1 - it.blk0, pr = 0;
        if (!(ok = open_block())) break;
        fetch(0, v[0], sb[0]);
        auto step = [&](uint4 (&vc)[RPT], uint32_t (&sc)[RPT], uint4 (&vn)[RPT], uint32_t (&sn)[RPT]) -> bool {
          if (++pr == np) {
            pr = 0;
            if (--left > 0 && !(ok = open_block())) return false;
          }
          if (left > 0) fetch(pr, vn, sn);
          if (!(ok = wait_warp(&sh.empty[st], stp ^ 1u))) return false;
          store(vc, sc);
          return left > 0;
        };
        while (step(v[0], sb[0], v[1], sb[1]) && step(v[1], sb[1], v[0], sb[0])) {
        }
      }
    }
  } else if (warp == kTmaWarp) {
    regs_down<kRegsIssue>();
    if constexpr (DT == MXQ_CACHE_BF16) {
      // --------------------------------- BF16 rows: copied as they are by TMA
      // Lane u < 8 copies unit u of the block, one box of 16 rows x 64 columns
      // per chunk.
      uint32_t st = 0, stp = 0, nb = 0;
      bool ok = true;
      Item it;
      for (uint32_t ni = 0; ok && read_item(ni, it); ++ni) {
        for (int blk = it.blk0; blk < it.blk1 && ok; ++blk) {
          if (!(ok = wait_warp(&sh.slot_full[nb % kSlots], (nb / kSlots) & 1u))) break;
          const int row = lane < kUnits ? sh.slots[nb % kSlots][lane] : -1;
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sh.slot_empty[nb % kSlots]);
          ++nb;
          const uint32_t boxes = (uint32_t)__popc(__ballot_sync(0xffffffffu, row >= 0));
          for (int pr = 0; pr < np; ++pr) {
            if (!(ok = wait_warp(&sh.empty[st], stp ^ 1u))) break;
            const int chunks = min(2, nch - pr * 2);
            if (lane == 0) ptx::mbar_arrive_expect_tx(&sh.full[st], boxes * (uint32_t)chunks * (kUnit * 128));
            __syncwarp();
            if (row >= 0)
              for (int c = 0; c < chunks; ++c)
                tma_load_2d(sm_stage + st * kStageBytes + c * kChunkBytes + lane * (kUnit * 128), &tm_kv,
                            &sh.full[st], (pr * 2 + c) * 64, row);
            if (++st == (uint32_t)k.stages) {
              st = 0;
              stp ^= 1u;
            }
          }
        }
      }
      // Copies in flight land before the shared memory goes away: every stage
      // that was filled is waited for (after an abort nobody else does).
      if (*abort_flag && lane == 0)
        for (int s = 0; s < k.stages; ++s)
          if (!ptx::mbar_wait(&sh.full[s], (uint32_t)s < st ? stp : stp ^ 1u, kWaitNs / 8)) break;
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    regs_down<kRegsIssue>();
    // Two cursors over the same sequence of blocks: the first product runs
    // ahead of the second by as much as the stages hold, two blocks at most
    // (the two S buffers).  Whatever is ready is issued, the second product
    // first, because it frees stages.
    const uint32_t dk0 = desc_lo(ptx::smem_u32(sm_stage), 16), dv0 = desc_lo(ptx::smem_u32(sm_stage), kChunkBytes);
    const uint32_t dp0 = desc_lo(ptx::smem_u32(sm_p), kChunkBytes), dq0 = desc_lo(ptx::smem_u32(sm_q), 16);
    constexpr uint32_t idesc_s = idesc_f16(BF, NR, false, false);
    constexpr uint32_t idesc_o = idesc_f16(BF, NV, true, true);
    // Items are read without blocking: those that see no key have nothing for
    // this warp, and the others may only move on once it has issued what is ready.
    uint32_t ni = 0;
    bool more = true;                 // the last item has not been read
    int qleft = 0, pleft = 0;         // blocks left of the two cursors' items
    int punits = 0, nwait = 0;        // units left of the second's; items it still has to begin,
    int wl0 = 0, wu0 = 0, wl1 = 0, wu1 = 0;  // at most two: it is two blocks behind at most
    bool pfirst = true;
    uint32_t gq = 0, gp = 0, nqi = 0;     // blocks issued by each, items begun
    uint32_t qs = 0, qsp = 0, ps = 0;     // stages of the two cursors
    int qpair = 0;
    bool q_ready = false;
    uint64_t t0 = 0;
    uint32_t idle = 0;
    while (more || qleft > 0 || pleft > 0) {
      bool did = false;
      if (more && qleft == 0 && nwait < 2 && ready(&sh.item_full[ni % kItems], (ni / kItems) & 1u)) {
        Item it;
        more = read_item(ni, it);
        ++ni;
        did = true;
        if (more && it.blk0 < it.blk1) {
          qleft = it.blk1 - it.blk0;
          const int u = it.units - it.blk0 * kUnits;
          if (pleft == 0) {
            pleft = qleft;
            punits = u;
          } else {
            if (nwait == 0) {
              wl0 = qleft;
              wu0 = u;
            } else {
              wl1 = qleft;
              wu1 = u;
            }
            ++nwait;
          }
        }
      }
      if (gp < gq && ready(&sh.p_full, gp & 1u)) {
        ptx::tc_fence_after();
        const int kk = min(kUnits, punits);  // units in use
        for (int m = 0; m < np; ++m) {
          if (ptx::elect_one()) {
            const uint32_t da = dv0 + ps * (kStageBytes >> 4);
            const uint32_t dd = tmem + m * NV;
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
              if (u >= kk) break;
              mma_f16(dd, da + u * 128, kDescHi, dp0 + u * 128, kDescHi, idesc_o, (pfirst && u == 0) ? 0u : 1u);
              if (NR == 64)  // the low parts, a buffer of their own
                mma_f16(dd, da + u * 128, kDescHi, dp0 + (kKeys * 8) + u * 128, kDescHi, idesc_o, 1u);
            }
            ptx::tc_commit(&sh.empty[ps]);
          }
          __syncwarp();
          if (++ps == (uint32_t)k.stages) ps = 0;
        }
        if (ptx::elect_one()) ptx::tc_commit(&sh.pv_done);
        ++gp;
        pfirst = false;
        punits -= kUnits;
        if (--pleft == 0) {
          pfirst = true;
          if (nwait > 0) {
            pleft = wl0;
            punits = wu0;
            wl0 = wl1;
            wu0 = wu1;
            --nwait;
          }
        }
        did = true;
      } else if (qleft > 0 && gq < gp + 2) {
        if (!q_ready) q_ready = ready(&sh.q_full[nqi & 3u], (nqi >> 2) & 1u);
        while (q_ready && ready(&sh.full[qs], qsp)) {
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            const uint32_t da = dk0 + qs * (kStageBytes >> 4), db = dq0 + qpair * (NR * 256 >> 4);
            const uint32_t ds = tmem + kTmemS + (gq & 1u) * 64;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (qpair * 2 + c >= nch) break;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                mma_f16(ds, da + c * (kChunkBytes >> 4) + e * 2, kDescHi, db + c * (NR * 128 >> 4) + e * 2, kDescHi,
                        idesc_s, (qpair | c | e) ? 1u : 0u);
            }
          }
          __syncwarp();
          did = true;
          if (++qs == (uint32_t)k.stages) {
            qs = 0;
            qsp ^= 1u;
          }
          if (++qpair == np) {
            qpair = 0;
            if (ptx::elect_one()) ptx::tc_commit(&sh.s_full[gq & 1u]);
            ++gq;
            if (--qleft == 0) {
              if (ptx::elect_one()) ptx::tc_commit(&sh.q_empty);
              ++nqi;
              q_ready = false;
            }
            break;
          }
        }
      }
      if (did) {
        idle = 0;
      } else if ((++idle & 63u) == 0) {
        if (idle == 64) t0 = ptx::globaltimer();
        int stop = *abort_flag;
        if (!stop && ptx::globaltimer() - t0 > kWaitNs) {
          stop = 1;
          if (lane == 0) {
            *abort_flag = 1;
            atomicOr(k.watchdog, kWdAttn);
          }
        }
        if (__any_sync(0xffffffffu, stop)) break;
      }
    }
    // Everything issued has completed before TMEM and shared memory go away.
    if (ptx::elect_one()) ptx::tc_commit(&sh.drain);
    __syncwarp();
    if (!ptx::mbar_wait(&sh.drain, 0, kWaitNs) && lane == 0) atomicOr(k.watchdog, kWdAttn);
  } else if (warp == kItemWarp) {
    // ------------------------------------------------------- work items
    // Decoded here once for all roles, up to four ahead.
    regs_down<kRegsIssue>();
    uint32_t i = 0;
    for (int item = blockIdx.x;; item += gridDim.x) {
      Item it;
      const bool end = item >= k.items;
      if (end) {
        it.b = -1;
      } else {
        it = get_item<NR>(k, item);
        if (it.nrows == 0) continue;
        if (lane == 0 && it.pad && a.err_flag != nullptr) atomicOr(a.err_flag, MXQ_DEVERR_LENGTH);
        // Without blocks: a row that sees nothing (written by split 0), or a
        // share of the keys that is empty.
        if (it.blk0 >= it.blk1 && (it.units > 0 || it.split > 0)) continue;
      }
      if (!wait_warp(&sh.item_empty[i % kItems], ((i / kItems) & 1u) ^ 1u)) break;
      if (lane == 0) {
        sh.items[i % kItems] = it;
        ptx::mbar_arrive(&sh.item_full[i % kItems]);
      }
      __syncwarp();
      if (end) break;
      ++i;
    }
  } else if (warp == kUnitWarp) {
    // ------------------------------------- where the units of a block lie
    // Lane u < 8 looks up unit u, a few blocks ahead of their use: the block
    // table's latency and the divisions stay out of the other warps' way.
    regs_down<kRegsIssue>();
    uint32_t nb = 0;
    bool ok = true;
    Item it;
    for (uint32_t ni = 0; ok && read_item(ni, it); ++ni) {
      for (int blk = it.blk0; blk < it.blk1; ++blk, ++nb) {
        const int x = blk * kUnits + lane;
        int slot = -1;
        if (lane < kUnits && x < it.units) {
          const int j = unit_key(it, x);
          const int pg = j / a.page_size;
          const int page = __ldg(a.block_table + (int64_t)it.b * a.max_pages + pg);
          const int64_t first = (int64_t)page * a.page_size + (j - pg * a.page_size);
          if (page >= 0 && first < a.num_slots) slot = (int)first;
          // A page outside the cache, or one that ends past it, hides keys.
          if (a.err_flag != nullptr && (slot < 0 || first + min(kUnit, it.p1 + 1 - j) > a.num_slots))
            atomicOr(a.err_flag, MXQ_DEVERR_SLOT);
        }
        if (!(ok = wait_warp(&sh.slot_empty[nb % kSlots], ((nb / kSlots) & 1u) ^ 1u))) break;
        if (lane < kUnits) sh.slots[nb % kSlots][lane] = slot;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.slot_full[nb % kSlots]);
      }
    }
  } else {
    // ------------------------------------------------- softmax and epilogue
    regs_up<kRegsSoft>();
    const int h = warp >> 2, quad = warp & 3;      // row half, TMEM lane quadrant
    const uint32_t tq = tmem + ((uint32_t)(quad * 32) << 16);
    const int key = quad * 32 + lane;              // this thread's key of a block
    const int c0 = h * NC;
    const uint32_t bar = 1 + h;
    const float c_all = a.sm_scale * kLog2e;
    const float4* negm4 = reinterpret_cast<const float4*>(sh.negm + c0);
    uint32_t g = 0;   // blocks so far
    int nq = 0;       // items with blocks so far
    uint32_t st = 0;  // first stage of the current block
    // A wait that gives up does not leave the loops by itself: the group's
    // next vote takes all of its threads out together.
    bool ok = true, dead = false;
    for (uint32_t ni = 0; !dead; ++ni) {
      // The item stays in shared memory until its output is on its way: only
      // what every block needs is held in registers.
      const volatile Item& held = sh.items[ni % kItems];
      const bool more = wait_warp(&sh.item_full[ni % kItems], (ni / kItems) & 1u) && held.b >= 0;
      if (named_any(bar, 128, !more)) break;
      struct {
        int nrows, p0, p1, u_lo, ns, units, blk0, blk1;
      } it = {held.nrows, held.p0, held.p1, held.u_lo, held.ns, held.units, held.blk0, held.blk1};
      const bool has = it.blk0 < it.blk1;
      // Rows of this group.
      if (quad == 0 && lane < NC) {
        const int r = c0 + lane;
        sh.negm[r] = r < it.nrows ? kNoKey : 0.0f;
        sh.rowt[r] = (uint8_t)((held.r0 + r) / a.H - held.r0 / a.H);
      }
      ptx::named_sync(bar, 128);
      float l[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) l[c] = 0.0f;
      const float4* crow4 = reinterpret_cast<const float4*>(sh.crow[nq % 3] + c0);
      if (has) {
        // The row scales come with the query.
        if (!BF) ok = wait(&sh.q_full[nq & 3], (uint32_t)(nq >> 2) & 1u) && ok;
        ++nq;
      }
      for (int blk = it.blk0; blk < it.blk1; ++blk) {
        // Which rows see this thread's key: all, none or some.
        const int x = blk * kUnits + (key >> 4);
        const bool in = x < it.units;
        const int j = unit_key(it, in ? x : 0) + (key & 15);
        const int weff = (a.window == 0 || j < a.sinks) ? 0x7fffffff : a.window;
        ok = wait(&sh.slot_full[g % kSlots], (g / kSlots) & 1u) && ok;
        const int unit_slot = sh.slots[g % kSlots][key >> 4];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.slot_empty[g % kSlots]);
        const bool some = in && j <= it.p1 && it.p0 - j < weff && unit_slot >= 0 &&
                          (int64_t)unit_slot + (key & 15) < a.num_slots;
        const bool all = some && j <= it.p0 && it.p1 - j < weff;
        const bool mixed = __any_sync(0xffffffffu, some && !all);
        auto sees = [&](int c) { return some && (uint32_t)(it.p0 + sh.rowt[c0 + c] - j) < (uint32_t)weff; };

        ok = wait(&sh.s_full[g & 1u], (g >> 1) & 1u) && ok;
        __syncwarp();
        ptx::tc_fence_after();
        uint32_t s[NC];
        tmem_ld<NC>(tq + kTmemS + (g & 1u) * 64 + c0, s);
        ptx::tmem_ld_wait();
        // Exponents d = s + negm in place of the scores.  Their largest is NaN
        // if one is: a cache row with a NaN or an infinity has no finite score.
        float d[NC], top, seen = -INFINITY;
        auto exponents = [&]() {
          top = -INFINITY;
#pragma unroll
          for (int q = 0; q < NC / 4; ++q) {
            const float4 n = negm4[q];
            const float4 cr = BF ? make_float4(c_all, c_all, c_all, c_all) : crow4[q];
            d[4 * q] = fmaf(__uint_as_float(s[4 * q]), cr.x, n.x);
            d[4 * q + 1] = fmaf(__uint_as_float(s[4 * q + 1]), cr.y, n.y);
            d[4 * q + 2] = fmaf(__uint_as_float(s[4 * q + 2]), cr.z, n.z);
            d[4 * q + 3] = fmaf(__uint_as_float(s[4 * q + 3]), cr.w, n.w);
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max_nan(top, d[4 * q + e]);
          }
        };
        exponents();
        if (mixed)
#pragma unroll
          for (int c = 0; c < NC; ++c) seen = fmaxf(seen, sees(c) ? d[c] : -INFINITY);
        const bool bad = in && !(fabsf(top) <= 3.4028234e38f);
        const bool raise = bad || (some && (mixed ? seen : top) > kSlack + kShift);
        if (named_any(bar, 128, raise || !ok)) {
          // ---- some maximum moves, something is not finite, or a wait gave up
          if (named_any(bar, 128, !ok)) {
            dead = true;
            break;
          }
          if (bad) {
            // A row that holds a NaN or an infinity must not reach the rows
            // that do not see it through 0 * NaN: it is cleared here, and the
            // rows that see it become NaN through their sums.
            bool rowbad = false;
            for (int pass = 0; pass < 2; ++pass)
              for (int ch = 0; ch < nch; ++ch) {
                const uint32_t sidx = (st + (ch >> 1)) % (uint32_t)k.stages;
                uint4* rp = reinterpret_cast<uint4*>(sm_stage + sidx * kStageBytes + (ch & 1) * kChunkBytes + key * 128);
                for (int e = 0; e < 8; ++e) {
                  if (pass == 1) {
                    if (rowbad) rp[e] = make_uint4(0, 0, 0, 0);
                    continue;
                  }
                  const uint4 w = rp[e];
                  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
                  const uint32_t m = BF ? 0x7F80u : 0x7C00u;
                  for (int q = 0; q < 4; ++q)
                    rowbad |= (ws[q] & m) == m || ((ws[q] >> 16) & m) == m;
                }
              }
          }
          // The scores again (s is not kept: registers), and their maxima.
          tmem_ld<NC>(tq + kTmemS + (g & 1u) * 64 + c0, s);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < NC / 4; ++q) {
            const float4 cr4 = BF ? make_float4(c_all, c_all, c_all, c_all) : crow4[q];
            const float cr[4] = {cr4.x, cr4.y, cr4.z, cr4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int c = 4 * q + e;
              const float v = __uint_as_float(s[c]);
              const bool fin = fabsf(v) <= 3.4028234e38f;
              const bool see = mixed ? sees(c) : all;
              if (bad && !fin && see) l[c] = NAN;
              d[c] = see && fin ? v * cr[e] : -INFINITY;
            }
          }
          const float m = lanes_reduce<NC, true>(d);
          if (lane < NC) sh.red[h][quad][lane] = m;
          ptx::named_sync(bar, 128);
          if (quad == 0 && lane < NC) {
            const int r = c0 + lane;
            const float mb = fmaxf(fmaxf(sh.red[h][0][lane], sh.red[h][1][lane]),
                                   fmaxf(sh.red[h][2][lane], sh.red[h][3][lane]));
            const float old = sh.negm[r];
            float f = 1.0f;
            if (r < it.nrows && mb > -INFINITY) {
              const float cur = old >= kNoKey ? -INFINITY : kShift - old;
              if (mb > cur) {
                if (old < kNoKey) f = ex2(cur - mb);
                sh.negm[r] = kShift - mb;
              }
            }
            sh.scale[r] = f;
          }
          ptx::named_sync(bar, 128);
          exponents();
          if (bad)
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if (!(fabsf(__uint_as_float(s[c])) <= 3.4028234e38f)) d[c] = -INFINITY;
          if (blk > it.blk0) {
            bool moved = false;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const float f = sh.scale[c0 + c];
              l[c] *= f;
              moved |= f != 1.0f;
            }
            ok = wait(&sh.pv_done, (g - 1) & 1u);
            __syncwarp();
            if (moved) {
              ptx::tc_fence_after();
              for (int m = 0; m < np * (NV / NR); ++m)
#pragma unroll
                for (int c = 0; c < NC; c += 8) {
                  uint32_t o[8];
                  const uint32_t ad = tq + m * NR + c0 + c;
                  ptx::tmem_ld_32x32b_x8(ad, o);
                  ptx::tmem_ld_wait();
#pragma unroll
                  for (int e = 0; e < 8; ++e)
                    o[e] = __float_as_uint(__uint_as_float(o[e]) * sh.scale[c0 + c + e]);
                  tmem_st8(ad, o);
                }
              tmem_st_wait();
            }
          }
        } else if (blk > it.blk0) {
          ok = wait(&sh.pv_done, (g - 1) & 1u);
          __syncwarp();
        }
        // ---- weights
#pragma unroll
        for (int q = 0; q < NC / 8; ++q) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float p[2];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const int c = q * 8 + e * 2 + f;
              const bool see = mixed ? sees(c) : all;
              p[f] = see ? ex2(d[c]) : 0.0f;
              l[c] += p[f];
            }
            hi[e] = pack16(BF, p[0], p[1]);
            lo[e] = pack16_rest(BF, p[0], p[1], hi[e]);
          }
          const int col = (c0 >> 3) + q;
          uint8_t* row = sm_p + key * 128;
          *reinterpret_cast<uint4*>(row + ((col ^ (key & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          const int lcol = NR == 64 ? col : col + NR / 8;
          *reinterpret_cast<uint4*>(row + (NR == 64 ? kKeys * 128 : 0) + ((lcol ^ (key & 7)) << 4)) =
              make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&sh.p_full);
        ++g;
        st = (st + np) % (uint32_t)k.stages;
      }
      if (dead) break;
      // ---- row sums over the 128 keys, then the output
      const float sum32 = lanes_reduce<NC, false>(l);
      if (lane < NC) sh.red[h][quad][lane] = sum32;
      if (has) {
        ok = wait(&sh.pv_done, (g - 1) & 1u) && ok;
        if (named_any(bar, 128, !ok)) {
          dead = true;
          break;
        }
      } else {
        ptx::named_sync(bar, 128);
      }
      ptx::tc_fence_after();
      if (quad == 0 && lane < NC) {
        const int r = c0 + lane;
        const float sum = (sh.red[h][0][lane] + sh.red[h][1][lane]) + (sh.red[h][2][lane] + sh.red[h][3][lane]);
        const float nm = sh.negm[r];
        if (k.splits > 1 && has) {
          k.part_ml[((int64_t)held.tile * k.splits + held.split) * NR + r] = make_float2(-nm, sum);
        } else {
          const float vs = DT == MXQ_CACHE_E4M3 ? __ldg(a.kv_scale) : 1.0f;
          sh.scale[r] = sum == 0.0f ? 0.0f : vs / sum;
          if (r < it.nrows && a.lse != nullptr)
            a.lse[held.qrow + r] = sum == 0.0f ? -INFINITY : (log2f(sum) - nm) * 0.6931471805599453f;
        }
      }
      ptx::named_sync(bar, 128);
      if (k.splits > 1 && has) {
        // Partial sums as they are: a warp stores 32 consecutive columns of a row.
        float* dst = k.part + (((int64_t)held.tile * k.splits + held.split) * NR + c0) * D + key;
        for (int m = 0; m < np; ++m) {
          uint32_t o[NC];
          tmem_ld<NC>(tq + m * NV + c0, o);
          if constexpr (NR < 64) {
            uint32_t lo[NC];
            tmem_ld<NC>(tq + m * NV + NR + c0, lo);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < NC; ++c)
              o[c] = __float_as_uint(__uint_as_float(o[c]) + __uint_as_float(lo[c]));
          } else {
            ptx::tmem_ld_wait();
          }
          if (m * 128 + key < D) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if (c0 + c < it.nrows) dst[(int64_t)c * D + m * 128] = __uint_as_float(o[c]);
          }
        }
      } else {
        // The output is turned around in shared memory (the group's half of
        // the P buffers), 256 columns at a time: 16-lane TMEM fragments,
        // rounded to BF16 pairs of rows, stored as transposed 8 x 8 matrices
        // into rows of 512 bytes whose 16-byte words are swizzled by row; then
        // whole rows go out with 16-byte stores.
        uint8_t* stage = sm_p + h * (p_bytes(NR) / 2);
        const uint32_t stage_a = ptx::smem_u32(stage);
        float2 sc[NC / 8];
#pragma unroll
        for (int q = 0; q < NC / 8; ++q)
          sc[q] = *reinterpret_cast<const float2*>(&sh.scale[c0 + q * 8 + (lane & 3) * 2]);
        uint8_t* dst = static_cast<uint8_t*>(a.out) + (held.qrow + c0) * D * 2;
        for (int m0 = 0; m0 < np; m0 += 2) {
          for (int m = m0; m < min(m0 + 2, np); ++m)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint32_t o[NC / 2];
              const uint32_t ad = tq + ((uint32_t)(hf * 16) << 16) + m * NV + c0;
              tmem_ld_16x256b<NC>(ad, o);
              if constexpr (NR < 64) {
                uint32_t lo[NC / 2];
                tmem_ld_16x256b<NC>(ad + NR, lo);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < NC / 2; ++c)
                  o[c] = __float_as_uint(__uint_as_float(o[c]) + __uint_as_float(lo[c]));
              } else {
                ptx::tmem_ld_wait();
              }
#pragma unroll
              for (int q = 0; q < NC / 8; ++q) {
                const uint32_t w0 = pack16(true, out_of(has, o[4 * q]) * sc[q].x, out_of(has, o[4 * q + 1]) * sc[q].y);
                const uint32_t w1 = pack16(true, out_of(has, o[4 * q + 2]) * sc[q].x, out_of(has, o[4 * q + 3]) * sc[q].y);
                // Lanes 0-7 name the rows of the first matrix, 8-15 of the second.
                const int row = q * 8 + (lane & 7);
                const int word = (m - m0) * 16 + quad * 4 + hf * 2 + ((lane >> 3) & 1);
                stmatrix_x2_trans(stage_a + row * 512 + ((word ^ (row & 7)) << 4), w0, w1);
              }
            }
          ptx::named_sync(bar, 128);
          for (int i = quad; i < NC; i += 4) {
            const int col = m0 * 128 + lane * 8;
            if (c0 + i < it.nrows && col < D)
              *reinterpret_cast<uint4*>(dst + ((int64_t)i * D + col) * 2) =
                  *reinterpret_cast<const uint4*>(stage + i * 512 + ((lane ^ (i & 7)) << 4));
          }
          ptx::named_sync(bar, 128);
        }
        // Both groups are done with the P buffers.
        ptx::named_sync(3, 256);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh.item_empty[ni % kItems]);
      ptx::tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, kTmemCols);
}

// Joins the partial sums of a tile's splits, one warp per row: the splits in
// index order, each weighted by 2^(its maximum - the largest).
template <int NR>
__global__ void __launch_bounds__(128) attn_join_kernel(const KernelArgs k) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const AttnArgs& a = k.a;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= (int64_t)k.tiles * NR) return;
  const int r = (int)(w % NR);
  // Item number of split 0 of this tile.
  const int tile = (int)(w / NR);
  const Item it = get_item<NR>(k, k.tiles - 1 - tile);
  if (r >= it.nrows || it.units == 0) return;
  const int nb = (it.units + kUnits - 1) / kUnits;
  const int per = (nb + k.splits - 1) / k.splits;
  const int used = (nb + per - 1) / per;
  const float2* ml = k.part_ml + ((int64_t)tile * k.splits) * NR + r;
  float mx = -INFINITY;
  for (int s = lane; s < used; s += 32) mx = fmaxf(mx, ml[(int64_t)s * NR].x);
  mx = warp_max(mx);
  float o[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) o[c] = 0.0f;
  float sum = 0.0f;
  const float* p = k.part + ((int64_t)tile * k.splits * NR + r) * a.D;
  for (int s = 0; s < used; ++s) {
    const float2 v = ml[(int64_t)s * NR];
    const float f = ex2(v.x - mx);
    sum += f * v.y;
    const float* ps = p + (int64_t)s * NR * a.D;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int d = c * 128 + lane * 4;
      if (d < a.D) {
        const float4 x = *reinterpret_cast<const float4*>(ps + d);
        o[4 * c] += f * x.x;
        o[4 * c + 1] += f * x.y;
        o[4 * c + 2] += f * x.z;
        o[4 * c + 3] += f * x.w;
      }
    }
  }
  const float vs = a.dtype == MXQ_CACHE_E4M3 ? __ldg(a.kv_scale) : 1.0f;
  const float inv = sum == 0.0f ? 0.0f : vs / sum;
  uint8_t* dst = static_cast<uint8_t*>(a.out) + (it.qrow + r) * a.D * 2;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int d = c * 128 + lane * 4;
    if (d < a.D)
      *reinterpret_cast<uint2*>(dst + d * 2) = make_uint2(pack16(true, o[4 * c] * inv, o[4 * c + 1] * inv),
                                                          pack16(true, o[4 * c + 2] * inv, o[4 * c + 3] * inv));
  }
  if (lane == 0 && a.lse != nullptr)
    a.lse[it.qrow + r] = sum == 0.0f ? -INFINITY : (log2f(sum) + mx) * 0.6931471805599453f;
}

// ---------------------------------------------------------------- host side
struct Plan {
  int NR, tiles, splits, stages;
  size_t part_bytes, bytes;
};

constexpr int kSms = 152;  // the plan must not depend on the device: workspace sizes come from it

Plan make_plan(const AttnArgs& a) {
  Plan p;
  const int64_t per_seq = a.T * a.H / a.B;
  p.NR = per_seq > 32 ? 64 : per_seq > 16 ? 32 : 16;
  p.tiles = (int)(a.T * a.H / p.NR + a.B);
  // Key blocks of a tile, at most.
  const int64_t cap = (int64_t)a.max_pages * a.page_size;
  int64_t keys = cap;
  if (a.window > 0) {
    const int64_t w = (int64_t)a.window + a.sinks + 2 * kUnit + (p.NR + a.H - 1) / a.H;
    keys = keys < w ? keys : w;
  }
  const int64_t nb = ceil_div(keys, kKeys);
  // Tiles that exist: the numbering above leaves gaps.
  const int64_t real = a.B * ceil_div(ceil_div(a.T * a.H, a.B), p.NR);
  int64_t splits = kSms / (real > 0 ? real : 1);
  if (splits > nb / 2) splits = nb / 2;  // two blocks at least: a join costs about one
  p.splits = splits < 1 ? 1 : (int)splits;
  p.stages = stages_for(p.NR, a.D);
  const size_t rows = (size_t)p.tiles * p.splits * p.NR;
  p.part_bytes = p.splits > 1 ? round_up_256(rows * a.D * 4) : 0;
  p.bytes = p.splits > 1 ? p.part_bytes + round_up_256(rows * 8) : 0;
  return p;
}

// BF16 cache rows as a 2-D map: boxes of 16 rows x 64 columns, 128-byte rows
// swizzled, zeros past the last row.
bool encode_rows(CUtensorMap* m, const void* base, uint64_t D, uint64_t rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {D, rows};
  cuuint64_t strides[1] = {D * 2};
  cuuint32_t box[2] = {64, kUnit};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NR, int DT>
cudaError_t launch_one(const KernelArgs& k, int num_sms, cudaStream_t s, const char** why) {
  auto kern = attn_kernel<NR, DT>;
  const int smem = smem_fixed(NR, k.a.D) + k.stages * kStageBytes;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // Per device, once: the shared-memory opt-in.
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_acq_rel);
  }
  CUtensorMap tm = {};
  if (DT == MXQ_CACHE_BF16 && !encode_rows(&tm, k.a.cache, (uint64_t)k.a.D, (uint64_t)k.a.num_slots)) {
    *why = "cuTensorMapEncodeTiled failed (driver entry point missing or arguments rejected)";
    return cudaErrorInvalidValue;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(k.items < num_sms ? k.items : num_sms), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, tm, k);
  if (e != cudaSuccess || k.splits == 1) return e;
  cfg.gridDim = dim3((unsigned)ceil_div((int64_t)k.tiles * NR, 4), 1, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, attn_join_kernel<NR>, k);
}

template <int NR>
cudaError_t launch_nr(const KernelArgs& k, int num_sms, cudaStream_t s, const char** why) {
  if (k.a.dtype == MXQ_CACHE_BF16) return launch_one<NR, MXQ_CACHE_BF16>(k, num_sms, s, why);
  if (k.a.dtype == MXQ_CACHE_E4M3) return launch_one<NR, MXQ_CACHE_E4M3>(k, num_sms, s, why);
  return launch_one<NR, MXQ_CACHE_E2M1>(k, num_sms, s, why);
}

}  // namespace

size_t attn_workspace_bytes(const AttnArgs& a) { return a.T > 0 ? make_plan(a).bytes : 0; }

cudaError_t launch_attn(const AttnArgs& a, void* ws, int num_sms, cudaStream_t s, const char** why) {
  const Plan p = make_plan(a);
  KernelArgs k = {};
  k.a = a;
  k.tiles = p.tiles;
  k.splits = p.splits;
  k.stages = p.stages;
  if ((int64_t)p.tiles * p.splits >= (int64_t)1 << 31) {
    *why = "too many tiles";
    return cudaErrorInvalidValue;
  }
  k.items = p.tiles * p.splits;
  k.part = static_cast<float*>(ws);
  k.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + p.part_bytes);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // Per device, once: the watchdog's address.
  static std::atomic<uint64_t> ready{0};
  static uint32_t* wd[64];
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = watchdog_address(&wd[dev & 63]);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_acq_rel);
  }
  k.watchdog = wd[dev & 63];
  if (p.NR == 64) return launch_nr<64>(k, num_sms, s, why);
  if (p.NR == 32) return launch_nr<32>(k, num_sms, s, why);
  return launch_nr<16>(k, num_sms, s, why);
}

}  // namespace mxq
