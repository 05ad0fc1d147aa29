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
// tile.  P = 2^(x + negm), x = s * log2(e).  BF16 has FP32's exponent range, so
// negm need not be minus the row's maximum: it is minus the score of one key
// of the item's first block that (nearly) all rows see, and moves only when a
// score passes it by more than 2^40, so that blocks need neither a maximum
// over the keys nor a rescale of O.  (O and the sums then reach 2^40 times the
// values they stand for, times the number of keys: 2^57 of them leave 2^70.)  Row sums are kept per thread (one key each) in FP32
// and joined at the end.
//
// The kernel is built for a small instruction footprint (70 to 90 KB; at 140 KB
// the roles missed the instruction cache on every block, and 8192 queries with a
// window of 128 took 681 us where half the code took 600): one copy of each
// piece of work, loops over unrolling wherever latency does not matter.
//
// Warps: NR / 4 for the softmax and the epilogue (a lane is a key, then a
// column; each group of four owns 16 of the tile's rows and never waits for
// another), one that issues the matrix instructions, one for the TMA copies of
// BF16 and E4M3 rows, one that hands out the work items, one that looks up the block
// table, and the loading warps, which fetch Q and the cache rows that are
// widened to 16 bits, into the 128-byte-swizzled layout.
//
// A BF16 cache's rows are copied into shared memory as they are, E2M1 rows are
// widened to BF16 (exactly, with their scales); both products then have BF16
// operands.  E4M3 rows are copied as they are too and multiplied as E4M3, which
// halves their shared memory, so that a block's rows arrive while the one before
// is in use, and spares widening them (the integer pipe's 64 results a cycle
// bound a kernel that did: 2048 queries with a window of 4096 took 2350 us).  The
// other operands are then sums of 8-bit parts: Q two E4M3 parts (4 + 4 significant
// bits, all of BF16's 8, relative to the row's largest value: a row is scaled by a
// power of two; half a step of the second part is 2^-21 of that value), P three
// E5M2 parts.  E5M2 is FP16's upper byte, so that a part is the upper byte of
// what the parts before it left, an FP16 number that holds it exactly: nothing is
// lost between the parts, whatever the weight.  A weight is off by 2^-8.8 of
// itself at most, or by half of E5M2's smallest step where that is more: the
// reference is held as 2^13, so that this is 2^-30 of it, met by weights below
// 2^-21 of it.  (E4M3 as the second part has a bit more, but ends seven octaves
// before E5M2: weights below 2^-16 of the reference lost 8 % of themselves.)
//
// P would lose to its rounding as much as the output to its own.  So wherever a
// weight is at least 1/16 of its row's sum so far, what is left of it after
// rounding multiplies its row too, as a second BF16 or a fourth 8-bit part;
// below that it is rounded once (BF16: by half an ulp, 2^-8 of itself at most,
// to either side).  An item's first two blocks, whose sums are not known yet,
// have all parts throughout.
//
// Work: with many tiles per SM, whole tiles are dealt out in turn, the last
// sequence's last tile first (in a sequence, those with the most keys).  Else the
// key blocks of all tiles, in one line, are cut into equal shares, one per CTA; a
// tile that is cut leaves FP32 partial sums, which a second kernel joins in the
// order of the keys.  Equal shares follow from the lengths on the device and stay
// balanced in ragged batches.  Whole tiles do not: a chunk of 1216 tiles or more
// together with a decode over many more keys leaves the latter's blocks to one CTA
// (64 heads, E4M3: 2048 tokens over 2048 keys and 8 tokens over 131072 keys each
// take 3.2 ms in one call, 0.41 and 0.19 ms in two).
//
// What bounds it, and what it measured (GB300, rows of 512 columns, 64 heads;
// products and bytes counted once):
//   2048 queries, window 4096, E4M3     1.36 ms   0.81 PFLOP/s
//   8192 queries, window 128, BF16      526 us    2.1 TB/s
//   16 x 1 query, window 8192, BF16     63 us     2.1 TB/s
//   32 x 1 query, 32768 keys, E2M1      179 us    1.0 TB/s, 0.47 PFLOP/s
//   1 query, 131072 keys, E2M1          51 us     0.70 TB/s
// E4M3: the products, which are being issued 80 % of the time: at 64 rows an
// instruction takes 55 to 60 cycles, 48 of them to read its operands (128 x 32
// and 64 x 32 bytes), where the arithmetic takes 32, and the three parts of the
// weights read the rows three times.  BF16 and E2M1 of 512 columns: one block of
// 128 keys fills the stages, so that the next one's copies and first product
// wait for the second product to free them; that chain takes 9000 cycles a block
// (2500 second product, 2000 copies, 800 first product, 2700 softmax, the rest
// handing over).  Blocks of 64 keys, of which two fit, were no faster (67 us in
// BF16) or slower (215 us in E2M1): the first product's rows past the block are
// read all the same.  Few keys: what a CTA does once, 20 to 25 thousand cycles of
// item decoding, first loads and output, and the join (10 us).
//
// Every wait is bounded in wall time (two seconds); on expiry the kernel sets a
// watchdog bit, stops, waits for the matrix instructions and the copies in
// flight, frees TMEM and returns.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "mxq.h"
#include "mxq_internal.h"
#include "mxq_ptx.cuh"
#include "quant_common.cuh"

namespace mxq {

// The driver's tensor-map encoder (bmm.cu), NULL where the driver lacks it.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace {

constexpr uint32_t kWaitNs = 2000000000u;
constexpr uint32_t kWdAttn = 64;  // watchdog bit of this kernel

constexpr int kKeys = 128;           // keys of a block (M of the first product)
constexpr int kUnit = 16;            // keys of a unit
constexpr int kUnits = kKeys / kUnit;
constexpr int kChunkBytes = kKeys * 128;   // 128 keys x 128 bytes: 64 columns of 16 bits, 128 of 8
// A stage holds 128 columns of the block's rows.
template <int DT>
struct Form {
  static constexpr bool F8 = DT == MXQ_CACHE_E4M3;
  static constexpr int CHUNKS = F8 ? 1 : 2;  // of a stage
  static constexpr int STAGE = CHUNKS * kChunkBytes;
  // Parts of a weight, of which the last is only used where it is large; log2
  // of what a weight equal to the reference's is held as, and of the most (8
  // bits: FP16 and E5M2 end below 2^16).
  static constexpr int PARTS = F8 ? 4 : 2, SURE = F8 ? 3 : 1;
  static constexpr float SHIFT = F8 ? 13.0f : 0.0f, MOST = F8 ? 15.0f : 40.0f;
  // Type of part i in an instruction descriptor: E5M2 three times and E4M3 (a
  // large weight's fourth part is in its range and has a bit more), or BF16.
  static constexpr uint32_t part_type(int i) { return F8 && i == 3 ? 0u : 1u; }
};
// Thread layout and registers (launch registers x threads is what setmaxnreg
// deals out again).  Next to nothing spills: with 227 KB of shared memory in use
// the L1 cache is too small for local memory.
template <int NR>
struct Roles {
  static constexpr int GROUPS = NR / 16;         // softmax groups of 4 warps, 16 rows each
  static constexpr int SOFT = 4 * GROUPS;        // their warps
  static constexpr int MMA = SOFT, TMA = SOFT + 1, ITEM = SOFT + 2, UNIT = SOFT + 3;
  static constexpr int LOAD0 = SOFT + 4, LOADS = 8;
  static constexpr int THREADS = (LOAD0 + LOADS) * 32;
  static constexpr int REGS = 65536 / THREADS / 8 * 8;
  static constexpr int REGS_SOFT = NR == 64 ? 80 : 112, REGS_ISSUE = NR == 64 ? 40 : 64,
                       REGS_LOAD = NR == 64 ? 72 : NR == 32 ? 88 : 128;
  static_assert(SOFT * 32 * REGS_SOFT + 128 * REGS_ISSUE + LOADS * 32 * REGS_LOAD <= THREADS * REGS, "register pool");
};
constexpr int kLoadThreads = 256;
constexpr int kMaxStages = 8;
constexpr uint32_t kTmemCols = 512, kTmemS = 256;
constexpr float kNoKey = 1e30f;      // negm of a row that has seen no key
constexpr float kLog2e = 1.4426950408889634f;

struct KernelArgs {
  AttnArgs a;
  float* part;      // [2 * gridDim][NR][D] partial sums of tiles that are cut
  float2* part_ml;  // [2 * gridDim][NR] (maximum, sum)
  int4* desc;       // [gridDim]: first row (low, high), rows, pieces of the tile that begins there and is cut
  uint32_t* watchdog;
  uint32_t wait_ns;  // the longest wait
  int shares;       // 1: blocks in equal shares; 0: whole tiles
  int stages;
};

// The query: rows of 16 bits, or two 8-bit parts of each row.
__host__ __device__ constexpr int q_bytes(int NR, int D, bool f8) {
  return f8 ? 2 * NR * ((D + 127) / 128 * 128) : NR * D * 2;
}

// What one work item (a tile, or a piece of its key blocks) covers.
struct alignas(16) Item {
  int b, r0, nrows, pos0;  // sequence, first row in it, rows, position of its first new token
  int p0, p1;              // positions of the tile's first and last row
  int u_lo, ns;            // first unit of the window, units of the sinks
  int units, blk0, blk1;   // units in all; this item's blocks of 8
  int piece;               // its slot among the partial sums, or -1: the whole tile
  int64_t qrow;            // first row of the tile in [T*H]
  int64_t pad;
};
static_assert(sizeof(Item) == 64, "four 16-byte words");
constexpr int kItems = 3;  // items handed out ahead
constexpr int kSlots = 2;  // blocks whose units are looked up, and fetched into L2, ahead

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], s_full[2], p_full, pv_done, q_full[4], q_empty, drain;
  uint64_t item_full[kItems], item_empty[kItems], slot_full[kSlots], slot_empty[kSlots], crow_empty[2];
  uint32_t tmem;
  int abort;
  alignas(16) Item items[kItems];
  int slots[kSlots][kUnits];  // cache row of each unit's first key; -1: none, -2: not needed
  alignas(16) float negm[64];
  float crow[2][64];  // 8-bit forms: what turns a row's products into scores
  float lthr[64];   // log2 of the weight from which the second part counts
  float scale[64];  // the rescale factors of a block; in the epilogue 1 / sum
  uint8_t rowt[64];  // a row's token, counted from the tile's first
  uint8_t hot[4][4];  // per group and quarter: units with such a weight (2 bits)
  float red[4][4][16];
};

// The weights P: part p of a key's NR rows lies p * NR elements into its row of
// 128 bytes, going on in further buffers of 128 such rows.
template <int NR, int DT>
constexpr int kPartBytes = NR * (Form<DT>::F8 ? 1 : 2);
template <int NR, int DT>
constexpr int kPBytes = (Form<DT>::PARTS * kPartBytes<NR, DT> + 127) / 128 * kChunkBytes;
constexpr int kSmemBudget = 232448;
template <int NR, int DT>
constexpr int smem_fixed(int D) {
  return kPBytes<NR, DT> + q_bytes(NR, D, Form<DT>::F8) + (int)sizeof(Shared);
}
template <int NR, int DT>
int stages_for(int D) {
  const int n = (kSmemBudget - smem_fixed<NR, DT>(D)) / Form<DT>::STAGE;
  return n < kMaxStages ? n : kMaxStages;
}
static_assert(smem_fixed<64, MXQ_CACHE_BF16>(512) + 4 * Form<MXQ_CACHE_BF16>::STAGE <= kSmemBudget, "a block fits");
static_assert(smem_fixed<64, MXQ_CACHE_E4M3>(512) + 8 * Form<MXQ_CACHE_E4M3>::STAGE <= kSmemBudget, "two blocks fit");

// A sequence: its first token, new tokens and keys.  Up to 32 at a time, one per lane.
struct Seq {
  int start, n, len, tiles;
  bool clamped;
};
template <int NR>
__device__ __forceinline__ Seq get_seq(const AttnArgs& a, int b) {
  Seq s = {0, 0, 0, 0, false};
  if (b < 0 || b >= a.B) return s;
  s.start = a.q_start != nullptr ? max(__ldg(a.q_start + b), 0) : b;
  const int end = a.q_start != nullptr ? (int)min((int64_t)__ldg(a.q_start + b + 1), a.T) : b + 1;
  s.n = max(end - s.start, 0);
  const int said = __ldg(a.seq_lens + b);
  s.len = min(max(said, 0), a.max_pages * a.page_size);
  s.clamped = said != s.len;
  s.tiles = (int)(((int64_t)s.n * a.H + NR - 1) / NR);
  return s;
}
// Tile t of a sequence: everything but its blocks and its piece.
template <int NR>
__device__ __forceinline__ Item get_tile(const AttnArgs& a, const Seq& s, int b, int t) {
  Item it;
  it.b = b;
  it.pos0 = s.len - s.n;
  it.r0 = t * NR;
  it.nrows = min(NR, s.n * a.H - it.r0);
  it.qrow = (int64_t)s.start * a.H + it.r0;
  it.p0 = it.pos0 + it.r0 / a.H;
  it.p1 = it.pos0 + (it.r0 + it.nrows - 1) / a.H;
  it.units = it.ns = it.u_lo = it.blk0 = it.blk1 = 0;
  it.piece = -1;
  it.pad = 0;
  if (it.p1 >= 0) {
    // (A tile may begin before its first key: p0 < 0, and the window be INT_MAX.)
    const int lo = a.window > 0 ? max(0, max(it.p0, 0) - a.window + 1) : 0;
    it.u_lo = lo / kUnit;
    const int sink_end = a.window > 0 ? min(a.sinks, lo) : 0;
    it.ns = min((sink_end + kUnit - 1) / kUnit, it.u_lo);
    it.units = it.ns + it.p1 / kUnit + 1 - it.u_lo;
  }
  return it;
}
// The work items of this CTA, in order; the lane that holds one gives it to
// `emit(item, lane)` (all lanes call it).  Tiles are walked from the last to
// the first, 32 at a time, one per lane: later tiles of a chunk see more keys.
template <int NR, typename Emit>
__device__ __forceinline__ void walk_items(const KernelArgs& k, Emit emit) {
  const AttnArgs& a = k.a;
  const int lane = threadIdx.x & 31;
  const int grid = (int)gridDim.x, cta = (int)blockIdx.x;
  if (k.shares && lane == 0) k.desc[cta] = make_int4(0, 0, 0, 0);
  __syncwarp();
  // Pass 0 (shares only) adds up the weights, pass 1 hands out the items.
  int share = 0, pos = 0, end = 0;  // this CTA's share of the line of all blocks
#pragma unroll 1
  for (int pass = k.shares ? 0 : 1; pass < 2; ++pass) {
    int run = 0;  // weight of the tiles so far; whole tiles: their number
#pragma unroll 1
    for (int base = (a.B - 1) & ~31; base >= 0; base -= 32) {
      const Seq s = get_seq<NR>(a, base + lane);
      int upto = s.tiles;  // tiles of this and the earlier sequences of the group
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
#pragma unroll 1
      for (int left = __shfl_sync(0xffffffffu, upto, 31); left > 0; left -= 32) {
        // This lane's tile of the group, and the sequence it belongs to: the
        // first whose count passes it.
        const int f = left - 1 - lane;
        int l = 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (__shfl_sync(0xffffffffu, upto, l + o - 1) <= f) l += o;
        Seq q;
        q.start = __shfl_sync(0xffffffffu, s.start, l);
        q.n = __shfl_sync(0xffffffffu, s.n, l);
        q.len = __shfl_sync(0xffffffffu, s.len, l);
        q.tiles = __shfl_sync(0xffffffffu, s.tiles, l);
        q.clamped = __shfl_sync(0xffffffffu, (int)s.clamped, l) != 0;
        const int t = f - (__shfl_sync(0xffffffffu, upto, l) - q.tiles);
        Item it = {};
        int nb = 0;
        if (f >= 0) {
          it = get_tile<NR>(a, q, base + l, t);
          nb = (it.units + kUnits - 1) / kUnits;
        }
        it.pad = q.clamped;
        // A tile weighs its blocks in the line; one that sees no key still has
        // its rows to write.  Whole tiles count one each.
        const int w = f < 0 ? 0 : k.shares ? max(nb, 1) : 1;
        int before = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += v;
        }
        const int sum = __shfl_sync(0xffffffffu, before, 31);
        before += run - w;  // weight before this tile
        run += sum;
        if (pass == 0) continue;
        bool mine;
        if (k.shares) {
          const int lo = max(pos - before, 0), hi = min(end - before, w);
          mine = lo < hi;
          it.blk0 = min(lo, nb);
          it.blk1 = min(hi, nb);
          if (mine && (lo > 0 || hi < w)) {
            // Slot 2c: the rest of a tile that an earlier CTA began; slot
            // 2c + 1: the beginning of one that the next CTA goes on with.
            it.piece = 2 * cta + (lo == 0 ? 1 : 0);
            if (lo == 0)
              k.desc[cta] = make_int4((int)(uint32_t)it.qrow, (int)(it.qrow >> 32), it.nrows,
                                      (before + w - 1) / share - cta + 1);
          }
        } else {
          it.blk1 = nb;
          mine = w > 0 && before % grid == cta;
        }
        for (uint32_t m = __ballot_sync(0xffffffffu, mine); m != 0; m &= m - 1)
          if (!emit(it, __ffs((int)m) - 1)) return;
        if (k.shares && run >= end) return;
      }
    }
    if (pass == 0) {
      // Equal shares; two blocks at least, since a cut costs about one.
      share = max((run + grid - 1) / grid, 2);
      pos = (int)min((int64_t)share * cta, (int64_t)run);
      end = pos + min(share, run - pos);
      if (pos == end) return;
    }
  }
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
// The same with 8-bit operands.
__device__ __forceinline__ void mma_f8(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                       uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 a, b;\n"
      "mov.b64 a, {%1, %2};\nmov.b64 b, {%3, %4};\n"
      "setp.ne.b32 p, %6, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Low and high words of a descriptor with 128-byte swizzle: address and
// leading offset; stride offset 1024 (eight 128-byte rows).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (ptx::kSwizzle128B << 29);
template <bool F8>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  if constexpr (F8)
    mma_f8(d, a_lo, kDescHi, b_lo, kDescHi, idesc, accumulate);
  else
    mma_f16(d, a_lo, kDescHi, b_lo, kDescHi, idesc, accumulate);
}

// Instruction descriptor: FP32 accumulation, operand types (kind::f16: 1 BF16;
// kind::f8f6f4: 0 E4M3, 1 E5M2), M = 128, N, and whether A and B are stored
// with M / N running fastest.
__host__ __device__ constexpr uint32_t idesc(uint32_t a, uint32_t b, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (a << 7) | (b << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | (8u << 24);
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
// One try of a barrier wait.  It returns as soon as the phase is over, and after
// 4 us if it is not (measured; a suspension hint of 20 ns to 2 us changes nothing).
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
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
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Two FP32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
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
__device__ __forceinline__ float out_of(bool has, uint32_t v) { return has ? __uint_as_float(v) : 0.0f; }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// What is left of two values after pack2, packed the same way.
__device__ __forceinline__ uint32_t pack2_rest(float lo, float hi, uint32_t w) {
  return pack2(lo - bf16_lo(w), hi - bf16_hi(w));
}
// Two values -> FP16, the first in the low half.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t v) { return __half22float2(*reinterpret_cast<__half2*>(&v)); }
__device__ __forceinline__ uint32_t add_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Four FP16 values -> four bytes: E5M2 cut, E5M2 and E4M3 to the nearest.
__device__ __forceinline__ uint32_t cut_e5m2(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7531); }
__device__ __forceinline__ uint32_t round_e5m2(uint32_t a, uint32_t b) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(lo) : "r"(a));
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(hi) : "r"(b));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ uint32_t round_e4m3(uint32_t a, uint32_t b) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(a));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(b));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
template <int N, int LAUNCH>
__device__ __forceinline__ void regs_set() {
  if constexpr (N > LAUNCH) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  if constexpr (N < LAUNCH) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(ptx::smem_u32(dst)),
      "l"(m), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

// --------------------------------------------------------------- widening
// A code's sign and its three magnitude bits, moved to BF16's sign and to the
// lowest two bits of its exponent and the highest of its fraction, are the code's
// value times 2^-126 (the code without exponent bits a subnormal one); a product
// with a power of two is then exact wherever the result is in BF16's range.  Two
// codes are moved by one multiplication: 2^a for the magnitudes and 2^b for the
// signs, which do not meet.  The codes that share a register are four apart: the
// stages hold the columns 0..7 in the order 0 4 1 5 2 6 3 7, as does Q, and the
// output is put back in order (1.1 operations of the half-rate pipe a value; a
// table by byte selection took 2.1, and the decode step of 32 sequences 193 us).
struct E2m1Scale {
  uint32_t m, past;  // 2^(sb - 1), or 2^127 and what is missing to it
};
__device__ __forceinline__ E2m1Scale e2m1_scale(uint32_t sb) {
  const uint32_t m = sb == 255u ? 0x7FFFu : (min(sb, 128u) + 126u) << 7, past = (max(sb, 128u) - 1u) << 7;
  return {m | (m << 16), past | (past << 16)};
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Eight codes -> eight BF16 values, in the order above.
__device__ __forceinline__ uint4 widen_e2m1x8(uint32_t w, const E2m1Scale& t, bool any_past) {
  constexpr uint32_t kKeep = 0x81C081C0u;
  const uint32_t v = w >> 8;
  uint32_t r[4] = {((w & 0x000F000Fu) * 0x1040u) & kKeep, ((w & 0x00F000F0u) * 0x104u) & kKeep,
                   ((v & 0x000F000Fu) * 0x1040u) & kKeep, ((v & 0x00F000F0u) * 0x104u) & kKeep};
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = mul_bf16x2(r[e], t.m);
  if (any_past)
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = mul_bf16x2(r[e], t.past);
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// Eight BF16 values, from the columns' order to the stages'.
template <int DT>
__device__ __forceinline__ uint4 to_stage_order(const uint4 v) {
  if constexpr (DT != MXQ_CACHE_E2M1) return v;
  return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                    __byte_perm(v.y, v.w, 0x7632));
}
// The column that place p of a stage holds.
template <int DT>
__device__ __forceinline__ int stage_column(int p) {
  return DT == MXQ_CACHE_E2M1 ? (p & ~7) | ((p >> 1) & 3) | ((p & 1) << 2) : p;
}

// Widening of a stage (128 keys x 128 columns) of E2M1 rows by NT threads:
// 16-byte pieces of the stored rows (32 codes, one scale), four to a row, RPT to a thread.
template <int NT>
struct Widen {
  static constexpr int TPR = 4, RPT = kKeys * TPR / NT;
  static constexpr int KSTEP = NT / TPR;     // key step between a thread's rows
  static_assert(KSTEP % 16 == 0 && RPT >= 1, "a thread's rows keep their place in a unit");
  const uint8_t* row[RPT];
  const uint8_t* sf[RPT];
  struct Piece {
    uint4 v[RPT];
    uint32_t sb[RPT];
  };

  // Rows t / TPR + i * KSTEP of a block whose units lie at su[0..7].
  __device__ __forceinline__ void open(const AttnArgs& a, const int* su, int t) {
    const int key0 = t / TPR, piece = t % TPR;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int u = su[(key0 + i * KSTEP) >> 4];
      const int64_t slot = (int64_t)u + (key0 & 15);
      const bool in = u >= 0 && slot < a.num_slots;
      row[i] = in ? static_cast<const uint8_t*>(a.cache) + slot * ((uint32_t)a.D / 2) + piece * 16 : nullptr;
      sf[i] = a.cache_sf + (in ? slot : 0) * (a.D >> 5) + piece;
    }
  }
  // The pieces (and scale bytes) of stage pr of the block.
  __device__ __forceinline__ void fetch(Piece& p, int D, int pr, int t) const {
    const bool in = pr * 128 + (t % TPR) * 32 < D;  // an odd last chunk: half a stage
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      p.v[i] = make_uint4(0, 0, 0, 0);
      p.sb[i] = 0;
      if (in && row[i] != nullptr) {
        p.v[i] = __ldg(reinterpret_cast<const uint4*>(row[i] + pr * (TPR * 16)));
        p.sb[i] = __ldg(sf[i] + pr * 4);
      }
    }
  }
  static __device__ __forceinline__ void store(const Piece& p, uint8_t* dst, int t) {
    const int key0 = t / TPR, piece = t % TPR, sw = key0 & 7;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      uint8_t* d = dst + (key0 + i * KSTEP) * 128;
      const E2m1Scale scale = e2m1_scale(p.sb[i]);
      const bool any_past = __any_sync(0xffffffffu, p.sb[i] > 128u);
      const int ch = piece >> 1, col = (piece & 1) * 4;
      d += ch * kChunkBytes;
      const uint32_t w[4] = {p.v[i].x, p.v[i].y, p.v[i].z, p.v[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // The second chunk's lanes take their words in another order, so that
        // eight lanes (two rows) always cover eight different 16-byte columns.
        const uint32_t we = ch ? w[e ^ 2] : w[e];
        *reinterpret_cast<uint4*>(d + (((col + (ch ? e ^ 2 : e)) ^ sw) << 4)) = widen_e2m1x8(we, scale, any_past);
      }
    }
  }
};

// ------------------------------------------------------------------ kernel
template <int NR, int DT>
__global__ void __launch_bounds__(Roles<NR>::THREADS, 1)
    attn_kernel(const __grid_constant__ CUtensorMap tm_kv, const KernelArgs k) {
  using R = Roles<NR>;
  using F = Form<DT>;
  constexpr bool F8 = F::F8;
  constexpr int NC = 16;                     // rows of a softmax group
  constexpr int kStageBytes = F::STAGE, kPart = kPartBytes<NR, DT>;
  extern __shared__ __align__(1024) uint8_t base[];
  const AttnArgs& a = k.a;
  const int D = a.D, nch = D >> 6, np = (nch + 1) >> 1;
  uint8_t* sm_stage = base;
  uint8_t* sm_p = sm_stage + (size_t)k.stages * kStageBytes;
  uint8_t* sm_q = sm_p + kPBytes<NR, DT>;
  Shared& sh = *reinterpret_cast<Shared*>(sm_q + q_bytes(NR, D, F8));
  volatile int* abort_flag = &sh.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    sh.abort = 0;
    for (int s = 0; s < k.stages; ++s) {
      ptx::mbar_init(&sh.full[s], DT == MXQ_CACHE_E2M1 ? R::LOADS : 1);
      ptx::mbar_init(&sh.empty[s], 1);
    }
    ptx::mbar_init(&sh.s_full[0], 1);
    ptx::mbar_init(&sh.s_full[1], 1);
    ptx::mbar_init(&sh.p_full, R::SOFT);
    ptx::mbar_init(&sh.crow_empty[0], R::SOFT);
    ptx::mbar_init(&sh.crow_empty[1], R::SOFT);
    ptx::mbar_init(&sh.pv_done, 1);
    for (int s = 0; s < 4; ++s) ptx::mbar_init(&sh.q_full[s], R::LOADS);
    ptx::mbar_init(&sh.q_empty, 1);
    ptx::mbar_init(&sh.drain, 1);
    for (int i = 0; i < kItems; ++i) {
      ptx::mbar_init(&sh.item_full[i], 1);
      // Readers: the softmax, loading, issuing and unit warps, and the TMA warp.
      ptx::mbar_init(&sh.item_empty[i], R::SOFT + R::LOADS + 2 + (DT == MXQ_CACHE_E2M1 ? 0 : 1));
    }
    for (int i = 0; i < kSlots; ++i) {
      ptx::mbar_init(&sh.slot_full[i], 1);
      ptx::mbar_init(&sh.slot_empty[i], R::SOFT + (DT == MXQ_CACHE_E2M1 ? R::LOADS : 1));
    }
    ptx::fence_barrier_init();
  }
  if (warp == R::MMA) {
    ptx::tmem_alloc(&sh.tmem, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();

  // A bounded wait; false once it or any other wait of the CTA gave up.  The
  // clock is read after a try that failed (its low word, whose differences have a
  // sign up to 2.1 s).
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    const uint32_t ad = ptx::smem_u32(bar);
    uint32_t end = 0;  // 0: no try has failed so far
#pragma unroll 1
    while (!try_wait(ad, parity)) {
      if (*abort_flag) return false;
      const uint32_t now = (uint32_t)ptx::globaltimer();
      if (end == 0) end = (now + k.wait_ns) | 1u;
      if ((int)(now - end) > 0) {
        *abort_flag = 1;
        return false;
      }
    }
    return true;
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

  uint32_t tma_st = 0, tma_stp = 0;  // the copying warp: the stage after its last, and that one's phase
  if (warp >= R::LOAD0) {
    // ------------------------------------- the query, and rows to be widened
    regs_set<R::REGS_LOAD, R::REGS>();
    const int lt = tid - R::LOAD0 * 32, lw = lt >> 5;
    int nq = 0;                // items with blocks so far
    [[maybe_unused]] uint32_t nb = 0;           // blocks so far
    [[maybe_unused]] uint32_t st = 0, stp = 0;  // stage and its phase
    bool ok = true;
    Item it;
    for (uint32_t ni = 0; ok && read_item(ni, it); ++ni) {
      if (it.blk0 >= it.blk1) continue;
      // Q rows, one per warp and step; rows past the tile's are zeros.
      if (nq > 0 && !(ok = wait_warp(&sh.q_empty, (uint32_t)(nq - 1) & 1u))) break;
      // The row scales of the item before the last are no longer read.
      if (F8 && !(ok = wait_warp(&sh.crow_empty[nq & 1], (uint32_t)((nq >> 1) & 1) ^ 1u))) break;
      const float kvs = DT == MXQ_CACHE_E4M3 ? __ldg(a.kv_scale) : 1.0f;
#pragma unroll 1
      for (int r0 = lw; r0 < NR; r0 += 4 * R::LOADS) {
        uint4 v[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            v[i][c] = make_uint4(0, 0, 0, 0);
            const int pc = c * 32 + lane, r = r0 + i * R::LOADS;
            if (pc < nch * 8 && r < it.nrows)
              v[i][c] = __ldg(reinterpret_cast<const uint4*>(a.q) + (it.qrow + r) * (nch * 8) + pc);
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + i * R::LOADS;
          if (r >= NR) break;
          float f = 1.0f;
          if constexpr (F8) {
            // Largest magnitude of the row -> the power of two that brings it
            // to [2^7, 2^8).  The products with both parts make up the score.
            uint32_t mx = 0;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t w[4] = {v[i][c].x, v[i][c].y, v[i][c].z, v[i][c].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) mx = max(mx, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
            }
            mx = __reduce_max_sync(0xffffffffu, mx);
            const int ex = (int)(mx >> 7);
            const int sft = mx == 0 ? 0 : min(134 - ex, 120);
            f = __uint_as_float((uint32_t)(127 + sft) << 23);
            // A row with a NaN or an infinity has no finite score.
            const float inv = ex == 255 ? NAN : __uint_as_float((uint32_t)(127 - sft) << 23);
            if (lane == 0) sh.crow[nq & 1][r] = r < it.nrows ? a.sm_scale * kLog2e * kvs * inv : 0.0f;
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int pc = c * 32 + lane;
            if (pc >= nch * 8) continue;
            if constexpr (!F8) {
              *reinterpret_cast<uint4*>(sm_q + (pc >> 3) * (NR * 128) + r * 128 + (((pc & 7) ^ (r & 7)) << 4)) =
                  to_stage_order<DT>(v[i][c]);
            } else {
              // BF16's 8 significant bits are two parts of E4M3's 4: rounded to
              // the nearest, and what is left, 16 times as large.
              float y[8];
              unpack8(v[i][c], y);
              uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                const float y0 = y[e] * f, y1 = y[e + 1] * f;
                const uint32_t h = e4m3x2(y0, y1);
                uint32_t b;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)h));
                const float2 w = __half22float2(*reinterpret_cast<__half2*>(&b));
                hi[e >> 2] |= h << (16 * ((e >> 1) & 1));
                lo[e >> 2] |= e4m3x2((y0 - w.x) * 16.0f, (y1 - w.y) * 16.0f) << (16 * ((e >> 1) & 1));
              }
              uint8_t* d = sm_q + (pc >> 4) * (2 * NR * 128) + r * 128 + ((((pc >> 1) & 7) ^ (r & 7)) << 4) + (pc & 1) * 8;
              *reinterpret_cast<uint2*>(d) = make_uint2(hi[0], hi[1]);
              *reinterpret_cast<uint2*>(d + NR * 128) = make_uint2(lo[0], lo[1]);
            }
          }
        }
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh.q_full[nq & 3]);
      ++nq;

      if constexpr (DT == MXQ_CACHE_E2M1) {
        // The next stage is fetched before the current one is stored; its rows
        // are in L2 by then (the unit warp's prefetch).
        using W = Widen<kLoadThreads>;
        W w;
        typename W::Piece p[2];
        int left = it.blk1 - it.blk0, pr = 0;
        auto open = [&]() -> bool {
          if (!wait_warp(&sh.slot_full[nb % kSlots], (nb / kSlots) & 1u)) return false;
          w.open(a, sh.slots[nb % kSlots], lt);
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sh.slot_empty[nb % kSlots]);
          ++nb;
          return true;
        };
        auto step = [&](const W::Piece& now, W::Piece& next) -> bool {
          if (++pr == np) {
            pr = 0;
            if (--left > 0 && !(ok = open())) return false;
          }
          if (left > 0) w.fetch(next, D, pr, lt);
          if (!(ok = wait_warp(&sh.empty[st], stp ^ 1u))) return false;
          W::store(now, sm_stage + st * kStageBytes, lt);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sh.full[st]);
          if (++st == (uint32_t)k.stages) {
            st = 0;
            stp ^= 1u;
          }
          return left > 0;
        };
        if (!(ok = open())) break;
        w.fetch(p[0], D, 0, lt);
        while (step(p[0], p[1]) && step(p[1], p[0])) {
        }
      }
    }
  } else if (warp == R::TMA) {
    regs_set<R::REGS_ISSUE, R::REGS>();
    if constexpr (DT != MXQ_CACHE_E2M1) {
      // ------------------------ BF16 and E4M3 rows: copied as they are by TMA
      // Lane u < 8 copies unit u of the block, one box of 16 rows x 128 bytes
      // per chunk.
      uint32_t st = 0, stp = 0, nb = 0;
      bool ok = true;
      Item it;
      for (uint32_t ni = 0; ok && read_item(ni, it); ++ni) {
        for (int blk = it.blk0; blk < it.blk1 && ok; ++blk) {
          if (!(ok = wait_warp(&sh.slot_full[nb % kSlots], (nb / kSlots) & 1u))) break;
          // A unit that is not in the cache is filled with its first rows (nothing
          // sees them): what lies in the stages depends on the arguments alone.
          int row = lane < kUnits ? sh.slots[nb % kSlots][lane] : -2;
          row = row == -1 ? 0 : row;
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sh.slot_empty[nb % kSlots]);
          ++nb;
          const uint32_t boxes = (uint32_t)__popc(__ballot_sync(0xffffffffu, row >= 0));
          for (int pr = 0; pr < np; ++pr) {
            if (!(ok = wait_warp(&sh.empty[st], stp ^ 1u))) break;
            const int chunks = F8 ? 1 : min(2, nch - pr * 2);
            if (lane == 0) ptx::mbar_arrive_expect_tx(&sh.full[st], boxes * (uint32_t)chunks * (kUnit * 128));
            __syncwarp();
            if (row >= 0)
              for (int c = 0; c < chunks; ++c)
                tma_load_2d(sm_stage + st * kStageBytes + c * kChunkBytes + lane * (kUnit * 128), &tm_kv,
                            &sh.full[st], F8 ? pr * 128 : (pr * 2 + c) * 64, row);
            if (++st == (uint32_t)k.stages) {
              st = 0;
              stp ^= 1u;
            }
          }
        }
      }
      tma_st = st;
      tma_stp = stp;
    }
  } else if (warp == R::MMA) {
    // ------------------------------------------------------------ products
    regs_set<R::REGS_ISSUE, R::REGS>();
    // Two cursors over the same sequence of blocks: the first product runs
    // ahead of the second by as much as the stages hold, two blocks at most
    // (the two S buffers).  Whatever is ready is issued, the second product
    // first, because it frees stages.
    const uint32_t dk0 = desc_lo(ptx::smem_u32(sm_stage), 16), dv0 = desc_lo(ptx::smem_u32(sm_stage), kChunkBytes);
    const uint32_t dp0 = desc_lo(ptx::smem_u32(sm_p), kChunkBytes), dq0 = desc_lo(ptx::smem_u32(sm_q), 16);
    constexpr uint32_t ta = F8 ? 0u : 1u;                    // type of the rows: E4M3 or BF16
    constexpr int kSteps = F8 ? kUnits / 2 : kUnits;         // second product: 32 or 16 keys at a time
    constexpr uint32_t kStep = F8 ? 256u : 128u;             // of descriptors: so many rows of 128 bytes
    constexpr uint32_t idesc_s = idesc(ta, F8 ? 0u : 1u, F8 ? 2 * NR : NR, false, false);
    constexpr uint32_t idesc_o = idesc(ta, 0u, NR, true, true), idesc_lo = idesc(ta, 0u, NC, true, true);
    // Where part i of the weights begins, in 16-byte units.
    auto part_at = [](int i) {
      return (uint32_t)((i * kPart / 128) * kChunkBytes + (i * kPart) % 128) >> 4;
    };
    // Items are read without blocking: those that see no key have nothing for
    // this warp, and the others may only move on once it has issued what is ready.
    uint32_t ni = 0;
    bool more = true;                 // the last item has not been read
    int qleft = 0, pleft = 0;         // blocks left of the two cursors' items
    int punits = 0, nwait = 0;        // units left of the second's; items it still has to begin,
    int wl0 = 0, wu0 = 0, wl1 = 0, wu1 = 0;  // at most two: it is two blocks behind at most
    int pdone = 0;                    // blocks of the second cursor's item that are behind it
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
        int kk = min(kUnits, punits);  // units in use; steps
        if (F8) kk = (kk + 1) >> 1;
        // Read before the products are issued: behind them a load waits for
        // the tensor pipe (measured: 7500 instead of 1700 cycles a block).
        uint32_t hot = 0;  // bit 8 q + i: group q, step i
        if (pdone >= 2)
#pragma unroll
          for (int q = 0; q < R::GROUPS; ++q) {
            // Byte i holds the units 2i and 2i + 1 in its low bits.
            const uint32_t w = *reinterpret_cast<const volatile uint32_t*>(sh.hot[q]);
            if constexpr (F8) {
              const uint32_t any = w | (w >> 1);
              hot |= ((any & 1u) | ((any >> 7) & 2u) | ((any >> 14) & 4u) | ((any >> 21) & 8u)) << (8 * q);
            } else {
              hot |= ((w | (w >> 6) | (w >> 12) | (w >> 18)) & 0xFFu) << (8 * q);
            }
          }
        hot &= 0x01010101u * ((1u << kk) - 1u);
        for (int m = 0; m < np; ++m) {
          if (ptx::elect_one()) {
            const uint32_t da = dv0 + ps * (kStageBytes >> 4);
            const uint32_t dd = tmem + m * NR;
            // The last parts: of all rows in the first two blocks, then 16 rows
            // at a time where there are any.
            const int parts = pdone < 2 ? F::PARTS : F::SURE;
#pragma unroll
            for (int i = 0; i < F::PARTS; ++i) {
              if (i >= parts) break;
#pragma unroll
              for (int u = 0; u < kSteps; ++u) {
                if (u >= kk) break;
                mma<F8>(dd, da + u * kStep, dp0 + part_at(i) + u * kStep, idesc_o | (F::part_type(i) << 10),
                        (pdone | i | u) ? 1u : 0u);
              }
            }
#pragma unroll 1
            for (uint32_t w = hot; w != 0; w &= w - 1) {
              const uint32_t bit = (uint32_t)__ffs((int)w) - 1u, q = bit >> 3, u = bit & 7u;
#pragma unroll
              for (int i = F::SURE; i < F::PARTS; ++i)
                mma<F8>(dd + q * NC, da + u * kStep, dp0 + part_at(i) + u * kStep + q * (F8 ? 1 : 2),
                        idesc_lo | (F::part_type(i) << 10), 1u);
            }
            ptx::tc_commit(&sh.empty[ps]);
          }
          __syncwarp();
          if (++ps == (uint32_t)k.stages) ps = 0;
        }
        if (ptx::elect_one()) ptx::tc_commit(&sh.pv_done);
        ++gp;
        ++pdone;
        punits -= kUnits;
        if (--pleft == 0) {
          pdone = 0;
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
            const uint32_t ds = tmem + kTmemS + (gq & 1u) * (F8 ? 2 * NR : 64);
#pragma unroll
            for (int e = 0; e < 4 * F::CHUNKS; ++e) {
              // 32 bytes of columns at a time; a chunk of 64 columns is 4 (2 of 8-bit ones).
              if (qpair * 2 + (F8 ? e >> 1 : e >> 2) >= nch) break;
              mma<F8>(ds, da + (e >> 2) * (kChunkBytes >> 4) + (e & 3) * 2, db + (e >> 2) * (NR * 128 >> 4) + (e & 3) * 2,
                      idesc_s, (qpair | e) ? 1u : 0u);
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
        if (!stop && ptx::globaltimer() - t0 > k.wait_ns) {
          stop = 1;
          if (lane == 0) *abort_flag = 1;
        }
        if (__any_sync(0xffffffffu, stop)) break;
      }
    }
    // Everything issued has completed before TMEM and shared memory go away.
    if (ptx::elect_one()) ptx::tc_commit(&sh.drain);
    __syncwarp();
    if (!ptx::mbar_wait(&sh.drain, 0, kWaitNs) && lane == 0) *abort_flag = 1;
  } else if (warp == R::ITEM) {
    // ------------------------------------------------------- work items
    // Decoded here once for all roles, up to three ahead.
    regs_set<R::REGS_ISSUE, R::REGS>();
    uint32_t i = 0;
    auto hand_out = [&](const Item& it, int owner) -> bool {
      if (!wait_warp(&sh.item_empty[i % kItems], ((i / kItems) & 1u) ^ 1u)) return false;
      if (lane == owner) {
        sh.items[i % kItems] = it;
        if (it.pad && a.err_flag != nullptr) atomicOr(a.err_flag, MXQ_DEVERR_LENGTH);
        ptx::mbar_arrive(&sh.item_full[i % kItems]);
      }
      __syncwarp();
      ++i;
      return true;
    };
    walk_items<NR>(k, hand_out);
    Item last = {};
    last.b = -1;
    hand_out(last, 0);
  } else if (warp == R::UNIT) {
    // ------------------------------------- where the units of a block lie
    // Lane u < 8 looks up unit u, a few blocks ahead of their use: the block
    // table's latency and the divisions stay out of the other warps' way.
    regs_set<R::REGS_ISSUE, R::REGS>();
    uint32_t nb = 0;
    bool ok = true;
    Item it;
    for (uint32_t ni = 0; ok && read_item(ni, it); ++ni) {
      for (int blk = it.blk0; blk < it.blk1; ++blk, ++nb) {
        const int x = blk * kUnits + lane;
        // The last 32 keys of an 8-bit form's product may end with a unit that is not there.
        int slot = x < (F8 ? (it.units + 1) & ~1 : it.units) ? -1 : -2;
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
        // The unit's rows lie one after the other: into L2, blocks ahead.
        if (slot >= 0) {
          const uint32_t row_bytes = (uint32_t)D * 2 / (DT == MXQ_CACHE_BF16 ? 1 : DT == MXQ_CACHE_E4M3 ? 2 : 4);
          const uint32_t rows = (uint32_t)min((int64_t)kUnit, a.num_slots - slot);
          ptx::prefetch_l2_bulk(static_cast<const uint8_t*>(a.cache) + (int64_t)slot * row_bytes, rows * row_bytes);
        }
        if (!(ok = wait_warp(&sh.slot_empty[nb % kSlots], ((nb / kSlots) & 1u) ^ 1u))) break;
        if (lane < kUnits) sh.slots[nb % kSlots][lane] = slot;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.slot_full[nb % kSlots]);
      }
    }
  } else {
    // ------------------------------------------------- softmax and epilogue
    regs_set<R::REGS_SOFT, R::REGS>();
    const int h = warp >> 2, quad = warp & 3;      // group, TMEM lane quadrant
    const uint32_t tq = tmem + ((uint32_t)(quad * 32) << 16);
    const int key = quad * 32 + lane;              // this thread's key of a block
    const int c0 = h * NC;
    const uint32_t bar = 1 + h;
    const float vs = DT == MXQ_CACHE_E4M3 ? __ldg(a.kv_scale) : 1.0f;
    const float c_all = a.sm_scale * kLog2e;  // of a 16-bit form's products
    const float4* negm4 = reinterpret_cast<const float4*>(sh.negm + c0);
    const float4* lthr4 = reinterpret_cast<const float4*>(sh.lthr + c0);
    uint32_t g = 0;   // blocks so far
    uint32_t st = 0;  // first stage of the current block
    int nq = 0;       // items with blocks so far
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
        sh.rowt[r] = (uint8_t)((held.r0 + r) / a.H - held.r0 / a.H);
        sh.lthr[r] = INFINITY;  // set before the third block
        if (F8) sh.negm[r] = r < it.nrows ? kNoKey : 0.0f;
      }
      // The key of the first block whose scores are the first reference: the
      // first of those that all rows see, where there is one.
      const int key_ref = has && a.window > 0 && it.ns == 0 && it.blk0 == 0
                              ? min(max(it.p1 - a.window + 1 - it.u_lo * kUnit, 0), kKeys - 1) : 0;
      ptx::named_sync(bar, 128);
      if (F8 && has) {
        // The row scales come with the query.
        ok = wait(&sh.q_full[nq & 3], (uint32_t)(nq >> 2) & 1u) && ok;
      }
      const float4* crow4 = reinterpret_cast<const float4*>(sh.crow[nq & 1] + c0);
      if (has) ++nq;
      float l[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) l[c] = 0.0f;
      for (int blk = it.blk0; blk < it.blk1; ++blk) {
        // Which rows see this thread's key: bit c for the group's row c.
        const int x = blk * kUnits + (key >> 4);
        const bool in = x < it.units;
        // Keys that the second product reaches (its steps may end with a unit that is not there).
        const bool live = F8 ? x < ((it.units + 1) & ~1) : in;
        const int j = unit_key(it, in ? x : 0) + (key & 15);
        const int weff = (a.window == 0 || j < a.sinks) ? 0x7fffffff : a.window;
        ok = wait(&sh.slot_full[g % kSlots], (g / kSlots) & 1u) && ok;
        const int unit_slot = sh.slots[g % kSlots][key >> 4];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.slot_empty[g % kSlots]);
        const bool some = in && j <= it.p1 && it.p0 - j < weff && unit_slot >= 0 &&
                          (int64_t)unit_slot + (key & 15) < a.num_slots;
        const bool all = some && j <= it.p0 && it.p1 - j < weff;
        uint32_t sees = all ? 0xFFFFu : 0u;
        if (__any_sync(0xffffffffu, some && !all)) {
          if (some && !all)
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if ((uint32_t)(it.p0 + sh.rowt[c0 + c] - j) < (uint32_t)weff) sees |= 1u << c;
          __syncwarp();
        }
        // Now and then, the sums so far: what a weight is measured against.
        const int done = blk - it.blk0;
        if (done >= 2 && (done & (done - 1)) == 0) {
          float v[NC];
#pragma unroll
          for (int c = 0; c < NC; ++c) v[c] = l[c];
          const float part = lanes_reduce<NC, false>(v);
          if (lane < NC) sh.red[h][quad][lane] = part;
          ptx::named_sync(bar, 128);
          if (quad == 0) {
            const int r = lane & 15;
            float t = INFINITY;
            if (c0 + r < it.nrows)
              t = __log2f((sh.red[h][0][r] + sh.red[h][1][r]) + (sh.red[h][2][r] + sh.red[h][3][r])) - 4.0f;
            sh.lthr[c0 + r] = t;
          }
          ptx::named_sync(bar, 128);
        }
        ok = wait(&sh.s_full[g & 1u], (g >> 1) & 1u) && ok;
        __syncwarp();
        ptx::tc_fence_after();
        const uint32_t ts = tq + kTmemS + (g & 1u) * (F8 ? 2 * NR : 64) + c0;
        // The scores of this thread's key, times log2(e), each plus add[c].
        auto scores = [&](float (&x)[NC], const float4* add) {
          uint32_t s[NC];
          if constexpr (F8) {
            uint32_t lo[NC];
            tmem_ld<NC>(ts, s);
            tmem_ld<NC>(ts + NR, lo);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < NC / 4; ++q) {
              const float4 cr = crow4[q], n = add != nullptr ? add[q] : make_float4(0.f, 0.f, 0.f, 0.f);
              const float2 ca = make_float2(cr.x, cr.y), cb = make_float2(cr.z, cr.w);
              const float2 sixteenth = make_float2(0.0625f, 0.0625f), zero = make_float2(0.f, 0.f);
              const float2 a0 = fma2(make_float2(__uint_as_float(lo[4 * q]), __uint_as_float(lo[4 * q + 1])), sixteenth,
                                     make_float2(__uint_as_float(s[4 * q]), __uint_as_float(s[4 * q + 1])));
              const float2 a1 = fma2(make_float2(__uint_as_float(lo[4 * q + 2]), __uint_as_float(lo[4 * q + 3])), sixteenth,
                                     make_float2(__uint_as_float(s[4 * q + 2]), __uint_as_float(s[4 * q + 3])));
              const float2 lo2 = fma2(a0, ca, add != nullptr ? make_float2(n.x, n.y) : zero);
              const float2 hi2 = fma2(a1, cb, add != nullptr ? make_float2(n.z, n.w) : zero);
              x[4 * q] = lo2.x;
              x[4 * q + 1] = lo2.y;
              x[4 * q + 2] = hi2.x;
              x[4 * q + 3] = hi2.y;
            }
          } else {
            tmem_ld<NC>(ts, s);
            ptx::tmem_ld_wait();
            const float2 cc = make_float2(c_all, c_all);
#pragma unroll
            for (int q = 0; q < NC / 4; ++q) {
              const float4 n = add != nullptr ? add[q] : make_float4(0.f, 0.f, 0.f, 0.f);
              const float2 lo2 = fma2(make_float2(__uint_as_float(s[4 * q]), __uint_as_float(s[4 * q + 1])), cc,
                                      make_float2(n.x, n.y));
              const float2 hi2 = fma2(make_float2(__uint_as_float(s[4 * q + 2]), __uint_as_float(s[4 * q + 3])), cc,
                                      make_float2(n.z, n.w));
              x[4 * q] = lo2.x;
              x[4 * q + 1] = lo2.y;
              x[4 * q + 2] = hi2.x;
              x[4 * q + 3] = hi2.y;
            }
          }
        };
        if (!F8 && done == 0) {
          uint32_t s[NC];
          if (quad == key_ref >> 5) {
            tmem_ld<NC>(ts, s);
            ptx::tmem_ld_wait();
            if (lane == (key_ref & 31))
#pragma unroll
              for (int c = 0; c < NC; ++c) {
                const float v = __uint_as_float(s[c]) * c_all;
                sh.negm[c0 + c] = ((sees >> c) & 1u) && fabsf(v) <= 3.4028234e38f ? -v
                                  : c0 + c < it.nrows ? kNoKey : 0.0f;
              }
          }
          ptx::named_sync(bar, 128);
        }
        float d[NC];
        // Units in which some weight is large against its row's sum so far.
        uint32_t hot = ~0u;
        // The 8-bit forms' weights have to stay near the reference, which is the
        // first block's maximum: there the weights are left for the second time.
        const bool skip = F8 && done == 0;
#pragma unroll 1
        for (bool again = false;;) {
          bool bad, raise = false;
          if (again || !skip) {
            // ---- exponents d = s + negm, and the weights in their place, before it
            // is known whether a reference has to move: it hardly ever has.
            scores(d, negm4);
            // The largest, NaN if one is: a cache row with a NaN or an infinity
            // has no finite score.
            float top = d[0];
#pragma unroll
            for (int c = 1; c + 1 < NC; c += 2) top = max3_nan(top, d[c], d[c + 1]);
            top = max_nan(top, d[NC - 1]);
            bad = live && !(fabsf(top) <= 3.4028234e38f);
            if (again && bad) {
              // A second time: what is not finite has no weight.
#pragma unroll
              for (int c = 0; c < NC; ++c)
                if (!(fabsf(d[c]) <= 3.4028234e38f)) d[c] = -INFINITY;
            }
            float most = top;  // of the rows that see the key
            if (some && !all) {
              most = -INFINITY;
#pragma unroll
              for (int c = 0; c < NC; ++c)
                if ((sees >> c) & 1u) most = fmaxf(most, d[c]);
            }
            raise = bad || (some && most > F::MOST);
            if (done >= 2) {
              bool big = false;
#pragma unroll
              for (int q = 0; q < NC / 4; ++q) {
                const float4 t = lthr4[q];
                big |= (d[4 * q] > t.x) | (d[4 * q + 1] > t.y) | (d[4 * q + 2] > t.z) | (d[4 * q + 3] > t.w);
              }
              hot = __ballot_sync(0xffffffffu, some && big);
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) d[c] = ex2(d[c]);
            if (sees != 0xFFFFu)
#pragma unroll
              for (int c = 0; c < NC; ++c)
                if (!((sees >> c) & 1u)) d[c] = 0.0f;
            if (again || !named_any(bar, 128, raise || !ok)) break;
          }
          again = true;
          // O is at rest once the previous block's second product is done.
          if (done > 0 && !wait(&sh.pv_done, (g - 1) & 1u)) ok = false;
          ptx::tc_fence_after();
          // ---- some reference moves, something is not finite, or a wait gave up
          if (named_any(bar, 128, !ok)) {
            dead = true;
            break;
          }
          // The scores again, and their maxima.
          scores(d, nullptr);
          bad = false;
#pragma unroll
          for (int c = 0; c < NC; ++c) bad |= !(fabsf(d[c]) <= 3.4028234e38f);
          bad = bad && live;
          if (bad) {
            // A row that holds a NaN or an infinity must not reach the rows
            // that do not see it through 0 * NaN: it is cleared here, and the
            // rows that see it become NaN through their sums.
            bool rowbad = false;
            const int words = F8 ? np * 8 : nch * 8;
#pragma unroll 1
            for (int e = 0; e < 2 * words; ++e) {  // the row's 16-byte words, twice over
              const int w8 = e >= words ? e - words : e, ch = w8 >> 3;
              const uint32_t sidx = (st + ch / F::CHUNKS) % (uint32_t)k.stages;
              uint4* wp = reinterpret_cast<uint4*>(sm_stage + sidx * kStageBytes + (ch % F::CHUNKS) * kChunkBytes +
                                                   key * 128) + (w8 & 7);
              if (e >= words) {
                if (rowbad) *wp = make_uint4(0, 0, 0, 0);
                continue;
              }
              const uint4 w = *wp;
              const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll 1
              for (int b = 0; b < 16; b += F8 ? 1 : 2) {
                // An exponent field of ones (E4M3: the one NaN code).
                const uint32_t v = ws[b >> 2] >> (8 * (b & 3));
                rowbad |= F8 ? (v & 0x7Fu) == 0x7Fu : (v & 0x7F80u) == 0x7F80u;
              }
            }
          }
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const bool fin = fabsf(d[c]) <= 3.4028234e38f, see = (sees >> c) & 1u;
            if (bad && !fin && see) l[c] = NAN;
            d[c] = see && fin ? d[c] : -INFINITY;
          }
          const float m = lanes_reduce<NC, true>(d);
          if (lane < NC) sh.red[h][quad][lane] = m;
          ptx::named_sync(bar, 128);
          if (quad == 0) {
            const int r = lane & 15;
            const float mb = fmaxf(fmaxf(sh.red[h][0][r], sh.red[h][1][r]), fmaxf(sh.red[h][2][r], sh.red[h][3][r]));
            const float old = sh.negm[c0 + r];
            float f = 1.0f, t = sh.lthr[c0 + r];
            __syncwarp();
            if (c0 + r < it.nrows && mb > -INFINITY && (old >= kNoKey || F::SHIFT - mb < old)) {
              if (old < kNoKey) f = ex2(F::SHIFT - mb - old);
              if (lane < NC) sh.negm[c0 + r] = F::SHIFT - mb;
              if (f != 1.0f) t += __log2f(f);  // stays infinite while it is
            }
            sh.scale[c0 + r] = f;
            sh.lthr[c0 + r] = t;
          }
          ptx::named_sync(bar, 128);
          if (done > 0) {
            bool moved = false;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const float f = sh.scale[c0 + c];
              l[c] *= f;
              moved |= f != 1.0f;
            }
            if (moved) {
#pragma unroll 1
              for (int o8 = 0; o8 < np * (NC / 8); ++o8) {
                uint32_t o[8];
                const int c = (o8 % (NC / 8)) * 8;
                const uint32_t ad = tq + (o8 / (NC / 8)) * NR + c0 + c;
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
        }
        if (dead) break;
#pragma unroll
        for (int c = 0; c < NC; c += 2) {
          const float2 v = add2(make_float2(l[c], l[c + 1]), make_float2(d[c], d[c + 1]));
          l[c] = v.x;
          l[c + 1] = v.y;
        }
        // ---- P, held back until the previous block's second product has read it
        auto free_p = [&]() {
          if (done > 0) {
            ok = wait(&sh.pv_done, (g - 1) & 1u) && ok;
            __syncwarp();
          }
          if (lane == 0) sh.hot[h][quad] = (uint8_t)(((hot & 0xFFFFu) ? 1 : 0) | ((hot >> 16) ? 2 : 0));
        };
        uint8_t* prow = sm_p + key * 128;
        // The 16 bytes of part i's row that begin `at` bytes into this group's.
        auto put = [&](int i, int at, const uint32_t* w) {
          const int b = i * kPart + c0 * (F8 ? 1 : 2) + at;
          *reinterpret_cast<uint4*>(prow + (b / 128) * kChunkBytes + (((b % 128) >> 4 ^ (key & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        };
        if constexpr (!F8) {
          free_p();
          uint32_t hi[NC / 2];
#pragma unroll
          for (int e = 0; e < NC / 2; ++e) hi[e] = pack2(d[2 * e], d[2 * e + 1]);
          put(0, 0, hi);
          put(0, 16, hi + 4);
          if (hot != 0) {
#pragma unroll
            for (int e = 0; e < NC / 2; ++e) hi[e] = pack2_rest(d[2 * e], d[2 * e + 1], hi[e]);
            put(1, 0, hi);
            put(1, 16, hi + 4);
          }
        } else {
          // The weights in FP16, whose upper bytes are the first parts; where some
          // weight is large, with what FP16 left of it, which joins the rest
          // before the third part is taken.
          uint32_t h[NC / 2], left[NC / 2], w[4][NC / 4];
#pragma unroll
          for (int e = 0; e < NC / 2; ++e) h[e] = pack_f16(d[2 * e], d[2 * e + 1]);
          if (hot != 0)
#pragma unroll
            for (int e = 0; e < NC / 2; ++e) {
              const float2 v = unpack_f16(h[e]);
              left[e] = pack_f16(d[2 * e] - v.x, d[2 * e + 1] - v.y);
            }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int q = 0; q < NC / 4; ++q) w[i][q] = cut_e5m2(h[2 * q], h[2 * q + 1]);
#pragma unroll
            for (int e = 0; e < NC / 2; ++e) h[e] = sub_f16x2(h[e], h[e] & 0xFF00FF00u);
          }
          if (hot == 0) {
#pragma unroll
            for (int q = 0; q < NC / 4; ++q) w[2][q] = round_e5m2(h[2 * q], h[2 * q + 1]);
          } else {
#pragma unroll
            for (int q = 0; q < NC / 4; ++q) {
              const uint32_t a0 = add_f16x2(h[2 * q], left[2 * q]), a1 = add_f16x2(h[2 * q + 1], left[2 * q + 1]);
              w[2][q] = round_e5m2(a0, a1);
              w[3][q] = round_e4m3(sub_f16x2(a0, __byte_perm(w[2][q], 0, 0x1404)),
                                   sub_f16x2(a1, __byte_perm(w[2][q], 0, 0x3424)));
            }
          }
          free_p();
          put(0, 0, w[0]);
          put(1, 0, w[1]);
          put(2, 0, w[2]);
          if (hot != 0) put(3, 0, w[3]);
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.p_full);
        ++g;
        st = (st + np) % (uint32_t)k.stages;
      }
      if (dead) break;
      if (F8 && has) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.crow_empty[(nq - 1) & 1]);
      }
      // ---- row sums over the 128 keys, then the output
      const float sum32 = lanes_reduce<NC, false>(l);
      if (lane < NC) sh.red[h][quad][lane] = sum32;
      if (has) ok = wait(&sh.pv_done, (g - 1) & 1u) && ok;
      if (named_any(bar, 128, !ok)) {
        dead = true;
        break;
      }
      ptx::tc_fence_after();
      if (quad == 0 && lane < NC) {
        const int r = c0 + lane;
        const float sum = (sh.red[h][0][lane] + sh.red[h][1][lane]) + (sh.red[h][2][lane] + sh.red[h][3][lane]);
        const float nm = has ? sh.negm[r] : kNoKey;
        if (held.piece >= 0) {
          k.part_ml[(int64_t)held.piece * NR + r] = make_float2(-nm, sum);
        } else {
          sh.scale[r] = sum == 0.0f ? 0.0f : vs / sum;
          if (r < it.nrows && a.lse != nullptr)
            a.lse[held.qrow + r] = sum == 0.0f ? -INFINITY : (__log2f(sum) - nm) * 0.6931471805599453f;
        }
      }
      ptx::named_sync(bar, 128);
      if (held.piece >= 0) {
        // Partial sums as they are: a lane holds a column, a warp stores 128
        // bytes of a row at a time.
        float* dst = k.part + ((int64_t)held.piece * NR + c0) * D + stage_column<DT>(key);
#pragma unroll 1
        for (int m = 0; m < np; ++m, dst += 128) {
          uint32_t o[NC];
          tmem_ld<NC>(tq + m * NR + c0, o);
          ptx::tmem_ld_wait();
          if (m * 128 + key < D) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
              if (c0 + c < held.nrows) dst[(int64_t)c * D] = __uint_as_float(o[c]);
          }
          __syncwarp();
        }
      } else {
        // The output: a lane holds a column, and the lanes of two neighbouring
        // columns swap halves of their rows, so that each stores pairs of columns
        // of eight rows.
        constexpr int kNext = DT == MXQ_CACHE_E2M1 ? 2 : 1;  // lane bit that is the column's lowest
        const bool odd = lane & kNext;
        const uint32_t pick = odd ? 0x3276u : 0x5410u;
        const int col = stage_column<DT>(key) & ~1, row = odd ? NC / 2 : 0;
        uint8_t* dst = static_cast<uint8_t*>(a.out) + ((held.qrow + c0 + row) * D + col) * 2;
        const int left = held.nrows - c0 - row;
        const float4* sc4 = reinterpret_cast<const float4*>(sh.scale + c0);
#pragma unroll 1
        for (int m = 0; m * 128 + col < D; ++m, dst += 256) {
          uint32_t o[NC];
          tmem_ld<NC>(tq + m * NR + c0, o);
          ptx::tmem_ld_wait();
          float v[NC];
#pragma unroll
          for (int q = 0; q < NC / 4; ++q) {
            const float4 sc = sc4[q];
            v[4 * q] = out_of(has, o[4 * q]) * sc.x;
            v[4 * q + 1] = out_of(has, o[4 * q + 1]) * sc.y;
            v[4 * q + 2] = out_of(has, o[4 * q + 2]) * sc.z;
            v[4 * q + 3] = out_of(has, o[4 * q + 3]) * sc.w;
          }
#pragma unroll
          for (int c = 0; c < NC / 2; ++c) {
            const uint32_t mine = pack2(v[c], v[c + NC / 2]);
            const uint32_t next = __shfl_xor_sync(0xffffffffu, mine, kNext);
            if (c < left) *reinterpret_cast<uint32_t*>(dst + (int64_t)c * D * 2) = __byte_perm(mine, next, pick);
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh.item_empty[ni % kItems]);
      ptx::tc_fence_before();
    }
  }
  __syncthreads();
  // After an abort, copies may be in flight that nobody has waited for: they land
  // before the shared memory goes away.  (Only here is it certain that no role
  // gives up any more: one may after the copying warp has issued its last copy.)
  if (DT != MXQ_CACHE_E2M1 && sh.abort && warp == R::TMA && lane == 0)
    for (int s = 0; s < k.stages; ++s)
      if (!ptx::mbar_wait(&sh.full[s], (uint32_t)s < tma_st ? tma_stp : tma_stp ^ 1u, kWaitNs / 8)) break;
  if (tid == 0 && sh.abort) atomicOr(k.watchdog, kWdAttn);
  if (warp == R::MMA) ptx::tmem_dealloc(tmem, kTmemCols);
}

// Joins the partial sums of the tiles that are cut: CTA (x, y) of the x-th of
// them, the one that begins in the x-th share c that has such a beginning.  Its
// pieces lie in the slots 2c + 1, 2(c + 1), 2(c + 2), ...; each counts
// 2^(its reference - the largest).  A warp adds up every WAYS-th piece of 128
// columns of a row, in order, BATCH at a time, so that their loads are under way
// together; the WAYS sums are added in order too: the result does not depend on
// timing.  Bound by latency: 9 to 12 us for 152 to 215 pieces of 64 rows x 512
// columns (20 to 28 MB from L2), 4 us for pieces of 16 rows, each by itself under
// the profiler; at most two rounds of CTAs, since each begins with the search
// (four rounds took 1 to 5 us more).
constexpr int kJoinThreads = 256, kJoinCtas = 1520;  // CTAs, about two to a place on the device
template <int NR, int WAYS>
__global__ void __launch_bounds__(kJoinThreads, WAYS == 8 ? 3 : 5) attn_join_kernel(const KernelArgs k, const int shares) {
  constexpr int WARPS = kJoinThreads / 32, ITEMS = WARPS / WAYS, BATCH = WAYS == 8 ? 8 : 4;
  __shared__ int pieces[kJoinThreads];
  __shared__ uint32_t begins[WARPS];
  __shared__ float4 part[WARPS][32];
  __shared__ float2 ml[WARPS];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const AttnArgs& a = k.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, way = warp % WAYS;
  const int np = (a.D + 127) >> 7;
  pieces[tid] = tid < shares ? k.desc[tid].w : 0;
  const uint32_t b = __ballot_sync(0xffffffffu, pieces[tid] != 0);
  if (lane == 0) begins[warp] = b;
  __syncthreads();
  int c = -1;
  for (int w = 0, skip = blockIdx.x; w * 32 < shares; ++w) {
    uint32_t m = begins[w];
    if (skip < __popc(m)) {
      for (; skip > 0; --skip) m &= m - 1;
      c = w * 32 + __ffs((int)m) - 1;
      break;
    }
    skip -= __popc(m);
  }
  if (c < 0) return;
  const int4 d = k.desc[c];
  const int used = pieces[c];
  // (NR rows of np parts are a whole number of rounds for every warp.)
#pragma unroll 1
  for (int item = blockIdx.y * ITEMS + warp / WAYS; item < NR * np; item += gridDim.y * ITEMS) {
    const int r = item / np, col = (item - r * np) * 128 + lane * 4;
    const bool here = r < d.z && col < a.D;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float mx = -INFINITY, sum = 0.0f;
    if (here) {
#pragma unroll 1
      for (int i0 = way; i0 < used; i0 += BATCH * WAYS) {
        float2 v[BATCH];
        float4 x[BATCH];
#pragma unroll
        for (int e = 0; e < BATCH; ++e) {
          const int i = i0 + e * WAYS;
          const int64_t at = (int64_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * NR + r;
          v[e] = i < used ? k.part_ml[at] : make_float2(-INFINITY, 0.f);
          x[e] = i < used ? *reinterpret_cast<const float4*>(k.part + at * a.D + col) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const float before = mx;
#pragma unroll
        for (int e = 0; e < BATCH; ++e) mx = fmaxf(mx, v[e].x);
        const float old = ex2(before - mx);
        sum *= old;
        o = make_float4(o.x * old, o.y * old, o.z * old, o.w * old);
#pragma unroll
        for (int e = 0; e < BATCH; ++e) {
          const float f = ex2(v[e].x - mx);
          sum += f * v[e].y;
          o.x += f * x[e].x;
          o.y += f * x[e].y;
          o.z += f * x[e].z;
          o.w += f * x[e].w;
        }
      }
    }
    if constexpr (WAYS > 1) {
      __syncthreads();  // the last ones have been read
      part[warp][lane] = o;
      if (lane == 0) ml[warp] = make_float2(mx, sum);
      __syncthreads();
      if (way != 0) continue;
#pragma unroll
      for (int w = 1; w < WAYS; ++w) mx = fmaxf(mx, ml[warp + w].x);
      sum = 0.0f;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WAYS; ++w) {
        const float f = ex2(ml[warp + w].x - mx);
        const float4 x = part[warp + w][lane];
        sum += f * ml[warp + w].y;
        o.x += f * x.x;
        o.y += f * x.y;
        o.z += f * x.z;
        o.w += f * x.w;
      }
    }
    if (!here) continue;
    const float vs = a.dtype == MXQ_CACHE_E4M3 ? __ldg(a.kv_scale) : 1.0f;
    const float inv = sum == 0.0f ? 0.0f : vs / sum;
    const int64_t row = (int64_t)(((uint64_t)(uint32_t)d.y << 32) | (uint32_t)d.x) + r;
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + (row * a.D + col) * 2) =
        make_uint2(pack2(o.x * inv, o.y * inv), pack2(o.z * inv, o.w * inv));
    if (col == 0 && a.lse != nullptr)
      a.lse[row] = sum == 0.0f ? -INFINITY : (__log2f(sum) + mx) * 0.6931471805599453f;
  }
}

// ---------------------------------------------------------------- host side
struct Plan {
  int NR, grid;
  int64_t tiles;  // at most, of this call
  bool shares;
  size_t part_bytes, ml_bytes, bytes;
};

// CTAs of the share form.  Workspace sizes come from the plan, which must not
// depend on the device; a device with fewer SMs runs them in turns.
constexpr int kShares = 152;
static_assert(kShares <= kJoinThreads, "a thread of the join looks at one share");

// Everything but `tiles` follows from what the workspace query takes, which is not
// told whether there is a q_start.
Plan make_plan(const AttnArgs& a) {
  Plan p;
  const int64_t rows = a.T * a.H, per_seq = rows / a.B;
  p.NR = per_seq > 32 ? 64 : per_seq > 16 ? 32 : 16;
  // Tiles, and key blocks of a tile, at most; T == B is taken as one token per
  // sequence, which a q_start need not bear out.
  const int64_t most = rows / p.NR + (a.B < rows ? a.B : rows);
  const int64_t tiles = a.T == a.B ? a.B * ceil_div(a.H, p.NR) : most;
  p.tiles = a.q_start == nullptr ? tiles : most;
  const int64_t cap = (int64_t)a.max_pages * a.page_size;
  int64_t keys = cap;
  if (a.window > 0) {
    const int64_t w = (int64_t)a.window + a.sinks + 2 * kUnit + (p.NR + a.H - 1) / a.H;
    keys = keys < w ? keys : w;
  }
  // Shares are even, but a cut costs about a block, and the pieces' sums and
  // their join about 16 stages (128 keys x 128 columns) of every CTA.  So whole
  // tiles where none has more than two blocks; where they leave fewer stages idle
  // in the last round of a few (301 tokens of each of 7 sequences, 12 heads of 192
  // columns, window 777: 53 us whole, 60 in shares; 500 of each of 2, 32 heads of
  // 256 columns over 4001 keys: 237 and 222); and from eight tiles a CTA, since
  // each CTA walks the line of all tiles before it begins its share.
  // (Weights are 32-bit numbers on the device.)
  const int64_t nb = ceil_div(keys, kKeys) + 1, idle = ceil_div(tiles, kShares) * kShares - tiles;
  p.shares = rows / p.NR < 8 * kShares && nb > 3 && most * nb < (int64_t)1 << 31 &&
             (tiles <= kShares || idle * nb * ceil_div(a.D, 128) > 16 * kShares);
  p.grid = p.shares || tiles > kShares ? kShares : (int)tiles;
  const size_t pieces = 2 * (size_t)p.grid;
  p.part_bytes = p.shares ? round_up_256(pieces * p.NR * a.D * 4) : 0;
  p.ml_bytes = p.shares ? round_up_256(pieces * p.NR * 8) : 0;
  p.bytes = p.shares ? p.part_bytes + p.ml_bytes + round_up_256((size_t)p.grid * 16) : 0;
  return p;
}

// BF16 or E4M3 cache rows as a 2-D map: boxes of 16 rows x 128 bytes, swizzled,
// zeros outside.
bool encode_rows(CUtensorMap* m, const void* base, bool f8, uint64_t D, uint64_t rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {D, rows};
  cuuint64_t strides[1] = {f8 ? D : D * 2};
  cuuint32_t box[2] = {f8 ? 128u : 64u, kUnit};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NR, int DT>
cudaError_t launch_one(KernelArgs k, int grid, int64_t tiles, cudaStream_t s, const char** why) {
  k.stages = stages_for<NR, DT>(k.a.D);
  auto kern = attn_kernel<NR, DT>;
  const int smem = smem_fixed<NR, DT>(k.a.D) + k.stages * Form<DT>::STAGE;
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
  if (DT != MXQ_CACHE_E2M1 && !encode_rows(&tm, k.a.cache, Form<DT>::F8, (uint64_t)k.a.D, (uint64_t)k.a.num_slots)) {
    *why = "cuTensorMapEncodeTiled failed (driver entry point missing or arguments rejected)";
    return cudaErrorInvalidValue;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(Roles<NR>::THREADS, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, tm, k);
  if (e != cudaSuccess || !k.shares) return e;
  // As many warps to a sum as a tile has a few pieces each for (shares over
  // tiles, at least).
  auto join = [&](auto join_kernel, int ways) {
    const int64_t rounds = NR * ceil_div(k.a.D, 128) * ways / (kJoinThreads / 32), x = tiles < grid ? tiles : grid;
    const int64_t y = ceil_div(kJoinCtas, x);
    cfg.gridDim = dim3((unsigned)x, (unsigned)(y < rounds ? y : rounds), 1);
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, join_kernel, k, grid);
  };
  if (tiles * 16 <= grid) return join(attn_join_kernel<NR, 8>, 8);
  if (tiles * 4 <= grid) return join(attn_join_kernel<NR, 4>, 4);
  return join(attn_join_kernel<NR, 1>, 1);
}

template <int NR>
cudaError_t launch_nr(const KernelArgs& k, int grid, int64_t tiles, cudaStream_t s, const char** why) {
  if (k.a.dtype == MXQ_CACHE_BF16) return launch_one<NR, MXQ_CACHE_BF16>(k, grid, tiles, s, why);
  if (k.a.dtype == MXQ_CACHE_E4M3) return launch_one<NR, MXQ_CACHE_E4M3>(k, grid, tiles, s, why);
  return launch_one<NR, MXQ_CACHE_E2M1>(k, grid, tiles, s, why);
}

}  // namespace

static std::atomic<uint32_t> g_wait_ns{kWaitNs};

uint32_t set_attn_wait(uint32_t ns) { return g_wait_ns.exchange(ns == 0 || ns > kWaitNs ? kWaitNs : ns); }

size_t attn_workspace_bytes(const AttnArgs& a) { return a.T > 0 ? make_plan(a).bytes : 0; }

cudaError_t launch_attn(const AttnArgs& a, void* ws, cudaStream_t s, const char** why) {
  const Plan p = make_plan(a);
  KernelArgs k = {};
  k.a = a;
  k.shares = p.shares;
  k.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
  uint8_t* w = static_cast<uint8_t*>(ws);
  k.part = reinterpret_cast<float*>(w);
  k.part_ml = reinterpret_cast<float2*>(w + p.part_bytes);
  k.desc = reinterpret_cast<int4*>(w + p.part_bytes + p.ml_bytes);
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
  if (p.NR == 64) return launch_nr<64>(k, p.grid, p.tiles, s, why);
  if (p.NR == 32) return launch_nr<32>(k, p.grid, p.tiles, s, why);
  return launch_nr<16>(k, p.grid, p.tiles, s, why);
}

}  // namespace mxq
