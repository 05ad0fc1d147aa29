// Products of E4M3 activations with 4-bit weights (E2M1 codes, an E8M0 scale
// per 32), dense and over routed experts.  Layouts and rules are stated in
// include/mxq.h.
//
// Mathematics:  out[t, n] = sum_k A[t, k] * W[n, k],
//   A = E4M3(a) * 2^(sa-127) (one sa per 128 k),
//   W = E2M1(w) * 2^(sw-127) (one sw per 32 k),
// with the products and scales exact on the tensor cores (kind::mxf8f6f4 takes
// E2M1 and E4M3 operands side by side) and fp32 sums.  The routed form makes
//   h = q8(silu(gate) * up)  and  out[t] = sum_j w_tj * W2[e_tj] h_tj
// of two such products, q8 being the group-128 quantisation of the other
// operators.
//
// Form: weight rows on the MMA's M axis (128), tokens on N (16..240), so that
// few tokens cost no padding.  The prepared weight is a sequence of 8704-byte
// blocks, each 128 rows x 128 columns of codes (64 bytes a row) and the
// 512-byte scale atom of those rows: one block is one pipeline stage's operand,
// and a row block's stages lie one behind the other in memory.  TMA unpacks the
// codes on the way into shared memory (16 codes in 8 bytes of a 16-byte chunk,
// 128-byte swizzle; the barrier counts the 8192 bytes read), where the MMA reads
// them; no instruction touches a weight.
//
// A unit is 128 weight rows (gate and up rows: twice 128) x a tile of tokens.
// Warp roles:
//   warp 0   copies: weight codes and scale atoms, and the token tile.
//   warp 1   TMEM owner; per stage tcgen05.cp of the scale atoms, four
//            tcgen05.mma for each 128 rows (K = 32 each, scale byte k of each
//            word), commit.  The MMA's N is the tile's own number of tokens,
//            rounded up to 16.
//   warp 2   token scales, one byte per row and stage, into the scale atom; for
//            few rows of the gate and up product also the token rows themselves,
//            gathered by index four to an instruction.
//   warp 3   prefetches into L2 (the epilogue's warps begin at a multiple of four).
//   warps 4- epilogue: groups of four warps, one for each TMEM lane quadrant, take
//            16 tokens at a time straight from TMEM: a lane holds one weight row.
//            Stores of a warp are contiguous along the rows; the abs-max of a
//            scale group (128 rows of a token) is a warp-wide maximum and an
//            exchange between the group's four warps.  (By way of shared memory, a lane
//            for eight rows, a call of 4096 tokens over 64 experts took a fifth longer.)
// Roles and operands are uniform to the compiler (a warp's role is broadcast, one
// elected lane issues): a warp that issues a copy or an MMA behind a lane's test
// spends its time moving operands (64 tokens over 128 experts took a third longer).
// Three forms:
//   split      few units: one unit for each cluster of up to 8 CTAs, which share
//              its K range.  Each CTA owns some of the tokens, receives the partial
//              sums for them through distributed shared memory and adds them in
//              rank order.
//   streaming  CTAs walk the units with a stride of the grid; copies run ahead
//              across units and the accumulator is doubled where TMEM allows it,
//              so that one unit's epilogue overlaps the next one's products.  Tiles of
//              up to 64 tokens, 128 in the dense product.
//   pairs      the same with two CTAs to a unit, for tiles of up to 240 tokens; see
//              w4_pair_kernel.
// A routed call is up to five kernels: plan (rows sorted by expert, tiles), rows
// (laid out by expert, for large tiles), gate and up, down, join (the sum over a
// token's experts).  Up to 16 rows take two; see w4_kernel.
//
// What bounds it, measured (floors: a copy's 6.78 TB/s, 3.78 PFLOP/s, twice the measured
// BF16 rate):
//   dense, 1 x 4096 x 4096      5.4 us (floor 1.3): launch, first copies, the sum over
//                               the cluster, one after the other
//   dense, 8192 x 4096 x 4096   79 us, 3.5 PFLOP/s (0.92); 2048 rows 24 us (0.76: two
//                               rounds of pairs, and the first copies and last epilogue)
//   64 tokens, 128 experts      127 us (0.98): HBM
//   1 token, 8 of 128           20 us (0.38): two kernels of 35 and 18 MB, each with the
//                               latencies of the first case
//   1024 tokens, 128 experts    232 us (0.55); over 64 145 (0.45): weights of an expert read
//                               for tiles of a few dozen rows, results written and read
//   4096 tokens, 64 experts     351 us (0.47): gate and up 143 us (tensor pipe 62 %
//                               active; one accumulator, so that the epilogue's fetches
//                               wait for the products and the other way round), down 116
//                               (copies from L2 and 402 MB of results at once), the sum 63
//                               and the rows 19 (both memory), the plan 11, each on cold
//                               caches
//
// Every wait is bounded in wall time; on expiry the kernel sets a watchdog bit,
// stops issuing, waits for its own copies and MMAs, frees TMEM and returns.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "kv_common.cuh"
#include "mxq.h"
#include "mxq_internal.h"
#include "mxq_ptx.cuh"
#include "quant_common.cuh"

namespace mxq {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // bmm.cu

namespace {

constexpr uint32_t kWaitNs = 2000000000u;  // default and longest bound on a wait
constexpr uint64_t kDrainNs = 2000000000ull;  // on what ends by itself once issuing has stopped
std::atomic<uint32_t> g_wait_ns{kWaitNs};  // see mxq_debug_set_w4_wait
constexpr uint32_t kHintNs = 20;
constexpr uint32_t kWdW4 = 0x80;  // a wait of these kernels ran out

constexpr int kCodeBytes = 128 * 64;    // a block's codes in memory
constexpr int kTileBytes = 128 * 128;   // the same, unpacked in shared memory
constexpr int kBlockBytes = kW4BlockBytes;
static_assert(kBlockBytes == kCodeBytes + kSfAtomBytes, "block layout");
constexpr int kChunk = 16;       // tokens drained at a time
constexpr int kMaxTokens = 240;  // of a tile (of CTA pairs): two accumulators and scale columns fit TMEM

enum Mode { kLinear = 0, kGateUp = 1, kDown = 2 };

// Device-side plan of a routed call: which sorted rows each tile holds.
struct alignas(16) Tile {
  int32_t expert, row0, count;
  uint32_t pairs;  // small calls: bit i: pair i (token * k + choice) is one of its rows;
                   // others: whether it is its expert's only tile
};
// Pairs and choices of a call that needs no plan: a warp sorts the pairs in its
// registers.
constexpr int kSmallPairs = 16;
constexpr int kMaxCluster = 8;    // CTAs of a cluster on any device
constexpr int kSmallChoices = kMaxCluster;

struct W4Args {
  const uint8_t* w;       // prepared weight
  const uint8_t* a_sf;    // [rows][KG]
  const Tile* tiles;      // routed forms
  const int32_t* n_tiles;
  const int32_t* perm;    // sorted row -> token * k + choice
  void* out;              // kLinear: BF16 [T][N]; kGateUp: codes [rows][N]; kDown: fp32 [rows][N]
  uint8_t* out_sf;        // kGateUp: [rows][NG]
  uint32_t* wd;           // watchdog word
  uint32_t wait_ns;       // bound on a wait
  int T, N, KG, KB, NB, NG, k;
  int per_tile, n_tiles_host;  // kLinear: tokens of a tile, tiles
  int splits, kb_per_split;  // CTAs of a cluster, K blocks of each
  int k_parts;               // small calls, down: CTAs of each choice
  // Small calls: ids instead of a plan; the gate and up product brings w2 into L2.
  const int32_t* ids;
  const float* wt;
  int32_t* err_flag;
  const uint8_t* w2;
  int E, KB2, NB2;
};

// The up to 16 pairs of a small call, sorted by expert in a warp's registers.
struct Pairs {
  int id;            // of pair `lane`
  bool valid;
  uint32_t peers;    // the pairs with the same expert
  uint32_t valids, leaders;  // valid pairs; the first pair of each expert

  __device__ __forceinline__ void load(const W4Args& p, int lane) {
    const int n = p.T * p.k;
    id = lane < n ? p.ids[lane] : -1;
    valid = id >= 0 && id < p.E;
    peers = __match_any_sync(0xffffffffu, valid ? id : -1 - lane);
    valids = __ballot_sync(0xffffffffu, valid);
    leaders = __ballot_sync(0xffffffffu, valid && (peers & ((1u << lane) - 1u)) == 0u);
  }
  // Pairs of the experts before the one that pair `leader` leads.
  __device__ __forceinline__ int before(int leader) const {
    return __popc(__ballot_sync(0xffffffffu, valid && __ffs(peers) - 1 < leader));
  }
  __device__ __forceinline__ Tile tile(int j) const {
    uint32_t m = leaders;
    for (int i = 0; i < j; ++i) m &= m - 1u;
    const int l = __ffs(m) - 1;
    Tile t;
    t.expert = __shfl_sync(0xffffffffu, id, l);
    t.pairs = __shfl_sync(0xffffffffu, peers, l);
    t.count = __popc(t.pairs);
    t.row0 = before(l);
    return t;
  }
  static __device__ __forceinline__ int row(const Tile& t, int i) {
    uint32_t m = t.pairs;
    for (; i > 0; --i) m &= m - 1u;
    return __ffs(m) - 1;
  }
  // The sorted row of pair `lane`.
  __device__ __forceinline__ int place(int lane) const {
    int r = 0;
    for (int l = 0; l < kSmallPairs; ++l) {
      const uint32_t o = __shfl_sync(0xffffffffu, peers, l);
      if ((valids >> l) & 1u) r += __ffs(o) < __ffs(peers) || (o == peers && l < lane) ? 1 : 0;
    }
    return r;
  }
};

// Two fp32 sums of a product at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n.reg .b64 a, b, c, r;\n"
      "mov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 r, a, b, c;\nmov.b64 {%0, %1}, r;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// Shape of an instance.  GATHER: the token rows are fetched by index.  SMALL: see
// w4_kernel.
template <int MODE, int NT, bool SPLIT, int SMALL = 0>
struct Cfg {
  static constexpr bool BY_CHOICE = SMALL != 0 && MODE == kDown;
  static constexpr int NA = MODE == kGateUp ? 2 : 1;
  static constexpr bool GATHER = MODE == kGateUp && NT <= 32;
  // Stages and CTAs per SM: as many bytes under way as shared memory allows; two
  // CTAs where the tile is small, so that one streams while the other turns
  // around.
  static constexpr int CTAS = SMALL == 2 ? 4 : NA == 1 && NT <= 64 ? 2 : 1;
  static constexpr int GROUPS = NT <= 64 || SPLIT ? 1 : 3;  // epilogue groups
  static constexpr int THREADS = 128 + 128 * GROUPS;
  static constexpr int TOK_TILE = NT * 128;
  static constexpr int STAGE = NA * (kTileBytes + kSfAtomBytes) + TOK_TILE + kSfAtomBytes;
  // Split K: the partial sums that the CTA receives, fp32
  // [rank][owned token][accumulator][row].
  static constexpr int SUM_BYTES = BY_CHOICE ? kSmallChoices * 512 : SPLIT ? NA * NT * 512 : 0;
  // For each epilogue group: two chunks' maxima of its four warps.
  static constexpr int MAX_BYTES = MODE == kGateUp ? GROUPS * 2 * 4 * kChunk * 4 : 0;
  static constexpr int LIMIT = (CTAS == 4 ? 56 * 1024 : CTAS == 2 ? 113 * 1024 : 232448) - 1024 - 512;
  static constexpr int FIT = (LIMIT - SUM_BYTES - MAX_BYTES) / STAGE;
  static constexpr int NSTAGE = FIT > 10 ? 10 : FIT;
  static constexpr int OFF_W = 0;
  static constexpr int OFF_TOK = NSTAGE * NA * kTileBytes;
  static constexpr int OFF_WSF = OFF_TOK + NSTAGE * TOK_TILE;
  static constexpr int OFF_TSF = OFF_WSF + NSTAGE * NA * kSfAtomBytes;
  static constexpr int OFF_SUM = OFF_TSF + NSTAGE * kSfAtomBytes;
  static constexpr int OFF_MAX = OFF_SUM + SUM_BYTES;
  static constexpr int OFF_BAR = OFF_MAX + MAX_BYTES;
  static constexpr int SMEM = OFF_BAR + (2 * NSTAGE + 5) * 8 + 32 + 1024;
  // TMEM: accumulators, then a ring of scale columns.  A copy of scales into
  // columns that earlier MMAs read is ordered behind them (both are issued by one
  // thread and execute in order); the ring keeps the copy from waiting.
  static constexpr int SF_COLS = 4 * NA + 4;
  static constexpr int NBUF = !SPLIT && 2 * NA * NT + 2 * SF_COLS <= 512 / CTAS ? 2 : 1;
  static constexpr int SF_RING = (512 / CTAS - NBUF * NA * NT) / SF_COLS >= 4 ? 4 : 2;
  static constexpr int TMEM_USED = NBUF * NA * NT + SF_RING * SF_COLS;
  static constexpr int TMEM_COLS = TMEM_USED <= 64 ? 64 : TMEM_USED <= 128 ? 128 : TMEM_USED <= 256 ? 256 : 512;
  // kind::mxf8f6f4: A E2M1 (format 5), B E4M3 (0), UE8M0 scales (bit 23), M >> 4
  // at bits 24-28; N >> 3 (bits 17-22) is the tile's; the scale byte of each
  // operand is chosen at bits 4-5 (B) and 29-30 (A).
  static constexpr uint32_t IDESC = (5u << 7) | (1u << 23) | ((128u >> 4) << 24);
  static_assert(NSTAGE >= 2 && SMEM <= 232448 && TMEM_COLS * CTAS <= 512, "budgets");
  static_assert(tmem_allowed(SMEM) >= TMEM_COLS, "TMEM beside other kernels' CTAs");
  static_assert(NT % kChunk == 0 && NT <= 128 && (!SPLIT || NT <= 32), "tokens of a tile");
};

// silu(g) * u.  The fast exponential (off by 2^-22 and 2^-23 |g| of itself) and
// quotient (2^-22) are far inside the step of the 8-bit codes that follow; the
// exact ones are a third of the epilogue's instructions.  Below g = -87, where silu(g) is
// smaller than 2^-119, the result is zero.
__device__ __forceinline__ float swiglu(float g, float u) {
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

// What four warps do with 16 tokens: v[a][i] is token i's sum for weight row
// n = 128 rb + 32 q + lane; `live` of them exist, the first being row `row` of the
// output.  max_: the group's maxima (double buffered), bar its barrier.
template <int MODE, int NA>
__device__ __forceinline__ void finish_chunk(const W4Args& p, float (&v)[NA][kChunk], int row,
                                             int live, int rb, int q, int lane, float* max_,
                                             int bar) {
  const int n = rb * 128 + q * 32 + lane;
  const bool in = n < p.N;
  if constexpr (MODE == kLinear) {
    // Neighbouring lanes swap a token each, so that a lane stores two rows of one.
    const int odd = lane & 1;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + (size_t)(row + odd) * p.N + (n - odd);
#pragma unroll
    for (int i = 0; i < kChunk; i += 2) {
      const float got = __shfl_xor_sync(0xffffffffu, odd ? v[0][i] : v[0][i + 1], 1);
      const uint32_t w = odd ? pack2(got, v[0][i + 1]) : pack2(v[0][i], got);
      if (in && i + odd < live) *reinterpret_cast<uint32_t*>(o + (size_t)i * p.N) = w;
    }
  } else if constexpr (MODE == kGateUp) {
    float h[kChunk];
    uint32_t mine = 0u;  // lane i: the warp's abs-max of token i, as bits
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      h[i] = swiglu(v[0][i], v[NA - 1][i]);
      const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(h[i]) & 0x7FFFFFFFu);
      if (lane == i) mine = m;
    }
    if (lane < kChunk) max_[q * kChunk + lane] = __uint_as_float(mine);
    ptx::named_sync(bar, 128);
    float inv = 0.0f;
    if (lane < kChunk) {
      uint32_t m = 0u;  // (as bits: a NaN counts as the largest)
#pragma unroll
      for (int w = 0; w < 4; ++w) m = max(m, __float_as_uint(max_[w * kChunk + lane]));
      uint32_t sb;
      inv = group_scale(__uint_as_float(m), &sb);
      if (q == 0 && lane < live && rb < p.NG) p.out_sf[(size_t)(row + lane) * p.NG + rb] = (uint8_t)sb;
    }
    // Four neighbouring lanes swap the codes of four tokens, so that each stores four
    // rows of one (64 tokens over 128 experts 1 us less than with single bytes).
    const int tok = lane & 3;
    const uint32_t pick2 = lane & 2 ? 0x3276u : 0x5410u, pick1 = lane & 1 ? 0x3715u : 0x6240u;
    uint8_t* o = static_cast<uint8_t*>(p.out) + (size_t)(row + tok) * p.N + (n - tok);
#pragma unroll
    for (int i = 0; i < kChunk; i += 4) {
      uint32_t w = 0u;
#pragma unroll
      for (int j = 0; j < 4; j += 2)
        w |= e4m3x2(__fmul_rn(h[i + j], __shfl_sync(0xffffffffu, inv, i + j)),
                    __fmul_rn(h[i + j + 1], __shfl_sync(0xffffffffu, inv, i + j + 1))) << (8 * j);
      w = __byte_perm(w, __shfl_xor_sync(0xffffffffu, w, 2), pick2);
      w = __byte_perm(w, __shfl_xor_sync(0xffffffffu, w, 1), pick1);
      if (in && i + tok < live) *reinterpret_cast<uint32_t*>(o + (size_t)i * p.N) = w;
    }
  } else {
    // FP32, as the sum over a token's experts takes them: what a column loses must not
    // hang on its neighbours, nor a token's result on the number of others in the call.
    float* o = static_cast<float*>(p.out) + (size_t)row * p.N + n;
    if (live >= kChunk && rb * 128 + 128 <= p.N) {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) o[(size_t)i * p.N] = v[0][i];
    } else {
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (in && i < live) o[(size_t)i * p.N] = v[0][i];
    }
  }
}

// The same for one token in a half-warp: v[a] are the lane's eight sums, from
// weight row n = 128 rb + 8 sub on.  All 32 lanes call it (in: the token exists).
template <int MODE, int NA>
__device__ __forceinline__ void finish_token(const W4Args& p, const float (&v)[NA][8], int row,
                                             int rb, int sub, bool in) {
  const int n = rb * 128 + 8 * sub;
  const bool store = in && n < p.N;
  if constexpr (MODE == kLinear) {
    if (store)
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + (size_t)row * p.N + n) =
          to_bf16x8(v[0]);
  } else if constexpr (MODE == kGateUp) {
    float h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = swiglu(v[0][e], v[NA - 1][e]);
    uint32_t sb;
    const float amax = half_warp_amax(h);
    const uint2 codes = encode8(h, amax, &sb);
    if (store) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + (size_t)row * p.N + n) = codes;
      if (sub == 0) p.out_sf[(size_t)row * p.NG + rb] = (uint8_t)sb;
    }
  } else {
    if (store) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + (size_t)row * p.N + n);
      o[0] = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
      o[1] = make_float4(v[0][4], v[0][5], v[0][6], v[0][7]);
    }
  }
}

// SMALL: a routed call of at most kSmallPairs rows and kSmallChoices choices, whose
// CTAs sort the rows themselves.  Its down product takes one token's 128 columns
// for each cluster and one of the token's experts (or, of few, a part of one's K
// range) for each CTA, and adds the experts' sums as a split K adds its parts: no
// results of single experts, and no kernel to add them.  One token over 8 of 128
// experts, 4096 x 1024: 20 us, with plan, results and sum half as long again.  SMALL == 2: the down
// product with four CTAs to an SM, of two stages each instead of five, for grids
// that fill more than two: 2 tokens over 8 of 128 (512 CTAs) 30.5 us against 34,
// one over 2 of 8, 4096 x 14336 (256 CTAs of 28 stages) 52 against 45.5.
template <int MODE, int NT, bool SPLIT, int SMALL>
__global__ void __launch_bounds__(Cfg<MODE, NT, SPLIT, SMALL>::THREADS, (Cfg<MODE, NT, SPLIT, SMALL>::CTAS))
    w4_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a,
              const W4Args p) {
  using C = Cfg<MODE, NT, SPLIT, SMALL>;
  constexpr int NA = C::NA, NSTAGE = C::NSTAGE;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + NSTAGE;
  uint64_t* acc_full = empty + NSTAGE;  // [2]
  uint64_t* acc_empty = acc_full + 2;   // [2]
  uint64_t* done = acc_empty + 2;       // every MMA has completed
  uint32_t* slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(slot + 1);
  volatile int* issued = reinterpret_cast<volatile int*>(slot + 2);  // [0] warp 0, [1] warp 2

  // (Broadcast: the compiler then knows that a warp's role and what follows from
  // it are the same in all lanes, and keeps the operands of copies and MMAs in
  // uniform registers instead of moving them there each time.)
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  const int split = SPLIT ? (int)ptx::cluster_rank() : 0;
  constexpr bool BY_CHOICE = C::BY_CHOICE;  // a cluster's CTAs are a token's choices
  static_assert(!BY_CHOICE || SPLIT, "choices are summed over a cluster");
  const int choice = BY_CHOICE ? split / p.k_parts : 0;
  const int kb0 = SPLIT ? (BY_CHOICE ? split - choice * p.k_parts : split) * p.kb_per_split : 0;
  int nk = SPLIT ? max(0, min(p.KB - kb0, p.kb_per_split)) : p.KB;
  const int u_first = SPLIT ? (int)(blockIdx.x / (uint32_t)p.splits) : (int)blockIdx.x;
  // The weight does not depend on what runs before: bring the first blocks into L2
  // while that finishes.  (Everything up to the wait runs beside it.)
  if (MODE == kLinear && warp == 3 && lane < NSTAGE && lane < nk)
    ptx::prefetch_l2_bulk(p.w + ((size_t)(u_first % p.NB) * p.KB + kb0 + lane) * kBlockBytes, kBlockBytes);
  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&tm_w);
    ptx::prefetch_tmap(&tm_a);
    for (int i = 0; i < NSTAGE; ++i) {
      ptx::mbar_init(&full[i], 2);
      ptx::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&acc_full[i], 1);
      ptx::mbar_init(&acc_empty[i], 4 * C::GROUPS);
    }
    ptx::mbar_init(done, 1);
    ptx::fence_barrier_init();
    *abort_flag = 0;
    issued[0] = issued[1] = 0;
  }
  if (warp == 1) {
    ptx::tmem_alloc(slot, C::TMEM_COLS);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);
  // Only now, with its TMEM in hand, may the next kernel begin: its CTAs may sit
  // beside this one and take theirs before they wait for this grid to end.
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  int units;
  Pairs pairs;
  if constexpr (MODE == kLinear) {
    units = p.n_tiles_host * p.NB;
  } else if constexpr (SMALL != 0) {
    pairs.load(p, lane);
    if constexpr (BY_CHOICE) {
      units = p.T * p.NB;
      // A choice that is no expert adds nothing.
      if (!((pairs.valids >> (u_first / p.NB * p.k + choice)) & 1u)) nk = 0;
    } else {
      units = __popc(pairs.leaders) * p.NB;
      if (blockIdx.x == 0 && warp == 0 && p.err_flag != nullptr && !pairs.valid && pairs.id != -1)
        atomicOr(p.err_flag, MXQ_DEVERR_EXPERT);
    }
  } else {
    units = *p.n_tiles * p.NB;
  }
  // The grid covers the most units that there can be; a CTA (the whole cluster
  // alike) without any leaves.
  if (u_first >= units) {
    if (warp == 1) ptx::tmem_dealloc(tmem, C::TMEM_COLS);
    return;
  }
  const int u_step = SPLIT ? units : (int)gridDim.x;  // split: one unit

  auto tile_of = [&](int u) {
    Tile t;
    if constexpr (MODE == kLinear) {
      t.expert = 0;
      t.pairs = 0u;
      t.row0 = (u / p.NB) * p.per_tile;
      t.count = min(p.per_tile, p.T - t.row0);
    } else if constexpr (BY_CHOICE) {
      const int pair = u / p.NB * p.k + choice;
      t.expert = __shfl_sync(0xffffffffu, pairs.id, pair);
      t.row0 = __shfl_sync(0xffffffffu, pairs.place(lane), pair);
      t.count = 1;
    } else if constexpr (SMALL != 0) {
      t = pairs.tile(u / p.NB);
    } else {
      const int4 v = *reinterpret_cast<const int4*>(p.tiles + u / p.NB);
      t.expert = __shfl_sync(0xffffffffu, v.x, 0);
      t.row0 = __shfl_sync(0xffffffffu, v.y, 0);
      t.count = __shfl_sync(0xffffffffu, v.z, 0);
      t.pairs = (uint32_t)__shfl_sync(0xffffffffu, v.w, 0);
    }
    return t;
  };
  if constexpr (SMALL != 0 && MODE == kGateUp) {
    // The first blocks on their way to L2 while barriers and TMEM are set up.
    if (warp == 3) {
      const Tile t = tile_of(u_first);
      const int mat = 2 * t.expert + (lane & 1), kk = lane >> 1;
      if (kk < nk && kk < NSTAGE)
        ptx::prefetch_l2_bulk(
            p.w + (((size_t)mat * p.NB + u_first % p.NB) * p.KB + kb0 + kk) * kBlockBytes, kBlockBytes);
    }
  }
  // The pair (token * k + choice) of row i of a tile.
  auto pair_of = [&](const Tile& t, int i) {
    if constexpr (SMALL != 0) return Pairs::row(t, i);
    else return (int)p.perm[t.row0 + i];
  };

  if constexpr (SPLIT) ptx::cluster_arrive();  // this CTA's shared memory may be written

  // A wait of a whole warp; false once it or another role has given up.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu,
                   !*abort_flag && ptx::mbar_wait_hint(bar, parity, p.wait_ns, kHintNs)))
      return true;
    if (lane == 0 && !*abort_flag) atomicOr(p.wd, kWdW4);
    *abort_flag = 1;
    return false;
  };

  if (warp == 0) {
    // ------------------------------------------------------------- copies
    // Weights that no other tile reads make way in L2 for what is read again: the rows,
    // the activation between the products, the results (64 tokens over 128 experts 3 %
    // less, 1024 over 64 5 %; with every expert's weights marked so, 4096 tokens, two tiles
    // each, take 2 % more).
    constexpr bool PLANNED = MODE != kLinear && SMALL == 0;
    const uint64_t once = ptx::policy_evict_first();
    int it = 0;
    bool ok = true;
    for (int u = u_first; u < units && ok; u += u_step) {
      const Tile t = tile_of(u);
      const uint32_t bytes = NA * kBlockBytes + (C::GATHER ? 0u : (uint32_t)C::TOK_TILE);
      const int rb = u % p.NB;
      const uint64_t keep = PLANNED && t.pairs ? once : ptx::policy_evict_normal();
      int row[NA];  // of a matrix's first block, in rows of 64 bytes
#pragma unroll
      for (int a = 0; a < NA; ++a)
        row[a] = (((MODE == kGateUp ? 2 * t.expert + a : t.expert) * p.NB + rb) * p.KB + kb0) *
                 (kBlockBytes / 64);
      for (int kk = 0; kk < nk; ++kk, ++it) {
        const int s = it % NSTAGE;
        ok = wait(&empty[s], ((uint32_t)(it / NSTAGE) & 1u) ^ 1u);
        if (!ok) break;
        if (ptx::elect_one()) {
          ptx::mbar_arrive_expect_tx(&full[s], bytes);
#pragma unroll
          for (int a = 0; a < NA; ++a) {
            if constexpr (PLANNED)
              ptx::tma_load_2d_hint(smem + C::OFF_W + (s * NA + a) * kTileBytes, &tm_w, &full[s], 0,
                                    row[a], keep);
            else
              ptx::tma_load_2d(smem + C::OFF_W + (s * NA + a) * kTileBytes, &tm_w, &full[s], 0, row[a]);
            ptx::bulk_load(smem + C::OFF_WSF + (s * NA + a) * kSfAtomBytes,
                           p.w + (size_t)(uint32_t)row[a] * 64 + kCodeBytes, kSfAtomBytes, &full[s]);
            row[a] += kBlockBytes / 64;
          }
          if constexpr (!C::GATHER)
            ptx::tma_load_2d(smem + C::OFF_TOK + s * C::TOK_TILE, &tm_a, &full[s], (kb0 + kk) * 128,
                             t.row0);
        }
        __syncwarp();
      }
    }
    if constexpr (SMALL != 0 && MODE == kGateUp) {
      // What is left to read is the experts' w2: each of an expert's CTAs brings
      // its share into L2.
      for (int u = u_first; u < units; u += u_step) {
        const int64_t blocks = (int64_t)p.NB2 * p.KB2;
        const int parts = p.NB * p.splits, part = (u % p.NB) * p.splits + split;
        const int64_t b0 = blocks * part / parts, b1 = blocks * (part + 1) / parts;
        const uint8_t* w2 = p.w2 + (size_t)tile_of(u).expert * blocks * kBlockBytes;
        for (int64_t b = b0 + lane; b < b1; b += 32)
          ptx::prefetch_l2_bulk(w2 + b * kBlockBytes, kBlockBytes);
      }
    }
    if (lane == 0) issued[0] = it;
  } else if (warp == 2) {
    // ------------------------------------- token scales (and gathered rows)
    // Lane i serves the rows i, i + 32, ...: the byte of a stage is fetched one
    // stage ahead, and the rows of a unit one unit ahead.
    constexpr int ROWS = (NT + 31) / 32;
    struct Rows {
      const uint8_t* src[ROWS];
      uint32_t byte[ROWS];  // of the first stage
      int g4[4];
      int count;
    };
    auto rows_of = [&](int u, Rows& r) {
      const Tile t = tile_of(u);
      r.count = t.count;
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        // Rows past the last stand for it: their columns are not stored.
        const int i = min(32 * j + lane, t.count - 1);
        r.src[j] = p.a_sf +
                   (size_t)(MODE == kGateUp ? pair_of(t, i) / p.k : t.row0 + i) * p.KG + kb0;
      }
      if constexpr (C::GATHER) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          r.g4[i] = pair_of(t, min(4 * lane + i, t.count - 1)) / p.k;
      }
#pragma unroll
      for (int j = 0; j < ROWS; ++j) r.byte[j] = nk > 0 ? r.src[j][0] : 127u;
    };
    Rows now, then;
    rows_of(u_first, now);
    int it = 0;
    bool ok = true;
    for (int u = u_first; u < units && ok; u += u_step) {
      if (u + u_step < units) rows_of(u + u_step, then);
      const int gathers = (now.count + 3) / 4;
      for (int kk = 0; kk < nk; ++kk, ++it) {
        const int s = it % NSTAGE;
        ok = wait(&empty[s], ((uint32_t)(it / NSTAGE) & 1u) ^ 1u);
        if (!ok) break;
        if constexpr (C::GATHER) {
          if (lane == 0) ptx::mbar_expect_tx(&full[s], (uint32_t)gathers * 512u);
          __syncwarp();
          if (lane < gathers)
            ptx::tma_gather4(smem + C::OFF_TOK + s * C::TOK_TILE + lane * 512, &tm_a, &full[s],
                             (kb0 + kk) * 128, now.g4[0], now.g4[1], now.g4[2], now.g4[3]);
        }
        // Row r of an atom owns word r / 32 of line r % 32; a group's
        // byte stands for its four blocks of 32.
        uint8_t* atom = smem + C::OFF_TSF + s * kSfAtomBytes;
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
          const uint32_t w = now.byte[j] * 0x01010101u;
          if (kk + 1 < nk) now.byte[j] = now.src[j][kk + 1];
          *reinterpret_cast<uint32_t*>(atom + lane * 16 + j * 4) = w;
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&full[s]);
      }
      now = then;
    }
    if (lane == 0) issued[1] = it;
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    int it = 0, n = 0;
    bool ok = true;
    for (int u = u_first; u < units && ok; u += u_step, ++n) {
      const int buf = C::NBUF == 2 ? n & 1 : 0;
      const uint32_t idesc = C::IDESC | ((uint32_t)((tile_of(u).count + 15) / 16 * 2) << 17);
      const uint32_t d = tmem + buf * NA * NT;
      ok = wait(&acc_empty[buf], ((uint32_t)(n / C::NBUF) & 1u) ^ 1u);
      if (!ok) break;
      ptx::tc_fence_after();
      for (int kk = 0; kk < nk; ++kk, ++it) {
        const int s = it % NSTAGE;
        ok = wait(&full[s], (uint32_t)(it / NSTAGE) & 1u);
        if (!ok) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint32_t sf = tmem + C::NBUF * NA * NT + (it % C::SF_RING) * C::SF_COLS;
          const uint32_t tok_sf = sf + 4 * NA;
          const uint64_t bdesc = ptx::smem_desc(
              ptx::smem_u32(smem + C::OFF_TOK + s * C::TOK_TILE), 16, 1024, ptx::kSwizzle128B);
#pragma unroll
          for (int a = 0; a < NA; ++a)
            ptx::tmem_cp_32x128b_x4(
                sf + 4 * a,
                ptx::smem_desc(ptx::smem_u32(smem + C::OFF_WSF + (s * NA + a) * kSfAtomBytes), 128,
                               128, ptx::kSwizzleNone));
          ptx::tmem_cp_32x128b_x4(
              tok_sf, ptx::smem_desc(ptx::smem_u32(smem + C::OFF_TSF + s * kSfAtomBytes), 128, 128,
                                     ptx::kSwizzleNone));
#pragma unroll
          for (int a = 0; a < NA; ++a) {
            const uint64_t adesc =
                ptx::smem_desc(ptx::smem_u32(smem + C::OFF_W + (s * NA + a) * kTileBytes), 16, 1024,
                               ptx::kSwizzle128B);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ptx::mma_mxf8(d + a * NT, adesc + 2 * k, bdesc + 2 * k,
                            idesc | ((uint32_t)k << 29) | ((uint32_t)k << 4), sf + 4 * a, tok_sf,
                            (kk > 0 || k > 0) ? 1u : 0u);
          }
          ptx::tc_commit(&empty[s]);
        }
        __syncwarp();
      }
      if (ptx::elect_one()) ptx::tc_commit(&acc_full[buf]);
      __syncwarp();
    }
    if (ptx::elect_one()) ptx::tc_commit(done);
  }
  __syncwarp();

  // ------------------------------------------------------------- epilogue
  float* sums = reinterpret_cast<float*>(smem + C::OFF_SUM);
  const int q = warp & 3, group = warp >= 4 ? (warp - 4) >> 2 : 0;
  float* max_ = reinterpret_cast<float*>(smem + C::OFF_MAX) + group * 2 * 4 * kChunk;
  if constexpr (!SPLIT) {
    if (warp >= 4) {
      int n = 0, chunk_no = 0;
      for (int u = u_first; u < units; u += u_step, ++n) {
        const int buf = C::NBUF == 2 ? n & 1 : 0;
        const Tile t = tile_of(u);
        const int rb = u % p.NB;
        const int chunks = (t.count + kChunk - 1) / kChunk;
        const bool ok = wait(&acc_full[buf], (uint32_t)(n / C::NBUF) & 1u);
        if (!ptx::named_sync_and(1 + group, 128, ok)) break;  // the group goes on, or leaves, together
        ptx::tc_fence_after();
        const uint32_t t0 = tmem + ((uint32_t)(q * 32) << 16) + buf * NA * NT;
        for (int c = group; c < chunks; c += C::GROUPS, ++chunk_no) {
          uint32_t r[NA][kChunk];
#pragma unroll
          for (int a = 0; a < NA; ++a) ptx::tmem_ld_32x32b_x16(t0 + a * NT + c * kChunk, r[a]);
          ptx::tmem_ld_wait();
          if (c + C::GROUPS >= chunks) {  // this group's last: the accumulator is free
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&acc_empty[buf]);
          }
          float v[NA][kChunk];
#pragma unroll
          for (int a = 0; a < NA; ++a)
#pragma unroll
            for (int i = 0; i < kChunk; ++i) v[a][i] = __uint_as_float(r[a][i]);
          finish_chunk<MODE, NA>(p, v, t.row0 + c * kChunk, t.count - c * kChunk, rb, q, lane,
                                 max_ + (chunk_no & 1) * 4 * kChunk, 1 + group);
        }
        if (group >= chunks) {  // no chunk for this group
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&acc_empty[buf]);
        }
      }
    }
    __syncthreads();
  } else {
    // One unit.  The four epilogue warps push each token's partial sums to the
    // CTA that owns the token.
    const Tile t = tile_of(u_first);
    const int rb = u_first % p.NB;
    const int own_log = BY_CHOICE ? 0 : __ffs(NT / p.splits) - 1;
    const int own = 1 << own_log;  // tokens of each CTA
    const float weight = BY_CHOICE && nk > 0 ? p.wt[u_first / p.NB * p.k + choice] : 1.0f;
    const int first = split * own;
    if (warp >= 4) {
      wait(&acc_full[0], 0);
      __syncwarp();
      ptx::tc_fence_after();
    }
    ptx::cluster_wait();  // every CTA of the cluster has begun
    if (warp >= 4) {
      const uint32_t t0 = tmem + ((uint32_t)(q * 32) << 16);
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          uint32_t v[16];
          ptx::tmem_ld_32x32b_x16(t0 + a * NT + c, v);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (c + i < t.count) {
              const int o = (c + i) >> own_log, tl = (c + i) & (own - 1);
              const uint32_t at =
                  ptx::smem_u32(sums + ((split * own + tl) * NA + a) * 128 + q * 32 + lane);
              ptx::st_shared_cluster_f32(ptx::map_shared_rank(at, (uint32_t)o),
                                         nk > 0 ? __uint_as_float(v[i]) * weight : 0.0f);
            }
          }
        }
      ptx::tc_fence_before();
    }
    __syncwarp();
    ptx::cluster_sync();  // all partial sums have arrived; nobody writes here again
    const int mine = min(own, t.count - first);
    if (!*abort_flag) {
      const int sub = lane & 15;
      for (int i = 2 * warp; i < mine; i += 2 * (C::THREADS / 32)) {
        const int tl = i + (lane >> 4);
        const bool in = tl < mine;
        float v[NA][8];
#pragma unroll
        for (int a = 0; a < NA; ++a) {
          const float* at = sums + ((in ? tl : i) * NA + a) * 128 + 8 * sub;
          *reinterpret_cast<float4*>(&v[a][0]) = *reinterpret_cast<const float4*>(at);
          *reinterpret_cast<float4*>(&v[a][4]) = *reinterpret_cast<const float4*>(at + 4);
          for (int r = 1; r < p.splits; ++r) {
            const float* ar = at + r * own * NA * 128;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[a][e] += ar[e];
          }
        }
        finish_token<BY_CHOICE ? kLinear : MODE, NA>(
            p, v, BY_CHOICE ? u_first / p.NB : t.row0 + first + tl, rb, sub, in);
      }
    }
  }
  if (*abort_flag) {
    // MMAs and copies in flight end before TMEM and shared memory are given up:
    // raise each issued stage's missing arrivals, then wait for its phase.
    if (threadIdx.x == 32) {
      ptx::mbar_wait(done, 0, kDrainNs);
      const int i0 = issued[0], i2 = issued[1], last = max(i0, i2);
      for (int i = min(i0, i2); i < last; ++i) ptx::mbar_arrive(&full[i % NSTAGE]);
      for (int i = max(0, last - NSTAGE); i < last; ++i)
        ptx::mbar_wait(&full[i % NSTAGE], (uint32_t)(i / NSTAGE) & 1u, kDrainNs);
    }
    __syncthreads();
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// The form for tiles of more than 128 tokens (routed: more than 64): CTA pairs.  One MMA
// (cta_group::2) takes
// 256 weight rows, 128 of each CTA (two row blocks side by side), against the
// tile's tokens, of which each CTA holds half.  Shared memory is what bounds the
// streaming form (128 bytes a cycle: a stage of 240 tokens writes 46 KB and the
// MMAs read 46 KB, 720 cycles where the products take 480; measured 712), and a
// pair writes and reads each token once for both CTAs (30 + 31 KB): 8192 x 4096 x
// 4096 99 us in the streaming form, 79 here; 4096 tokens over 64 experts 6 % less.
// Roles and epilogue are those of the streaming form, with these differences: the even
// CTA issues the MMAs and scale copies for both; the odd CTA's copies and scale
// words count on the even CTA's barriers; stages and accumulators are handed
// back to, and released by, both.  With an odd number of row blocks the last
// pair's odd CTA repeats the last block and stores nothing.  Three epilogue groups: with
// two or four a call of 4096 tokens takes 2 % longer, with five 3 % (fewer registers each);
// fetching a chunk ahead of its arithmetic: no faster.
template <int MODE>
struct PairCfg {
  static constexpr int NA = MODE == kGateUp ? 2 : 1;
  static constexpr int NT = kMaxTokens;
  static constexpr int GROUPS = 3, THREADS = 128 + 128 * GROUPS;
  static constexpr int TOK_ATOMS = 2;
  static constexpr int BOX_ROWS = 40;  // rows of a copy of tokens
  static constexpr int TOK_TILE = NT / 2 * 128;
  static_assert((NT / 2) % BOX_ROWS == 0 && BOX_ROWS % 8 == 0, "token copies");
  static constexpr int STAGE = NA * (kTileBytes + kSfAtomBytes) + TOK_TILE + TOK_ATOMS * kSfAtomBytes;
  static constexpr int MAX_BYTES = MODE == kGateUp ? GROUPS * 2 * 4 * kChunk * 4 : 0;
  static constexpr int NSTAGE = (232448 - 1024 - 512 - MAX_BYTES) / STAGE;
  static constexpr int OFF_W = 0;
  static constexpr int OFF_TOK = NSTAGE * NA * kTileBytes;
  static constexpr int OFF_WSF = OFF_TOK + NSTAGE * TOK_TILE;
  static constexpr int OFF_TSF = OFF_WSF + NSTAGE * NA * kSfAtomBytes;
  static constexpr int OFF_MAX = OFF_TSF + NSTAGE * TOK_ATOMS * kSfAtomBytes;
  static constexpr int OFF_BAR = OFF_MAX + MAX_BYTES;
  static constexpr int SMEM = OFF_BAR + (2 * NSTAGE + 5) * 8 + 32 + 1024;
  static constexpr int SF_COLS = 4 * NA + 4 * TOK_ATOMS;
  static constexpr int NBUF = 2 * NA * NT + 2 * SF_COLS <= 512 ? 2 : 1;
  static constexpr int SF_RING = 2;
  static constexpr uint32_t IDESC = (5u << 7) | (1u << 23) | ((256u >> 4) << 24);
  static_assert(NBUF * NA * NT + SF_RING * SF_COLS <= 512 && SMEM <= 232448 && TOK_TILE % 1024 == 0,
                "budgets");
  static_assert(tmem_allowed(SMEM) >= 512, "TMEM beside other kernels' CTAs");
};

template <int MODE>
__global__ void __launch_bounds__(PairCfg<MODE>::THREADS, 1)
    w4_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_sf,
                   const __grid_constant__ CUtensorMap tm_a, const W4Args p) {
  using C = PairCfg<MODE>;
  constexpr int NA = C::NA, NSTAGE = C::NSTAGE, NT = C::NT;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // the even CTA's count
  uint64_t* empty = full + NSTAGE;
  uint64_t* acc_full = empty + NSTAGE;  // [2]
  uint64_t* acc_empty = acc_full + 2;   // [2], the even CTA's count
  uint64_t* done = acc_empty + 2;
  uint32_t* slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(slot + 1);
  volatile int* issued = reinterpret_cast<volatile int*>(slot + 2);  // [0] warp 0, [1] warp 2
  // What the other CTA leaves here at its end: whether it gave up, and its `issued`.
  volatile int* other = reinterpret_cast<volatile int*>(slot + 4);  // [3]

  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)ptx::cluster_rank();

  const int nk = p.KB, NBP = (p.NB + 1) / 2;
  const int u_first = (int)(blockIdx.x >> 1), u_step = (int)(gridDim.x >> 1);
  auto block_of = [&](int u) { return 2 * (u % NBP) + rank; };  // may be NB: nothing of it is stored
  if (MODE == kLinear && warp == 3 && lane < NSTAGE && lane < nk)
    ptx::prefetch_l2_bulk(
        p.w + ((size_t)min(block_of(u_first), p.NB - 1) * p.KB + lane) * kBlockBytes, kBlockBytes);
  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&tm_w);
    ptx::prefetch_tmap(&tm_sf);
    ptx::prefetch_tmap(&tm_a);
    for (int i = 0; i < NSTAGE; ++i) {
      ptx::mbar_init(&full[i], 3);  // the expected bytes, and both CTAs' token scales
      ptx::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&acc_full[i], 1);
      ptx::mbar_init(&acc_empty[i], 2 * 4 * C::GROUPS);
    }
    ptx::mbar_init(done, 1);
    ptx::fence_barrier_init();
    *abort_flag = 0;
    issued[0] = issued[1] = 0;
    other[0] = other[1] = other[2] = 0;
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(slot, 512);
    ptx::tmem_relinquish_pair();
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::cluster_sync();  // both CTAs' barriers are set up
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);
  ptx::griddep_launch_dependents();  // (TMEM in hand, as above)
  ptx::griddep_wait();
  const int units = (MODE == kLinear ? p.n_tiles_host : *p.n_tiles) * NBP;
  if (u_first >= units) {  // both CTAs alike
    if (warp == 1) ptx::tmem_dealloc_pair(tmem, 512);
    return;
  }

  auto tile_of = [&](int u) {
    Tile t;
    if constexpr (MODE == kLinear) {
      t.expert = 0;
      t.pairs = 0u;
      t.row0 = (u / NBP) * p.per_tile;
      t.count = min(p.per_tile, p.T - t.row0);
    } else {
      const int4 v = *reinterpret_cast<const int4*>(p.tiles + u / NBP);
      t.expert = __shfl_sync(0xffffffffu, v.x, 0);
      t.row0 = __shfl_sync(0xffffffffu, v.y, 0);
      t.count = __shfl_sync(0xffffffffu, v.z, 0);
      t.pairs = (uint32_t)__shfl_sync(0xffffffffu, v.w, 0);
    }
    return t;
  };

  const uint32_t even_full = ptx::map_shared_rank(ptx::smem_u32(full), 0);
  const uint32_t even_acc = ptx::map_shared_rank(ptx::smem_u32(acc_empty), 0);

  // Bytes of one CTA's copies of a stage of a tile.
  auto boxes_of = [&](const Tile& t) { return ((t.count + 15) / 16 * 8 + C::BOX_ROWS - 1) / C::BOX_ROWS; };
  auto bytes_of = [&](const Tile& t) { return (uint32_t)(NA * kBlockBytes + boxes_of(t) * C::BOX_ROWS * 128); };

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu,
                   !*abort_flag && ptx::mbar_wait_hint(bar, parity, p.wait_ns, kHintNs)))
      return true;
    if (lane == 0 && !*abort_flag) atomicOr(p.wd, kWdW4);
    *abort_flag = 1;
    return false;
  };

  if (warp == 0) {
    // ------------------------------------------------------------- copies
    const uint64_t once = ptx::policy_evict_first();  // (as above)
    int it = 0;
    bool ok = true;
    for (int u = u_first; u < units && ok; u += u_step) {
      const Tile t = tile_of(u);
      const int half = (t.count + 15) / 16 * 8;  // tokens held by each CTA
      const int boxes = boxes_of(t);
      const uint32_t bytes = 2u * bytes_of(t);
      const int rb = min(block_of(u), p.NB - 1);
      const uint64_t keep = MODE != kLinear && t.pairs ? once : ptx::policy_evict_normal();
      int blk[NA];
#pragma unroll
      for (int a = 0; a < NA; ++a)
        blk[a] = ((MODE == kGateUp ? 2 * t.expert + a : t.expert) * p.NB + rb) * p.KB;
      for (int kk = 0; kk < nk; ++kk, ++it) {
        const int s = it % NSTAGE;
        ok = wait(&empty[s], ((uint32_t)(it / NSTAGE) & 1u) ^ 1u);
        if (!ok) break;
        if (ptx::elect_one()) {
          const uint32_t bar = even_full + 8u * (uint32_t)s;
          if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], bytes);
#pragma unroll
          for (int a = 0; a < NA; ++a) {
            ptx::tma_load_2d_pair_hint(smem + C::OFF_W + (s * NA + a) * kTileBytes, &tm_w, bar, 0,
                                       blk[a] * (kBlockBytes / 64), keep);
            ptx::tma_load_2d_pair(smem + C::OFF_WSF + (s * NA + a) * kSfAtomBytes, &tm_sf, bar, 0,
                                  blk[a] * (kBlockBytes / 256) + kCodeBytes / 256);
            ++blk[a];
          }
#pragma unroll
          for (int b = 0; b < NT / 2 / C::BOX_ROWS; ++b)
            if (b < boxes)
              ptx::tma_load_2d_pair(smem + C::OFF_TOK + s * C::TOK_TILE + b * C::BOX_ROWS * 128, &tm_a,
                                    bar, kk * 128, t.row0 + rank * half + b * C::BOX_ROWS);
        }
        __syncwarp();
      }
    }
    if (lane == 0) issued[0] = it;
  } else if (warp == 2) {
    // ------------------------------------------------------- token scales
    constexpr int ROWS = (NT + 31) / 32;
    struct Rows {
      const uint8_t* src[ROWS];
      uint32_t byte[ROWS];
    };
    auto rows_of = [&](int u, Rows& r) {
      const Tile t = tile_of(u);
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const int i = t.row0 + min(32 * j + lane, t.count - 1);
        r.src[j] = p.a_sf + (size_t)(MODE == kGateUp ? p.perm[i] / p.k : i) * p.KG;
      }
#pragma unroll
      for (int j = 0; j < ROWS; ++j) r.byte[j] = r.src[j][0];
    };
    Rows now, then;
    rows_of(u_first, now);
    int it = 0;
    bool ok = true;
    for (int u = u_first; u < units && ok; u += u_step) {
      if (u + u_step < units) rows_of(u + u_step, then);
      for (int kk = 0; kk < nk; ++kk, ++it) {
        const int s = it % NSTAGE;
        ok = wait(&empty[s], ((uint32_t)(it / NSTAGE) & 1u) ^ 1u);
        if (!ok) break;
        uint8_t* atom = smem + C::OFF_TSF + s * C::TOK_ATOMS * kSfAtomBytes;
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
          const uint32_t w = now.byte[j] * 0x01010101u;
          if (kk + 1 < nk) now.byte[j] = now.src[j][kk + 1];
          *reinterpret_cast<uint32_t*>(atom + (j >> 2) * kSfAtomBytes + lane * 16 + (j & 3) * 4) = w;
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote(even_full + 8u * (uint32_t)s);
      }
      now = then;
    }
    if (lane == 0) issued[1] = it;
  } else if (warp == 1 && rank == 0) {
    // ----------------------------------------------------------------- MMA
    int it = 0, n = 0;
    bool ok = true;
    for (int u = u_first; u < units && ok; u += u_step, ++n) {
      const int buf = C::NBUF == 2 ? n & 1 : 0;
      const uint32_t idesc = C::IDESC | ((uint32_t)((tile_of(u).count + 15) / 16 * 2) << 17);
      const uint32_t d = tmem + buf * NA * NT;
      ok = wait(&acc_empty[buf], ((uint32_t)(n / C::NBUF) & 1u) ^ 1u);
      if (!ok) break;
      ptx::tc_fence_after();
      for (int kk = 0; kk < nk; ++kk, ++it) {
        const int s = it % NSTAGE;
        ok = wait(&full[s], (uint32_t)(it / NSTAGE) & 1u);
        if (!ok) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint32_t sf = tmem + C::NBUF * NA * NT + (it % C::SF_RING) * C::SF_COLS;
          const uint32_t tok_sf = sf + 4 * NA;
          const uint64_t bdesc = ptx::smem_desc(
              ptx::smem_u32(smem + C::OFF_TOK + s * C::TOK_TILE), 16, 1024, ptx::kSwizzle128B);
#pragma unroll
          for (int a = 0; a < NA; ++a)
            ptx::tmem_cp_32x128b_x4_pair(
                sf + 4 * a,
                ptx::smem_desc(ptx::smem_u32(smem + C::OFF_WSF + (s * NA + a) * kSfAtomBytes), 128,
                               128, ptx::kSwizzleNone));
#pragma unroll
          for (int a = 0; a < C::TOK_ATOMS; ++a)
            ptx::tmem_cp_32x128b_x4_pair(
                tok_sf + 4 * a,
                ptx::smem_desc(
                    ptx::smem_u32(smem + C::OFF_TSF + (s * C::TOK_ATOMS + a) * kSfAtomBytes), 128,
                    128, ptx::kSwizzleNone));
#pragma unroll
          for (int a = 0; a < NA; ++a) {
            const uint64_t adesc =
                ptx::smem_desc(ptx::smem_u32(smem + C::OFF_W + (s * NA + a) * kTileBytes), 16, 1024,
                               ptx::kSwizzle128B);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              ptx::mma_mxf8_pair(d + a * NT, adesc + 2 * k, bdesc + 2 * k,
                                 idesc | ((uint32_t)k << 29) | ((uint32_t)k << 4), sf + 4 * a, tok_sf,
                                 (kk > 0 || k > 0) ? 1u : 0u);
          }
          ptx::tc_commit_pair_mc(&empty[s], 3);  // frees the stage in both CTAs
        }
        __syncwarp();
      }
      if (ptx::elect_one()) ptx::tc_commit_pair_mc(&acc_full[buf], 3);
      __syncwarp();
    }
    if (ptx::elect_one()) ptx::tc_commit_pair_mc(done, 1);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, group = (warp - 4) >> 2;
    float* max_ = reinterpret_cast<float*>(smem + C::OFF_MAX) + group * 2 * 4 * kChunk;
    int n = 0, chunk_no = 0;
    for (int u = u_first; u < units; u += u_step, ++n) {
      const int buf = C::NBUF == 2 ? n & 1 : 0;
      const Tile t = tile_of(u);
      const int rb = block_of(u);
      const int chunks = (t.count + kChunk - 1) / kChunk;
      const bool ok = wait(&acc_full[buf], (uint32_t)(n / C::NBUF) & 1u);
      if (!ptx::named_sync_and(1 + group, 128, ok)) break;
      ptx::tc_fence_after();
      const uint32_t t0 = tmem + ((uint32_t)(q * 32) << 16) + buf * NA * NT;
      for (int c = group; c < chunks; c += C::GROUPS, ++chunk_no) {
        uint32_t r[NA][kChunk];
#pragma unroll
        for (int a = 0; a < NA; ++a) ptx::tmem_ld_32x32b_x16(t0 + a * NT + c * kChunk, r[a]);
        ptx::tmem_ld_wait();
        if (c + C::GROUPS >= chunks) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_remote(even_acc + 8u * (uint32_t)buf);
        }
        float v[NA][kChunk];
#pragma unroll
        for (int a = 0; a < NA; ++a)
#pragma unroll
          for (int i = 0; i < kChunk; ++i) v[a][i] = __uint_as_float(r[a][i]);
        finish_chunk<MODE, NA>(p, v, t.row0 + c * kChunk, t.count - c * kChunk, rb, q, lane,
                               max_ + (chunk_no & 1) * 4 * kChunk, 1 + group);
      }
      if (group >= chunks) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote(even_acc + 8u * (uint32_t)buf);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const int left[3] = {*abort_flag, issued[0], issued[1]};
    for (int i = 0; i < 3; ++i)
      ptx::st_shared_cluster_u32(
          ptx::map_shared_rank(ptx::smem_u32(const_cast<int*>(other + i)), (uint32_t)(rank ^ 1)),
          (uint32_t)left[i]);
  }
  ptx::cluster_sync();  // neither CTA leaves while the other may still use it
  if (*abort_flag || other[0]) {  // (both CTAs alike)
    // MMAs and copies in flight, all of which the even CTA's barriers count, end before TMEM
    // and shared memory are given up: raise each issued stage's missing arrivals and
    // bytes, then wait for its phase.
    if (rank == 0 && warp == 0) {
      const int i0 = issued[0], i2 = issued[1], o0 = other[1], o2 = other[2];
      const int last = max(max(i0, i2), max(o0, o2));
      ptx::mbar_wait(done, 0, kDrainNs);
      for (int i = min(min(i0, i2), min(o0, o2)); i < last; ++i) {
        const uint32_t bytes = bytes_of(tile_of(u_first + i / nk * u_step));
        uint64_t* bar = &full[i % NSTAGE];
        if (lane == 0) {
          if (i >= i0 && i < o0) ptx::mbar_arrive_expect_tx(bar, bytes);
          if (i >= i0 && i >= o0) ptx::mbar_arrive(bar);
          if (i < i0 && i >= o0) ptx::mbar_complete_tx(bar, bytes);
          if (i >= i2) ptx::mbar_arrive(bar);
          if (i >= o2) ptx::mbar_arrive(bar);
        }
        __syncwarp();
      }
      for (int i = max(0, last - NSTAGE); i < last; ++i)
        ptx::mbar_wait(&full[i % NSTAGE], (uint32_t)(i / NSTAGE) & 1u, kDrainNs);
    }
    ptx::cluster_sync();
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------ plan and join
// One cluster counts the rows of each expert, lays out the tiles and sorts the rows
// by expert: perm gives a sorted row's token and choice, pos the other way round
// (-1: no expert).  The order of an expert's rows does not matter: each is summed by
// itself, and lands at its own place.
constexpr int kPlanThreads = 1024;
constexpr int kPlanBatch = 8;
constexpr int kSizes = kMaxTokens / 16 + 1;  // tiles of 16 i tokens and less

__global__ void __launch_bounds__(kPlanThreads) w4_plan_kernel(const int32_t* ids, int R, int E,
                                                               int nt, int ctas, Tile* tiles,
                                                               int32_t* n_tiles, int32_t* perm,
                                                               int32_t* pos, int32_t* err_flag) {
  __shared__ int cnt[kMaxExperts], cur[kMaxExperts];
  __shared__ int wsum[32], size_n[kSizes], size_at[kSizes];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  static_assert(kMaxExperts <= kPlanThreads, "one expert per thread");
  // CTA `rank` of the cluster takes the rows [first, end); shared-memory atomics
  // of one SM alone take 19 us for 24576 rows.
  const uint32_t rank = ptx::cluster_rank();
  const int share = (R + ctas - 1) / ctas, first = min(R, (int)rank * share), end = min(R, first + share);
  if (tid < kMaxExperts) cnt[tid] = 0;
  __syncthreads();
  bool bad = false;
  // (Eight loads at a time: with one after the other their latency is the time.)
  for (int i0 = first + tid; i0 < end; i0 += kPlanBatch * kPlanThreads) {
    int e[kPlanBatch];
#pragma unroll
    for (int j = 0; j < kPlanBatch; ++j)
      e[j] = i0 + j * kPlanThreads < end ? ids[i0 + j * kPlanThreads] : -1;
#pragma unroll
    for (int j = 0; j < kPlanBatch; ++j) {
      if (e[j] >= 0 && e[j] < E)
        atomicAdd(&cnt[e[j]], 1);
      else
        bad |= e[j] != -1;
    }
  }
  if (bad && err_flag != nullptr) atomicOr(err_flag, MXQ_DEVERR_EXPERT);
  ptx::cluster_sync();
  // All CTAs' rows of expert `tid`, and those of the CTAs before this one.
  int c = 0, earlier = 0;
  if (tid < E) {
    const uint32_t at = ptx::smem_u32(&cnt[tid]);
    for (int r = 0; r < ctas; ++r) {
      const int v = (int)ptx::ld_shared_cluster_u32(ptx::map_shared_rank(at, (uint32_t)r));
      c += v;
      earlier += r < (int)rank ? v : 0;
    }
  }
  // Even tiles of at most nt rows, each a multiple of 16 but for the last.
  const int even = (c + nt - 1) / nt;
  const int rows = c > 0 ? ((c + even - 1) / even + 15) / 16 * 16 : 16;
  const int nt_e = (c + rows - 1) / rows;
  int sc = c;  // inclusive sums over the warp, then over warps
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, sc, m);
    if (lane >= m) sc += a;
  }
  if (lane == 31) wsum[warp] = sc;
  // The largest tiles come first: CTAs take units in order, so the last round,
  // which is seldom full, is one of small ones.  An expert's tiles stay together, so
  // that its weights come from HBM once (the last tile may be smaller than the others).
  const int full16 = rows / 16;
  if (tid < kSizes) size_n[tid] = 0;
  __syncthreads();
  if (nt_e > 0) atomicAdd(&size_n[full16], nt_e);
  __syncthreads();
  int pc = 0;
  for (int w = 0; w < warp; ++w) pc += wsum[w];
  if (tid < kSizes) {
    int before = 0;
    for (int i = tid + 1; i < kSizes; ++i) before += size_n[i];
    size_at[tid] = before;
  }
  const int row0 = pc + sc - c;
  if (tid < E) cur[tid] = row0 + earlier;
  __syncthreads();
  if (rank == 0) {
    if (tid == 0) *n_tiles = size_at[0] + size_n[0];
    Tile t;
    t.expert = tid;
    t.pairs = nt_e == 1 ? 1u : 0u;
    if (nt_e > 0) {
      const int at = atomicAdd(&size_at[full16], nt_e);
      for (int i = 0; i < nt_e; ++i) {
        t.row0 = row0 + i * rows;
        t.count = min(rows, c - i * rows);
        tiles[at + i] = t;
      }
    }
  }
  ptx::cluster_sync();  // (also: nobody reads this CTA's counts any more)
  for (int i0 = first + tid; i0 < end; i0 += kPlanBatch * kPlanThreads) {
    int e[kPlanBatch];
#pragma unroll
    for (int j = 0; j < kPlanBatch; ++j)
      e[j] = i0 + j * kPlanThreads < end ? ids[i0 + j * kPlanThreads] : -1;
#pragma unroll
    for (int j = 0; j < kPlanBatch; ++j) {
      const int i = i0 + j * kPlanThreads;
      if (i >= end) break;
      int at = -1;
      if (e[j] >= 0 && e[j] < E) {
        at = atomicAdd(&cur[e[j]], 1);
        perm[at] = i;
      }
      pos[i] = at;
    }
  }
}

// The activation rows laid out by expert, for the plain copies of large tiles: every
// 128 weight rows read a tile's tokens anew, and a copy by index moves four rows (in
// 44 ns) where a plain one moves a box of them: with tiles of 128 tokens by index a call of
// 4096 tokens over 64 experts took half as long again as with rows laid out, which takes
// 19 us of it.  A warp reads 2 KB of a token's row once and writes it to each of the row's
// places.
constexpr int kRowWarps = 8;
constexpr int kRowChunks = 128;  // of 16 bytes, of a warp

__global__ void __launch_bounds__(kRowWarps * 32) w4_rows_kernel(const uint4* a, const int32_t* pos,
                                                                 int64_t items, int parts, int k,
                                                                 int chunks, uint4* out) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t it = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (it >= items) return;
  const int64_t t = it / parts;
  const int c0 = (int)(it - t * parts) * kRowChunks + lane;
  uint4 v[kRowChunks / 32];
#pragma unroll
  for (int i = 0; i < kRowChunks / 32; ++i)
    if (c0 + 32 * i < chunks) v[i] = a[(size_t)t * chunks + c0 + 32 * i];
  const int mine = lane < k ? pos[t * k + lane] : -1;  // (k is 32 at most)
  for (int j = 0; j < k; ++j) {
    const int row = __shfl_sync(0xffffffffu, mine, j);
    if (row < 0) continue;
#pragma unroll
    for (int i = 0; i < kRowChunks / 32; ++i)
      if (c0 + 32 * i < chunks) out[(size_t)row * chunks + c0 + 32 * i] = v[i];
  }
}

// out[t] = weighted sum over the token's choices, in their order, of the FP32
// results that the down product left.  (Adding in the down product's last CTA of a token
// instead, found by a counter, was no faster.)
constexpr int kJoinWarps = 8;
constexpr int kJoinCols = 256;  // of a warp

// One warp: kJoinCols columns of a token, four and four to a lane.  The lanes fetch the
// token's rows and weights at once and pass them round, so that the results' loads wait
// for nothing else.
__global__ void __launch_bounds__(kJoinWarps * 32) w4_join_kernel(const float* part, const int32_t* pos,
                                                                  const float* wt, __nv_bfloat16* out,
                                                                  int64_t items, int segs, int N, int k) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t it = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (it >= items) return;
  const int64_t t = it / segs;
  const int c = (int)(it - t * segs) * kJoinCols + lane * 4;
  const int my_row = lane < k ? pos[t * k + lane] : -1;  // (k is 32 at most)
  const float my_weight = lane < k ? wt[t * k + lane] : 0.0f;
  const bool in[2] = {c < N, c + kJoinCols / 2 < N};
  float2 y[2][2] = {};
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int row = __shfl_sync(0xffffffffu, my_row, j);
    const float weight = __shfl_sync(0xffffffffu, my_weight, j);
    if (row < 0) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!in[h]) continue;
      // (Read once: 4096 tokens over 64 experts 350 us, 358 with loads that stay in L2.)
      const float4 v = __ldcs(reinterpret_cast<const float4*>(part + (size_t)row * N + c + h * (kJoinCols / 2)));
      y[h][0] = fma2(make_float2(v.x, v.y), make_float2(weight, weight), y[h][0]);
      y[h][1] = fma2(make_float2(v.z, v.w), make_float2(weight, weight), y[h][1]);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (in[h])
      *reinterpret_cast<uint2*>(out + (size_t)t * N + c + h * (kJoinCols / 2)) =
          make_uint2(pack2(y[h][0].x, y[h][0].y), pack2(y[h][1].x, y[h][1].y));
}

// Codes and scales of B matrices [N][K] into blocks; one thread per 16 bytes.
__global__ void __launch_bounds__(256) prepare_w4_kernel(const uint8_t* w, const uint8_t* sf,
                                                         uint4* out, int64_t items, int N, int K,
                                                         int NB, int KB) {
  const int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (it >= items) return;
  constexpr int kPer = kBlockBytes / 16;
  const int64_t blk = it / kPer;
  const int i = (int)(it - blk * kPer);
  const int kb = (int)(blk % KB);
  const int64_t r = blk / KB;
  const int nb = (int)(r % NB);
  const int64_t b = r / NB;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (i < kCodeBytes / 16) {
    const int n = nb * 128 + (i >> 2), at = kb * 64 + (i & 3) * 16;  // bytes of the row
    if (n < N && at < K / 2)
      v = *reinterpret_cast<const uint4*>(w + ((size_t)b * N + n) * (size_t)(K / 2) + at);
  } else {
    const int line = i - kCodeBytes / 16;
    uint32_t word[4];
    for (int j = 0; j < 4; ++j) {
      const int n = nb * 128 + 32 * j + line;
      word[j] = 0;
      for (int q = 0; q < 4; ++q) {
        const int g = kb * 4 + q;
        const uint32_t s = n < N && g < K / 32 ? sf[((size_t)b * N + n) * (size_t)(K / 32) + g] : 127u;
        word[j] |= s << (8 * q);
      }
    }
    v = make_uint4(word[0], word[1], word[2], word[3]);
  }
  out[it] = v;
}

// --------------------------------------------------------------- host side
bool encode_weight(CUtensorMap* m, const void* base, uint64_t blocks) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  // Rows of 128 codes (64 bytes); a block is 136 of them, the last eight its
  // scale atom.
  cuuint64_t dims[2] = {128, blocks * (kBlockBytes / 64)};
  cuuint64_t strides[1] = {64};
  cuuint32_t box[2] = {128, 128};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_rows(CUtensorMap* m, const void* base, uint64_t K, uint64_t rows, uint32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {K, rows};
  cuuint64_t strides[1] = {K};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int NT, bool SPLIT, int SMALL = 0>
cudaError_t launch_cfg(const void* a, uint64_t a_rows, uint64_t K, uint64_t blocks, W4Args args,
                       int64_t units, int num_sms, cudaStream_t s, const char** why) {
  using C = Cfg<MODE, NT, SPLIT, SMALL>;
  CUtensorMap tm_w, tm_a;
  if (!encode_weight(&tm_w, args.w, blocks) ||
      !encode_rows(&tm_a, a, K, a_rows, C::GATHER ? 1 : NT)) {
    *why = "cuTensorMapEncodeTiled failed (driver entry point missing or arguments rejected)";
    return cudaErrorInvalidValue;
  }
  auto kern = w4_kernel<MODE, NT, SPLIT, SMALL>;
  static std::atomic<uint64_t> smem_set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(smem_set.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    smem_set.fetch_or(bit, std::memory_order_acq_rel);
  }
  const int64_t slots = (int64_t)num_sms * C::CTAS;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(SPLIT ? units * args.splits : units < slots ? units : slots), 1, 1);
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (SPLIT) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)args.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kern, tm_w, tm_a, args);
}

// Scale atoms of the prepared weight, as two rows of 256 bytes each.
bool encode_atoms(CUtensorMap* m, const void* base, uint64_t blocks) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {256, blocks * (kBlockBytes / 256)};
  cuuint64_t strides[1] = {256};
  cuuint32_t box[2] = {256, kSfAtomBytes / 256};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
cudaError_t launch_pair(const void* a, uint64_t a_rows, uint64_t K, uint64_t blocks, const W4Args& args,
                        int64_t tiles, int num_sms, cudaStream_t s, const char** why) {
  using C = PairCfg<MODE>;
  CUtensorMap tm_w, tm_sf, tm_a;
  if (!encode_weight(&tm_w, args.w, blocks) || !encode_atoms(&tm_sf, args.w, blocks) ||
      !encode_rows(&tm_a, a, K, a_rows, C::BOX_ROWS)) {
    *why = "cuTensorMapEncodeTiled failed (driver entry point missing or arguments rejected)";
    return cudaErrorInvalidValue;
  }
  auto kern = w4_pair_kernel<MODE>;
  static std::atomic<uint64_t> smem_set{0};
  static std::atomic<int> pair_slots[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(smem_set.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    smem_set.fetch_or(bit, std::memory_order_acq_rel);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // One pair for each place that the device has for it.
  int slots = pair_slots[dev & 63].load(std::memory_order_acquire);
  if (slots == 0) {
    cfg.gridDim = dim3(2u * (unsigned)(num_sms / 2), 1, 1);
    e = cudaOccupancyMaxActiveClusters(&slots, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (slots <= 0) {
      *why = "no CTA pair fits on this device";
      return cudaErrorInvalidConfiguration;
    }
    pair_slots[dev & 63].store(slots, std::memory_order_release);
  }
  const int64_t units = tiles * ((args.NB + 1) / 2);
  cfg.gridDim = dim3(2u * (unsigned)(units < slots ? units : slots), 1, 1);
  return cudaLaunchKernelEx(&cfg, kern, tm_w, tm_sf, tm_a, args);
}

// The product for tiles of at most `nt` tokens (16, 32, 64, dense 128, 240), its K
// split where the caller chose so (16 and, dense, 32 tokens only).
template <int MODE>
cudaError_t launch_tokens(int nt, const void* a, uint64_t a_rows, uint64_t K, uint64_t blocks,
                          const W4Args& g, int64_t units, int num_sms, cudaStream_t s,
                          const char** why) {
  if constexpr (MODE != kLinear) {
    if (g.ids != nullptr) {
      if constexpr (MODE == kGateUp) {
        if (g.splits == 1)
          return launch_cfg<MODE, 16, false, 1>(a, a_rows, K, blocks, g, units, num_sms, s, why);
      } else if (units * g.splits > 2 * num_sms) {
        return launch_cfg<MODE, 16, true, 2>(a, a_rows, K, blocks, g, units, num_sms, s, why);
      }
      return launch_cfg<MODE, 16, true, 1>(a, a_rows, K, blocks, g, units, num_sms, s, why);
    }
  }
  if (nt <= 16)
    return g.splits > 1 ? launch_cfg<MODE, 16, true>(a, a_rows, K, blocks, g, units, num_sms, s, why)
                        : launch_cfg<MODE, 16, false>(a, a_rows, K, blocks, g, units, num_sms, s, why);
  if (nt <= 32) {
    if constexpr (MODE == kLinear) {
      if (g.splits > 1)
        return launch_cfg<MODE, 32, true>(a, a_rows, K, blocks, g, units, num_sms, s, why);
    }
    return launch_cfg<MODE, 32, false>(a, a_rows, K, blocks, g, units, num_sms, s, why);
  }
  if (nt <= 64) return launch_cfg<MODE, 64, false>(a, a_rows, K, blocks, g, units, num_sms, s, why);
  if constexpr (MODE == kLinear) {
    if (nt <= 128) return launch_cfg<MODE, 128, false>(a, a_rows, K, blocks, g, units, num_sms, s, why);
  }
  return launch_pair<MODE>(a, a_rows, K, blocks, g, units / g.NB, num_sms, s, why);
}

// CTAs that the device holds at once in clusters of c, with one or two to an SM: a
// cluster's SMs are neighbours, and some of their groups are short of a few (152 SMs
// hold 36 clusters of 4 and 15 of 8, and twice 37 and 18 with two CTAs to an SM).
int64_t held(int num_sms, int ctas, int c) {
  const int64_t all = (int64_t)num_sms * ctas;
  return c < 4 ? all : c > 4 && ctas == 1 ? all * 15 / 19 : all * 18 / 19;
}
// CTAs along K of each of a unit's `per` products of KB blocks: powers of two up to
// the portable cluster size that the device holds at once, two blocks each at least
// (1 x 4096 x 4096 5.6 us on 8, unsplit 11.7), and none where K has less than eight (32 x
// 4096 x 512 3.9 us, on two 4.6; 16 x 2048 x 1024 on four 4.2, on two 4.6, unsplit 4.7).
int pick_splits(int64_t units, int KB, int num_sms, int ctas, int per = 1) {
  int s = 1;
  while (2 * s * per <= kMaxCluster && units * 2 * s * per <= held(num_sms, ctas, 2 * s * per) &&
         KB >= 8 && KB >= 4 * s)
    s *= 2;
  return s;
}

}  // namespace

uint32_t set_w4_wait(uint32_t ns) {
  return g_wait_ns.exchange(ns == 0 || ns > kWaitNs ? kWaitNs : ns);
}

cudaError_t launch_prepare_w4(const uint8_t* w, const uint8_t* sf, int64_t B, int N, int K,
                              uint8_t* out, cudaStream_t s) {
  const int NB = (int)ceil_div(N, 128), KB = (int)ceil_div(K, kGroup);
  const int64_t items = B * NB * KB * (kBlockBytes / 16);
  prepare_w4_kernel<<<(unsigned)ceil_div(items, 256), 256, 0, s>>>(
      w, sf, reinterpret_cast<uint4*>(out), items, N, K, NB, KB);
  return cudaGetLastError();
}

cudaError_t launch_linear_a8w4(const uint8_t* a, const uint8_t* a_sf, const uint8_t* w, void* out,
                               int64_t T, int N, int K, int num_sms, cudaStream_t s,
                               const char** why) {
  W4Args g = {};
  g.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
  g.w = w;
  g.a_sf = a_sf;
  g.out = out;
  g.T = (int)T;
  g.N = N;
  g.KG = g.KB = (int)ceil_div(K, kGroup);
  g.NB = (int)ceil_div(N, 128);
  g.splits = 1;
  cudaError_t e = watchdog_address(&g.wd);
  if (e != cudaSuccess) return e;
  if (T <= 32) {
    g.splits = pick_splits(g.NB, g.KB, num_sms, 2);
    g.per_tile = T <= 16 ? 16 : 32;
  } else {
    // Tiles of even size.  A stage of n tokens costs about 256 + 2 n cycles of
    // shared memory (the weight tile's write and read, and the tokens'), or, above
    // 128 tokens, 256 + n in each CTA of a pair: the number of tiles is the one with
    // the least rounds x that.
    int64_t best = -1;
    const int64_t least = ceil_div(T, kMaxTokens);
    for (int64_t n = least; n <= least + 24; ++n) {
      const int64_t per = ceil_div(ceil_div(T, n), 16) * 16, tiles = ceil_div(T, per);
      const int64_t cost = per > 128 ? ceil_div(tiles * ((g.NB + 1) / 2), num_sms / 2) * (256 + per)
                                     : ceil_div(tiles * g.NB, num_sms) * (256 + 2 * per);
      if (best < 0 || cost < best) {
        best = cost;
        g.per_tile = (int)per;
      }
    }
  }
  g.kb_per_split = (int)ceil_div(g.KB, g.splits);
  g.n_tiles_host = (int)ceil_div(T, g.per_tile);
  return launch_tokens<kLinear>(g.per_tile, a, (uint64_t)T, (uint64_t)K, (uint64_t)g.NB * g.KB, g,
                                (int64_t)g.n_tiles_host * g.NB, num_sms, s, why);
}

namespace {
bool small_call(int64_t R, int k) { return R <= kSmallPairs && k <= kSmallChoices; }
// Most tokens of a tile, by the rows that an expert gets on average: above that
// some experts take two tiles, which read their weights twice (from L2).  128 experts,
// 8 choices, 4096 x 1024, us, with tiles of 16 / 32 / 64 / 128 / 240 (taken with results of
// 16 bits; FP32 ones add nothing at 4 rows, 2 us at 12 to 40 and 11 at 64, whatever the tile):
//   rows an expert on average
//    4    128 / 127 / 134 / 159 / 154      24   279 / 212 / 179 / 202 / 198
//    5    144 / 135 / 142 / 170 / 163      40   406 / 289 / 206 / 216 / 210
//   12    188 / 161 / 162 / 190 / 186      48   461 / 331 / 224 / 231 / 216
//   14    206 / 176 / 166 / 194 / 189      64   586 / 409 / 268 / 252 / 228
int expert_tile(int64_t R, int k, int E) {
  const int64_t avg = ceil_div(R, E);
  if (small_call(R, k)) return 16;
  return avg <= 3 ? 16 : avg <= 12 ? 32 : avg <= 40 ? 64 : kMaxTokens;
}
// An expert of c rows has ceil(c / nt) tiles at most (fewer where even tiles
// round up to 16), that is c / nt and one more if it has any.
int64_t most_tiles(int64_t R, int E, int nt) { return R / nt + (R < E ? R : E); }
// Whether the rows are laid out by expert first (see w4_rows_kernel); up to 32 tokens
// it made no difference, and the launch and the workspace are saved.
bool lays_out_rows(int nt) { return nt > 32; }
}  // namespace

ExpertsLayout experts_layout(int64_t T, int k, int E, int K, int I, int N) {
  const int64_t R = T * k;
  const int nt = expert_tile(R, k, E);
  ExpertsLayout l;
  l.tiles = 256;  // their number lies before them
  l.perm = l.tiles + round_up_256((size_t)most_tiles(R, E, nt) * sizeof(Tile));
  l.pos = l.perm + round_up_256((size_t)R * 4);
  l.rows = l.pos + round_up_256((size_t)R * 4);
  l.h = l.rows + (lays_out_rows(nt) ? round_up_256((size_t)R * K) : 0);
  l.h_sf = l.h + round_up_256((size_t)R * I);
  l.part = l.h_sf + round_up_256((size_t)R * (size_t)ceil_div(I, kGroup));
  l.total = l.part + round_up_256((size_t)R * N * 4);
  return l;
}

cudaError_t launch_experts_a8w4(const uint8_t* a, const uint8_t* a_sf, const int32_t* ids,
                                const float* wt, const uint8_t* w13, const uint8_t* w2, void* out,
                                int64_t T, int k, int E, int K, int I, int N, int32_t* err_flag,
                                void* ws, int num_sms, cudaStream_t s, const char** why) {
  const int64_t R = T * k;
  const int nt = expert_tile(R, k, E);
  const ExpertsLayout l = experts_layout(T, k, E, K, I, N);
  uint8_t* base = static_cast<uint8_t*>(ws);
  int32_t* n_tiles = reinterpret_cast<int32_t*>(base);
  Tile* tiles = reinterpret_cast<Tile*>(base + l.tiles);
  int32_t* perm = reinterpret_cast<int32_t*>(base + l.perm);
  int32_t* pos = reinterpret_cast<int32_t*>(base + l.pos);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(kPlanThreads, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  W4Args g = {};
  g.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
  cudaError_t e = watchdog_address(&g.wd);
  if (e != cudaSuccess) return e;
  const bool small = small_call(R, k);
  if (small) {
    g.ids = ids;
    g.wt = wt;
    g.err_flag = err_flag;
    g.w2 = w2;
    g.E = E;
    g.KB2 = (int)ceil_div(I, kGroup);
    g.NB2 = (int)ceil_div(N, 128);
  }
  if (!small) {
    // (2048 rows 1.5 us faster on eight CTAs, 24576 rows 13; 1024 rows as on one.)
    const int ctas = R > kPlanThreads ? kMaxCluster : 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, w4_plan_kernel, ids, (int)R, E, nt, ctas, tiles, n_tiles, perm, pos,
                           err_flag);
    cfg.numAttrs = 1;
    if (e != cudaSuccess) return e;
  }
  const uint8_t* rows = a;
  int64_t n_rows = T;
  if (lays_out_rows(nt)) {
    const int chunks = K / 16, parts = (int)ceil_div(chunks, kRowChunks);
    cfg.gridDim = dim3((unsigned)ceil_div(T * parts, kRowWarps), 1, 1);
    cfg.blockDim = dim3(kRowWarps * 32, 1, 1);
    e = cudaLaunchKernelEx(&cfg, w4_rows_kernel, reinterpret_cast<const uint4*>(a),
                           static_cast<const int32_t*>(pos), T * parts, parts, k, chunks,
                           reinterpret_cast<uint4*>(base + l.rows));
    if (e != cudaSuccess) return e;
    rows = base + l.rows;
    n_rows = R;
  }

  g.tiles = tiles;
  g.n_tiles = n_tiles;
  g.perm = perm;
  g.k = k;
  const int64_t most = most_tiles(R, E, nt);
  // Gate and up.
  g.w = w13;
  g.a_sf = a_sf;
  g.out = base + l.h;
  g.out_sf = base + l.h_sf;
  g.T = (int)T;
  g.N = I;
  g.KG = g.KB = (int)ceil_div(K, kGroup);
  g.NB = g.NG = (int)ceil_div(I, 128);
  g.splits = nt == 16 ? pick_splits(most * g.NB, g.KB, num_sms, 1) : 1;
  g.kb_per_split = (int)ceil_div(g.KB, g.splits);
  e = launch_tokens<kGateUp>(nt, rows, (uint64_t)n_rows, (uint64_t)K, 2 * (uint64_t)E * g.NB * g.KB, g,
                             most * g.NB, num_sms, s, why);
  if (e != cudaSuccess) return e;
  // Down.
  g.w = w2;
  g.a_sf = base + l.h_sf;
  g.out = base + l.part;
  g.N = N;
  g.KG = g.KB = (int)ceil_div(I, kGroup);
  g.NB = (int)ceil_div(N, 128);
  int64_t units = most * g.NB;
  if (small) {
    g.out = out;
    // One CTA for each choice, or several that share its K range.
    units = T * g.NB;
    g.k_parts = pick_splits(units, g.KB, num_sms, 2, k);
    g.splits = k * g.k_parts;
  } else {
    g.k_parts = 1;
    g.splits = nt == 16 ? pick_splits(units, g.KB, num_sms, 2) : 1;
  }
  g.kb_per_split = (int)ceil_div(g.KB, small ? g.k_parts : g.splits);
  e = launch_tokens<kDown>(nt, base + l.h, (uint64_t)R, (uint64_t)I, (uint64_t)E * g.NB * g.KB, g,
                           units, num_sms, s, why);
  if (e != cudaSuccess || small) return e;
  const int segs = (int)ceil_div(N, kJoinCols);
  cfg.gridDim = dim3((unsigned)ceil_div(T * segs, kJoinWarps), 1, 1);
  cfg.blockDim = dim3(kJoinWarps * 32, 1, 1);
  return cudaLaunchKernelEx(&cfg, w4_join_kernel, reinterpret_cast<const float*>(base + l.part),
                            static_cast<const int32_t*>(pos), wt, static_cast<__nv_bfloat16*>(out), T * segs,
                            segs, N, k);
}

}  // namespace mxq
