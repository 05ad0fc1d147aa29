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
// Form: weight rows on the MMA's M axis (128), tokens on N (16..256), so that
// few tokens cost no padding.  The prepared weight is a sequence of 8704-byte
// blocks, each 128 rows x 128 columns of codes (64 bytes a row) and the
// 512-byte scale atom of those rows: one block is one pipeline stage's operand,
// and a CTA's blocks lie one behind the other in memory.  TMA unpacks the codes
// on the way into shared memory (16 codes in 8 bytes of a 16-byte chunk, 128-byte
// swizzle), where the MMA reads them; no instruction touches a weight.
//
// A CTA makes one unit: 128 weight rows (gate and up rows: twice 128) x NT
// tokens over its share of K.  Warp roles in the main loop:
//   warp 0   copies: weight codes and scale atoms, and the token tile (dense and
//            down products).
//   warp 1   TMEM owner; per stage tcgen05.cp of the scale atoms, four
//            tcgen05.mma (K = 32 each, scale byte k of each word), commit.
//   warp 2   token scales, one byte per row and stage, into the scale atom; in
//            the gate and up product also the token rows themselves, gathered
//            by index four to an instruction.
// Then all eight warps drain the accumulator to shared memory, row-contiguous
// per token, and a half-warp takes a token's 128 values: 16-byte stores, and
// the abs-max of a scale group is four shuffles.  Few units: the K range is
// split over a cluster of up to 8 CTAs, each of which owns some of the tokens,
// receives the partial sums for them through distributed shared memory and adds
// them in rank order.
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

constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint32_t kHintNs = 20;
constexpr uint32_t kWdW4 = 0x80;  // a wait of these kernels ran out
constexpr int kThreads = 256;

constexpr int kCodeBytes = 128 * 64;    // a block's codes in memory
constexpr int kTileBytes = 128 * 128;   // the same, unpacked in shared memory
constexpr int kBlockBytes = kW4BlockBytes;
static_assert(kBlockBytes == kCodeBytes + kSfAtomBytes, "block layout");

enum Mode { kLinear = 0, kGateUp = 1, kDown = 2 };

// Device-side plan of a routed call: which rows each tile holds.
struct Tile {
  int32_t expert, row0, count, pad;
};

struct W4Args {
  const uint8_t* w;       // prepared weight
  const uint8_t* a_sf;    // [rows][KG]
  const Tile* tiles;      // routed forms
  const int32_t* n_tiles;
  const int32_t* perm;    // sorted row -> token * k + choice
  const float* wt;        // [T][k], down product
  void* out;              // kLinear: BF16 [T][N]; kGateUp: codes [rows][N]; kDown: fp32 [T*k][N]
  uint8_t* out_sf;        // kGateUp: [rows][NG]
  uint32_t* wd;           // watchdog word
  int T, N, KG, KB, NB, NG, k;
  int splits, kb_per_split;
};

template <int MODE, int NT, int NSTAGE, bool SPLIT>
struct Cfg {
  static constexpr int NA = MODE == kGateUp ? 2 : 1;
  static constexpr int TOK_ATOMS = (NT + 127) / 128;
  static constexpr int TOK_TILE = NT * 128;
  static constexpr int OFF_W = 0;
  static constexpr int OFF_TOK = NSTAGE * NA * kTileBytes;
  static constexpr int OFF_WSF = OFF_TOK + NSTAGE * TOK_TILE;
  static constexpr int OFF_TSF = OFF_WSF + NSTAGE * NA * kSfAtomBytes;
  static constexpr int PIPE = OFF_TSF + NSTAGE * TOK_ATOMS * kSfAtomBytes;
  // Sums on their way to the epilogue, fp32 [token][weight row] for each
  // accumulator: over the pipeline's buffers, or with a split K, whose other
  // CTAs may still be in their main loop, in a place of its own.
  static constexpr int SUM_BYTES = NA * NT * 128 * 4;
  static constexpr int OFF_SUM = SPLIT ? PIPE : 0;
  static constexpr int OFF_BAR = SPLIT ? PIPE + SUM_BYTES : (PIPE > SUM_BYTES ? PIPE : SUM_BYTES);
  static constexpr int SMEM = OFF_BAR + (2 * NSTAGE + 1) * 8 + 32 + 1024;
  static constexpr int SF_COLS = 4 * NA + 4 * TOK_ATOMS;
  static constexpr int TMEM_USED = NA * NT + NSTAGE * SF_COLS;
  static constexpr int TMEM_COLS = TMEM_USED <= 32    ? 32
                                   : TMEM_USED <= 64  ? 64
                                   : TMEM_USED <= 128 ? 128
                                   : TMEM_USED <= 256 ? 256
                                                      : 512;
  // kind::mxf8f6f4: A E2M1 (format 5), B E4M3 (0), N >> 3 at bits 17-22, UE8M0
  // scales (bit 23), M >> 4 at bits 24-28; the scale byte of each operand is
  // chosen at bits 4-5 (B) and 29-30 (A).
  static constexpr uint32_t IDESC =
      (5u << 7) | (1u << 23) | ((uint32_t)(NT >> 3) << 17) | ((128u >> 4) << 24);
  // Two CTAs share an SM where their shared memory and TMEM allow it: one
  // streams while the other starts or finishes.
  static constexpr int CTAS_PER_SM = SMEM <= 113 * 1024 && TMEM_COLS <= 256 ? 2 : 1;
  static_assert(TMEM_USED <= 512 && SMEM <= 232448, "budgets");
  static_assert(NT % 16 == 0 && NT <= 256, "MMA N");
};

template <int MODE, int NT, int NSTAGE, bool SPLIT>
__global__ void __launch_bounds__(kThreads, (Cfg<MODE, NT, NSTAGE, SPLIT>::CTAS_PER_SM))
    w4_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a,
              const W4Args p) {
  using C = Cfg<MODE, NT, NSTAGE, SPLIT>;
  constexpr int NA = C::NA;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + NSTAGE;
  uint64_t* acc = empty + NSTAGE;
  uint32_t* slot = reinterpret_cast<uint32_t*>(acc + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(slot + 1);
  volatile int* issued = reinterpret_cast<volatile int*>(slot + 2);  // [0] warp 0, [1] warp 2

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ptx::griddep_launch_dependents();

  const int split = SPLIT ? (int)ptx::cluster_rank() : 0;
  const uint32_t unit = blockIdx.x / (uint32_t)p.splits;
  const int tile = (int)(unit / (uint32_t)p.NB);
  const int rb = (int)(unit - (uint32_t)tile * (uint32_t)p.NB);
  const int kb0 = split * p.kb_per_split;
  const int nk = max(0, min(p.KB - kb0, p.kb_per_split));

  int expert = 0, row0, count;
  if constexpr (MODE == kLinear) {
    row0 = tile * NT;
    count = min(NT, p.T - row0);
    // The weight does not depend on what runs before: bring the first blocks
    // into L2 while that finishes.
    if (warp == 0 && lane < NSTAGE && lane < nk)
      ptx::prefetch_l2_bulk(p.w + ((size_t)rb * p.KB + kb0 + lane) * kBlockBytes, kBlockBytes);
    ptx::griddep_wait();
  } else {
    ptx::griddep_wait();
    // The grid covers the most tiles that there can be; the whole cluster
    // leaves where there is none.
    if (tile >= *p.n_tiles) return;
    const Tile t = p.tiles[tile];
    expert = t.expert;
    row0 = t.row0;
    count = t.count;
  }

  if (threadIdx.x == 0) {
    ptx::prefetch_tmap(&tm_w);
    ptx::prefetch_tmap(&tm_a);
    for (int i = 0; i < NSTAGE; ++i) {
      ptx::mbar_init(&full[i], 2);
      ptx::mbar_init(&empty[i], 1);
    }
    ptx::mbar_init(acc, 1);
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
  const uint32_t tmem = *slot;
  if constexpr (SPLIT) ptx::cluster_arrive();  // this CTA's shared memory may be written

  if (warp == 0) {
    // ------------------------------------------------------------- copies
    const uint32_t mat = MODE == kGateUp ? 2u * (uint32_t)expert + (lane & 1) : (uint32_t)expert;
    const size_t blk0 = ((size_t)mat * p.NB + rb) * p.KB + kb0;
    int it = 0;
    for (; it < nk; ++it) {
      const int s = it % NSTAGE;
      if (*abort_flag ||
          !ptx::mbar_wait_hint(&empty[s], ((uint32_t)(it / NSTAGE) & 1u) ^ 1u, kWaitNs, kHintNs)) {
        if (lane == 0 && !*abort_flag) atomicOr(p.wd, kWdW4);
        *abort_flag = 1;
        break;
      }
      if (lane == 0)
        ptx::mbar_arrive_expect_tx(&full[s], NA * kBlockBytes + (MODE == kGateUp ? 0 : C::TOK_TILE));
      __syncwarp();
      // Lanes 0..NA-1: codes; the next NA: their scale atoms; then the tokens.
      if (lane < NA) {
        ptx::tma_load_2d(smem + C::OFF_W + (s * NA + lane) * kTileBytes, &tm_w, &full[s], 0,
                         (int)((blk0 + it) * (kBlockBytes / 64)));
      } else if (lane >= 2 && lane < 2 + NA) {
        ptx::bulk_load(smem + C::OFF_WSF + (s * NA + lane - 2) * kSfAtomBytes,
                       p.w + (blk0 + it) * kBlockBytes + kCodeBytes, kSfAtomBytes, &full[s]);
      } else if (MODE != kGateUp && lane == 4) {
        ptx::tma_load_2d(smem + C::OFF_TOK + s * C::TOK_TILE, &tm_a, &full[s], (kb0 + it) * 128,
                         row0);
      }
      __syncwarp();
    }
    if (lane == 0) issued[0] = it;
  } else if (warp == 2) {
    // ------------------------------------- token scales (and gathered rows)
    // Lane i serves the rows i, i + 32, ...: their bytes of stage `it` are
    // fetched one stage ahead.
    constexpr int ROWS = NT >= 32 ? NT / 32 : 1;
    const uint8_t* src[ROWS];
    bool live[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int r = 32 * j + lane;
      live[j] = r < count;
      int row = row0 + (live[j] ? r : 0);
      if constexpr (MODE == kGateUp) row = p.perm[row] / p.k;
      src[j] = p.a_sf + (size_t)row * p.KG + kb0;
    }
    int g4[4];
    if constexpr (MODE == kGateUp) {
      // The rows past the tile's last repeat its first.
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * lane + i;
        g4[i] = p.perm[row0 + (r < count ? r : 0)] / p.k;
      }
    }
    uint32_t next[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) next[j] = live[j] && nk > 0 ? src[j][0] : 127u;
    int it = 0;
    for (; it < nk; ++it) {
      const int s = it % NSTAGE;
      if (*abort_flag ||
          !ptx::mbar_wait_hint(&empty[s], ((uint32_t)(it / NSTAGE) & 1u) ^ 1u, kWaitNs, kHintNs)) {
        if (lane == 0 && !*abort_flag) atomicOr(p.wd, kWdW4);
        *abort_flag = 1;
        break;
      }
      if constexpr (MODE == kGateUp) {
        if (lane == 0) ptx::mbar_expect_tx(&full[s], C::TOK_TILE);
        __syncwarp();
        for (int i = lane; i < NT / 4; i += 32)
          ptx::tma_gather4(smem + C::OFF_TOK + s * C::TOK_TILE + i * 512, &tm_a, &full[s],
                           (kb0 + it) * 128, g4[0], g4[1], g4[2], g4[3]);
        static_assert(MODE != kGateUp || NT <= 128, "one gather per lane");
      }
      uint32_t cur[ROWS];
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        cur[j] = next[j] * 0x01010101u;
        if (live[j] && it + 1 < nk) next[j] = src[j][it + 1];
      }
      uint8_t* atom = smem + C::OFF_TSF + s * C::TOK_ATOMS * kSfAtomBytes;
      // Row r of an atom owns word (r % 128) / 32 of line r % 32.
#pragma unroll
      for (int j = 0; j < ROWS; ++j)
        *reinterpret_cast<uint32_t*>(atom + (j >> 2) * kSfAtomBytes + lane * 16 + (j & 3) * 4) =
            cur[j];
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&full[s]);
    }
    if (lane == 0) issued[1] = it;
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    for (int it = 0; it < nk; ++it) {
      const int s = it % NSTAGE;
      if (*abort_flag ||
          !ptx::mbar_wait_hint(&full[s], (uint32_t)(it / NSTAGE) & 1u, kWaitNs, kHintNs)) {
        if (lane == 0 && !*abort_flag) atomicOr(p.wd, kWdW4);
        *abort_flag = 1;
        break;
      }
      ptx::tc_fence_after();
      if (lane == 0) {
        const uint32_t sf = tmem + NA * NT + s * C::SF_COLS;
        const uint32_t tok_sf = sf + 4 * NA;
        const uint64_t bdesc = ptx::smem_desc(
            ptx::smem_u32(smem + C::OFF_TOK + s * C::TOK_TILE), 16, 1024, ptx::kSwizzle128B);
#pragma unroll
        for (int a = 0; a < NA; ++a)
          ptx::tmem_cp_32x128b_x4(
              sf + 4 * a, ptx::smem_desc(ptx::smem_u32(smem + C::OFF_WSF + (s * NA + a) * kSfAtomBytes),
                                         128, 128, ptx::kSwizzleNone));
#pragma unroll
        for (int a = 0; a < C::TOK_ATOMS; ++a)
          ptx::tmem_cp_32x128b_x4(
              tok_sf + 4 * a,
              ptx::smem_desc(ptx::smem_u32(smem + C::OFF_TSF + (s * C::TOK_ATOMS + a) * kSfAtomBytes),
                             128, 128, ptx::kSwizzleNone));
#pragma unroll
        for (int a = 0; a < NA; ++a) {
          const uint64_t adesc =
              ptx::smem_desc(ptx::smem_u32(smem + C::OFF_W + (s * NA + a) * kTileBytes), 16, 1024,
                             ptx::kSwizzle128B);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            ptx::mma_mxf8(tmem + a * NT, adesc + 2 * k, bdesc + 2 * k,
                          C::IDESC | ((uint32_t)k << 29) | ((uint32_t)k << 4), sf + 4 * a, tok_sf,
                          (it > 0 || k > 0) ? 1u : 0u);
        }
        ptx::tc_commit(&empty[s]);
      }
      __syncwarp();
    }
    // Everything issued completes before the accumulator is read or freed.
    if (lane == 0) ptx::tc_commit(acc);
  }
  __syncwarp();

  // ------------------------------------------------------------- epilogue
  if (!ptx::mbar_wait(acc, 0, 2 * kWaitNs)) {
    if (lane == 0) atomicOr(p.wd, kWdW4);
    *abort_flag = 1;
  }
  __syncwarp();
  ptx::tc_fence_after();
  if constexpr (SPLIT) ptx::cluster_wait();  // every CTA of the cluster has begun
  {
    // Warp w drains lanes 32 (w % 4)... of half the columns.
    constexpr int CH = NA * NT / 2;
    constexpr int STEP = CH >= 32 ? 32 : CH;
    constexpr int TOK_OWN = NT / 8;  // smallest share of tokens; see below
    static_assert(TOK_OWN >= 2 && CH % STEP == 0 && STEP % 8 == 0, "drain");
    const int row = (warp & 3) * 32 + lane;
    const uint32_t t0 = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (warp >> 2) * CH;
    float* sum = reinterpret_cast<float*>(smem + C::OFF_SUM);
    const int own = NT / p.splits;  // tokens owned by each CTA
#pragma unroll
    for (int c = 0; c < CH; c += STEP) {
      uint32_t v[STEP];
      if constexpr (STEP == 32) {
        ptx::tmem_ld_32x32b_x32(t0 + c, v);
      } else {
#pragma unroll
        for (int i = 0; i < STEP; i += 8) ptx::tmem_ld_32x32b_x8(t0 + c + i, v + i);
      }
      ptx::tmem_ld_wait();
      const int col = (warp >> 2) * CH + c;
#pragma unroll
      for (int i = 0; i < STEP; ++i) {
        const int a = (col + i) / NT, tok = (col + i) % NT;
        const float f = nk > 0 ? __uint_as_float(v[i]) : 0.0f;
        if constexpr (SPLIT) {
          // [rank][owned token][accumulator][row] at the token's owner.
          const int o = tok / own, tl = tok - o * own;
          const uint32_t at =
              ptx::smem_u32(sum + ((split * own + tl) * NA + a) * 128 + row);
          ptx::st_shared_cluster_f32(ptx::map_shared_rank(at, (uint32_t)o), f);
        } else {
          sum[(tok * NA + a) * 128 + row] = f;
        }
      }
    }
  }
  ptx::tc_fence_before();
  if constexpr (SPLIT)
    ptx::cluster_sync();  // all partial sums have arrived; nobody writes here again
  else
    __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if (*abort_flag) {
    __syncthreads();
    // Copies in flight land before the CTA's shared memory is given up: raise
    // each issued stage's missing arrivals, then wait for its phase.
    if (threadIdx.x == 0) {
      const int i0 = issued[0], i2 = issued[1];
      for (int i = min(i0, i2); i < max(i0, i2); ++i) ptx::mbar_arrive(&full[i % NSTAGE]);
      for (int i = max(0, max(i0, i2) - NSTAGE); i < max(i0, i2); ++i)
        ptx::mbar_wait(&full[i % NSTAGE], (uint32_t)(i / NSTAGE) & 1u, kWaitNs);
    }
    __syncthreads();
    return;
  }
  {
    const float* sum = reinterpret_cast<const float*>(smem + C::OFF_SUM);
    const int own = NT / p.splits;
    const int first = SPLIT ? split * own : 0;
    const int mine = min(own, count - first);  // tokens of this CTA
    const int sub = lane & 15;
    for (int i = 2 * warp; i < mine; i += 2 * (kThreads / 32)) {
      const int tl = i + (lane >> 4);
      const bool in = tl < mine;
      float v[NA][8];
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        const float* at = sum + ((in ? tl : i) * NA + a) * 128 + 8 * sub;
        *reinterpret_cast<float4*>(&v[a][0]) = *reinterpret_cast<const float4*>(at);
        *reinterpret_cast<float4*>(&v[a][4]) = *reinterpret_cast<const float4*>(at + 4);
        if constexpr (SPLIT) {
          for (int r = 1; r < p.splits; ++r) {
            const float* ar = at + r * own * NA * 128;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[a][e] += ar[e];
          }
        }
      }
      const int n = rb * 128 + 8 * sub;
      const int tok = first + tl;
      if constexpr (MODE == kLinear) {
        if (in && n < p.N)
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) +
                                    (size_t)(row0 + tok) * p.N + n) = to_bf16x8(v[0]);
      } else if constexpr (MODE == kGateUp) {
        float h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = v[0][e] / (1.0f + expf(-v[0][e])) * v[NA - 1][e];
        uint32_t sb;
        const float amax = half_warp_amax(h);
        const uint2 codes = encode8(h, amax, &sb);
        if (in && n < p.N) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + (size_t)(row0 + tok) * p.N + n) =
              codes;
          if (sub == 0) p.out_sf[(size_t)(row0 + tok) * p.NG + rb] = (uint8_t)sb;
        }
      } else {
        if (in && n < p.N) {
          const int pair = p.perm[row0 + tok];
          const float w = p.wt[pair];
          float* o = static_cast<float*>(p.out) + (size_t)pair * p.N + n;
          *reinterpret_cast<float4*>(o) =
              make_float4(v[0][0] * w, v[0][1] * w, v[0][2] * w, v[0][3] * w);
          *reinterpret_cast<float4*>(o + 4) =
              make_float4(v[0][4] * w, v[0][5] * w, v[0][6] * w, v[0][7] * w);
        }
      }
    }
  }
}

// ------------------------------------------------------------ plan and join
// One CTA counts the rows of each expert, lays out the tiles and sorts the rows
// by expert.  The order of an expert's rows does not matter: each is summed by
// itself, and lands at its own place.
constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads) w4_plan_kernel(const int32_t* ids, int R, int E,
                                                               int nt, Tile* tiles,
                                                               int32_t* n_tiles, int32_t* perm,
                                                               int32_t* err_flag) {
  __shared__ int cnt[kMaxExperts], cur[kMaxExperts];
  __shared__ int wsum[32], wtile[32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  static_assert(kMaxExperts <= kPlanThreads, "one expert per thread");
  if (tid < kMaxExperts) cnt[tid] = 0;
  __syncthreads();
  bool bad = false;
  for (int i = tid; i < R; i += kPlanThreads) {
    const int e = ids[i];
    if (e >= 0 && e < E)
      atomicAdd(&cnt[e], 1);
    else
      bad |= e != -1;
  }
  if (bad && err_flag != nullptr) atomicOr(err_flag, MXQ_DEVERR_EXPERT);
  __syncthreads();
  const int c = tid < E ? cnt[tid] : 0;
  const int nt_e = (c + nt - 1) / nt;
  int sc = c, st = nt_e;  // inclusive sums over the warp, then over warps
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, sc, m), b = __shfl_up_sync(0xffffffffu, st, m);
    if (lane >= m) {
      sc += a;
      st += b;
    }
  }
  if (lane == 31) {
    wsum[warp] = sc;
    wtile[warp] = st;
  }
  __syncthreads();
  int pc = 0, pt = 0;
  for (int w = 0; w < warp; ++w) {
    pc += wsum[w];
    pt += wtile[w];
  }
  const int row0 = pc + sc - c, tile0 = pt + st - nt_e;
  if (tid < E) {
    cur[tid] = row0;
    for (int i = 0; i < nt_e; ++i) {
      Tile t;
      t.expert = tid;
      t.row0 = row0 + i * nt;
      t.count = min(nt, c - i * nt);
      t.pad = 0;
      tiles[tile0 + i] = t;
    }
  }
  if (tid == kPlanThreads - 1) *n_tiles = pt + st;
  __syncthreads();
  for (int i = tid; i < R; i += kPlanThreads) {
    const int e = ids[i];
    if (e >= 0 && e < E) perm[atomicAdd(&cur[e], 1)] = i;
  }
}

// out[t] = sum over the token's choices, in their order.
__global__ void __launch_bounds__(256) w4_join_kernel(const float* part, const int32_t* ids,
                                                      uint4* out, int64_t items, int chunks, int k,
                                                      int E) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (it >= items) return;
  const int64_t t = it / chunks;
  const int c = (int)(it - t * chunks);
  float y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < k; ++j) {
    const int e = ids[t * k + j];
    if (e < 0 || e >= E) continue;
    const float4* s = reinterpret_cast<const float4*>(part) + ((size_t)(t * k + j) * chunks + c) * 2;
    const float4 a = s[0], b = s[1];
    y[0] += a.x;
    y[1] += a.y;
    y[2] += a.z;
    y[3] += a.w;
    y[4] += b.x;
    y[5] += b.y;
    y[6] += b.z;
    y[7] += b.w;
  }
  out[it] = to_bf16x8(y);
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

template <int MODE, int NT, int NSTAGE, bool SPLIT>
cudaError_t launch_cfg(const void* a, uint64_t a_rows, uint64_t K, uint64_t blocks, W4Args args,
                       int64_t units, cudaStream_t s, const char** why) {
  using C = Cfg<MODE, NT, NSTAGE, SPLIT>;
  CUtensorMap tm_w, tm_a;
  if (!encode_weight(&tm_w, args.w, blocks) ||
      !encode_rows(&tm_a, a, K, a_rows, MODE == kGateUp ? 1 : NT)) {
    *why = "cuTensorMapEncodeTiled failed (driver entry point missing or arguments rejected)";
    return cudaErrorInvalidValue;
  }
  auto kern = w4_kernel<MODE, NT, NSTAGE, SPLIT>;
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * args.splits), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
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

// CTAs along K for `units` units of KB blocks each: about two CTAs for each SM,
// powers of two up to the portable cluster size, and two blocks each at least.
int pick_splits(int64_t units, int KB, int slots) {
  int s = 1;
  while (s < 8 && units * s * 2 <= slots && KB >= 4 * s) s *= 2;
  return s;
}

}  // namespace

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
  g.w = w;
  g.a_sf = a_sf;
  g.out = out;
  g.T = (int)T;
  g.N = N;
  g.KG = g.KB = (int)ceil_div(K, kGroup);
  g.NB = (int)ceil_div(N, 128);
  g.splits = 1;
  g.kb_per_split = g.KB;
  cudaError_t e = watchdog_address(&g.wd);
  if (e != cudaSuccess) return e;
  const uint64_t blocks = (uint64_t)g.NB * g.KB;
  if (T <= 32) {
    g.splits = pick_splits(g.NB, g.KB, 2 * num_sms);
    g.kb_per_split = (int)ceil_div(g.KB, g.splits);
  }
  if (T <= 16) {
    return g.splits > 1 ? launch_cfg<kLinear, 16, 5, true>(a, T, K, blocks, g, g.NB, s, why)
                        : launch_cfg<kLinear, 16, 5, false>(a, T, K, blocks, g, g.NB, s, why);
  }
  if (T <= 32) {
    return g.splits > 1 ? launch_cfg<kLinear, 32, 4, true>(a, T, K, blocks, g, g.NB, s, why)
                        : launch_cfg<kLinear, 32, 4, false>(a, T, K, blocks, g, g.NB, s, why);
  }
  if (T <= 64) return launch_cfg<kLinear, 64, 4, false>(a, T, K, blocks, g, g.NB, s, why);
  return launch_cfg<kLinear, 128, 3, false>(a, T, K, blocks, g, ceil_div(T, 128) * g.NB, s, why);
}

namespace {
// Tokens of a tile of the routed products.
int expert_tile(int64_t R, int E) {
  const int64_t avg = ceil_div(R, E);
  return avg <= 8 ? 16 : avg <= 24 ? 32 : avg <= 48 ? 64 : 128;
}
int64_t most_tiles(int64_t R, int E, int nt) { return R / nt + (R < E ? R : E); }
}  // namespace

ExpertsLayout experts_layout(int64_t T, int k, int E, int I, int N) {
  const int64_t R = T * k;
  ExpertsLayout l;
  l.tiles = 256;  // the number of tiles lies before them
  l.perm = l.tiles + round_up_256((size_t)most_tiles(R, E, expert_tile(R, E)) * sizeof(Tile));
  l.h = l.perm + round_up_256((size_t)R * 4);
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
  const int nt = expert_tile(R, E);
  const ExpertsLayout l = experts_layout(T, k, E, I, N);
  uint8_t* base = static_cast<uint8_t*>(ws);
  int32_t* n_tiles = reinterpret_cast<int32_t*>(base);
  Tile* tiles = reinterpret_cast<Tile*>(base + l.tiles);
  int32_t* perm = reinterpret_cast<int32_t*>(base + l.perm);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(kPlanThreads, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  W4Args g = {};
  cudaError_t e = watchdog_address(&g.wd);
  if (e != cudaSuccess) return e;
  e = cudaLaunchKernelEx(&cfg, w4_plan_kernel, ids, (int)R, E, nt, tiles, n_tiles, perm, err_flag);
  if (e != cudaSuccess) return e;

  g.tiles = tiles;
  g.n_tiles = n_tiles;
  g.perm = perm;
  g.wt = wt;
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
  g.splits = nt == 16 ? pick_splits(most * g.NB, g.KB, num_sms) : 1;
  g.kb_per_split = (int)ceil_div(g.KB, g.splits);
  uint64_t blocks = 2 * (uint64_t)E * g.NB * g.KB;
  int64_t units = most * g.NB;
  if (nt == 16) {
    e = g.splits > 1 ? launch_cfg<kGateUp, 16, 5, true>(a, T, K, blocks, g, units, s, why)
                     : launch_cfg<kGateUp, 16, 3, false>(a, T, K, blocks, g, units, s, why);
  } else if (nt == 32) {
    e = launch_cfg<kGateUp, 32, 5, false>(a, T, K, blocks, g, units, s, why);
  } else if (nt == 64) {
    e = launch_cfg<kGateUp, 64, 5, false>(a, T, K, blocks, g, units, s, why);
  } else {
    e = launch_cfg<kGateUp, 128, 4, false>(a, T, K, blocks, g, units, s, why);
  }
  if (e != cudaSuccess) return e;
  // Down.
  g.w = w2;
  g.a_sf = base + l.h_sf;
  g.out = base + l.part;
  g.out_sf = nullptr;
  g.N = N;
  g.KG = g.KB = (int)ceil_div(I, kGroup);
  g.NB = (int)ceil_div(N, 128);
  g.splits = nt == 16 ? pick_splits(most * g.NB, g.KB, 2 * num_sms) : 1;
  g.kb_per_split = (int)ceil_div(g.KB, g.splits);
  blocks = (uint64_t)E * g.NB * g.KB;
  units = most * g.NB;
  const uint8_t* h = base + l.h;
  if (nt == 16) {
    e = g.splits > 1 ? launch_cfg<kDown, 16, 5, true>(h, R, I, blocks, g, units, s, why)
                     : launch_cfg<kDown, 16, 5, false>(h, R, I, blocks, g, units, s, why);
  } else if (nt == 32) {
    e = launch_cfg<kDown, 32, 4, false>(h, R, I, blocks, g, units, s, why);
  } else if (nt == 64) {
    e = launch_cfg<kDown, 64, 4, false>(h, R, I, blocks, g, units, s, why);
  } else {
    e = launch_cfg<kDown, 128, 3, false>(h, R, I, blocks, g, units, s, why);
  }
  if (e != cudaSuccess) return e;
  const int chunks = N / 8;
  const int64_t items = T * chunks;
  cfg.gridDim = dim3((unsigned)ceil_div(items, 256), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  return cudaLaunchKernelEx(&cfg, w4_join_kernel, reinterpret_cast<const float*>(base + l.part), ids,
                            static_cast<uint4*>(out), items, chunks, k, E);
}

}  // namespace mxq
