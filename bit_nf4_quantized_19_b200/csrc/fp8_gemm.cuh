// Block-scaled 8-bit GEMM of the linear layer on an 8-bit base (sm_100a).
//
//   forward:  Y[m, n]  = sum_k deq(X)[m, k] deq(W)[n, k]  +  sum_j s XA[m, j] B[j, n]
//   dX:       dX[m, k] = sum_n deq(dY)[m, n] deq(W)[n, k] +  sum_j s G[m, j] A[k, j]
//
// Codes are fp8, factors powers of two for each 1 x 128 (tokens) or 128 x 128 (weight)
// block, and the tensor core applies them: tcgen05.mma kind::mxf8f6f4 multiplies each
// 32-value step of a row by that row's UE8M0 byte, so the accumulator holds the finished
// fp32 sum and no CUDA core touches a partial product.  A block of 128 is four such steps
// under one byte.  The factor tile in TMEM holds one 32-bit word per row, and the
// instruction names which of its four bytes to use: word g of a row is the bytes of
// blocks 4g .. 4g+3, so one factor tile serves 512 values of the contraction.
//
// CTA pairs (cta_group::2): a tile is 256 tokens x 256 outputs; each CTA holds 128 token
// rows (A operand, K-major) and 128 of the 256 output columns (B operand; forward K-major
// rows of W, dX MN-major: the same row-major W read as [contraction n][128 outputs k]),
// so W has one copy for both directions (its blocks are square, so are its factors).
// The rank-r term is appended as bf16 steps (kind::f16) into the same accumulator: the
// token side is s XA (or s G) as bf16 hi | lo halves, each padded with zero columns to
// r16 = r rounded up to 16; the output side is B [r, N] (MN-major) or A [K, r] (K-major),
// once for each half, its rows or columns past r zero-filled by TMA.
//
// Few tokens (forward, M <= kFwTokens): the operands change places.  The weight's 256 rows are the
// MMA's rows and the tokens, rounded up to 32, its columns, so the tensor core takes nt / 256 of
// the time and HBM is the bound; the smaller stage (16 KB of weight, at most 8 KB of tokens) makes
// eight of them.  The epilogue's lanes are outputs: it stores a token's 32 of them at once, no
// staging.  13 tokens, no adapter, weights in turn, replayed: 8192 x 22016 35 us (40 as 256 token
// rows), 22016 x 8192 35 (54), floor 28; with r 64 and so XA in front 38 (43) and 39 (60).
//
// TMEM: two 256-column accumulators that overlap by 32 columns, [0, 256) and [224, 480),
// leave 32 columns for two factor slots.  The epilogue drains the shared columns of a
// tile first and then lets the next tile's MMAs start, so the rest of its stores run
// beside them, as with two full accumulators.
//
// Warps (384 threads, one CTA per SM, persistent over tiles):
//   0     TMA producer of this CTA's operand tiles (completing on the leader's barrier)
//   1     TMEM allocator; in the leader the MMA issuer
//   4..7  epilogue: TMEM -> bf16 (or fp32 partials) -> shared memory -> TMA store
//   8..11 factor writers: each TMEM lane quadrant needs its own copy of the factor tile
// Measured: forward of 8192 tokens, 22016 x 8192, r 64: one launch takes 1.455 M cycles, 1.03 ms alone
// (2.9 PFLOP/s, where twice the measured bf16 rate is 3.39) and 1.17 ms under a continuous load.  The
// tensor pipe is active 89% of them, 96% of the cycles in which the SMs are: the power limit bounds
// it, with the SM clock at 1.41 GHz and 1.24 GHz.  dX of 8192 tokens, 8192 x 8192: 345 to 362 us.
// The rest is the switch between tiles (about 1500 cycles), start and end, and, with few tiles, the
// last round: 1024 tokens of 18944 x 8192, four whole rounds: active 84%; 4096 x 4096 x 4096,
// 3.46 rounds: 60 us for 41.  Dividing a last round's tiles as well cost more in its exchange than
// the half round (57 to 70 us).
#pragma once
#include "common.cuh"
#include "fp8_quant.cuh"
#include "pipeline.cuh"

namespace qlora {

constexpr int kFgThreads = 384;
constexpr int kFgRows = 128;                      // tokens and outputs per CTA of a pair
constexpr int kFgTile = 256;                      // tokens and outputs per tile
constexpr int kFgStages = 6;
constexpr int kFgOpBytes = kFgRows * 128;         // one operand tile: 128 rows x 128 bytes
constexpr int kFgStageBytes = 2 * kFgOpBytes;
constexpr int kFgOutBytes = 4096;                 // one store box: 32 rows x 128 bytes
constexpr int kFgTmemCols = 512;
// The form for up to kFwTokens tokens: the weight is the MMA's A operand, the tokens its B
constexpr int kFwTokens = 128;
constexpr int kFwStages = 8;
constexpr int kFwStageBytes = kFgOpBytes + kFwTokens / 2 * 128;
constexpr int kFwSmemBytes = 1024 + kFwStages * kFwStageBytes + 256;
constexpr int kFgAcc1 = 224;                      // first column of the odd tiles' accumulator
constexpr int kFgSf = 480;                        // factor slots: 16 columns each (4 A + 8 B used)
constexpr int kFgSfSlots = 2;
constexpr int kFgSmemBytes = 1024 + kFgStages * kFgStageBytes + 4 * 2 * kFgOutBytes + 256;
static_assert(kFgSmemBytes <= 227 * 1024, "shared memory of the 8-bit GEMM exceeds the per-CTA limit");
static_assert(kFgSfSlots == 2, "the MMA issuer alternates two factor slots");
static_assert(kFgSf + 16 * kFgSfSlots <= kFgTmemCols && kFgAcc1 + kFgTile <= kFgSf, "TMEM columns overlap");

struct Fp8GemmParams {
  int M;               // tokens
  int n_out;           // output row length
  int num_m_tiles, num_w_tiles, group_m;
  int kb_main;         // 128-value blocks of the contraction
  int kb_lora;         // 64-wide bf16 steps of the rank-r term, both halves (0: no adapter)
  int r16;
  int splits;          // parts of the contraction; > 1: fp32 partials [splits][M][n_out]
  int groups_per_split;   // 512-value groups per part
  const uint8_t *sa;   // factors of the tokens' rows [M, sa_pitch]
  int sa_pitch;
  const uint8_t *sw;   // factors of W [ceil(N / 128), sw_pitch]
  int sw_pitch;
  int out_blocks;      // 128-wide blocks of the output (forward: factor rows, dX: factor columns)
  uint32_t a_fmt;      // token codes: 0 e4m3, 1 e5m2
  int late_wait;       // the kernel before wrote hl alone: only the first rank-r step waits for it
  int nt;              // few tokens: M rounded up to 32, the MMA's N
  void *out;           // few tokens: bf16 [M, n_out], or the fp32 partials
  uint64_t limit_ns;
};

// ------------------------------------------------------------------ instruction forms
// Instruction descriptor of kind::mxf8f6f4 with UE8M0 factors and fp32 accumulation.
__host__ __device__ constexpr uint32_t make_idesc_mxf8(int M, int N, uint32_t a_fmt, uint32_t b_fmt, bool b_mn_major) {
  return (a_fmt << 7) | (b_fmt << 10) | (static_cast<uint32_t>(b_mn_major) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24);
}
// Byte of the factor words the instruction uses, for A and B.
__host__ __device__ constexpr uint32_t idesc_sf_id(uint32_t id) { return (id << 4) | (id << 29); }

QDEV void mma_mxf8_ss_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                           uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb));
}
QDEV void tmem_st_32x32b_x4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
QDEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// TMA load into this CTA whose completion is counted on `bar` (a shared::cluster
// address, here the barrier of the pair's leader).  No multicast.
QDEV void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
QDEV void tma_store_3d(const CUtensorMap *map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}
QDEV void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
QDEV void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }

// ------------------------------------------------------------------ work items
// Item i of unit u (a CTA pair) of G: tile and part of the contraction.
struct Fp8Item {
  int m0, w0;          // first token, first output
  int kb0, kb1;        // 128-value blocks
  int split;
  bool lora;
};
QDEV bool fp8_item(const Fp8GemmParams &p, int it, Fp8Item &w) {
  const int tiles = p.num_m_tiles * p.num_w_tiles;
  const int i = static_cast<int>(blockIdx.x >> 1) + it * static_cast<int>(gridDim.x >> 1);
  if (i >= tiles * p.splits) return false;
  const int t = i / p.splits;
  w.split = i - t * p.splits;
  // groups of group_m token tiles, the token tile fastest within a group (see tile_coords)
  const int per_group = p.group_m * p.num_w_tiles;
  const int grp = t / per_group;
  const int m_base = grp * p.group_m;
  const int gm = min(p.group_m, p.num_m_tiles - m_base);
  const int idx = t - grp * per_group;
  w.m0 = (m_base + idx % gm) * kFgTile;
  w.w0 = (idx / gm) * kFgTile;
  w.kb0 = w.split * p.groups_per_split * 4;
  w.kb1 = min(p.kb_main, w.kb0 + p.groups_per_split * 4);
  w.lora = w.split == 0 && p.kb_lora > 0;
  return true;
}

template <bool DX, bool FEW>
__global__ void __launch_bounds__(kFgThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tm_a,     // token codes u8 [M, contraction], box {128, 128}
                    const __grid_constant__ CUtensorMap tm_w,     // weight codes u8 [N, K], box {128, 128}
                    const __grid_constant__ CUtensorMap tm_hl,    // bf16 [M, 2 r16], box {64, 128}
                    const __grid_constant__ CUtensorMap tm_lw,    // B [r, N], box {64, 64}; A [K, r], box {64, 128}
                    const __grid_constant__ CUtensorMap tm_out,   // [splits, M, n_out], box {128 bytes, 32, 1}
                    const __grid_constant__ Fp8GemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  static_assert(!(DX && FEW), "few tokens: forward only");
  constexpr int kStages = FEW ? kFwStages : kFgStages, kStageBytes = FEW ? kFwStageBytes : kFgStageBytes;
  uint8_t *sOut = smem + kStages * kStageBytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(sOut + (FEW ? 0 : 4 * 2 * kFgOutBytes));   // used at the leader
  uint64_t *empty = full + kStages;
  uint64_t *sf_full = empty + kStages;                                      // used at the leader
  uint64_t *sf_empty = sf_full + kFgSfSlots;
  uint64_t *tmem_full = sf_empty + kFgSfSlots;
  uint64_t *tmem_empty = tmem_full + 1;                                       // used at the leader
  uint64_t *drain = tmem_empty + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int half = static_cast<int>(rank) * kFgRows;   // this CTA's tokens and outputs within a tile

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], 1); }
    for (int i = 0; i < kFgSfSlots; ++i) { mbar_init(&sf_full[i], 8); mbar_init(&sf_empty[i], 1); }
    mbar_init(tmem_full, 1);
    mbar_init(tmem_empty, 8);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_a);
    prefetch_tmap(&tm_w);
    if (!FEW) prefetch_tmap(&tm_out);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kFgTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // both CTAs' barriers are initialized before either arrives on the other's
  tc_fence_after();
  if (!p.late_wait) pdl_wait();
  pdl_trigger();
  // The allocation is all of TMEM, so it starts at address 0 (in both CTAs) and every TMEM
  // address below is a constant.  Should it not, no role runs and the status says so.
  const uint32_t tmem_base = *tmem_slot;
  if (tmem_base != 0u && tid == 0) atomicOr(&g_device_status, kStatLayout);
  const Waiter wt{abort_flag, p.limit_ns};
  volatile int no_abort = 0;
  const Waiter final_wt{&no_abort, drain_limit_ns(p.limit_ns)};

  if (tmem_base != 0u) {
  } else if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint32_t bytes = FEW ? 2u * kFgOpBytes + 128u * static_cast<uint32_t>(p.nt) : 2u * kStageBytes;   // both CTAs'
      uint32_t armed = 0, last = 0;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true, waited = !p.late_wait;
      Fp8Item w;
      for (int it = 0; ok && fp8_item(p, it, w); ++it) {
        const int m0 = FEW ? static_cast<int>(rank) * (p.nt >> 1) : w.m0 + half;
        const int nst = (w.kb1 - w.kb0) + (w.lora ? p.kb_lora : 0);
        for (int j = 0; j < nst; ++j) {
          if (!wait_bar(&empty[s], ph ^ 1u, wt)) { ok = false; break; }
          // the MMA's A operand lies first: the tokens' tile, or with few tokens the weight's
          const uint32_t a0 = smem_u32(smem + s * kStageBytes);
          const uint32_t a = FEW ? a0 + kFgOpBytes : a0, b = FEW ? a0 : a0 + kFgOpBytes;
          const uint32_t bar = map_rank(smem_u32(&full[s]), 0u);
          const int kb = w.kb0 + j;
          const int ls = kb - w.kb1;
          if (ls < 0) {
            // the leader's barrier counts both CTAs' bytes; the peer's may land before
            // the leader arms the phase, which cannot complete without that arrival
            if (leader) mbar_arrive_expect_tx(&full[s], bytes);
            tma_load_2d_pair(a, &tm_a, bar, kb * 128, m0);
            if (DX) tma_load_2d_pair(b, &tm_w, bar, w.w0 + half, kb * 128);
            else tma_load_2d_pair(b, &tm_w, bar, kb * 128, w.w0 + half);
          } else {
            // rank-r step: columns 64 cc .. of the hi (then the lo) halves, and the same
            // 64 rows (forward) or columns (dX) of the weight-side operand for both
            if (!waited) {
              pdl_wait();
              waited = true;
            }
            const int lo = ls >= p.kb_lora / 2 ? 1 : 0, cc = ls - lo * (p.kb_lora / 2);
            if (leader) mbar_arrive_expect_tx(&full[s], bytes);
            tma_load_2d_pair(a, &tm_hl, bar, lo * p.r16 + cc * 64, m0);
            if (DX) {
              tma_load_2d_pair(b, &tm_lw, bar, cc * 64, w.w0 + half);
            } else {
              tma_load_2d_pair(b, &tm_lw, bar, w.w0 + half, cc * 64);
              tma_load_2d_pair(b + kFgOpBytes / 2, &tm_lw, bar, w.w0 + half + 64, cc * 64);
            }
          }
          armed |= 1u << s;
          last = (last & ~(1u << s)) | (ph << s);
          if (++s == kStages) { s = 0; ph ^= 1u; }
        }
      }
      if (!waited) pdl_wait();   // this grid ends after the one before
      if (leader) {
        // every copy that the armed phases count (both CTAs') has landed before the
        // cluster barrier at the end (bounded)
        for (int i = 0; i < kStages; ++i)
          if (armed & (1u << i)) wait_bar(&full[i], (last >> i) & 1u, final_wt);
      }
      if (!ok) {
        // given up: copies may be in flight that no armed phase counts; they land in
        // microseconds, long before this delay ends
        for (int i = 0; i < 200; ++i) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    // The whole warp walks the loop and one elected lane issues: with warp-uniform control
    // flow the descriptors stay in uniform registers.  (One lane inside a divergent branch
    // took 570 cycles to issue a stage's four MMAs and its commit, longer than the 512 the
    // tensor core needs for them.)
    if (leader) {
      const bool el = elect_one();
      const uint32_t idesc = FEW ? make_idesc_mxf8(kFgTile, p.nt, 0u, p.a_fmt, false)
                                 : make_idesc_mxf8(kFgTile, kFgTile, p.a_fmt, 0u, DX);
      const uint32_t idesc_lora = FEW ? make_idesc_bf16(kFgTile, p.nt, true, false)
                                      : make_idesc_bf16(kFgTile, kFgTile, false, !DX);
      constexpr uint32_t b_step = DX ? (4096u >> 4) : (32u >> 4);   // 32 rows, or 32 bytes of a row
      const uint32_t a0 = smem_u32(smem), b0 = a0 + kFgOpBytes;
      const uint64_t ad0 = sw128_desc(a0, 16, 1024);
      const uint64_t bd0 = sw128_desc(b0, 16, 1024);               // MN-major: 8-row groups 1024 apart
      // rank-r operands: of the weight's side, forward MN-major, two 64-wide groups of 64 rows; dX
      // K-major.  The tokens' side is K-major.
      constexpr uint32_t mn_step = 2048u >> 4, k_step = 32u >> 4;
      const uint64_t al0 = FEW ? sw128_desc(a0, kFgOpBytes / 2, 1024) : ad0;
      const uint64_t bl0 = DX || FEW ? sw128_desc(b0, 16, 1024) : sw128_desc(b0, kFgOpBytes / 2, 1024);
      constexpr uint32_t al_step = FEW ? mn_step : k_step, bl_step = DX || FEW ? k_step : mn_step;
      int s = 0, slot = 0;
      uint32_t ph = 0, sfph = 0;
      bool ok = true;
      // the next stage's (and factor slot's) completion is asked for before a stage's MMAs
      // are issued and answered behind them, so that a wait costs nothing when it is early
      bool full_seen = false, sf_seen = false;
      Fp8Item w;
      for (int it = 0; ok && fp8_item(p, it, w); ++it) {
        // the previous tile's shared columns (and all of the tile before it) are drained
        if (it > 0 && !wait_bar_warp(tmem_empty, static_cast<uint32_t>(it - 1) & 1u, wt)) break;
        tc_fence_after();
        const uint32_t d = (it & 1) ? kFgAcc1 : 0;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          const uint32_t sf = kFgSf + slot * 16;
          if ((kb & 3) == 0 && !sf_seen && !wait_bar_warp(&sf_full[slot], sfph, wt)) { ok = false; break; }
          if (!full_seen && !wait_bar_warp(&full[s], ph, wt)) { ok = false; break; }
          tc_fence_after();
          const bool group_end = (kb & 3) == 3 || kb + 1 == w.kb1;
          const int s1 = s + 1 == kStages ? 0 : s + 1, slot1 = slot ^ 1;
          const uint32_t ph1 = s1 ? ph : ph ^ 1u, sfph1 = slot1 ? sfph : sfph ^ 1u;
          const uint32_t peek = (mbar_test(&full[s1], ph1) ? 1u : 0u) |
                                (group_end && mbar_test(&sf_full[slot1], sfph1) ? 2u : 0u);
          const uint64_t ad = ad0 + static_cast<uint64_t>(s * (kStageBytes >> 4));
          const uint64_t bd = bd0 + static_cast<uint64_t>(s * (kStageBytes >> 4));
          const uint32_t id = idesc | idesc_sf_id(static_cast<uint32_t>(kb & 3));
          if (el) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_mxf8_ss_pair(d, ad + k * 2, bd + k * b_step, id, sf, sf + 4, (kb > w.kb0 || k) ? 1u : 0u);
            mma_commit_pair(&empty[s], static_cast<uint16_t>(0x3));
            if (group_end) mma_commit_pair(&sf_empty[slot], static_cast<uint16_t>(0x3));
          }
          full_seen = __all_sync(0xffffffffu, peek & 1u) != 0;
          sf_seen = __all_sync(0xffffffffu, peek & 2u) != 0;
          if (group_end) { slot = slot1; sfph = sfph1; }
          s = s1;
          ph = ph1;
        }
        for (int ls = 0; ok && w.lora && ls < p.kb_lora; ++ls) {
          if (!full_seen && !wait_bar_warp(&full[s], ph, wt)) { ok = false; break; }
          full_seen = false;
          tc_fence_after();
          const uint64_t ad = al0 + static_cast<uint64_t>(s * (kStageBytes >> 4));
          const uint64_t bd = bl0 + static_cast<uint64_t>(s * (kStageBytes >> 4));
          const int nk = min(4, p.r16 / 16 - (ls % (p.kb_lora / 2)) * 4);
          if (el) {
            for (int k = 0; k < nk; ++k) mma_bf16_ss_pair(d, ad + k * al_step, bd + k * bl_step, idesc_lora, 1u);
            mma_commit_pair(&empty[s], static_cast<uint16_t>(0x3));
          }
          if (++s == kStages) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        if (el) mma_commit_pair(tmem_full, static_cast<uint16_t>(0x3));
      }
      if (el) mma_commit_pair(drain, static_cast<uint16_t>(0x3));
      __syncwarp();
    }
    // the MMAs read both CTAs' shared memory and write both TMEMs: they complete before
    // either CTA releases its own (bounded)
    if (lane == 0) wait_bar(drain, 0, final_wt);
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const uint32_t tq = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t buf0 = smem_u32(sOut + q * 2 * kFgOutBytes);
    uint32_t nbuf = 0;
    Fp8Item w;
    for (int it = 0; fp8_item(p, it, w); ++it) {
      if (!__all_sync(0xffffffffu, wait_bar(tmem_full, static_cast<uint32_t>(it) & 1u, wt) ? 1 : 0)) break;
      tc_fence_after();
      const uint32_t acc = tq + ((it & 1) ? kFgAcc1 : 0);
      if (FEW) {
        // lanes are outputs, columns tokens; the accumulators do not overlap, and the other one
        // was read before this tile was waited for
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tmem_empty, 0u);
        const int n = w.w0 + half + q * 32 + lane;
        for (int c = 0; c < p.nt; c += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(acc + c, v);
          tmem_wait_ld();
          if (n >= p.n_out) continue;
          if (p.splits > 1) {
            float *o = static_cast<float *>(p.out) + (static_cast<int64_t>(w.split) * p.M + c) * p.n_out + n;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c + j < p.M) o[static_cast<int64_t>(j) * p.n_out] = __uint_as_float(v[j]);
          } else {
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + static_cast<int64_t>(c) * p.n_out + n;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c + j < p.M) o[static_cast<int64_t>(j) * p.n_out] = __float2bfloat16_rn(__uint_as_float(v[j]));
          }
        }
        continue;
      }
      const int row0 = w.m0 + half + q * 32;
      const bool partial = p.splits > 1;
      const int chunks = partial ? 8 : 4;          // boxes of 128 bytes: 32 fp32 or 64 bf16 columns
      for (int i = 0; i < chunks; ++i) {
        // the columns shared with the next tile's accumulator first
        const int c = (it & 1) ? i : chunks - 1 - i;
        const uint32_t buf = buf0 + (nbuf & 1u) * kFgOutBytes + lane * 128;
        uint32_t v[32], u[32];
        if (partial) {
          tmem_ld_32x32b_x32(acc + c * 32, v);
          tmem_wait_ld();
        } else {
          tmem_ld_32x32b_x32(acc + c * 64, v);
          tmem_ld_32x32b_x32(acc + c * 64 + 32, u);
          tmem_wait_ld();
        }
        if (i == 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(tmem_empty, 0u);
        }
        if (!partial) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            v[j] = pack_bf16x2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) v[16 + j] = pack_bf16x2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
        }
        if (lane == 0) bulk_wait_read<1>();        // the store that read this buffer two boxes ago
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          st_shared_v4(buf + ((j ^ (lane & 7)) << 4), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          const int x = w.w0 + c * (partial ? 32 : 64);
          if (row0 < p.M && x < p.n_out) tma_store_3d(&tm_out, buf, x, row0, w.split);
          bulk_commit();
        }
        ++nbuf;
      }
    }
    if (lane == 0) bulk_wait_read<0>();
  } else if (warp >= 8) {
    // ------------------------------------------------------------ factor writers
    const int q = warp & 3;
    const uint32_t tq = (static_cast<uint32_t>(q * 32) << 16) + kFgSf;
    int slot = 0;
    uint32_t ph = 0;
    bool ok = true;
    Fp8Item w;
    for (int it = 0; ok && fp8_item(p, it, w); ++it) {
      const int ob = w.w0 >> 7;
      for (int g = w.kb0 >> 2; 4 * g < w.kb1; ++g) {
        uint32_t a[4], b[2] = {0x7F7F7F7Fu, 0x7F7F7F7Fu};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int m = (FEW ? 0 : w.m0 + half) + lane + 32 * j;
          a[j] = 0x7F7F7F7Fu;    // rows past the end hold zero codes; their factor is one
          if (m < p.M) a[j] = ld_global_u32(p.sa + static_cast<int64_t>(m) * p.sa_pitch + 4 * g);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (ob + h >= p.out_blocks) continue;
          if (!DX) {
            b[h] = ld_global_u32(p.sw + static_cast<int64_t>(ob + h) * p.sw_pitch + 4 * g);
          } else {
            uint32_t x = 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (4 * g + j < p.kb_main)
                x |= ld_global_u8(p.sw + static_cast<int64_t>(4 * g + j) * p.sw_pitch + ob + h) << (8 * j);
            b[h] = x;
          }
        }
        if (!__all_sync(0xffffffffu, wait_bar(&sf_empty[slot], ph ^ 1u, wt) ? 1 : 0)) { ok = false; break; }
        tc_fence_after();
        const uint32_t dst = tq + slot * 16;
        if (FEW) {
          const uint32_t f = rank ? b[1] : b[0];          // of this CTA's 128 weight rows
          tmem_st_32x32b_x4(dst, f, f, f, f);
          tmem_st_32x32b_x4(dst + 4, a[0], a[1], a[2], a[3]);
        } else {
          tmem_st_32x32b_x4(dst, a[0], a[1], a[2], a[3]);
          tmem_st_32x32b_x4(dst + 4, b[0], b[0], b[0], b[0]);
          tmem_st_32x32b_x4(dst + 8, b[1], b[1], b[1], b[1]);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(&sf_full[slot], 0u);
        if (++slot == kFgSfSlots) { slot = 0; ph ^= 1u; }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // neither CTA leaves while the other may still arrive on its barriers
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kFgTmemCols);
  }
}

// Y = bf16(sum of the splits' fp32 partials, in order).  total is a multiple of 4.
__global__ void __launch_bounds__(256) fp8_reduce_kernel(const float *part, int splits, int64_t total,
                                                         uint16_t *out) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  pdl_trigger();
  pdl_wait();
  if (i >= total) return;
  // two parts' loads before their adds: one at a time takes 0.3 us more of 8 (9 tokens, 4096 x 4096);
  // eight need registers past 32, and its CTAs no longer start beside the GEMM's (128 tokens of
  // 22016 x 8192: 46 us, 44)
  const float *src = part + i;
  float4 v = ld_global_f4(src);
  int s = 1;
#pragma unroll 1
  for (; s + 1 < splits; s += 2) {
    const float4 f = ld_global_f4(src + s * total), g = ld_global_f4(src + (s + 1) * total);
    v.x += f.x; v.y += f.y; v.z += f.z; v.w += f.w;
    v.x += g.x; v.y += g.y; v.z += g.z; v.w += g.w;
  }
  if (s < splits) {
    const float4 f = ld_global_f4(src + s * total);
    v.x += f.x; v.y += f.y; v.z += f.z; v.w += f.w;
  }
  *reinterpret_cast<uint2 *>(out + i) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

}  // namespace qlora
