// Rank-r products of the adapter around the 8-bit operators (sm_100a):
//   projections   XA = deq(X8) A,  G = dY B^T (and, in the same pass, dY quantized)
//   gradients     dA = deq(X8)^T (sG),  dB^T = dY^T (sXA)
// Each is D[rows, r] = Act[rows, c] Q[c, r], a tall-skinny product bound by reading the
// activation once: 1 byte per value for X8, 2 for dY (3 with its codes written).
//
// One CTA owns 128 output rows and one split of the contraction; the splits of a row tile
// form a cluster (at most 16) that adds its partial tiles in rank order through
// distributed shared memory.  Stages are 64 contraction values, in pairs of 128:
//   warps 0, 3  TMA: 0 the Q tile of each stage, and a bf16 activation, into the operand ring;
//               3 the 8-bit codes, 128 x 128 per pair, into a raw ring.
//   warp 1      MMA issuer (tcgen05 kind::f16, M = 128).
//   warp 2      8-bit activations: the factors of each raw tile's 128 rows, into shared memory.
//               Their bytes lie a row pitch apart in HBM, so every lane's load is a sector of
//               its own; loaded by each worker thread they took more of the load pipe than
//               the codes.
//   warps 4..11 drain: every four stages the partial sums leave TMEM and are added to fp32
//               registers, two TMEM buffers in turn.  The tensor core's fp32 accumulation
//               truncates, which biases a chain of n MMAs by about (2/3) n 2^-24 of its
//               sum: 1.2e-5 measured on dA over 8192 tokens in one chain, 4e-7 for the 16
//               MMAs of four stages; the adds between chains round to nearest.
//   warps 12..27 workers, four groups of four:
//               8-bit activations: two groups turn a raw tile into its two operand stages, the
//               other two the next, a thread 64 codes of a row: bf16 (exact), scaled by the
//               row's power of two, dropped-out elements zeroed;
//               G with QUANT: two groups take a pair, the other two the next, two lanes a row,
//               whose 128 values are one block: amax, factor byte and codes.
// Stages of 64 rather than 128 halve what a slot holds (G 18 to 24 KB, XA 24, gradients 24 to 40): a slot's Q load, conversion
// and MMAs follow one another, so the number of slots sets how much of that latency is
// hidden.
// The activation is the MMA's A operand: K-major for projections (128 rows of 64 values),
// MN-major for gradients (two groups of 64 features, 64 tokens each).  Q is K-major
// (B [r, N], for G) or MN-major: A [K, r], or for the gradients the fp32 factor sG / sXA as three
// bf16 terms side by side [M, 3 w], whose sum carries all 24 bits; the drain adds the
// three column ranges.  A launch computes up to 64 columns (32 sums per drain thread);
// wider adapters take two.
// Measured (8192 x 8192, r 64, events around each launch): XA 38 us, dA 45 (67 MB each: the path of a
// stage through conversion, MMAs and barriers, about 1500 cycles for 128 values of the 700 that HBM
// allows), G with the quantization 43 (201 MB, 4.6 TB/s), dB 38 (134 MB, 3.5 TB/s).  Start, cluster skew
// and reduction are 7 to 11 us of each, and the clusters of few row tiles leave SMs idle: 64 row
// tiles in two parts are 128 CTAs for 148 SMs, dB of 11008 columns 86.  r 128 takes two launches
// of each: forward 440 us (402 at r 64), backward 577 (468).
// Ring slots of two stages, for one wait and commit per 128 values, changed nothing.
#pragma once
#include "common.cuh"
#include "fp8_quant.cuh"
#include "pipeline.cuh"

namespace qlora {

constexpr int kAmWorkers = 16;                    // worker warps
constexpr int kAmThreads = 32 * (12 + kAmWorkers);
constexpr int kAmPass = 64;                       // columns of the result one launch computes at most
constexpr int kAmRows = 128;
constexpr int kAmRawBytes = 128 * 128;            // codes of one pair of stages
constexpr int kAmOpBytes = kAmRows * 128;         // bf16 operand tile of one stage
constexpr int kAmMaxOp = 8, kAmMaxRaw = 4;        // ring limits
static_assert(kAmMaxRaw % 2 == 0, "a raw slot belongs to one team of workers");
constexpr int kAmChain = 4;                       // stages accumulated in TMEM between two drains
constexpr int kAmSmemMax = 227 * 1024;
constexpr int kAmClusterMax = 16;                 // splits of a row tile; more than 8 is opt-in

enum AmAct : int { kActBf16 = 0, kActE4M3 = 1, kActE5M2 = 2 };
enum AmQuant : int { kQuantNone = 0, kQuantE4M3 = 1, kQuantE5M2 = 2 };

struct AdapterParams {
  int rows;               // output rows: tokens (projection) or features (gradient)
  int tokens;             // M
  int pairs_total, pairs_per_split, splits;   // in pairs of stages (128 contraction values)
  int n_op, n_raw;        // ring slots (n_op = 8 under QUANT: see the workers)
  int n;                  // MMA N, a multiple of 16
  uint32_t tmem_cols;     // two buffers of n columns
  int q_kmajor;           // Q box of a stage: 1: {64 c, r16 rows}; 0: {64 columns, 64 c} per 64-column group
  int q_bytes;
  int r, r16;             // columns of the result in this pass, and rounded up to 16
  int j0, ld;             // first column of this pass, and the columns of all passes (the rank)
  float s, out_scale;
  // 8-bit activation
  const uint8_t *scales;
  int64_t pitch;
  const uint8_t *keep;    // bit-packed keep mask of the activation [M, act_cols], or null
  int64_t act_cols;
  // QUANT (codes of the call's workspace, on a 256-byte address; rows of a multiple of 128)
  uint8_t *q_codes, *q_scales;
  int64_t q_pitch;
  // projection, each may be null: fp32 [rows, ld]; bf16 hi|lo of s*value [rows, 2 half]
  // (columns >= ld of a half zero); three terms of s*value for the gradients (see am_store_terms)
  float *out;
  uint16_t *hl;
  int half;
  uint16_t *terms;
  const float *split_in;  // a second fp32 [rows, ld], and its three terms of s*value
  uint16_t *split_terms;
  unsigned int *zero;     // words a later kernel of the call expects to find zero
  int zero_n;
  int late_wait;          // nothing of the kernel before is needed: wait for it at the end
  // gradient: 0 out[row][j0 + j] of row length ld, 1 out[j0 + j][row]
  int layout, accumulate;
  uint64_t limit_ns;
};

// Row pitch (floats) of the partial tile: whole 16-byte groups, and 4 mod 32 banks at most
// widths, so that eight rows' groups fall on distinct banks.
constexpr __host__ __device__ int am_pitch(int r16) { return r16 + 4; }
constexpr int am_smem_bytes(int n_op, int n_raw, int q_bytes) {
  return 1024 + n_op * (kAmOpBytes + q_bytes) + n_raw * (kAmRawBytes + 256) + 512;
}
static_assert(am_smem_bytes(4, 4, 3 * 8192) <= kAmSmemMax && am_smem_bytes(8, 0, kAmPass * 128) <= kAmSmemMax,
              "the smallest rings of the widest products must fit");

// The three bf16 terms of s*v for four values: each the rounding of what the ones before
// left over, so their sum is s*v to 2^-25.
QDEV void am_split4(const float (&v)[4], float s, uint2 (&t)[3]) {
  float rest[4] = {s * v[0], s * v[1], s * v[2], s * v[3]};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    t[k].x = pack_bf16x2(rest[0], rest[1]);
    t[k].y = pack_bf16x2(rest[2], rest[3]);
    rest[0] -= bf16_lo(t[k].x); rest[1] -= bf16_hi(t[k].x);
    rest[2] -= bf16_lo(t[k].y); rest[3] -= bf16_hi(t[k].y);
  }
}
// Columns j .. j+3 of a row of the terms of a pass: [M, 3 w], one term after the other in a
// row, columns past the rank zero; the block of pass i follows those of the passes before.
QDEV void am_store_terms(uint16_t *dst, int64_t M, int64_t row, int j, int j0, int w, const uint2 (&t)[3]) {
  uint16_t *d = dst + M * 3 * j0 + row * 3 * w + j;
#pragma unroll
  for (int k = 0; k < 3; ++k) *reinterpret_cast<uint2 *>(d + k * w) = t[k];
}
QDEV float4 ld_dsmem_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// Four codes -> two bf16x2 words before the factor: the code's exponent and mantissa
// moved under bf16's, which scales the value by 2^-120 (e4m3) or 2^-112 (e5m2), exactly,
// format subnormals included.
template <int ACT>
QDEV void am_spread4(uint32_t w, uint32_t &a, uint32_t &b) {
  const uint32_t x = prmt(w, 0u, 0x1404u), y = prmt(w, 0u, 0x3424u);
  if (ACT == kActE5M2) {
    a = (x & 0x80008000u) | ((x >> 3) & 0x0FE00FE0u);
    b = (y & 0x80008000u) | ((y >> 3) & 0x0FE00FE0u);
  } else {
    a = (x & 0x80008000u) | ((x >> 4) & 0x07F007F0u);
    b = (y & 0x80008000u) | ((y >> 4) & 0x07F007F0u);
  }
}
// The factor that goes with am_spread4 for an exponent byte, 2^(byte - 127 + 120 or 112), as
// bf16 bits.  Beyond 2^127 (byte > 134 or 142) the sign bit is set and the bits hold what is
// left after a first factor of 2^127; byte 255 gives NaN.
constexpr uint32_t kAm2To127 = 0x7F007F00u;
template <int ACT>
QDEV uint16_t am_factor(uint32_t byte) {
  const uint32_t field = byte + (ACT == kActE5M2 ? 112u : 120u);
  if (byte == 255u) return 0x7FC0u;
  return static_cast<uint16_t>(field <= 254u ? field << 7 : 0x8000u | ((field - 254u + 127u) << 7));
}
QDEV uint32_t mul_bf16x2(uint32_t a, uint32_t f) {
  const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                   *reinterpret_cast<const __nv_bfloat162 *>(&f));
  return *reinterpret_cast<const uint32_t *>(&p);
}
// (p on a 32-byte address)
QDEV void st_global_v8(void *p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
QDEV void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr));
}

// A producer's end: every copy it issued has landed before the block's shared memory is
// reused or given up (bounded): the last use of each ring slot.  After a wait that ran out,
// copies may be in flight whose phases never complete; they land in microseconds.
QDEV void am_copies_landed(uint64_t *full, int slots, int uses, bool ok, const Waiter &w) {
  if (ok) {
    for (int i = max(0, uses - slots); i < uses; ++i) wait_bar(&full[i % slots], static_cast<uint32_t>((i / slots) & 1), w);
  } else {
    for (int i = 0; i < 200; ++i) __nanosleep(1000);
  }
}
QDEV void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Barrier of the drain and worker warps.
QDEV void am_rings_idle() { asm volatile("bar.sync 1, 768;" ::: "memory"); }

template <int ACT, bool GRAD, int QUANT>
__global__ void __launch_bounds__(kAmThreads, 1)
    adapter_mma_kernel(const __grid_constant__ CUtensorMap tm_act, const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ AdapterParams p) {
  constexpr bool F8 = ACT != kActBf16;
  static_assert(!QUANT || (!F8 && !GRAD), "only a bf16 projection quantizes its activation");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int op_stage = kAmOpBytes + p.q_bytes;
  uint8_t *sRaw = smem + p.n_op * op_stage;
  uint16_t *sFac = reinterpret_cast<uint16_t *>(sRaw + p.n_raw * kAmRawBytes);   // [n_raw][128] factors
  uint64_t *op_full = reinterpret_cast<uint64_t *>(sFac + p.n_raw * 128);
  uint64_t *op_empty = op_full + kAmMaxOp;
  uint64_t *raw_full = op_empty + kAmMaxOp;
  uint64_t *raw_empty = raw_full + kAmMaxRaw;
  uint64_t *acc_full = raw_empty + kAmMaxRaw;
  uint64_t *acc_empty = acc_full + 2;
  uint64_t *drain = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row0 = static_cast<int>(blockIdx.x) * kAmRows;
  const int pr0 = static_cast<int>(blockIdx.y) * p.pairs_per_split;
  const int npr = max(0, min(p.pairs_total, pr0 + p.pairs_per_split) - pr0);
  const int nst = 2 * npr;
  if (tid == 0) {
    prefetch_tmap(&tm_act);
    prefetch_tmap(&tm_q);
    for (int i = 0; i < kAmMaxOp; ++i) {
      mbar_init(&op_full[i], F8 ? 5 : 1);        // the TMA's arrival, and four worker warps
      mbar_init(&op_empty[i], QUANT ? 9 : 1);    // the MMAs' commit, and eight worker warps
    }
    for (int i = 0; i < kAmMaxRaw; ++i) { mbar_init(&raw_full[i], 2); mbar_init(&raw_empty[i], 8); }
    for (int i = 0; i < 2; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], 8); }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!p.late_wait) pdl_wait();
  pdl_trigger();
  if (p.zero && blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = tid; i < p.zero_n; i += kAmThreads) p.zero[i] = 0u;
  const uint32_t tmem_base = *tmem_slot;
  const Waiter wt{abort_flag, p.limit_ns};
  volatile int no_abort = 0;
  const Waiter final_wt{&no_abort, drain_limit_ns(p.limit_ns)};

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer: operand ring
    if (lane == 0) {
      const uint32_t bytes = static_cast<uint32_t>((F8 ? 0 : kAmOpBytes) + p.q_bytes);
      bool ok = true;
      int s = 0;
      uint32_t ph = 1;
      for (int i = 0, c = 128 * pr0; i < nst; ++i, c += 64) {
        if (!wait_bar(&op_empty[s], ph, wt)) { ok = false; break; }   // the slots' first use passes at once
        if (QUANT) fence_proxy_async_smem();   // the quantizers read the slot through the generic proxy
        uint8_t *op = smem + s * op_stage, *sq = op + kAmOpBytes;
        mbar_arrive_expect_tx(&op_full[s], bytes);
        if (!F8) {
          if (GRAD) tma_load_3d(op, &tm_act, &op_full[s], 0, c, row0 >> 6);
          else tma_load_2d(op, &tm_act, &op_full[s], c, row0);
        }
        if (GRAD) tma_load_3d(sq, &tm_q, &op_full[s], 0, c, 0);
        else if (p.q_kmajor) tma_load_2d(sq, &tm_q, &op_full[s], c, 0);
        else tma_load_2d(sq, &tm_q, &op_full[s], 0, c);
        if (++s == p.n_op) { s = 0; ph ^= 1u; }
      }
      am_copies_landed(op_full, p.n_op, nst, ok, final_wt);
    }
  } else if (warp == 3 && F8) {
    // ------------------------------------------------------------ TMA producer: raw codes
    if (lane == 0) {
      bool ok = true;
      int s = 0;
      uint32_t ph = 1;
      for (int i = 0, c = 128 * pr0; i < npr; ++i, c += 128) {
        if (!wait_bar(&raw_empty[s], ph, wt)) { ok = false; break; }
        // the slot's codes were read through the generic proxy, the TMA rewrites them
        // through the async proxy: order the two
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(&raw_full[s], kAmRawBytes);
        if (GRAD) tma_load_2d(sRaw + s * kAmRawBytes, &tm_act, &raw_full[s], row0, c);
        else tma_load_2d(sRaw + s * kAmRawBytes, &tm_act, &raw_full[s], c, row0);
        if (++s == p.n_raw) { s = 0; ph ^= 1u; }
      }
      am_copies_landed(raw_full, p.n_raw, npr, ok, final_wt);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // (lean: the descriptors of slot 0 are built once, a slot adds its offset)
    const bool el = elect_one();
    const uint32_t idesc = make_idesc_bf16(kAmRows, p.n, GRAD, !p.q_kmajor);
    const uint32_t a0 = smem_u32(smem), q0 = a0 + kAmOpBytes;
    const uint64_t ad0 = GRAD ? sw128_desc(a0, kAmOpBytes / 2, 1024) : sw128_desc(a0, 16, 1024);
    const uint64_t bd0 = p.q_kmajor ? sw128_desc(q0, 16, 1024) : sw128_desc(q0, 8192, 1024);
    constexpr uint32_t a_step = GRAD ? (2048u >> 4) : (32u >> 4);
    const uint32_t b_step = p.q_kmajor ? (32u >> 4) : (2048u >> 4);
    const uint64_t slot_step = static_cast<uint64_t>(op_stage >> 4);
    const uint32_t d1 = static_cast<uint32_t>(p.n);
    uint64_t ad = ad0, bd = bd0;
    int s = 0;
    uint32_t ph = 0;
    bool ready = false;   // this stage's tile was seen complete while the last one was issued
    bool issued = false;
    for (int i = 0; i < nst; ++i) {
      const bool first = (i & (kAmChain - 1)) == 0;
      const bool last = (i & (kAmChain - 1)) == kAmChain - 1 || i + 1 == nst;
      const int ch = i / kAmChain, b = ch & 1;
      if (first && !wait_bar_warp(&acc_empty[b], static_cast<uint32_t>((ch >> 1) & 1) ^ 1u, wt)) break;
      if (!ready && !wait_bar_warp(&op_full[s], ph, wt)) break;
      tc_fence_after();
      const bool wrap = s + 1 == p.n_op;
      const uint32_t peek = mbar_test(&op_full[wrap ? 0 : s + 1], wrap ? ph ^ 1u : ph) ? 1u : 0u;
      if (el) {
        const uint32_t d = tmem_base + (b ? d1 : 0u);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_bf16_ss(d, ad + k * a_step, bd + k * b_step, idesc, (!first || k) ? 1u : 0u);
        mma_commit(&op_empty[s]);
        if (last) mma_commit(&acc_full[b]);
      }
      ad += slot_step;
      bd += slot_step;
      issued = true;
      ready = __all_sync(0xffffffffu, peek) != 0;
      if (++s == p.n_op) { s = 0; ph ^= 1u; ad = ad0; bd = bd0; }
    }
    // every MMA issued has completed before the block gives up its shared memory and TMEM
    // (bounded); unless a wait ran out, the last drain has seen the same
    if (issued) {
      if (el) mma_commit(drain);
      wait_bar_warp(drain, 0, final_wt);
    }
    __syncwarp();
  } else if (warp == 2 && F8) {
    // ------------------------------------------------------------ factors
    // Row rr of pair i's tile: token row0 + rr, block pr0 + i (projection), or token
    // 128 (pr0 + i) + rr, block row0 / 128 (gradient).  Rows past the end hold zero codes:
    // their factor is one.  A pair's bytes are requested before the last pair's are stored.
    auto load = [&](int i, uint32_t (&b)[4]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t m = (GRAD ? static_cast<int64_t>(pr0 + i) * 128 : row0) + lane + 32 * j;
        const int64_t blk = GRAD ? (row0 >> 7) : pr0 + i;
        b[j] = (i < npr && m < p.tokens) ? ld_global_u8(p.scales + m * p.pitch + blk) : 127u;
      }
    };
    uint32_t cur[4], nxt[4];
    load(0, cur);
    int rs = 0;
    uint32_t ph = 1;
    for (int i = 0; i < npr; ++i) {
      load(i + 1, nxt);
      if (!wait_bar_warp(&raw_empty[rs], ph, wt)) break;     // the slots' first use passes at once
#pragma unroll
      for (int j = 0; j < 4; ++j) { sFac[rs * 128 + lane + 32 * j] = am_factor<ACT>(cur[j]); cur[j] = nxt[j]; }
      __syncwarp();
      if (lane == 0) mbar_arrive(&raw_full[rs]);
      if (++rs == p.n_raw) { rs = 0; ph ^= 1u; }
    }
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------ drain
    const int h = (warp - 4) >> 2, q = warp & 3;
    const int cols = p.r16 / 2;               // columns of this warp, a multiple of 8
    float acc[kAmPass / 2];                   // [h cols, (h + 1) cols) of this thread's row
#pragma unroll
    for (int i = 0; i < kAmPass / 2; ++i) acc[i] = 0.f;
    const int chains = (nst + kAmChain - 1) / kAmChain;
    for (int i = 0; i < chains; ++i) {
      const int b = i & 1;
      if (!wait_bar_warp(&acc_full[b], static_cast<uint32_t>((i >> 1) & 1), wt)) break;
      tc_fence_after();
      const uint32_t t = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(b * p.n + h * cols);
#pragma unroll
      for (int c = 0; c < kAmPass / 16; ++c) {
        if (c * 8 < cols) {
          uint32_t v[8];
          tmem_ld_32x32b_x8(t + c * 8, v);
          if (GRAD) {
            uint32_t u[8], z[8];
            tmem_ld_32x32b_x8(t + p.r16 + c * 8, u);
            tmem_ld_32x32b_x8(t + 2 * p.r16 + c * 8, z);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              acc[c * 8 + j] += __uint_as_float(v[j]) + (__uint_as_float(u[j]) + __uint_as_float(z[j]));
          } else {
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[c * 8 + j] += __uint_as_float(v[j]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[b]);
    }
    // the rings become the partial tile: every MMA (so every copy it read) is done, and the
    // workers have left the rings
    if (F8 || QUANT) am_rings_idle();
    float *dst = reinterpret_cast<float *>(smem) + (q * 32 + lane) * am_pitch(p.r16) + h * cols;
#pragma unroll
    for (int c = 0; c < kAmPass / 8; ++c)
      if (c * 4 < cols)
        *reinterpret_cast<float4 *>(dst + c * 4) = make_float4(acc[c * 4], acc[c * 4 + 1], acc[c * 4 + 2], acc[c * 4 + 3]);
  } else if (warp >= 12 && (F8 || QUANT)) {
    // ------------------------------------------------------------ workers
    const int g = (warp - 12) >> 2;
    const int t = (tid - 12 * 32) & 127;
    if (F8) {
      // Two teams of two groups take alternate pairs (n_raw is even, so a raw slot belongs to
      // one team); within a team group g writes stage 2 i2 + (g mod 2) of pair i2, from columns
      // 64 (g mod 2) .. of the raw tile (projection, thread t = row t) or tokens 64 (g mod 2) ..
      // (gradient, thread t = token t mod 64 of them, features 64 (t / 64) ..), 64 codes
      // each.  A group's stage i - 4 saw the MMAs of stage i - 4 - n_op done, and the MMAs run in
      // order, so those of stage i - 2 n_op are done (n_op >= 4): the parity wait below cannot
      // see a phase two behind.
      const int team = g >> 1, sub = g & 1;
      const int srow = GRAD ? 64 * sub + (t & 63) : t;
      const int shalf = GRAD ? t >> 6 : sub;
      const int drow = GRAD ? (t & 63) : t;
      const uint32_t sswz = static_cast<uint32_t>(srow & 7), dswz = static_cast<uint32_t>(drow & 7);
      const uint32_t src0 = smem_u32(sRaw) + static_cast<uint32_t>(srow * 128);
      const uint32_t dst0 = smem_u32(smem) + static_cast<uint32_t>((GRAD ? (t >> 6) * (kAmOpBytes / 2) : 0) + drow * 128);
      // the keep bits of this thread's codes, and the step from one of its pairs to the next
      const int64_t m0 = (GRAD ? static_cast<int64_t>(pr0 + team) * 128 : row0) + srow;
      int64_t m_left = p.keep ? p.tokens - m0 : 0;
      const int m_step = GRAD ? 256 : 0;
      const uint8_t *kp = p.keep + ((m0 * p.act_cols + static_cast<int64_t>(GRAD ? (row0 >> 7) : pr0 + team) * 128 + 64 * shalf) >> 3);
      const int64_t kp_step = GRAD ? 32 * p.act_cols : 32;
      auto keep_now = [&]() -> uint2 {
        return m_left > 0 ? ld_global_v2(kp) : make_uint2(~0u, ~0u);
      };
      uint2 kb = team < npr ? keep_now() : make_uint2(~0u, ~0u);
      int rs = team, s = 2 * team + sub;
      uint32_t rph = 0, oph = 1;
      while (s >= p.n_op) { s -= p.n_op; oph ^= 1u; }
      for (int i2 = team; i2 < npr; i2 += 2) {
        m_left -= m_step;
        kp += kp_step;
        const uint2 next_kb = i2 + 2 < npr ? keep_now() : make_uint2(~0u, ~0u);
        if (!wait_bar_warp(&raw_full[rs], rph, wt)) break;
        const uint32_t src = src0 + static_cast<uint32_t>(rs * kAmRawBytes);
        uint32_t f = sFac[rs * 128 + srow];
        uint4 w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = ld_shared_v4(src + ((static_cast<uint32_t>(4 * shalf + c) ^ sswz) << 4));
        // the codes are in registers: their slot is free once every warp has read its part
        __syncwarp();
        if (lane == 0) mbar_arrive(&raw_empty[rs]);
        const bool two = (f & 0x8000u) != 0u;
        f = (f & 0x7FFFu) * 0x10001u;
        if (!wait_bar_warp(&op_empty[s], oph, wt)) break;      // the slots' first use passes at once
        const uint32_t dst = dst0 + static_cast<uint32_t>(s * op_stage);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t in[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) am_spread4<ACT>(in[j], o[2 * j], o[2 * j + 1]);
          if (two) {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = mul_bf16x2(o[j], kAm2To127);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = mul_bf16x2(o[j], f);
          if (p.keep) {
            const uint32_t bits = (c < 2 ? kb.x : kb.y) >> (16 * (c & 1));
#pragma unroll
            for (int j = 0; j < 8; ++j)
              o[j] &= (((bits >> (2 * j)) & 1u) ? 0x0000FFFFu : 0u) | (((bits >> (2 * j + 1)) & 1u) ? 0xFFFF0000u : 0u);
          }
          st_shared_v4(dst + ((static_cast<uint32_t>(2 * c) ^ dswz) << 4), o[0], o[1], o[2], o[3]);
          st_shared_v4(dst + ((static_cast<uint32_t>(2 * c + 1) ^ dswz) << 4), o[4], o[5], o[6], o[7]);
        }
        kb = next_kb;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&op_full[s]);
        rs += 2;
        if (rs >= p.n_raw) { rs -= p.n_raw; rph ^= 1u; }
        s += 4;
        while (s >= p.n_op) { s -= p.n_op; oph ^= 1u; }
      }
    } else {
      // Two teams of two groups take alternate pairs.  With 8 slots a slot belongs to one team,
      // which has consumed its previous use: a parity wait cannot see a phase two behind.  Two
      // neighbouring lanes share a row: lane h holds the 64 values of the pair's stage h, read
      // once, in an order (16-byte pieces c ^ 4 h) that keeps the eight lanes of a shared-memory
      // phase on eight columns of the swizzle.  (A thread for each whole row read it twice from
      // shared memory, whose pipe was the bound: G of 8192 x 8192, r 64, took 66 us, now 52.)
      const int team = g >> 1, h = t & 1, lr = (((g & 1) << 7) | t) >> 1;
      const int64_t row = row0 + lr;
      const uint32_t swz = static_cast<uint32_t>(lr & 7) ^ static_cast<uint32_t>(h << 2);
      const uint32_t src0 = smem_u32(smem) + static_cast<uint32_t>(h * op_stage + lr * 128);
      uint8_t *dst0 = p.q_codes + row * p.act_cols + static_cast<int64_t>(pr0) * 128 + h * 64;
      bool bad = false;
      int s = 2 * team;
      uint32_t par = 0;
      for (int i2 = team; i2 < npr; i2 += 2) {
        if (!wait_bar_warp(&op_full[s], par, wt) || !wait_bar_warp(&op_full[s + 1], par, wt)) break;
        const uint32_t src = src0 + static_cast<uint32_t>(s * op_stage);
        uint4 v[8];
        uint32_t m = 0u;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          v[c] = ld_shared_v4(src + ((static_cast<uint32_t>(c) ^ swz) << 4));
          m = f8_amax8(m, v[c]);
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&op_empty[s]);
          mbar_arrive(&op_empty[s + 1]);
        }
        m = max(m & 0xFFFFu, m >> 16);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const bool nan = m >= 0x7F80u;
        const uint32_t byte = nan ? kF8NanScale : f8_exp_byte<QUANT == kQuantE5M2>(m);
        const float inv = f8_inv_scale(nan ? 127u : byte);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint2 x = f8_encode8<QUANT == kQuantE5M2>(v[4 * k + e], inv);
            o[2 * e] = nan ? kF8NanCodes : x.x;
            o[2 * e + 1] = nan ? kF8NanCodes : x.y;
          }
          if (row < p.rows) st_global_v8(dst0 + static_cast<int64_t>(i2) * 128 + ((k ^ h) << 5), o);
        }
        if (row < p.rows) {
          if (h == 0) p.q_scales[row * p.q_pitch + pr0 + i2] = static_cast<uint8_t>(byte);
          bad = bad || nan;
        }
        s += 4;
        if (s >= kAmMaxOp) { s -= kAmMaxOp; par ^= 1u; }
      }
      if (bad) atomicOr(&g_device_status, kStatNonFinite);
    }
    am_rings_idle();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }

  // ---- cluster reduction: rank q finishes rows [q R, (q+1) R) of the tile, four columns
  // of a row at a time (one row of out[j][row] is written by neighbouring threads)
  cluster_sync_all();
  {
    const int rank = static_cast<int>(cluster_ctarank());
    const int R = (kAmRows + p.splits - 1) / p.splits;
    const int r0 = rank * R, nr = max(0, min(kAmRows, r0 + R) - r0);
    const uint32_t base = smem_u32(smem);
    const int quads = p.r16 >> 2, pitch = am_pitch(p.r16);
    for (int i = tid; i < nr * quads; i += kAmThreads) {
      int rr, j;
      if (GRAD && p.layout == 1) { j = i / nr; rr = i - j * nr; }
      else { rr = i / quads; j = i - rr * quads; }
      j *= 4;
      const int row = row0 + r0 + rr;
      if (row >= p.rows) continue;
      const uint32_t a = base + 4u * static_cast<uint32_t>((r0 + rr) * pitch + j);
      // the sum runs in rank order; eight ranks' loads are issued before they are added
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      for (int q0 = 0; q0 < p.splits; q0 += 8) {
        float4 pa[8];
#pragma unroll
        for (int qq = 0; qq < 8; ++qq)
          if (q0 + qq < p.splits) pa[qq] = ld_dsmem_v4(map_rank(a, static_cast<uint32_t>(q0 + qq)));
#pragma unroll
        for (int qq = 0; qq < 8; ++qq)
          if (q0 + qq < p.splits) { v[0] += pa[qq].x; v[1] += pa[qq].y; v[2] += pa[qq].z; v[3] += pa[qq].w; }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = j + e < p.r ? __fmul_rn(v[e], p.out_scale) : 0.f;
      if (GRAD) {
        // r is a multiple of 8, so a group of four is whole or absent
        if (j >= p.r) continue;
        if (p.layout == 0) {
          float4 *o = reinterpret_cast<float4 *>(p.out + static_cast<int64_t>(row) * p.ld + p.j0 + j);
          if (p.accumulate) {
            const float4 old = *o;
            v[0] = __fadd_rn(old.x, v[0]); v[1] = __fadd_rn(old.y, v[1]);
            v[2] = __fadd_rn(old.z, v[2]); v[3] = __fadd_rn(old.w, v[3]);
          }
          *o = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float *o = p.out + static_cast<int64_t>(p.j0 + j + e) * p.rows + row;
            *o = p.accumulate ? __fadd_rn(*o, v[e]) : v[e];
          }
        }
      } else {
        if (p.out && j < p.r)
          *reinterpret_cast<float4 *>(p.out + static_cast<int64_t>(row) * p.ld + p.j0 + j) =
              make_float4(v[0], v[1], v[2], v[3]);
        const bool in_half = p.hl && p.j0 + j < p.half;
        if (p.terms || in_half) {
          uint2 t[3];
          am_split4(v, p.s, t);
          if (in_half) {
            uint16_t *h = p.hl + static_cast<int64_t>(row) * 2 * p.half + p.j0 + j;
            *reinterpret_cast<uint2 *>(h) = t[0];
            *reinterpret_cast<uint2 *>(h + p.half) = t[1];
          }
          if (p.terms) am_store_terms(p.terms, p.rows, row, j, p.j0, p.r16, t);
        }
        if (p.split_terms) {
          float x[4] = {0.f, 0.f, 0.f, 0.f};
          if (j < p.r) {
            const float4 f = ld_global_f4(p.split_in + static_cast<int64_t>(row) * p.ld + p.j0 + j);
            x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
          }
          uint2 t[3];
          am_split4(x, p.s, t);
          am_store_terms(p.split_terms, p.rows, row, j, p.j0, p.r16, t);
        }
      }
    }
  }
  if (p.late_wait && tid == 0) pdl_wait();
  __syncwarp();
  cluster_sync_all();   // no CTA leaves while a peer may still read its partial tile
}

}  // namespace qlora
