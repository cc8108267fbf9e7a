// Host side of the 8-bit operators: argument checks, workspace plans, launches and the
// C ABI entry points.  Part of the translation unit of qlora_nf4.cu, whose helpers
// (device_info, make_map_2d, Workspace, LaunchTimer, the rank-r launches) it uses.
#pragma once

namespace {

// ------------------------------------------------------------------ checks
qlora_status check_fp8(const qlora_fp8_t *t, int block_rows) {
  if (!t || !t->codes || !t->scales) return QLORA_ERR_INVALID_ARG;
  if (t->rows <= 0 || t->cols <= 0) return QLORA_ERR_INVALID_ARG;
  if (t->block_rows != 1 && t->block_rows != kF8Block) return QLORA_ERR_INVALID_ARG;
  if (block_rows != 0 && t->block_rows != block_rows) return QLORA_ERR_INVALID_ARG;
  if (t->fmt != QLORA_FP8_E4M3 && (t->fmt != QLORA_FP8_E5M2 || t->block_rows != 1)) return QLORA_ERR_INVALID_ARG;
  if (!aligned16(t->codes) || !aligned16(t->scales)) return QLORA_ERR_MISALIGNED;
  if ((t->cols % 8) != 0 || t->rows > (1ll << 30) || t->cols > (1ll << 30)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  // the streaming kernels count blocks in 32 bits
  if (t->rows * ((t->cols + kF8Block - 1) / kF8Block) >= (1ll << 31)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  return QLORA_OK;
}

// r = 0 (A and B null): no adapter.
qlora_status check_fp8_layer(int64_t M, const qlora_fp8_t *W, const uint16_t *A, const uint16_t *B, int r, float s) {
  const qlora_status st = check_fp8(W, kF8Block);
  if (st != QLORA_OK) return st;
  if (M < 1 || M > (1ll << 30)) return QLORA_ERR_INVALID_ARG;
  if (r != 0 && (r < 8 || r > 128 || (r % 8) != 0)) return QLORA_ERR_INVALID_ARG;
  if (r ? (!A || !B) : (A || B)) return QLORA_ERR_INVALID_ARG;
  if (!(s == s)) return QLORA_ERR_INVALID_ARG;
  if (W->rows % 128 != 0 || W->cols % 128 != 0) return QLORA_ERR_UNSUPPORTED_SHAPE;
  if (W->rows > (1ll << 24) || W->cols > (1ll << 24)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  return QLORA_OK;
}

// ------------------------------------------------------------------ launches
// Launch of a kernel that calls pdl_wait before it touches global memory, as a programmatic
// dependent of what is before it in the stream; cluster_x * cluster_y > 1: clusters.
template <typename K, typename... Args>
qlora_status launch_pdl(K kernel, dim3 grid, int threads, int smem, int cluster_x, int cluster_y, cudaStream_t st,
                        const Args &...args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster_x);
  attr[1].val.clusterDim.y = static_cast<unsigned>(cluster_y);
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster_x * cluster_y > 1 ? 2 : 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, args...));
}

unsigned f8_grid(uint32_t blocks) {
  const uint32_t per = (kF8Threads / 8) * kF8Unroll;
  return (blocks + per - 1) / per;
}

qlora_status launch_fp8_quantize(const uint16_t *X, const qlora_fp8_t &t, cudaStream_t st) {
  const int kb = static_cast<int>((t.cols + kF8Block - 1) / kF8Block);
  const int pitch = static_cast<int>(f8_pitch(t.cols));
  LaunchTimer lt(QLORA_K_FP8_QUANTIZE, st);
  if (t.block_rows == kF8Block) {
    const int64_t grid = ((t.rows + kF8Block - 1) / kF8Block) * kb;
    fp8_quantize_weight_kernel<<<static_cast<unsigned>(grid), kF8Threads, 0, st>>>(
        X, static_cast<int>(t.rows), static_cast<int>(t.cols), pitch, t.codes, t.scales);
  } else {
    const Fp8QuantParams p{X, t.codes, t.scales, static_cast<int>(t.cols), kb, pitch,
                           static_cast<uint32_t>(t.rows * kb)};
    return t.fmt == QLORA_FP8_E5M2
               ? launch_pdl(fp8_quantize_kernel<true>, dim3(f8_grid(p.blocks)), kF8Threads, 0, 1, 1, st, p)
               : launch_pdl(fp8_quantize_kernel<false>, dim3(f8_grid(p.blocks)), kF8Threads, 0, 1, 1, st, p);
  }
  return cuda_status(cudaGetLastError());
}

qlora_status launch_fp8_dequant(const qlora_fp8_t &t, uint16_t *out, cudaStream_t st) {
  const int kb = static_cast<int>((t.cols + kF8Block - 1) / kF8Block);
  const Fp8DequantParams p{t.codes, t.scales, out, static_cast<int>(t.cols), kb,
                           static_cast<int>(f8_pitch(t.cols)), t.block_rows == 1 ? 0 : 7,
                           static_cast<uint32_t>(t.rows * kb)};
  LaunchTimer lt(QLORA_K_FP8_DEQUANT, st);
  if (t.fmt == QLORA_FP8_E5M2) fp8_dequant_kernel<true><<<f8_grid(p.blocks), kF8Threads, 0, st>>>(p);
  else fp8_dequant_kernel<false><<<f8_grid(p.blocks), kF8Threads, 0, st>>>(p);
  return cuda_status(cudaGetLastError());
}

// Parts of the contraction of one 8-bit GEMM: the 512-value groups are divided over more
// items, whose fp32 partials a second launch sums in order.
//   few (forward, M <= kFwTokens): HBM bounds the items, so the rounds are evened out: the least
//     of rounds times (groups of a part, and 0.75 for its start), in units of a group's 1.25 us,
//     plus 2 for the second launch and 13 MB of partials written and read per unit.  It takes
//     the best number of parts, or one 2% from it, in 30 cases (6 layers, 9 to 128 tokens); 9
//     tokens of 22016 x 8192, 86 tiles: 34 us in 4 parts, 43 undivided.
//   otherwise, with fewer than half as many tiles as CTA pairs, as many parts as the pairs
//     hold: the best in 38 of 42 such cases (to 1024 tokens), at most 8% from it in the others.
struct Fp8Plan {
  int splits = 1, groups_per_split = 0;
  size_t scratch_bytes = 0;
};
Fp8Plan fp8_plan(int64_t M, int64_t n_out, int64_t contraction, const GemmUnits &u, bool few) {
  Fp8Plan g;
  const int64_t groups = (contraction / 128 + 3) / 4;
  const int64_t tiles = ((M + kFgTile - 1) / kFgTile) * ((n_out + kFgTile - 1) / kFgTile);
  const int64_t pairs = u.pairs > 0 ? u.pairs : 1;
  int64_t per = groups;
  if (few) {
    int64_t best = -1;
    for (int64_t s = 1; s <= groups && s <= 32; ++s) {
      const int64_t p = (groups + s - 1) / s;
      const int64_t parts = (groups + p - 1) / p;
      if (parts != s) continue;
      const int64_t cost = ((tiles * s + pairs - 1) / pairs) * (4 * p + 3) + (s > 1 ? 8 + s * M * n_out * 8 / 3275000 : 0);
      if (best < 0 || cost < best) {
        best = cost;
        per = p;
      }
    }
  } else {
    int64_t s = tiles > 0 ? u.pairs / tiles : 1;
    if (s > groups) s = groups;
    if (s < 1) s = 1;
    per = (groups + s - 1) / s;
  }
  g.groups_per_split = static_cast<int>(per);
  g.splits = static_cast<int>((groups + per - 1) / per);   // no part is empty
  if (g.splits > 1) g.scratch_bytes = static_cast<size_t>(g.splits) * M * n_out * 4;
  return g;
}

// CTA pairs of the GEMM's launch.
int64_t fp8_units(const Fp8Plan &plan, int64_t M, int64_t n_out, const GemmUnits &u) {
  const int64_t items = ((M + kFgTile - 1) / kFgTile) * ((n_out + kFgTile - 1) / kFgTile) * plan.splits;
  return items < u.pairs ? items : u.pairs;
}

bool make_map_3d(CUtensorMap *m, CUtensorMapDataType dt, void *base, uint64_t inner, uint64_t mid, uint64_t outer,
                 uint64_t row_bytes, uint32_t box_inner, uint32_t box_mid) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {inner, mid, outer};
  cuuint64_t strides[2] = {row_bytes, row_bytes * mid};
  cuuint32_t box[3] = {box_inner, box_mid, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, dt, 3, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 [rows, ld] as {64 columns, rows, groups of 64 columns}: a box is box_rows rows of
// box_groups groups, one group after the other in shared memory.
bool make_map_groups(CUtensorMap *m, const void *base, uint64_t rows, uint64_t ld, uint64_t groups, uint32_t box_rows,
                     uint32_t box_groups) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {64, rows, groups};
  cuuint64_t strides[2] = {ld * 2, 128};
  cuuint32_t box[3] = {64, box_rows, box_groups};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

qlora_status fp8_gemm_ready() {
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return QLORA_ERR_NO_DEVICE;
  std::lock_guard<std::mutex> lk(mu);
  if (done[dev]) return QLORA_OK;
  if (cudaFuncSetAttribute(fp8_gemm_kernel<false, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFgSmemBytes) !=
          cudaSuccess ||
      cudaFuncSetAttribute(fp8_gemm_kernel<false, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFwSmemBytes) !=
          cudaSuccess ||
      cudaFuncSetAttribute(fp8_gemm_kernel<true, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFgSmemBytes) !=
          cudaSuccess)
    return QLORA_ERR_CUDA;
  done[dev] = true;
  return QLORA_OK;
}

// out [M, n_out] bf16 = deq(act) deq(W)^T (forward) or deq(act) deq(W) (DX) + hl * lw,
// with hl [M, 2 r16] the bf16 hi | lo halves and lw the weight side, B [r, N] or A [K, r]
// (r = 0: neither).
template <bool DX>
qlora_status launch_fp8_gemm(const qlora_fp8_t &act, const qlora_fp8_t &W, const uint16_t *hl, const uint16_t *lw,
                             int r, uint16_t *out, float *scratch, const Fp8Plan &plan, const GemmUnits &u,
                             cudaStream_t st, int late_wait = 0) {
  const int64_t M = act.rows, N = W.rows, K = W.cols;
  const int64_t n_out = DX ? K : N, contraction = DX ? N : K;
  if (u.pairs < 1) return QLORA_ERR_UNSUPPORTED_SHAPE;   // no room for clusters of two
  qlora_status e = fp8_gemm_ready();
  if (e != QLORA_OK) return e;
  const bool partial = plan.splits > 1;
  // few tokens: the weight on the MMA's 256 rows and the tokens, rounded up to 32, on its columns
  const bool few = !DX && M <= kFwTokens;
  const int nt = static_cast<int>((M + 31) / 32) * 32;
  const uint32_t tok_rows = few ? static_cast<uint32_t>(nt / 2) : kFgRows;      // of one CTA of a pair
  CUtensorMap tm_a, tm_w, tm_hl, tm_lw, tm_out;
  tm_out = tm_a = CUtensorMap{};
  if (!make_map_2d(&tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, act.codes, contraction, M, contraction, 128, tok_rows,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, W.codes, K, N, K, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      (!few && !make_map_3d(&tm_out, partial ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                            partial ? static_cast<void *>(scratch) : static_cast<void *>(out), n_out, M, plan.splits,
                            n_out * (partial ? 4 : 2), partial ? 32 : 64, 32)))
    return QLORA_ERR_CUDA;
  tm_hl = tm_a;
  tm_lw = tm_w;
  const int r16 = nn_proj(r);
  if (r && (!make_map_2d(&tm_hl, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, hl, 2 * r16, M, 4 * r16, 64, tok_rows,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
            !(DX ? make_map_2d(&tm_lw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, lw, r, K, r * 2, 64, kFgRows,
                               CU_TENSOR_MAP_SWIZZLE_128B)
                 : make_map_2d(&tm_lw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, lw, N, r, N * 2, 64, 64,
                               CU_TENSOR_MAP_SWIZZLE_128B))))
    return QLORA_ERR_CUDA;
  Fp8GemmParams p{};
  p.M = static_cast<int>(M);
  p.n_out = static_cast<int>(n_out);
  p.num_m_tiles = static_cast<int>((M + kFgTile - 1) / kFgTile);
  p.num_w_tiles = static_cast<int>((n_out + kFgTile - 1) / kFgTile);
  {
    // token tiles per raster group, as in the NF4 GEMM: a weight within the budget stays
    // in L2 by itself, a larger one is swept by groups of token tiles that do
    // (8192 tokens, forward: at 72 MB 22016 x 8192 takes 8% longer, at 16 MB 8192 x 22016 6%,
    // at 28 MB between -1% and 2% over 20 shapes)
    constexpr int64_t budget = 40ll << 20;
    int64_t g = (n_out * contraction <= budget) ? 1 : budget / (static_cast<int64_t>(kFgTile) * contraction);
    if (g < 1) g = 1;
    if (g > p.num_m_tiles) g = p.num_m_tiles;
    p.group_m = static_cast<int>(g);
  }
  p.nt = nt;
  p.out = partial ? static_cast<void *>(scratch) : static_cast<void *>(out);
  p.late_wait = late_wait;
  p.kb_main = static_cast<int>(contraction / 128);
  p.kb_lora = 2 * ((r16 + 63) / 64);
  p.r16 = r16;
  p.splits = plan.splits;
  p.groups_per_split = plan.groups_per_split;
  p.sa = act.scales;
  p.sa_pitch = static_cast<int>(f8_pitch(contraction));
  p.sw = W.scales;
  p.sw_pitch = static_cast<int>(f8_pitch(K));
  p.out_blocks = static_cast<int>(n_out / 128);
  p.a_fmt = act.fmt == QLORA_FP8_E5M2 ? 1u : 0u;
  p.limit_ns = static_cast<uint64_t>(g_wait_limit_us.load()) * 1000ull;
  if (static_cast<int64_t>(p.num_m_tiles) * p.num_w_tiles * plan.splits > (1ll << 30)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  const int64_t units = fp8_units(plan, M, n_out, u);
  {
    LaunchTimer lt(DX ? QLORA_K_FP8_GEMM_DX : QLORA_K_FP8_GEMM_FWD, st);
    const dim3 grid(static_cast<unsigned>(2 * units));
    e = few ? launch_pdl(fp8_gemm_kernel<false, true>, grid, kFgThreads, kFwSmemBytes, 2, 1, st, tm_a, tm_w, tm_hl, tm_lw,
                         tm_out, p)
            : launch_pdl(fp8_gemm_kernel<DX, false>, grid, kFgThreads, kFgSmemBytes, 2, 1, st, tm_a, tm_w, tm_hl, tm_lw,
                         tm_out, p);
  }
  if (e != QLORA_OK || !partial) return e;
  LaunchTimer lt(QLORA_K_PREP, st);
  const int64_t total = M * n_out;
  return launch_pdl(fp8_reduce_kernel, dim3(static_cast<unsigned>((total / 4 + 255) / 256)), 256, 0, 1, 1, st,
                    static_cast<const float *>(scratch), plan.splits, total, out);
}

// ------------------------------------------------------------------ cluster occupancy
// Clusters of one kernel that the current device holds at once, by cluster size and shared
// memory (0: none, or the runtime cannot say).  Each kernel has its own cache, of plain
// values; a full cache asks again.
struct ClusterCache {
  std::mutex mu;
  struct Entry {
    int dev, size, smem, n;
  } e[128];
  int count = 0;
};

template <typename K>
int max_clusters(ClusterCache &cache, K kernel, int threads, int cx, int cy, int smem) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lk(cache.mu);
  for (int i = 0; i < cache.count; ++i)
    if (cache.e[i].dev == dev && cache.e[i].size == cx * cy && cache.e[i].smem == smem) return cache.e[i].n;
  int n = 0;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess ||
      (cx * cy > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)) {
    (void)cudaGetLastError();
    return 0;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(cx), static_cast<unsigned>(cy), 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cx);
  attr[0].val.clusterDim.y = static_cast<unsigned>(cy);
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    n = 0;
  }
  if (cache.count < 128) cache.e[cache.count++] = {dev, cx * cy, smem, n};
  return n;
}

// ------------------------------------------------------------------ rank-r products

// The operands of one rank-r product: the activation [act_rows, act_cols] (codes or bf16),
// Q [q_rows, q_cols] bf16 with a row pitch of q_ld elements.
struct AmOperands {
  const void *act;
  int64_t act_rows, act_cols;
  const uint16_t *q;
  int64_t q_rows, q_cols, q_ld;
};

// Fills the geometry of p (rows, columns, q_kmajor, n, outputs set by the caller) and launches.
// `room` > 0: SMs that a GEMM launched to run beside this leaves free.
template <int ACT, bool GRAD, int QUANT>
qlora_status launch_adapter(const AmOperands &o, AdapterParams p, cudaStream_t st, int64_t room = 0) {
  constexpr bool F8 = ACT != kActBf16;
  const int64_t contraction = GRAD ? o.act_rows : o.act_cols;
  p.tokens = static_cast<int>(o.act_rows);
  p.act_cols = o.act_cols;
  p.pairs_total = static_cast<int>((contraction + 127) / 128);
  const int q_groups = (p.n + 63) / 64;
  p.q_bytes = p.q_kmajor ? p.r16 * 128 : q_groups * 8192;
  p.tmem_cols = 32;
  while (static_cast<int>(p.tmem_cols) < 2 * p.n) p.tmem_cols <<= 1;
  // rings: 64 KB of raw codes in flight, the rest operand slots
  p.n_raw = F8 ? kAmMaxRaw : 0;
  p.n_op = 4;
  while (p.n_op < kAmMaxOp && am_smem_bytes(p.n_op + 1, p.n_raw, p.q_bytes) <= kAmSmemMax) ++p.n_op;
  const int smem = am_smem_bytes(p.n_op, p.n_raw, p.q_bytes);
  const int64_t tiles = (p.rows + kAmRows - 1) / kAmRows;
  // splits: fewest waves of clusters times the length of a CTA, its pairs plus about
  // eight pairs' worth of setup, first load and reduction
  static ClusterCache cache;
  int64_t best = -1;
  for (int c = kAmClusterMax; c >= 1; c >>= 1) {
    const int per = (p.pairs_total + c - 1) / c;
    const int splits = (p.pairs_total + per - 1) / per;
    const int active = max_clusters(cache, adapter_mma_kernel<ACT, GRAD, QUANT>, kAmThreads, 1, splits, smem);
    if (active <= 0) continue;
    // a CTA fills an SM: where fewer splits fit into the room, more would hold the GEMM up
    if (tiles <= room && tiles * splits > room && splits > 1) continue;
    const int64_t cost = ((tiles + active - 1) / active) * (per + 8);
    if (best < 0 || cost < best) {
      best = cost;
      p.pairs_per_split = per;
      p.splits = splits;
    }
  }
  if (best < 0) return QLORA_ERR_CUDA;
  p.limit_ns = static_cast<uint64_t>(g_wait_limit_us.load()) * 1000ull;
  CUtensorMap tm_act, tm_q;
  // Gradients take 64-column groups as a third dimension, one copy for all of a stage's.
  // The last group of Q may reach past its rows (the workspace is padded for the last row's);
  // those columns are past the MMA's N.
  constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kU8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const bool act_ok =
      F8 ? make_map_2d(&tm_act, kU8, o.act, o.act_cols, o.act_rows, o.act_cols, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B)
      : GRAD ? make_map_groups(&tm_act, o.act, o.act_rows, o.act_cols, o.act_cols / 64, 64, 2)
             : make_map_2d(&tm_act, kBf16, o.act, o.act_cols, o.act_rows, o.act_cols * 2, 64, 128,
                           CU_TENSOR_MAP_SWIZZLE_128B);
  const bool maps =
      act_ok && (GRAD ? make_map_groups(&tm_q, o.q, o.q_rows, o.q_ld, q_groups, 64, q_groups)
                      : make_map_2d(&tm_q, kBf16, o.q, o.q_cols, o.q_rows, o.q_ld * 2, 64,
                                    p.q_kmajor ? static_cast<uint32_t>(p.r16) : 64u, CU_TENSOR_MAP_SWIZZLE_128B));
  if (!maps) return QLORA_ERR_CUDA;
  LaunchTimer lt(GRAD ? QLORA_K_GRAD : QLORA_K_PROJECT, st);
  return launch_pdl(adapter_mma_kernel<ACT, GRAD, QUANT>,
                    dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(p.splits)), kAmThreads, smem, 1, p.splits, st,
                    tm_act, tm_q, p);
}

// Column pass i of a product of rank r: columns [j0, j0 + r of the pass).
int am_passes(int r) { return (r + kAmPass - 1) / kAmPass; }
void am_pass(AdapterParams &p, int i, int r) {
  p.ld = r;
  p.j0 = i * kAmPass;
  p.r = r - p.j0 < kAmPass ? r - p.j0 : kAmPass;
  p.r16 = nn_proj(p.r);
}

// XA = (deq(X) (.) keep) A * scale: fp32 [M, r], hi|lo of s*XA [M, 2 r16] and the three
// terms of s*XA, each where given.
qlora_status launch_xa8(const qlora_fp8_t &X, const uint16_t *A, int r, float s, float *out, uint16_t *hl,
                        uint16_t *terms, const uint8_t *keep, float scale, cudaStream_t st, int64_t room = 0) {
  AdapterParams p{};
  p.rows = static_cast<int>(X.rows);
  p.half = nn_proj(r);
  p.s = s;
  p.out_scale = scale;
  p.out = out;
  p.hl = hl;
  p.terms = terms;
  p.scales = X.scales;
  p.pitch = f8_pitch(X.cols);
  p.keep = keep;
  for (int i = 0; i < am_passes(r); ++i) {
    am_pass(p, i, r);
    p.n = p.r16;
    // the columns of A from j0 on: the row pitch stays r
    const AmOperands o{X.codes, X.rows, X.cols, A + p.j0, X.cols, p.r, r};
    const qlora_status e = X.fmt == QLORA_FP8_E5M2 ? launch_adapter<kActE5M2, false, kQuantNone>(o, p, st, room)
                                                   : launch_adapter<kActE4M3, false, kQuantNone>(o, p, st, room);
    if (e != QLORA_OK) return e;
  }
  return QLORA_OK;
}

// G = dY B^T: hi|lo of s*G [M, 2 half], its three terms, the three terms of s*XA when the saved
// XA is given; with `q` the 8-bit form of dY, from the same pass over it.  `clear` as in
// launch_projection.
qlora_status launch_g(const uint16_t *dY, int64_t M, int64_t N, const uint16_t *B, int r, float s, uint16_t *hl,
                      int half, uint16_t *terms, const float *XA, uint16_t *xa_terms, const qlora_fp8_t *q,
                      const SplitScratch *clear, cudaStream_t st) {
  AdapterParams p{};
  p.rows = static_cast<int>(M);
  p.half = half;
  p.q_kmajor = 1;
  p.s = s;
  p.out_scale = 1.0f;
  p.hl = hl;
  p.terms = terms;
  p.split_in = XA;
  p.split_terms = XA ? xa_terms : nullptr;
  if (clear && clear->g.count) {
    p.zero = clear->flags;
    p.zero_n = clear->g.count * clear->g.parts();
  }
  for (int i = 0; i < am_passes(r); ++i) {
    am_pass(p, i, r);
    p.n = p.r16;
    const AmOperands o{dY, M, N, B + static_cast<int64_t>(p.j0) * N, p.r, N, N};
    qlora_status e;
    if (!q || i > 0) {
      e = launch_adapter<kActBf16, false, kQuantNone>(o, p, st);
    } else {
      p.q_codes = q->codes;
      p.q_scales = q->scales;
      p.q_pitch = f8_pitch(N);
      e = q->fmt == QLORA_FP8_E5M2 ? launch_adapter<kActBf16, false, kQuantE5M2>(o, p, st)
                                   : launch_adapter<kActBf16, false, kQuantE4M3>(o, p, st);
    }
    if (e != QLORA_OK) return e;
  }
  return QLORA_OK;
}

// One adapter gradient from the three terms of its factor:
// dA [K, r] = scale * (deq(X) (.) keep)^T (sG), or dB [r, N] = (sXA)^T dY.
template <int ACT>
qlora_status launch_grad(const void *act, int64_t M, int64_t cols, const uint16_t *terms, int r, AdapterParams p,
                         cudaStream_t st) {
  p.rows = static_cast<int>(cols);
  for (int i = 0; i < am_passes(r); ++i) {
    am_pass(p, i, r);
    if (i) p.late_wait = 1;   // the passes are independent of one another
    p.n = 3 * p.r16;
    const AmOperands o{act, M, cols, terms + M * 3 * p.j0, M, p.n, p.n};
    const qlora_status e = launch_adapter<ACT, true, kQuantNone>(o, p, st);
    if (e != QLORA_OK) return e;
  }
  return QLORA_OK;
}

qlora_status launch_da8(const qlora_fp8_t &X, const uint16_t *terms, int r, float *dA, int accumulate,
                        const uint8_t *keep, float scale, cudaStream_t st, int late_wait = 0) {
  AdapterParams p{};
  p.late_wait = late_wait;
  p.out_scale = scale;
  p.out = dA;
  p.accumulate = accumulate;
  p.scales = X.scales;
  p.pitch = f8_pitch(X.cols);
  p.keep = keep;
  return X.fmt == QLORA_FP8_E5M2 ? launch_grad<kActE5M2>(X.codes, X.rows, X.cols, terms, r, p, st)
                                 : launch_grad<kActE4M3>(X.codes, X.rows, X.cols, terms, r, p, st);
}

qlora_status launch_db(const uint16_t *dY, int64_t M, int64_t N, const uint16_t *terms, int r, float *dB,
                       int accumulate, cudaStream_t st) {
  AdapterParams p{};
  p.late_wait = 1;   // launched behind dA, of which it needs nothing
  p.out_scale = 1.0f;
  p.out = dB;
  p.layout = 1;
  p.accumulate = accumulate;
  return launch_grad<kActBf16>(dY, M, N, terms, r, p, st);
}

// ------------------------------------------------------------------ few tokens
// Clusters over which the few-token XA divides K: about 32 KB of A per CTA.  Smaller parts end
// sooner, but their CTAs take the places of the weight pass's: 1 token, r 16, N 4096, K 11008,
// replayed, takes 15.3 us with 64 of them and 12.3 us with 16; at 16 KB each N 8192, K 22016
// takes 37 us for 32.5 us.
int xa8_parts(int64_t K, int r) {
  const int64_t n = (K * r * 2 + kXaCluster * 32768 - 1) / (kXaCluster * 32768);
  return static_cast<int>(n < kS8MaxXaParts ? n : kS8MaxXaParts);
}
size_t xa8_bytes(int64_t M, int64_t K, int r) { return r ? static_cast<size_t>(xa8_parts(K, r)) * M * r * 4 : 0; }

// Rows of A per pass of XA: what an SM's shared memory leaves beside two CTAs of the weight
// pass (each launch takes 1 KB more than it asks for).
int xa8_chunk(int r, int kx, int skinny_smem) {
  const int left = 228 * 1024 - 2 * (skinny_smem + 1024) - 1024;
  const int rows = (left - xa_smem_bytes(r, 0, kS8MaxTokens)) / (2 * (r + kS8MaxTokens)) / 16 * 16;
  return rows > kx ? kx : rows < 64 ? 64 : rows;
}

template <bool XE5M2>
qlora_status launch_skinny8(const qlora_fp8_t &X, const qlora_fp8_t &W, const uint16_t *A, const uint16_t *B, int r,
                            float s, uint16_t *Y, float *xa, float *xa_out, cudaStream_t st) {
  const int64_t M = X.rows, N = W.rows, K = W.cols;
  // cluster size: fewest waves times the blocks of a CTA plus 14, what a wave costs beside them
  // (with 4, 1 token of 22016 x 4096 takes 24.3 us, with 14 19.5; 11008 x 8192 24.0 and 20.0;
  // 15 other layers the same)
  static ClusterCache cache;
  Skinny8Plan pl{};
  int64_t best = -1;
  for (int C = kS8MaxCluster; C >= 1; C >>= 1) {
    const Skinny8Plan cand = skinny8_plan(static_cast<int>(M), static_cast<int>(K), r, C);
    if (cand.smem > 227 * 1024 || (C > 1 && C > K / 128)) continue;
    const int active = max_clusters(cache, fp8_skinny_kernel<XE5M2>, kS8Threads, C, 1, cand.smem);
    if (active <= 0) continue;
    const int64_t cost = ((N / kS8Rows + active - 1) / active) * (cand.blocks + 14);
    if (best < 0 || cost < best) {
      best = cost;
      pl = cand;
    }
  }
  if (best < 0) return QLORA_ERR_CUDA;
  const uint64_t limit_ns = static_cast<uint64_t>(g_wait_limit_us.load()) * 1000ull;
  const int pitch = static_cast<int>(f8_pitch(K));
  const int parts = r ? xa8_parts(K, r) : 0;
  if (r) {
    // it lets the weight pass start when everything before it in the stream has finished, so
    // the weight pass may read X and W at once
    XaParams xp{};
    xp.scale = 1.0f;
    xp.A = A;
    xp.xa = xa;
    xp.M = static_cast<int>(M);
    xp.K = static_cast<int>(K);
    xp.r = r;
    xp.kx = static_cast<int>((K / (kXaCluster * parts) + 15) / 16 * 16);
    xp.chunk = xa8_chunk(r, xp.kx, pl.smem);
    xp.limit_ns = limit_ns;
    xp.codes = X.codes;
    xp.scales = X.scales;
    xp.pitch = pitch;
    xp.e5m2 = XE5M2 ? 1 : 0;
    LaunchTimer lt(QLORA_K_PROJECT, st);
    const qlora_status e = launch_pdl(qlora_xa_kernel<true>, dim3(kXaCluster, static_cast<unsigned>(parts)), 256,
                                      xa_smem_bytes(r, xp.chunk, kS8MaxTokens), kXaCluster, 1, st, xp);
    if (e != QLORA_OK) return e;
  }
  const int R = kS8Rows / pl.C;
  CUtensorMap tm_w, tm_x, tm_b;
  if (!make_map_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, W.codes, K, N, K, 128, kS8Rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map_2d(&tm_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, X.codes, K, M, K, 128, kS8MaxTokens, CU_TENSOR_MAP_SWIZZLE_NONE))
    return QLORA_ERR_CUDA;
  tm_b = tm_w;
  if (r && !make_map_2d(&tm_b, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, B, N, r, 2 * N, R, r, CU_TENSOR_MAP_SWIZZLE_NONE))
    return QLORA_ERR_CUDA;
  Skinny8Params p{};
  p.xs = X.scales;
  p.ws = W.scales;
  p.pitch = pitch;
  p.xa = xa;
  p.xa_parts = parts;
  p.xa_out = xa_out;
  p.Y = Y;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.r = r;
  p.blocks = pl.blocks;
  p.s = s;
  p.off_b = pl.off_b;
  p.off_recv = pl.off_recv;
  p.off_xa = pl.off_xa;
  p.off_bar = pl.off_bar;
  p.limit_ns = limit_ns;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(pl.C), static_cast<unsigned>(N / kS8Rows), 1);
  cfg.blockDim = dim3(kS8Threads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(pl.smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(pl.C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = r ? 2 : 1;   // a dependent of the XA launch, or a plain launch
  LaunchTimer lt(QLORA_K_FP8_SKINNY, st);
  return cuda_status(cudaLaunchKernelEx(&cfg, fp8_skinny_kernel<XE5M2>, tm_w, tm_x, tm_b, p));
}

// ------------------------------------------------------------------ workspaces
size_t fp8_hl_bytes(int64_t M, int r) { return align256(static_cast<size_t>(M) * 2 * nn_proj(r) * 2); }
// (128 bytes more than the terms: a 64-column group may reach past the last row)
size_t fp8_terms_bytes(int64_t M, int r) { return align256(static_cast<size_t>(M) * 3 * nn_proj(r) * 2 + 128); }

// The calls of the few-token kernel.  Each of its CTAs adds the parts of XA, M r values, and takes the
// rank-r product of its rows without the tensor core; the GEMM's form pays two more launches and,
// past rank 64, a second pass for XA.  Both forced on 6 layers (4096 x 4096 to 8192 x 22016), ranks 8 to
// 128, 1 to 8 tokens, replayed, us:
//   8192 x 8192   1 token, r 16: 16.2 (GEMM 17.9); 8 tokens, r 64: 18.6 (18.5); 8 tokens, r 128: 23.0 (26.6)
//   11008 x 4096  1 token, r 16: 13.9 (14.6); 8 tokens, r 64: 17.2 (14.8); 8 tokens, r 128: 19.7 (21.3)
//   4096 x 11008  1 token, r 16: 12.4 (15.0); 8 tokens, r 64: 17.4 (15.5); 8 tokens, r 128: 18.9 (24.8)
// This rule takes the faster form, or one within 2% of it, in 232 of the 252 calls, and one at most 10%
// slower in the others.  The launch has a row of clusters for each 128 weight rows, at most 65535.
bool fp8_few_tokens(int64_t M, int64_t N, int r) {
  return M <= kS8MaxTokens && (M * r <= 384 || r > kAmPass) && N / kS8Rows <= 65535;
}

size_t fp8_fwd_workspace(int64_t M, int64_t N, int64_t K, int r, const GemmUnits &u) {
  // few tokens: the parts of XA; otherwise s*XA hi|lo and the parts of a divided contraction
  if (fp8_few_tokens(M, N, r)) return 256 + align256(xa8_bytes(M, K, r));
  return 256 + fp8_hl_bytes(M, r) + align256(fp8_plan(M, N, K, u, M <= kFwTokens).scratch_bytes);
}

size_t fp8_bwd_workspace(int64_t M, int64_t N, int64_t K, int r, const GemmUnits &u) {
  // q(dY), s*G hi|lo, the terms of s*G and s*XA, and the parts of a divided contraction
  return 256 + align256(static_cast<size_t>(M) * N) + align256(static_cast<size_t>(M) * f8_pitch(N)) +
         fp8_hl_bytes(M, r) + 2 * fp8_terms_bytes(M, r) + align256(fp8_plan(M, K, N, u, false).scratch_bytes);
}

size_t ckpt_workspace(int64_t M, int64_t N, int64_t K, int r, const GemmUnits &u) {
  // s*G hi|lo, the terms of s*G and s*XA, and the NF4 GEMM's last-round partial tiles
  return 256 + align256(static_cast<size_t>(M) * 2 * r * 2) + 2 * fp8_terms_bytes(M, r) +
         split_workspace_any(M, K, N, u);
}

// ------------------------------------------------------------------ the linear layer on an 8-bit base
qlora_status fp8_fwd_impl(const qlora_fp8_t *X, const qlora_fp8_t *W, const uint16_t *A, const uint16_t *B, int r,
                          float s, uint16_t *Y, float *XA_out, void *workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
  qlora_status st = check_fp8(X, 1);
  if (st != QLORA_OK) return st;
  const int64_t M = X->rows;
  if ((st = check_fp8_layer(M, W, A, B, r, s)) != QLORA_OK) return st;
  if (!Y || X->cols != W->cols || (!r && XA_out)) return QLORA_ERR_INVALID_ARG;
  if ((A && !aligned16(A)) || (B && !aligned16(B)) || !aligned16(Y) || (XA_out && !aligned16(XA_out)) ||
      (workspace && !aligned16(workspace)))
    return QLORA_ERR_MISALIGNED;
  DeviceInfo *d = nullptr;
  if ((st = device_info(&d)) != QLORA_OK) return st;
  const int64_t N = W->rows, K = W->cols;
  if (!workspace || workspace_bytes < fp8_fwd_workspace(M, N, K, r, d->units)) return QLORA_ERR_WORKSPACE;
  Workspace ws{static_cast<char *>(workspace), 0, workspace_bytes};
  if (fp8_few_tokens(M, N, r)) {
    float *xa = static_cast<float *>(ws.take(xa8_bytes(M, K, r)));
    if (!xa) return QLORA_ERR_WORKSPACE;
    return X->fmt == QLORA_FP8_E5M2 ? launch_skinny8<true>(*X, *W, A, B, r, s, Y, xa, XA_out, stream)
                                    : launch_skinny8<false>(*X, *W, A, B, r, s, Y, xa, XA_out, stream);
  }
  const Fp8Plan plan = fp8_plan(M, N, K, d->units, M <= kFwTokens);
  float *scratch = static_cast<float *>(ws.take(plan.scratch_bytes));
  if (!scratch) return QLORA_ERR_WORKSPACE;
  // The GEMM, the dependent of XA, reads X and W beside it and waits for hl only at its first
  // rank-r step.
  uint16_t *hl = nullptr;
  if (r) {
    hl = static_cast<uint16_t *>(ws.take(fp8_hl_bytes(M, r)));
    if (!hl) return QLORA_ERR_WORKSPACE;
    if ((st = launch_xa8(*X, A, r, s, XA_out, hl, nullptr, nullptr, 1.0f, stream, d->sms - 2 * fp8_units(plan, M, N, d->units))) !=
        QLORA_OK)
      return st;
  }
  return launch_fp8_gemm<false>(*X, *W, hl, B, r, Y, scratch, plan, d->units, stream, r > 0 ? 1 : 0);
}

qlora_status fp8_bwd_impl(const uint16_t *dY, int64_t M, const qlora_fp8_t *X, const float *XA, const qlora_fp8_t *W,
                          const uint16_t *A, const uint16_t *B, int r, float s, int grad_fmt, int accumulate,
                          uint16_t *dX, float *dA, float *dB, void *workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
  qlora_status st = check_fp8_layer(M, W, A, B, r, s);
  if (st != QLORA_OK) return st;
  if (!dY || (grad_fmt != QLORA_FP8_E4M3 && grad_fmt != QLORA_FP8_E5M2)) return QLORA_ERR_INVALID_ARG;
  if (r ? (!X || !dA || !dB) : (X || XA || dA || dB || !dX)) return QLORA_ERR_INVALID_ARG;
  const int64_t N = W->rows, K = W->cols;
  if (r) {
    if ((st = check_fp8(X, 1)) != QLORA_OK) return st;
    if (X->rows != M || X->cols != K) return QLORA_ERR_INVALID_ARG;
  }
  if (!aligned16(dY) || (A && !aligned16(A)) || (B && !aligned16(B)) || (dA && !aligned16(dA)) ||
      (dB && !aligned16(dB)) || (dX && !aligned16(dX)) || (XA && !aligned16(XA)) ||
      (workspace && !aligned16(workspace)))
    return QLORA_ERR_MISALIGNED;
  if (dX && overlap_bf16(dX, M * K, dY, M * N)) return QLORA_ERR_INVALID_ARG;
  if (M * (N / 128) >= (1ll << 31)) return QLORA_ERR_UNSUPPORTED_SHAPE;
  DeviceInfo *d = nullptr;
  if ((st = device_info(&d)) != QLORA_OK) return st;
  if (!workspace || workspace_bytes < fp8_bwd_workspace(M, N, K, r, d->units)) return QLORA_ERR_WORKSPACE;
  Workspace ws{static_cast<char *>(workspace), 0, workspace_bytes};
  const Fp8Plan plan = fp8_plan(M, K, N, d->units, false);
  float *scratch = static_cast<float *>(ws.take(plan.scratch_bytes));
  qlora_fp8_t q{};
  q.rows = M;
  q.cols = N;
  q.fmt = grad_fmt;
  q.block_rows = 1;
  q.codes = static_cast<uint8_t *>(ws.take(static_cast<size_t>(M) * N));
  q.scales = static_cast<uint8_t *>(ws.take(static_cast<size_t>(M) * f8_pitch(N)));
  if (!scratch || !q.codes || !q.scales) return QLORA_ERR_WORKSPACE;
  if (!r) {
    if ((st = launch_fp8_quantize(dY, q, stream)) != QLORA_OK) return st;
    return launch_fp8_gemm<true>(q, *W, nullptr, nullptr, 0, dX, scratch, plan, d->units, stream);
  }
  uint16_t *ghl = static_cast<uint16_t *>(ws.take(fp8_hl_bytes(M, r)));
  uint16_t *gt = static_cast<uint16_t *>(ws.take(fp8_terms_bytes(M, r)));
  uint16_t *xat = static_cast<uint16_t *>(ws.take(fp8_terms_bytes(M, r)));
  if (!ghl || !gt || !xat) return QLORA_ERR_WORKSPACE;
  if (!XA && (st = launch_xa8(*X, A, r, s, nullptr, nullptr, xat, nullptr, 1.0f, stream)) != QLORA_OK) return st;
  if ((st = launch_g(dY, M, N, B, r, s, ghl, nn_proj(r), gt, XA, xat, dX ? &q : nullptr, nullptr, stream)) != QLORA_OK)
    return st;
  // dX waits for G, so once it runs, dA and dB (which need nothing of it) take the SMs that its
  // last round leaves: 4096 tokens of 22016 x 8192, r 16, 615 us in a graph, 640 with dX behind
  // them; small layers the same
  if (dX && (st = launch_fp8_gemm<true>(q, *W, ghl, A, r, dX, scratch, plan, d->units, stream)) != QLORA_OK) return st;
  if ((st = launch_da8(*X, gt, r, dA, accumulate, nullptr, 1.0f, stream, dX ? 1 : 0)) != QLORA_OK) return st;
  return launch_db(dY, M, N, xat, r, dB, accumulate, stream);
}

// ------------------------------------------------------------------ the NF4 layer's backward from a checkpoint
qlora_status bwd_ckpt_impl(const uint16_t *dY, const qlora_fp8_t *X, const float *XA, const qlora_nf4_t *Wq,
                           const uint16_t *A, const uint16_t *B, int r, float s, const uint8_t *keep, float drop_p,
                           int accumulate, uint16_t *dX, float *dA, float *dB, void *workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  qlora_status st = check_fp8(X, 1);
  if (st != QLORA_OK || (st = check_nf4(Wq)) != QLORA_OK) return st;
  if (!dY || !A || !B || !dA || !dB || X->cols != Wq->cols) return QLORA_ERR_INVALID_ARG;
  const int64_t M = X->rows, N = Wq->rows, K = Wq->cols;
  if ((st = check_linear_shape(M, Wq, r)) != QLORA_OK) return st;
  if (!aligned16(dY) || !aligned16(A) || !aligned16(B) || !aligned16(dA) || !aligned16(dB) ||
      (dX && !aligned16(dX)) || (XA && !aligned16(XA)) || (workspace && !aligned16(workspace)))
    return QLORA_ERR_MISALIGNED;
  if (!(s == s) || (dX && overlap_bf16(dX, M * K, dY, M * N))) return QLORA_ERR_INVALID_ARG;
  if ((st = check_dropout(keep, drop_p)) != QLORA_OK) return st;
  DeviceInfo *d = nullptr;
  if ((st = device_info(&d)) != QLORA_OK) return st;
  if (!workspace || workspace_bytes < ckpt_workspace(M, N, K, r, d->units)) return QLORA_ERR_WORKSPACE;
  Workspace ws{static_cast<char *>(workspace), 0, workspace_bytes};
  const float xscale = keep ? 1.0f / (1.0f - drop_p) : 1.0f;
  uint16_t *ghl = static_cast<uint16_t *>(ws.take(static_cast<size_t>(M) * 2 * r * 2));
  uint16_t *gt = static_cast<uint16_t *>(ws.take(fp8_terms_bytes(M, r)));
  uint16_t *xat = static_cast<uint16_t *>(ws.take(fp8_terms_bytes(M, r)));
  SplitScratch sp;
  if (!ghl || !gt || !xat) return QLORA_ERR_WORKSPACE;
  if (dX && !take_split(ws, gemm_plan(M, K, N, d->units), sp)) return QLORA_ERR_WORKSPACE;
  if (!XA && (st = launch_xa8(*X, A, r, s, nullptr, nullptr, xat, keep, xscale, stream)) != QLORA_OK) return st;
  if ((st = launch_g(dY, M, N, B, r, s, ghl, r, gt, XA, xat, nullptr, &sp, stream)) != QLORA_OK) return st;
  // dA waits for G; dB, which needs nothing of dA, runs beside it
  if ((st = launch_da8(*X, gt, r, dA, accumulate, keep, xscale, stream)) != QLORA_OK) return st;
  if ((st = launch_db(dY, M, N, xat, r, dB, accumulate, stream)) != QLORA_OK || !dX) return st;
  return launch_gemm<kModeDx>(dY, M, Wq, ghl, A, r, dX, sp, d->units, stream, keep, xscale);
}

}  // namespace

// ==================================================================== C ABI
extern "C" {

size_t qlora_fp8_bytes(int64_t rows, int64_t cols, int block_rows, size_t *codes_bytes, size_t *scales_bytes) {
  size_t c = 0, s = 0;
  if (rows > 0 && cols > 0 && (block_rows == 1 || block_rows == kF8Block)) {
    c = static_cast<size_t>(rows) * static_cast<size_t>(cols);
    s = static_cast<size_t>((rows + block_rows - 1) / block_rows) * static_cast<size_t>(f8_pitch(cols));
  }
  if (codes_bytes) *codes_bytes = c;
  if (scales_bytes) *scales_bytes = s;
  return c + s;
}

qlora_status qlora_fp8_quantize(const uint16_t *X, int64_t rows, int64_t cols, const qlora_fp8_t *out,
                                qlora_stream_t stream) {
  if (!X || !out || rows <= 0 || cols <= 0) return QLORA_ERR_INVALID_ARG;
  if (out->rows != rows || out->cols != cols) return QLORA_ERR_INVALID_ARG;
  qlora_status st = check_fp8(out, 0);
  if (st != QLORA_OK) return st;
  if (!aligned16(X)) return QLORA_ERR_MISALIGNED;
  DeviceInfo *d = nullptr;
  if ((st = device_info(&d)) != QLORA_OK) return st;
  return launch_fp8_quantize(X, *out, stream);
}

qlora_status qlora_fp8_dequant(const qlora_fp8_t *X, uint16_t *out, qlora_stream_t stream) {
  qlora_status st = check_fp8(X, 0);
  if (st != QLORA_OK) return st;
  if (!out) return QLORA_ERR_INVALID_ARG;
  if (!aligned16(out)) return QLORA_ERR_MISALIGNED;
  DeviceInfo *d = nullptr;
  if ((st = device_info(&d)) != QLORA_OK) return st;
  return launch_fp8_dequant(*X, out, stream);
}

size_t qlora_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K, int r) {
  if (M < 1 || N < 1 || K < 1 || r < 0) return 0;
  GemmUnits u;
  DeviceInfo *d = nullptr;
  if (device_info(&d) == QLORA_OK) u = d->units;
  const size_t f = fp8_fwd_workspace(M, N, K, r, u), b = fp8_bwd_workspace(M, N, K, r, u);
  return f > b ? f : b;
}

qlora_status qlora_fp8_linear_fwd(const qlora_fp8_t *X, const qlora_fp8_t *W, const uint16_t *A, const uint16_t *B,
                                  int r, float s, uint16_t *Y, float *XA_out, void *workspace,
                                  size_t workspace_bytes, qlora_stream_t stream) {
  return fp8_fwd_impl(X, W, A, B, r, s, Y, XA_out, workspace, workspace_bytes, stream);
}

qlora_status qlora_fp8_linear_bwd(const uint16_t *dY, int64_t M, const qlora_fp8_t *X, const float *XA,
                                  const qlora_fp8_t *W, const uint16_t *A, const uint16_t *B, int r, float s,
                                  int grad_fmt, int accumulate, uint16_t *dX, float *dA, float *dB, void *workspace,
                                  size_t workspace_bytes, qlora_stream_t stream) {
  return fp8_bwd_impl(dY, M, X, XA, W, A, B, r, s, grad_fmt, accumulate, dX, dA, dB, workspace, workspace_bytes,
                      stream);
}

size_t qlora_linear_ckpt_workspace_bytes(int64_t M, int64_t N, int64_t K, int r) {
  if (M < 1 || N < 1 || K < 1 || r < 1) return 0;
  GemmUnits u;
  DeviceInfo *d = nullptr;
  if (device_info(&d) == QLORA_OK) u = d->units;
  return ckpt_workspace(M, N, K, r, u);
}

qlora_status qlora_linear_bwd_ckpt(const uint16_t *dY, const qlora_fp8_t *X, const float *XA, const qlora_nf4_t *Wq,
                                   const uint16_t *A, const uint16_t *B, int r, float s, const uint8_t *keep,
                                   float dropout_p, int accumulate, uint16_t *dX, float *dA, float *dB,
                                   void *workspace, size_t workspace_bytes, qlora_stream_t stream) {
  return bwd_ckpt_impl(dY, X, XA, Wq, A, B, r, s, keep, dropout_p, accumulate, dX, dA, dB, workspace, workspace_bytes,
                       stream);
}

}  // extern "C"
