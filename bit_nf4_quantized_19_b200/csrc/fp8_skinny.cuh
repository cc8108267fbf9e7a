// Few-token forward (M <= 8; fp8_few_tokens says for which ranks) of the linear layer on an 8-bit base:
//     Y = deq(X) deq(W)^T + s (XA) B
// Bound by reading the 8-bit weight once, so the design keeps the weight stream deep and
// everything else beside it.  XA comes from qlora_xa_kernel<true> (clusters of eight
// CTAs, each a part of K), launched just before; this kernel is its programmatic dependent,
// runs beside it, and one warp waits for it and adds its parts.
//   - A CTA owns 128 weight rows and one slice of K; the C CTAs of a row tile form a cluster
//     that exchanges fp32 partials through distributed shared memory (summed in a fixed
//     order).
//   - The codes arrive by TMA in 128 x 128 boxes (16 KB, one block: one factor byte) through
//     a ring of kS8Stages; two CTAs fit an SM, 128 KB in flight.
//   - The products run on mma.sync m16n8k16 f16: every e4m3 and e5m2 code is exact in f16 (one
//     conversion for two codes), products accumulate in fp32 and each block's sum is scaled
//     by 2^(eW + eX) as it is added, in two factors of half the exponent each (see s8_factors).  The
//     contraction index is permuted inside a block so
//     that a lane takes 16 consecutive codes of its rows: step w of a 16-byte piece is its
//     word w, codes 0, 1 and 2, 3 the fragment's two halves, for W and X alike.
//   - The CTAs of XA fit beside two of these on an SM (72 and 40 registers, small chunks), so the
//     weight pass has its places from the start: with XA on SMs of its own, whole clusters
//     waited for it (1 token, r 64, N 8192, K 22016, replayed: 40 us, now 34; the weight
//     alone at 6.45 TB/s is 28).
//   - X's codes come by TMA too, and two warps, on alternate blocks, convert them for all: they
//     stage each block's f16 fragments, in the order the product warps' registers take them,
//     and the tokens' factors, beside the codes.  (With every product warp converting X
//     itself the kernel was bound by issue: 414 instructions per warp and block.)
#pragma once
#include "common.cuh"
#include "fp8_quant.cuh"
#include "pipeline.cuh"
#include "skinny_kernel.cuh"

namespace qlora {

constexpr int kS8MaxTokens = 8;            // one n8 group of the MMA; 9 tokens and more are faster on the GEMM
constexpr int kS8Threads = 384;            // eight product warps, the TMA producer, two X warps, the XA warp
// Two CTAs at 72 registers leave the 10240 that a CTA of the XA kernel takes (launch bounds of 448
// threads hold the compiler to that).
constexpr int kS8RegThreads = 448;
constexpr int kS8Rows = 128;
constexpr int kS8BoxBytes = kS8Rows * 128;
constexpr int kS8Stages = 4;
constexpr int kS8MaxCluster = 8;
constexpr int kS8MaxXaParts = 8;

struct Skinny8Params {
  const uint8_t *xs;       // factors [M, pitch]
  const uint8_t *ws;       // factors [N / 128, pitch]
  int pitch;
  const float *xa;         // [xa_parts][M, r] partial sums, written by the kernel before; r = 0: none
  int xa_parts;
  float *xa_out;           // their sum, or null
  uint16_t *Y;
  int M, N, K, r;
  int blocks;              // 128-value blocks per cluster rank
  float s;
  int off_b, off_recv, off_xa, off_bar;   // byte offsets from the 1024-aligned base
  uint64_t limit_ns;
};

struct Skinny8Plan {
  int C, blocks, off_b, off_recv, off_xa, off_bar, smem;
};
// X in one stage: the codes of eight tokens, their f16 fragments, eight pairs of factors.
constexpr int kS8XCodes = 1024, kS8XFrags = 2048;
constexpr int kS8XBytes = kS8XCodes + kS8XFrags + 128;
inline Skinny8Plan skinny8_plan(int M, int K, int r, int C) {
  Skinny8Plan pl{};
  const int nb = K / 128;
  pl.C = C;
  pl.blocks = (nb + C - 1) / C;
  int off = kS8Stages * (kS8BoxBytes + kS8XBytes);
  pl.off_b = off;     off += (r * (kS8Rows / C) * 2 + 127) & ~127;
  pl.off_recv = off;  off += kS8Rows * M * 4;
  pl.off_xa = off;    off += (M * r * 4 + 15) & ~15;
  pl.off_bar = off;   off += 8 * (3 * kS8Stages + 1) + 16;
  pl.smem = off + 1024;
  return pl;
}

QDEV void mma_16816_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Codes 0, 1 and 2, 3 of a word as two f16 pairs (exact).
template <bool E5M2>
QDEV void f8_to_f16x2(uint32_t w, uint32_t &lo, uint32_t &hi) {
  const uint16_t a = static_cast<uint16_t>(w), b = static_cast<uint16_t>(w >> 16);
  if (E5M2) {
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(lo) : "h"(a));
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(hi) : "h"(b));
  } else {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(a));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(b));
  }
}

// 2^(eX + eW) as two powers of two that fp32 holds whatever the bytes are, each with half of the
// exponent: a block's sum d is taken times the first and, as it is added, times the second.  d is 0
// or 2^-25 to 2^32 in size, so either the first product is exact (halves of -101 to 95) or the
// whole one is beyond fp32 in the same direction.  (The one factor 2^(eX + eW) is infinite past 127,
// which turns 0 into NaN and loses what codes below 1 bring back, and 0 below -149, where d still
// brings products back.)
QDEV float2 s8_factors(uint32_t bx, uint32_t bw) {
  if (bx == kF8NanScale || bw == kF8NanScale) return make_float2(f8_scale(kF8NanScale), 1.0f);
  const uint32_t sum = bx + bw;
  return make_float2(f8_scale(sum >> 1), f8_scale(sum - (sum >> 1)));
}

// XE5M2: format of X.
template <bool XE5M2>
__global__ void __launch_bounds__(kS8RegThreads, 2)
    fp8_skinny_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                      const __grid_constant__ CUtensorMap tm_b,
                      const __grid_constant__ Skinny8Params p) {
  extern __shared__ __align__(16) uint8_t s8_raw[];
  uint8_t *sm = s8_raw + ((1024u - (smem_u32(s8_raw) & 1023u)) & 1023u);
  uint8_t *sX = sm + kS8Stages * kS8BoxBytes;
  uint16_t *sB = reinterpret_cast<uint16_t *>(sm + p.off_b);          // [r][R]
  float *sRecv = reinterpret_cast<float *>(sm + p.off_recv);          // [C ranks][R rows][M tokens]
  float *sXA = reinterpret_cast<float *>(sm + p.off_xa);              // [M][r]
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + p.off_bar);
  uint64_t *empty = full + kS8Stages;
  uint64_t *x_full = empty + kS8Stages;
  uint64_t *bar_b = x_full + kS8Stages;
  int *abort_flag = reinterpret_cast<int *>(bar_b + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int C = static_cast<int>(gridDim.x), R = kS8Rows / C;
  const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int nb_all = p.K >> 7;
  const int b0 = min(nb_all, rank * p.blocks), nb = min(nb_all, b0 + p.blocks) - b0;
  const int w0 = static_cast<int>(blockIdx.y) * kS8Rows;
  const int pg = ((g & 1) << 2) | (g >> 1);
  const int ra = warp * 16 + pg;                     // first of a product lane's two weight rows, ra and ra + 8
  const Waiter wt{abort_flag, p.limit_ns};
  volatile int no_abort = 0;
  const Waiter final_wt{&no_abort, drain_limit_ns(p.limit_ns)};

  if (tid == 0) {
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_x);
    for (int i = 0; i < kS8Stages; ++i) { mbar_init(&full[i], 2); mbar_init(&empty[i], 8); mbar_init(&x_full[i], 1); }
    mbar_init(bar_b, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (C > 1) cluster_arrive();
  pdl_trigger();

  if (warp == 8) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      bool ok = true;
      int s = 0;
      uint32_t ph = 1;
      for (int i = 0; i < nb; ++i) {
        if (!wait_bar(&empty[s], ph, wt)) { ok = false; break; }
        if (i >= kS8Stages) fence_proxy_async_smem();   // generic reads of the slot before its TMA refill
        mbar_arrive_expect_tx(&full[s], kS8BoxBytes);
        tma_load_2d(sm + s * kS8BoxBytes, &tm_w, &full[s], (b0 + i) * 128, w0);
        mbar_arrive_expect_tx(&x_full[s], kS8XCodes);
        tma_load_2d(sX + s * kS8XBytes, &tm_x, &x_full[s], (b0 + i) * 128, 0);
        if (i == 0 && p.r) {
          mbar_arrive_expect_tx(bar_b, static_cast<uint32_t>(p.r * R * 2));
          tma_load_2d(sB, &tm_b, bar_b, w0 + rank * R, 0);
        }
        if (++s == kS8Stages) { s = 0; ph ^= 1u; }
      }
      if (nb == 0 && p.r) {
        mbar_arrive_expect_tx(bar_b, static_cast<uint32_t>(p.r * R * 2));
        tma_load_2d(sB, &tm_b, bar_b, w0 + rank * R, 0);
      }
      // every copy has landed before the block may end (bounded)
      if (ok) {
        for (int i = max(0, nb - kS8Stages); i < nb; ++i) {
          wait_bar(&full[i % kS8Stages], static_cast<uint32_t>((i / kS8Stages) & 1), final_wt);
          wait_bar(&x_full[i % kS8Stages], static_cast<uint32_t>((i / kS8Stages) & 1), final_wt);
        }
      } else {
        for (int i = 0; i < 200; ++i) __nanosleep(1000);
      }
    }
  } else if (warp == 11) {
    // ------------------------------------------------------------ XA
    // the sum of the parts, once the kernel before has finished
    pdl_wait();
    // (r is a multiple of 8: four values at a time, every part's load issued before the sum)
    const int n4 = (p.M * p.r) >> 2;
#pragma unroll 2
    for (int i = lane; i < n4; i += 32) {
      float4 pa[kS8MaxXaParts], v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < kS8MaxXaParts; ++q) pa[q] = q < p.xa_parts ? ld_global_f4(p.xa + 4 * (q * n4 + i)) : v;
#pragma unroll
      for (int q = 0; q < kS8MaxXaParts; ++q) { v.x += pa[q].x; v.y += pa[q].y; v.z += pa[q].z; v.w += pa[q].w; }
      reinterpret_cast<float4 *>(sXA)[i] = v;
      if (p.xa_out && blockIdx.x == 0 && blockIdx.y == 0) reinterpret_cast<float4 *>(p.xa_out)[i] = v;
    }
  } else if (warp >= 9) {
    // ------------------------------------------------------------ X
    // lane (g, c) converts 16 codes of token g at columns 64 h + 16 c of a block; lane t < 8 makes the
    // factors of token t with the weight block's, from bytes requested 2 kAhead blocks before.
    // Warp 9 + j takes the blocks i with i mod 2 = j (the ring is even, so its slots are its own).
    constexpr int kAhead = 2;
    static_assert(kS8Stages % 2 == 0, "a ring slot belongs to one X warp");
    const int j0 = warp - 9;
    uint32_t fx[kAhead], fw[kAhead];
    const uint8_t *px = p.xs + static_cast<int64_t>(min(lane, p.M - 1)) * p.pitch + b0;
    const uint8_t *pw = p.ws + static_cast<int64_t>(blockIdx.y) * p.pitch + b0;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = j0 + 2 * u;
      fx[u] = i < nb ? ld_global_u8(px + i) : 0u;
      fw[u] = i < nb ? ld_global_u8(pw + i) : 0u;
    }
    int s = j0;
    uint32_t ph = 0;
    bool ok = true;
    for (int i0 = j0; ok && i0 < nb; i0 += 2 * kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + 2 * u;
        if (!ok || i >= nb) continue;
        const float2 f = s8_factors(fx[u], fw[u]);
        if (i + 2 * kAhead < nb) {
          fx[u] = ld_global_u8(px + i + 2 * kAhead);
          fw[u] = ld_global_u8(pw + i + 2 * kAhead);
        }
        // the slot's product warps are done with it: its copies were issued after they were
        ok = wait_bar_warp(&x_full[s], ph, wt);
        if (!ok) continue;
        const uint32_t src = smem_u32(sX + s * kS8XBytes) + static_cast<uint32_t>(g * 128 + 16 * c);
        const uint32_t dst = smem_u32(sX + s * kS8XBytes + kS8XCodes) + lane * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 x = ld_shared_v4(src + h * 64);
          uint32_t o[8];
          f8_to_f16x2<XE5M2>(x.x, o[0], o[1]);
          f8_to_f16x2<XE5M2>(x.y, o[2], o[3]);
          f8_to_f16x2<XE5M2>(x.z, o[4], o[5]);
          f8_to_f16x2<XE5M2>(x.w, o[6], o[7]);
          st_shared_v4(dst + h * 1024, o[0], o[1], o[2], o[3]);
          st_shared_v4(dst + h * 1024 + 512, o[4], o[5], o[6], o[7]);
        }
        if (lane < kS8MaxTokens) reinterpret_cast<float2 *>(sX + s * kS8XBytes + kS8XCodes + kS8XFrags)[lane] = f;
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
        s += 2;
        if (s >= kS8Stages) { s -= kS8Stages; ph ^= 1u; }
      }
    }
  } else {
    // ------------------------------------------------------------ products
    // Fragment rows g and g + 8 of a warp are weight rows perm(g) and 8 + perm(g) of its 16:
    // neighbouring g differ in bit 2 of the row, so the eight lanes of a shared-memory
    // phase (two rows, four pieces) fall on eight distinct 16-byte columns of the 128B swizzle.
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    const uint32_t row0 = smem_u32(sm) + static_cast<uint32_t>(ra * 128);
    const uint32_t ch0 = static_cast<uint32_t>((c ^ pg) << 4), ch1 = static_cast<uint32_t>(((4 + c) ^ pg) << 4);   // ra & 7 = pg
    const uint32_t x0 = smem_u32(sX) + kS8XCodes + lane * 16;
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < nb; ++i) {
      if (!wait_bar_warp(&full[s], ph, wt)) break;
      const uint32_t row = row0 + static_cast<uint32_t>(s * kS8BoxBytes), xb = x0 + static_cast<uint32_t>(s * kS8XBytes);
      uint4 wa[2], wb[2], xv[2][2];
      wa[0] = ld_shared_v4(row + ch0);
      wb[0] = ld_shared_v4(row + 8 * 128 + ch0);
      wa[1] = ld_shared_v4(row + ch1);
      wb[1] = ld_shared_v4(row + 8 * 128 + ch1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        xv[h][0] = ld_shared_v4(xb + h * 1024);
        xv[h][1] = ld_shared_v4(xb + h * 1024 + 512);
      }
      const float4 f = reinterpret_cast<const float4 *>(sX + s * kS8XBytes + kS8XCodes + kS8XFrags)[c];   // tokens 2c, 2c + 1
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t va[4] = {wa[h].x, wa[h].y, wa[h].z, wa[h].w}, vb[4] = {wb[h].x, wb[h].y, wb[h].z, wb[h].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a[4];
          f8_to_f16x2<false>(va[w], a[0], a[2]);
          f8_to_f16x2<false>(vb[w], a[1], a[3]);
          const uint4 q = xv[h][w >> 1];
          mma_16816_f16(d, a, (w & 1) ? q.z : q.x, (w & 1) ? q.w : q.y);
        }
      }
      acc[0] = fmaf(d[0] * f.x, f.y, acc[0]);
      acc[1] = fmaf(d[1] * f.z, f.w, acc[1]);
      acc[2] = fmaf(d[2] * f.x, f.y, acc[2]);
      acc[3] = fmaf(d[3] * f.z, f.w, acc[3]);
      if (++s == kS8Stages) { s = 0; ph ^= 1u; }
    }
    // push the partial rows to the rank that finishes them, [this rank][row][token], once the
    // cluster's CTAs have all started
    __syncwarp();
    if (C > 1) cluster_wait();
    const uint32_t recv = smem_u32(sRecv);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = ra + 8 * h, owner = row / R;
      const uint32_t base = recv + 4u * static_cast<uint32_t>((rank * R + row % R) * p.M);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tk = 2 * c + e;
        if (tk < p.M)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_rank(base + 4u * tk, static_cast<uint32_t>(owner))),
                       "f"(acc[2 * h + e])
                       : "memory");
      }
    }
  }
  if (warp >= 8) {
    __syncwarp();
    if (C > 1) cluster_wait();
  }
  pdl_wait();   // before the first write of Y
  if (p.r) wait_bar_warp(bar_b, 0, final_wt);
  if (C > 1) cluster_sync_all(); else __syncthreads();
  // L lanes finish an output, as many as leave one round for the CTA's first 256 threads: lane e
  // adds the partials of the ranks q mod L = e and the terms j mod L = e of the rank-r product,
  // then the lanes are added pairwise.  (One lane alone took 128 dependent steps at r 128; more
  // rounds take issue slots from the CTA beside.)
  int lg = 0;
  while (lg < 3 && (R * p.M << (lg + 1)) <= 256) ++lg;
  const int L = 1 << lg, e = tid & (L - 1), lr = 31 - __clz(R);   // C, and with it R, is a power of two
  for (int i = tid >> lg; i < R * p.M; i += kS8Threads >> lg) {
    const int tk = i >> lr, rr = i & (R - 1);
    float v = 0.f, lora = 0.f;
    for (int q = e; q < C; q += L) v += sRecv[(q * R + rr) * p.M + tk];
#pragma unroll 8
    for (int j = e; j < p.r; j += L)
      lora = fmaf(sXA[tk * p.r + j], __uint_as_float(static_cast<uint32_t>(sB[j * R + rr]) << 16), lora);
    if (p.r) v = fmaf(p.s, lora, v);
    // (a warp leaves the loop whole: R M is a multiple of 16, 32 / L lanes' worth of outputs at L > 1)
    for (int d = L >> 1; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    const __nv_bfloat16 h = __float2bfloat16_rn(v);
    if (e == 0) p.Y[static_cast<int64_t>(tk) * p.N + w0 + rank * R + rr] = *reinterpret_cast<const uint16_t *>(&h);
  }
}

}  // namespace qlora
