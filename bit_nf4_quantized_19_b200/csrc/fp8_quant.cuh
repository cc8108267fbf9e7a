// Blockwise 8-bit floating point: quantizers and dequant (sm_100a).
//
// A block's values are e4m3 (or e5m2) codes times one power of two 2^e, stored as the
// byte e + 127:
//   e      = the smallest integer >= -127 with amax <= FMAX 2^e   (FMAX 448, or 57344),
//   code_i = RNE(x_i 2^-e)     (x_i 2^-e is exact in fp32, so this is the only rounding).
// Blocks are 128 values along a row (activations, gradients) or 128 x 128 values
// (weights).  A power of two costs at most one of the format's 16 (or 30) binades against an
// exact amax / FMAX and buys three things: the codes are reproducible bit for bit, the
// tensor core applies the factors itself (block-scaled MMA), and code 2^e is exact in
// bf16.  FMAX = 1.75 2^8 (2^15), so with amax = 1.f 2^k the smallest e is k - 8 (k - 15),
// plus one when f > 0.75: one integer add on the fp32 bits.
//
// All three kernels stream: 2 bytes in and 1 out per value (or the reverse), so HBM
// bounds them.  Eight lanes share a block of 128 (two 16-byte loads each, the 8 lanes'
// loads contiguous), the amax is a packed integer maximum over |bf16| bits and three
// shuffles, and the values wait in registers: one pass over the data.  Measured: 8192 x 22016
// 91 us (5.9 TB/s, of 6.45 for a copy), a 22016 x 8192 weight 83 us (6.5), one row of 4096 1.5 us
// replayed in a graph; dequant of 8192 x 22016 82 us (6.6), of 8192 x 8192 33 (6.1).
#pragma once
#include "common.cuh"
#include "pipeline.cuh"

namespace qlora {

constexpr int kF8Block = 128;
constexpr int kF8Threads = 256;
constexpr int kF8Unroll = 4;              // blocks in flight per 8-lane group
constexpr uint8_t kF8NanScale = 255;      // the exponent byte of a block with a non-finite value
constexpr uint32_t kF8NanCodes = 0x7F7F7F7Fu;   // NaN in e4m3 and in e5m2

// Row pitch in bytes of the exponent bytes of `cols` columns: one per 128 columns, padded
// so that each group of four (512 columns) is an aligned 32-bit word.
__host__ __device__ constexpr int64_t f8_pitch(int64_t cols) { return 4 * ((cols + 511) / 512); }

// Exponent byte of a block from the bf16 magnitude bits of its amax (finite).
template <bool E5M2>
QDEV uint32_t f8_exp_byte(uint32_t amax16) {
  const int b = static_cast<int>(((amax16 << 16) + 0x1FFFFFu) >> 23) - (E5M2 ? 15 : 8);
  return static_cast<uint32_t>(max(b, 0));
}
// 2^(127 - byte): the factor x is multiplied by (byte <= 247, so the result is normal).
QDEV float f8_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// 2^(byte - 127); byte 0 is the subnormal 2^-127, byte 255 gives NaN.
QDEV float f8_scale(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

// Two fp32 values -> two codes (lo in bits 0-7).
template <bool E5M2>
QDEV uint32_t f8_pack2(float lo, float hi) {
  uint16_t r;
  if (E5M2) asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two codes (bits 0-7, 8-15) -> two fp32 values (exact).
template <bool E5M2>
QDEV float2 f8_unpack2(uint32_t w) {
  uint32_t h;
  const uint16_t c = static_cast<uint16_t>(w);
  if (E5M2) asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(c));
  else asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// |bf16| maximum of a packed pair (the bits of non-negative bf16 order like integers,
// NaN and infinity above every finite value).
QDEV uint32_t f8_amax2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }
QDEV uint32_t f8_amax8(uint32_t m, const uint4 &v) {
  return f8_amax2(f8_amax2(f8_amax2(f8_amax2(m, v.x), v.y), v.z), v.w);
}
// Eight bf16 -> eight codes.
template <bool E5M2>
QDEV uint2 f8_encode8(const uint4 &v, float inv) {
  auto four = [inv](uint32_t a, uint32_t b) {
    return f8_pack2<E5M2>(bf16_lo(a) * inv, bf16_hi(a) * inv) |
           (f8_pack2<E5M2>(bf16_lo(b) * inv, bf16_hi(b) * inv) << 16);
  };
  return make_uint2(four(v.x, v.y), four(v.z, v.w));
}
// Eight codes -> eight bf16, times a power of two.
template <bool E5M2>
QDEV uint4 f8_decode8(uint2 c, float scale) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = f8_unpack2<E5M2>(((i & 2) ? c.y : c.x) >> (16 * (i & 1)));
    o[i] = pack_bf16x2(f.x * scale, f.y * scale);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

struct Fp8QuantParams {
  const uint16_t *x;    // bf16 [rows, cols], cols a multiple of 8
  uint8_t *codes;       // [rows, cols]
  uint8_t *scales;      // [rows, pitch]
  int cols;
  int kb;               // blocks per row, ceil(cols / 128)
  int pitch;
  uint32_t blocks;      // rows * kb
};

// Activations: 128-value blocks along the rows.
template <bool E5M2>
__global__ void __launch_bounds__(kF8Threads) fp8_quantize_kernel(const __grid_constant__ Fp8QuantParams p) {
  pdl_trigger();
  pdl_wait();
  const int g = threadIdx.x >> 3, sub = threadIdx.x & 7;
  constexpr uint32_t kGroups = kF8Threads / 8;
  uint32_t row[kF8Unroll];
  int col[kF8Unroll];
  uint4 v[kF8Unroll][2];
  const uint32_t first = blockIdx.x * (kGroups * kF8Unroll) + static_cast<uint32_t>(g);
#pragma unroll
  for (int u = 0; u < kF8Unroll; ++u) {
    const uint32_t blk = first + u * kGroups;
    row[u] = blk / static_cast<uint32_t>(p.kb);
    col[u] = static_cast<int>(blk - row[u] * static_cast<uint32_t>(p.kb));
    const uint16_t *src = p.x + static_cast<int64_t>(row[u]) * p.cols + col[u] * kF8Block + sub * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v[u][h] = make_uint4(0u, 0u, 0u, 0u);
      if (blk < p.blocks && col[u] * kF8Block + sub * 8 + h * 64 < p.cols) v[u][h] = ld_global_v4(src + h * 64);
    }
  }
  bool bad = false;
#pragma unroll
  for (int u = 0; u < kF8Unroll; ++u) {
    uint32_t m = f8_amax8(f8_amax8(0u, v[u][0]), v[u][1]);
    m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
    for (int o = 4; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t blk = first + u * kGroups;
    if (blk >= p.blocks) continue;
    const bool nan = m >= 0x7F80u;
    const uint32_t byte = nan ? kF8NanScale : f8_exp_byte<E5M2>(m);
    const float inv = f8_inv_scale(nan ? 127u : byte);
    uint8_t *dst = p.codes + static_cast<int64_t>(row[u]) * p.cols + col[u] * kF8Block + sub * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint2 c = f8_encode8<E5M2>(v[u][h], inv);
      if (nan) c = make_uint2(kF8NanCodes, kF8NanCodes);
      if (col[u] * kF8Block + sub * 8 + h * 64 < p.cols) *reinterpret_cast<uint2 *>(dst + h * 64) = c;
    }
    if (sub == 0) {
      uint8_t *sc = p.scales + static_cast<int64_t>(row[u]) * p.pitch;
      sc[col[u]] = static_cast<uint8_t>(byte);
      if (col[u] == p.kb - 1)
        for (int j = p.kb; j < p.pitch; ++j) sc[j] = 0;
    }
    bad = bad || nan;
  }
  if (bad) atomicOr(&g_device_status, kStatNonFinite);
}

// Weights: one CTA per 128 x 128 block (e4m3).  32 row slots x 8 lanes, four rows each.
__global__ void __launch_bounds__(kF8Threads) fp8_quantize_weight_kernel(const uint16_t *__restrict__ w, int rows,
                                                                         int cols, int pitch,
                                                                         uint8_t *__restrict__ codes,
                                                                         uint8_t *__restrict__ scales) {
  __shared__ uint32_t warp_max[kF8Threads / 32];
  const int tid = threadIdx.x, g = tid >> 3, sub = tid & 7;
  const int kb = (cols + kF8Block - 1) / kF8Block;
  const int bc = static_cast<int>(blockIdx.x % static_cast<unsigned>(kb));
  const int br = static_cast<int>(blockIdx.x / static_cast<unsigned>(kb));
  const int c0 = bc * kF8Block + sub * 8;
  uint4 v[4][2];
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = br * kF8Block + i * 32 + g;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v[i][h] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows && c0 + h * 64 < cols) v[i][h] = ld_global_nc_v4(w + static_cast<int64_t>(r) * cols + c0 + h * 64);
      m = f8_amax8(m, v[i][h]);
    }
  }
  m = max(m & 0xFFFFu, m >> 16);
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) warp_max[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kF8Threads / 32; ++i) m = max(m, warp_max[i]);
  const bool nan = m >= 0x7F80u;
  const uint32_t byte = nan ? kF8NanScale : f8_exp_byte<false>(m);
  const float inv = f8_inv_scale(nan ? 127u : byte);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = br * kF8Block + i * 32 + g;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint2 c = f8_encode8<false>(v[i][h], inv);
      if (nan) c = make_uint2(kF8NanCodes, kF8NanCodes);
      if (r < rows && c0 + h * 64 < cols)
        *reinterpret_cast<uint2 *>(codes + static_cast<int64_t>(r) * cols + c0 + h * 64) = c;
    }
  }
  if (tid == 0) {
    uint8_t *sc = scales + static_cast<int64_t>(br) * pitch;
    sc[bc] = static_cast<uint8_t>(byte);
    if (bc == kb - 1)
      for (int j = kb; j < pitch; ++j) sc[j] = 0;
    if (nan) atomicOr(&g_device_status, kStatNonFinite);
  }
}

// bf16 values of a quantized tensor.
struct Fp8DequantParams {
  const uint8_t *codes, *scales;
  uint16_t *out;
  int cols, kb, pitch;
  int row_shift;         // log2 of the block's rows: 0 or 7
  uint32_t blocks;       // rows * kb
};

template <bool E5M2>
__global__ void __launch_bounds__(kF8Threads) fp8_dequant_kernel(const __grid_constant__ Fp8DequantParams p) {
  const int g = threadIdx.x >> 3, sub = threadIdx.x & 7;
  constexpr uint32_t kGroups = kF8Threads / 8;
  const uint32_t first = blockIdx.x * (kGroups * kF8Unroll) + static_cast<uint32_t>(g);
  uint2 c[kF8Unroll][2];
  uint32_t sc[kF8Unroll];
  int64_t off[kF8Unroll];
  int col[kF8Unroll];
#pragma unroll
  for (int u = 0; u < kF8Unroll; ++u) {
    const uint32_t blk = first + u * kGroups;
    const uint32_t row = blk / static_cast<uint32_t>(p.kb);
    const int b = static_cast<int>(blk - row * static_cast<uint32_t>(p.kb));
    // blocks past the end are given a column past the end: no load and no store
    col[u] = blk < p.blocks ? b * kF8Block + sub * 8 : p.cols;
    off[u] = static_cast<int64_t>(row) * p.cols + col[u];
    sc[u] = blk < p.blocks ? p.scales[static_cast<int64_t>(row >> p.row_shift) * p.pitch + b] : 127u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (col[u] + h * 64 >= p.cols) continue;
      c[u][h] = __ldg(reinterpret_cast<const uint2 *>(p.codes + off[u] + h * 64));
    }
  }
#pragma unroll
  for (int u = 0; u < kF8Unroll; ++u) {
    const float f = f8_scale(sc[u]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (col[u] + h * 64 >= p.cols) continue;
      *reinterpret_cast<uint4 *>(p.out + off[u] + h * 64) = f8_decode8<E5M2>(c[u][h], f);
    }
  }
}

}  // namespace qlora
