// gdn_pack8.h -- activation checkpoints in 8 bits on gfx950.
//
// A row's channels are held in blocks of 32 (the last one may be shorter): one
// byte b for the block's scale s = 2^(b - 127), the least power of two with
// max|x| <= 127 s (at least 2^-126, at most 2^121), and one signed byte per
// channel, the quotient x / s rounded to the nearest integer, ties to even, and
// held to [-127, 127].  A power of two makes the quotient, and the value
// code * s that the checkpoint stands for, exact: the only rounding is that to
// the integer, by at most s/2 <= max|x| / 127.  (Scales max|x|/127 would round
// by up to half as much, but the stored value then depends on the order of two
// more roundings, and the scale takes four bytes instead of one.)
// A block that holds an infinity or a NaN stores b = 255 and stands for NaN.
//
// Copy-bound: e + 1 + 1/32 bytes per element each way.  Eight channels per lane,
// so a lane's load is 16 bytes of bf16 (32 of fp32) and its codes 8; four lanes
// share a block and agree on its maximum by two lane exchanges.
#pragma once
#include "gdn_layer.h"

namespace gdn {

constexpr int kPackUnroll = 4;  // vectors in flight per thread

// The scale byte of a block whose largest |x| has the bits m.
__device__ __forceinline__ uint32_t pack_byte(uint32_t m) {
  if (m >= 0x7f800000u) return 255u;
  // max = f 2^k: 127 2^(k-6) holds it if f <= 127/64, else 127 2^(k-5) does
  const int b = (int)(m >> 23) - 6 + ((m & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return (uint32_t)min(max(b, 1), 248);
}
__device__ __forceinline__ int pack_code(float x, uint32_t b) {
  if (b == 255u) return 0;
  const float q = rintf(x * __uint_as_float((254u - b) << 23));
  return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// Vectors of 8 channels: C % 8 == 0, ld % 8 == 0, 16-byte aligned x.  Lane groups
// of four per block; `vpr` = 4 * ceil(C / 32) vector places per row, those at or
// beyond C / 8 hold nothing.  rows * vpr < 2^31.
template <typename E>
__global__ __launch_bounds__(256) void gdn_pack8_vec_kernel(const E* __restrict__ x, int64_t ld,
                                                            int8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales,
                                                            uint32_t rows, int C, uint32_t vpr) {
  const uint32_t total = rows * vpr, step = gridDim.x * 256u;
  const uint32_t nblk = vpr >> 2;
  for (uint32_t i0 = blockIdx.x * 256u + threadIdx.x; i0 < total; i0 += step * kPackUnroll) {
    u32x4 w[kPackUnroll][sizeof(E) / 2];
    uint32_t row[kPackUnroll], v[kPackUnroll];
    bool in[kPackUnroll];
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
      const uint32_t i = i0 + u * step;
      // i0 + u * step may pass total (and, near 2^32, wrap): both hold nothing
      const bool any = i < total && i >= i0;
      row[u] = any ? i / vpr : 0;
      v[u] = any ? i - row[u] * vpr : 0;
      in[u] = any && (int)(v[u] * 8) < C;
      const u32x4* q = reinterpret_cast<const u32x4*>(x + (int64_t)row[u] * ld + v[u] * 8);
#pragma unroll
      for (int k = 0; k < (int)sizeof(E) / 2; ++k) w[u][k] = in[u] ? q[k] : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
      float f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (sizeof(E) == 2) f[k] = (k & 1) ? bf16_hi(w[u][0][k >> 1]) : bf16_lo(w[u][0][k >> 1]);
        else f[k] = __uint_as_float(w[u][k >> 2][k & 3]);
      }
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(f[k]) & 0x7fffffffu);
      // lanes xor 1, then xor 2 (quad permutations)
      m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xf, 0xf, true));
      m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xf, 0xf, true));
      const uint32_t b = pack_byte(m);
      u32x2 c = {0, 0};
#pragma unroll
      for (int k = 0; k < 8; ++k) c[k >> 2] |= ((uint32_t)pack_code(f[k], b) & 255u) << (8 * (k & 3));
      if (in[u]) {
        *reinterpret_cast<u32x2*>(codes + (int64_t)row[u] * C + v[u] * 8) = c;
        if ((v[u] & 3) == 0) scales[(int64_t)row[u] * nblk + (v[u] >> 2)] = (uint8_t)b;
      }
    }
  }
}

// Any C, stride and alignment: 32 lanes per block, one channel each.
template <typename E>
__global__ __launch_bounds__(256) void gdn_pack8_scalar_kernel(const E* __restrict__ x, int64_t ld,
                                                               int8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales,
                                                               int64_t rows, int C, int nblk) {
  const int64_t total = rows * nblk, step = (int64_t)gridDim.x * 8;
  const int l = threadIdx.x & 31;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += step) {
    const int64_t row = i / nblk;
    const int c = (int)(i - row * nblk) * kPackBlock + l;
    const float f = c < C ? (float)x[row * ld + c] : 0.f;
    uint32_t m = __float_as_uint(f) & 0x7fffffffu;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 32));
    const uint32_t b = pack_byte(m);
    if (c < C) codes[row * C + c] = (int8_t)pack_code(f, b);
    if (l == 0) scales[i] = (uint8_t)b;
  }
}

// The values a checkpoint stands for, rows contiguous.  Vectors of 8 channels:
// C % 8 == 0, 16-byte aligned y, 8-byte aligned codes; rows * C / 8 < 2^31.
template <typename E>
__global__ __launch_bounds__(256) void gdn_unpack8_vec_kernel(const int8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales,
                                                              E* __restrict__ y, uint32_t rows,
                                                              uint32_t vpr, uint32_t nblk) {
  const uint32_t total = rows * vpr, step = gridDim.x * 256u;
  for (uint32_t i0 = blockIdx.x * 256u + threadIdx.x; i0 < total; i0 += step * kPackUnroll) {
    u32x2 c[kPackUnroll];
    uint32_t b[kPackUnroll];
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
      const uint32_t i = i0 + u * step;
      const bool any = i < total && i >= i0;
      const uint32_t j = any ? i : i0;
      const uint32_t row = j / vpr;
      c[u] = reinterpret_cast<const u32x2*>(codes)[j];
      b[u] = scales[(int64_t)row * nblk + ((j - row * vpr) >> 2)];
    }
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
      const uint32_t i = i0 + u * step;
      if (!(i < total && i >= i0)) continue;
      const float s = pack_scale(b[u]);
      float f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = (float)(int8_t)(c[u][k >> 2] >> (8 * (k & 3))) * s;
      E* q = y + (int64_t)i * 8;
      if constexpr (sizeof(E) == 2) {
        vec_store<E, 8>(q, f);
      } else {
        reinterpret_cast<f32x4*>(q)[0] = f32x4{f[0], f[1], f[2], f[3]};
        reinterpret_cast<f32x4*>(q)[1] = f32x4{f[4], f[5], f[6], f[7]};
      }
    }
  }
}

template <typename E>
__global__ __launch_bounds__(256) void gdn_unpack8_scalar_kernel(const int8_t* __restrict__ codes,
                                                                 const uint8_t* __restrict__ scales,
                                                                 E* __restrict__ y, int64_t n, int C,
                                                                 int nblk) {
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
    const int64_t row = i / C;
    const int c = (int)(i - row * C);
    y[i] = (E)((float)codes[i] * pack_scale(scales[row * nblk + (c >> 5)]));
  }
}

}  // namespace gdn
