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
// share a block and agree on its maximum by two lane exchanges.  Rows whose length
// is no multiple of eight, and addresses that are no multiple of a lane's bytes,
// take the same kernels: gfx950's vector loads and stores need no alignment beyond
// the element's.  A row's last lane then has fewer than eight channels; it loads
// eight (the memory behind them is the next row's; the last row's lane takes them
// one by one) and stores its own in pieces of 4, 2 and 1 (TAIL; where no row has such
// a lane the test for it is left out, which is worth a tenth in small calls).
//
// Measured, us: 32768 rows of 2048 bf16 (207 MB) pack 34, unpack 32 where the same rows
// come again and are in part in the caches (a copy there, 8 TB/s: 26), 40 and 38 with two
// sets in turn; 262144 rows 383 and 354 (from memory, 4.2 and 4.6 TB/s); 65536 of 1001 34
// and 34, where a lane per channel took 135 and 73.  Next to memory it is the VALU: 18
// operations per channel in pack, with clamps, conversions and shifts of their own for each
// code, were 37 us at the first size.  fp32, the same two sizes of 2048 channels: pack 62 (65
// in turn) and 578, unpack 95 and 735 (4.7 and 3.7 TB/s).
#pragma once
#include <type_traits>

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
// 1 / scale (0 for a block of NaN: its codes are taken as 0).
__device__ __forceinline__ float pack_inverse(uint32_t b) { return b == 255u ? 0.f : __uint_as_float((254u - b) << 23); }
// A code in the low byte (what is above it is of no use).  x / s is at most 127, and just
// below 128 where the scale is at its upper end: held to 127, then 1.5 * 2^23 added, which
// rounds to the nearest integer, ties to even, and leaves it in the low bits, in two's
// complement.
__device__ __forceinline__ uint32_t pack_code(float x, float inverse) {
  return __float_as_uint(__builtin_amdgcn_fmed3f(x * inverse, -127.f, 127.f) + 12582912.f);
}
// Four codes' low bytes in a word: byte selectors 0..3 take from the second operand, 4..7
// from the first, 12 gives 0.
__device__ __forceinline__ uint32_t pack_word(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0c0c0400u), __builtin_amdgcn_perm(b, a, 0x0c0c0400u), 0x05040100u);
}

typedef uint32_t u32x4_e2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_e4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_e1 __attribute__((ext_vector_type(2), aligned(1)));

// Eight channels of E as loaded from an address aligned to the element; `n` < 8: of those
// only n, one by one, the others 0.
template <typename E> struct Oct {
  uint32_t w[2 * sizeof(E)];
  __device__ __forceinline__ void load(const E* p) {
    using V = std::conditional_t<sizeof(E) == 2, u32x4_e2, u32x4_e4>;
#pragma unroll
    for (int k = 0; k < (int)sizeof(E) / 2; ++k) {
      const u32x4 q = reinterpret_cast<const V*>(p)[k];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[4 * k + i] = q[i];
    }
  }
  __device__ __forceinline__ void load(const E* p, int n) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if constexpr (sizeof(E) == 4) {
        w[k] = k < n ? reinterpret_cast<const uint32_t*>(p)[k] : 0u;
      } else {
        const uint32_t v = k < n ? reinterpret_cast<const uint16_t*>(p)[k] : 0u;
        w[k >> 1] = (k & 1) ? w[k >> 1] | v << 16 : v;
      }
    }
  }
  __device__ __forceinline__ float operator[](int k) const {
    if constexpr (sizeof(E) == 2) return (k & 1) ? bf16_hi(w[k >> 1]) : bf16_lo(w[k >> 1]);
    else return __uint_as_float(w[k]);
  }
};

// Any C >= 8.  Lane groups of four per block; `vpr` = 4 * ceil(C / 32) places of eight
// channels per row, those at or beyond C hold nothing.  rows * vpr < 2^31.
template <typename E, bool TAIL>
__global__ __launch_bounds__(256) void gdn_pack8_vec_kernel(const E* __restrict__ x, int64_t ld,
                                                            int8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales,
                                                            uint32_t rows, int C, uint32_t vpr) {
  const uint32_t total = rows * vpr, step = gridDim.x * 256u;
  const uint32_t nblk = vpr >> 2;
  for (uint32_t i0 = blockIdx.x * 256u + threadIdx.x; i0 < total; i0 += step * kPackUnroll) {
    Oct<E> w[kPackUnroll];
    uint32_t row[kPackUnroll], v[kPackUnroll];
    int cnt[kPackUnroll];  // channels of the lane's own
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
      const uint32_t i = i0 + u * step;
      // i0 + u * step may pass total (and, near 2^32, wrap): both hold nothing
      const bool any = i < total && i >= i0;
      row[u] = any ? i / vpr : 0;
      v[u] = any ? i - row[u] * vpr : 0;
      cnt[u] = any ? min(max(C - (int)(v[u] * 8), 0), 8) : 0;
      if (!TAIL) cnt[u] = cnt[u] ? 8 : 0;
      const E* q = x + (int64_t)row[u] * ld + (cnt[u] ? v[u] * 8 : 0);  // (without channels: the row's first)
      if (TAIL && (cnt[u] & 7) && row[u] == rows - 1) w[u].load(q, cnt[u]);
      else w[u].load(q);
    }
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t e = __float_as_uint(w[u][k]) & 0x7fffffffu;
        m = max(m, !TAIL || k < cnt[u] ? e : 0u);
      }
      if (!TAIL) m = cnt[u] ? m : 0u;
      // lanes xor 1, then xor 2 (quad permutations)
      m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xf, 0xf, true));
      m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xf, 0xf, true));
      const uint32_t b = pack_byte(m);
      const float inverse = pack_inverse(b);
      u32x2 c;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        c[k] = pack_word(pack_code(w[u][4 * k], inverse), pack_code(w[u][4 * k + 1], inverse),
                         pack_code(w[u][4 * k + 2], inverse), pack_code(w[u][4 * k + 3], inverse));
      if (b == 255u) c = {0, 0};
      uint8_t* q = reinterpret_cast<uint8_t*>(codes) + (int64_t)row[u] * C + v[u] * 8;
      if (cnt[u] == 8) {
        *reinterpret_cast<u32x2_e1*>(q) = c;
      } else if (TAIL && cnt[u]) {
        uint32_t d = c.x;
        if (cnt[u] & 4) {
          __builtin_memcpy(q, &d, 4);
          d = c.y;
          q += 4;
        }
        if (cnt[u] & 2) {
          const uint16_t h = (uint16_t)d;
          __builtin_memcpy(q, &h, 2);
          d >>= 16;
          q += 2;
        }
        if (cnt[u] & 1) *q = (uint8_t)d;
      }
      if (cnt[u] && (v[u] & 3) == 0) scales[(int64_t)row[u] * nblk + (v[u] >> 2)] = (uint8_t)b;
    }
  }
}

// Rows of fewer than eight channels: 32 lanes per block, one channel each.
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
    if (c < C) codes[row * C + c] = b == 255u ? (int8_t)0 : (int8_t)pack_code(f, pack_inverse(b));
    if (l == 0) scales[i] = (uint8_t)b;
  }
}

// The values a checkpoint stands for, rows contiguous.  Any C >= 8: `vpr` = ceil(C / 8)
// places of eight channels per row; rows * vpr < 2^31.
template <typename E, bool TAIL>
__global__ __launch_bounds__(256) void gdn_unpack8_vec_kernel(const int8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales,
                                                              E* __restrict__ y, uint32_t rows, int C,
                                                              uint32_t vpr, uint32_t nblk) {
  const uint32_t total = rows * vpr, step = gridDim.x * 256u;
  for (uint32_t i0 = blockIdx.x * 256u + threadIdx.x; i0 < total; i0 += step * kPackUnroll) {
    u32x2 c[kPackUnroll];
    uint32_t b[kPackUnroll];
    int64_t at[kPackUnroll];
    int cnt[kPackUnroll];
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
      const uint32_t i = i0 + u * step;
      const bool any = i < total && i >= i0;
      const uint32_t j = any ? i : i0, row = j / vpr, v = j - row * vpr;
      const int own = TAIL ? min(C - (int)(v * 8), 8) : 8;
      cnt[u] = any ? own : 0;
      at[u] = (int64_t)row * C + v * 8;
      const uint8_t* q = reinterpret_cast<const uint8_t*>(codes) + at[u];
      if (TAIL && own < 8 && row == rows - 1) {
        c[u] = {0, 0};
#pragma unroll
        for (int k = 0; k < 7; ++k)
          if (k < own) c[u][k >> 2] |= (uint32_t)q[k] << (8 * (k & 3));
      } else {
        c[u] = *reinterpret_cast<const u32x2_e1*>(q);
      }
      b[u] = scales[(int64_t)row * nblk + (v >> 2)];
    }
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
      if (!cnt[u]) continue;
      const float s = pack_scale(b[u]);
      float f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = (float)(int8_t)(c[u][k >> 2] >> (8 * (k & 3))) * s;
      E* q = y + at[u];
      typedef E E4 __attribute__((ext_vector_type(4), aligned(sizeof(E))));
      typedef E E2 __attribute__((ext_vector_type(2), aligned(sizeof(E))));
      if (!TAIL || cnt[u] == 8) {
        if constexpr (sizeof(E) == 2) {
          typedef E E8 __attribute__((ext_vector_type(8), aligned(2)));
          *reinterpret_cast<E8*>(q) = E8{(E)f[0], (E)f[1], (E)f[2], (E)f[3], (E)f[4], (E)f[5], (E)f[6], (E)f[7]};
        } else {
          reinterpret_cast<E4*>(q)[0] = E4{f[0], f[1], f[2], f[3]};
          reinterpret_cast<E4*>(q)[1] = E4{f[4], f[5], f[6], f[7]};
        }
        continue;
      }
      if (cnt[u] & 4) {
        *reinterpret_cast<E4*>(q) = E4{(E)f[0], (E)f[1], (E)f[2], (E)f[3]};
        f[0] = f[4];
        f[1] = f[5];
        f[2] = f[6];
        q += 4;
      }
      if (cnt[u] & 2) {
        *reinterpret_cast<E2*>(q) = E2{(E)f[0], (E)f[1]};
        f[0] = f[2];
        q += 2;
      }
      if (cnt[u] & 1) *q = (E)f[0];
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
