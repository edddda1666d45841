// gdn_norm.h -- the norms around a block, on gfx950:
//
//     r(u) = u / sqrt(mean(u^2) + eps)   over the channels of a row
//     gated norm      y = r(x) w silu(z)  or  r(x silu(z)) w  or (no gate) r(x) w
//     residual norm   p = r(x) post_w  or  x;   s = residual + scale p;   h = r(s) w
//
// and their gradients.  With n = r(u) = u c, c = (mean(u^2) + eps)^-1/2, and dn the gradient
// towards n, that towards u is  c (dn - n mean(n dn)).
//
// Rows are independent and read once, so the passes are bound by memory.  A row is held in
// the registers of LPR lanes (of one wave, or of a workgroup), NV vectors of VEC channels
// each; all arithmetic is fp32 and every output is rounded once.  The weights' gradients are
// sums over all rows: a lane keeps its channels' sums over the rows that its workgroup walks,
// the workgroup writes them to its row of `partial`, and a second kernel adds those rows, in a
// fixed order.
//
// Measured (us and TB/s of a pass; 5.2 is a copy's, more comes from the caches), bf16: gated norm of
// B=4, T=8192, 16 heads of 128: 74 and 5.4; of a token of 64 sequences 3.0 (a launch).  Its backward
// pass, B=2, T=2048: 18.5 and 4.5, with 4.6 of sums.  Residual norm, T=5003, C=1000 fp32: 13.8 and
// 5.8; backward, B=4, T=4096, C=2048: 78 and 5.2, with 4.8 of sums.
#pragma once
#include "gdn_layer.h"

namespace gdn {

enum { kGateNone = 0, kGateAfter = 1, kGateFirst = 2 };

// VEC channels of a row as loaded.  Rows of any width are read and written 16 bytes at a time: the
// device takes such accesses at any element's address, and only the row's last vector, where `left`
// channels are fewer than VEC, is put together, zeros behind them (gated norm's backward pass over
// 8M channels in bf16 rows of 2049: 39 us, by single channels 961).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
template <int BYTES> struct RawBytes;
template <> struct RawBytes<32> { u32x4 a, b; };
template <> struct RawBytes<16> { u32x4 a; };
template <> struct RawBytes<4> { uint32_t a; };
template <> struct RawBytes<2> { uint16_t a; };
template <typename E, int VEC> struct Chan {
  RawBytes<VEC * (int)sizeof(E)> r;
  __device__ __forceinline__ void load(const E* p, int left) {
    if constexpr (VEC == 1) {
      r.a = *reinterpret_cast<const decltype(r.a)*>(p);
    } else if (left >= VEC) {
      r.a = *reinterpret_cast<const u32x4_any*>(p);
      if constexpr (sizeof(r) == 32) r.b = *reinterpret_cast<const u32x4_any*>(p + 4);
    } else if constexpr (sizeof(E) == 2) {  // the row's last VEC channels, moved down
      typedef unsigned __int128 bits;
      const bits v = __builtin_bit_cast(bits, (u32x4)*reinterpret_cast<const u32x4_any*>(p + left - VEC));
      r.a = __builtin_bit_cast(u32x4, v >> (16 * (VEC - left)));
    } else {
      uint32_t v[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = i < left ? __float_as_uint(p[i]) : 0;
      r.a = u32x4{v[0], v[1], v[2], v[3]};
      if constexpr (sizeof(r) == 32) r.b = u32x4{v[4], v[5], v[6], v[7]};
    }
  }
  __device__ __forceinline__ void zero() { r = {}; }
  __device__ __forceinline__ void get(float (&v)[VEC]) const {
    typedef E vec __attribute__((ext_vector_type(VEC)));
    if constexpr (VEC == 1) {
      v[0] = (float)__builtin_bit_cast(E, r.a);
    } else if constexpr (sizeof(r) == 32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(r.a[i]);
        v[4 + i] = __uint_as_float(r.b[i]);
      }
    } else {
      const vec x = __builtin_bit_cast(vec, r.a);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = (float)x[i];
    }
  }
};
template <typename E, int VEC> __device__ __forceinline__ void chan_store(E* p, const float (&v)[VEC], int left) {
  if constexpr (VEC == 1) {
    *p = (E)v[0];
  } else if (left < VEC) {
#pragma unroll
    for (int i = 0; i < VEC - 1; ++i)
      if (i < left) p[i] = (E)v[i];
  } else if constexpr (VEC * sizeof(E) == 32) {
    typedef float any __attribute__((ext_vector_type(4), aligned(4)));
    reinterpret_cast<any*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
    reinterpret_cast<any*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    typedef E vec __attribute__((ext_vector_type(VEC)));
    vec x;
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = (E)v[i];
    *reinterpret_cast<u32x4_any*>(p) = __builtin_bit_cast(u32x4, x);
  }
}

// Sum over the 16 lanes of a DPP row, in every lane (rotations by 8, 4, 2, 1).
__device__ __forceinline__ float row16_sum(float v) {
  auto rot = [](float x, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  v += rot(v, std::integral_constant<int, 0x128>{});
  v += rot(v, std::integral_constant<int, 0x124>{});
  v += rot(v, std::integral_constant<int, 0x122>{});
  v += rot(v, std::integral_constant<int, 0x121>{});
  return v;
}

// Sums over the LPR lanes that hold a row, in every one of them.  In workgroups of several
// waves per row, `slot` is LDS of two rows of waves: calls alternate between the two, so that
// one barrier per call is enough.
template <int LPR> struct RowSum {
  float (*slot)[LPR / 64 > 0 ? LPR / 64 : 1];
  int turn = 0;
  __device__ __forceinline__ float operator()(float v) {
    if constexpr (LPR == 8) {
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) v += __shfl_xor(v, d);
      return v;
    } else {
      v = row16_sum(v);
      if constexpr (LPR >= 32) v += __shfl_xor(v, 16);
      if constexpr (LPR >= 64) v += __shfl_xor(v, 32);
      if constexpr (LPR > 64) {
        constexpr int W = LPR / 64;
        if (lane_id() == 0) slot[turn][threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += slot[turn][w];
        turn ^= 1;
      }
      return v;
    }
  }
};

struct NormGeo {
  int64_t rows;      // of D channels; rows / H tokens
  int H, D;
  int64_t ldx, ldz;  // elements between tokens (residual norm: of x and of the residual)
  float eps;
  int mode;          // the gate's place
};

// Where a row begins in a tensor whose tokens are `ld` elements apart.
__device__ __forceinline__ int64_t norm_row(const NormGeo& g, int64_t row, int64_t ld) {
  if (ld == (int64_t)g.H * g.D) return row * g.D;
  const uint32_t t = (uint32_t)row / (uint32_t)g.H;  // (rows are below 2^31)
  return t * ld + ((uint32_t)row - t * g.H) * (int64_t)g.D;
}

// Channels of a row of D from c on, as a vector's load or store asks (WHOLE: D is a multiple of VEC).
template <bool WHOLE, int VEC> __device__ __forceinline__ int channels_left(int D, int c) { return WHOLE ? VEC : D - c; }

// Threads of a workgroup, and the rows that it holds at a time.
constexpr int norm_threads(int lpr) { return lpr <= 256 ? 256 : lpr; }

template <typename E, int VEC, int LPR, int NV, bool WHOLE>
__global__ __launch_bounds__(norm_threads(LPR)) void gdn_gated_norm_kernel(NormGeo g, const E* __restrict__ x,
                                                                          const float* __restrict__ w,
                                                                          const E* __restrict__ z, E* __restrict__ y) {
  constexpr int RPB = norm_threads(LPR) / LPR;
  __shared__ float slot[2][LPR / 64 > 0 ? LPR / 64 : 1];
  RowSum<LPR> sum{slot};
  const int sub = threadIdx.x / LPR, l = threadIdx.x % LPR;
  Chan<float, VEC> wv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * LPR + l) * VEC;
    if (c < g.D) wv[i].load(w + c, channels_left<WHOLE, VEC>(g.D, c));
    else wv[i].zero();
  }
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < g.rows; base += (int64_t)gridDim.x * RPB) {
    const int64_t row = base + sub;
    const bool live = row < g.rows;
    const E* xr = x + norm_row(g, live ? row : 0, g.ldx);
    const E* zr = z ? z + norm_row(g, live ? row : 0, g.ldz) : nullptr;
    Chan<E, VEC> xv[NV], zv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * LPR + l) * VEC;
      xv[i].zero();
      zv[i].zero();
      if (c < g.D && live) {
        xv[i].load(xr + c, channels_left<WHOLE, VEC>(g.D, c));
        if (z) zv[i].load(zr + c, channels_left<WHOLE, VEC>(g.D, c));
      }
    }
    float u[NV][VEC], gate[NV][VEC], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xv[i].get(u[i]);
      zv[i].get(gate[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        gate[i][j] = gate[i][j] * fast_sigmoid(gate[i][j]);
        if (g.mode == kGateFirst) u[i][j] *= gate[i][j];
        ss += u[i][j] * u[i][j];
      }
    }
    const float c = __builtin_amdgcn_rsqf(sum(ss) / (float)g.D + g.eps);
    if (!live) continue;
    E* yr = y + row * g.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = (i * LPR + l) * VEC;
      float wf[VEC], out[VEC];
      wv[i].get(wf);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        out[j] = u[i][j] * c * wf[j];
        if (g.mode == kGateAfter) out[j] *= gate[i][j];
      }
      if (ch < g.D) chan_store<E, VEC>(yr + ch, out, channels_left<WHOLE, VEC>(g.D, ch));
    }
  }
}

// The workgroup's sums of K weights' gradients, from its row groups, to partial[block][k][D].
template <int VEC, int LPR, int NV, bool WHOLE, int K>
__device__ __forceinline__ void norm_partials(float (&acc)[K][NV][VEC], float* __restrict__ partial, int D) {
  constexpr int RPB = norm_threads(LPR) / LPR;
  const int sub = threadIdx.x / LPR, l = threadIdx.x % LPR;
  if constexpr (RPB == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * LPR + l) * VEC;
        if (c < D) chan_store<float, VEC>(partial + ((int64_t)blockIdx.x * K + k) * D + c, acc[k][i], channels_left<WHOLE, VEC>(D, c));
      }
  } else {
    __shared__ float sums[norm_threads(LPR) * VEC];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < VEC; ++j) sums[(sub * LPR + l) * VEC + j] = acc[k][i][j];
        __syncthreads();
        for (int t = threadIdx.x; t < LPR * VEC; t += norm_threads(LPR)) {
          float s = 0.f;
#pragma unroll
          for (int r = 0; r < RPB; ++r) s += sums[r * LPR * VEC + t];
          const int c = i * LPR * VEC + t;
          if (c < D) partial[((int64_t)blockIdx.x * K + k) * D + c] = s;
        }
      }
  }
}

// The factor of a row's norm from its mean square.  Rows behind the last one (not live) hold zeros,
// which without an eps have an infinite one: theirs is 0, so that what they add to the sums is 0.
__device__ __forceinline__ float row_factor(float mean, const NormGeo& g, bool live) {
  return live ? __builtin_amdgcn_rsqf(mean + g.eps) : 0.f;
}

template <typename E, int VEC, int LPR, int NV, bool WHOLE>
__global__ __launch_bounds__(norm_threads(LPR)) void gdn_gated_norm_bwd_kernel(
    NormGeo g, const E* __restrict__ x, const float* __restrict__ w, const E* __restrict__ z,
    const E* __restrict__ dy, E* __restrict__ dx, E* __restrict__ dz, float* __restrict__ partial) {
  constexpr int RPB = norm_threads(LPR) / LPR;
  __shared__ float slot[2][LPR / 64 > 0 ? LPR / 64 : 1];
  RowSum<LPR> sum{slot};
  const int sub = threadIdx.x / LPR, l = threadIdx.x % LPR;
  Chan<float, VEC> wv[NV];
  float acc[1][NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * LPR + l) * VEC;
    if (c < g.D) wv[i].load(w + c, channels_left<WHOLE, VEC>(g.D, c));
    else wv[i].zero();
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc[0][i][j] = 0.f;
  }
  const float inv = 1.f / (float)g.D;
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < g.rows; base += (int64_t)gridDim.x * RPB) {
    const int64_t row = base + sub;
    const bool live = row < g.rows;
    const int64_t at = live ? row : 0;
    const E* xr = x + norm_row(g, at, g.ldx);
    const E* zr = z ? z + norm_row(g, at, g.ldz) : nullptr;
    Chan<E, VEC> xv[NV], zv[NV], dv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * LPR + l) * VEC;
      xv[i].zero();
      zv[i].zero();
      dv[i].zero();
      if (c < g.D && live) {
        xv[i].load(xr + c, channels_left<WHOLE, VEC>(g.D, c));
        dv[i].load(dy + at * g.D + c, channels_left<WHOLE, VEC>(g.D, c));
        if (z) zv[i].load(zr + c, channels_left<WHOLE, VEC>(g.D, c));
      }
    }
    float u[NV][VEC], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float zf[VEC];
      xv[i].get(u[i]);
      if (g.mode == kGateFirst) {
        zv[i].get(zf);
#pragma unroll
        for (int j = 0; j < VEC; ++j) u[i][j] *= zf[j] * fast_sigmoid(zf[j]);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss += u[i][j] * u[i][j];
    }
    const float c = row_factor(sum(ss) * inv, g, live);
    // n = u c;  m = mean(n dn), dn = dy w (times the gate behind the norm)
    float dn[NV][VEC], m = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float wf[VEC], df[VEC], zf[VEC];
      wv[i].get(wf);
      dv[i].get(df);
      zv[i].get(zf);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float n = u[i][j] * c;
        float d = df[j];
        if (g.mode == kGateAfter) d *= zf[j] * fast_sigmoid(zf[j]);
        acc[0][i][j] += d * n;
        dn[i][j] = d * wf[j];
        m += n * dn[i][j];
      }
    }
    m = sum(m) * inv;
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = (i * LPR + l) * VEC;
      float wf[VEC], df[VEC], zf[VEC], xf[VEC], ox[VEC], oz[VEC];
      wv[i].get(wf);
      dv[i].get(df);
      zv[i].get(zf);
      xv[i].get(xf);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float n = u[i][j] * c, du = c * (dn[i][j] - n * m);
        const float s = fast_sigmoid(zf[j]);
        if (g.mode == kGateFirst) {
          ox[j] = du * (zf[j] * s);
          oz[j] = du * xf[j] * silu_slope(zf[j], s);
        } else {
          ox[j] = du;
          oz[j] = df[j] * n * wf[j] * silu_slope(zf[j], s);
        }
      }
      if (ch < g.D) {
        chan_store<E, VEC>(dx + row * g.D + ch, ox, channels_left<WHOLE, VEC>(g.D, ch));
        if (z) chan_store<E, VEC>(dz + row * g.D + ch, oz, channels_left<WHOLE, VEC>(g.D, ch));
      }
    }
  }
  norm_partials<VEC, LPR, NV, WHOLE, 1>(acc, partial, g.D);
}

template <typename E, typename R, int VEC, int LPR, int NV, bool WHOLE>
__global__ __launch_bounds__(norm_threads(LPR)) void gdn_residual_norm_kernel(
    NormGeo g, const E* __restrict__ x, const R* residual, const float* __restrict__ w,
    const float* __restrict__ post, const float* __restrict__ scale, E* __restrict__ h, R* out) {
  constexpr int RPB = norm_threads(LPR) / LPR;
  __shared__ float slot[2][LPR / 64 > 0 ? LPR / 64 : 1];
  RowSum<LPR> sum{slot};
  const int sub = threadIdx.x / LPR, l = threadIdx.x % LPR;
  const float inv = 1.f / (float)g.D;
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < g.rows; base += (int64_t)gridDim.x * RPB) {
    const int64_t row = base + sub;
    const bool live = row < g.rows;
    const E* xr = x + (live ? row : 0) * g.ldx;
    const R* rr = residual + (live ? row : 0) * g.ldz;
    Chan<E, VEC> xv[NV];
    Chan<R, VEC> rv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * LPR + l) * VEC;
      xv[i].zero();
      rv[i].zero();
      if (c < g.D && live) {
        xv[i].load(xr + c, channels_left<WHOLE, VEC>(g.D, c));
        rv[i].load(rr + c, channels_left<WHOLE, VEC>(g.D, c));
      }
    }
    float s[NV][VEC];
    float cp = 1.f;
    if (post) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float xf[VEC];
        xv[i].get(xf);
#pragma unroll
        for (int j = 0; j < VEC; ++j) ss += xf[j] * xf[j];
      }
      cp = __builtin_amdgcn_rsqf(sum(ss) * inv + g.eps);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * LPR + l) * VEC;
      float xf[VEC], pf[VEC], sf[VEC];
      xv[i].get(xf);
      rv[i].get(s[i]);
      Chan<float, VEC> pv, sv;
      pv.zero();
      sv.zero();
      if (c < g.D) {
        if (post) pv.load(post + c, channels_left<WHOLE, VEC>(g.D, c));
        if (scale) sv.load(scale + c, channels_left<WHOLE, VEC>(g.D, c));
      }
      pv.get(pf);
      sv.get(sf);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float p = post ? xf[j] * cp * pf[j] : xf[j];
        s[i][j] += scale ? sf[j] * p : p;
        ss += s[i][j] * s[i][j];
      }
    }
    const float c = __builtin_amdgcn_rsqf(sum(ss) * inv + g.eps);
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = (i * LPR + l) * VEC;
      if (ch >= g.D) continue;
      Chan<float, VEC> wv;
      float wf[VEC], hf[VEC];
      wv.load(w + ch, channels_left<WHOLE, VEC>(g.D, ch));
      wv.get(wf);
#pragma unroll
      for (int j = 0; j < VEC; ++j) hf[j] = s[i][j] * c * wf[j];
      chan_store<R, VEC>(out + row * g.D + ch, s[i], channels_left<WHOLE, VEC>(g.D, ch));
      chan_store<E, VEC>(h + row * g.D + ch, hf, channels_left<WHOLE, VEC>(g.D, ch));
    }
  }
}

// s is formed again from x and the residual, in fp32, so that the gradients are those of the
// values that h was formed from (and not of s as it was rounded).
template <typename E, typename R, int VEC, int LPR, int NV, bool WHOLE>
__global__ __launch_bounds__(norm_threads(LPR)) void gdn_residual_norm_bwd_kernel(
    NormGeo g, const E* __restrict__ x, const R* __restrict__ residual, const float* __restrict__ w,
    const float* __restrict__ post, const float* __restrict__ scale, const E* __restrict__ dh,
    const R* __restrict__ ds, E* __restrict__ dx, R* __restrict__ dr, float* __restrict__ partial) {
  constexpr int RPB = norm_threads(LPR) / LPR;
  __shared__ float slot[2][LPR / 64 > 0 ? LPR / 64 : 1];
  RowSum<LPR> sum{slot};
  const int sub = threadIdx.x / LPR, l = threadIdx.x % LPR;
  const float inv = 1.f / (float)g.D;
  float acc[3][NV][VEC];  // towards w, post and scale
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[k][i][j] = 0.f;
  auto read = [&](const float* p, int c, float (&v)[VEC]) {
    Chan<float, VEC> t;
    if (p && c < g.D) {
      t.load(p + c, channels_left<WHOLE, VEC>(g.D, c));
      t.get(v);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = 1.f;
    }
  };
  // Where a lane has one vector, it keeps the weights' as well, and loads a row ahead of its use
  // (B=4, T=4096, C=2048 bf16: 108 us without either in 1024 workgroups, 86 with both in 512).
  constexpr bool HOLD = NV == 1 && LPR <= 512;
  float held[3][VEC];
  if constexpr (HOLD) {
    read(w, l * VEC, held[0]);
    read(post, l * VEC, held[1]);
    read(scale, l * VEC, held[2]);
  }
  auto vec = [&](auto which, int c, float (&v)[VEC]) {
    constexpr int k = decltype(which)::value;
    if constexpr (HOLD) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = held[k][j];
    } else {
      read(k == 0 ? w : k == 1 ? post : scale, c, v);
    }
  };
  constexpr std::integral_constant<int, 0> kW{};
  constexpr std::integral_constant<int, 1> kPost{};
  constexpr std::integral_constant<int, 2> kScale{};
  struct Row {
    Chan<E, VEC> x[NV], h[NV];
    Chan<R, VEC> r[NV], s[NV];
  };
  auto load = [&](Row& o, int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * LPR + l) * VEC;
      o.x[i].zero();
      o.h[i].zero();
      o.r[i].zero();
      o.s[i].zero();
      if (c < g.D && row < g.rows) {
        o.x[i].load(x + row * g.ldx + c, channels_left<WHOLE, VEC>(g.D, c));
        o.r[i].load(residual + row * g.ldz + c, channels_left<WHOLE, VEC>(g.D, c));
        o.h[i].load(dh + row * g.D + c, channels_left<WHOLE, VEC>(g.D, c));
        if (ds) o.s[i].load(ds + row * g.D + c, channels_left<WHOLE, VEC>(g.D, c));
      }
    }
  };
  Row next;
  if constexpr (HOLD) load(next, (int64_t)blockIdx.x * RPB + sub);
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < g.rows; base += (int64_t)gridDim.x * RPB) {
    const int64_t row = base + sub;
    const bool live = row < g.rows;
    Row cur;
    if constexpr (HOLD) {
      cur = next;
      load(next, row + (int64_t)gridDim.x * RPB);
    } else {
      load(cur, row);
    }
    const auto &xv = cur.x, &hv = cur.h;
    const auto &rv = cur.r, &sv = cur.s;
    float cp = 1.f;
    if (post) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float xf[VEC];
        xv[i].get(xf);
#pragma unroll
        for (int j = 0; j < VEC; ++j) ss += xf[j] * xf[j];
      }
      cp = row_factor(sum(ss) * inv, g, live);
    }
    float s[NV][VEC], ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * LPR + l) * VEC;
      float xf[VEC], pf[VEC], cf[VEC];
      xv[i].get(xf);
      rv[i].get(s[i]);
      vec(kPost, c, pf);
      vec(kScale, c, cf);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        s[i][j] += cf[j] * (xf[j] * cp * pf[j]);
        ss += s[i][j] * s[i][j];
      }
    }
    const float c = row_factor(sum(ss) * inv, g, live);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float hf[VEC], wf[VEC];
      hv[i].get(hf);
      vec(kW, (i * LPR + l) * VEC, wf);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float n = s[i][j] * c;
        acc[0][i][j] += hf[j] * n;
        m += n * (hf[j] * wf[j]);
      }
    }
    m = sum(m) * inv;
    // d = gradient towards s; q = mean(r(x) dn) of the norm behind the block
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = (i * LPR + l) * VEC;
      float hf[VEC], wf[VEC], d[VEC], xf[VEC], pf[VEC], cf[VEC];
      hv[i].get(hf);
      sv[i].get(d);
      xv[i].get(xf);
      vec(kW, ch, wf);
      vec(kPost, ch, pf);
      vec(kScale, ch, cf);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float n = s[i][j] * c;
        d[j] += c * (hf[j] * wf[j] - n * m);
        s[i][j] = d[j];
        const float nx = xf[j] * cp, dp = d[j] * cf[j];
        acc[1][i][j] += dp * nx;
        acc[2][i][j] += d[j] * (nx * pf[j]);
        q += nx * (dp * pf[j]);
      }
    }
    if (post) q = sum(q) * inv;
    else q = 0.f;
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int ch = (i * LPR + l) * VEC;
      if (ch >= g.D) continue;
      float xf[VEC], pf[VEC], cf[VEC];
      xv[i].get(xf);
      vec(kPost, ch, pf);
      vec(kScale, ch, cf);
#pragma unroll
      for (int j = 0; j < VEC; ++j) xf[j] = cp * (s[i][j] * cf[j] * pf[j] - xf[j] * cp * q);
      chan_store<R, VEC>(dr + row * g.D + ch, s[i], channels_left<WHOLE, VEC>(g.D, ch));
      chan_store<E, VEC>(dx + row * g.D + ch, xf, channels_left<WHOLE, VEC>(g.D, ch));
    }
  }
  norm_partials<VEC, LPR, NV, WHOLE, 3>(acc, partial, g.D);
}

// out[k][c] = sum over the rows of partial[row][k][c], for the K outputs that are wanted.  A
// workgroup has 64 channels of one output, VEC of them per lane and so 16 VEC groups of rows;
// their sums are added in the groups' order.
struct NormSums {
  float* out[3];
};
constexpr int kSumAhead = 8;  // rows of a group that are loaded at a time
template <int VEC>
__global__ __launch_bounds__(1024) void gdn_norm_sums_kernel(const float* __restrict__ partial, int rows, int K, int D,
                                                             NormSums o) {
  constexpr int LANES = 64 / VEC, GROUPS = 1024 / LANES;
  __shared__ float s[GROUPS][64 + 1], t[16][64 + 1];
  const int blocks = (D + 63) / 64, k = blockIdx.x / blocks, c0 = (blockIdx.x - k * blocks) * 64;
  if (!o.out[k]) return;
  const int g = threadIdx.x / LANES, x = threadIdx.x % LANES * VEC;
  float a[VEC] = {};
  if (c0 + x < D) {
    const float* p = partial + (int64_t)k * D + c0 + x;
    for (int r = g; r < rows; r += GROUPS * kSumAhead) {
      Chan<float, VEC> v[kSumAhead];
#pragma unroll
      for (int i = 0; i < kSumAhead; ++i) {
        v[i].zero();
        if (r + i * GROUPS < rows) v[i].load(p + (int64_t)(r + i * GROUPS) * K * D, VEC);
      }
#pragma unroll
      for (int i = 0; i < kSumAhead; ++i) {
        float f[VEC];
        v[i].get(f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) a[j] += f[j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) s[g][x + j] = a[j];
  __syncthreads();
  const int w = threadIdx.x >> 6, c = lane_id();
  float b = 0.f;
#pragma unroll
  for (int r = 0; r < GROUPS / 16; ++r) b += s[w * (GROUPS / 16) + r][c];
  t[w][c] = b;
  __syncthreads();
  if (w == 0 && c0 + c < D) {
    b = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) b += t[r][c];
    o.out[k][c0 + c] = b;
  }
}

}  // namespace gdn
