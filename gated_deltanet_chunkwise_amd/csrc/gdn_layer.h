// gdn_layer.h -- device helpers shared by the layer operators around the gated
// delta rule (short causal convolution, selective scan, 8-bit checkpoints).
#pragma once
#include "gdn_common.h"

namespace gdn {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));

// A pointer into global memory with its address space spelled out.
template <typename E> using Global = __attribute__((address_space(1))) E*;

// A lane's offset, in a form that the compiler adds to a uniform pointer within the load
// itself (it would otherwise form 64-bit sums in vector registers).
__device__ __forceinline__ uint32_t lane_offset(uint32_t bytes) {
  asm("" : "+v"(bytes));
  return bytes;
}

// p + n, in a form that the compiler does not fold into other sums: the walks below step
// their row pointers token by token, and without this it keeps every multiple of every
// stride in scalar registers, which then spill.
template <typename T> __device__ __forceinline__ Global<T> stepped(Global<T> p, int64_t n) {
  p += n;
  asm("" : "+s"(p));
  return p;
}

constexpr int kPackBlock = 32;  // channels that share one checkpoint scale

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 1 / (1 + e^-x).  v_exp_f32 and v_rcp_f32 are within about 1 ulp; e^-x
// overflowing to infinity gives exactly 0.
__device__ __forceinline__ float fast_sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-x * kLog2e));
}

// gate_softplus (gdn_common.h: the same formula and error) without branches, for a value
// that every lane needs, and without its range below 2^-126: a time step that small
// changes no state, and here is 0.
__device__ __forceinline__ float softplus_flat(float x) {
  const float y = __builtin_amdgcn_exp2f(x * kLog2e);
  const float u = 1.f + y;
  const float r = (__builtin_amdgcn_logf(u) * __builtin_amdgcn_rcpf(u - 1.f)) * (y * 0.693147180559945309f);
  return x > 20.f ? x : u == 1.f ? y : r;
}

// d/dx x sigmoid(x) = s (1 + x (1 - s)), s = sigmoid(x).  1 - s is off by at most 2^-24,
// which x (1 - s) + 1 loses only |x| 2^-24 to.
__device__ __forceinline__ float silu_slope(float x, float s) { return s * fmaf(x, 1.f - s, 1.f); }

// The checkpoint scale of a stored byte b: 2^(b - 127), and NaN for 255 (a block
// that held an infinity or a NaN).
__device__ __forceinline__ float pack_scale(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7fc00000u : b ? b << 23 : 0x00400000u);
}

// Activations [tokens][C] as a kernel reads them: rows of E with a row stride, or
// (scales != nullptr) a checkpoint's codes [tokens][C] and scales [tokens][ceil(C/32)].
struct Src {
  const void* p;
  const uint8_t* scales;
  int64_t ld;  // elements between rows (codes: C)
};

// VEC consecutive channels of one row, as loaded (not yet converted), so that loads can
// be issued well before their use; two at most from a checkpoint.
template <typename E, int VEC> struct RawVec;
template <> struct RawVec<bf16, 4> { u32x2 w; uint32_t s; };
template <> struct RawVec<bf16, 2> { uint32_t w, s; };
template <> struct RawVec<float, 4> { u32x4 w; uint32_t s; };
template <typename E> struct RawVec<E, 1> { uint32_t w, s; };

template <typename E, int VEC>
__device__ __forceinline__ RawVec<E, VEC> raw_load(const Src& s, int64_t row, int c, int nblk) {
  RawVec<E, VEC> r = {};
  if (s.scales) {  // VEC divides 32: one scale for the vector
    const uint8_t* q = static_cast<const uint8_t*>(s.p) + row * s.ld + c;
    if constexpr (VEC == 1) r.w = *q;
    else if constexpr (VEC == 2) r.w = *reinterpret_cast<const uint16_t*>(q);
    r.s = s.scales[row * nblk + (c >> 5)];
  } else {
    const E* q = static_cast<const E*>(s.p) + row * s.ld + c;
    if constexpr (VEC == 1 && sizeof(E) == 2) r.w = *reinterpret_cast<const uint16_t*>(q);
    else r.w = *reinterpret_cast<const decltype(r.w)*>(q);
  }
  return r;
}

// The same at a wave-uniform row and a lane's offset in bytes (in a checkpoint: the same
// of its code; `soff` that of its scale).
template <typename E, int VEC, bool CK>
__device__ __forceinline__ RawVec<E, VEC> raw_load_at(Global<const char> row, Global<const uint8_t> srow,
                                                      uint32_t off, uint32_t soff) {
  RawVec<E, VEC> r = {};
  Global<const char> q = row + off;
  if constexpr (!CK) {
    if constexpr (VEC == 1 && sizeof(E) == 2) r.w = *(Global<const uint16_t>)q;
    else r.w = *(Global<const decltype(r.w)>)q;
  } else {
    static_assert(VEC <= 2, "");
    if constexpr (VEC == 1) r.w = *(Global<const uint8_t>)q;
    else r.w = *(Global<const uint16_t>)q;
    r.s = srow[soff];
  }
  return r;
}

// The raw vector as fp32; `packed` as the load's (s.scales != nullptr).
template <typename E, int VEC>
__device__ __forceinline__ void raw_unpack(const RawVec<E, VEC>& r, bool packed, float (&v)[VEC]) {
  if constexpr (VEC <= 2) {
    if (packed) {
      const float sc = pack_scale(r.s);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = (float)(int8_t)(r.w >> (8 * i)) * sc;
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    if constexpr (VEC == 1) v[0] = __uint_as_float(sizeof(E) == 2 ? r.w << 16 : r.w);
    else if constexpr (VEC == 2) v[i] = i ? bf16_hi(r.w) : bf16_lo(r.w);
    else if constexpr (sizeof(E) == 2) v[i] = (i & 1) ? bf16_hi(r.w[i >> 1]) : bf16_lo(r.w[i >> 1]);
    else v[i] = __uint_as_float(r.w[i]);
  }
}

// VEC consecutive elements of E from a plain pointer, and to one (round to nearest even).
template <typename E, int VEC>
__device__ __forceinline__ void vec_load(const E* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = (float)*p;
  } else {
    const Src s{p, nullptr, 0};
    raw_unpack<E, VEC>(raw_load<E, VEC>(s, 0, 0, 0), false, v);
  }
}
template <typename E, int VEC>
__device__ __forceinline__ void vec_store(E* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    *p = (E)v[0];
  } else if constexpr (VEC == 2) {
    *reinterpret_cast<bf16x2*>(p) = bf16x2{(bf16)v[0], (bf16)v[1]};
  } else {
    static_assert(sizeof(E) == 4, "");
    *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  }
}

// U tokens of one vector of channels as loaded, so that the loads are all in flight
// before the first is converted.  CK: from a checkpoint, codes and scale.
template <typename E, int VEC, int U, bool CK> struct TokenVals {
  RawVec<E, VEC> v[U];
  // tokens t .. t + U - 1, those from `end` on held to the last before it; `off`: the
  // lane's offset in bytes, `soff` that of its scale
  __device__ __forceinline__ void fetch(const Src& src, int t, int end, uint32_t off, uint32_t soff, int nblk) {
    if (t + U <= end) walk(src, t, off, soff, nblk, [](int) { return true; });
    else walk(src, t, off, soff, nblk, [&](int k) { return t + k + 1 < end; });
  }
  template <typename F>
  __device__ __forceinline__ void walk(const Src& src, int t, uint32_t off, uint32_t soff, int nblk, F&& more) {
    const int64_t step = src.ld * (CK ? 1 : (int)sizeof(E));
    Global<const char> p = (Global<const char>)src.p + t * step;
    Global<const uint8_t> q = (Global<const uint8_t>)src.scales + (CK ? (int64_t)t * nblk : 0);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      v[k] = raw_load_at<E, VEC, CK>(p, q, off, soff);
      p = stepped<const char>(p, more(k) ? step : 0);
      if constexpr (CK) q = stepped<const uint8_t>(q, more(k) ? nblk : 0);
    }
  }
  __device__ __forceinline__ float operator[](int k) const {
    static_assert(VEC == 1, "");
    float f[1];
    raw_unpack<E, 1>(v[k], CK, f);
    return f[0];
  }
};

// Packed sequences.  Offsets are read clamped to [0, T], so that ill-formed ones
// never lead outside the buffers.
__device__ __forceinline__ int seq_offset(const int64_t* cu, int n, int T) {
  const int64_t v = cu[n];
  return v < 0 ? 0 : v > T ? T : (int)v;
}
// The last n in [0, N) whose offset is at most t (0 if there is none): the sequence
// of token t, unless t lies behind the last sequence.
__device__ __forceinline__ int seq_of_token(const int64_t* cu, int N, int T, int t) {
  int lo = 0, hi = N;  // offset[lo] <= t is taken for granted, offset[hi] > t or hi == N
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (seq_offset(cu, mid, T) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A wave-uniform value that the compiler cannot see to be one, in a scalar register.
template <bool UNIFORM> __device__ __forceinline__ int uniform(int v) {
  return UNIFORM ? __builtin_amdgcn_readfirstlane(v) : v;
}

// A maximal stretch [ta, tb) of a tile within one sequence n = [start, end), all in
// tokens of the flattened batch; done() once the tile is exhausted.  Every step
// moves n or ta forward, so the walk ends for any offsets.  UNIFORM: all lanes of the
// wave walk the same tile.
template <bool UNIFORM> struct Run {
  int n, N, T, start, end, ta, tb, t1;
  int rest;  // once done: the tile's first token behind the last sequence, or t1
  const int64_t* cu;

  __device__ __forceinline__ void init(const int64_t* cu_, int T_, int N_, int tile, int ntiles, int len) {
    place(cu_, T_, N_, tile, ntiles, len);
    locate();
  }
  // The tile's tokens [ta, t1), which need no offset; then its first run.
  __device__ __forceinline__ void place(const int64_t* cu_, int T_, int N_, int tile, int ntiles, int len) {
    cu = cu_;
    T = T_;
    N = N_;
    if (cu) {
      ta = tile * len;
      t1 = rest = ta + min(len, T - ta);  // (ta + len may pass 2^31)
    } else {
      n = tile / ntiles;
      start = n * T;
      end = start + T;
      ta = start + (tile - n * ntiles) * len;
      t1 = rest = tb = ta + min(len, end - ta);
    }
  }
  __device__ __forceinline__ void locate() {
    if (!cu) return;
    n = uniform<UNIFORM>(seq_of_token(cu, N, T, ta));
    fit();
  }
  __device__ __forceinline__ bool done() const { return ta >= t1; }
  __device__ __forceinline__ void next() {
    ta = tb;
    if (cu && ta < t1) {
      ++n;
      fit();
      // the identity for well-formed offsets: only a tile's first run continues a sequence
      start = max(start, ta);
    }
  }
  // The sequence that holds token ta, from n on: past empty ones by a search (offsets padded
  // to a fixed count hold thousands of them); behind the last sequence the walk ends.
  __device__ __forceinline__ void fit() {
    for (; n < N; n = max(n + 1, uniform<UNIFORM>(seq_of_token(cu, N, T, ta)))) {
      start = uniform<UNIFORM>(seq_offset(cu, n, T));
      end = uniform<UNIFORM>(seq_offset(cu, n + 1, T));
      if (end > ta && end > start) {
        if (start > ta) ta = min(start, t1);  // only for ill-formed offsets
        tb = min(end, t1);
        return;
      }
    }
    rest = ta;
    ta = tb = t1;
  }
};

}  // namespace gdn
