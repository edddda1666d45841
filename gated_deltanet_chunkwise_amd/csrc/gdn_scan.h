// gdn_scan.h -- selective state space scan on gfx950, forward pass and decode step.
//
//     D = softplus(dt + dt_bias),  a = exp(-exp(A_log) D)
//     h[d,n] <- a[d,n] h[d,n] + D Bm[n] x,   y = (sum_n Cm[n] h[d,n] + skip x) silu(z)
//
// A wave owns 64 channels of one group, a lane one channel with NS of its states in
// registers; Bm and Cm of a token are the same for all its lanes and come through
// scalar loads into scalar registers.  With more than NS states the workgroup has
// ceil(N / NS) waves for the same channels, which add their parts of y through LDS.
//
// Per token, channel and state the recurrence takes one v_exp_f32 and four other
// VALU operations (D A, D x B, the state's and y's multiply-adds), so at N = 16 it is
// bound by the VALU and not by the 8 bytes of x, dt, z and y.
//
// Few channels leave most of the device idle, so the tokens are cut into tiles that
// run side by side: (1) each tile's end state from a zero start, and its sum of D,
// whose exp(A sum) is the tile's decay; (2) the tiles' start states, tile after tile;
// (3) every tile again from its true start.  That forms the states twice; where the
// waves of one tile per sequence already fill the device, (3) alone runs the whole
// sequence.
#pragma once
#include "gdn_layer.h"

namespace gdn {

struct ScanGeo {
  int B, T, D, G, N, S;  // S = sequences
  int DG, wpg, cgroups;  // channels per group, waves per group, waves for all channels
  int len, ntiles;       // tokens per tile; tiles per row of the batch
  int nw, np;            // waves per workgroup; nw * NS
  const int64_t* cu;
  int64_t lddt;
  int64_t ldb, ldc;      // elements between rows of Bm and Cm, and between groups
  int bgs, cgs;
};

constexpr int kScanGroup = 8;  // tokens whose loads are in flight together
constexpr int kScanMaxWaves = 4;

typedef const __attribute__((address_space(4))) uint32_t* scalar_ptr;

// NS consecutive elements at a wave-uniform, 4-byte aligned address, in scalar registers.
template <typename BE, int NS> struct ScalarRow {
  static constexpr int kWords = NS * (int)sizeof(BE) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const BE* p) {
    scalar_ptr q = (scalar_ptr)(uintptr_t)p;
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = q[i];
  }
  __device__ __forceinline__ float operator[](int j) const {
    if constexpr (sizeof(BE) == 4) return __uint_as_float(w[j]);
    else return (j & 1) ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
  }
};

// One channel of one row as loaded.
template <typename E> __device__ __forceinline__ uint32_t load1(const E* p) {
  if constexpr (sizeof(E) == 2) return *reinterpret_cast<const uint16_t*>(p);
  else return *reinterpret_cast<const uint32_t*>(p);
}
template <typename E> __device__ __forceinline__ float value1(uint32_t w) {
  return __uint_as_float(sizeof(E) == 2 ? w << 16 : w);
}

// -exp(A_log) log2(e), the rate in base 2 that the kernels hold.  0 beyond N: such a
// state keeps the 0 it starts with.
template <int NS>
__device__ __forceinline__ void scan_rates(const float* A_log, const ScanGeo& g, int d, int n0, float (&A2)[NS]) {
#pragma unroll
  for (int j = 0; j < NS; ++j)
    A2[j] = n0 + j < g.N ? -expf(A_log[(int64_t)d * g.N + n0 + j]) * kLog2e : 0.f;
}

template <int NS>
__device__ __forceinline__ void state_load(const float* st, const ScanGeo& g, int n, int d, int n0, float (&h)[NS]) {
  const float* p = st ? st + ((int64_t)n * g.D + d) * g.N : nullptr;
#pragma unroll
  for (int j = 0; j < NS; ++j) h[j] = p && n0 + j < g.N ? p[n0 + j] : 0.f;
}
template <int NS>
__device__ __forceinline__ void state_store(float* st, const ScanGeo& g, int n, int d, int n0, const float (&h)[NS]) {
  float* p = st + ((int64_t)n * g.D + d) * g.N;
#pragma unroll
  for (int j = 0; j < NS; ++j)
    if (n0 + j < g.N) p[n0 + j] = h[j];
}

// Block id -> (tile of the whole batch, group of 64 channels); the lane's channel d,
// `on` where it has one of its own.
struct ScanPlace {
  int tile, gi, d, lane, wave, n0;
  bool on;
  template <int NS> __device__ __forceinline__ void init(const ScanGeo& g, uint32_t block) {
    tile = block / g.cgroups;
    const int cg = block - tile * g.cgroups;
    gi = cg / g.wpg;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int dl = (cg - gi * g.wpg) * 64 + lane;
    on = dl < g.DG;
    d = gi * g.DG + min(dl, g.DG - 1);
    n0 = wave * NS;
  }
};

// A sequence without tokens ends as it starts.
__device__ __forceinline__ void scan_empty_state(const ScanGeo& g, int n, const float* from, float* to) {
  const int64_t start = g.cu ? seq_offset(g.cu, n, g.T) : 0;
  const int64_t end = g.cu ? seq_offset(g.cu, n + 1, g.T) : g.T;
  if (end > start || !to) return;
  const int64_t w = (int64_t)g.D * g.N;
  for (int64_t i = threadIdx.x; i < w; i += blockDim.x) to[n * w + i] = from ? from[n * w + i] : 0.f;
}

// Tiles' end states from a zero start (ENDS: `states` [tile][np][D] and sums
// [tile][D] written; a sum of -1 says that a sequence starts in the tile, so nothing
// passes through it), or the outputs (`states` holds the tiles' start states).
// Blocks behind the last tile's copy the states of empty sequences (not ENDS).
template <typename E, typename BE, int NS, bool SPLIT, bool ENDS>
__global__ __launch_bounds__(SPLIT ? 64 * kScanMaxWaves : 64) void gdn_scan_kernel(
    ScanGeo g, Src x, const E* __restrict__ dt, Src z, const float* __restrict__ A_log,
    const BE* __restrict__ Bm, const BE* __restrict__ Cm, const float* __restrict__ skip,
    const float* __restrict__ dt_bias, const float* __restrict__ h0, float* __restrict__ states,
    float* __restrict__ sums, E* __restrict__ y, float* __restrict__ fin) {
  constexpr int U = kScanGroup;
  __shared__ float part[SPLIT && !ENDS ? 2 : 1][SPLIT && !ENDS ? kScanMaxWaves : 1][U][SPLIT && !ENDS ? 64 : 1];
  const int tiles = g.ntiles * (g.cu ? 1 : g.B);
  const uint32_t main_blocks = (uint32_t)tiles * g.cgroups;
  if constexpr (ENDS) {
    if ((int)(blockIdx.x / g.cgroups) % g.ntiles == g.ntiles - 1) return;  // nobody starts from it
  } else if (blockIdx.x >= main_blocks) {
    scan_empty_state(g, blockIdx.x - main_blocks, h0, fin);
    return;
  }
  ScanPlace w;
  w.init<NS>(g, blockIdx.x);
  float A2[NS], h[NS];
  scan_rates<NS>(A_log, g, w.d, w.n0, A2);
  const float bias = dt_bias ? dt_bias[w.d] : 0.f, sk = skip ? skip[w.d] : 0.f;
  const E* xd = static_cast<const E*>(x.p) + w.d;
  const E* dtd = dt + w.d;
  const E* zd = static_cast<const E*>(z.p) + w.d;
  const bool gate = z.p != nullptr && !ENDS;
  const BE* bp = Bm + (int64_t)w.gi * g.bgs + w.n0;
  const BE* cp = Cm + (int64_t)w.gi * g.cgs + w.n0;
  float sum = 0.f;
  int buf = 0;

  Run<true> run;
  run.init(g.cu, g.T, g.S, w.tile, g.ntiles, g.len);
#pragma unroll
  for (int j = 0; j < NS; ++j) h[j] = 0.f;
  for (; !run.done(); run.next()) {
    if (run.ta > run.start) {
      if constexpr (!ENDS) {
        const float* p = states + ((int64_t)w.tile * g.np + w.n0) * g.D + w.d;
#pragma unroll
        for (int j = 0; j < NS; ++j) h[j] = p[(int64_t)j * g.D];
      }
    } else {
      state_load<NS>(h0, g, run.n, w.d, w.n0, h);
      sum = -1.f;
    }
    uint32_t rx[U], rd[U], rz[U] = {};
    auto fetch = [&](int t) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int64_t q = min(t + k, run.tb - 1);
        rx[k] = load1<E>(xd + q * x.ld);
        rd[k] = load1<E>(dtd + q * g.lddt);
        if (gate) rz[k] = load1<E>(zd + q * z.ld);
      }
    };
    ScalarRow<BE, NS> b, c;
    fetch(run.ta);
    b.load(bp + run.ta * g.ldb);
    if constexpr (!ENDS) c.load(cp + run.ta * g.ldc);
    for (int t = run.ta; t < run.tb; t += U) {
      float xv[U], dl[U], zv[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        xv[k] = value1<E>(rx[k]);
        zv[k] = value1<E>(rz[k]);
        dl[k] = softplus_flat(value1<E>(rd[k]) + bias);
      }
      if (t + U < run.tb) fetch(t + U);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (t + k >= run.tb) break;
        const ScalarRow<BE, NS> bt = b, ct = c;
        const int64_t q = min(t + k + 1, run.tb - 1);
        b.load(bp + q * g.ldb);
        if constexpr (!ENDS) c.load(cp + q * g.ldc);
        const float u = dl[k] * xv[k];
        float acc0 = 0.f, acc1 = 0.f;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          h[j] = fmaf(fast_exp2(dl[k] * A2[j]), h[j], bt[j] * u);
          if constexpr (!ENDS) {
            if (j & 1) acc1 = fmaf(ct[j], h[j], acc1);
            else acc0 = fmaf(ct[j], h[j], acc0);
          }
        }
        if constexpr (ENDS) {
          if (sum >= 0.f) sum += dl[k];
        } else if constexpr (SPLIT) {
          part[buf][w.wave][k][w.lane] = acc0 + acc1;
        } else {
          float o = fmaf(sk, xv[k], acc0 + acc1);
          if (gate) o *= zv[k] * fast_sigmoid(zv[k]);
          if (w.on) y[(int64_t)(t + k) * g.D + w.d] = (E)o;
        }
      }
      if constexpr (SPLIT && !ENDS) {
        // each wave finishes every nw-th token; the other buffer is written next, and
        // the barrier after that keeps this one until all have read it
        __syncthreads();
#pragma unroll
        for (int k = 0; k < U; ++k) {
          if (k % g.nw != w.wave || t + k >= run.tb) continue;
          float o = sk * xv[k];
          for (int q = 0; q < g.nw; ++q) o += part[buf][q][k][w.lane];
          if (gate) o *= zv[k] * fast_sigmoid(zv[k]);
          if (w.on) y[(int64_t)(t + k) * g.D + w.d] = (E)o;
        }
        buf ^= 1;
      }
    }
    if constexpr (!ENDS)
      if (fin && w.on && run.tb == run.end) state_store<NS>(fin, g, run.n, w.d, w.n0, h);
  }
  if constexpr (ENDS) {
    if (!w.on) return;
    float* p = states + ((int64_t)w.tile * g.np + w.n0) * g.D + w.d;
#pragma unroll
    for (int j = 0; j < NS; ++j) p[(int64_t)j * g.D] = h[j];
    if (w.wave == 0) sums[(int64_t)w.tile * g.D + w.d] = sum;
  }
}

// (2): states [row of the batch][tile][np][D] from end states to start states, in
// place; one lane per (row, state, channel).
static __global__ __launch_bounds__(256) void gdn_scan_join_kernel(ScanGeo g, const float* __restrict__ A_log,
                                                            const float* __restrict__ h0,
                                                            float* __restrict__ states,
                                                            const float* __restrict__ sums) {
  constexpr int U = 8;
  const int64_t per = (int64_t)g.np * g.D;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int rows = g.cu ? 1 : g.B;
  if (i >= rows * per) return;
  const int row = (int)(i / per);
  const int64_t r = i - row * per;
  const int n = (int)(r / g.D), d = (int)(r - (int64_t)n * g.D);
  const float A2 = n < g.N ? -expf(A_log[(int64_t)d * g.N + n]) * kLog2e : 0.f;
  float H = !g.cu && h0 && n < g.N ? h0[((int64_t)row * g.D + d) * g.N + n] : 0.f;
  float* p = states + (int64_t)row * g.ntiles * per + r;
  const float* s = sums + (int64_t)row * g.ntiles * g.D + d;
  for (int t = 0; t < g.ntiles; t += U) {
    float e[U], sm[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int q = min(t + k, g.ntiles - 1);
      e[k] = p[q * per];  // the last tile's is not written by (1) and not used
      sm[k] = s[(int64_t)q * g.D];
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (t + k >= g.ntiles) break;
      p[(t + k) * per] = H;
      H = sm[k] < 0.f ? e[k] : fmaf(fast_exp2(A2 * sm[k]), H, e[k]);
    }
  }
}

// Rows of Bm and Cm as fp32, groups padded with zeros to np: for element counts,
// strides or addresses that scalar loads cannot take.
template <typename E>
__global__ __launch_bounds__(256) void gdn_scan_rows_kernel(const E* __restrict__ Bm, const E* __restrict__ Cm,
                                                            int64_t ldb, int64_t ldc, int64_t tok, int G,
                                                            int N, int np, float* __restrict__ Bw,
                                                            float* __restrict__ Cw) {
  const int64_t total = tok * G * np, step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += step) {
    const int64_t r = i / np;
    const int n = (int)(i - r * np);
    const int64_t t = r / G;
    const int gi = (int)(r - t * G);
    Bw[i] = n < N ? (float)Bm[t * ldb + (int64_t)gi * N + n] : 0.f;
    Cw[i] = n < N ? (float)Cm[t * ldc + (int64_t)gi * N + n] : 0.f;
  }
}

// Decode: nl = a power of two of lanes per channel, four states each (nl >= N / 4),
// 64 / nl channels per wave, T tokens one after the other.  The state's read and
// write bound it (8 N bytes per channel); `vec`: rows of the state are 16-byte
// aligned multiples of four.
template <typename E>
__global__ __launch_bounds__(256) void gdn_scan_decode_kernel(
    ScanGeo g, Src x, const E* __restrict__ dt, Src z, const float* __restrict__ A_log,
    const E* __restrict__ Bm, const E* __restrict__ Cm, const float* __restrict__ skip,
    const float* __restrict__ dt_bias, const float* state_in, float* state_out, E* __restrict__ y,
    int nl, int vec) {
  const int64_t item = ((int64_t)blockIdx.x * 256 + threadIdx.x) / nl;
  const int part = threadIdx.x & (nl - 1), n0 = 4 * part;
  const bool on = item < (int64_t)g.B * g.D;  // lanes without a channel stay for the sums
  const int64_t it = on ? item : 0;
  const int64_t b = it / g.D;
  const int d = (int)(it - b * g.D), gi = d / g.DG;
  float A2[4], h[4];
  const float* hp = state_in + it * g.N + n0;
  if (vec && n0 < g.N) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(hp);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = v[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = n0 + j < g.N ? hp[j] : 0.f;
  }
  scan_rates<4>(A_log, g, d, n0, A2);
  const float bias = dt_bias ? dt_bias[d] : 0.f, sk = skip ? skip[d] : 0.f;
  for (int t = 0; t < g.T; ++t) {
    const int64_t tok = b * g.T + t;
    const float xv = (float)static_cast<const E*>(x.p)[tok * x.ld + d];
    const float dl = gate_softplus((float)dt[tok * g.lddt + d] + bias);
    const float u = dl * xv;
    const E* bp = Bm + tok * g.ldb + (int64_t)gi * g.N + n0;
    const E* cp = Cm + tok * g.ldc + (int64_t)gi * g.N + n0;
    float acc = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = n0 + j < g.N;
      h[j] = fmaf(fast_exp2(dl * A2[j]), h[j], in ? (float)bp[j] * u : 0.f);
      if (in) acc = fmaf((float)cp[j], h[j], acc);
    }
    for (int o = nl >> 1; o; o >>= 1) acc += __shfl_xor(acc, o, 64);
    if (on && part == 0) {
      float v = fmaf(sk, xv, acc);
      if (z.p) {
        const float zv = (float)static_cast<const E*>(z.p)[tok * z.ld + d];
        v *= zv * fast_sigmoid(zv);
      }
      y[tok * g.D + d] = (E)v;
    }
  }
  if (!on) return;
  float* op = state_out + it * g.N + n0;
  if (vec && n0 < g.N) {
    *reinterpret_cast<f32x4*>(op) = f32x4{h[0], h[1], h[2], h[3]};
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n0 + j < g.N) op[j] = h[j];
  }
}

}  // namespace gdn
