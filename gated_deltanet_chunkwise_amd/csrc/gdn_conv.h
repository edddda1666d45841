// gdn_conv.h -- short causal depthwise convolution on gfx950.
//
//     s[t,c] = bias[c] + sum_{j<W} weight[c,j] x[t-W+1+j,c],   y = s or s/(1+e^-s)
// per sequence, W in {2, 3, 4}; inputs before a sequence's first token come from
// its initial state [W-1][C] (oldest first) or are 0.  The final state holds the
// sequence's last W-1 inputs.
//
// Copy-bound: a lane owns VEC neighbouring channels (16 bytes) and walks down a
// tile of tokens with the W-1 previous inputs in registers, so each input is read
// once per tile (W-1 rows more at a tile's start, which its neighbour has just
// brought into the L2).  All sums are fp32; y is rounded once.
#pragma once
#include "gdn_layer.h"

namespace gdn {

struct ConvGeo {
  int B, T, C, N;    // N = sequences; packed sequences: B = 1
  int cvn;           // vectors per row
  int nblk;          // checkpoint scales per row
  int tile, ntiles;  // tokens per tile; tiles per row of the batch
  int silu;
  const int64_t* cu;  // packed offsets or nullptr
};

__device__ __forceinline__ float conv_act(float s, bool silu) { return silu ? s * fast_sigmoid(s) : s; }

// Row of the sequence's inputs at place p (p < 0: the initial state), as fp32.
template <typename E, int W, int VEC>
__device__ __forceinline__ void conv_before(const ConvGeo& g, const Src& x, const E* h0, int n,
                                            int64_t start, int64_t p, int c, float (&v)[VEC]) {
  if (p >= 0) {
    raw_unpack<E, VEC>(raw_load<E, VEC>(x, start + p, c, g.nblk), x.scales != nullptr, v);
  } else if (h0) {
    vec_load<E, VEC>(h0 + ((int64_t)n * (W - 1) + (W - 1 + p)) * g.C + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = 0.f;
  }
}

template <int W, int VEC>
__device__ __forceinline__ void conv_params(const float* weight, const float* bias, int c,
                                            float (&w)[VEC][W], float (&b)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[i][j] = weight[(int64_t)(c + i) * W + j];
    b[i] = bias ? bias[c + i] : 0.f;
  }
}

constexpr int kConvGroup = 8;  // tokens whose loads are in flight together

// Work items: (tile, vector of channels), then (sequence, state row, vector) for
// the final state.  Consecutive lanes take consecutive vectors of a row.
template <typename E, int W, int VEC>
__global__ __launch_bounds__(256) void gdn_conv_fwd_kernel(ConvGeo g, Src x,
                                                           const float* __restrict__ weight,
                                                           const float* __restrict__ bias,
                                                           const E* __restrict__ h0,
                                                           E* __restrict__ y, E* __restrict__ fin) {
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t unit = item / g.cvn;
  const int c = (int)(item - unit * g.cvn) * VEC;
  const int64_t tiles = (int64_t)g.ntiles * (g.cu ? 1 : g.B);
  if (unit >= tiles) {
    const int64_t r = unit - tiles;
    if (!fin || r >= (int64_t)g.N * (W - 1)) return;
    const int n = (int)(r / (W - 1)), row = (int)(r - (int64_t)n * (W - 1));
    const int64_t start = g.cu ? seq_offset(g.cu, n, g.T) : (int64_t)n * g.T;
    const int64_t end = g.cu ? seq_offset(g.cu, n + 1, g.T) : start + g.T;
    const int64_t len = end > start ? end - start : 0;
    float v[VEC];
    conv_before<E, W, VEC>(g, x, h0, n, start, len - (W - 1) + row, c, v);
    vec_store<E, VEC>(fin + r * g.C + c, v);
    return;
  }
  float w[VEC][W], b[VEC];
  conv_params<W, VEC>(weight, bias, c, w, b);
  const bool silu = g.silu;
  Run<false> run;
  run.init(g.cu, g.T, g.N, (int)unit, g.ntiles, g.tile);
  for (; !run.done(); run.next()) {
    float win[W - 1][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      conv_before<E, W, VEC>(g, x, h0, run.n, run.start, run.ta - run.start - (W - 1) + j, c, win[j]);
    for (int t = run.ta; t < run.tb; t += kConvGroup) {
      RawVec<E, VEC> raw[kConvGroup];
#pragma unroll
      for (int k = 0; k < kConvGroup; ++k)
        raw[k] = raw_load<E, VEC>(x, min(t + k, run.tb - 1), c, g.nblk);
#pragma unroll
      for (int k = 0; k < kConvGroup; ++k) {
        if (t + k >= run.tb) break;
        float cur[VEC], out[VEC];
        raw_unpack<E, VEC>(raw[k], x.scales != nullptr, cur);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          float s = b[i];
#pragma unroll
          for (int j = 0; j < W - 1; ++j) s = fmaf(w[i][j], win[j][i], s);
          s = fmaf(w[i][W - 1], cur[i], s);
          out[i] = conv_act(s, silu);
        }
        vec_store<E, VEC>(y + (int64_t)(t + k) * g.C + c, out);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
#pragma unroll
          for (int j = 0; j < W - 2; ++j) win[j][i] = win[j + 1][i];
          win[W - 2][i] = cur[i];
        }
      }
    }
  }
}

// T tokens of each of B sequences after its state [B][W-1][C], which is written
// back (state_out may be state_in: a lane reads its channels' rows before it
// writes them, and no other lane touches them).
template <typename E, int W, int VEC>
__global__ __launch_bounds__(256) void gdn_conv_decode_kernel(ConvGeo g, Src x,
                                                              const float* __restrict__ weight,
                                                              const float* __restrict__ bias,
                                                              const E* state_in, E* state_out,
                                                              E* __restrict__ y) {
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t n = item / g.cvn;
  if (n >= g.B) return;
  const int c = (int)(item - n * g.cvn) * VEC;
  float win[W - 1][VEC];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) vec_load<E, VEC>(state_in + (n * (W - 1) + j) * g.C + c, win[j]);
  RawVec<E, VEC> next = raw_load<E, VEC>(x, n * g.T, c, g.nblk);
  float w[VEC][W], b[VEC];
  conv_params<W, VEC>(weight, bias, c, w, b);
  for (int t = 0; t < g.T; ++t) {
    float cur[VEC], out[VEC];
    raw_unpack<E, VEC>(next, false, cur);
    if (t + 1 < g.T) next = raw_load<E, VEC>(x, n * g.T + t + 1, c, g.nblk);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float s = b[i];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) s = fmaf(w[i][j], win[j][i], s);
      s = fmaf(w[i][W - 1], cur[i], s);
      out[i] = conv_act(s, g.silu);
    }
    vec_store<E, VEC>(y + (n * g.T + t) * g.C + c, out);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
      for (int j = 0; j < W - 2; ++j) win[j][i] = win[j + 1][i];
      win[W - 2][i] = cur[i];
    }
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) vec_store<E, VEC>(state_out + (n * (W - 1) + j) * g.C + c, win[j]);
}

// ---- backward --------------------------------------------------------------------
// With p[t] = dL/ds[t] = dy[t] act'(s[t]) (s formed again from x):
//     dx[t]       = sum_{i<W, t+i<end} weight[W-1-i] p[t+i]  (+ d_final of the row that holds x[t])
//     dweight[j]  = sum_t p[t] x[t-W+1+j],   dbias = sum_t p[t]
//     d_initial[r] = sum_{q<=r, q<len} weight[r-q] p[q]      (+ d_final of the row that holds it)
// A lane walks down its tile as the forward pass does, W-1 tokens further than it
// owns (they are formed again by the next tile), and holds the last W values of p.
// The weight's and bias's sums stay in registers over the tile; the lanes of a
// workgroup that own the same channels add theirs through LDS, and each workgroup
// writes one row of partial sums, added up in a fixed order by the sums kernel.

template <int W>
__device__ __forceinline__ float conv_dact(float s, float dy, bool silu) {
  if (!silu) return dy;
  const float sg = fast_sigmoid(s);
  // d/ds s sg = sg + s sg (1 - sg); 1 - sg formed as sigmoid(-s) keeps it exact
  // where sg rounds to 1
  return dy * fmaf(s * sg, fast_sigmoid(-s), sg);
}

// Workgroup: cl lanes (a power of two) of neighbouring vectors times 256 / cl tiles.
// Block id = (group of tiles, channel group of cl vectors), the latter fastest.
// partial [tile groups][W + 1][C]: dweight's W rows, then dbias.
template <typename E, int W, int VEC>
__global__ __launch_bounds__(256) void gdn_conv_bwd_kernel(ConvGeo g, Src x,
                                                           const float* __restrict__ weight,
                                                           const float* __restrict__ bias,
                                                           const E* __restrict__ h0,
                                                           const E* __restrict__ d_y,
                                                           const E* __restrict__ d_fin,
                                                           E* __restrict__ dx,
                                                           float* __restrict__ partial, int cl,
                                                           int cgroups) {
  __shared__ float sm[256 * VEC];
  const int tl = 256 / cl, lc = threadIdx.x & (cl - 1), lt = threadIdx.x / cl;
  const int tg = blockIdx.x / cgroups, cg = blockIdx.x - tg * cgroups;
  const int v = cg * cl + lc;
  const bool on = v < g.cvn;
  const int c = (on ? v : 0) * VEC;
  const int64_t tiles = (int64_t)g.ntiles * (g.cu ? 1 : g.B);
  const int64_t tile = (int64_t)tg * tl + lt;
  const bool silu = g.silu, packed = x.scales != nullptr;
  const Src dys{d_y, nullptr, g.C};

  float dw[W][VEC], db[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    db[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
  }
  if (on && tile < tiles) {
    float w[VEC][W], b[VEC];
    conv_params<W, VEC>(weight, bias, c, w, b);
    Run<false> run;
    run.init(g.cu, g.T, g.N, (int)tile, g.ntiles, g.tile);
    if (g.cu) {  // rows behind the last sequence get a zero gradient
      const int64_t last = seq_offset(g.cu, g.N, g.T);
      const float zero[VEC] = {};
      for (int64_t t = max((int64_t)tile * g.tile, last); t < min((int64_t)(tile + 1) * g.tile, (int64_t)g.T); ++t)
        vec_store<E, VEC>(dx + t * g.C + c, zero);
    }
    for (; !run.done(); run.next()) {
      float win[W - 1][VEC], p[W][VEC];  // p[i]: p of the token i before the current one
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        conv_before<E, W, VEC>(g, x, h0, run.n, run.start, run.ta - run.start - (W - 1) + j, c, win[j]);
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) p[j][i] = 0.f;
      const int lim = run.tb + (W - 1);  // tokens at or beyond the sequence's end have p = 0
      const int stop = min(lim, run.end);
      for (int t = run.ta; t < lim; t += kConvGroup / 2) {
        RawVec<E, VEC> rx[kConvGroup / 2], rd[kConvGroup / 2];
#pragma unroll
        for (int k = 0; k < kConvGroup / 2; ++k) {
          const int q = min(t + k, stop - 1);
          rx[k] = raw_load<E, VEC>(x, q, c, g.nblk);
          rd[k] = raw_load<E, VEC>(dys, q, c, 0);
        }
#pragma unroll
        for (int k = 0; k < kConvGroup / 2; ++k) {
          const int u = t + k;
          if (u >= lim) break;
          float cur[VEC], d[VEC];
          raw_unpack<E, VEC>(rx[k], packed, cur);
          raw_unpack<E, VEC>(rd[k], false, d);
          const bool live = u < stop, own = u < run.tb;
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
#pragma unroll
            for (int j = W - 1; j > 0; --j) p[j][i] = p[j - 1][i];
            float s = b[i];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) s = fmaf(w[i][j], win[j][i], s);
            s = fmaf(w[i][W - 1], cur[i], s);
            p[0][i] = live ? conv_dact<W>(s, d[i], silu) : 0.f;
            if (own) {
              db[i] += p[0][i];
#pragma unroll
              for (int j = 0; j < W - 1; ++j) dw[j][i] = fmaf(p[0][i], win[j][i], dw[j][i]);
              dw[W - 1][i] = fmaf(p[0][i], cur[i], dw[W - 1][i]);
            }
#pragma unroll
            for (int j = 0; j < W - 2; ++j) win[j][i] = win[j + 1][i];
            win[W - 2][i] = cur[i];
          }
          const int o = u - (W - 1);  // its later outputs are all known now
          if (o >= run.ta) {
            float out[VEC];
            const int row = o - run.end + (W - 1);  // >= 0: held in the final state
            if (d_fin && row >= 0) vec_load<E, VEC>(d_fin + ((int64_t)run.n * (W - 1) + row) * g.C + c, out);
            else
#pragma unroll
              for (int i = 0; i < VEC; ++i) out[i] = 0.f;
#pragma unroll
            for (int i = 0; i < VEC; ++i)
#pragma unroll
              for (int j = 0; j < W; ++j) out[i] = fmaf(w[i][j], p[j][i], out[i]);
            vec_store<E, VEC, true>(dx + (int64_t)o * g.C + c, out);
          }
        }
      }
    }
  }
  // partial sums over the workgroup's tiles, one of the W + 1 rows at a time
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VEC; ++i) sm[i * 256 + threadIdx.x] = k < W ? dw[k < W ? k : 0][i] : db[i];
    __syncthreads();
    for (int e = threadIdx.x; e < cl * VEC; e += 256) {
      const int i = e / cl, l = e - i * cl;
      float s = 0.f;
      for (int q = 0; q < tl; ++q) s += sm[i * 256 + q * cl + l];
      const int ch = (cg * cl + l) * VEC + i;
      if (ch < g.C) partial[((int64_t)tg * (W + 1) + k) * g.C + ch] = s;
    }
  }
}

// d_initial, one lane per (sequence, vector): the first W-1 outputs' p once more.
template <typename E, int W, int VEC>
__global__ __launch_bounds__(256) void gdn_conv_bwd_state_kernel(
    ConvGeo g, Src x, const float* __restrict__ weight, const float* __restrict__ bias,
    const E* __restrict__ h0, const E* __restrict__ d_y, const E* __restrict__ d_fin,
    E* __restrict__ dh0) {
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t n = item / g.cvn;
  if (n >= g.N) return;
  const int c = (int)(item - n * g.cvn) * VEC;
  const int64_t start = g.cu ? seq_offset(g.cu, (int)n, g.T) : n * g.T;
  const int64_t end = g.cu ? seq_offset(g.cu, (int)n + 1, g.T) : start + g.T;
  const int64_t len = end > start ? end - start : 0;
  float w[VEC][W], b[VEC], line[2 * (W - 1)][VEC], out[W - 1][VEC];
  conv_params<W, VEC>(weight, bias, c, w, b);
#pragma unroll
  for (int j = 0; j < 2 * (W - 1); ++j) {  // places -(W-1) .. W-2
    const int64_t q = j - (W - 1);
    conv_before<E, W, VEC>(g, x, h0, (int)n, start, len > 0 ? min(q, len - 1) : min(q, (int64_t)-1), c, line[j]);
  }
#pragma unroll
  for (int r = 0; r < W - 1; ++r) {
    const int64_t kept = r - len;  // the final row that holds row r, if any
    if (d_fin && kept >= 0) vec_load<E, VEC>(d_fin + (n * (W - 1) + kept) * g.C + c, out[r]);
    else
#pragma unroll
      for (int i = 0; i < VEC; ++i) out[r][i] = 0.f;
  }
#pragma unroll
  for (int q = 0; q < W - 1; ++q) {
    if (q >= len) break;
    float d[VEC];
    vec_load<E, VEC>(d_y + (start + q) * g.C + c, d);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float s = b[i];
#pragma unroll
      for (int j = 0; j < W; ++j) s = fmaf(w[i][j], line[q + j][i], s);
      const float p = conv_dact<W>(s, d[i], g.silu);
#pragma unroll
      for (int r = q; r < W - 1; ++r) out[r][i] = fmaf(w[i][r - q], p, out[r][i]);
    }
  }
#pragma unroll
  for (int r = 0; r < W - 1; ++r) vec_store<E, VEC>(dh0 + (n * (W - 1) + r) * g.C + c, out[r]);
}

// dweight [C][W] and dbias [C] from the partial rows: a workgroup adds 64
// neighbouring values, four lanes of rows each.
template <int W>
__global__ __launch_bounds__(256) void gdn_conv_bwd_sums_kernel(const float* __restrict__ partial,
                                                                int rows, int C,
                                                                float* __restrict__ dweight,
                                                                float* __restrict__ dbias) {
  __shared__ float sm[256];
  const int64_t e = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63), n = (int64_t)(W + 1) * C;
  const int q = threadIdx.x >> 6;
  float s = 0.f;
  if (e < n)
    for (int r = q; r < rows; r += 4) s += partial[r * n + e];
  sm[threadIdx.x] = s;
  __syncthreads();
  if (q || e >= n) return;
  s = (sm[threadIdx.x] + sm[64 + threadIdx.x]) + (sm[128 + threadIdx.x] + sm[192 + threadIdx.x]);
  const int k = (int)(e / C), c = (int)(e - (int64_t)k * C);
  if (k < W) dweight[(int64_t)c * W + k] = s;
  else if (dbias) dbias[c] = s;
}

}  // namespace gdn
