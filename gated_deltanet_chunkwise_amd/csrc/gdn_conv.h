// gdn_conv.h -- short causal depthwise convolution on gfx950.
//
//     s[t,c] = bias[c] + sum_{j<W} weight[c,j] x[t-W+1+j,c],   y = s or s/(1+e^-s)
// per sequence, W in {2, 3, 4}; inputs before a sequence's first token come from
// its initial state [W-1][C] (oldest first) or are 0.  The final state holds the
// sequence's last W-1 inputs.
//
// Copy-bound: a lane owns VEC neighbouring channels and walks down a tile of tokens
// with the W-1 previous inputs in registers, so each input is read once per tile (W-1
// rows more at a tile's start, which its neighbour has just brought into the L2).  All
// sums are fp32; y is rounded once.
//
// Channels per lane, forward, W=4, us from memory (with the number of waves per CU that
// suits each): B=4, T=8192, C=2048 bf16 (268 MB) one 69, two 51 (5.2 TB/s, a copy's), four 53,
// eight 55; B=2, T=2048 13.0, 11.1, 11.5, 15.0; B=1, T=300 4.1, 4.3, 4.8, 6.7: fewer bytes per
// load, but more waves and fewer registers.  fp32 T=8192 one 111, four 109; T=5003, C=1000 one
// 10.0, four 11.0, packed in seven sequences with W=3 14.3 and 10.9.  Hence two of bf16 and
// four of fp32; an odd number of channels goes one by one (us a call, bf16 T=8192: C=2048 49,
// C=2047 66; backward 96 and 137).
#pragma once
#include "gdn_layer.h"

namespace gdn {

struct ConvGeo {
  int B, T, C, N;    // N = sequences; packed sequences: B = 1
  int cvn;           // vectors per row
  int nblk;          // checkpoint scales per row
  int tile, ntiles;  // tokens per tile; tiles per row of the batch
  int silu;
  int zero;          // forward: y's rows behind the last sequence are set to 0
  const int64_t* cu;  // packed offsets or nullptr
};

__device__ __forceinline__ float conv_act(float s, bool silu) { return silu ? s * fast_sigmoid(s) : s; }

// The inputs at place q of sequence n (q < 0: rows of the initial state, or zeros),
// behind one load whatever the place, so that loads of several rows are in flight
// together.  x from a checkpoint: the initial state is read on its own.
template <typename E, int W, int VEC>
__device__ __forceinline__ RawVec<E, VEC> conv_row(const ConvGeo& g, const Src& x, const E* h0, int n,
                                                   int start, int q, int c) {
  if (x.scales) {
    if (q >= 0) return raw_load<E, VEC>(x, start + q, c, g.nblk);
    RawVec<E, VEC> r = {};
    if (h0) r = raw_load<E, VEC>(Src{h0, nullptr, g.C}, (int64_t)n * (W - 1) + (W - 1 + q), c, 0);
    return r;
  }
  const E* p = static_cast<const E*>(x.p) + (int64_t)(start + max(q, 0)) * x.ld;
  const bool before = q < 0;
  if (before && h0) p = h0 + ((int64_t)n * (W - 1) + (W - 1 + q)) * g.C;
  RawVec<E, VEC> r = raw_load<E, VEC>(Src{p, nullptr, 0}, 0, c, 0);
  if (before && !h0) r = {};
  return r;
}
template <typename E, int W, int VEC>
__device__ __forceinline__ void conv_value(const RawVec<E, VEC>& r, bool packed, int q, float (&v)[VEC]) {
  raw_unpack<E, VEC>(r, packed && q >= 0, v);
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
// the final state.  Consecutive lanes take consecutive vectors of a row.  The rows of a
// tile's first group are sent for before the weights, and before the search for the
// sequence that they are in: a lane's life is little more than its loads' latency.
template <typename E, int W, int VEC>
__global__ __launch_bounds__(256) void gdn_conv_fwd_kernel(ConvGeo g, Src x,
                                                           const float* __restrict__ weight,
                                                           const float* __restrict__ bias,
                                                           const E* __restrict__ h0,
                                                           E* __restrict__ y, E* __restrict__ fin) {
  const uint32_t item = blockIdx.x * 256u + threadIdx.x;  // below 2^32, see the host
  const uint32_t unit = item / (uint32_t)g.cvn;
  const int c = (int)(item - unit * g.cvn) * VEC;
  const uint32_t tiles = (uint32_t)g.ntiles * (g.cu ? 1 : g.B);
  if (unit >= tiles) {
    const uint32_t r = unit - tiles;
    if (!fin || r >= (uint64_t)g.N * (W - 1)) return;
    const int n = r / (W - 1), row = r - n * (W - 1);
    const int start = g.cu ? seq_offset(g.cu, n, g.T) : n * g.T;
    const int end = g.cu ? seq_offset(g.cu, n + 1, g.T) : start + g.T;
    const int len = max(end - start, 0);
    float v[VEC];
    // (a row of the initial state where there are no tokens at all)
    if (len == 0 && !h0)
      for (int i = 0; i < VEC; ++i) v[i] = 0.f;
    else conv_value<E, W, VEC>(conv_row<E, W, VEC>(g, x, h0, n, start, len - (W - 1) + row, c), false, 0, v);
    vec_store<E, VEC>(fin + (int64_t)r * g.C + c, v);
    return;
  }
  const bool silu = g.silu;
  Run<false> run;
  run.place(g.cu, g.T, g.N, (int)unit, g.ntiles, g.tile);
  const int ta = run.ta;
  RawVec<E, VEC> old[W - 1], raw[kConvGroup];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) old[j] = raw_load<E, VEC>(x, max(ta - (W - 1) + j, 0), c, 0);
#pragma unroll
  for (int k = 0; k < kConvGroup; ++k) raw[k] = raw_load<E, VEC>(x, min(ta + k, run.t1 - 1), c, 0);
  // the inputs before a run: those already on their way, unless its sequence has just begun
  auto before = [&]() {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      old[j] = conv_row<E, W, VEC>(g, x, h0, run.n, run.start, run.ta - run.start - (W - 1) + j, c);
  };
  auto first = [&]() {
    before();
#pragma unroll
    for (int k = 0; k < kConvGroup; ++k) raw[k] = raw_load<E, VEC>(x, min(run.ta + k, run.tb - 1), c, 0);
  };
  auto leave = [&]() {
    if (!g.zero) return;
    const float none[VEC] = {};
    for (int t = run.rest; t < run.t1; ++t) vec_store<E, VEC>(y + (int64_t)t * g.C + c, none);
  };
  run.locate();
  if (run.done()) return leave();
  if (run.ta != ta) first();  // only with ill-formed offsets
  else if (run.ta - run.start < W - 1) before();
  float w[VEC][W], b[VEC];
  conv_params<W, VEC>(weight, bias, c, w, b);
  for (;;) {
    float win[W - 1][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) conv_value<E, W, VEC>(old[j], false, 0, win[j]);
    for (int t = run.ta; t < run.tb; t += kConvGroup) {
      if (t > run.ta) {
#pragma unroll
        for (int k = 0; k < kConvGroup; ++k) raw[k] = raw_load<E, VEC>(x, min(t + k, run.tb - 1), c, 0);
      }
#pragma unroll
      for (int k = 0; k < kConvGroup; ++k) {
        if (t + k >= run.tb) break;
        float cur[VEC], out[VEC];
        raw_unpack<E, VEC>(raw[k], false, cur);
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
    run.next();
    if (run.done()) return leave();
    first();
  }
}

// T tokens of each of B sequences after its state [B][W-1][C], which is written
// back (state_out may be state_in: a lane reads its channels' rows before it
// writes them, and no other lane touches them).  One token, W=4, us with two channels of
// bf16 per lane and with eight: B=64, C=2048 2.6 and 4.0 (the latency of one lane's loads),
// B=256, C=8192 7.2 (29 MB, in the caches) and 14.7.  fp32, us a call, with one channel per
// lane and with four: B=64, C=2048 10.1 and 10.1 (the host), B=256, C=8192 11.8 and 12.8,
// B=2048, C=8192 91 and 110.
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

// dy times the activation's slope at s.
__device__ __forceinline__ float conv_dact(float s, float dy, bool silu) {
  return silu ? dy * silu_slope(s, fast_sigmoid(s)) : dy;
}

// d_initial of one (sequence, vector): the first W-1 outputs' p once more.
template <typename E, int W, int VEC>
__device__ __forceinline__ void conv_bwd_state(const ConvGeo& g, const Src& x, const float* weight,
                                               const float* bias, const E* h0, const E* d_y,
                                               const E* d_fin, E* dh0, int n, int c) {
  const int start = g.cu ? seq_offset(g.cu, n, g.T) : n * g.T;
  const int end = g.cu ? seq_offset(g.cu, n + 1, g.T) : start + g.T;
  const int len = max(end - start, 0);
  const bool packed = x.scales != nullptr;
  float out[W - 1][VEC];
#pragma unroll
  for (int r = 0; r < W - 1; ++r) {
    const int kept = r - len;  // the final row that holds row r, if any
    if (d_fin && kept >= 0) vec_load<E, VEC>(d_fin + ((int64_t)n * (W - 1) + kept) * g.C + c, out[r]);
    else
#pragma unroll
      for (int i = 0; i < VEC; ++i) out[r][i] = 0.f;
  }
  if (len > 0) {
    RawVec<E, VEC> raw[2 * (W - 1)], rd[W - 1];  // places -(W-1) .. W-2, held to the last
#pragma unroll
    for (int j = 0; j < 2 * (W - 1); ++j)
      raw[j] = conv_row<E, W, VEC>(g, x, h0, n, start, min(j - (W - 1), len - 1), c);
#pragma unroll
    for (int q = 0; q < W - 1; ++q) rd[q] = raw_load<E, VEC>(Src{d_y, nullptr, g.C}, start + min(q, len - 1), c, 0);
    float w[VEC][W], b[VEC], line[2 * (W - 1)][VEC];
    conv_params<W, VEC>(weight, bias, c, w, b);
#pragma unroll
    for (int j = 0; j < 2 * (W - 1); ++j) conv_value<E, W, VEC>(raw[j], packed, j - (W - 1), line[j]);
#pragma unroll
    for (int q = 0; q < W - 1; ++q) {
      if (q >= len) break;
      float d[VEC];
      raw_unpack<E, VEC>(rd[q], false, d);
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        float s = b[i];
#pragma unroll
        for (int j = 0; j < W; ++j) s = fmaf(w[i][j], line[q + j][i], s);
        const float p = conv_dact(s, d[i], g.silu);
#pragma unroll
        for (int r = q; r < W - 1; ++r) out[r][i] = fmaf(w[i][r - q], p, out[r][i]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < W - 1; ++r) vec_store<E, VEC>(dh0 + ((int64_t)n * (W - 1) + r) * g.C + c, out[r]);
}

constexpr int kConvTiles = 4;  // tiles per workgroup, a wave each

// A wave owns 64 neighbouring vectors of channels (its last lanes beyond C hold the last
// vector once more: they store the same values again and their sums are not used) and a
// tile.  Block id = (group of tiles, channel group), the latter fastest; blocks behind
// those form d_initial.  partial [tile groups][W + 1][C]: dweight's W rows, then dbias.
//
// Bound by memory, and by how much of it is in flight: the loads of U tokens are sent for
// ahead of the U being computed (144 us without that, 105 with, four channels per lane at
// the first size below).  B=4, T=8192, C=2048, W=4 bf16 (403 MB, 79 us at a copy's 5.1 TB/s):
// 96 us.  Channels per lane, us, before the tiles were held to 80 tokens: there one 112, two
// 109, four 114; B=4, T=4096 57, 56, 64; B=2, T=2048 21, 23, 28; fp32 T=8192 one 184, four
// 189.  Hence two of bf16 and one of fp32; U = 4 in fp32 (128 us against 141 with 8 where
// x and d_y were one tensor).
// Tiles are uniform over a wave, so the row pointers are scalar and the middle of a tile
// has no branches: with stores under a lane's condition, every wait for loads is also one
// for the stores before them (154 us).
template <typename E, int W, int VEC, bool CK>
__global__ __launch_bounds__(64 * kConvTiles, 2) void gdn_conv_bwd_kernel(
    ConvGeo g, Src x, const float* __restrict__ weight, const float* __restrict__ bias,
    const E* __restrict__ h0, const E* __restrict__ d_y, const E* __restrict__ d_fin, E* __restrict__ dx,
    E* __restrict__ dh0, float* __restrict__ partial, int cgroups, int main_blocks) {
  constexpr int U = sizeof(E) == 2 ? kConvGroup : kConvGroup / 2;
  __shared__ float sm[64 * kConvTiles * VEC];
  if ((int)blockIdx.x >= main_blocks) {
    const uint32_t item = (blockIdx.x - main_blocks) * (64u * kConvTiles) + threadIdx.x;
    const uint32_t n = item / (uint32_t)g.cvn;
    if (n < (uint32_t)g.N)
      conv_bwd_state<E, W, VEC>(g, x, weight, bias, h0, d_y, d_fin, dh0, (int)n, (int)(item - n * g.cvn) * VEC);
    return;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tg = blockIdx.x / cgroups, cg = blockIdx.x - tg * cgroups;
  const int c = min(cg * 64 + lane, g.cvn - 1) * VEC;
  const int tiles = g.ntiles * (g.cu ? 1 : g.B);
  const int tile = tg * kConvTiles + wave;
  const bool silu = g.silu;
  const Src dys{d_y, nullptr, g.C};
  const uint32_t off = lane_offset(c * (uint32_t)sizeof(E)), xoff = CK ? lane_offset(c) : off;
  const uint32_t soff = CK ? lane_offset((uint32_t)c >> 5) : 0;

  float dw[W][VEC], db[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    db[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
  }
  if (tile < tiles) {
    if (g.cu) {  // rows behind the last sequence get a zero gradient
      const int last = uniform<true>(seq_offset(g.cu, g.N, g.T));
      const float zero[VEC] = {};
      for (int t = max(tile * g.tile, last); t < min((tile + 1) * g.tile, g.T); ++t)
        vec_store<E, VEC>(dx + (int64_t)t * g.C + c, zero);
    }
    Run<true> run;
    run.init(g.cu, g.T, g.N, tile, g.ntiles, g.tile);
    float w[VEC][W], b[VEC];
    if (!run.done()) conv_params<W, VEC>(weight, bias, c, w, b);
    for (; !run.done(); run.next()) {
      const int lim = run.tb + (W - 1);  // tokens at or beyond the sequence's end have p = 0
      const int stop = min(lim, run.end);
      RawVec<E, VEC> old[W - 1];
      TokenVals<E, VEC, U, CK> rx;
      TokenVals<E, VEC, U, false> rd;
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        old[j] = conv_row<E, W, VEC>(g, x, h0, run.n, run.start, run.ta - run.start - (W - 1) + j, c);
      rx.fetch(x, run.ta, stop, xoff, soff, g.nblk);
      rd.fetch(dys, run.ta, stop, off, 0, 0);
      float win[W - 1][VEC], p[W][VEC];  // p[i]: p of the token i before the current one
#pragma unroll
      for (int j = 0; j < W - 1; ++j) conv_value<E, W, VEC>(old[j], CK, run.ta - run.start - (W - 1) + j, win[j]);
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) p[j][i] = 0.f;
      // one token; `edge`: one of the tile's first or last, whose conditions it checks
      auto token = [&](int u, const RawVec<E, VEC>& rawx, const RawVec<E, VEC>& rawd, bool edge) {
        float cur[VEC], d[VEC];
        raw_unpack<E, VEC>(rawx, CK, cur);
        raw_unpack<E, VEC>(rawd, false, d);
        const bool live = !edge || u < stop;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
#pragma unroll
          for (int j = W - 1; j > 0; --j) p[j][i] = p[j - 1][i];
          float s = b[i];
#pragma unroll
          for (int j = 0; j < W - 1; ++j) s = fmaf(w[i][j], win[j][i], s);
          s = fmaf(w[i][W - 1], cur[i], s);
          p[0][i] = live ? conv_dact(s, d[i], silu) : 0.f;
        }
        if (!edge || u < run.tb) {  // a token of this tile's own
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            db[i] += p[0][i];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) dw[j][i] = fmaf(p[0][i], win[j][i], dw[j][i]);
            dw[W - 1][i] = fmaf(p[0][i], cur[i], dw[W - 1][i]);
          }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
#pragma unroll
          for (int j = 0; j < W - 2; ++j) win[j][i] = win[j + 1][i];
          win[W - 2][i] = cur[i];
        }
        const int o = u - (W - 1);  // its later outputs are all known now
        if (!edge || o >= run.ta) {
          float out[VEC];
          const int row = o - run.end + (W - 1);  // >= 0: held in the final state
          if (edge && d_fin && row >= 0) vec_load<E, VEC>(d_fin + ((int64_t)run.n * (W - 1) + row) * g.C + c, out);
          else
#pragma unroll
            for (int i = 0; i < VEC; ++i) out[i] = 0.f;
#pragma unroll
          for (int i = 0; i < VEC; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) out[i] = fmaf(w[i][j], p[j][i], out[i]);
          vec_store<E, VEC>(reinterpret_cast<E*>(reinterpret_cast<char*>(dx + (int64_t)o * g.C) + off), out);
        }
        __builtin_amdgcn_sched_barrier(0);  // token by token: interleaved they take all registers
      };
      for (int t = run.ta; t < lim; t += U) {
        const TokenVals<E, VEC, U, CK> cx = rx;
        const TokenVals<E, VEC, U, false> cd = rd;
        const int next = min(t + U, stop - 1);
        rx.fetch(x, next, stop, xoff, soff, g.nblk);
        rd.fetch(dys, next, stop, off, 0, 0);
        if (t >= run.ta + W - 1 && t + U <= run.tb) {
#pragma unroll
          for (int k = 0; k < U; ++k) token(t + k, cx.v[k], cd.v[k], false);
        } else {
#pragma unroll
          for (int k = 0; k < U; ++k)
            if (t + k < lim) token(t + k, cx.v[k], cd.v[k], true);
        }
      }
    }
  }
  // partial sums over the workgroup's tiles, one of the W + 1 rows at a time
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VEC; ++i) sm[(wave * VEC + i) * 64 + lane] = k < W ? dw[k < W ? k : 0][i] : db[i];
    __syncthreads();
    for (int e = threadIdx.x; e < 64 * VEC; e += 64 * kConvTiles) {
      const int i = e / 64, l = e - i * 64;
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < kConvTiles; ++q) s += sm[(q * VEC + i) * 64 + l];
      const int ch = (cg * 64 + l) * VEC + i;
      if (ch < g.C) partial[((int64_t)tg * (W + 1) + k) * g.C + ch] = s;
    }
  }
}

// dweight [C][W] and dbias [C] from the partial rows: a workgroup adds 64
// neighbouring values, 16 lanes of rows each.
template <int W>
__global__ __launch_bounds__(1024) void gdn_conv_bwd_sums_kernel(const float* __restrict__ partial,
                                                                 int rows, int C,
                                                                 float* __restrict__ dweight,
                                                                 float* __restrict__ dbias) {
  __shared__ float sm[1024];
  const int64_t e = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63), n = (int64_t)(W + 1) * C;
  const int q = threadIdx.x >> 6;
  float s = 0.f;
  if (e < n) {
#pragma unroll 8
    for (int r = q; r < rows; r += 16) s += partial[r * n + e];
  }
  sm[threadIdx.x] = s;
  __syncthreads();
  if (q || e >= n) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += sm[64 * i + threadIdx.x];
  const int k = (int)(e / C), c = (int)(e - (int64_t)k * C);
  if (k < W) dweight[(int64_t)c * W + k] = s;
  else if (dbias) dbias[c] = s;
}

}  // namespace gdn
