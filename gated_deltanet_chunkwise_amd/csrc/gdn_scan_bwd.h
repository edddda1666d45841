// gdn_scan_bwd.h -- the selective scan's backward pass on gfx950.
//
// With r_t = dy_t silu(z_t) and l_t = dL/dh_t:
//     l_t     = Cm_t r_t + a_{t+1} l_{t+1}        (from d_final at a sequence's end)
//     q_t     = l_t a_t h_{t-1}                   (towards the exponent D A)
//     dBm_t   = sum_d l_t D x,   dCm_t = sum_d h_t r_t      (over a group's channels)
//     dx_t    = D sum_n l_t Bm_t + skip r_t
//     dD_t    = x sum_n l_t Bm_t + sum_n A q_t,   ddt = dD softplus'(dt + dt_bias)
//     dz_t    = dy silu'(z) (sum_n Cm h + skip x)
//     dA_log  = A sum_t D q_t,  dskip = sum_t r x,  ddt_bias = sum_t ddt,  d_initial = a_1 l_1
//
// The states are formed again.  Tokens are cut into tiles that run side by side, as in
// the forward pass: (1) each tile's end state from a zero start and, in the same walk,
// what its own tokens send to the state before it (R = sum_t (a_1 .. a_t) Cm_t r_t);
// (2) both joined over the tiles, forwards for the states and backwards for their
// gradients; (3) every tile on its own: forwards once, the state before every group of
// SUB tokens kept in LDS; then, from the last group to the first, forwards again with
// the group's states in registers and backwards through them; (4) sums over waves and
// tiles.  VALU-bound like the forward pass, with about three times its operations.
//
// dBm and dCm need sums over channels, that is over lanes: 2 NS values of a token are
// added over 64 lanes by halving (in each step a lane keeps half of its values and
// hands the others to its partner), 2.2 operations per value instead of 6.
#pragma once
#include "gdn_scan.h"

namespace gdn {

constexpr int kScanBwdStates = 8;  // states per lane
constexpr int kScanBwdSub = 8;     // tokens per group
// Tokens per tile: 64, or 32 where the kept states of eight waves would not fit in LDS.
constexpr int scan_bwd_tile(int waves) { return waves > 4 ? 32 : 64; }

// One channel of one row, codes and scale of a checkpoint in one word.
template <typename E> __device__ __forceinline__ uint32_t src_load1(const Src& s, int64_t row, int d, int nblk) {
  if (s.scales)
    return static_cast<const uint8_t*>(s.p)[row * s.ld + d] | (uint32_t)s.scales[row * nblk + (d >> 5)] << 8;
  return load1<E>(static_cast<const E*>(s.p) + row * s.ld + d);
}
template <typename E> __device__ __forceinline__ float src_value1(const Src& s, uint32_t w) {
  return s.scales ? (float)(int8_t)(w & 255u) * pack_scale(w >> 8) : value1<E>(w);
}

// Sums over the wave's 64 lanes of V values each (V = 16 or 32): returns the sum of
// value lane / (64 / V).
template <int V> __device__ __forceinline__ float wave_sums(float (&v)[V]) {
  static_assert(V == 16 || V == 32, "");
  // lanes 32 apart: the lower half keeps the values below V / 2
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i + V / 2]), false, false);
    v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  // rows of 16 lanes, 16 apart
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[i + V / 4]), false, false);
    v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  auto dpp = [](float x, auto ctrl) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  const int lane = threadIdx.x & 63;
  auto half = [&](int i, int j, int bit, auto ctrl) {
    const bool up = lane & bit;
    const float keep = up ? v[j] : v[i], send = up ? v[i] : v[j];
    v[i] = keep + dpp(send, ctrl);
  };
  using Ror8 = std::integral_constant<int, 0x128>;    // lane xor 8 within a row
  using Mirror = std::integral_constant<int, 0x141>;  // lane -> 7 - lane within 8: bit 2 differs
  using Xor2 = std::integral_constant<int, 0x4E>;
  using Xor1 = std::integral_constant<int, 0xB1>;
#pragma unroll
  for (int i = 0; i < V / 8; ++i) half(i, i + V / 8, 8, Ror8{});
#pragma unroll
  for (int i = 0; i < V / 16; ++i) half(i, i + V / 16, 4, Mirror{});
  if constexpr (V == 32) half(0, 1, 2, Xor2{});
  else v[0] += dpp(v[0], Xor2{});
  return v[0] + dpp(v[0], Xor1{});
}

struct ScanBwdGeo {
  ScanGeo g;
  int nblk;  // checkpoint scales per row
};

// silu'(z) = s + z s (1 - s), s = sigmoid(z); 1 - s as sigmoid(-z).
__device__ __forceinline__ float dsilu(float z, float s) { return fmaf(z * s, fast_sigmoid(-z), s); }

// (1).  states, rev [tile][np][D]; sums, rsums [tile][D] (-1: nothing passes through).
template <typename E, typename BE, int NS, int NW>
__global__ __launch_bounds__(64 * NW) void gdn_scan_bwd_ends_kernel(
    ScanBwdGeo bg, Src x, const E* __restrict__ dt, Src z, const float* __restrict__ A_log,
    const BE* __restrict__ Bm, const BE* __restrict__ Cm, const float* __restrict__ dt_bias,
    const float* __restrict__ h0, const E* __restrict__ d_y, const float* __restrict__ d_fin,
    float* __restrict__ states, float* __restrict__ rev, float* __restrict__ sums,
    float* __restrict__ rsums) {
  constexpr int U = kScanGroup;
  const ScanGeo& g = bg.g;
  ScanPlace w;
  w.init<NS>(g, blockIdx.x);
  float A2[NS], h[NS], P[NS], R[NS];
  scan_rates<NS>(A_log, g, w.d, w.n0, A2);
  const float bias = dt_bias ? dt_bias[w.d] : 0.f;
  const BE* bp = Bm + (int64_t)w.gi * g.bgs + w.n0;
  const BE* cp = Cm + (int64_t)w.gi * g.cgs + w.n0;
  float sum = 0.f, rsum = -1.f;
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    h[j] = R[j] = 0.f;
    P[j] = 1.f;
  }
  Run<true> run;
  run.init(g.cu, g.T, g.S, w.tile, g.ntiles, g.len);
  for (; !run.done(); run.next()) {
    const bool cont = run.ta > run.start;  // only a tile's first run can be
    if (!cont) {
      state_load<NS>(h0, g, run.n, w.d, w.n0, h);
      sum = -1.f;
    }
    float pass = 0.f;
    for (int t = run.ta; t < run.tb; t += U) {
      uint32_t rx[U], rd[U], ry[U] = {}, rz[U] = {};
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int64_t q = min(t + k, run.tb - 1);
        rx[k] = src_load1<E>(x, q, w.d, bg.nblk);
        rd[k] = load1<E>(dt + q * g.lddt + w.d);
        if (cont) {
          ry[k] = load1<E>(d_y + q * g.D + w.d);
          if (z.p) rz[k] = src_load1<E>(z, q, w.d, bg.nblk);
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (t + k >= run.tb) break;
        ScalarRow<BE, NS> b;
        b.load(bp + (int64_t)(t + k) * g.ldb);
        const float dl = softplus_flat(value1<E>(rd[k]) + bias);
        const float u = dl * src_value1<E>(x, rx[k]);
        if (cont) {
          ScalarRow<BE, NS> c;
          c.load(cp + (int64_t)(t + k) * g.ldc);
          float r = value1<E>(ry[k]);
          if (z.p) {
            const float zv = src_value1<E>(z, rz[k]);
            r *= zv * fast_sigmoid(zv);
          }
          pass += dl;
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            const float a = fast_exp2(dl * A2[j]);
            h[j] = fmaf(a, h[j], b[j] * u);
            P[j] *= a;
            R[j] = fmaf(P[j], c[j] * r, R[j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < NS; ++j) h[j] = fmaf(fast_exp2(dl * A2[j]), h[j], b[j] * u);
        }
      }
    }
    if (sum >= 0.f) sum += pass;
    if (cont) {
      if (run.tb == run.end) {
        float f[NS];
        state_load<NS>(d_fin, g, run.n, w.d, w.n0, f);
#pragma unroll
        for (int j = 0; j < NS; ++j) R[j] = fmaf(P[j], f[j], R[j]);
      } else {
        rsum = pass;
      }
    }
  }
  if (!w.on) return;
  const int64_t at = ((int64_t)w.tile * g.np + w.n0) * g.D + w.d;
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    states[at + (int64_t)j * g.D] = h[j];
    rev[at + (int64_t)j * g.D] = R[j];
  }
  if (w.wave == 0) {
    sums[(int64_t)w.tile * g.D + w.d] = sum;
    rsums[(int64_t)w.tile * g.D + w.d] = rsum;
  }
}

// (2), backwards: rev from what each tile sends to the state before it to the gradient
// of each tile's end state, in place.
__global__ __launch_bounds__(256) void gdn_scan_bwd_join_kernel(ScanGeo g, const float* __restrict__ A_log,
                                                                float* __restrict__ rev,
                                                                const float* __restrict__ rsums) {
  constexpr int U = 8;
  const int64_t per = (int64_t)g.np * g.D;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int rows = g.cu ? 1 : g.B;
  if (i >= rows * per) return;
  const int row = (int)(i / per);
  const int64_t r = i - row * per;
  const int n = (int)(r / g.D), d = (int)(r - (int64_t)n * g.D);
  const float A2 = n < g.N ? -expf(A_log[(int64_t)d * g.N + n]) * kLog2e : 0.f;
  float G = 0.f;
  float* p = rev + (int64_t)row * g.ntiles * per + r;
  const float* s = rsums + (int64_t)row * g.ntiles * g.D + d;
  for (int t = g.ntiles - 1; t >= 0; t -= U) {
    float e[U], sm[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int q = max(t - k, 0);
      e[k] = p[q * per];
      sm[k] = s[(int64_t)q * g.D];
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (t - k < 0) break;
      p[(t - k) * per] = G;
      G = sm[k] < 0.f ? e[k] : fmaf(fast_exp2(A2 * sm[k]), G, e[k]);
    }
  }
}

// (3).  states holds the tiles' start states and is overwritten with the tile's part of
// sum_t D q; rev the end states' gradients.  pbc [channel wave][token][2][np]: the
// wave's parts of dBm and dCm.  psum [tile][NW][2][D]: of dskip and ddt_bias.  Blocks
// behind the last tile's copy d_final to d_initial for empty sequences.
template <typename E, typename BE, int NS, int NW, int SUB>
__global__ __launch_bounds__(64 * NW) void gdn_scan_bwd_kernel(
    ScanBwdGeo bg, Src x, const E* __restrict__ dt, Src z, const float* __restrict__ A_log,
    const BE* __restrict__ Bm, const BE* __restrict__ Cm, const float* __restrict__ skip,
    const float* __restrict__ dt_bias, const float* __restrict__ h0, const E* __restrict__ d_y,
    const float* __restrict__ d_fin, float* __restrict__ states, const float* __restrict__ rev,
    E* __restrict__ dx, E* __restrict__ ddt, E* __restrict__ dz, float* __restrict__ pbc,
    float* __restrict__ psum, float* __restrict__ dh0) {
  __shared__ float hs[scan_bwd_tile(NW) / SUB][NW][NS][64];
  __shared__ float part[NW > 1 ? NW : 1][NW > 1 ? SUB : 1][3][NW > 1 ? 64 : 1];
  const ScanGeo& g = bg.g;
  const int64_t ntok = (int64_t)g.B * g.T;
  const uint32_t main_blocks = (uint32_t)(g.ntiles * (g.cu ? 1 : g.B)) * g.cgroups;
  if (blockIdx.x >= main_blocks) {
    scan_empty_state(g, blockIdx.x - main_blocks, d_fin, dh0);
    return;
  }
  ScanPlace w;
  w.init<NS>(g, blockIdx.x);
  const int cg = blockIdx.x % g.cgroups;
  float A2[NS], dA[NS], h[NS], l[NS];
  scan_rates<NS>(A_log, g, w.d, w.n0, A2);
  const float bias = dt_bias ? dt_bias[w.d] : 0.f, sk = skip ? skip[w.d] : 0.f;
  const BE* bp = Bm + (int64_t)w.gi * g.bgs + w.n0;
  const BE* cp = Cm + (int64_t)w.gi * g.cgs + w.n0;
  float dskip = 0.f, dbias = 0.f;
  const int64_t at = ((int64_t)w.tile * g.np + w.n0) * g.D + w.d;
  // this wave's place in a token's row of pbc: lane v of dBm and dCm's 2 NS values
  constexpr int kRep = 64 / (2 * NS);
  const int v = w.lane / kRep;
  float* pb = pbc + ((int64_t)cg * ntok) * 2 * g.np + (v / NS) * g.np + w.n0 + v % NS;
#pragma unroll
  for (int j = 0; j < NS; ++j) dA[j] = 0.f;

  if (g.cu) {  // rows behind the last sequence
    const int last = max(uniform<true>(seq_offset(g.cu, g.S, g.T)), w.tile * g.len);
    for (int t = last; t < min((w.tile + 1) * g.len, g.T); ++t) {
      if (w.on && w.wave == 0) {
        dx[(int64_t)t * g.D + w.d] = (E)0.f;
        ddt[(int64_t)t * g.D + w.d] = (E)0.f;
        if (z.p) dz[(int64_t)t * g.D + w.d] = (E)0.f;
      }
      if (w.lane % kRep == 0) pb[(int64_t)t * 2 * g.np] = 0.f;
    }
  }

  Run<true> run;
  run.init(g.cu, g.T, g.S, w.tile, g.ntiles, g.len);
  for (; !run.done(); run.next()) {
    if (run.ta > run.start) {
#pragma unroll
      for (int j = 0; j < NS; ++j) h[j] = states[at + (int64_t)j * g.D];
    } else {
      state_load<NS>(h0, g, run.n, w.d, w.n0, h);
    }
    if (run.tb == run.end) {
      state_load<NS>(d_fin, g, run.n, w.d, w.n0, l);
    } else {
#pragma unroll
      for (int j = 0; j < NS; ++j) l[j] = rev[at + (int64_t)j * g.D];
    }
#pragma unroll
    for (int j = 0; j < NS; ++j) l[j] = w.on ? l[j] : 0.f;  // lanes without a channel add nothing

    const int nsub = (run.tb - run.ta + SUB - 1) / SUB;
    uint32_t rx[SUB], rd[SUB], ry[SUB], rz[SUB] = {};
    auto fetch = [&](int t, bool all) {
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        const int64_t q = min(t + k, run.tb - 1);
        rx[k] = src_load1<E>(x, q, w.d, bg.nblk);
        rd[k] = load1<E>(dt + q * g.lddt + w.d);
        if (all) {
          ry[k] = load1<E>(d_y + q * g.D + w.d);
          if (z.p) rz[k] = src_load1<E>(z, q, w.d, bg.nblk);
        }
      }
    };
    // forwards: the state before every group
    fetch(run.ta, nsub == 1);
    for (int s = 0; s < nsub; ++s) {
#pragma unroll
      for (int j = 0; j < NS; ++j) hs[s][w.wave][j][w.lane] = h[j];
      if (s == nsub - 1) break;
      const int t = run.ta + s * SUB;
      float xv[SUB], dl[SUB];
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        xv[k] = src_value1<E>(x, rx[k]);
        dl[k] = softplus_flat(value1<E>(rd[k]) + bias);
      }
      fetch(t + SUB, s + 1 == nsub - 1);
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        ScalarRow<BE, NS> b;
        b.load(bp + (int64_t)(t + k) * g.ldb);
        const float u = dl[k] * xv[k];
#pragma unroll
        for (int j = 0; j < NS; ++j) h[j] = fmaf(fast_exp2(dl[k] * A2[j]), h[j], b[j] * u);
      }
    }
    // backwards, group by group
    for (int s = nsub - 1; s >= 0; --s) {
      const int t = run.ta + s * SUB, cnt = min(SUB, run.tb - t);
      float xv[SUB], dl[SUB], raw[SUB], dyv[SUB], zv[SUB], hp[SUB][NS];
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        xv[k] = w.on ? src_value1<E>(x, rx[k]) : 0.f;
        raw[k] = value1<E>(rd[k]) + bias;
        dl[k] = softplus_flat(raw[k]);
        dyv[k] = w.on ? value1<E>(ry[k]) : 0.f;
        zv[k] = src_value1<E>(z, rz[k]);
      }
      if (s > 0) fetch(t - SUB, true);
#pragma unroll
      for (int j = 0; j < NS; ++j) hp[0][j] = hs[s][w.wave][j][w.lane];
#pragma unroll
      for (int k = 0; k + 1 < SUB; ++k) {
        if (k + 1 >= cnt) break;
        ScalarRow<BE, NS> b;
        b.load(bp + (int64_t)(t + k) * g.ldb);
        const float u = dl[k] * xv[k];
#pragma unroll
        for (int j = 0; j < NS; ++j) hp[k + 1][j] = fmaf(fast_exp2(dl[k] * A2[j]), hp[k][j], b[j] * u);
      }
      float yraw[SUB], lb[SUB], aq[SUB];  // sums over the states: Cm h, l Bm, A q
#pragma unroll
      for (int k = SUB - 1; k >= 0; --k) {
        if (k >= cnt) continue;
        ScalarRow<BE, NS> b, c;
        b.load(bp + (int64_t)(t + k) * g.ldb);
        c.load(cp + (int64_t)(t + k) * g.ldc);
        const float u = dl[k] * xv[k];
        const float r = z.p ? dyv[k] * zv[k] * fast_sigmoid(zv[k]) : dyv[k];
        float bc[2 * NS], sy = 0.f, sb = 0.f, sq = 0.f;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const float a = fast_exp2(dl[k] * A2[j]);
          const float ah = a * hp[k][j];
          const float ht = fmaf(b[j], u, ah);
          const float lam = fmaf(c[j], r, l[j]);
          sy = fmaf(c[j], ht, sy);
          sb = fmaf(b[j], lam, sb);
          const float q = lam * ah;
          sq = fmaf(q, A2[j], sq);
          dA[j] = fmaf(q, dl[k], dA[j]);
          bc[j] = lam * u;
          bc[NS + j] = ht * r;
          l[j] = a * lam;
        }
        yraw[k] = sy;
        lb[k] = sb;
        aq[k] = sq;
        const float tot = wave_sums<2 * NS>(bc);
        if (w.lane % kRep == 0) pb[(int64_t)(t + k) * 2 * g.np] = tot;
      }
      if constexpr (NW > 1) {
        __syncthreads();  // the last group's sums are all read
#pragma unroll
        for (int k = 0; k < SUB; ++k) {
          if (k >= cnt) break;
          part[w.wave][k][0][w.lane] = yraw[k];
          part[w.wave][k][1][w.lane] = lb[k];
          part[w.wave][k][2][w.lane] = aq[k];
        }
        __syncthreads();
      }
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        if (k >= cnt) break;
        if constexpr (NW > 1) {
          if (k % g.nw != w.wave) continue;
          yraw[k] = lb[k] = aq[k] = 0.f;
          for (int q = 0; q < g.nw; ++q) {
            yraw[k] += part[q][k][0][w.lane];
            lb[k] += part[q][k][1][w.lane];
            aq[k] += part[q][k][2][w.lane];
          }
        }
        float r = dyv[k];
        const int64_t o = (int64_t)(t + k) * g.D + w.d;
        if (z.p) {
          const float sg = fast_sigmoid(zv[k]);
          if (w.on) dz[o] = (E)(dyv[k] * dsilu(zv[k], sg) * fmaf(sk, xv[k], yraw[k]));
          r *= zv[k] * sg;
        }
        const float dD = fmaf(lb[k], xv[k], aq[k] * 0.693147180559945309f);
        const float dr = raw[k] > 20.f ? dD : dD * fast_sigmoid(raw[k]);
        if (w.on) {
          dx[o] = (E)fmaf(dl[k], lb[k], sk * r);
          ddt[o] = (E)dr;
        }
        dskip = fmaf(r, xv[k], dskip);
        dbias += dr;
      }
    }
    if (dh0 && w.on && run.ta == run.start) state_store<NS>(dh0, g, run.n, w.d, w.n0, l);
  }
  if (!w.on) return;
#pragma unroll
  for (int j = 0; j < NS; ++j) states[at + (int64_t)j * g.D] = dA[j];
  float* ps = psum + ((int64_t)w.tile * g.nw + w.wave) * 2 * g.D + w.d;
  ps[0] = dskip;
  ps[g.D] = dbias;
}

// (4): dBm and dCm, a lane per value, summed over the group's channel waves.
template <typename E>
__global__ __launch_bounds__(256) void gdn_scan_bwd_rows_kernel(ScanGeo g, const float* __restrict__ pbc,
                                                                E* __restrict__ dBm, E* __restrict__ dCm) {
  const int64_t ntok = (int64_t)g.B * g.T, total = ntok * g.G * 2 * g.np;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += step) {
    const int64_t per = ntok * 2 * g.np;
    const int gi = (int)(i / per);
    const int64_t r = i - gi * per;
    const int64_t t = r / (2 * g.np);
    const int m = (int)(r - t * 2 * g.np), c = m / g.np, n = m - c * g.np;
    if (n >= g.N) continue;
    const float* p = pbc + (int64_t)gi * g.wpg * per + r;
    float s = 0.f;
    for (int k = 0; k < g.wpg; ++k) s += p[k * per];
    (c ? dCm : dBm)[(t * g.G + gi) * g.N + n] = (E)s;
  }
}

// (4): dA_log, dskip and ddt_bias, summed over the tiles: 64 neighbouring values per
// workgroup, four lanes of tiles each.  Values: np rows of D for dA_log, then two rows.
__global__ __launch_bounds__(256) void gdn_scan_bwd_params_kernel(ScanGeo g, int tiles,
                                                                  const float* __restrict__ A_log,
                                                                  const float* __restrict__ states,
                                                                  const float* __restrict__ psum,
                                                                  float* __restrict__ dA_log,
                                                                  float* __restrict__ dskip,
                                                                  float* __restrict__ ddt_bias) {
  __shared__ float sm[256];
  const int64_t e = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63), per = (int64_t)g.np * g.D;
  const int q = threadIdx.x >> 6;
  const int64_t n = e / g.D, d = e - n * g.D;
  float s = 0.f;
  if (n < g.np) {
    for (int t = q; t < tiles; t += 4) s += states[t * per + e];
  } else if (n < g.np + 2) {
    const int64_t row = (int64_t)2 * g.D;
    for (int t = q; t < tiles * g.nw; t += 4) s += psum[t * row + (n - g.np) * g.D + d];
  }
  sm[threadIdx.x] = s;
  __syncthreads();
  if (q) return;
  s = (sm[threadIdx.x] + sm[64 + threadIdx.x]) + (sm[128 + threadIdx.x] + sm[192 + threadIdx.x]);
  if (n < g.N) dA_log[d * g.N + n] = -expf(A_log[d * g.N + n]) * s;
  else if (n == g.np && dskip) dskip[d] = s;
  else if (n == g.np + 1 && ddt_bias) ddt_bias[d] = s;
}

}  // namespace gdn
