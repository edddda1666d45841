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
// SUB tokens kept in LDS; then, from the last group to the first, forwards again within
// the group, its states in registers, and backwards through them; (4) sums over waves and
// tiles.  VALU-bound like the forward pass: B=2, T=2048, D=2048, N=16 bf16, us: (1) 43,
// (2) 13, (3) 167 with its vector units busy for 78 % of them, (4) 9; the bytes alone
// would be 15 from the caches, 23 from memory.  Calls there, us: bf16 231 (fp32 248), N=8
// 129, N=32 439, N=64 916; other N run as the next of those (N=13 249, N=17 463, N=33 963).
//
// Eight states per lane and eight tokens per group: (3) then takes 241 registers, two
// waves per SIMD, which 45 KB of LDS per workgroup allow as well (from checkpoints 256 and
// up to 36 bytes of scratch per lane).  Held to three waves per SIMD the registers spill;
// groups of four tokens took a tenth more.
//
// dBm and dCm need sums over channels, that is over lanes: 2 NS values of a token are
// added over 64 lanes by halving (in each step a lane keeps half of its values and
// hands the others to its partner), 2.2 operations per value instead of 6.
#pragma once
#include "gdn_scan.h"

namespace gdn {

constexpr int kScanBwdStates = 8;  // states per lane
constexpr int kScanBwdSub = 8;     // tokens per group
// Tokens per tile.  B=2, T=2048, D=2048, N=16 bf16, us a call: 231 with 32, 238 with 64, 249
// with 16 (more tiles to join); B=2, T=1024, D=1024: 81 with 32 and 16, 115 with 64.
constexpr int kScanBwdTile = 32;
constexpr int scan_bwd_units(int waves) { return waves >= 4 ? 1 : 4 / waves; }  // per workgroup

// Sums over the wave's 64 lanes of 16 values each: returns the sum of value lane / 4.
__device__ __forceinline__ float wave_sums(float (&v)[16]) {
  constexpr int V = 16;
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
  v[0] += dpp(v[0], Xor2{});
  return v[0] + dpp(v[0], Xor1{});
}

struct ScanBwdGeo {
  ScanGeo g;
  int nblk;  // checkpoint scales per row
};

// softplus_flat(x) and its derivative, sigmoid(x) (1 where softplus is taken as x).
__device__ __forceinline__ float softplus_both(float x, float& slope) {
  const float y = __builtin_amdgcn_exp2f(x * kLog2e);
  const float u = 1.f + y;
  const float r = (__builtin_amdgcn_logf(u) * __builtin_amdgcn_rcpf(u - 1.f)) * (y * 0.693147180559945309f);
  slope = x > 20.f ? 1.f : y * __builtin_amdgcn_rcpf(u);
  return x > 20.f ? x : u == 1.f ? y : r;
}

// (1).  states, rev [tile][np][D]; sums, rsums [tile][D] (-1: nothing passes through).
// R needs no walk backwards: with P_t = a_1 .. a_t it is sum_t P_t Cm_t r_t.  VALU-bound;
// B=2, T=2048, D=2048, N=16 bf16: 43 us with four tokens' loads in flight (122 registers, so
// the launch's four waves per SIMD run side by side); a tenth more with eight (154 registers).
template <typename E, typename BE, int NS, bool WHOLE, bool CK>
__global__ __launch_bounds__(64 * kScanMaxWaves) void gdn_scan_bwd_ends_kernel(
    ScanBwdGeo bg, Src x, const E* __restrict__ dt, Src z, const float* __restrict__ A_log,
    const BE* __restrict__ Bm, const BE* __restrict__ Cm, const float* __restrict__ dt_bias,
    const float* __restrict__ h0, const E* __restrict__ d_y, const float* __restrict__ d_fin,
    float* __restrict__ states, float* __restrict__ rev, float* __restrict__ sums,
    float* __restrict__ rsums) {
  constexpr int U = kScanGroup / 2;
  const ScanGeo& g = bg.g;
  ScanPlace w;
  w.init<NS>(g, blockIdx.x);
  if (!w.valid) return;
  float A2[NS], h[NS], P[NS], R[NS];
  scan_rates<NS, WHOLE>(A_log, g, w.d, w.n0, A2);
  // lane offsets: of E, of a checkpoint's codes and scales
  const uint32_t off = lane_offset(w.d * (uint32_t)sizeof(E)), xoff = CK ? lane_offset(w.d) : off;
  const uint32_t soff = CK ? lane_offset((uint32_t)w.d >> 5) : 0;
  const float bias = dt_bias ? dt_bias[w.d] : 0.f;
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
      state_load<NS, WHOLE>(h0, g, run.n, w.d, w.n0, h);
      sum = -1.f;
    }
    float pass = 0.f;
    Global<const BE> br = (Global<const BE>)Bm + run.ta * g.ldb + (int64_t)w.gi * g.bgs + w.n0;
    Global<const BE> cr = (Global<const BE>)Cm + run.ta * g.ldc + (int64_t)w.gi * g.cgs + w.n0;
    TokenVals<E, 1, U, CK> rx, rz = {};
    TokenVals<E, 1, U, false> rd, ry = {};
    auto fetch = [&](int t) {
      rx.fetch(x, t, run.tb, xoff, soff, bg.nblk);
      rd.fetch(Src{dt, nullptr, g.lddt}, t, run.tb, off, 0, 0);
      if (cont) {
        ry.fetch(Src{d_y, nullptr, g.D}, t, run.tb, off, 0, 0);
        if (z.p) rz.fetch(z, t, run.tb, xoff, soff, bg.nblk);
      }
    };
    RowAhead ahead;
    static_assert(kScanBwdTile <= 64, "one round of rows sent for ahead");
    ahead.send<BE>((Global<const BE>)Bm + (int64_t)w.gi * g.bgs + w.n0, (Global<const BE>)Cm + (int64_t)w.gi * g.cgs + w.n0,
                   g.ldb, g.ldc, run.ta, run.tb);
    ScalarRow<BE, NS> b, c;
    b.load(br);
    c.load(cr);
    fetch(run.ta);
    for (int t = run.ta; t < run.tb; t += U) {
      float u[U], dl[U], r[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        dl[k] = softplus_flat(rd[k] + bias);
        u[k] = dl[k] * rx[k];
        r[k] = ry[k];
      }
      if (z.p) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const float zv = rz[k];
          r[k] *= zv * fast_sigmoid(zv);
        }
      }
      if (t + U < run.tb) fetch(t + U);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (t + k >= run.tb) break;
        scalar_loads_done();
        const ScalarRow<BE, NS> bt = b, ct = c;
        if (t + k + 1 < run.tb) {
          br = stepped<const BE>(br, g.ldb);
          cr = stepped<const BE>(cr, g.ldc);
        }
        b.load(br);
        c.load(cr);
        float a[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) a[j] = fast_exp2(dl[k] * A2[j]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NS; ++j) h[j] = fmaf(a[j], h[j], bt[j] * u[k]);
        if (cont) {
          pass += dl[k];
#pragma unroll
          for (int j = 0; j < NS; ++j) {
            P[j] *= a[j];
            R[j] = fmaf(P[j], ct[j] * r[k], R[j]);
          }
        }
      }
    }
    ahead.land();
    if (sum >= 0.f) sum += pass;
    if (cont) {
      if (run.tb == run.end) {
        float f[NS];
        state_load<NS, WHOLE>(d_fin, g, run.n, w.d, w.n0, f);
#pragma unroll
        for (int j = 0; j < NS; ++j) R[j] = fmaf(P[j], f[j], R[j]);
      } else {
        rsum = pass;
      }
    }
  }
  if (!w.on) return;
  tile_state_store<NS>(states, g, w, h);
  tile_state_store<NS>(rev, g, w, R);
  if (w.wave == 0) {
    sums[(int64_t)w.tile * g.D + w.d] = sum;
    rsums[(int64_t)w.tile * g.D + w.d] = rsum;
  }
}

// (3).  states holds the tiles' start states and is overwritten with the tile's part of
// sum_t D q; rev the end states' gradients.  pbc [channel wave][token][2][np]: the
// wave's parts of dBm and dCm.  psum [tile][NW][2][D]: of dskip and ddt_bias.  Blocks
// behind the last tile's copy d_final to d_initial for empty sequences.
//
// The waves of a workgroup (NS states each) add their sums over the states, three per
// token, through LDS: token k of a group is finished by wave k % NW.
template <typename E, typename BE, int NS, bool WHOLE, int NW, int SUB, bool CK>
__global__ __launch_bounds__(64 * NW * scan_bwd_units(NW), 2) void gdn_scan_bwd_kernel(
    ScanBwdGeo bg, Src x, const E* __restrict__ dt, Src z, const float* __restrict__ A_log,
    const BE* __restrict__ Bm, const BE* __restrict__ Cm, const float* __restrict__ skip,
    const float* __restrict__ dt_bias, const float* __restrict__ h0, const E* __restrict__ d_y,
    const float* __restrict__ d_fin, float* __restrict__ states, const float* __restrict__ rev,
    E* __restrict__ dx, E* __restrict__ ddt, E* __restrict__ dz, float* __restrict__ pbc,
    float* __restrict__ psum, float* __restrict__ dh0) {
  constexpr int UPW = scan_bwd_units(NW);
  __shared__ float hs[kScanBwdTile / SUB][UPW * NW][NS][64];
  __shared__ float part_[NW > 1 ? UPW : 1][NW > 1 ? SUB : 1][NW > 1 ? NW - 1 : 1][3][NW > 1 ? 64 : 1];
  const ScanGeo& g = bg.g;
  const int64_t ntok = (int64_t)g.B * g.T;
  const uint32_t main_blocks = (uint32_t)(g.ntiles * (g.cu ? 1 : g.B)) * g.cgb;
  if (blockIdx.x >= main_blocks) {
    scan_empty_state(g, blockIdx.x - main_blocks, d_fin, dh0);
    return;
  }
  ScanPlace w;
  w.init<NS>(g, blockIdx.x);
  if (!w.valid) {  // no channels: only the workgroup's barriers
    if constexpr (NW > 1) {
      Run<true> run;
      for (run.init(g.cu, g.T, g.S, w.tile, g.ntiles, g.len); !run.done(); run.next())
        for (int s = 0; s < 2 * ((run.tb - run.ta + SUB - 1) / SUB); ++s) __syncthreads();
    }
    return;
  }
  auto& part = part_[NW > 1 ? w.unit : 0];
  const int kept = w.unit * NW + w.wave;
  // lane offsets: of E, of a checkpoint's codes and scales
  const uint32_t off = lane_offset(w.d * (uint32_t)sizeof(E)), xoff = CK ? lane_offset(w.d) : off;
  const uint32_t soff = CK ? lane_offset((uint32_t)w.d >> 5) : 0;
  const bool gate = z.p != nullptr;
  float A2[NS], dA[NS], h[NS], l[NS];
  scan_rates<NS, WHOLE>(A_log, g, w.d, w.n0, A2);
  const float bias = dt_bias ? dt_bias[w.d] : 0.f, sk = skip ? skip[w.d] : 0.f;
  const Global<const BE> bp = (Global<const BE>)Bm + (int64_t)w.gi * g.bgs + w.n0;
  const Global<const BE> cp = (Global<const BE>)Cm + (int64_t)w.gi * g.cgs + w.n0;
  float dskip = 0.f, dbias = 0.f;
  // this wave's place in a token's row of pbc: lane v of dBm and dCm's 2 NS values
  constexpr int kRep = 64 / (2 * NS);
  const int v = w.lane / kRep;
  const Global<float> pb = (Global<float>)pbc + (int64_t)w.cg * ntok * 2 * g.np;
  const uint32_t pboff = lane_offset(((v / NS) * g.np + w.n0 + v % NS) * 4u);
#pragma unroll
  for (int j = 0; j < NS; ++j) dA[j] = 0.f;

  if (g.cu) {  // rows behind the last sequence
    const int last = max(uniform<true>(seq_offset(g.cu, g.S, g.T)), w.tile * g.len);
    for (int t = last; t < min((w.tile + 1) * g.len, g.T); ++t) {
      if (w.wave == 0) {
        store1<E>((Global<E>)dx + (int64_t)t * g.D, off, 0.f);
        store1<E>((Global<E>)ddt + (int64_t)t * g.D, off, 0.f);
        if (gate) store1<E>((Global<E>)dz + (int64_t)t * g.D, off, 0.f);
      }
      store1<float>(pb + (int64_t)t * 2 * g.np, pboff, 0.f);
    }
  }

  Run<true> run;
  run.init(g.cu, g.T, g.S, w.tile, g.ntiles, g.len);
  for (; !run.done(); run.next()) {
    if (run.ta > run.start) tile_state_load<NS>(states, g, w, h);
    else state_load<NS, WHOLE>(h0, g, run.n, w.d, w.n0, h);
    if (run.tb == run.end) state_load<NS, WHOLE>(d_fin, g, run.n, w.d, w.n0, l);
    else tile_state_load<NS>(rev, g, w, l);
    // groups of SUB tokens, the last one maybe shorter (its rows held to the run's last)
    const int nsub = (run.tb - run.ta + SUB - 1) / SUB;
    TokenVals<E, 1, SUB, CK> rx, rz = {};
    TokenVals<E, 1, SUB, false> rd, ry;
    auto fetch = [&](int t, bool all) {
      rx.fetch(x, t, run.tb, xoff, soff, bg.nblk);
      rd.fetch(Src{dt, nullptr, g.lddt}, t, run.tb, off, 0, 0);
      if (all) {
        ry.fetch(Src{d_y, nullptr, g.D}, t, run.tb, off, 0, 0);
        if (gate) rz.fetch(z, t, run.tb, xoff, soff, bg.nblk);
      }
    };
    RowAhead ahead;
    ahead.send<BE>(bp, cp, g.ldb, g.ldc, run.ta, run.tb);
    // forwards: the state before every group
    ScalarRow<BE, NS> b, c;
    Global<const BE> br = bp + run.ta * g.ldb;
    b.load(br);
    fetch(run.ta, nsub == 1);
    for (int s = 0; s < nsub; ++s) {
#pragma unroll
      for (int j = 0; j < NS; ++j) hs[s][kept][j][w.lane] = h[j];
      if (s == nsub - 1) break;
      float u[SUB], dl[SUB];
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        dl[k] = softplus_flat(rd[k] + bias);
        u[k] = dl[k] * rx[k];
      }
      fetch(run.ta + (s + 1) * SUB, s + 1 == nsub - 1);
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        scalar_loads_done();
        const ScalarRow<BE, NS> bt = b;
        br = stepped<const BE>(br, g.ldb);  // there is a later group
        b.load(br);
        float a[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) a[j] = fast_exp2(dl[k] * A2[j]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NS; ++j) h[j] = fmaf(a[j], h[j], bt[j] * u[k]);
      }
    }
    ahead.land();
    // backwards, group by group
    for (int s = nsub - 1; s >= 0; --s) {
      const int t = run.ta + s * SUB, cnt = min(SUB, run.tb - t);
      // per token: x, D, softplus', r = dy silu(z), dy silu'(z)
      float xv[SUB], dl[SUB], sig[SUB], r[SUB], rz2[SUB], hp[SUB + 1][NS];
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        xv[k] = rx[k];
        dl[k] = softplus_both(rd[k] + bias, sig[k]);
        r[k] = ry[k];
        rz2[k] = 0.f;
      }
      if (gate) {
#pragma unroll
        for (int k = 0; k < SUB; ++k) {
          const float zv = rz[k], sg = fast_sigmoid(zv);
          rz2[k] = r[k] * silu_slope(zv, sg);
          r[k] *= zv * sg;
        }
      }
      if (s > 0) fetch(t - SUB, true);
      br = bp + t * g.ldb;
      b.load(br);
#pragma unroll
      for (int j = 0; j < NS; ++j) hp[0][j] = hs[s][kept][j][w.lane];
      // hp[k]: the state before token k; the last is the next group's first, where there is one
      const bool last = s == nsub - 1;
      if (!last) {
#pragma unroll
        for (int j = 0; j < NS; ++j) hp[SUB][j] = hs[s + 1][kept][j][w.lane];
      }
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        if (k + 1 >= cnt + (last ? 1 : 0)) break;
        scalar_loads_done();
        const ScalarRow<BE, NS> bt = b;
        if (k + 1 < cnt) br = stepped<const BE>(br, g.ldb);
        b.load(br);
        const float u = dl[k] * xv[k];
        float a[NS];
#pragma unroll
        for (int j = 0; j < NS; ++j) a[j] = fast_exp2(dl[k] * A2[j]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NS; ++j) hp[k + 1][j] = fmaf(a[j], hp[k][j], bt[j] * u);
      }
      float own[(SUB + NW - 1) / NW][3];  // sums over the states of the tokens this wave finishes
      br = bp + (int64_t)(t + cnt - 1) * g.ldb;
      Global<const BE> cr = cp + (int64_t)(t + cnt - 1) * g.ldc;
      Global<float> pr = pb + (int64_t)(t + cnt - 1) * 2 * g.np;
      b.load(br);
      c.load(cr);
      if constexpr (NW > 1) __syncthreads();  // the last group's sums are all read
#pragma unroll
      for (int k = SUB - 1; k >= 0; --k) {
        if (k >= cnt) continue;
        scalar_loads_done();
        const ScalarRow<BE, NS> bt = b, ct = c;
        if (k > 0) {
          br = stepped<const BE>(br, -g.ldb);
          cr = stepped<const BE>(cr, -g.ldc);
        }
        b.load(br);
        c.load(cr);
        // lanes without a channel of their own hold the last channel's once more; to the
        // sums over channels they add nothing
        const float um = w.on ? dl[k] * xv[k] : 0.f, rm = w.on ? r[k] : 0.f;
        float a[NS], bc[2 * NS], sy = 0.f, sb = 0.f, sq = 0.f;
#pragma unroll
        for (int j = 0; j < NS; ++j) a[j] = fast_exp2(dl[k] * A2[j]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const float ht = hp[k + 1][j];
          const float lam = fmaf(ct[j], r[k], l[j]);
          sy = fmaf(ct[j], ht, sy);
          sb = fmaf(bt[j], lam, sb);
          l[j] = a[j] * lam;
          const float q = l[j] * hp[k][j];
          sq = fmaf(q, A2[j], sq);
          dA[j] = fmaf(q, dl[k], dA[j]);
          bc[j] = lam * um;
          bc[NS + j] = ht * rm;
        }
        store1<float>(pr, pboff, wave_sums(bc));  // kRep lanes the same value
        pr = stepped<float>(pr, -2 * g.np);
        if (NW == 1 || k % NW == w.wave) {
          own[k / NW][0] = sy;
          own[k / NW][1] = sb;
          own[k / NW][2] = sq;
        } else {
          const int slot = w.wave - (w.wave > k % NW ? 1 : 0);
          part[k][slot][0][w.lane] = sy;
          part[k][slot][1][w.lane] = sb;
          part[k][slot][2][w.lane] = sq;
        }
      }
      if constexpr (NW > 1) __syncthreads();
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        if (k >= cnt) break;
        if (NW > 1 && k % NW != w.wave) continue;
        float sy = own[k / NW][0], sb = own[k / NW][1], sq = own[k / NW][2];
        if constexpr (NW > 1) {
#pragma unroll
          for (int q = 0; q < NW - 1; ++q) {
            sy += part[k][q][0][w.lane];
            sb += part[k][q][1][w.lane];
            sq += part[k][q][2][w.lane];
          }
        }
        const int64_t o = (int64_t)(t + k) * g.D;
        const float dr = fmaf(sb, xv[k], sq * 0.693147180559945309f) * sig[k];
        if (gate) store1<E>((Global<E>)dz + o, off, rz2[k] * fmaf(sk, xv[k], sy));
        store1<E>((Global<E>)dx + o, off, fmaf(dl[k], sb, sk * r[k]));
        store1<E>((Global<E>)ddt + o, off, dr);
        dskip = fmaf(r[k], xv[k], dskip);
        dbias += dr;
      }
    }
    if (dh0 && w.on && run.ta == run.start) state_store<NS, WHOLE>(dh0, g, run.n, w.d, w.n0, l);
  }
  if (!w.on) return;
  tile_state_store<NS>(states, g, w, dA);
  Global<float> ps = (Global<float>)psum + ((int64_t)w.tile * NW + w.wave) * 2 * g.D;
  store1<float>(ps, w.d * 4u, dskip);
  store1<float>(ps + g.D, w.d * 4u, dbias);
}

// (4).  Blocks below `row_blocks`: dBm and dCm, a value at a time per lane, summed over the
// group's channel waves.  The others: dA_log, dskip and ddt_bias, summed over the tiles, 64
// neighbouring values per workgroup, four lanes of tiles each; np rows of D values for
// dA_log, then two rows.
template <typename E>
__global__ __launch_bounds__(256) void gdn_scan_bwd_sums_kernel(
    ScanGeo g, int tiles, uint32_t row_blocks, const float* __restrict__ A_log,
    const float* __restrict__ pbc, const float* __restrict__ states, const float* __restrict__ psum,
    E* __restrict__ dBm, E* __restrict__ dCm, float* __restrict__ dA_log, float* __restrict__ dskip,
    float* __restrict__ ddt_bias) {
  __shared__ float sm[256];
  if (blockIdx.x < row_blocks) {
    const int64_t per = (int64_t)g.B * g.T * 2 * g.np, total = per * g.G;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)row_blocks * 256) {
      const int gi = (int)(i / per);
      const int64_t r = i - gi * per;
      const uint32_t w2 = 2 * g.np;
      const int64_t t = r / w2;
      const int m = (int)(r - t * w2), c = m >= g.np, n = m - c * g.np;
      if (n >= g.N) continue;
      const float* p = pbc + (int64_t)gi * g.wpg * per + r;
      float s = 0.f;
#pragma unroll 8
      for (int k = 0; k < g.wpg; ++k) s += p[k * per];
      (c ? dCm : dBm)[(t * g.G + gi) * g.N + n] = (E)s;
    }
    return;
  }
  const int64_t e = (int64_t)(blockIdx.x - row_blocks) * 64 + (threadIdx.x & 63), per = (int64_t)g.np * g.D;
  const int q = threadIdx.x >> 6;
  const int64_t n = e / g.D, d = e - n * g.D;
  float s = 0.f;
  if (n < g.np) {
#pragma unroll 8
    for (int t = q; t < tiles; t += 4) s += states[t * per + e];
  } else if (n < g.np + 2) {
    const int64_t row = (int64_t)2 * g.D;
#pragma unroll 8
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
