// gdn_scan.h -- selective state space scan on gfx950, forward pass and decode step.
//
//     D = softplus(dt + dt_bias),  a = exp(-exp(A_log) D)
//     h[d,n] <- a[d,n] h[d,n] + D Bm[n] x,   y = (sum_n Cm[n] h[d,n] + skip x) silu(z)
//
// A wave owns 64 channels of one group, a lane one channel with NS of its states in
// registers; Bm and Cm of a token are the same for all its lanes and come through
// scalar loads into scalar registers.  With more than NS states the workgroup has
// ceil(N / NS) waves for the same channels, which add their parts of y through LDS; eight
// states per lane where there are no more.  B=2, T=2048, D=2048 bf16, us a call: N=8 50,
// N=16 72, N=32 129.  Other N run as the next of those (N=9 to 13 90, the copies of Bm and
// Cm included, N=17 to 20 159), and a group of fewer than 64 channels leaves lanes without
// one (N=16 in groups of 32 channels 118, of 16 206).
//
// Per token, channel and state the recurrence takes one v_exp_f32 and four other
// VALU operations (D A, D x B, the state's and y's multiply-adds), measured at 8.8 and 4.6
// cycles of a SIMD each, so at N = 16 it is bound by the VALU and not by the 8 bytes of x,
// dt, z and y.  B=2, T=2048, D=2048, N=16 bf16: the main kernel 34 us, its vector units
// busy for 86 % of them; the tiles' end states 31 us (78 %); the bytes alone would be 8
// from the caches, 13 from memory.
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
  int nw, np;            // waves per 64 channels; nw * NS
  int upw, cgb;          // units of nw waves per workgroup, workgroups for all channels
  int zero;              // forward: y's rows behind the last sequence are set to 0
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
  __device__ __forceinline__ void load(Global<const BE> p) {
    scalar_ptr q = (scalar_ptr)(uintptr_t)p;
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = q[i];
  }
  __device__ __forceinline__ float operator[](int j) const {
    if constexpr (sizeof(BE) == 4) return __uint_as_float(w[j]);
    else return (j & 1) ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
  }
};

// Brings the rows of Bm and Cm of 64 tokens from `t` on (those before `end`) into the L2,
// a lane per token, by loading a value of each.  The scalar loads that follow token by
// token wait for one row at a time, a longer wait from memory than from the L2, which the
// token before hides.  Measured in tiles of 64 tokens, us of kernels: B=3, T=777, D=1002,
// G=2, N=13 fp32 38 -> 30; T=32768 packed, D=2048, N=16 bf16, the first kernel 273 -> 259.
// The values are of no use: land() takes them, late enough that nothing waits for them.
struct RowAhead {
  uint32_t b = 0, c = 0;
  template <typename BE>
  __device__ __forceinline__ void send(Global<const BE> Bt, Global<const BE> Ct, int64_t ldb, int64_t ldc, int t, int end) {
    const int q = min(t + (int)(threadIdx.x & 63), end - 1);
    b = *(Global<const uint16_t>)(Bt + q * ldb);
    c = *(Global<const uint16_t>)(Ct + q * ldc);
  }
  __device__ __forceinline__ void land() { asm volatile("" ::"v"(b), "v"(c)); }
};

// One channel of one row as loaded: `row` is wave-uniform, `off` the lane's offset in
// bytes, so that the address takes no vector arithmetic.
template <typename E> __device__ __forceinline__ uint32_t load1(Global<const E> row, uint32_t off) {
  Global<const char> p = (Global<const char>)row + off;
  if constexpr (sizeof(E) == 2) return *(Global<const uint16_t>)p;
  else return *(Global<const uint32_t>)p;
}
template <typename E> __device__ __forceinline__ void store1(Global<E> row, uint32_t off, float v) {
  *(Global<E>)((Global<char>)row + off) = (E)v;
}
// Waits for the scalar loads in flight, and lets nothing later move before the wait.
// Scalar loads return out of order, so the compiler's own wait for one row would, placed
// at its first use, also wait for the next row's loads issued meanwhile.
__device__ __forceinline__ void scalar_loads_done() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_sched_barrier(0);
}
template <typename E> __device__ __forceinline__ float value1(uint32_t w) {
  return __uint_as_float(sizeof(E) == 2 ? w << 16 : w);
}

// NS consecutive values of a row of N from n0 on, 0 beyond the row.  WHOLE: the row is a
// multiple of NS, and is read four values at a time (dword alignment is enough for that).
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
template <int NS, bool WHOLE>
__device__ __forceinline__ void row_load(const float* p, int N, int n0, float (&v)[NS]) {
  if constexpr (WHOLE) {
#pragma unroll
    for (int j = 0; j < NS; j += 4) {
      const f32x4 q = *reinterpret_cast<const f32x4_u*>(p + n0 + j);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j + i] = q[i];
    }
  } else {
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const float q = p[min(n0 + j, N - 1)];
      v[j] = n0 + j < N ? q : 0.f;
    }
  }
}

// -exp(A_log) log2(e), the rate in base 2 that the kernels hold.  0 beyond N: such a
// state keeps the 0 it starts with.
__device__ __forceinline__ float scan_rate(float a_log) { return -fast_exp2(a_log * kLog2e) * kLog2e; }
template <int NS, bool WHOLE>
__device__ __forceinline__ void scan_rates(const float* A_log, const ScanGeo& g, int d, int n0, float (&A2)[NS]) {
  row_load<NS, WHOLE>(A_log + (int64_t)d * g.N, g.N, n0, A2);
#pragma unroll
  for (int j = 0; j < NS; ++j) A2[j] = WHOLE || n0 + j < g.N ? scan_rate(A2[j]) : 0.f;
}

template <int NS, bool WHOLE>
__device__ __forceinline__ void state_load(const float* st, const ScanGeo& g, int n, int d, int n0, float (&h)[NS]) {
  if (st) {
    row_load<NS, WHOLE>(st + ((int64_t)n * g.D + d) * g.N, g.N, n0, h);
  } else {
#pragma unroll
    for (int j = 0; j < NS; ++j) h[j] = 0.f;
  }
}
template <int NS, bool WHOLE>
__device__ __forceinline__ void state_store(float* st, const ScanGeo& g, int n, int d, int n0, const float (&h)[NS]) {
  float* p = st + ((int64_t)n * g.D + d) * g.N;
  if constexpr (WHOLE) {
#pragma unroll
    for (int j = 0; j < NS; j += 4)
      *reinterpret_cast<f32x4_u*>(p + n0 + j) = f32x4{h[j], h[j + 1], h[j + 2], h[j + 3]};
  } else {
#pragma unroll
    for (int j = 0; j < NS; ++j)
      if (n0 + j < g.N) p[n0 + j] = h[j];
  }
}

// Block id -> (tile of the whole batch, upw groups of 64 channels); the lane's channel d,
// `on` where it has one of its own; cg the wave's group, `unit` its place in the
// workgroup.  Workgroups have four waves where they can: with one or two, the waves of a
// launch were spread unevenly over the SIMDs (2048 of one wave each: 66 us of kernel for
// waves that lived 41 us).
struct ScanPlace {
  int tile, cg, gi, d, lane, unit, wave, n0;
  bool on, valid;
  template <int NS> __device__ __forceinline__ void init(const ScanGeo& g, uint32_t block) {
    tile = block / g.cgb;
    lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    unit = w / g.nw;
    wave = w - unit * g.nw;
    cg = (block - tile * g.cgb) * g.upw + unit;
    valid = cg < g.cgroups;
    cg = min(cg, g.cgroups - 1);
    gi = cg / g.wpg;
    const int dl = (cg - gi * g.wpg) * 64 + lane;
    on = valid && dl < g.DG;
    d = gi * g.DG + min(dl, g.DG - 1);
    n0 = wave * NS;
  }
};

// The lane's states in [tile][np][D].
template <int NS>
__device__ __forceinline__ void tile_state_load(const float* st, const ScanGeo& g, const ScanPlace& w, float (&h)[NS]) {
  Global<const float> row = (Global<const float>)st + ((int64_t)w.tile * g.np + w.n0) * g.D;
  const uint32_t off = lane_offset(w.d * 4u);
#pragma unroll
  for (int j = 0; j < NS; ++j, row = stepped<const float>(row, g.D)) h[j] = __uint_as_float(load1<float>(row, off));
}
template <int NS>
__device__ __forceinline__ void tile_state_store(float* st, const ScanGeo& g, const ScanPlace& w, const float (&h)[NS]) {
  Global<float> row = (Global<float>)st + ((int64_t)w.tile * g.np + w.n0) * g.D;
  const uint32_t off = lane_offset(w.d * 4u);
#pragma unroll
  for (int j = 0; j < NS; ++j, row = stepped<float>(row, g.D)) store1<float>(row, off, h[j]);
}

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
template <typename E, typename BE, int NS, bool WHOLE, bool SPLIT, bool ENDS>
__global__ __launch_bounds__(64 * kScanMaxWaves) void gdn_scan_kernel(
    ScanGeo g, Src x, const E* __restrict__ dt, Src z, const float* __restrict__ A_log,
    const BE* __restrict__ Bm, const BE* __restrict__ Cm, const float* __restrict__ skip,
    const float* __restrict__ dt_bias, const float* __restrict__ h0, float* __restrict__ states,
    float* __restrict__ sums, E* __restrict__ y, float* __restrict__ fin) {
  constexpr int U = kScanGroup;
  // [buffer][unit * nw + wave]
  __shared__ float part[SPLIT && !ENDS ? 2 : 1][SPLIT && !ENDS ? kScanMaxWaves : 1][U][SPLIT && !ENDS ? 64 : 1];

  const int tiles = g.ntiles * (g.cu ? 1 : g.B);
  const uint32_t main_blocks = (uint32_t)tiles * g.cgb;
  if constexpr (ENDS) {
    if ((int)(blockIdx.x / g.cgb) % g.ntiles == g.ntiles - 1) return;  // nobody starts from it
  } else if (blockIdx.x >= main_blocks) {
    scan_empty_state(g, blockIdx.x - main_blocks, h0, fin);
    return;
  }
  ScanPlace w;
  w.init<NS>(g, blockIdx.x);
  if (!SPLIT && !w.valid) return;
  float A2[NS], h[NS];
  scan_rates<NS, WHOLE>(A_log, g, w.d, w.n0, A2);
  if (SPLIT && !w.valid) {  // no channels: only the workgroup's barriers
    if constexpr (!ENDS) {
      Run<true> run;
      for (run.init(g.cu, g.T, g.S, w.tile, g.ntiles, g.len); !run.done(); run.next()) {
        const int n = run.tb - run.ta;
        for (int i = 0; i < n % U + n / U; ++i) __syncthreads();
      }
    }
    return;
  }
  const float bias = dt_bias ? dt_bias[w.d] : 0.f, sk = skip ? skip[w.d] : 0.f;
  const uint32_t off = lane_offset(w.d * (uint32_t)sizeof(E));
  const bool gate = !ENDS && z.p != nullptr;
  float sum = 0.f;
  int buf = 0;

  Run<true> run;
  run.init(g.cu, g.T, g.S, w.tile, g.ntiles, g.len);
#pragma unroll
  for (int j = 0; j < NS; ++j) h[j] = 0.f;
  for (; !run.done(); run.next()) {
    if (run.ta > run.start) {
      if constexpr (!ENDS) tile_state_load<NS>(states, g, w, h);
    } else {
      state_load<NS, WHOLE>(h0, g, run.n, w.d, w.n0, h);
      sum = -1.f;
    }
    Global<const E> xr = (Global<const E>)x.p + run.ta * x.ld, dr = (Global<const E>)dt + run.ta * g.lddt;
    Global<const E> zr = (Global<const E>)z.p + run.ta * z.ld;
    Global<E> yr = (Global<E>)y + (int64_t)run.ta * g.D;
    Global<const BE> br = (Global<const BE>)Bm + run.ta * g.ldb + (int64_t)w.gi * g.bgs + w.n0;
    Global<const BE> cr = (Global<const BE>)Cm + run.ta * g.ldc + (int64_t)w.gi * g.cgs + w.n0;
    const Global<const BE> b0 = (Global<const BE>)Bm + (int64_t)w.gi * g.bgs + w.n0;
    const Global<const BE> c0 = (Global<const BE>)Cm + (int64_t)w.gi * g.cgs + w.n0;
    RowAhead ahead;
    ahead.send<BE>(b0, ENDS ? b0 : c0, g.ldb, ENDS ? g.ldb : g.ldc, run.ta, run.tb);
    ScalarRow<BE, NS> b, c;
    b.load(br);
    if constexpr (!ENDS) c.load(cr);
    // One token with its row of Bm and Cm in flight; `more`: the run goes on, so the next
    // token's rows are sent for.  Returns sum_n Cm h.
    auto step = [&](float xv, float dl, bool more) {
      scalar_loads_done();
      const ScalarRow<BE, NS> bt = b, ct = c;
      if (more) {
        br = stepped<const BE>(br, g.ldb);
        cr = stepped<const BE>(cr, g.ldc);
      }
      b.load(br);
      if constexpr (!ENDS) c.load(cr);
      const float u = dl * xv;
      float a[NS];
#pragma unroll
      for (int j = 0; j < NS; ++j) a[j] = fast_exp2(dl * A2[j]);
      __builtin_amdgcn_sched_barrier(0);
      float acc0 = 0.f, acc1 = 0.f;
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        h[j] = fmaf(a[j], h[j], bt[j] * u);
        if constexpr (!ENDS) {
          if (j & 1) acc1 = fmaf(ct[j], h[j], acc1);
          else acc0 = fmaf(ct[j], h[j], acc0);
        }
      }
      return acc0 + acc1;
    };
    // Lanes without a channel of their own hold the last channel's once more and store the
    // same value to the same place: a store under a condition would make every later wait
    // for a load wait for the stores as well.
    auto finish = [&](float acc, float xv, float gv, Global<E> row) {
      store1<E>(row, off, fmaf(sk, xv, acc) * gv);
    };
    // SPLIT: the waves' parts of a group's outputs are added through LDS, each wave
    // finishing every nw-th token.  The other buffer is written next, and the barrier
    // after that keeps this one until all have read it.
    auto add_waves = [&](const float (&xv)[U], const float (&gv)[U], int n) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (k >= n || k % g.nw != w.wave) continue;
        float acc = 0.f;
        for (int q = 0; q < g.nw; ++q) acc += part[buf][w.unit * g.nw + q][k][w.lane];
        finish(acc, xv[k], gv[k], yr + (int64_t)k * g.D);
      }
      buf ^= 1;
    };
    // first what is over whole groups, token by token, then the groups, the next one's
    // rows on their way while one is computed
    const int over = (run.tb - run.ta) % U;
    for (int k = 0; k < over; ++k) {
      const float xv = value1<E>(load1<E>(xr, off)), dl = softplus_flat(value1<E>(load1<E>(dr, off)) + bias);
      float gv = 1.f;
      if (gate) {
        const float zv = value1<E>(load1<E>(zr, off));
        gv = zv * fast_sigmoid(zv);
      }
      const float acc = step(xv, dl, run.ta + k + 1 < run.tb);
      if constexpr (ENDS) {
        if (sum >= 0.f) sum += dl;
      } else if constexpr (SPLIT) {
        float xs[U] = {xv}, gs[U] = {gv};
        part[buf][w.unit * g.nw + w.wave][0][w.lane] = acc;
        add_waves(xs, gs, 1);
      } else {
        finish(acc, xv, gv, yr);
      }
      xr += x.ld;
      dr += g.lddt;
      zr += z.ld;
      yr += g.D;
    }
    uint32_t rx[U], rd[U], rz[U] = {};
    auto fetch = [&]() {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        rx[k] = load1<E>(xr, off);
        rd[k] = load1<E>(dr, off);
        xr = stepped<const E>(xr, x.ld);
        dr = stepped<const E>(dr, g.lddt);
      }
      if (gate) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
          rz[k] = load1<E>(zr, off);
          zr = stepped<const E>(zr, z.ld);
        }
      }
    };
    if (run.ta + over < run.tb) fetch();
    for (int t = run.ta + over; t < run.tb; t += U) {
      float xv[U], dl[U], gv[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        xv[k] = value1<E>(rx[k]);
        dl[k] = softplus_flat(value1<E>(rd[k]) + bias);
        gv[k] = 1.f;
      }
      if (gate) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const float zv = value1<E>(rz[k]);
          gv[k] = zv * fast_sigmoid(zv);
        }
      }
      const bool more = t + U < run.tb;
      if (more) fetch();
      if (((t - run.ta - over) & 63) == 0 && t + 64 < run.tb) {
        ahead.land();
        ahead.send<BE>(b0, ENDS ? b0 : c0, g.ldb, ENDS ? g.ldb : g.ldc, t + 64, run.tb);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float acc = step(xv[k], dl[k], k + 1 < U || more);
        if constexpr (ENDS) {
          if (sum >= 0.f) sum += dl[k];
        } else if constexpr (SPLIT) {
          part[buf][w.unit * g.nw + w.wave][k][w.lane] = acc;
        } else {
          finish(acc, xv[k], gv[k], yr);
          yr = stepped<E>(yr, g.D);
        }
      }
      if constexpr (SPLIT && !ENDS) {
        add_waves(xv, gv, U);
        yr += (int64_t)U * g.D;
      }
    }
    ahead.land();
    if constexpr (!ENDS)
      if (fin && w.on && run.tb == run.end) state_store<NS, WHOLE>(fin, g, run.n, w.d, w.n0, h);
  }
  if constexpr (!ENDS) {
    if (g.zero && w.wave == 0)
      for (int t = run.rest; t < run.t1; ++t) store1<E>((Global<E>)y + (int64_t)t * g.D, off, 0.f);
  } else {
    if (!w.on) return;
    tile_state_store<NS>(states, g, w, h);
    if (w.wave == 0) sums[(int64_t)w.tile * g.D + w.d] = sum;
  }
}

// (2): end states [row of the batch][tile][np][D] to start states, in place; one lane per
// (row, state, channel).  Back: from the last tile to the first, from what each tile adds
// to the state gradient before it to the gradient of its end state (the backward pass's;
// blocks with z = 1).  A chain of a few operations per tile: what it takes is the latency
// of its loads, so U tiles are sent for ahead of the U being joined, and before anything
// else.  B=2, T=2048, D=2048, N=16, 64 tiles: 9.2 us for one chain, 13.3 for both (67 MB,
// 5.0 TB/s; 19 in two launches).
struct JoinArgs {
  float* states;
  const float* sums;
};
static __global__ __launch_bounds__(256) void gdn_scan_join_kernel(ScanGeo g, const float* __restrict__ A_log,
                                                                   JoinArgs fore, JoinArgs aft) {
  constexpr int U = 16;
  const uint32_t per = (uint32_t)g.np * g.D;  // checked on the host: below 2^31
  const uint32_t r = blockIdx.x * 256u + threadIdx.x;
  if (r >= per) return;
  const bool back = blockIdx.z;
  const JoinArgs& j = back ? aft : fore;
  const int row = blockIdx.y, last = g.ntiles - 1;
  const uint32_t n = r / g.D, d = r - n * g.D;
  // the chain's first tile, and the steps to the next
  const int64_t first = (int64_t)row * g.ntiles + (back ? last : 0);
  float* p = j.states + first * per;
  const float* s = j.sums + first * g.D;
  const int64_t pstep = back ? -(int64_t)per : per, sstep = back ? -(int64_t)g.D : g.D;
  float e[U], sm[U];
  auto fetch = [&](int t) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t q = min(t + k, last);
      e[k] = (p + q * pstep)[r];
      sm[k] = (s + q * sstep)[d];
    }
  };
  fetch(0);
  const int64_t sd = (int64_t)d * g.N + min(n, (uint32_t)g.N - 1);
  const bool in = n < (uint32_t)g.N;
  // a row's first tile starts its sequence, from a state that the tile reads itself; behind
  // its last tile there is nothing
  float H = 0.f;
  const float A2 = in ? scan_rate(A_log[sd]) : 0.f;
  for (int t = 0; t <= last; t += U) {
    float out[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {  // beyond the last tile: not stored
      out[k] = H;
      H = sm[k] < 0.f ? e[k] : fmaf(fast_exp2(A2 * sm[k]), H, e[k]);
    }
    if (t + U <= last) fetch(t + U);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (t + k > last) break;
      (p + (t + k) * pstep)[r] = out[k];
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
// write bound it (8 N bytes per channel).  VEC: N is a multiple of four, and a lane's four
// values of the states, of A_log, Bm and Cm are one aligned load each.  Bound by how many
// loads a lane needs for its 32 bytes of state: one token each of B=256, D=4096, N=16 bf16
// (143 MB) 32 us = 4.4 TB/s, 49 us without VEC; B=64, D=2048 6.6 against 8.3 (N=13: 8.6).
// The fp32 state is nearly all of it in either type: calls with two sets of inputs in turn
// take 36 us in bf16 and 37 in fp32 at the first size.
template <typename E, bool VEC>
__global__ __launch_bounds__(256) void gdn_scan_decode_kernel(
    ScanGeo g, Src x, const E* __restrict__ dt, Src z, const float* __restrict__ A_log,
    const E* __restrict__ Bm, const E* __restrict__ Cm, const float* __restrict__ skip,
    const float* __restrict__ dt_bias, const float* state_in, float* state_out, E* __restrict__ y,
    int nl) {
  const int64_t item = ((int64_t)blockIdx.x * 256 + threadIdx.x) / nl;
  const int part = threadIdx.x & (nl - 1);
  const bool on = item < (int64_t)g.B * g.D;  // lanes without a channel stay for the sums
  const int64_t it = on ? item : 0;
  const int64_t b = it / g.D;
  const int d = (int)(it - b * g.D), gi = d / g.DG;
  // the lane's states, of which it has `cnt` (VEC: four or none; with none it reads the
  // row's first ones, and its rates and rows count as 0)
  const int cnt = max(min(g.N - 4 * part, 4), 0), n0 = cnt ? 4 * part : 0;
  auto four = [&](const auto* p, float (&v)[4]) {
    using P = std::remove_cv_t<std::remove_pointer_t<decltype(p)>>;
    if constexpr (VEC) {
      vec_load<P, 4>(p, v);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = (float)p[max(min(j, cnt - 1), 0)];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < cnt ? v[j] : 0.f;
  };
  float A2[4], h[4];
  four(state_in + it * g.N + n0, h);
  four(A_log + (int64_t)d * g.N + n0, A2);
  const float bias = dt_bias ? dt_bias[d] : 0.f, sk = skip ? skip[d] : 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) A2[j] = scan_rate(A2[j]);
  for (int t = 0; t < g.T; ++t) {
    const int64_t tok = b * g.T + t;
    const float xv = (float)static_cast<const E*>(x.p)[tok * x.ld + d];
    const float dv = (float)dt[tok * g.lddt + d];
    float zv = 0.f, bv[4], cv[4];
    if (z.p) zv = (float)static_cast<const E*>(z.p)[tok * z.ld + d];
    four(Bm + tok * g.ldb + (int64_t)gi * g.N + n0, bv);
    four(Cm + tok * g.ldc + (int64_t)gi * g.N + n0, cv);
    const float dl = gate_softplus(dv + bias), u = dl * xv;
    float acc = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[j] = fmaf(fast_exp2(dl * A2[j]), h[j], j < cnt ? bv[j] * u : 0.f);
      if (j < cnt) acc = fmaf(cv[j], h[j], acc);
    }
    for (int o = nl >> 1; o; o >>= 1) acc += __shfl_xor(acc, o, 64);
    if (on && part == 0) {
      float v = fmaf(sk, xv, acc);
      if (z.p) v *= zv * fast_sigmoid(zv);
      y[tok * g.D + d] = (E)v;
    }
  }
  if (!on) return;
  float* op = state_out + it * g.N + n0;
  if constexpr (VEC) {
    if (cnt) vec_store<float, 4>(op, h);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < cnt) op[j] = h[j];
  }
}

}  // namespace gdn
