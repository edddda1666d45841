// gdn_scan_bwd_api.hip -- entry point of the selective scan's backward pass.  See
// include/gdn.h.
#include "gdn_scan_bwd.h"
#include "gdn_scan_host.h"

namespace {

struct BwdSpace {
  size_t states, rev, sums, rsums, psum, pbc, rows, total;
};

BwdSpace bwd_space(const ScanPlan& pl) {
  const gdn::ScanGeo& g = pl.geo;
  const size_t tiles = pl.tok > 0 ? (size_t)scan_all_tiles(pl) : 0;
  const size_t state = align_up(tiles * g.np * g.D * 4), row = align_up(tiles * g.D * 4);
  BwdSpace w{};
  size_t off = 0;
  w.states = off; off += state;
  w.rev = off;    off += state;
  w.sums = off;   off += row;
  w.rsums = off;  off += row;
  w.psum = off;   off = align_up(off + tiles * g.nw * 2 * g.D * 4);
  w.pbc = off;    off = align_up(off + (size_t)g.cgroups * pl.tok * 2 * g.np * 4);
  w.rows = off;   off += 2 * scan_rows_bytes(pl);
  w.total = off;
  return w;
}

gdn_status_t bwd_sizes(const gdn_scan_params_t* p, bool packed, ScanPlan* pl) {
  gdn_status_t st = scan_sizes(p, packed, pl);
  if (st != GDN_OK) return st;
  // 1, 2, 4 or 8 waves
  int nw = 1;
  while (nw * gdn::kScanBwdStates < p->N) nw *= 2;
  scan_waves(&pl->geo, gdn::kScanBwdStates, nw);
  scan_tiles(pl, gdn::kScanBwdTile);
  return GDN_OK;
}

struct BwdArgs {
  const void* x;
  const uint8_t* x_scales;
  const void* dt;
  const float* A_log;
  const void *Bm, *Cm;
  const float* skip;
  const void* z;
  const uint8_t* z_scales;
  const float *dt_bias, *h0;
  const void* dy;
  const float* dfin;
  void *dx, *ddt;
  float* dA_log;
  void *dBm, *dCm;
  float* dskip;
  void* dz;
  float *dbias, *dh0;
};

gdn_status_t scan_bwd_run(ScanPlan pl, const BwdArgs& a, void* ws, hipStream_t s) {
  gdn::ScanGeo& g = pl.geo;
  const BwdSpace sp = bwd_space(pl);
  char* w = static_cast<char*>(ws);
  auto F = [&](size_t off) { return reinterpret_cast<float*>(w + off); };
  const bool direct = scan_rows_direct(pl, a.Bm, a.Cm);
  const void *Bm = a.Bm, *Cm = a.Cm;
  hipError_t err = hipSuccess;
  auto ok = [&](hipError_t e) {
    if (e != hipSuccess && err == hipSuccess) err = e;
  };
  const int64_t tiles = pl.tok > 0 ? scan_all_tiles(pl) : 0;
  const int64_t main_blocks = tiles * g.cgb;
  const int64_t empties = (g.cu || g.T == 0) && a.dh0 ? g.S : 0;
  // rows of dBm and dCm: workgroups beyond that loop
  const int64_t row_blocks = std::min<int64_t>(pl.tok > 0 ? ceil_div(pl.tok * g.G * 2 * g.np, 256) : 0, 1 << 16);
  const int64_t param_blocks = ceil_div((int64_t)(g.np + 2) * g.D, 64);
  // (the first kernel has no more threads than the main one)
  if (!grid_fits(main_blocks + empties, 64 * g.nw * g.upw) || !grid_fits(row_blocks + param_blocks, 256))
    return GDN_ERR_UNSUPPORTED;
  if (!direct && pl.tok > 0) {
    float *Bw = F(sp.rows), *Cw = F(sp.rows + scan_rows_bytes(pl));
    ok(pl.esz == 2 ? scan_copy_rows<gdn::bf16>(&pl, Bm, Cm, Bw, Cw, s) : scan_copy_rows<float>(&pl, Bm, Cm, Bw, Cw, s));
    Bm = Bw;
    Cm = Cw;
  }
  if (pl.tok == 0) g.ntiles = 0;
  auto run = [&](auto e, auto be, auto whole, auto nw, auto ck) {
    using E = decltype(e);
    using BE = decltype(be);
    constexpr int NS = gdn::kScanBwdStates, NW = decltype(nw)::value;
    constexpr bool WHOLE = decltype(whole)::value, CK = decltype(ck)::value;
    const gdn::ScanBwdGeo bg{g, (int)ceil_div(g.D, gdn::kPackBlock)};
    const gdn::Src x{a.x, a.x_scales, a.x_scales ? g.D : pl.ldx}, z{a.z, a.z_scales, a.z_scales ? g.D : pl.ldz};
    const E *dt = static_cast<const E*>(a.dt), *dy = static_cast<const E*>(a.dy);
    const BE *b = static_cast<const BE*>(Bm), *c = static_cast<const BE*>(Cm);
    if (g.ntiles > 1) {
      // sixteen states per lane where there are as many: half the work per token that
      // does not depend on the states
      auto ends = [&](auto n) {
        constexpr int M = decltype(n)::value;
        gdn::ScanBwdGeo eg = bg;
        scan_waves(&eg.g, M, g.np / M);
        ok(launch(gdn::gdn_scan_bwd_ends_kernel<E, BE, M, WHOLE, CK>, dim3((unsigned)(tiles * eg.g.cgb)),
                  dim3(64 * eg.g.nw * eg.g.upw), s, eg, x, dt, z, a.A_log, b, c, a.dt_bias, a.h0, dy, a.dfin, F(sp.states), F(sp.rev), F(sp.sums),
                  F(sp.rsums)));
      };
      if constexpr (NW == 1) ends(std::integral_constant<int, 8>{});
      else ends(std::integral_constant<int, 16>{});
      ok(launch(gdn::gdn_scan_join_kernel, scan_join_grid(g, 2), dim3(256), s, g, a.A_log,
                gdn::JoinArgs{F(sp.states), F(sp.sums)}, gdn::JoinArgs{F(sp.rev), F(sp.rsums)}));
    }
    if (main_blocks + empties > 0)
      ok(launch(gdn::gdn_scan_bwd_kernel<E, BE, NS, WHOLE, NW, gdn::kScanBwdSub, CK>, dim3((unsigned)(main_blocks + empties)),
                dim3(64 * NW * g.upw), s, bg, x, dt, z, a.A_log, b, c, a.skip, a.dt_bias, a.h0, dy, a.dfin, F(sp.states),
                F(sp.rev), static_cast<E*>(a.dx), static_cast<E*>(a.ddt), static_cast<E*>(a.dz), F(sp.pbc), F(sp.psum),
                a.dh0));
    ok(launch(gdn::gdn_scan_bwd_sums_kernel<E>, dim3((unsigned)(row_blocks + param_blocks)), dim3(256), s, g, (int)tiles,
              (uint32_t)row_blocks, a.A_log, F(sp.pbc), F(sp.states), F(sp.psum), static_cast<E*>(a.dBm),
              static_cast<E*>(a.dCm), a.dA_log, a.dskip, a.dbias));
  };
  auto waves = [&](auto e, auto be, auto whole) {
    auto kind = [&](auto nw) {
      if (a.x_scales) run(e, be, whole, nw, std::true_type{});
      else run(e, be, whole, nw, std::false_type{});
    };
    if (g.nw == 1) kind(std::integral_constant<int, 1>{});
    else if (g.nw == 2) kind(std::integral_constant<int, 2>{});
    else if (g.nw == 4) kind(std::integral_constant<int, 4>{});
    else kind(std::integral_constant<int, 8>{});
  };
  using Yes = std::true_type;
  using No = std::false_type;
  if (pl.esz == 4) direct ? waves(0.f, 0.f, Yes{}) : waves(0.f, 0.f, No{});
  else direct ? waves(gdn::bf16{}, gdn::bf16{}, Yes{}) : waves(gdn::bf16{}, 0.f, No{});
  return err == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // namespace

extern "C" {

size_t gdn_scan_bwd_workspace_size(const gdn_scan_params_t* p, int packed) {
  ScanPlan pl;
  return bwd_sizes(p, packed != 0, &pl) == GDN_OK ? bwd_space(pl).total : 0;
}

gdn_status_t gdn_scan_bwd(const gdn_scan_params_t* p, const void* x, const uint8_t* x_scales, const void* dt,
                          const float* A_log, const void* Bm, const void* Cm, const float* skip, const void* z,
                          const uint8_t* z_scales, const float* dt_bias, const int64_t* cu_seqlens,
                          const float* initial_state, const void* d_y, const float* d_final_state, void* dx,
                          void* ddt, float* dA_log, void* dBm, void* dCm, float* dskip, void* dz,
                          float* ddt_bias, float* d_initial_state, void* workspace, size_t workspace_bytes,
                          void* stream) {
  ScanPlan pl;
  gdn_status_t st = bwd_sizes(p, cu_seqlens != nullptr, &pl);
  if (st != GDN_OK) return st;
  if (z && !x_scales != !z_scales) return GDN_ERR_SHAPE;
  if ((x_scales && pl.ldx != p->D) || (z_scales && pl.ldz != p->D)) return GDN_ERR_SHAPE;  // codes are dense
  if (pl.tok > 0 && (!x || !dt || !Bm || !Cm || !d_y || !dx || !ddt || !dBm || !dCm || (z && !dz)))
    return GDN_ERR_NULL;
  if (!A_log || !dA_log) return GDN_ERR_NULL;
  const size_t need = bwd_space(pl).total;
  if (need > 0 && !workspace) return GDN_ERR_NULL;
  for (const void* q : {x_scales ? nullptr : x, dt, Bm, Cm, z_scales ? nullptr : z, d_y, (const void*)dx,
                        (const void*)ddt, (const void*)dBm, (const void*)dCm, (const void*)dz})
    if (!aligned(q, pl.esz)) return GDN_ERR_ALIGN;
  for (const float* q : {A_log, skip, dt_bias, initial_state, d_final_state, (const float*)dA_log,
                         (const float*)dskip, (const float*)ddt_bias, (const float*)d_initial_state})
    if (!aligned(q, 4)) return GDN_ERR_ALIGN;
  if (!aligned(cu_seqlens, 8) || !aligned(workspace, kWsAlign)) return GDN_ERR_ALIGN;
  if (workspace_bytes < need) return GDN_ERR_WORKSPACE;
  pl.geo.cu = cu_seqlens;
  return scan_bwd_run(pl,
                      {x, x_scales, dt, A_log, Bm, Cm, skip, z, z_scales, dt_bias, initial_state, d_y,
                       d_final_state, dx, ddt, dA_log, dBm, dCm, dskip, dz, ddt_bias, d_initial_state},
                      workspace, static_cast<hipStream_t>(stream));
}

}  // extern "C"
