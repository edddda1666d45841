// gdn_scan_api.hip -- entry points of the selective scan's forward pass and decode
// step: validation, tiles and launches.  See include/gdn.h.
#include "gdn_scan_host.h"

namespace {

// Tokens per tile.  256 CUs are taken for granted, so that sizes alone decide and the
// workspace is the same on every device.  Measured on MI355X, N = 16 bf16, us per call:
//   one tile per sequence, which forms the states once, from a wave per SIMD on (1024;
//   packed sequences are one row and are always cut): T=512, D=4096, B=16 (1024 waves)
//   197 against 228 in tiles; B=12 (768) 196 either way; B=64, T=128, D=2048 (2048) 72
//   against 137;
//   else tiles for about 8192 waves, of 32 tokens at least: B=2, T=2048, D=2048 (64 waves
//   a tile) 72 with 32 tokens, 76 with 64, 78 with 128, 78 with 16; T=32768 packed (32
//   waves) 428 with 128, 438 with 64, 441 with 256, 483 with 32 (the join's chain grows);
//   16 tokens where 32 leave less than 2048 waves: B=3, T=777, D=1002, G=2 fp32 (48 waves)
//   50 against 53 with 32, and 53 with 8.
constexpr int kOneTileWaves = 1024, kTileWaves = 8192, kTile = 32, kShortTile = 16;

int scan_fwd_len(const ScanPlan& pl) {
  const gdn::ScanGeo& g = pl.geo;
  const int64_t waves = (int64_t)g.cgroups * g.nw * (pl.packed ? 1 : g.B);  // of one tile per row
  if (g.T <= kTile || (!pl.packed && waves >= kOneTileWaves)) return std::max(g.T, 1);
  if (waves * ceil_div(g.T, kTile) < kOneTileWaves * 2) return kShortTile;
  const int64_t tiles = std::max<int64_t>(kTileWaves / waves, 1);
  const int64_t len = ceil_div(ceil_div(g.T, tiles), gdn::kScanGroup) * gdn::kScanGroup;
  return (int)std::max<int64_t>(len, kTile);
}

gdn_status_t fwd_sizes(const gdn_scan_params_t* p, bool packed, ScanPlan* pl) {
  const gdn_status_t st = scan_sizes(p, packed, pl);
  if (st != GDN_OK) return st;
  const int ns = p->N <= 8 ? 8 : 16;
  scan_waves(&pl->geo, ns, (int)ceil_div(p->N, ns));
  scan_tiles(pl, scan_fwd_len(*pl));
  return GDN_OK;
}

// f(E, BE, NS, WHOLE, SPLIT) as default-constructed tags.
template <typename F> gdn_status_t scan_dispatch(const ScanPlan& pl, bool direct, F&& f) {
  using Yes = std::true_type;
  using No = std::false_type;
  auto states = [&](auto e, auto be, auto whole) {
    if (pl.geo.np == 8) return f(e, be, std::integral_constant<int, 8>{}, whole, No{});
    const std::integral_constant<int, 16> ns;
    return pl.geo.nw > 1 ? f(e, be, ns, whole, Yes{}) : f(e, be, ns, whole, No{});
  };
  if (pl.esz == 4) return direct ? states(0.f, 0.f, Yes{}) : states(0.f, 0.f, No{});
  return direct ? states(gdn::bf16{}, gdn::bf16{}, Yes{}) : states(gdn::bf16{}, 0.f, No{});
}

struct FwdSpace {
  size_t states, sums, rows, total;
};
FwdSpace fwd_space(const ScanPlan& pl) {
  FwdSpace w{};
  const size_t tiles = pl.geo.ntiles > 1 ? (size_t)scan_all_tiles(pl) : 0;
  size_t off = 0;
  w.states = off; off = align_up(off + tiles * pl.geo.np * pl.geo.D * 4);
  w.sums = off;   off = align_up(off + tiles * pl.geo.D * 4);
  w.rows = off;   off += 2 * scan_rows_bytes(pl);
  w.total = off;
  return w;
}

struct FwdArgs {
  const void *x, *dt;
  const float* A_log;
  const void *Bm, *Cm;
  const float* skip;
  const void* z;
  const float *dt_bias, *h0;
  void* y;
  float* fin;
};

gdn_status_t scan_fwd_run(ScanPlan pl, const FwdArgs& a, void* ws, hipStream_t s) {
  gdn::ScanGeo& g = pl.geo;
  const int64_t main_blocks = pl.tok > 0 ? scan_all_tiles(pl) * g.cgb : 0;
  const int64_t empties = (g.cu || g.T == 0) && a.fin ? g.S : 0;
  if (!grid_fits(main_blocks + empties, 64 * g.nw * g.upw)) return GDN_ERR_UNSUPPORTED;
  const FwdSpace sp = fwd_space(pl);
  char* w = static_cast<char*>(ws);
  float* states = reinterpret_cast<float*>(w + sp.states);
  float* sums = reinterpret_cast<float*>(w + sp.sums);
  const bool direct = scan_rows_direct(pl, a.Bm, a.Cm);
  const void *Bm = a.Bm, *Cm = a.Cm;
  hipError_t err = hipSuccess;
  auto ok = [&](hipError_t e) {
    if (e != hipSuccess && err == hipSuccess) err = e;
  };
  if (!direct && pl.tok > 0) {
    float* Bw = reinterpret_cast<float*>(w + sp.rows);
    float* Cw = reinterpret_cast<float*>(w + sp.rows + scan_rows_bytes(pl));
    ok(pl.esz == 2 ? scan_copy_rows<gdn::bf16>(&pl, Bm, Cm, Bw, Cw, s) : scan_copy_rows<float>(&pl, Bm, Cm, Bw, Cw, s));
    Bm = Bw;
    Cm = Cw;
  }
  if (pl.tok == 0) g.ntiles = 0;  // no tile blocks: the first block is the first sequence's
  if (main_blocks + empties == 0) return GDN_OK;
  gdn_status_t st = scan_dispatch(pl, direct, [&](auto e, auto be, auto ns, auto whole, auto split) {
    using E = decltype(e);
    using BE = decltype(be);
    constexpr int NS = decltype(ns)::value;
    constexpr bool WHOLE = decltype(whole)::value, SPLIT = decltype(split)::value;
    const gdn::Src x{a.x, nullptr, pl.ldx}, z{a.z, nullptr, pl.ldz};
    const E* dt = static_cast<const E*>(a.dt);
    const BE *b = static_cast<const BE*>(Bm), *c = static_cast<const BE*>(Cm);
    E* y = static_cast<E*>(a.y);
    const dim3 block(64 * g.nw * g.upw);
    if (g.ntiles > 1) {
      ok(launch(gdn::gdn_scan_kernel<E, BE, NS, WHOLE, SPLIT, true>, dim3((unsigned)main_blocks), block, s, g, x, dt, z,
                a.A_log, b, c, a.skip, a.dt_bias, a.h0, states, sums, y, a.fin));
      ok(launch(gdn::gdn_scan_join_kernel, scan_join_grid(g, 1), dim3(256), s, g, a.A_log, gdn::JoinArgs{states, sums},
                gdn::JoinArgs{}));
    }
    ok(launch(gdn::gdn_scan_kernel<E, BE, NS, WHOLE, SPLIT, false>, dim3((unsigned)(main_blocks + empties)), block, s, g, x,
              dt, z, a.A_log, b, c, a.skip, a.dt_bias, a.h0, states, sums, y, a.fin));
    return GDN_OK;
  });
  if (st != GDN_OK) return st;
  return err == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // namespace

extern "C" {

size_t gdn_scan_fwd_workspace_size(const gdn_scan_params_t* p, int packed) {
  ScanPlan pl;
  return fwd_sizes(p, packed != 0, &pl) == GDN_OK ? fwd_space(pl).total : 0;
}

gdn_status_t gdn_scan_fwd(const gdn_scan_params_t* p, const void* x, const void* dt, const float* A_log,
                          const void* Bm, const void* Cm, const float* skip, const void* z,
                          const float* dt_bias, const int64_t* cu_seqlens, const float* initial_state,
                          void* y, float* final_state, void* workspace, size_t workspace_bytes,
                          void* stream) {
  ScanPlan pl;
  gdn_status_t st = fwd_sizes(p, cu_seqlens != nullptr, &pl);
  if (st != GDN_OK) return st;
  if (pl.tok > 0 && (!x || !dt || !A_log || !Bm || !Cm || !y)) return GDN_ERR_NULL;
  const size_t need = fwd_space(pl).total;
  if (need > 0 && !workspace) return GDN_ERR_NULL;
  for (const void* q : {x, dt, Bm, Cm, z, (const void*)y})
    if (!aligned(q, pl.esz)) return GDN_ERR_ALIGN;
  for (const float* q : {A_log, skip, dt_bias, initial_state, (const float*)final_state})
    if (!aligned(q, 4)) return GDN_ERR_ALIGN;
  if (!aligned(cu_seqlens, 8) || !aligned(workspace, kWsAlign)) return GDN_ERR_ALIGN;
  if (workspace_bytes < need) return GDN_ERR_WORKSPACE;
  pl.geo.cu = cu_seqlens;
  return scan_fwd_run(pl, {x, dt, A_log, Bm, Cm, skip, z, dt_bias, initial_state, y, final_state},
                      workspace, static_cast<hipStream_t>(stream));
}

gdn_status_t gdn_scan_decode(const gdn_scan_params_t* p, const void* x, const void* dt, const float* A_log,
                             const void* Bm, const void* Cm, const float* skip, const void* z,
                             const float* dt_bias, const float* state, float* new_state, void* y,
                             void* stream) {
  ScanPlan pl;
  gdn_status_t st = scan_sizes(p, false, &pl);
  if (st != GDN_OK) return st;
  if (p->num_seqs != 0) return GDN_ERR_SHAPE;
  if (p->B > 0 && (!state || !new_state)) return GDN_ERR_NULL;
  if ((pl.tok > 0 && (!x || !dt || !Bm || !Cm || !y)) || (p->B > 0 && !A_log)) return GDN_ERR_NULL;
  for (const void* q : {x, dt, Bm, Cm, z, (const void*)y})
    if (!aligned(q, pl.esz)) return GDN_ERR_ALIGN;
  for (const float* q : {A_log, skip, dt_bias, state, (const float*)new_state})
    if (!aligned(q, 4)) return GDN_ERR_ALIGN;
  if (p->B == 0) return GDN_OK;
  const gdn::ScanGeo& g = pl.geo;
  int nl = 1;
  while (nl * 4 < g.N) nl <<= 1;
  const size_t four = 4 * pl.esz;
  const bool vec = g.N % 4 == 0 && aligned(state, 16) && aligned(new_state, 16) && aligned(A_log, 16) &&
                   aligned(Bm, four) && aligned(Cm, four) && g.ldb % 4 == 0 && g.ldc % 4 == 0;
  const int64_t blocks = ceil_div((int64_t)g.B * g.D * nl, 256);
  if (!grid_fits(blocks, 256)) return GDN_ERR_UNSUPPORTED;
  auto go = [&](auto e) {
    using E = decltype(e);
    return launch(vec ? gdn::gdn_scan_decode_kernel<E, true> : gdn::gdn_scan_decode_kernel<E, false>,
                  dim3((unsigned)blocks), dim3(256),
                  static_cast<hipStream_t>(stream), g, gdn::Src{x, nullptr, pl.ldx}, static_cast<const E*>(dt),
                  gdn::Src{z, nullptr, pl.ldz}, A_log, static_cast<const E*>(Bm), static_cast<const E*>(Cm),
                  skip, dt_bias, state, new_state, static_cast<E*>(y), nl);
  };
  return (pl.esz == 2 ? go(gdn::bf16{}) : go(0.f)) == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // extern "C"
