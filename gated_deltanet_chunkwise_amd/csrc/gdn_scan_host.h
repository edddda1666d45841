// gdn_scan_host.h -- sizes, tiles and workspace that the scan's entry points share.
#pragma once
#include "gdn_host.h"
#include "gdn_scan.h"

namespace {

struct ScanPlan {
  gdn::ScanGeo geo;
  int64_t ldx, ldz;
  size_t esz;
  int64_t tok;   // tokens in all
  bool packed;
};

// Sizes only.
inline gdn_status_t scan_sizes(const gdn_scan_params_t* p, bool packed, ScanPlan* out) {
  if (!p) return GDN_ERR_NULL;
  const int32_t dtype = p->dtype & ~GDN_ZERO_REST;
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (p->D <= 0 || p->G <= 0 || p->N <= 0 || p->D % p->G) return GDN_ERR_SHAPE;
  gdn_status_t st = check_batch(p->B, p->T, p->num_seqs, packed);
  if (st != GDN_OK) return st;
  if (p->N > 64) return GDN_ERR_UNSUPPORTED;
  const int64_t bn = (int64_t)p->G * p->N;
  // 32-bit indices of a row of states; rows of the batch in a grid's second dimension
  if (bn > INT32_MAX || (int64_t)p->D * 64 > INT32_MAX || p->B > 65535) return GDN_ERR_UNSUPPORTED;
  // beyond any memory; workspaces take up to about 1 KB per token and channel, counted in 64 bits
  if ((int64_t)p->B * p->T > ((int64_t)1 << 48) / p->D) return GDN_ERR_UNSUPPORTED;
  auto bad = [](int64_t ld, int64_t least) { return ld != 0 && ld < least; };
  if (bad(p->x_stride, p->D) || bad(p->dt_stride, p->D) || bad(p->z_stride, p->D) ||
      bad(p->b_stride, bn) || bad(p->c_stride, bn))
    return GDN_ERR_SHAPE;
  ScanPlan pl{};
  pl.packed = packed;
  pl.esz = dtype == GDN_BF16 ? 2 : 4;
  pl.tok = (int64_t)p->B * p->T;
  pl.ldx = p->x_stride ? p->x_stride : p->D;
  pl.ldz = p->z_stride ? p->z_stride : p->D;
  gdn::ScanGeo& g = pl.geo;
  g.B = p->B; g.T = p->T; g.D = p->D; g.G = p->G; g.N = p->N;
  g.S = packed ? p->num_seqs : p->B;
  g.DG = p->D / p->G;
  g.zero = packed && (p->dtype & GDN_ZERO_REST);
  g.wpg = (int)ceil_div(g.DG, 64);
  g.cgroups = g.G * g.wpg;
  g.lddt = p->dt_stride ? p->dt_stride : p->D;
  g.ldb = p->b_stride ? p->b_stride : bn;
  g.ldc = p->c_stride ? p->c_stride : bn;
  g.bgs = g.cgs = p->N;
  *out = pl;
  return GDN_OK;
}

// ns states per lane and nw waves per 64 channels; workgroups of four waves where nw
// divides into them.
inline void scan_waves(gdn::ScanGeo* g, int ns, int nw) {
  g->nw = nw;
  g->np = nw * ns;
  g->upw = nw < 4 ? 4 / nw : 1;
  g->cgb = (int)ceil_div(g->cgroups, g->upw);
}

inline void scan_tiles(ScanPlan* pl, int len) {
  pl->geo.len = len;
  pl->geo.ntiles = (int)std::max<int64_t>(ceil_div(pl->geo.T, len), 1);
}
inline int64_t scan_all_tiles(const ScanPlan& pl) {
  return (int64_t)pl.geo.ntiles * (pl.packed ? 1 : pl.geo.B);
}

inline dim3 scan_join_grid(const gdn::ScanGeo& g, int chains) {
  return dim3((unsigned)ceil_div((int64_t)g.np * g.D, 256), g.cu ? 1 : g.B, chains);
}

// Whether Bm and Cm can be read in place: whole rows of np states at 4-byte aligned
// addresses (fp32: the addresses are always aligned).
inline bool scan_rows_direct(const ScanPlan& pl, const void* Bm, const void* Cm) {
  const gdn::ScanGeo& g = pl.geo;
  if (g.N != g.np) return false;
  if (pl.esz == 4) return true;
  return g.ldb % 2 == 0 && g.ldc % 2 == 0 && aligned(Bm, 4) && aligned(Cm, 4);
}
// Bytes of one of the two fp32 copies otherwise.
inline size_t scan_rows_bytes(const ScanPlan& pl) {
  return align_up((size_t)pl.tok * pl.geo.G * pl.geo.np * 4);
}

template <typename E>
hipError_t scan_copy_rows(ScanPlan* pl, const void* Bm, const void* Cm, float* Bw, float* Cw, hipStream_t s) {
  gdn::ScanGeo& g = pl->geo;
  const int64_t n = pl->tok * g.G * g.np;
  const int64_t blocks = std::min(ceil_div(n, 256), (int64_t)device_cus() * 16);
  const hipError_t e = launch(gdn::gdn_scan_rows_kernel<E>, dim3((unsigned)blocks), dim3(256), s,
                              static_cast<const E*>(Bm), static_cast<const E*>(Cm), g.ldb, g.ldc, pl->tok,
                              g.G, g.N, g.np, Bw, Cw);
  g.ldb = g.ldc = (int64_t)g.G * g.np;
  g.bgs = g.cgs = g.np;
  return e;
}

}  // namespace
