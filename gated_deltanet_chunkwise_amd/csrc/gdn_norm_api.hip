// gdn_norm_api.hip -- entry points of the norms around a block: validation and launches.
// See include/gdn.h.
#include "gdn_host.h"
#include "gdn_norm.h"

namespace {

using gdn::NormGeo;

constexpr int kMostChannels = 16384;  // a row is held by 1024 lanes of 16 channels at most

struct NormPlan {
  NormGeo geo;
  int32_t dtype, rdtype;  // residual norm: of the residual
};

gdn_status_t norm_sizes(int32_t B, int32_t T, int32_t H, int32_t D, int32_t dtype, int64_t x_stride, int64_t z_stride,
                        float eps, NormPlan* out) {
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (B < 0 || T < 0 || H <= 0 || D <= 0 || !(eps >= 0.f)) return GDN_ERR_SHAPE;
  // rows are 32-bit indices
  if (D > kMostChannels || (int64_t)B * T > (INT32_MAX - 65536) / H) return GDN_ERR_UNSUPPORTED;
  const int64_t width = (int64_t)H * D;
  if ((x_stride != 0 && x_stride < width) || (z_stride != 0 && z_stride < width)) return GDN_ERR_SHAPE;
  NormPlan pl{};
  pl.geo.rows = (int64_t)B * T * H;
  pl.geo.H = H;
  pl.geo.D = D;
  pl.geo.ldx = x_stride ? x_stride : width;
  pl.geo.ldz = z_stride ? z_stride : width;
  pl.geo.eps = eps;
  pl.dtype = pl.rdtype = dtype;
  *out = pl;
  return GDN_OK;
}

gdn_status_t gated_sizes(const gdn_gated_norm_params_t* p, NormPlan* out) {
  if (!p) return GDN_ERR_NULL;
  if (p->gate_first != 0 && p->gate_first != 1) return GDN_ERR_SHAPE;
  return norm_sizes(p->B, p->T, p->H, p->D, p->dtype, p->x_stride, p->z_stride, p->eps, out);
}

gdn_status_t residual_sizes(const gdn_residual_norm_params_t* p, NormPlan* out) {
  if (!p) return GDN_ERR_NULL;
  const gdn_status_t st = norm_sizes(p->B, p->T, 1, p->C, p->dtype, p->x_stride, p->residual_stride, p->eps, out);
  if (st != GDN_OK) return st;
  if (p->residual_dtype != p->dtype && p->residual_dtype != GDN_F32) return GDN_ERR_DTYPE;
  out->rdtype = p->residual_dtype;
  return GDN_OK;
}

inline size_t esize(int32_t dtype) { return dtype == GDN_BF16 ? 2 : 4; }

// f(VEC, LPR, NV, WHOLE) for the lanes and vectors of 16 bytes that hold a row: one vector per lane
// as long as 1024 lanes hold the row, so that the three sums of a backward pass stay in registers,
// then as few as do.  Beyond 8192 channels they do not stay there: the backward kernels spill 74 to
// 176 registers (8M channels bf16 in rows of 8192 and of 16384: gated norm 36 and 84 us, residual norm
// 49 and 159).  WHOLE: no vector is cut off by the row's end, which spares the passes the
// question (backward of a residual norm, B=4, T=4096, C=2048 bf16: 89 us with it, 82 without).  Rows
// below 16 bytes go by channels.
template <typename E, typename F> hipError_t norm_shape(int D, F&& f) {
  constexpr int VEC = 16 / (int)sizeof(E);
  using std::integral_constant;
  auto go = [&](auto lpr, auto nv) {
    return D % VEC ? f(integral_constant<int, VEC>{}, lpr, nv, std::false_type{})
                   : f(integral_constant<int, VEC>{}, lpr, nv, std::true_type{});
  };
  using One = integral_constant<int, 1>;
  using All = integral_constant<int, 1024>;
  if (D < VEC) return f(One{}, integral_constant<int, 8>{}, One{}, std::true_type{});
  const int n = (D + VEC - 1) / VEC;
  if (n <= 8) return go(integral_constant<int, 8>{}, One{});
  if (n <= 16) return go(integral_constant<int, 16>{}, One{});
  if (n <= 32) return go(integral_constant<int, 32>{}, One{});
  if (n <= 64) return go(integral_constant<int, 64>{}, One{});
  if (n <= 256) return go(integral_constant<int, 256>{}, One{});
  if (n <= 512) return go(integral_constant<int, 512>{}, One{});
  if (n <= 1024) return go(All{}, One{});
  if constexpr (VEC == 4)
    if (n > 2048) return go(All{}, integral_constant<int, 4>{});
  return go(All{}, integral_constant<int, 2>{});
}

template <int LPR> int64_t rows_per_block() { return gdn::norm_threads(LPR) / LPR; }

// Workgroups of a backward pass, each with a row of partial sums: as many as fill the device at the
// rows they were measured with (256 CUs are taken for granted, so that the workspace is the same on
// every device).  us, 512, 768 and 1024: gated norm of B=2, T=2048, 16 heads of 128 bf16 23.3, 22.1 and
// 21.4; residual norm of B=4, T=4096, C=2048 bf16 86, 88 and 104 (three workgroups of it fit a CU).
// Wide rows take more than they need, since a workgroup of 1024 lanes fills a CU by itself: at 8192
// channels the partial sums are as many bytes as the data of 8M channels.
constexpr int64_t kGatedBlocks = 1024, kResidualBlocks = 512;
int64_t norm_blocks(const NormPlan& pl, int64_t rpb, int64_t most) { return std::min(ceil_div(pl.geo.rows, rpb), most); }
size_t norm_ws(const NormPlan& pl, int K, int64_t most) {
  return align_up((size_t)std::min(pl.geo.rows, most) * K * pl.geo.D * 4);
}

hipError_t norm_sums(const NormPlan& pl, const float* partial, int64_t rows, int K, gdn::NormSums o, hipStream_t s) {
  return launch(pl.geo.D % 4 ? gdn::gdn_norm_sums_kernel<1> : gdn::gdn_norm_sums_kernel<4>, dim3((unsigned)(K * ceil_div(pl.geo.D, 64))), dim3(1024), s, partial,
                (int)rows, K, pl.geo.D, o);
}

gdn_status_t status(hipError_t e) { return e == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH; }

bool all_aligned(std::initializer_list<const void*> ps, size_t a) {
  for (const void* q : ps)
    if (!aligned(q, a)) return false;
  return true;
}

template <typename E>
gdn_status_t gated_fwd(const NormPlan& pl, const void* x, const float* w, const void* z, void* y, hipStream_t s) {
  return status(norm_shape<E>(pl.geo.D, [&](auto v, auto lpr, auto nv, auto whole) {
    constexpr int LPR = decltype(lpr)::value;
    const int64_t blocks = std::min(ceil_div(pl.geo.rows, rows_per_block<LPR>()), (int64_t)device_cus() * 32);
    return launch(gdn::gdn_gated_norm_kernel<E, decltype(v)::value, LPR, decltype(nv)::value, decltype(whole)::value>, dim3((unsigned)blocks),
                  dim3(gdn::norm_threads(LPR)), s, pl.geo, static_cast<const E*>(x), w, static_cast<const E*>(z),
                  static_cast<E*>(y));
  }));
}

template <typename E>
gdn_status_t gated_bwd(const NormPlan& pl, const void* x, const float* w, const void* z, const void* dy, void* dx,
                       void* dz, float* dw, float* partial, hipStream_t s) {
  int64_t blocks = 0;
  hipError_t err = hipSuccess;
  if (pl.geo.rows > 0)
    err = norm_shape<E>(pl.geo.D, [&](auto v, auto lpr, auto nv, auto whole) {
      constexpr int LPR = decltype(lpr)::value;
      blocks = norm_blocks(pl, rows_per_block<LPR>(), kGatedBlocks);
      return launch(gdn::gdn_gated_norm_bwd_kernel<E, decltype(v)::value, LPR, decltype(nv)::value, decltype(whole)::value>,
                    dim3((unsigned)blocks), dim3(gdn::norm_threads(LPR)), s, pl.geo, static_cast<const E*>(x), w,
                    static_cast<const E*>(z), static_cast<const E*>(dy), static_cast<E*>(dx), static_cast<E*>(dz),
                    partial);
    });
  const hipError_t e = norm_sums(pl, partial, blocks, 1, {{dw, nullptr, nullptr}}, s);
  return status(err != hipSuccess ? err : e);
}

template <typename E, typename R>
gdn_status_t residual_fwd(const NormPlan& pl, const void* x, const void* r, const float* w, const float* post,
                          const float* scale, void* h, void* out, hipStream_t s) {
  return status(norm_shape<E>(pl.geo.D, [&](auto v, auto lpr, auto nv, auto whole) {
    constexpr int LPR = decltype(lpr)::value;
    const int64_t blocks = std::min(ceil_div(pl.geo.rows, rows_per_block<LPR>()), (int64_t)device_cus() * 32);
    return launch(gdn::gdn_residual_norm_kernel<E, R, decltype(v)::value, LPR, decltype(nv)::value, decltype(whole)::value>,
                  dim3((unsigned)blocks), dim3(gdn::norm_threads(LPR)), s, pl.geo, static_cast<const E*>(x),
                  static_cast<const R*>(r), w, post, scale, static_cast<E*>(h), static_cast<R*>(out));
  }));
}

struct ResidualBwd {
  const void *x, *r;
  const float *w, *post, *scale;
  const void *dh, *ds;
  void *dx, *dr;
  float *dw, *dpost, *dscale;
};

template <typename E, typename R>
gdn_status_t residual_bwd(const NormPlan& pl, const ResidualBwd& a, float* partial, hipStream_t s) {
  int64_t blocks = 0;
  hipError_t err = hipSuccess;
  if (pl.geo.rows > 0)
    err = norm_shape<E>(pl.geo.D, [&](auto v, auto lpr, auto nv, auto whole) {
      constexpr int LPR = decltype(lpr)::value;
      blocks = norm_blocks(pl, rows_per_block<LPR>(), kResidualBlocks);
      return launch(gdn::gdn_residual_norm_bwd_kernel<E, R, decltype(v)::value, LPR, decltype(nv)::value, decltype(whole)::value>,
                    dim3((unsigned)blocks), dim3(gdn::norm_threads(LPR)), s, pl.geo, static_cast<const E*>(a.x),
                    static_cast<const R*>(a.r), a.w, a.post, a.scale, static_cast<const E*>(a.dh),
                    static_cast<const R*>(a.ds), static_cast<E*>(a.dx), static_cast<R*>(a.dr), partial);
    });
  const hipError_t e = norm_sums(pl, partial, blocks, 3, {{a.dw, a.dpost, a.dscale}}, s);
  return status(err != hipSuccess ? err : e);
}

}  // namespace

extern "C" {

gdn_status_t gdn_gated_norm_fwd(const gdn_gated_norm_params_t* p, const void* x, const float* weight, const void* z,
                                void* y, void* stream) {
  NormPlan pl;
  gdn_status_t st = gated_sizes(p, &pl);
  if (st != GDN_OK) return st;
  if (!weight || (pl.geo.rows > 0 && (!x || !y))) return GDN_ERR_NULL;
  const size_t e = esize(pl.dtype);
  if (!all_aligned({x, z, y}, e) || !aligned(weight, 4)) return GDN_ERR_ALIGN;
  if (pl.geo.rows == 0) return GDN_OK;
  if (!z) pl.geo.ldz = (int64_t)p->H * p->D;
  pl.geo.mode = !z ? gdn::kGateNone : p->gate_first ? gdn::kGateFirst : gdn::kGateAfter;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return e == 2 ? gated_fwd<gdn::bf16>(pl, x, weight, z, y, s) : gated_fwd<float>(pl, x, weight, z, y, s);
}

size_t gdn_gated_norm_bwd_workspace_size(const gdn_gated_norm_params_t* p) {
  NormPlan pl;
  return gated_sizes(p, &pl) == GDN_OK ? norm_ws(pl, 1, kGatedBlocks) : 0;
}

gdn_status_t gdn_gated_norm_bwd(const gdn_gated_norm_params_t* p, const void* x, const float* weight, const void* z,
                                const void* d_y, void* dx, void* dz, float* dweight, void* workspace,
                                size_t workspace_bytes, void* stream) {
  NormPlan pl;
  gdn_status_t st = gated_sizes(p, &pl);
  if (st != GDN_OK) return st;
  const bool any = pl.geo.rows > 0;
  if (!weight || !dweight || (any && (!x || !d_y || !dx || (z && !dz)))) return GDN_ERR_NULL;
  const size_t need = norm_ws(pl, 1, kGatedBlocks), e = esize(pl.dtype);
  if (need > 0 && !workspace) return GDN_ERR_NULL;
  if (!all_aligned({x, z, d_y, dx, dz}, e) || !all_aligned({weight, dweight}, 4) || !aligned(workspace, kWsAlign))
    return GDN_ERR_ALIGN;
  if (workspace_bytes < need) return GDN_ERR_WORKSPACE;
  if (!z) pl.geo.ldz = (int64_t)p->H * p->D;
  pl.geo.mode = !z ? gdn::kGateNone : p->gate_first ? gdn::kGateFirst : gdn::kGateAfter;
  hipStream_t s = static_cast<hipStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  return e == 2 ? gated_bwd<gdn::bf16>(pl, x, weight, z, d_y, dx, dz, dweight, part, s)
                : gated_bwd<float>(pl, x, weight, z, d_y, dx, dz, dweight, part, s);
}

gdn_status_t gdn_residual_norm_fwd(const gdn_residual_norm_params_t* p, const void* x, const void* residual,
                                   const float* weight, const float* post_weight, const float* scale, void* h,
                                   void* new_residual, void* stream) {
  NormPlan pl;
  gdn_status_t st = residual_sizes(p, &pl);
  if (st != GDN_OK) return st;
  if (!weight || (pl.geo.rows > 0 && (!x || !residual || !h || !new_residual))) return GDN_ERR_NULL;
  if (!all_aligned({x, h}, esize(pl.dtype)) || !all_aligned({residual, new_residual}, esize(pl.rdtype)) ||
      !all_aligned({weight, post_weight, scale}, 4))
    return GDN_ERR_ALIGN;
  if (pl.geo.rows == 0) return GDN_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (pl.dtype == GDN_F32)
    return residual_fwd<float, float>(pl, x, residual, weight, post_weight, scale, h, new_residual, s);
  return pl.rdtype == GDN_F32
             ? residual_fwd<gdn::bf16, float>(pl, x, residual, weight, post_weight, scale, h, new_residual, s)
             : residual_fwd<gdn::bf16, gdn::bf16>(pl, x, residual, weight, post_weight, scale, h, new_residual, s);
}

size_t gdn_residual_norm_bwd_workspace_size(const gdn_residual_norm_params_t* p) {
  NormPlan pl;
  return residual_sizes(p, &pl) == GDN_OK ? norm_ws(pl, 3, kResidualBlocks) : 0;
}

gdn_status_t gdn_residual_norm_bwd(const gdn_residual_norm_params_t* p, const void* x, const void* residual,
                                   const float* weight, const float* post_weight, const float* scale, const void* d_h,
                                   const void* d_new_residual, void* dx, void* dresidual, float* dweight,
                                   float* dpost_weight, float* dscale, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  NormPlan pl;
  gdn_status_t st = residual_sizes(p, &pl);
  if (st != GDN_OK) return st;
  if (!weight || !dweight || (pl.geo.rows > 0 && (!x || !residual || !d_h || !dx || !dresidual))) return GDN_ERR_NULL;
  const size_t need = norm_ws(pl, 3, kResidualBlocks);
  if (need > 0 && !workspace) return GDN_ERR_NULL;
  if (!all_aligned({x, d_h, dx}, esize(pl.dtype)) ||
      !all_aligned({residual, d_new_residual, dresidual}, esize(pl.rdtype)) ||
      !all_aligned({weight, post_weight, scale, dweight, dpost_weight, dscale}, 4) || !aligned(workspace, kWsAlign))
    return GDN_ERR_ALIGN;
  if (workspace_bytes < need) return GDN_ERR_WORKSPACE;
  const ResidualBwd a{x, residual, weight, post_weight, scale, d_h, d_new_residual, dx, dresidual, dweight,
                      post_weight ? dpost_weight : nullptr, scale ? dscale : nullptr};
  hipStream_t s = static_cast<hipStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  if (pl.dtype == GDN_F32) return residual_bwd<float, float>(pl, a, part, s);
  return pl.rdtype == GDN_F32 ? residual_bwd<gdn::bf16, float>(pl, a, part, s)
                              : residual_bwd<gdn::bf16, gdn::bf16>(pl, a, part, s);
}

}  // extern "C"
