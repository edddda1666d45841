// gdn_conv_api.hip -- entry points of the short causal convolution and the 8-bit
// activation checkpoints: validation and launches.  See include/gdn.h.
#include "gdn_conv.h"
#include "gdn_host.h"
#include "gdn_pack8.h"

namespace {

struct ConvPlan {
  gdn::ConvGeo geo;
  int64_t ld;     // elements between x's rows
  size_t esz;
  int64_t rows;   // backward: rows of partial sums
  size_t total;   // backward workspace bytes
};

// Sizes only.
gdn_status_t conv_sizes(const gdn_conv_params_t* p, bool packed, ConvPlan* out) {
  if (!p) return GDN_ERR_NULL;
  const int32_t dtype = p->dtype & ~GDN_ZERO_REST;
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (p->C <= 0 || p->W <= 0 || (p->activation != 0 && p->activation != 1)) return GDN_ERR_SHAPE;
  gdn_status_t st = check_batch(p->B, p->T, p->num_seqs, packed);
  if (st != GDN_OK) return st;
  if (p->W < 2 || p->W > 4) return GDN_ERR_UNSUPPORTED;
  if (p->x_stride != 0 && p->x_stride < p->C) return GDN_ERR_SHAPE;
  ConvPlan pl{};
  pl.ld = p->x_stride ? p->x_stride : p->C;
  pl.esz = dtype == GDN_BF16 ? 2 : 4;
  gdn::ConvGeo& g = pl.geo;
  g.B = p->B; g.T = p->T; g.C = p->C;
  g.N = packed ? p->num_seqs : p->B;
  g.silu = p->activation;
  g.zero = packed && (p->dtype & GDN_ZERO_REST);
  g.nblk = (int)ceil_div(p->C, gdn::kPackBlock);
  // beyond any grid, and near where three rows of states per sequence pass 64 bits
  if ((int64_t)g.N * p->C > ((int64_t)1 << 38) / 3) return GDN_ERR_UNSUPPORTED;
  *out = pl;
  return GDN_OK;
}

// Channels per lane where rows and addresses allow: two of bf16; of fp32 four forward, one
// in the decode step and backward (see the kernels).
constexpr int kFwd32 = 4;
int conv_vec(const ConvPlan& pl, int fp32 = 1) { return pl.esz == 2 ? 2 : fp32; }

// The backward pass's tiles: each lane's tile as long as leaves about 12 waves per
// CU (256 CUs are taken for granted, so that the workspace is the same on every
// device), 16 tokens at least (its W-1 tokens of overlap are then at most a fifth)
// and 80 at most, the overlap included.  us, W=4: at most 80 and 256 tokens: B=4, T=8192,
// C=2048 bf16 96 and 108, C=2044 119 and 130; 12, 16 and 24 waves: B=1, T=32768, C=512 bf16
// 32, 34 and 40, B=2, T=4096, C=1000 fp32 30, 33 and 36.
void conv_bwd_tiles(const gdn_conv_params_t* p, bool packed, int vec, ConvPlan* pl) {
  gdn::ConvGeo& g = pl->geo;
  g.cvn = p->C / vec;
  const int64_t ntok = (int64_t)p->B * p->T;
  int64_t tile = ntok * g.cvn / (256 * 12 * 64);
  // whole groups of loads for the tile and the W-1 tokens after it
  tile = std::min<int64_t>(std::max<int64_t>(tile / gdn::kConvGroup, 2), 10) * gdn::kConvGroup - (p->W - 1);
  g.tile = (int)tile;
  g.ntiles = (int)std::max<int64_t>(ceil_div(p->T, tile), 1);
  const int64_t tiles = (int64_t)g.ntiles * (packed ? 1 : p->B);
  pl->rows = ceil_div(tiles, gdn::kConvTiles);
  pl->total = align_up((size_t)pl->rows * (p->W + 1) * p->C * 4);
}

size_t conv_ws(const gdn_conv_params_t* p, bool packed, ConvPlan pl) {
  conv_bwd_tiles(p, packed, 1, &pl);  // what misaligned pointers would take
  const size_t total = pl.total;
  if (p->C % conv_vec(pl) == 0) conv_bwd_tiles(p, packed, conv_vec(pl), &pl);
  return std::max(total, pl.total);
}

// Whether rows of C elements from these addresses split into vectors of `vec` elements.
bool vec_ok(const ConvPlan& pl, int vec, std::initializer_list<const void*> rows) {
  if (pl.geo.C % vec || pl.ld % vec) return false;
  for (const void* q : rows)
    if (!aligned(q, vec * pl.esz)) return false;
  return true;
}

template <typename E, int W, int VEC>
gdn_status_t conv_fwd_run(ConvPlan pl, const void* x, const float* w, const float* b,
                          const void* h0, void* y, void* fin, hipStream_t s) {
  gdn::ConvGeo& g = pl.geo;
  g.cvn = g.C / VEC;
  // Tokens per lane: as long as leaves about 16 waves per CU, at least one group of
  // loads, at most 64.  8, 16 and 32 waves, us, bf16: B=1, T=2000, C=8192 20, 16, 17; T=32768,
  // C=512 19, 17, 16; B=4, T=4096, C=2044 31, 32, 31.
  const int64_t ntok = (int64_t)g.B * g.T;
  const int64_t lanes = (int64_t)device_cus() * 16 * 64;
  const int64_t tile = ntok * g.cvn / std::max<int64_t>(lanes, 1) / gdn::kConvGroup * gdn::kConvGroup;
  g.tile = (int)std::min<int64_t>(std::max<int64_t>(tile, gdn::kConvGroup), 64);
  g.ntiles = (int)ceil_div(g.T, g.tile);
  const int64_t units = (int64_t)g.ntiles * (g.cu ? 1 : g.B) + (fin ? (int64_t)g.N * (W - 1) : 0);
  const int64_t blocks = ceil_div(units * g.cvn, 256);
  if (blocks == 0) return GDN_OK;
  if (!grid_fits(blocks, 256)) return GDN_ERR_UNSUPPORTED;  // (the kernel's work items are 32 bits as well)
  return launch(gdn::gdn_conv_fwd_kernel<E, W, VEC>, dim3((unsigned)blocks), dim3(256), s, g,
                gdn::Src{x, nullptr, pl.ld}, w, b, static_cast<const E*>(h0), static_cast<E*>(y),
                static_cast<E*>(fin)) == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

template <typename E, int W, int VEC>
gdn_status_t conv_decode_run(ConvPlan pl, const void* x, const float* w, const float* b,
                             const void* in, void* out, void* y, hipStream_t s) {
  gdn::ConvGeo& g = pl.geo;
  g.cvn = g.C / VEC;
  const int64_t blocks = ceil_div((int64_t)g.B * g.cvn, 256);
  if (!grid_fits(blocks, 256)) return GDN_ERR_UNSUPPORTED;
  return launch(gdn::gdn_conv_decode_kernel<E, W, VEC>, dim3((unsigned)blocks), dim3(256), s, g,
                gdn::Src{x, nullptr, pl.ld}, w, b, static_cast<const E*>(in), static_cast<E*>(out),
                static_cast<E*>(y)) == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

struct ConvBwdArgs {
  const void* x;
  const uint8_t* scales;
  const float *w, *b;
  const void *h0, *dy, *dfin;
  void* dx;
  float *dw, *db;
  void* dh0;
};

template <typename E, int W, int VEC>
gdn_status_t conv_bwd_run(const ConvPlan& pl, const ConvBwdArgs& a, void* ws, hipStream_t s) {
  const gdn::ConvGeo& g = pl.geo;
  const gdn::Src x{a.x, a.scales, pl.ld};
  float* partial = static_cast<float*>(ws);
  hipError_t err = hipSuccess;
  auto ok = [&](hipError_t e) {
    if (e != hipSuccess && err == hipSuccess) err = e;
  };
  const bool tokens = (int64_t)g.B * g.T > 0;
  const int cgroups = (int)ceil_div(g.cvn, 64);
  const int64_t main_blocks = tokens ? pl.rows * cgroups : 0;
  const int64_t states = a.dh0 ? ceil_div((int64_t)g.N * g.cvn, 256) : 0;
  const int64_t sums = ceil_div((int64_t)(W + 1) * g.C, 64);
  if (!grid_fits(main_blocks + states, 64 * gdn::kConvTiles) || !grid_fits(sums, 1024)) return GDN_ERR_UNSUPPORTED;
  if (main_blocks + states > 0)
    ok(launch(a.scales ? gdn::gdn_conv_bwd_kernel<E, W, VEC, true> : gdn::gdn_conv_bwd_kernel<E, W, VEC, false>,
              dim3((unsigned)(main_blocks + states)), dim3(64 * gdn::kConvTiles), s, g, x, a.w, a.b,
              static_cast<const E*>(a.h0), static_cast<const E*>(a.dy), static_cast<const E*>(a.dfin),
              static_cast<E*>(a.dx), static_cast<E*>(a.dh0), partial, cgroups, (int)main_blocks));
  ok(launch(gdn::gdn_conv_bwd_sums_kernel<W>, dim3((unsigned)sums), dim3(1024), s, partial, tokens ? (int)pl.rows : 0, g.C, a.dw, a.db));
  return err == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

// F<E, W, VEC>::run for the call's type and width; `vec`: VEC = conv_vec(.., V32), else 1.
template <template <typename, int, int> class F, int V32, typename... A>
gdn_status_t conv_dispatch(const ConvPlan& pl, int W, bool vec, A&&... a) {
  auto width = [&](auto e, auto v) {
    using E = decltype(e);
    constexpr int V = decltype(v)::value;
    if (W == 2) return F<E, 2, V>::run(pl, a...);
    if (W == 3) return F<E, 3, V>::run(pl, a...);
    return F<E, 4, V>::run(pl, a...);
  };
  using One = std::integral_constant<int, 1>;
  if (pl.esz == 4) return vec ? width(0.f, std::integral_constant<int, V32>{}) : width(0.f, One{});
  return vec ? width(gdn::bf16{}, std::integral_constant<int, 2>{}) : width(gdn::bf16{}, One{});
}
template <typename E, int W, int VEC> struct FwdRun {
  template <typename... A> static gdn_status_t run(A&&... a) { return conv_fwd_run<E, W, VEC>(a...); }
};
template <typename E, int W, int VEC> struct DecodeRun {
  template <typename... A> static gdn_status_t run(A&&... a) { return conv_decode_run<E, W, VEC>(a...); }
};
template <typename E, int W, int VEC> struct BwdRun {
  template <typename... A> static gdn_status_t run(A&&... a) { return conv_bwd_run<E, W, VEC>(a...); }
};

gdn_status_t pack_sizes(int dt, int64_t rows, int32_t C) {
  if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_DTYPE;
  if (rows < 0 || C < 1) return GDN_ERR_SHAPE;
  if (rows > INT64_MAX / 8 / C) return GDN_ERR_SHAPE;
  return GDN_OK;
}

template <typename E>
gdn_status_t pack_run(const void* xv, int64_t ld, int64_t rows, int C, int8_t* codes,
                      uint8_t* scales, hipStream_t s) {
  const E* x = static_cast<const E*>(xv);
  const int nblk = (int)ceil_div(C, gdn::kPackBlock);
  const int64_t cap = (int64_t)device_cus() * 16;  // workgroups beyond that loop
  if (C < 8) {
    const int64_t blocks = std::min(ceil_div(rows * nblk, 8), cap);
    return launch(gdn::gdn_pack8_scalar_kernel<E>, dim3((unsigned)blocks), dim3(256), s, x, ld, codes,
                  scales, rows, C, nblk) == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
  }
  const int64_t vpr = (int64_t)nblk * 4;
  const int64_t most = std::max<int64_t>(((int64_t)1 << 30) / vpr, 1);  // rows per launch
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = std::min(most, rows - r);
    const int64_t blocks = std::min(ceil_div(n * vpr, 256 * gdn::kPackUnroll), cap);
    if (launch(C % 8 ? gdn::gdn_pack8_vec_kernel<E, true> : gdn::gdn_pack8_vec_kernel<E, false>, dim3((unsigned)blocks), dim3(256), s, x + r * ld, ld,
               codes + r * C, scales + r * nblk, (uint32_t)n, C, (uint32_t)vpr) != hipSuccess)
      return GDN_ERR_LAUNCH;
  }
  return GDN_OK;
}

template <typename E>
gdn_status_t unpack_run(const int8_t* codes, const uint8_t* scales, int64_t rows, int C, void* yv,
                        hipStream_t s) {
  E* y = static_cast<E*>(yv);
  const int nblk = (int)ceil_div(C, gdn::kPackBlock);
  const int64_t cap = (int64_t)device_cus() * 16;
  if (C < 8) {
    const int64_t blocks = std::min(ceil_div(rows * C, 256), 2 * cap);
    return launch(gdn::gdn_unpack8_scalar_kernel<E>, dim3((unsigned)blocks), dim3(256), s, codes, scales,
                  y, rows * C, C, nblk) == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
  }
  const int64_t vpr = ceil_div(C, 8), most = std::max<int64_t>(((int64_t)1 << 30) / vpr, 1);
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = std::min(most, rows - r);
    const int64_t blocks = std::min(ceil_div(n * vpr, 256 * gdn::kPackUnroll), cap);
    if (launch(C % 8 ? gdn::gdn_unpack8_vec_kernel<E, true> : gdn::gdn_unpack8_vec_kernel<E, false>, dim3((unsigned)blocks), dim3(256), s, codes + r * C,
               scales + r * nblk, y + r * C, (uint32_t)n, C, (uint32_t)vpr, (uint32_t)nblk) != hipSuccess)
      return GDN_ERR_LAUNCH;
  }
  return GDN_OK;
}

int enum_int(const gdn_dtype_t& e) {  // any int may stand in an enum argument (see gdn_api.hip)
  int v;
  __builtin_memcpy(&v, &e, sizeof v);
  return v;
}

}  // namespace

extern "C" {

gdn_status_t gdn_conv_fwd(const gdn_conv_params_t* p, const void* x, const float* weight,
                          const float* bias, const int64_t* cu_seqlens, const void* initial_state,
                          void* y, void* final_state, void* stream) {
  ConvPlan pl;
  gdn_status_t st = conv_sizes(p, cu_seqlens != nullptr, &pl);
  if (st != GDN_OK) return st;
  const bool tokens = (int64_t)p->B * p->T > 0;
  if (tokens && (!x || !weight || !y)) return GDN_ERR_NULL;
  if (!aligned(x, pl.esz) || !aligned(y, pl.esz) || !aligned(initial_state, pl.esz) ||
      !aligned(final_state, pl.esz) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(cu_seqlens, 8))
    return GDN_ERR_ALIGN;
  pl.geo.cu = cu_seqlens;
  return conv_dispatch<FwdRun, kFwd32>(pl, p->W, vec_ok(pl, conv_vec(pl, kFwd32), {x, y, initial_state, final_state}), x, weight,
                                       bias, initial_state, y, final_state, static_cast<hipStream_t>(stream));
}

gdn_status_t gdn_conv_decode(const gdn_conv_params_t* p, const void* x, const float* weight,
                             const float* bias, const void* state, void* new_state, void* y,
                             void* stream) {
  ConvPlan pl;
  gdn_status_t st = conv_sizes(p, false, &pl);
  if (st != GDN_OK) return st;
  if (p->num_seqs != 0) return GDN_ERR_SHAPE;
  if (p->B > 0 && (!state || !new_state)) return GDN_ERR_NULL;
  if ((int64_t)p->B * p->T > 0 && (!x || !weight || !y)) return GDN_ERR_NULL;
  if (!aligned(x, pl.esz) || !aligned(y, pl.esz) || !aligned(state, pl.esz) ||
      !aligned(new_state, pl.esz) || !aligned(weight, 4) || !aligned(bias, 4))
    return GDN_ERR_ALIGN;
  if (p->B == 0 || (p->T == 0 && state == new_state)) return GDN_OK;
  if (p->T == 0) {  // no weights to read: the state passes through
    pl.geo.cu = nullptr;
    return conv_dispatch<FwdRun, kFwd32>(pl, p->W, vec_ok(pl, conv_vec(pl, kFwd32), {state, new_state}), x, weight, bias, state,
                                         y, new_state, static_cast<hipStream_t>(stream));
  }
  return conv_dispatch<DecodeRun, 1>(pl, p->W, vec_ok(pl, conv_vec(pl), {x, y, state, new_state}), x, weight, bias, state,
                                     new_state, y, static_cast<hipStream_t>(stream));
}

size_t gdn_conv_bwd_workspace_size(const gdn_conv_params_t* p, int packed) {
  ConvPlan pl;
  if (conv_sizes(p, packed != 0, &pl) != GDN_OK) return 0;
  return conv_ws(p, packed != 0, pl);
}

gdn_status_t gdn_conv_bwd(const gdn_conv_params_t* p, const void* x, const uint8_t* x_scales,
                          const float* weight, const float* bias, const int64_t* cu_seqlens,
                          const void* initial_state, const void* d_y, const void* d_final_state,
                          void* dx, float* dweight, float* dbias, void* d_initial_state,
                          void* workspace, size_t workspace_bytes, void* stream) {
  const bool packed = cu_seqlens != nullptr;
  ConvPlan pl;
  gdn_status_t st = conv_sizes(p, packed, &pl);
  if (st != GDN_OK) return st;
  if (x_scales && p->x_stride != 0 && p->x_stride != p->C) return GDN_ERR_SHAPE;  // codes are dense
  const bool tokens = (int64_t)p->B * p->T > 0;
  if ((tokens && (!x || !weight || !d_y || !dx)) || !dweight) return GDN_ERR_NULL;
  const size_t need = conv_ws(p, packed, pl);
  if (need > 0 && !workspace) return GDN_ERR_NULL;
  const size_t xa = x_scales ? 1 : pl.esz;
  if (!aligned(x, xa) || !aligned(d_y, pl.esz) || !aligned(dx, pl.esz) ||
      !aligned(initial_state, pl.esz) || !aligned(d_final_state, pl.esz) ||
      !aligned(d_initial_state, pl.esz) || !aligned(weight, 4) || !aligned(bias, 4) ||
      !aligned(dweight, 4) || !aligned(dbias, 4) || !aligned(cu_seqlens, 8) || !aligned(workspace, kWsAlign))
    return GDN_ERR_ALIGN;
  if (workspace_bytes < need) return GDN_ERR_WORKSPACE;
  const int v = conv_vec(pl);
  const bool vec = vec_ok(pl, v, {x_scales ? nullptr : x, d_y, dx, initial_state, d_final_state, d_initial_state}) &&
                   aligned(x, v);
  conv_bwd_tiles(p, packed, vec ? v : 1, &pl);
  pl.geo.cu = cu_seqlens;
  const ConvBwdArgs a{x, x_scales, weight, bias, initial_state, d_y, d_final_state,
                      dx, dweight, dbias, d_initial_state};
  return conv_dispatch<BwdRun, 1>(pl, p->W, vec, a, workspace, static_cast<hipStream_t>(stream));
}

gdn_status_t gdn_pack8(const void* x, gdn_dtype_t dtype, int64_t rows, int32_t C, int64_t x_stride,
                       int8_t* codes, uint8_t* scales, void* stream) {
  const int dt = enum_int(dtype);
  gdn_status_t st = pack_sizes(dt, rows, C);
  if (st != GDN_OK) return st;
  if (x_stride != 0 && x_stride < C) return GDN_ERR_SHAPE;
  if (rows == 0) return GDN_OK;
  if (!x || !codes || !scales) return GDN_ERR_NULL;
  if (!aligned(x, dt == GDN_F32 ? 4 : 2)) return GDN_ERR_ALIGN;
  const int64_t ld = x_stride ? x_stride : C;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dt == GDN_F32 ? pack_run<float>(x, ld, rows, C, codes, scales, s)
                       : pack_run<gdn::bf16>(x, ld, rows, C, codes, scales, s);
}

gdn_status_t gdn_unpack8(const int8_t* codes, const uint8_t* scales, int64_t rows, int32_t C, void* y,
                         gdn_dtype_t dtype, void* stream) {
  const int dt = enum_int(dtype);
  gdn_status_t st = pack_sizes(dt, rows, C);
  if (st != GDN_OK) return st;
  if (rows == 0) return GDN_OK;
  if (!codes || !scales || !y) return GDN_ERR_NULL;
  if (!aligned(y, dt == GDN_F32 ? 4 : 2)) return GDN_ERR_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return dt == GDN_F32 ? unpack_run<float>(codes, scales, rows, C, y, s)
                       : unpack_run<gdn::bf16>(codes, scales, rows, C, y, s);
}

}  // extern "C"
