// gdn_linattn_api.hip -- entry points of linear attention with a decay for each head:
// validation, segments and launches.  See include/gdn.h.
#include "gdn_host.h"
#include "gdn_linattn.h"

namespace {

using gdn::AttnGeo;
using gdn::AttnRows;
using gdn::AttnState;
using gdn::kChunk;

struct AttnPlan {
  AttnGeo geo;
  int K, V;
  size_t esz;
  int64_t tok;  // tokens in all
  bool packed;
  bool one;     // no sequence has more than one segment
  float scale;
  int64_t ldq, ldk, ldv;
};

// Sizes only.
gdn_status_t attn_sizes(const gdn_linattn_params_t* p, bool packed, AttnPlan* out) {
  if (!p) return GDN_ERR_NULL;
  const int32_t dtype = p->dtype & ~GDN_ZERO_REST;
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (p->H <= 0 || p->HV <= 0 || p->HV % p->H) return GDN_ERR_SHAPE;
  gdn_status_t st = check_batch(p->B, p->T, p->num_seqs, packed);
  if (st != GDN_OK) return st;
  if ((p->K != 64 && p->K != 128) || (p->V != 64 && p->V != 128)) return GDN_ERR_UNSUPPORTED;
  AttnPlan pl{};
  pl.esz = dtype == GDN_BF16 ? 2 : 4;
  // token's offsets within a row are 32 bits, and so are sums over rows of all heads below
  if (p->HV > INT32_MAX / 1024) return GDN_ERR_UNSUPPORTED;
  const int64_t qk = (int64_t)p->H * p->K, vw = (int64_t)p->HV * p->V;
  auto bad = [](int64_t ld, int64_t least) { return ld != 0 && ld < least; };
  if (bad(p->q_stride, qk) || bad(p->k_stride, qk) || bad(p->v_stride, vw)) return GDN_ERR_SHAPE;
  pl.ldq = p->q_stride ? p->q_stride : qk;
  pl.ldk = p->k_stride ? p->k_stride : qk;
  pl.ldv = p->v_stride ? p->v_stride : vw;
  AttnGeo& g = pl.geo;
  g.B = p->B; g.T = p->T; g.H = p->H; g.HV = p->HV;
  g.G = p->HV / p->H;
  g.N = packed ? p->num_seqs : p->B;
  g.zero = packed && (p->dtype & GDN_ZERO_REST);
  pl.K = p->K; pl.V = p->V;
  pl.packed = packed;
  pl.tok = (int64_t)p->B * p->T;
  pl.scale = p->scale;
  // beyond any memory: states, and tokens' partial sums, counted in 64 bits below
  if ((int64_t)g.N * g.HV > (int64_t)1 << 40 || pl.tok > ((int64_t)1 << 48) / g.HV) return GDN_ERR_UNSUPPORTED;

  // Segments: about kWorkgroups of them over all heads, of kLeast chunks at least.
  constexpr int64_t kWorkgroups = 512, kLeast = 2;
  const int64_t chunks = ceil_div(std::max(g.T, 1), kChunk);  // of a sequence, or of the packed row
  const int64_t units = std::max<int64_t>((int64_t)(packed ? 1 : std::max(g.B, 1)) * g.HV, 1);
  const int64_t want = std::max<int64_t>(kWorkgroups / units, 1);
  g.chunks = (int)std::min(std::max(ceil_div(chunks, want), kLeast), chunks);
  g.nseg = (int)ceil_div(chunks, g.chunks);
  const int64_t slots = packed ? (int64_t)g.T / kChunk / g.chunks + g.N : (int64_t)g.nseg * g.N;
  if (slots > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  g.slots = (int)slots;
  pl.one = g.nseg == 1;
  *out = pl;
  return GDN_OK;
}

// Bytes of the segments' states; workspaces of both passes.
size_t attn_states(const AttnPlan& pl) {
  if (pl.one || pl.tok == 0) return 0;
  return align_up((size_t)pl.geo.slots * pl.geo.HV * pl.K * pl.V * 4);
}
size_t attn_partial(const AttnPlan& pl) {
  return pl.geo.G == 1 ? 0 : align_up((size_t)pl.tok * pl.geo.HV * pl.K * 4);
}

bool attn_fits(const AttnPlan& pl) {
  return grid_fits((int64_t)pl.geo.slots * pl.geo.HV, gdn::kAttnThreads) &&
         grid_fits((int64_t)pl.geo.N * pl.geo.HV * (pl.K * pl.V / 1024), 256);
}

struct Weights {
  float intra, inter, update;
};

template <typename E, typename OT, int KD, int VD, bool REV, bool OUT>
hipError_t pass_run(const AttnGeo& g, AttnRows a, AttnRows b, AttnRows c, const float* ld, AttnState st, OT* out,
                    Weights w, hipStream_t s) {
  // three parts where states go out as fp32
  constexpr bool exact = sizeof(E) == 4;
  const dim3 grid((unsigned)((int64_t)g.slots * g.HV)), block(gdn::kAttnThreads);
  if constexpr (exact)
    return launch(gdn::gdn_linattn_kernel<E, OT, KD, VD, REV, OUT, 1>, grid, block, s, g, a, b, c, ld, st, out,
                  w.intra, w.inter, w.update);
  else if (st.end)
    return launch(gdn::gdn_linattn_kernel<E, OT, KD, VD, REV, OUT, 3>, grid, block, s, g, a, b, c, ld, st, out,
                  w.intra, w.inter, w.update);
  else
    return launch(gdn::gdn_linattn_kernel<E, OT, KD, VD, REV, OUT, 2>, grid, block, s, g, a, b, c, ld, st, out,
                  w.intra, w.inter, w.update);
}

template <typename E, typename OT, bool REV, bool OUT>
hipError_t pass(const AttnPlan& pl, int KD, int VD, AttnRows a, AttnRows b, AttnRows c, const float* ld,
                AttnState st, void* out, Weights w, hipStream_t s) {
  OT* o = static_cast<OT*>(out);
  if (KD == 64)
    return VD == 64 ? pass_run<E, OT, 64, 64, REV, OUT>(pl.geo, a, b, c, ld, st, o, w, s)
                    : pass_run<E, OT, 64, 128, REV, OUT>(pl.geo, a, b, c, ld, st, o, w, s);
  return VD == 64 ? pass_run<E, OT, 128, 64, REV, OUT>(pl.geo, a, b, c, ld, st, o, w, s)
                  : pass_run<E, OT, 128, 128, REV, OUT>(pl.geo, a, b, c, ld, st, o, w, s);
}

template <bool REV>
hipError_t join(const AttnPlan& pl, const float* ld, const float* start, float* w, float* end, hipStream_t s) {
  const int kv = pl.K * pl.V;
  const dim3 grid((unsigned)((int64_t)pl.geo.N * pl.geo.HV * (kv / 1024))), block(256);
  auto kern = kv == 4096 ? gdn::gdn_linattn_join_kernel<4096, REV>
              : kv == 8192 ? gdn::gdn_linattn_join_kernel<8192, REV> : gdn::gdn_linattn_join_kernel<16384, REV>;
  return launch(kern, grid, block, s, pl.geo, ld, start, w, end);
}

// The states alone pass to `end` where there is no token.
hipError_t pass_on(const AttnPlan& pl, const float* ld, const float* start, float* end, hipStream_t s) {
  return end && pl.geo.N > 0 ? join<false>(pl, ld, start, nullptr, end, s) : hipSuccess;
}

template <typename E>
gdn_status_t fwd_run(const AttnPlan& pl, const void* q, const void* k, const void* v, const float* ld,
                     const float* h0, void* o, float* fin, void* ws, hipStream_t s) {
  hipError_t err = hipSuccess;
  auto ok = [&](hipError_t e) {
    if (e != hipSuccess && err == hipSuccess) err = e;
  };
  const AttnRows a{q, pl.ldq, pl.geo.G}, b{k, pl.ldk, pl.geo.G}, c{v, pl.ldv, 1};
  const int K = pl.K, V = pl.V;
  const Weights w{pl.scale, pl.scale, 1.f};
  if (pl.tok == 0) {
    ok(pass_on(pl, ld, h0, fin, s));
  } else if (pl.one) {
    ok(pass<E, E, false, true>(pl, K, V, a, b, c, ld, {h0, fin, V, 1, false}, o, w, s));
  } else {
    float* st = static_cast<float*>(ws);
    ok(pass<E, E, false, false>(pl, K, V, a, b, c, ld, {nullptr, st, V, 1, true}, nullptr, w, s));
    ok(join<false>(pl, ld, h0, st, fin, s));
    ok(pass<E, E, false, true>(pl, K, V, a, b, c, ld, {st, nullptr, V, 1, true}, o, w, s));
  }
  return err == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

struct AttnBwd {
  const void *q, *k, *v;
  const float *ld, *h0;
  const void* d_o;
  const float* d_fin;
  void *dq, *dk, *dv;
  float* dh0;
};

template <typename E>
gdn_status_t bwd_run(AttnPlan pl, const AttnBwd& x, void* ws, hipStream_t s) {
  hipError_t err = hipSuccess;
  auto ok = [&](hipError_t e) {
    if (e != hipSuccess && err == hipSuccess) err = e;
  };
  const int K = pl.K, V = pl.V, G = pl.geo.G;
  const AttnRows q{x.q, pl.ldq, G}, k{x.k, pl.ldk, G}, v{x.v, pl.ldv, 1}, d_o{x.d_o, (int64_t)pl.geo.HV * V, 1};
  const Weights fw{pl.scale, pl.scale, 1.f}, bw{pl.scale, 1.f, pl.scale};
  pl.geo.zero = pl.packed;
  if (pl.tok == 0) {
    ok(pass_on(pl, x.ld, x.d_fin, x.dh0, s));
    return err == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
  }
  char* base = static_cast<char*>(ws);
  float* part = reinterpret_cast<float*>(base + 2 * attn_states(pl));
  AttnState sq, sk, sv;  // the states of the passes that form dq, dk and dv
  if (pl.one) {
    sq = {x.h0, nullptr, 1, V, false};
    sk = {x.d_fin, nullptr, 1, V, false};
    sv = {x.d_fin, x.dh0, V, 1, false};
  } else {
    float* sth = reinterpret_cast<float*>(base);
    float* std_ = reinterpret_cast<float*>(base + attn_states(pl));
    ok(pass<E, E, false, false>(pl, K, V, q, k, v, x.ld, {nullptr, sth, V, 1, true}, nullptr, fw, s));
    ok(pass<E, E, true, false>(pl, K, V, k, q, d_o, x.ld, {nullptr, std_, V, 1, true}, nullptr, bw, s));
    ok(join<false>(pl, x.ld, x.h0, sth, nullptr, s));
    ok(join<true>(pl, x.ld, x.d_fin, std_, x.dh0, s));
    sq = {sth, nullptr, 1, V, true};
    sk = {std_, nullptr, 1, V, true};
    sv = {std_, nullptr, V, 1, true};
  }
  // gradients of shared heads: each value head's own, then their sum
  auto shared = [&](void* out) {
    const int64_t quads = pl.tok * pl.geo.H * (K / 4);
    const int64_t blocks = std::min(ceil_div(quads, 256), (int64_t)device_cus() * 16);
    ok(launch(gdn::gdn_linattn_sum_kernel<E>, dim3((unsigned)blocks), dim3(256), s, part, static_cast<E*>(out), quads,
              G, K / 4));
  };
  if (G == 1) {
    ok(pass<E, E, false, true>(pl, V, K, d_o, v, k, x.ld, sq, x.dq, fw, s));
    ok(pass<E, E, true, true>(pl, V, K, v, d_o, q, x.ld, sk, x.dk, bw, s));
  } else {
    ok(pass<E, float, false, true>(pl, V, K, d_o, v, k, x.ld, sq, part, fw, s));
    shared(x.dq);
    ok(pass<E, float, true, true>(pl, V, K, v, d_o, q, x.ld, sk, part, bw, s));
    shared(x.dk);
  }
  ok(pass<E, E, true, true>(pl, K, V, k, q, d_o, x.ld, sv, x.dv, bw, s));
  return err == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

// Rows are read 16 bytes at a time.
bool rows_ok(std::initializer_list<const void*> rows, std::initializer_list<int64_t> strides, size_t esz) {
  for (const void* q : rows)
    if (!aligned(q, 16)) return false;
  for (int64_t ld : strides)
    if (ld * (int64_t)esz % 16) return false;
  return true;
}

}  // namespace

extern "C" {

size_t gdn_linattn_fwd_workspace_size(const gdn_linattn_params_t* p, int packed) {
  AttnPlan pl;
  return attn_sizes(p, packed != 0, &pl) == GDN_OK ? attn_states(pl) : 0;
}

gdn_status_t gdn_linattn_fwd(const gdn_linattn_params_t* p, const void* q, const void* k, const void* v,
                             const float* log_decay, const int64_t* cu_seqlens, const float* initial_state, void* o,
                             float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
  AttnPlan pl;
  gdn_status_t st = attn_sizes(p, cu_seqlens != nullptr, &pl);
  if (st != GDN_OK) return st;
  if (!log_decay || (pl.tok > 0 && (!q || !k || !v || !o))) return GDN_ERR_NULL;
  const size_t need = attn_states(pl);
  if (need > 0 && !workspace) return GDN_ERR_NULL;
  if (!rows_ok({q, k, v, o, initial_state, final_state}, {pl.ldq, pl.ldk, pl.ldv}, pl.esz) || !aligned(log_decay, 4) ||
      !aligned(cu_seqlens, 8) || !aligned(workspace, kWsAlign))
    return GDN_ERR_ALIGN;
  if (workspace_bytes < need) return GDN_ERR_WORKSPACE;
  if (!attn_fits(pl)) return GDN_ERR_UNSUPPORTED;
  pl.geo.cu = cu_seqlens;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return pl.esz == 2 ? fwd_run<gdn::bf16>(pl, q, k, v, log_decay, initial_state, o, final_state, workspace, s)
                     : fwd_run<float>(pl, q, k, v, log_decay, initial_state, o, final_state, workspace, s);
}

size_t gdn_linattn_bwd_workspace_size(const gdn_linattn_params_t* p, int packed) {
  AttnPlan pl;
  return attn_sizes(p, packed != 0, &pl) == GDN_OK ? 2 * attn_states(pl) + attn_partial(pl) : 0;
}

gdn_status_t gdn_linattn_bwd(const gdn_linattn_params_t* p, const void* q, const void* k, const void* v,
                             const float* log_decay, const int64_t* cu_seqlens, const float* initial_state,
                             const void* d_o, const float* d_final_state, void* dq, void* dk, void* dv,
                             float* d_initial_state, void* workspace, size_t workspace_bytes, void* stream) {
  AttnPlan pl;
  gdn_status_t st = attn_sizes(p, cu_seqlens != nullptr, &pl);
  if (st != GDN_OK) return st;
  if (!log_decay || (pl.tok > 0 && (!q || !k || !v || !d_o || !dq || !dk || !dv))) return GDN_ERR_NULL;
  const size_t need = 2 * attn_states(pl) + attn_partial(pl);
  if (need > 0 && !workspace) return GDN_ERR_NULL;
  if (!rows_ok({q, k, v, d_o, dq, dk, dv, initial_state, d_final_state, d_initial_state}, {pl.ldq, pl.ldk, pl.ldv},
               pl.esz) || !aligned(log_decay, 4) || !aligned(cu_seqlens, 8) || !aligned(workspace, kWsAlign))
    return GDN_ERR_ALIGN;
  if (workspace_bytes < need) return GDN_ERR_WORKSPACE;
  if (!attn_fits(pl)) return GDN_ERR_UNSUPPORTED;
  pl.geo.cu = cu_seqlens;
  const AttnBwd x{q, k, v, log_decay, initial_state, d_o, d_final_state, dq, dk, dv, d_initial_state};
  hipStream_t s = static_cast<hipStream_t>(stream);
  return pl.esz == 2 ? bwd_run<gdn::bf16>(pl, x, workspace, s) : bwd_run<float>(pl, x, workspace, s);
}

gdn_status_t gdn_linattn_decode(const gdn_linattn_params_t* p, const void* q, const void* k, const void* v,
                                const float* log_decay, const float* state, float* new_state, void* o, void* stream) {
  AttnPlan pl;
  gdn_status_t st = attn_sizes(p, false, &pl);
  if (st != GDN_OK) return st;
  if (p->num_seqs != 0) return GDN_ERR_SHAPE;
  if (p->B > 0 && (!state || !new_state || !log_decay)) return GDN_ERR_NULL;
  if (pl.tok > 0 && (!q || !k || !v || !o)) return GDN_ERR_NULL;
  if (!rows_ok({q, k, v, o, state, new_state}, {pl.ldq, pl.ldk, pl.ldv}, pl.esz) || !aligned(log_decay, 4)) return GDN_ERR_ALIGN;
  if (p->B == 0 || (p->T == 0 && state == new_state)) return GDN_OK;
  constexpr int VB = 32;
  const int64_t blocks = (int64_t)p->B * p->HV * (p->V / VB);
  if (!grid_fits(blocks, 256)) return GDN_ERR_UNSUPPORTED;
  auto go = [&](auto e, auto kd, auto vd) {
    using E = decltype(e);
    return launch(gdn::gdn_linattn_decode_kernel<E, decltype(kd)::value, decltype(vd)::value, VB>, dim3((unsigned)blocks),
                  dim3(256), static_cast<hipStream_t>(stream), pl.geo, AttnRows{q, pl.ldq, pl.geo.G},
                  AttnRows{k, pl.ldk, pl.geo.G}, AttnRows{v, pl.ldv, 1}, log_decay, state, new_state,
                  static_cast<E*>(o), pl.scale);
  };
  using S = std::integral_constant<int, 64>;
  using L = std::integral_constant<int, 128>;
  auto sized = [&](auto e) {
    if (p->K == 64) return p->V == 64 ? go(e, S{}, S{}) : go(e, S{}, L{});
    return p->V == 64 ? go(e, L{}, S{}) : go(e, L{}, L{});
  };
  return (pl.esz == 2 ? sized(gdn::bf16{}) : sized(0.f)) == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // extern "C"
