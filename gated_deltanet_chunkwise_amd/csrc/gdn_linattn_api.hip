// gdn_linattn_api.hip -- entry points of linear attention with a decay for each head:
// validation, segments and launches.  See include/gdn.h.
#include <cmath>

#include "gdn_host.h"
#include "gdn_linattn.h"

namespace {

using gdn::AttnGeo;
using gdn::AttnPass;
using gdn::AttnRows;
using gdn::AttnState;
using gdn::kChunk;

// Segments of a sequence up to which each sums its start itself.
constexpr int kSumMost = 8;

struct AttnPlan {
  AttnGeo geo;
  int K, V;
  size_t esz;
  int64_t tok;  // tokens in all
  bool packed;
  bool one;     // no sequence has more than one segment
  int64_t states;  // of segments, per head, in the workspace
  float scale;
  int64_t ldq, ldk, ldv;
};

// Chunks per segment, for sequences of `chunks` in `units` (sequence, head) pairs or, packed, one
// row of them per head that holds `packed` sequences; `passes` in one launch (3 backwards); G heads
// share a key head.  256 CUs in 8 XCDs are taken for granted, so that the workspace is the same on
// every device, and that a CU runs one workgroup of the last launch at a time: so it is but for bf16
// 64 x 64, of which two or three fit, and the forward pass of 128 x 64, two, which the rounds below do
// not count.  Packed sequences end with a
// short segment each; no more than 32 are counted, since offsets may be padded with empty ones, which
// cost a workgroup per head that ends at once.
//
// Of the lengths that fill 1 to 8 rounds of workgroups and the shortest ones, that of the least time
// by figures in us as measured at widths of 128: a chunk in the last launch 4.1 (bf16, with operands in
// one part; a quarter less where few CUs are busy) or 14 (fp32: matrix cores), in the first 2 or 5.5.
// In two parts a bf16 chunk takes 4.6, with which one call in twenty would choose another length; of
// narrower widths it takes down to 2.1, and lengths are then up to a fifth off the best.  Further: a
// workgroup's own start 5, a state that it reads for it 0.7; the first launch 5, the join 6, 0.065
// per segment of a sequence and the states that it reads and writes.  Segments of one length run in
// whole rounds of an XCD; those of packed sequences in whatever order, a part of one behind the mean.
//
// Measured (us; with the forward pass's rounds alone and two chunks at least, and so): backward, 2
// sequences of 2048 tokens, 16 heads of 128 bf16, 98 and 89 (4 and 7 chunks); 5003 packed tokens, 8
// value heads of 128 x 64, 72 and 69 (2 and 5); 3 sequences of 777 tokens, 5 heads of 64 x 128 fp32,
// 33 and 28 (2 and 1); one of 32768, one head of 64 bf16 46 and 39 (2 and 3; with 5 it would take 36).
int64_t segment_chunks(int64_t chunks, int64_t units, int64_t packed, int G, int passes, int K, int V, bool fp32) {
  int64_t best = chunks;
  double least = 1e300;
  const double ends = (double)std::min<int64_t>(packed, 32), area = K * V / 16384.;
  const double chunk = fp32 ? 3.5 + 10.5 * area : 4.1, first = fp32 ? 1.5 + 4. * area : 2.;
  const int sums = passes > 1 ? 2 : 1;  // kinds of states
  const double row = (double)units * passes / 256.;
  for (int i = 0; i <= 16; ++i) {
    // as many segments per row of chunks as fill 0 (one segment) to 8 rounds; 1 to 8 chunks each
    const int64_t fill = std::max<int64_t>((int64_t)(i / row - 0.5 * ends), 1);
    const int64_t len = i <= 8 ? ceil_div(chunks, fill) : std::min<int64_t>(i - 8, chunks), n = ceil_div(chunks, len);
    const double start = 5. + 0.7 * area * (n == 1 ? 0 : n <= kSumMost ? n : 2);
    const double wgs = packed ? row * (n + ends) : ceil_div(units / G * n, 8) * G * passes / 32.;
    const double one = len * chunk, whole = std::floor(wgs);
    double cost;
    if (wgs <= 1.) cost = one * (0.75 + 0.25 * wgs) + start;
    else if (packed) cost = row * chunks * chunk + wgs * start + 0.3 * (one + start);
    else cost = whole * (one + start) + (wgs > whole ? one * (0.75 + 0.25 * (wgs - whole)) + start : 0.);
    const double states = units * (n + 0.5 * ends) * sums;
    if (n > 1) cost += 5. + len * first * std::max(1., (states - units * sums) / 256.);
    if (n > kSumMost) cost += 6. + 0.065 * n / std::max(ends, 1.) + states * area * (16384. * 4 * 3 / 5e6);
    if (cost < least) {
      least = cost;
      best = len;
    }
  }
  return best;
}

// Sizes only; `passes` of the last launch.
gdn_status_t attn_sizes(const gdn_linattn_params_t* p, bool packed, int passes, AttnPlan* out) {
  if (!p) return GDN_ERR_NULL;
  const int32_t dtype = p->dtype & ~GDN_ZERO_REST;
  if (dtype != GDN_F32 && dtype != GDN_BF16) return GDN_ERR_DTYPE;
  if (p->H <= 0 || p->HV <= 0 || p->HV % p->H) return GDN_ERR_SHAPE;
  gdn_status_t st = check_batch(p->B, p->T, p->num_seqs, packed);
  if (st != GDN_OK) return st;
  if ((p->K != 64 && p->K != 128) || (p->V != 64 && p->V != 128)) return GDN_ERR_UNSUPPORTED;
  AttnPlan pl{};
  pl.esz = dtype == GDN_BF16 ? 2 : 4;
  const int64_t qk = (int64_t)p->H * p->K, vw = (int64_t)p->HV * p->V;
  auto bad = [](int64_t ld, int64_t least) { return ld != 0 && ld < least; };
  if (bad(p->q_stride, qk) || bad(p->k_stride, qk) || bad(p->v_stride, vw)) return GDN_ERR_SHAPE;
  pl.ldq = p->q_stride ? p->q_stride : qk;
  pl.ldk = p->k_stride ? p->k_stride : qk;
  pl.ldv = p->v_stride ? p->v_stride : vw;
  // a chunk's rows are 32-bit byte offsets apart
  if (std::max({pl.ldq, pl.ldk, pl.ldv, vw}) > (int64_t)UINT32_MAX / (kChunk * 4)) return GDN_ERR_UNSUPPORTED;
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

  const int64_t chunks = ceil_div(std::max(g.T, 1), kChunk);  // of a sequence, or of the packed row
  g.chunks = (int)segment_chunks(chunks, packed ? g.HV : (int64_t)std::max(g.B, 1) * g.HV, packed ? g.N : 0,
                                 g.G, passes, pl.K, pl.V, pl.esz == 4);
  g.nseg = (int)ceil_div(chunks, g.chunks);
  const int64_t slots = packed ? (int64_t)g.T / kChunk / g.chunks + g.N : (int64_t)g.nseg * g.N;
  if (slots > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  g.slots = (int)slots;
  pl.one = g.nseg == 1;
  const int64_t whole = (int64_t)g.T / kChunk / g.chunks;
  pl.states = pl.one || pl.tok == 0 ? 0 : packed ? whole + std::min<int64_t>(g.N, whole) : slots;  // (Segment)
  *out = pl;
  return GDN_OK;
}

// Bytes of the segments' states; workspaces of both passes.
size_t attn_states(const AttnPlan& pl) { return align_up((size_t)pl.states * pl.geo.HV * pl.K * pl.V * 4); }
size_t attn_partial(const AttnPlan& pl) {
  return pl.geo.G == 1 ? 0 : align_up((size_t)pl.tok * pl.geo.HV * pl.K * 4 * 2);
}

int64_t attn_blocks(const AttnGeo& g) { return ceil_div((int64_t)g.slots * g.H, 8) * 8 * g.G; }
int64_t join_blocks(const AttnPlan& pl) { return (int64_t)pl.geo.N * pl.geo.HV * (pl.K * pl.V / 1024); }

// `f` for widths KD and VD.
template <typename F> hipError_t sized(int KD, int VD, F&& f) {
  using S = std::integral_constant<int, 64>;
  using L = std::integral_constant<int, 128>;
  if (KD == 64) return VD == 64 ? f(S{}, S{}) : f(S{}, L{});
  return VD == 64 ? f(L{}, S{}) : f(L{}, L{});
}

// Without any token the states pass through.
hipError_t pass_on(const AttnPlan& pl, const float* start, float* end, hipStream_t s) {
  const int64_t n = (int64_t)pl.geo.N * pl.geo.HV * pl.K * pl.V / 4;
  if (!end || n == 0) return hipSuccess;
  const int64_t blocks = std::min(ceil_div(n, 256), (int64_t)device_cus() * 16);
  return launch(gdn::gdn_linattn_copy_kernel, dim3((unsigned)blocks), dim3(256), s, start, end, n);
}

// How segments get their starts.
int attn_mode(const AttnPlan& pl) {
  return pl.one ? gdn::kWholeSequence : pl.geo.nseg <= kSumMost ? gdn::kSumSegments : gdn::kJoined;
}

// Whether the launches of a call with `passes` in its last one (3 backwards) fit the grid.
bool attn_fits(const AttnPlan& pl, int passes) {
  if (pl.tok == 0) return true;
  return grid_fits(attn_blocks(pl.geo) * passes, gdn::attn_threads(passes == 1 ? pl.V : std::max(pl.K, pl.V))) &&
         (attn_mode(pl) != gdn::kJoined || grid_fits(join_blocks(pl), 256));
}

template <typename E>
gdn_status_t fwd_run(const AttnPlan& pl, const void* q, const void* k, const void* v, const float* ld,
                     const float* h0, void* o, float* fin, void* ws, hipStream_t s) {
  hipError_t err = hipSuccess;
  auto ok = [&](hipError_t e) {
    if (e != hipSuccess && err == hipSuccess) err = e;
  };
  const AttnRows a{q, pl.ldq, pl.geo.G}, b{k, pl.ldk, pl.geo.G}, c{v, pl.ldv, 1};
  const AttnState st{h0, fin, pl.V, 1, static_cast<float*>(ws), attn_mode(pl), false};
  const AttnPass x{a, b, c, st, o, pl.scale, pl.scale, 1.f};
  if (pl.tok == 0) {
    ok(pass_on(pl, h0, fin, s));
  } else {
    ok(sized(pl.K, pl.V, [&](auto kd, auto vd) {
      constexpr int K = decltype(kd)::value, V = decltype(vd)::value;
      const dim3 grid((unsigned)attn_blocks(pl.geo)), block(gdn::attn_threads(V));
      if (!pl.one) {
        ok(launch(gdn::gdn_linattn_kernel<E, E, K, V, false, false>, grid, block, s, pl.geo, x, ld));
        if (st.mode == gdn::kJoined)
          ok(launch(gdn::gdn_linattn_join_kernel<K, V>, dim3((unsigned)join_blocks(pl)), dim3(256), s, pl.geo, st, ld));
      }
      return launch(gdn::gdn_linattn_kernel<E, E, K, V, false, true>, grid, block, s, pl.geo, x, ld);
    }));
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
  pl.geo.zero = pl.packed;
  if (pl.tok == 0) {
    ok(pass_on(pl, x.d_fin, x.dh0, s));
    return err == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
  }
  char* base = static_cast<char*>(ws);
  float* part = reinterpret_cast<float*>(base + 2 * attn_states(pl));  // of dq, then of dk
  float* wh = reinterpret_cast<float*>(base);
  float* wd = reinterpret_cast<float*>(base + attn_states(pl));
  const int mode = attn_mode(pl);
  const int64_t row = pl.tok * pl.geo.HV * K;
  // dq goes by H^T, dk by dH^T, dv by dH
  const AttnPass xq{d_o, v, k, {x.h0, nullptr, 1, V, wh, mode, false}, G == 1 ? x.dq : part, pl.scale, pl.scale, 1.f};
  const AttnPass xk{v, d_o, q, {x.d_fin, nullptr, 1, V, wd, mode, true}, G == 1 ? x.dk : part + row, pl.scale, 1.f, pl.scale};
  const AttnPass xv{k, q, d_o, {x.d_fin, x.dh0, V, 1, wd, mode, false}, x.dv, pl.scale, 1.f, pl.scale};
  ok(sized(K, V, [&](auto kd, auto vd) {
    constexpr int KD = decltype(kd)::value, VD = decltype(vd)::value;
    const int blocks = (int)attn_blocks(pl.geo);
    const dim3 block(gdn::attn_threads(std::max(KD, VD)));
    if (!pl.one) {
      ok(launch(gdn::gdn_linattn_bwd_kernel<E, E, KD, VD, false>, dim3((unsigned)blocks * 2), block, s, pl.geo, xq, xk,
                xv, x.ld, blocks));
      if (mode == gdn::kJoined)
        ok(launch(gdn::gdn_linattn_bwd_join_kernel<KD, VD>, dim3((unsigned)join_blocks(pl), 2), dim3(256), s, pl.geo,
                  xq.st, xv.st, x.ld));
    }
    const dim3 grid((unsigned)blocks * 3);
    if (G == 1) return launch(gdn::gdn_linattn_bwd_kernel<E, E, KD, VD, true>, grid, block, s, pl.geo, xq, xk, xv, x.ld, blocks);
    // of shared heads: each value head's own, then their sum
    ok(launch(gdn::gdn_linattn_bwd_kernel<E, float, KD, VD, true>, grid, block, s, pl.geo, xq, xk, xv, x.ld, blocks));
    const int64_t quads = pl.tok * pl.geo.H * (K / 4);
    const int64_t n = std::min(ceil_div(quads, 256), (int64_t)device_cus() * 16);
    return launch(gdn::gdn_linattn_sum_kernel<E>, dim3((unsigned)n, 2), dim3(256), s, part, part + row,
                  static_cast<E*>(x.dq), static_cast<E*>(x.dk), quads, G, K / 4);
  }));
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
  return attn_sizes(p, packed != 0, 1, &pl) == GDN_OK ? attn_states(pl) : 0;
}

gdn_status_t gdn_linattn_fwd(const gdn_linattn_params_t* p, const void* q, const void* k, const void* v,
                             const float* log_decay, const int64_t* cu_seqlens, const float* initial_state, void* o,
                             float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
  AttnPlan pl;
  gdn_status_t st = attn_sizes(p, cu_seqlens != nullptr, 1, &pl);
  if (st != GDN_OK) return st;
  if (!log_decay || (pl.tok > 0 && (!q || !k || !v || !o))) return GDN_ERR_NULL;
  const size_t need = attn_states(pl);
  if (need > 0 && !workspace) return GDN_ERR_NULL;
  if (!rows_ok({q, k, v, o, initial_state, final_state}, {pl.ldq, pl.ldk, pl.ldv}, pl.esz) || !aligned(log_decay, 4) ||
      !aligned(cu_seqlens, 8) || !aligned(workspace, kWsAlign))
    return GDN_ERR_ALIGN;
  if (workspace_bytes < need) return GDN_ERR_WORKSPACE;
  if (!attn_fits(pl, 1)) return GDN_ERR_UNSUPPORTED;
  pl.geo.cu = cu_seqlens;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return pl.esz == 2 ? fwd_run<gdn::bf16>(pl, q, k, v, log_decay, initial_state, o, final_state, workspace, s)
                     : fwd_run<float>(pl, q, k, v, log_decay, initial_state, o, final_state, workspace, s);
}

size_t gdn_linattn_bwd_workspace_size(const gdn_linattn_params_t* p, int packed) {
  AttnPlan pl;
  return attn_sizes(p, packed != 0, 3, &pl) == GDN_OK ? 2 * attn_states(pl) + attn_partial(pl) : 0;
}

gdn_status_t gdn_linattn_bwd(const gdn_linattn_params_t* p, const void* q, const void* k, const void* v,
                             const float* log_decay, const int64_t* cu_seqlens, const float* initial_state,
                             const void* d_o, const float* d_final_state, void* dq, void* dk, void* dv,
                             float* d_initial_state, void* workspace, size_t workspace_bytes, void* stream) {
  AttnPlan pl;
  gdn_status_t st = attn_sizes(p, cu_seqlens != nullptr, 3, &pl);
  if (st != GDN_OK) return st;
  if (!log_decay || (pl.tok > 0 && (!q || !k || !v || !d_o || !dq || !dk || !dv))) return GDN_ERR_NULL;
  const size_t need = 2 * attn_states(pl) + attn_partial(pl);
  if (need > 0 && !workspace) return GDN_ERR_NULL;
  if (!rows_ok({q, k, v, d_o, dq, dk, dv, initial_state, d_final_state, d_initial_state}, {pl.ldq, pl.ldk, pl.ldv},
               pl.esz) || !aligned(log_decay, 4) || !aligned(cu_seqlens, 8) || !aligned(workspace, kWsAlign))
    return GDN_ERR_ALIGN;
  if (workspace_bytes < need) return GDN_ERR_WORKSPACE;
  if (!attn_fits(pl, 3)) return GDN_ERR_UNSUPPORTED;
  pl.geo.cu = cu_seqlens;
  const AttnBwd x{q, k, v, log_decay, initial_state, d_o, d_final_state, dq, dk, dv, d_initial_state};
  hipStream_t s = static_cast<hipStream_t>(stream);
  return pl.esz == 2 ? bwd_run<gdn::bf16>(pl, x, workspace, s) : bwd_run<float>(pl, x, workspace, s);
}

gdn_status_t gdn_linattn_decode(const gdn_linattn_params_t* p, const void* q, const void* k, const void* v,
                                const float* log_decay, const float* state, float* new_state, void* o, void* stream) {
  AttnPlan pl;
  gdn_status_t st = attn_sizes(p, false, 1, &pl);
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
  auto typed = [&](auto e) { return sized(p->K, p->V, [&](auto kd, auto vd) { return go(e, kd, vd); }); };
  return (pl.esz == 2 ? typed(gdn::bf16{}) : typed(0.f)) == hipSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

}  // extern "C"
