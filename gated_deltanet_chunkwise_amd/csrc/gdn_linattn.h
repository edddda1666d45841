// gdn_linattn.h -- linear attention with a decay for each head, on gfx950.
//
// Per sequence and value head, with a = exp(log_decay[hv]):
//     H_t = a H_{t-1} + k_t v_t^T            (K x V, fp32)
//     o_t = scale H_t^T q_t
//
// Chunks of 64 tokens.  With H the state ahead of a chunk of n tokens, its tokens counted
// from 0,
//     o_t = scale (sum_{s<=t} a^(t-s) (q_t . k_s) v_s + a^(t+1) H^T q_t)
//     H'  = a^n H + sum_s a^(n-1-s) k_s v_s^T
// Powers of a are formed as exp2((t-s) log2 a), never as quotients, so that no decay however
// fast overflows.
//
// The gradients have the same form with the operands in other places.  With dH the gradient
// of the state behind the chunk,
//     dq_t = scale (sum_{s<=t} a^(t-s) (d_o_t . v_s) k_s + a^(t+1) H d_o_t)
//     dk_s = scale sum_{t>=s} a^(t-s) (v_s . d_o_t) q_t + a^(n-1-s) dH v_s
//     dv_s = scale sum_{t>=s} a^(t-s) (k_s . q_t) d_o_t + a^(n-1-s) dH^T k_s
//     dH'  = a^n dH + scale sum_t a^(t+1) q_t d_o_t^T       (the state's ahead of the chunk)
// so one kernel computes all four: three operands (a, b, c), rows a_i . b_j weighted and
// applied to c_j, and a state of b_j c_j^T that is carried from chunk to chunk, forwards or
// (REV) backwards:
//                a     b     c     state      direction
//     o          q     k     v     H          forwards
//     dq         d_o   v     k     H^T        forwards
//     dv         k     q     d_o   dH         backwards
//     dk         v     d_o   q     dH^T       backwards
//
// Sequences are cut into segments of whole chunks, which run side by side: one launch forms
// each segment's own contribution to the state, a second joins them (the decay of a segment
// is known without its data), a third runs every segment from its true start.  Where the
// heads and sequences alone fill the device there is one segment per sequence and only the
// third launch.
#pragma once
#include "gdn_layer.h"

namespace gdn {

struct AttnGeo {
  int B, T, H, HV, G, N;  // N sequences; G = HV / H
  int chunks;             // chunks per segment
  int nseg;               // segments per sequence (without offsets)
  int slots;              // segments in all, or (packed) an upper bound
  const int64_t* cu;
  bool zero;              // rows of the output behind the last sequence are set to 0
};

// Rows of one operand: token t's values of head `hv / div` at p + t ld + (hv / div) width.
struct AttnRows {
  const void* p;
  int64_t ld;
  int div;
};

// What a pass does with the states: element [i][j] of a head's (rows as operand b, columns as
// operand c) at i rs + j cs.
struct AttnState {
  const float* start;  // [starts][HV][..], or nullptr: zero
  float* end;          // [ends][HV][..], or nullptr: not written
  int rs, cs;
  bool by_slot;        // start and end by segment (else by sequence)
};

// log_decay as the base-2 exponent; a^n for a whole n >= 0 (a = 0: 0^0 = 1).
__device__ __forceinline__ float decay_power(float l2, int n) {
  return n == 0 ? 1.f : __builtin_amdgcn_exp2f((float)n * l2);
}

// The segment of a slot: sequence n, its number in the sequence, tokens [t0, t0 + len).
//
// Packed sequences have slot floor(cu[n] / L) + n + i for segment i of sequence n (L tokens
// per segment): ceil((y - x) / L) <= floor(y / L) - floor(x / L) + 1 keeps the sequences'
// slots apart, and no table has to be made on the device first; T / L + N slots hold all.
// The search for n compares 64 offsets at a time.
struct Segment {
  int n, i, t0, len;

  __device__ __forceinline__ static int seq_slot(const AttnGeo& g, int n) {
    return (seq_offset(g.cu, n, g.T) / kChunk) / g.chunks + n;
  }
  // False for a slot that no token is in: i == 0 then still tells a sequence without tokens.
  __device__ __forceinline__ bool find(const AttnGeo& g, int slot) {
    const int64_t L = (int64_t)g.chunks * kChunk;
    int64_t start, end;
    if (!g.cu) {
      n = slot / g.nseg;
      i = slot - n * g.nseg;
      start = (int64_t)n * g.T;
      end = start + g.T;
    } else {
      int lo = 0, hi = g.N;  // slot(lo) <= slot is taken for granted
      while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64;
        const int64_t at = lo + (int64_t)lane_id() * step;
        const bool in = lane_id() == 0 || (at < hi && seq_slot(g, (int)at) <= slot);
        const uint64_t out = ~__ballot(in);  // (lane 0 is never among them)
        lo += ((out ? __builtin_ctzll(out) : 64) - 1) * step;
        hi = min(lo + step, hi);
      }
      n = __builtin_amdgcn_readfirstlane(lo);
      start = seq_offset(g.cu, n, g.T);
      end = max((int64_t)seq_offset(g.cu, n + 1, g.T), start);
      i = slot - seq_slot(g, n);
    }
    t0 = len = 0;
    const int64_t at = start + i * L;
    if (i < 0 || at >= end) return false;
    t0 = (int)at;
    len = (int)min(L, end - at);
    return true;
  }
};

// A chunk's rows in LDS: 64 rows of D, padded so that the transposed reads below (four rows
// of 32 bytes per 16 lanes, two such groups at a time) meet no bank twice.
template <typename E, int D> struct AttnTile {
  static constexpr int LD = D + (sizeof(E) == 2 ? 16 : 4);
  static constexpr int VECS = D * (int)sizeof(E) / 16;  // 16-byte vectors per row
  static constexpr int PER = kChunk * VECS / 256;       // per thread
  E x[kChunk * LD];
};

constexpr int kAttnThreads = 256;

// The rows of a chunk, as loaded: rows from `len` on are the last one's again (whatever is
// formed from them is not used), so that no row of another sequence is read.
template <typename E, int D, int PER>
__device__ __forceinline__ void attn_fetch(u32x4 (&r)[PER], const E* base, int64_t ld, int len) {
  using Tl = AttnTile<E, D>;
  static_assert(PER == Tl::PER, "");
#pragma unroll
  for (int i = 0; i < Tl::PER; ++i) {
    const int idx = threadIdx.x + kAttnThreads * i;
    const int row = min(idx / Tl::VECS, len - 1), col = idx % Tl::VECS;
    r[i] = *reinterpret_cast<const u32x4*>(base + row * ld + col * (16 / (int)sizeof(E)));
  }
}
template <typename E, int D, int PER>
__device__ __forceinline__ void attn_place(AttnTile<E, D>& t, const u32x4 (&r)[PER]) {
  using Tl = AttnTile<E, D>;
  static_assert(PER == Tl::PER, "");
#pragma unroll
  for (int i = 0; i < Tl::PER; ++i) {
    const int idx = threadIdx.x + kAttnThreads * i;
    *reinterpret_cast<u32x4*>(t.x + idx / Tl::VECS * Tl::LD + idx % Tl::VECS * (16 / (int)sizeof(E))) = r[i];
  }
}

// k32 fragment of 32 rows from s0 on, the lane's column c0 + lane % 16: ds_read_b64_tr_b16
// gives a lane of a group of 16 the four values of its column from the four rows that the
// group's lanes address (four lanes of 8 bytes per row).
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ Frag<bf16> frag_from_columns(const bf16* x, int ld, int s0, int c0) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const int g = lane_id() >> 4, m = lane_id() & 15;
  const bf16* p = x + (s0 + 4 * g + (m >> 2)) * ld + c0 + 4 * (m & 3);
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * ld));
  const auto both = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  return {__builtin_bit_cast(bf16x8, both)};
}
__device__ __forceinline__ Frag<float> frag_from_columns(const float* x, int ld, int s0, int c0) {
  const int g = lane_id() >> 4, m = lane_id() & 15;
  const float* p = x + (s0 + 4 * g) * ld + c0 + m;
  Frag<float> f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.lo[i] = p[i * ld];
    f.hi[i] = p[(16 + i) * ld];
  }
  return f;
}

// c_s w_s as a sum of NP fragments.  A bf16 operand of the state's update is c_s (8 bits)
// times an fp32 weight: one bf16 would leave 2^-9 of every state, which fp32 states must not
// have; two parts leave 2^-17 (states that only ever meet bf16 operands), three 2^-25.
template <int NP>
__device__ __forceinline__ void weighted_parts(const Frag<bf16>& c, const float (&w)[8], Frag<bf16> (&out)[NP]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f = (float)c.x[i] * w[i];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      out[p].x[i] = (bf16)f;
      f -= (float)out[p].x[i];
    }
  }
}
template <int NP>
__device__ __forceinline__ void weighted_parts(const Frag<float>& c, const float (&w)[8], Frag<float> (&out)[NP]) {
  static_assert(NP == 1, "");
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[0].lo[i] = c.lo[i] * w[i];
    out[0].hi[i] = c.hi[i] * w[i + 4];
  }
}

// Rows [from, T) of head hv of the output set to 0, shared out over the slots.
template <typename OT, int D>
__device__ __forceinline__ void attn_zero_rest(const AttnGeo& g, int hv, int slot, OT* out) {
  constexpr int PER_ROW = D * (int)sizeof(OT) / 16, ROWS = kAttnThreads / PER_ROW;
  const int sub = threadIdx.x / PER_ROW, col = threadIdx.x % PER_ROW;
  for (int64_t t = seq_offset(g.cu, g.N, g.T) + (int64_t)slot * ROWS + sub; t < g.T; t += (int64_t)g.slots * ROWS)
    *reinterpret_cast<u32x4*>(out + (t * g.HV + hv) * D + col * (16 / (int)sizeof(OT))) = u32x4{0, 0, 0, 0};
}

// One pass over a segment of one value head by four waves; wave w owns columns
// [w VD/4, (w+1) VD/4) of the state and of the output.  KD, VD: widths of operands a and b,
// and of c.  OUT: rows of the output are formed (else the state alone, from zero).  NP: parts
// of the update's operands.
template <typename E, int KD, int VD, bool OUT> struct AttnLds {
  AttnTile<E, KD> b;
  AttnTile<E, VD> c;
};
template <typename E, int KD, int VD> struct AttnLds<E, KD, VD, true> {
  AttnTile<E, KD> b;
  AttnTile<E, VD> c;
  AttnTile<E, KD> a;
  static constexpr int PLD = kChunk + (sizeof(E) == 2 ? 8 : 4);
  E p[kChunk * PLD];
};

template <typename E, typename OT, int KD, int VD, bool REV, bool OUT, int NP>
__global__ __launch_bounds__(kAttnThreads, sizeof(E) == 2 ? 2 : 1) void gdn_linattn_kernel(
    AttnGeo geo, AttnRows ar, AttnRows br, AttnRows cr, const float* __restrict__ log_decay, AttnState st,
    OT* __restrict__ out, float s_intra, float s_inter, float s_update) {
  constexpr int CT = VD / 64, KT = KD / 16, TT = kChunk / 16;
  using Lds = AttnLds<E, KD, VD, OUT>;
  __shared__ __attribute__((aligned(16))) char smem[sizeof(Lds)];
  Lds& L = *reinterpret_cast<Lds*>(smem);

  int hv, slot;
  xcd_slot_block(blockIdx.x, geo.H, geo.G, geo.slots, hv, slot);
  if constexpr (OUT) {
    if (geo.cu && geo.zero) attn_zero_rest<OT, VD>(geo, hv, slot, out);
  }
  Segment seg;
  // (a sequence without tokens passes its state on)
  if (!seg.find(geo, slot) && (!st.end || st.by_slot || seg.i != 0)) return;
  const int nch = (seg.len + kChunk - 1) / kChunk;
  const int lane = lane_id(), g = lane >> 4, m = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col0 = wave * 16 * CT;
  const float l2 = log_decay[hv] * kLog2e;

  const E* ap = static_cast<const E*>(ar.p) + (int64_t)seg.t0 * ar.ld + (hv / ar.div) * KD;
  const E* bp = static_cast<const E*>(br.p) + (int64_t)seg.t0 * br.ld + (hv / br.div) * KD;
  const E* cp = static_cast<const E*>(cr.p) + (int64_t)seg.t0 * cr.ld + (hv / cr.div) * VD;

  // the state: tile kt holds rows 16 kt + 4 g + r, column col0 + 16 ct + m
  f32x4 H[KT][CT];
  const int64_t sbase = ((int64_t)(st.by_slot ? slot : seg.n) * geo.HV + hv) * (KD * VD);
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      H[kt][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (OUT && st.start) {
        const float* s = st.start + sbase + (int64_t)(16 * kt + 4 * g) * st.rs + (col0 + 16 * ct + m) * st.cs;
#pragma unroll
        for (int r = 0; r < 4; ++r) H[kt][ct][r] = s[r * st.rs];
      }
    }

  u32x4 ra[OUT ? AttnTile<E, KD>::PER : 1], rb[AttnTile<E, KD>::PER], rc[AttnTile<E, VD>::PER];
  auto fetch = [&](int c) {
    const int n = min(kChunk, seg.len - c * kChunk);
    if constexpr (OUT) attn_fetch<E, KD>(ra, ap + (int64_t)c * kChunk * ar.ld, ar.ld, n);
    attn_fetch<E, KD>(rb, bp + (int64_t)c * kChunk * br.ld, br.ld, n);
    attn_fetch<E, VD>(rc, cp + (int64_t)c * kChunk * cr.ld, cr.ld, n);
  };
  if (nch > 0) fetch(REV ? nch - 1 : 0);

  for (int it = 0; it < nch; ++it) {
    const int c = REV ? nch - 1 - it : it;
    const int n = min(kChunk, seg.len - c * kChunk);
    __syncthreads();  // the last chunk's reads are done
    if constexpr (OUT) attn_place<E, KD>(L.a, ra);
    attn_place<E, KD>(L.b, rb);
    attn_place<E, VD>(L.c, rc);
    __syncthreads();
    if (it + 1 < nch) fetch(REV ? c - 1 : c + 1);

    if constexpr (OUT) {
      constexpr int ALD = AttnTile<E, KD>::LD;
      // rows of operand a: tile `wave`; the weighted products with every row of b that they see
      {
        const int t = 16 * wave + m;
        Frag<E> fa[KD / 32];
#pragma unroll
        for (int kb = 0; kb < KD / 32; ++kb) fa[kb] = frag_from_row(L.a.x + t * ALD + 32 * kb);
#pragma unroll
        for (int sg = 0; sg < TT; ++sg) {
          f32x4 p = {0.f, 0.f, 0.f, 0.f};
          if (REV ? sg >= wave : sg <= wave) {
#pragma unroll
            for (int kb = 0; kb < KD / 32; ++kb)
              mma_k32(p, frag_from_row(L.b.x + (16 * sg + m) * ALD + 32 * kb), fa[kb]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int s = 16 * sg + 4 * g + r, gap = REV ? s - t : t - s;
              // (a select, so that nothing of a masked product stays)
              p[r] = gap >= 0 && s < n ? p[r] * (s_intra * decay_power(l2, gap)) : 0.f;
            }
          }
          // rows in blocks of 32 of which at least one is seen are read below
          if (REV ? sg >= (wave & ~1) : sg <= (wave | 1))
            *reinterpret_cast<Quad<E>*>(L.p + t * Lds::PLD + 16 * sg + 4 * g) = make_quad<E>(p);
        }
      }
      // the state's part: O^T = H^T a^T, then weighted by row
      f32x4 acc[CT][TT];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) acc[ct][tt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KD / 32; ++kb) {
        Frag<E> h[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) h[ct] = frag_from_tiles<E>(H[2 * kb][ct], H[2 * kb + 1][ct]);
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          const Frag<E> a = frag_from_row(L.a.x + (16 * tt + m) * ALD + 32 * kb);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) mma_k32(acc[ct][tt], h[ct], a);
        }
      }
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        const int t = 16 * tt + m;
        const float w = s_inter * decay_power(l2, REV ? max(n - 1 - t, 0) : t + 1);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) acc[ct][tt] *= w;
      }
      __syncthreads();  // the weighted products are there
#pragma unroll
      for (int sb = 0; sb < kChunk / 32; ++sb) {
        Frag<E> v[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) v[ct] = frag_from_columns(L.c.x, AttnTile<E, VD>::LD, 32 * sb, col0 + 16 * ct);
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          if (REV ? 2 * sb + 1 < tt : 2 * sb > tt) continue;
          const Frag<E> p = frag_from_row(L.p + (16 * tt + m) * Lds::PLD + 32 * sb);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) mma_k32(acc[ct][tt], v[ct], p);
        }
      }
      OT* orow = out + ((int64_t)(seg.t0 + c * kChunk) * geo.HV + hv) * VD + col0;
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        const int t = 16 * tt + m;
        if (t < n) {
#pragma unroll
          for (int ct = 0; ct < CT; ++ct)
            *reinterpret_cast<Quad<OT>*>(orow + (int64_t)t * geo.HV * VD + 16 * ct + 4 * g) = make_quad<OT>(acc[ct][tt]);
        }
      }
    }

    if (!OUT || st.end || it + 1 < nch) {
      const float a = decay_power(l2, n);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) H[kt][ct] *= a;
#pragma unroll
      for (int sb = 0; sb < kChunk / 32; ++sb) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int s = 32 * sb + (i < 4 ? 4 * g + i : 12 + 4 * g + i);
          w[i] = s < n ? s_update * decay_power(l2, REV ? s + 1 : n - 1 - s) : 0.f;
        }
        Frag<E> v[CT][NP];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
          weighted_parts<NP>(frag_from_columns(L.c.x, AttnTile<E, VD>::LD, 32 * sb, col0 + 16 * ct), w, v[ct]);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          const Frag<E> k = frag_from_columns(L.b.x, AttnTile<E, KD>::LD, 32 * sb, 16 * kt);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int p = 0; p < NP; ++p) mma_k32(H[kt][ct], k, v[ct][p]);
        }
      }
    }
  }

  if (st.end) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        float* s = st.end + sbase + (int64_t)(16 * kt + 4 * g) * st.rs + (col0 + 16 * ct + m) * st.cs;
#pragma unroll
        for (int r = 0; r < 4; ++r) s[r * st.rs] = H[kt][ct][r];
      }
  }
}

// Segments joined: per sequence, head and four elements of the state, in the segments' order
// (REV: from the last),  w[segment] <- cur;  cur <- a^len cur + (what w[segment] held),
// from `start` (or 0); the last cur goes to `end`.  Sequences without tokens pass `start` on
// (w is not read where there is no token at all).
// Loads run kAttnAhead segments ahead.
constexpr int kAttnAhead = 8;

template <int KV, bool REV>
__global__ __launch_bounds__(256) void gdn_linattn_join_kernel(AttnGeo geo, const float* __restrict__ log_decay,
                                                               const float* __restrict__ start, float* w,
                                                               float* __restrict__ end) {
  constexpr int PER = KV / 4 / 256;  // workgroups per head
  const int part = blockIdx.x % PER, unit = blockIdx.x / PER;
  const int hv = unit % geo.HV, n = unit / geo.HV;
  const int64_t at = 4 * ((int64_t)part * 256 + threadIdx.x);
  const float l2 = log_decay[hv] * kLog2e;
  int64_t t0, t1;
  int first;
  if (geo.cu) {
    t0 = seq_offset(geo.cu, n, geo.T);
    t1 = max((int64_t)seq_offset(geo.cu, n + 1, geo.T), t0);
    first = Segment::seq_slot(geo, n);
  } else {
    t0 = 0;
    t1 = geo.T;
    first = n * geo.nseg;
  }
  const int64_t L = (int64_t)geo.chunks * kChunk;
  const int count = (int)((t1 - t0 + L - 1) / L);
  const int64_t head = ((int64_t)n * geo.HV + hv) * KV + at;
  f32x4 cur = {0.f, 0.f, 0.f, 0.f};
  if (start) cur = *reinterpret_cast<const f32x4*>(start + head);
  auto place = [&](int i) {
    return reinterpret_cast<f32x4*>(w + ((int64_t)(first + (REV ? count - 1 - i : i)) * geo.HV + hv) * KV + at);
  };
  const float whole = decay_power(l2, (int)min(L, t1 - t0));
  const float tail = decay_power(l2, (int)(t1 - t0 - (int64_t)(count - 1) * L));
  for (int i = 0; i < count; i += kAttnAhead) {
    f32x4 own[kAttnAhead];
#pragma unroll
    for (int j = 0; j < kAttnAhead; ++j)
      if (i + j < count) own[j] = *place(i + j);
#pragma unroll
    for (int j = 0; j < kAttnAhead; ++j)
      if (i + j < count) {
        *place(i + j) = cur;
        cur = cur * ((REV ? i + j == 0 : i + j == count - 1) ? tail : whole) + own[j];
      }
  }
  if (end) *reinterpret_cast<f32x4*>(end + head) = cur;
}

// Gradients of shared key heads: out[row][h][k] = sum over the G value heads of part[row][h G + j][k],
// in their order.
template <typename E>
__global__ __launch_bounds__(256) void gdn_linattn_sum_kernel(const float* __restrict__ part, E* __restrict__ out,
                                                              int64_t quads, int G, int KQ) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < quads; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / KQ;
    const f32x4* p = reinterpret_cast<const f32x4*>(part) + row * G * KQ + (i - row * KQ);
    f32x4 s = p[0];
    for (int j = 1; j < G; ++j) s += p[(int64_t)j * KQ];
    *reinterpret_cast<Quad<E>*>(out + 4 * i) = make_quad<E>(s);
  }
}

// A few tokens of every sequence, in order, the state in registers: per workgroup one
// (sequence, value head, VB columns), a lane four columns of every 256/(VB/4)-th row.  Bound by
// the state, which is read and written once.
template <typename E, int K, int V, int VB>
__global__ __launch_bounds__(256) void gdn_linattn_decode_kernel(AttnGeo geo, AttnRows qr, AttnRows kr, AttnRows vr,
                                                                 const float* __restrict__ log_decay, const float* state,
                                                                 float* new_state, E* __restrict__ o, float scale) {
  constexpr int LPR = VB / 4, RG = 256 / LPR, R = K / RG, NB = V / VB;
  static_assert(R >= 1 && 64 % LPR == 0, "");
  __shared__ float sk[K], sq[K];
  __shared__ f32x4 so[4][LPR];
  const int blk = blockIdx.x % NB, unit = blockIdx.x / NB;
  const int hv = unit % geo.HV, n = unit / geo.HV;
  const int x = threadIdx.x % LPR, rg = threadIdx.x / LPR, wave = threadIdx.x >> 6;
  const int64_t base = ((int64_t)n * geo.HV + hv) * (K * V) + blk * VB + 4 * x;
  f32x4 H[R];
#pragma unroll
  for (int r = 0; r < R; ++r) H[r] = *reinterpret_cast<const f32x4*>(state + base + (int64_t)(r * RG + rg) * V);
  const float a = decay_power(log_decay[hv] * kLog2e, 1);
  for (int t = 0; t < geo.T; ++t) {
    const int64_t tok = (int64_t)n * geo.T + t;
    if (t) __syncthreads();  // the last token's reads are done
    for (int i = threadIdx.x; i < 2 * K; i += 256) {
      const int h = hv / geo.G;
      if (i < K) sk[i] = (float)(static_cast<const E*>(kr.p) + tok * kr.ld + h * K)[i];
      else sq[i - K] = (float)(static_cast<const E*>(qr.p) + tok * qr.ld + h * K)[i - K];
    }
    float v[4];
    const E* vp = static_cast<const E*>(vr.p) + tok * vr.ld + hv * V + blk * VB + 4 * x;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (float)vp[j];
    const f32x4 vv = {v[0], v[1], v[2], v[3]};
    __syncthreads();
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      H[r] = H[r] * a + vv * sk[r * RG + rg];
      acc += H[r] * sq[r * RG + rg];
    }
#pragma unroll
    for (int d = LPR; d < 64; d <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] += __shfl_xor(acc[j], d);
    if (lane_id() < LPR) so[wave][x] = acc;
    __syncthreads();
    if (threadIdx.x < LPR)
      *reinterpret_cast<Quad<E>*>(o + (tok * geo.HV + hv) * V + blk * VB + 4 * x) =
          make_quad<E>((so[0][x] + so[1][x] + so[2][x] + so[3][x]) * scale);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) *reinterpret_cast<f32x4*>(new_state + base + (int64_t)(r * RG + rg) * V) = H[r];
}

}  // namespace gdn
