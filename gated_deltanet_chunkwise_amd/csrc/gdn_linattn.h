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
// what each segment adds to the state, the next runs every segment from its true start, which
// it sums from what the segments ahead of it added (their decays are known without their data)
// -- or, where sequences have many segments, a launch in between forms the starts.  Where the
// heads and sequences alone fill the device there is one segment per sequence and one launch.
//
// Measured, bf16, 128 x 128.  With 256 workgroups a chunk takes 4.6 us of the launch that forms
// outputs (64 KB per workgroup: 3.6 TB/s, where a copy from memory reaches 5.2; 5.0 where final states
// are asked for, in three parts), with 64 3.8.  Matrix instructions are a fifth to a quarter of it;
// the rest is reads of LDS, barriers and waits: every wave reads all rows of a and, transposed at half
// rate, of b.  Of 64 x 64 a chunk takes 2.1.  A workgroup's start, and the states that it writes, take 4
// to 7 us.
//     B=2, T=2048, 16 heads: outputs 30 us, what segments add 13 (backward 76 and 24)
//     32768 packed tokens, 16 value heads: 190 and 61, the join 10
// The comparisons that follow, and those at weighted_parts, attn_join and segment_chunks, were made
// with one bf16 part of what operand_parts now gives in two, which takes 7 to 12 % less time on
// either side of each.
// Tried and slower: four waves of 32 columns, two workgroups per CU (43 to 48 us for the first shape,
// 41 with eight of 16); loads two chunks ahead (44; backward 111 for 99); the backward pass's three
// passes next to one another in the grid (102 for 97); segments' sums by waves of 32 columns and half
// of the rows (packed 243 for 225).  No faster: c's columns held from the
// outputs' product for the update.
#pragma once
#include <type_traits>

#include "gdn_layer.h"

namespace gdn {

struct AttnGeo {
  int B, T, H, HV, G, N;  // N sequences; G = HV / H
  int chunks;             // chunks per segment
  int nseg;               // segments per sequence (without offsets)
  int slots;              // segments in all, or (packed) an upper bound that counts empty sequences too
  const int64_t* cu;
  bool zero;              // rows of the output behind the last sequence are set to 0
};

// Rows of one operand: token t's values of head `hv / div` at p + t ld + (hv / div) width.
struct AttnRows {
  const void* p;
  int64_t ld;
  int div;
};

// What a pass does with the states.  The caller's are [sequences][HV][..] with element [i][j]
// of a head (row as operand b, column as operand c) at i rs + j cs.  Those of segments are in
// the workspace, [Segment::state][HV] of them, in the order in which lanes hold them (state_place).
enum { kWholeSequence, kSumSegments, kJoined };
struct AttnState {
  const float* start;  // or nullptr: zero
  float* end;          // or nullptr: not written
  int rs, cs;
  float* w;            // what segments add to the state, or (kJoined) their starts
  int mode;
  bool transposed;     // w was written by a pass whose b and c were the other way round
};

// log_decay as the base-2 exponent; a^n for a whole n >= 0 (a = 0: 0^0 = 1).
__device__ __forceinline__ float decay_power(float l2, int n) {
  return n == 0 ? 1.f : __builtin_amdgcn_exp2f((float)n * l2);
}

// The segment of a slot: sequence n, its number i of `count` in the sequence, tokens
// [t0, t0 + len).
//
// Packed sequences have slot floor(cu[n] / L) + n + i for segment i of sequence n (L tokens
// per segment): ceil((y - x) / L) <= floor(y / L) - floor(x / L) + 1 keeps the sequences'
// slots apart, and no table has to be made on the device first; T / L + N slots hold all.
// The search for n compares 64 offsets at a time.
//
// States in the workspace are those of sequences of several segments alone, whose x < y are more
// than L apart: with f = floor(x / L), theirs are f + min(n, f) + i, which are apart as well (such a
// sequence takes f a step further, and so min(n, f)) and below T / L + min(N, T / L), however many
// short sequences there are.
struct Segment {
  int n, i, count, t0, len;
  int state;  // place of the segment's state, where the sequence has several

  __device__ __forceinline__ static int whole(const AttnGeo& g, int n) {
    return (seq_offset(g.cu, n, g.T) / kChunk) / g.chunks;
  }
  __device__ __forceinline__ static int seq_slot(const AttnGeo& g, int n) { return whole(g, n) + n; }
  // the place of a sequence's first state
  __device__ __forceinline__ static int seq_state(const AttnGeo& g, int n) {
    const int f = whole(g, n);
    return f + min(n, f);
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
      state = slot;
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
      const int f = whole(g, n);
      i = slot - (f + n);
      state = f + min(n, f) + i;
    }
    count = (int)((end - start + L - 1) / L);
    t0 = len = 0;
    const int64_t at = start + i * L;
    if (i < 0 || at >= end) return false;
    t0 = (int)at;
    len = (int)min(L, end - at);
    return true;
  }
};

// Block id -> (slot, value head): the G value heads of a (slot, key head) go to one XCD
// (workgroups are dispatched to the 8 XCDs round-robin by id), one after the other, so that
// the query and key rows they share come through one L2.  False for the ids that fill up the
// last group of eight.
__device__ __forceinline__ bool attn_block(const AttnGeo& g, int b, int& slot, int& hv) {
  const int j = b >> 3, unit = j / g.G * 8 + (b & 7);
  slot = unit / g.H;
  hv = (unit - slot * g.H) * g.G + j % g.G;
  return slot < g.slots;
}

// A state of KD x VD lies in the lanes as tiles of 16 x 16: tile kt = 2 kb + j holds, in lane
// (g, m) and element r, row 32 kb + 8 g + 4 j + r and column 16 ct + m, so that the two tiles
// of a block of 32 rows are a fragment whose lane holds eight consecutive rows, which an
// operand's fragment reads from LDS as 16 bytes.
__device__ __forceinline__ int state_row(int kt) { return 32 * (kt >> 1) + 8 * (lane_id() >> 4) + 4 * (kt & 1); }
// A lane's four elements of a tile in the workspace.
__device__ __forceinline__ int state_place(int kt, int ct, int cts) { return ((kt * cts + ct) * 64 + lane_id()) * 4; }
// The same of a state that was written the other way round, with KD columns: its element [col][row]
// for a lane's row (state_row(kt) + r) and column (c + m, c a multiple of 16), as a lane's part
// (in bytes) and a uniform one.
template <int KD> __device__ __forceinline__ uint32_t state_lane_transposed() {
  const int g = lane_id() >> 4, m = lane_id() & 15;
  return 4 * ((((m >> 2 & 1) * (KD / 16) + (g >> 1)) * 64 + (m >> 3) * 16 + 8 * (g & 1)) * 4 + (m & 3));
}
template <int KD> __device__ __forceinline__ int state_transposed(int kt, int r, int c) {
  return ((c / 32 * 2 * (KD / 16) + (kt >> 1) * 2) * 64 + c / 8 % 4 * 16 + 4 * (kt & 1) + r) * 4;
}

// A wave per 16 columns of the state.
constexpr int attn_threads(int vd) { return 4 * vd; }

// A chunk's rows in LDS: 64 rows of D elements in 16-byte pieces, whose places within a row are
// exchanged (piece c of row r is at c ^ turn(r)) so that neither reads of one piece of 16 rows
// nor the transposed reads below (two or four pieces of four rows) meet a bank twice.
template <typename E, int D, int THREADS> struct AttnTile {
  static constexpr int VECS = D * (int)sizeof(E) / 16;     // pieces per row
  static constexpr int STEP = THREADS / VECS;              // rows between a thread's pieces
  static constexpr int PER = kChunk / STEP;                // pieces per thread
  E x[kChunk * D];
  __device__ __forceinline__ static int turn(int row) {
    if (sizeof(E) == 4) return (row >> 3 & 3) << 2 | (row & 3);  // (its columns are read element by element)
    return VECS == 8 ? (row >> 1 & 1) << 2 | (row >> 2 & 3) : (row & 3) << 2 | (row >> 2 & 3);
  }
  // the elements from [row][col] on, to the end of their piece
  __device__ __forceinline__ E* at(int row, int col) {
    constexpr int N = 16 / (int)sizeof(E);
    return x + row * D + ((col / N) ^ turn(row)) * N + col % N;
  }
  __device__ __forceinline__ const E* at(int row, int col) const { return const_cast<AttnTile*>(this)->at(row, col); }
  struct Rows {
    u32x4 r[PER];
  };
  // The rows of a chunk, as loaded: rows from `len` on are the last one's again (whatever is
  // formed from them is not used), so that no row of another sequence is read.  `base` is
  // uniform, `ld` in bytes (offsets within a chunk are 32 bits).
  __device__ __forceinline__ static void fetch(Rows& f, const void* base, uint32_t ld, int len) {
    const int row = threadIdx.x / VECS, col = threadIdx.x % VECS * 16;
    Global<const char> p = (Global<const char>)base;
    if (len == kChunk) {
      const uint32_t off = lane_offset(row * ld + col);
#pragma unroll
      for (int i = 0; i < PER; ++i) f.r[i] = *(Global<const u32x4>)(p + (uint64_t)(i * STEP) * ld + off);
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        f.r[i] = *(Global<const u32x4>)(p + lane_offset(min(row + i * STEP, len - 1) * ld + col));
    }
  }
  __device__ __forceinline__ void place(const Rows& f) {
    const int row = threadIdx.x / VECS, col = threadIdx.x % VECS * (16 / (int)sizeof(E));
#pragma unroll
    for (int i = 0; i < PER; ++i) *reinterpret_cast<u32x4*>(at(row + i * STEP, col)) = f.r[i];
  }
  // k32 fragment of a row, whose lane holds eight consecutive elements: 32 kb + 8 g on
  __device__ __forceinline__ Frag<E> of_row(int row, int kb) const {
    const int c = 32 * kb + 8 * (lane_id() >> 4);
    if constexpr (sizeof(E) == 2) return {*reinterpret_cast<const bf16x8*>(at(row, c))};
    else return {*reinterpret_cast<const f32x4*>(at(row, c)), *reinterpret_cast<const f32x4*>(at(row, c + 4))};
  }
  // k32 fragment of rows s0 .. s0 + 31 in the same order, the lane's column c0 + APART (m / 4) +
  // m % 4: ds_read_b64_tr_b16 gives lane m of a group of 16 element m % 4 of what its lanes
  // 4 i + m / 4 (i = 0..3) address
  template <int APART> __device__ __forceinline__ Frag<E> of_columns(int s0, int c0) const {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    if constexpr (sizeof(E) == 2) {
      const int g = lane_id() >> 4, m = lane_id() & 15;
      const int row = s0 + 8 * g + (m >> 2), col = c0 + APART * (m & 3);
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at(row, col));
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at(row + 4, col));
      const auto both = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
      return {__builtin_bit_cast(bf16x8, both)};
    } else {
      int lane = lane_id();
      // where the tiles are of two widths, addresses kept from chunk to chunk need more registers
      // than there are: formed here each time
      if constexpr (D * 4 != THREADS) asm volatile("" : "+v"(lane));
      const int row = s0 + 8 * (lane >> 4), col = c0 + APART * ((lane & 15) >> 2) + (lane & 3);
      Frag<E> f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f.lo[i] = *at(row + i, col);
        f.hi[i] = *at(row + 4 + i, col);
      }
      return f;
    }
  }
};

// c_s w_s as a sum of NP fragments.  A bf16 operand of the state's update is c_s (8 bits)
// times an fp32 weight: one bf16 would leave 2^-9 of every state, which fp32 states must not
// have; two parts leave 2^-17 (as operand_parts does of a state that only ever meets bf16 rows),
// three 2^-25.  They are
// rounded two elements at a time: the vector unit is half busy here (packed, as above: 225 us one at a
// time, 219 so).
template <int NP>
__device__ __forceinline__ void weighted_parts(const Frag<bf16>& c, const float (&w)[8], Frag<bf16> (&out)[NP]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const u32x4 x = __builtin_bit_cast(u32x4, c.x);
  u32x4 part[NP];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // two at a time, which one instruction rounds
    float lo = __uint_as_float(x[i] << 16) * w[2 * i], hi = __uint_as_float(x[i] & 0xffff0000u) * w[2 * i + 1];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      part[p][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
      lo -= __uint_as_float(part[p][i] << 16);
      hi -= __uint_as_float(part[p][i] & 0xffff0000u);
    }
  }
#pragma unroll
  for (int p = 0; p < NP; ++p) out[p].x = __builtin_bit_cast(bf16x8, part[p]);
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

// What fp32 values become as operands (a chunk's weighted products, and the state where it meets
// rows), as a sum of NP fragments.  Of bf16 there are two, which leave 2^-17, so that a result's own
// rounding is the one that it shows: with one part results were off by 0.0023 where that rounding
// alone is 0.0017.  Times with one and with two (us): B=2, T=2048, 16 heads of 128 38 and 40, its
// backward pass 87 and 96; 32768 packed tokens, 16 value heads 220 and 245 (239 since the join passes
// over single segments).
template <typename E> constexpr int attn_parts() { return sizeof(E) == 2 ? 2 : 1; }
template <typename E, int NP> __device__ __forceinline__ void operand_parts(f32x4 x, Quad<E> (&out)[NP]) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    out[p] = make_quad<E>(x);
    if (p + 1 < NP) x -= quad_f32(out[p]);
  }
}
// The same of two tiles of a state, which are a fragment's halves.
template <typename E, int NP> __device__ __forceinline__ void state_parts(f32x4 d0, f32x4 d1, Frag<E> (&out)[NP]) {
  Quad<E> lo[NP], hi[NP];
  operand_parts(d0, lo);
  operand_parts(d1, hi);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    if constexpr (sizeof(E) == 2) out[p] = {__builtin_shufflevector(lo[p].x, hi[p].x, 0, 1, 2, 3, 4, 5, 6, 7)};
    else out[p] = {lo[p].x, hi[p].x};
  }
}

// Rows behind the last sequence, of head hv's columns of the output, set to 0: shared out over
// the slots.
template <typename OT, int D, int THREADS>
__device__ __forceinline__ void attn_zero_rest(const AttnGeo& g, int hv, int slot, OT* out) {
  constexpr int PER_ROW = D * (int)sizeof(OT) / 16, ROWS = THREADS / PER_ROW;
  const int sub = threadIdx.x / PER_ROW, col = threadIdx.x % PER_ROW;
  for (int64_t t = seq_offset(g.cu, g.N, g.T) + (int64_t)slot * ROWS + sub; t < g.T; t += (int64_t)g.slots * ROWS)
    *reinterpret_cast<u32x4*>(out + (t * g.HV + hv) * D + col * (16 / (int)sizeof(OT))) = u32x4{0, 0, 0, 0};
}

// The phases of a chunk stay apart: mixed by the scheduler they need more registers than there are.
#define ATTN_PHASE __builtin_amdgcn_sched_barrier(0)

// Within a phase (bf16): `ahead` reads of LDS, then per step `mfma` products and `reads` more, so
// that products find their operands there.  Left alone the scheduler saves registers and waits
// for every read.
template <typename E, int AHEAD, int STEPS, int MFMA, int READS> __device__ __forceinline__ void attn_interleave() {
  if constexpr (sizeof(E) == 2) {
    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, MFMA, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
    }
  }
}

// H <- a H + b^T (c weighted), H the state's tiles: NP parts of the weighted operand.
template <int NP, typename E, int KT, typename B, typename C>
__device__ __forceinline__ void attn_update(f32x4 (&H)[KT], const B& b, const C& c, int col0, const float* weight) {
  const int g = lane_id() >> 4;
#pragma unroll
  for (int sb = 0; sb < kChunk / 32; ++sb) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const f32x4 q = *reinterpret_cast<const f32x4*>(weight + 32 * sb + 8 * g + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[i + j] = q[j];
    }
    Frag<E> vw[NP];
    weighted_parts<NP>(c.template of_columns<4>(32 * sb, col0), w, vw);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const Frag<E> k = b.template of_columns<8>(32 * sb, 32 * (kt >> 1) + 4 * (kt & 1));
#pragma unroll
      for (int p = 0; p < NP; ++p) mma_k32(H[kt], k, vw[p]);
    }
    attn_interleave<E, 4 + 6, KT, NP, 2>();
  }
}

// One pass over a segment of one value head; a wave per 16 columns of the state and of the
// output.  KD, VD: widths of operands a and b, and of c.  OUT: rows of the output are formed
// (else what the segment adds to the state).
//
// Per chunk: rows from registers (loaded a chunk ahead) to LDS; the weighted products a.b, tiles of
// 16 x 16 shared out over the waves, to LDS as the next product's operand; the state's part and
// the products' part of the output, whose rows go through LDS to be stored whole; the state's
// update.  Powers of the decay are formed by one lane each and read from LDS: of the products
// (`gap`) once, the weights of a chunk's update and of the state in each of its rows per chunk.
template <typename E, typename OT, int KD, int VD, int THREADS, bool OUT> struct AttnLds {
  AttnTile<E, KD, THREADS> b;
  AttnTile<E, VD, THREADS> c;
  float update[kChunk];
};
template <typename E, typename OT, int KD, int VD, int THREADS> struct AttnLds<E, OT, KD, VD, THREADS, true> {
  AttnTile<E, KD, THREADS> b;
  AttnTile<E, VD, THREADS> c;
  AttnTile<E, KD, THREADS> a;
  AttnTile<OT, VD, THREADS> o;
  AttnTile<E, kChunk, THREADS> p[attn_parts<E>()];
  float update[kChunk], inter[kChunk], gap[2 * kChunk];  // gap: 0 for rows that are not seen
};

struct AttnPass {
  AttnRows a, b, c;
  AttnState st;
  void* out;
  float s_intra, s_inter, s_update;  // what products a.b, the state's part and its update are scaled by
};

template <typename E, typename OT, int KD, int VD, int THREADS, bool REV, bool OUT>
__device__ __forceinline__ void attn_pass(const AttnGeo& geo, int block, const AttnPass& x,
                                          const float* __restrict__ log_decay, char* smem) {
  const AttnRows &ar = x.a, &br = x.b, &cr = x.c;
  const AttnState& st = x.st;
  OT* out = static_cast<OT*>(x.out);
  const float s_intra = x.s_intra, s_inter = x.s_inter, s_update = x.s_update;
  constexpr int KT = KD / 16, TT = kChunk / 16, WAVES = VD / 16, NP = attn_parts<E>();
  using Lds = AttnLds<E, OT, KD, VD, THREADS, OUT>;
  using KTile = AttnTile<E, KD, THREADS>;
  using VTile = AttnTile<E, VD, THREADS>;
  using OTile = AttnTile<OT, VD, THREADS>;
  Lds& L = *reinterpret_cast<Lds*>(smem);

  int hv, slot;
  if (!attn_block(geo, block, slot, hv)) return;
  if constexpr (OUT) {
    if (geo.cu && geo.zero) attn_zero_rest<OT, VD, THREADS>(geo, hv, slot, out);
  }
  Segment seg;
  const bool tokens = seg.find(geo, slot);
  // in the order of the pass: segments done before this one, and whether it is the last
  const int before = REV ? seg.count - 1 - seg.i : seg.i;
  const bool last = before >= seg.count - 1;
  if constexpr (OUT) {
    // (a sequence without tokens passes its state on)
    if (!tokens && !(st.end && seg.i == 0)) return;
  } else {
    if (!tokens || last) return;  // nobody asks what the last segment adds
  }
  const int nch = (seg.len + kChunk - 1) / kChunk;
  const int lane = lane_id(), g = lane >> 4, m = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // (waves beyond the columns, where another pass of the launch has more, load and store)
  const bool owner = THREADS == attn_threads(VD) || wave < WAVES;
  const int col0 = owner ? 16 * wave : 0;
  const float l2 = log_decay[hv] * kLog2e;

  const E* ap = static_cast<const E*>(ar.p) + (int64_t)seg.t0 * ar.ld + (hv / ar.div) * KD;
  const E* bp = static_cast<const E*>(br.p) + (int64_t)seg.t0 * br.ld + (hv / br.div) * KD;
  const E* cp = static_cast<const E*>(cr.p) + (int64_t)seg.t0 * cr.ld + (hv / cr.div) * VD;

  struct Rows {
    typename KTile::Rows a, b;
    typename VTile::Rows c;
  };
  Rows ahead;  // the next chunk's
  auto fetch_ab = [&](int it) {
    const int c = REV ? nch - 1 - it : it, n = min(kChunk, seg.len - c * kChunk);
    if constexpr (OUT) KTile::fetch(ahead.a, ap + (int64_t)c * kChunk * ar.ld, (uint32_t)(ar.ld * sizeof(E)), n);
    KTile::fetch(ahead.b, bp + (int64_t)c * kChunk * br.ld, (uint32_t)(br.ld * sizeof(E)), n);
  };
  auto fetch_c = [&](int it) {
    const int c = REV ? nch - 1 - it : it, n = min(kChunk, seg.len - c * kChunk);
    VTile::fetch(ahead.c, cp + (int64_t)c * kChunk * cr.ld, (uint32_t)(cr.ld * sizeof(E)), n);
  };
  if (nch > 0) {
    fetch_ab(0);
    fetch_c(0);
  }

  f32x4 H[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) H[kt] = f32x4{0.f, 0.f, 0.f, 0.f};
  if constexpr (OUT) {
    const bool joined = st.mode == kJoined && seg.count > 1;
    if (st.start && !joined) {
      const float* s = st.start + ((int64_t)seg.n * geo.HV + hv) * (KD * VD) + (col0 + m) * st.cs;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r) H[kt][r] = s[(state_row(kt) + r) * st.rs];
    }
    // H <- a^len H + what the segment adds, over the segments done before, AHEAD of them loaded
    // at a time; or the start itself
    const int sums = joined ? 1 : st.mode == kSumSegments ? before : 0;
    constexpr int AHEAD = sizeof(E) == 2 ? 4 : 1;
    for (int j0 = 0; j0 < sums; j0 += AHEAD) {
      f32x4 e[AHEAD][KT];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const int k = min(j0 + j, sums - 1);
        const int at = joined ? seg.state : REV ? seg.state + before - k : seg.state - before + k;
        const float* w = st.w + ((int64_t)at * geo.HV + hv) * (KD * VD);
        if (!st.transposed) {
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) e[j][kt] = *reinterpret_cast<const f32x4*>(w + state_place(kt, col0 / 16, VD / 16));
        } else {
          const uint32_t off = lane_offset(state_lane_transposed<KD>());
#pragma unroll
          for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              e[j][kt][r] = *(Global<const float>)((Global<const char>)(w + state_transposed<KD>(kt, r, col0)) + off);
        }
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (j0 + j >= sums) break;
        const int64_t len = (int64_t)geo.chunks * kChunk;
        // (backwards, the sequence's last segment may be short; forwards those before are whole)
        int64_t n = len;
        if (REV && j0 + j == 0) {
          const int64_t end = geo.cu ? seq_offset(geo.cu, seg.n + 1, geo.T) : (int64_t)(seg.n + 1) * geo.T;
          n = end - (seg.t0 - (int64_t)seg.i * len) - (int64_t)(seg.count - 1) * len;
        }
        // (a start replaces what is there: nothing, times 0)
        const float a = joined ? 0.f : decay_power(l2, (int)n);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) H[kt] = H[kt] * a + e[j][kt];
      }
    }
    if (wave < 2) L.gap[threadIdx.x] = wave == 0 ? 0.f : s_intra * decay_power(l2, lane);
  }

  // the output's rows of chunk `it`, from LDS
  auto store = [&](int it) {
    if constexpr (OUT) {
      const int c = REV ? nch - 1 - it : it, n = min(kChunk, seg.len - c * kChunk);
      const uint32_t row = (uint32_t)(geo.HV * VD * sizeof(OT));
      Global<char> o = (Global<char>)(out + ((int64_t)(seg.t0 + c * kChunk) * geo.HV + hv) * VD);
      const int r0 = threadIdx.x / OTile::VECS, col = threadIdx.x % OTile::VECS * 16;
      const uint32_t off = lane_offset(r0 * row + col);
#pragma unroll
      for (int i = 0; i < OTile::PER; ++i) {
        const int r = r0 + i * OTile::STEP;
        const u32x4 v = *reinterpret_cast<const u32x4*>(L.o.at(r, col / (int)sizeof(OT)));
        if (r < n) *(Global<u32x4>)(o + (uint64_t)(i * OTile::STEP) * row + off) = v;
      }
    }
  };

  auto chunk = [&](int it, auto more) {
    const int c = REV ? nch - 1 - it : it;
    const int n = min(kChunk, seg.len - c * kChunk);
    if (it) __syncthreads();  // the last chunk's reads are done, its rows of the output written
    if constexpr (OUT) L.a.place(ahead.a);
    L.b.place(ahead.b);
    L.c.place(ahead.c);
    if (wave == 0) L.update[lane] = lane < n ? s_update * decay_power(l2, REV ? lane + 1 : n - 1 - lane) : 0.f;
    if constexpr (OUT) {
      if (wave == 1) L.inter[lane] = lane < n ? s_inter * decay_power(l2, REV ? n - 1 - lane : lane + 1) : 0.f;
    }
    __syncthreads();
    if constexpr (decltype(more)::value) fetch_ab(it + 1);
    if constexpr (!OUT && decltype(more)::value) fetch_c(it + 1);
    if (it) store(it - 1);

    f32x4 acc[TT];
    if constexpr (OUT && decltype(more)::value) fetch_c(it + 1);
    if constexpr (OUT) {
      // the weighted products of a tile of rows of a with those rows of b that they see, two
      // tiles of b at a time; two waves share a tile of a where there are eight (all of them, also
      // those beyond the columns)
      {
        constexpr int SHARE = THREADS / 64 / TT;
        const int tt = wave / SHARE, t = 16 * tt + m;
        Frag<E> fa[KD / 32];
#pragma unroll
        for (int kb = 0; kb < KD / 32; ++kb) fa[kb] = L.a.of_row(t, kb);
#pragma unroll
        for (int i = 0; i < 2 / SHARE; ++i) {
          const int sb = SHARE == 2 ? wave % 2 : i;
          // (blocks of 32 rows of which none is seen are not read below)
          if (REV ? 2 * sb + 1 < tt : 2 * sb > tt) continue;
          f32x4 p[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
          float w[2][4];
          const int apart = 32 * sb + 4 * g - t;  // s - t at j = r = 0
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) w[j][r] = L.gap[kChunk + (REV ? 1 : -1) * (apart + 16 * j + r)];
#pragma unroll
          for (int kb = 0; kb < KD / 32; ++kb)
#pragma unroll
            for (int j = 0; j < 2; ++j) mma_k32(p[j], L.b.of_row(32 * sb + 16 * j + m, kb), fa[kb]);
          attn_interleave<E, 16, KD / 32, 2, 0>();
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              asm("" : "+v"(w[j][r]));  // (read above, and not behind a branch here)
              // (a select, so that nothing of a masked product stays)
              const int gap = apart + 16 * j + r;
              p[j][r] = (REV ? gap >= 0 && 32 * sb + 4 * g + 16 * j + r < n : gap <= 0) ? p[j][r] * w[j][r] : 0.f;
            }
            Quad<E> part[NP];
            operand_parts(p[j], part);
#pragma unroll
            for (int i = 0; i < NP; ++i) *reinterpret_cast<Quad<E>*>(L.p[i].at(t, 32 * sb + 16 * j + 4 * g)) = part[i];
          }
          ATTN_PHASE;
        }
      }
    }
    if constexpr (OUT) if (owner) {
      // the state's part: O^T = H^T a^T, then weighted by row
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) acc[tt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KD / 32; ++kb) {
        Frag<E> h[NP];
        state_parts(H[2 * kb], H[2 * kb + 1], h);
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          const Frag<E> q = L.a.of_row(16 * tt + m, kb);
#pragma unroll
          for (int i = 0; i < NP; ++i) mma_k32(acc[tt], h[i], q);
        }
      }
      attn_interleave<E, 6, (KD / 32) * TT * NP, 1, 1>();
      ATTN_PHASE;
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) acc[tt] *= L.inter[16 * tt + m];
    }
    if constexpr (OUT) __syncthreads();  // the weighted products are there
    if constexpr (OUT) if (owner) {
#pragma unroll
      for (int sb = 0; sb < kChunk / 32; ++sb) {
        const Frag<E> v = L.c.template of_columns<4>(32 * sb, col0);
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          if (REV ? 2 * sb + 1 < tt : 2 * sb > tt) continue;
#pragma unroll
          for (int i = 0; i < NP; ++i) mma_k32(acc[tt], v, L.p[i].of_row(16 * tt + m, sb));
        }
      }
      attn_interleave<E, 8, 12, 1, 1>();
#pragma unroll
      for (int tt = 0; tt < TT; ++tt)
        *reinterpret_cast<Quad<OT>*>(L.o.at(16 * tt + m, col0 + 4 * g)) = make_quad<OT>(acc[tt]);
    }
    ATTN_PHASE;
    const bool end = OUT && last && st.end;
    if (owner && (!OUT || end || it + 1 < nch)) {
      const float a = decay_power(l2, n);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) H[kt] *= a;
      // three parts where the states go out as fp32, two where they only meet bf16 operands
      if constexpr (sizeof(E) == 4) attn_update<1, E>(H, L.b, L.c, col0, L.update);
      else if (!OUT || end) attn_update<3, E>(H, L.b, L.c, col0, L.update);
      else attn_update<2, E>(H, L.b, L.c, col0, L.update);
    }
  };
  // (the loop's loads are unconditional: the compiler then knows how many are under way)
  int it = 0;
  for (; it + 1 < nch; ++it) chunk(it, std::true_type{});
  if (nch > 0) chunk(it, std::false_type{});

  if constexpr (OUT) {
    if (nch > 0) {
      __syncthreads();
      store(nch - 1);
    }
    if (last && st.end && owner) {
      float* s = st.end + ((int64_t)seg.n * geo.HV + hv) * (KD * VD) + (col0 + m) * st.cs;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r) s[(state_row(kt) + r) * st.rs] = H[kt][r];
    }
  } else if (owner) {
    float* w = st.w + ((int64_t)seg.state * geo.HV + hv) * (KD * VD);
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) *reinterpret_cast<f32x4*>(w + state_place(kt, col0 / 16, VD / 16)) = H[kt];
  }
}

template <typename E, int VD, bool OUT> constexpr int attn_waves() {  // per SIMD, that registers are left for
  return sizeof(E) == 4 || (VD == 64 && OUT) ? 1 : 2;
}

template <typename E, typename OT, int KD, int VD, bool REV, bool OUT>
__global__ __launch_bounds__(attn_threads(VD), (attn_waves<E, VD, OUT>())) void gdn_linattn_kernel(
    AttnGeo geo, AttnPass x, const float* __restrict__ log_decay) {
  __shared__ __attribute__((aligned(16))) char smem[sizeof(AttnLds<E, OT, KD, VD, attn_threads(VD), OUT>)];
  attn_pass<E, OT, KD, VD, attn_threads(VD), REV, OUT>(geo, blockIdx.x, x, log_decay, smem);
}

// The backward pass's passes of one kind in one launch, `blocks` workgroups each: what segments
// add to H^T and dH (two passes), or dq, dk and dv.  OT: the type of dq and dk.  Workgroups have
// the threads that the wider of keys and values takes.
template <typename E, typename OT, int K, int V, bool OUT>
__global__ __launch_bounds__(attn_threads(K > V ? K : V), (attn_waves<E, (K > V ? K : V), OUT>())) void gdn_linattn_bwd_kernel(
    AttnGeo geo, AttnPass q, AttnPass k, AttnPass v, const float* __restrict__ log_decay, int blocks) {
  constexpr int THREADS = attn_threads(K > V ? K : V);
  constexpr size_t QK = sizeof(AttnLds<E, OT, V, K, THREADS, OUT>), VV = sizeof(AttnLds<E, E, K, V, THREADS, OUT>);
  __shared__ __attribute__((aligned(16))) char smem[QK > VV ? QK : VV];
  const int role = blockIdx.x / blocks, block = blockIdx.x - role * blocks;
  if (role == 0) attn_pass<E, OT, V, K, THREADS, false, OUT>(geo, block, q, log_decay, smem);
  else if (OUT && role == 1) attn_pass<E, OT, V, K, THREADS, true, OUT>(geo, block, k, log_decay, smem);
  else attn_pass<E, E, K, V, THREADS, true, OUT>(geo, block, v, log_decay, smem);
}

// The starts of the segments of sequences that have several: per sequence, head and four elements
// of the state, in the segments' order (REV: from the last),  w[segment] <- cur;  cur <- a^len cur +
// (what w[segment] held),  from `start` (or 0).  Loads run kAttnAhead segments ahead (backward, 5003
// packed tokens, 8 value heads of 128 x 64 in segments of two chunks: 8 ahead 76.8 us, 16 74.9, 32
// 76.1).  Bound by the states' bytes: 75 MB read and written in 10 us at 32768 tokens, 16 heads.
// Packed sequences of one segment are passed over: their states would go to the workspace and back
// (1000 of 64 tokens, 16 heads of 128 bf16: 1272 and 887 us a call, backward 3471 and 2673).
constexpr int kAttnAhead = 16;

template <int KD, int VD, bool REV>
__device__ __forceinline__ void attn_join(const AttnGeo& geo, const float* __restrict__ log_decay, const AttnState& st) {
  constexpr int KV = KD * VD, PER = KV / 4 / 256;  // workgroups per head
  const float* start = st.start;
  float* w = st.w;
  const int rs = st.rs, cs = st.cs;
  const int part = blockIdx.x % PER, unit = blockIdx.x / PER;
  const int hv = unit % geo.HV, n = unit / geo.HV;
  const int tile = part * 4 + (threadIdx.x >> 6), at = (tile * 64 + lane_id()) * 4;
  const float l2 = log_decay[hv] * kLog2e;
  const int64_t L = (int64_t)geo.chunks * kChunk;
  int64_t t0, t1;
  int first;
  if (geo.cu) {
    t0 = seq_offset(geo.cu, n, geo.T);
    t1 = max((int64_t)seq_offset(geo.cu, n + 1, geo.T), t0);
    if (t1 - t0 <= L) return;  // (its one segment starts from `start` itself)
    first = Segment::seq_state(geo, n);
  } else {
    t0 = 0;
    t1 = geo.T;
    first = n * geo.nseg;
  }
  const int count = (int)((t1 - t0 + L - 1) / L);
  f32x4 cur = {0.f, 0.f, 0.f, 0.f};
  if (start) {
    const float* s = start + ((int64_t)n * geo.HV + hv) * KV + (tile % (VD / 16) * 16 + (lane_id() & 15)) * cs;
    const int row = state_row(tile / (VD / 16));
#pragma unroll
    for (int r = 0; r < 4; ++r) cur[r] = s[(row + r) * rs];
  }
  auto place = [&](int i) {
    return reinterpret_cast<f32x4*>(w + ((int64_t)(first + (REV ? count - 1 - i : i)) * geo.HV + hv) * KV + at);
  };
  const float whole = decay_power(l2, (int)min(L, t1 - t0));
  const float tail = decay_power(l2, (int)(t1 - t0 - (int64_t)(count - 1) * L));
  for (int i = 0; i < count; i += kAttnAhead) {
    f32x4 add[kAttnAhead];
#pragma unroll
    for (int j = 0; j < kAttnAhead; ++j)
      if (i + j + 1 < count) add[j] = *place(i + j);  // (the last segment's is not formed)
#pragma unroll
    for (int j = 0; j < kAttnAhead; ++j)
      if (i + j < count) {
        *place(i + j) = cur;
        if (i + j + 1 < count) cur = cur * (REV && i + j == 0 ? tail : whole) + add[j];
      }
  }
}

template <int K, int V>
__global__ __launch_bounds__(256) void gdn_linattn_join_kernel(AttnGeo geo, AttnState h, const float* __restrict__ log_decay) {
  attn_join<K, V, false>(geo, log_decay, h);
}
// H^T and (second row of the grid) dH of the backward pass.
template <int K, int V>
__global__ __launch_bounds__(256) void gdn_linattn_bwd_join_kernel(AttnGeo geo, AttnState ht, AttnState dh,
                                                                   const float* __restrict__ log_decay) {
  if (blockIdx.y == 0) attn_join<V, K, false>(geo, log_decay, ht);
  else attn_join<K, V, true>(geo, log_decay, dh);
}

// States without a token: start (or 0) passed to end.
static __global__ __launch_bounds__(256) void gdn_linattn_copy_kernel(const float* __restrict__ start,
                                                                      float* __restrict__ end, int64_t quads) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < quads; i += (int64_t)gridDim.x * 256)
    reinterpret_cast<f32x4*>(end)[i] = start ? reinterpret_cast<const f32x4*>(start)[i] : f32x4{0.f, 0.f, 0.f, 0.f};
}

// Gradients of shared key heads: out[row][h][k] = sum over the G value heads of part[row][h G + j][k],
// in their order; of dq, and (second row of the grid) of dk.
template <typename E>
__global__ __launch_bounds__(256) void gdn_linattn_sum_kernel(const float* __restrict__ partq, const float* __restrict__ partk,
                                                              E* __restrict__ dq, E* __restrict__ dk, int64_t quads,
                                                              int G, int KQ) {
  const f32x4* part = reinterpret_cast<const f32x4*>(blockIdx.y ? partk : partq);
  E* out = blockIdx.y ? dk : dq;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < quads; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / KQ;
    const f32x4* p = part + row * G * KQ + (i - row * KQ);
    f32x4 s = p[0];
    for (int j = 1; j < G; ++j) s += p[(int64_t)j * KQ];
    *reinterpret_cast<Quad<E>*>(out + 4 * i) = make_quad<E>(s);
  }
}

// A few tokens of every sequence, in order, the state in registers: per workgroup one
// (sequence, value head, VB columns), a lane four columns of every 256/(VB/4)-th row.  Bound by
// the state, which is read and written once: 64 sequences, 16 heads of 128 bf16, 135 MB in 21.7 us
// (6.2 TB/s, part of it from the caches); VB = 32 21.0, 64 and 128 22.0.
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
