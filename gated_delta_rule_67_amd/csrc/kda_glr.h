// The gated linear recurrence: arguments (validated by the C ABI), the gate's arithmetic and how its
// kernels share work, for the forward, backward and one-token kernels.
#pragma once

#include <type_traits>

#include "kda_rows.h"
#include "kda_sequence.h"

namespace kda {

struct GlrArgs {
  Source x, r, in;      // input, decay gate's input, input gate's input (p null: no input gate)
  const float* A_log;   // [D]
  const float* dt_bias; // [D] or null
  const float* init;    // [N, D] or null
  Sequences seqs;
  int N, T, D;
  float* states;        // [ceil(T / kGlrBlock), D]: the state in front of every block; out, in (backward), or null
  // forward
  float* final;         // [N, D] or null
  void* y;              // null: only states are wanted
  int zero_rest;
  // backward
  Source dy;
  const float* dfinal;  // [N, D] or null
  void *dx, *dr, *din;  // din null without an input gate
  float* dinit;         // [N, D] or null
  float* part;          // partial sums [tiles][2][D]: dA_log, ddt_bias
  float *dA_log, *ddt_bias;  // or null
  // step
  float* pool;
  const int* slots;
  int nslots, B;
  int normalise;
  bool bf, packed;
};

constexpr int kGlrBlock = 64;  // tokens between kept states

size_t glr_fwd_workspace_bytes(int T, int D);
size_t glr_bwd_workspace_bytes(int T, int D, bool kept_states);
hipError_t launch_glr_fwd(GlrArgs a, void* workspace, hipStream_t stream);
hipError_t launch_glr_bwd(GlrArgs a, void* workspace, hipStream_t stream);
hipError_t launch_glr_step(const GlrArgs& a, hipStream_t stream);

namespace glr {

// ---- Gates. Per channel: -exp(A_log) (an exp(A_log) above 2e38 counts as that, so that products with
// it and a constant are finite), and the bias.
struct Channel {
  float neg_rate, bias;
};
__device__ __forceinline__ Channel channel(float A_log, float dt_bias) {
  const float rate = fast_exp2(A_log * kLog2e);
  return {-(rate > 2.0e38f ? 2.0e38f : rate), dt_bias};
}
__device__ __forceinline__ Channel channel(const GlrArgs& a, int c) {
  return channel(a.A_log[c], a.dt_bias ? a.dt_bias[c] : 0.f);
}

// log2 of the decay, g2 <= 0, for the gate's input; e = 2^-|z2| and u = fl(1 + e) are left for the
// softplus' slope. z = x + bias is rounded before it is scaled: x log2 e + (bias log2 e) in one instruction
// carries the second product's rounding, which stays where a large bias cancels (softplus off by 6e-6 at 100;
// the instruction more costs the backward pass 2 of 267 us, the forward pass nothing). With z2 = z log2 e,
// softplus(z) log2 e = max(z2, 0) + log2(1 + e), and the rounding d of 1 + e is taken back at first order,
// log2(1 + e) = log2(u) - d log2 e (the factor 1 / u of that term is left out: it is off by e d at most, under
// 2^-24 of the result), so that the value keeps its relative accuracy however small e is.
__device__ __forceinline__ float decay_log2(float x, const Channel& ch, float& z2, float& e, float& u) {
  z2 = (x + ch.bias) * kLog2e;
  e = fast_exp2(-fabsf(z2));
  u = 1.f + e;
  const float d = (u - 1.f) - e;
  return ch.neg_rate * fmaf(d, -kLog2e, fmaxf(z2, 0.f) + __builtin_amdgcn_logf(u));
}
__device__ __forceinline__ float decay_log2(float x, const Channel& ch) {
  float z2, e, u;
  return decay_log2(x, ch, z2, e, u);
}
// The same held above -1e30, so that products with it stay finite (the decay is 0 long before), and the
// slope of the softplus, logistic(z).
__device__ __forceinline__ float decay_log2(float x, const Channel& ch, float& slope) {
  float z2, e, u;
  const float g2 = decay_log2(x, ch, z2, e, u), r = __builtin_amdgcn_rcpf(u);
  slope = z2 >= 0.f ? r : e * r;
  return g2 < -1e30f ? -1e30f : g2;
}

// logistic(z), the input gate.
__device__ __forceinline__ float sigmoid_fast(float z) {
  return __builtin_amdgcn_rcpf(1.f + fast_exp2(-z * kLog2e));
}

// sqrt(1 - a^2) for a = 2^g2. Near a = 1 the difference would cancel: there 1 - e^-v, v = -2 g2 ln 2, by
// its series in g2 (relative error v^5 / 720 < 5e-8 at v = 1/8); elsewhere from a, whose last bit costs
// 1e-6 at most.
__device__ __forceinline__ float input_weight_squared(float a, float g2) {
  constexpr float k = -2.f * kLn2;
  constexpr float c1 = k, c2 = -k * k / 2, c3 = k * k * k / 6, c4 = -k * k * k * k / 24, c5 = k * k * k * k * k / 120;
  const float p = g2 * fmaf(g2, fmaf(g2, fmaf(g2, fmaf(g2, c5, c4), c3), c2), c1);
  return g2 > -0.125f / (2.f * kLn2) ? p : fmaf(-a, a, 1.f);
}
__device__ __forceinline__ float input_weight(float a, float g2) {
  return __builtin_amdgcn_sqrtf(input_weight_squared(a, g2));
}
// The same and its reciprocal, which is held below 2^63: it is multiplied by the softplus' slope, which is as
// small as the weight's square, so that a weight of 0 has no part in a gradient.
__device__ __forceinline__ float input_weight(float a, float g2, float& inv) {
  const float v = input_weight_squared(a, g2);
  inv = __builtin_amdgcn_rsqf(v < 0x1p-126f ? 0x1p-126f : v);
  return v * inv;
}

// ---- Work. A workgroup's tile is kWaves consecutive spans of tokens (one a wave) by 64 VEC channels
// (VEC a lane). A tile's effect on the state is h -> A h + B per channel; tiles of one column follow
// each other along the tokens (backward: against them), `q` counting from the first.
//
// The token axis is scanned in one pass, every tensor read once: a tile leaves (A, B) for the tiles
// behind it as soon as it has them, the last tile of every kGroup leaves the state behind it, and a
// tile gathers the state in front of it from the state behind the previous group and the (A, B) of its
// own group's tiles in front of it, always folded in the same order: results do not depend on timing.
// Workgroups take their tiles from a counter and work on them one after the other. A tile waits only for
// tiles of its column that come before it in the counter's order, so the first one that is not finished
// never waits for one that is not: every wait ends, however many workgroups run at a time.
//
// A word that is not there yet is all ones, which no value that is stored has (NaN is stored as
// 0x7fc00000 where it could be mistaken): value and presence arrive together, in one relaxed atomic
// access of the whole device (the XCDs' L2 caches are not coherent for plain ones).
//
// One more wave of the workgroup does this (the chain wave), while the others load their next tile: a wave's loads
// return in order, so a wave with a tile's loads in flight would see an answer only after them. A workgroup a tile
// and no such wave: forward 186 us, backward 409, at 4 x 8192 x 2048 bf16, where they take 127 and 265.
// Groups of 4, 8 and 16 tiles: forward 141, 139 and 140 us, backward 265, 267 and 271, and from checkpoints,
// 8192 x 2048, 200, 203 and 229 (all before later steps).
constexpr int kGroup = 8;
constexpr unsigned kAbsent = 0xffffffffu;
constexpr int kPolls = 1 << 20;  // looks at the words in front of a tile at most (about half a second): then NaN
constexpr unsigned kGaveUp = 1;  // left behind the ticket by a wait that ran out of them

struct Chain {
  unsigned* ticket;    // counter; behind it, kGaveUp once a wait has given up (no kernel clears it)
  uint64_t* map;       // [nq][D]: A in the upper, B in the lower half
  unsigned* state;     // [groups][D]
  int nq, ncol;        // tiles along the tokens, columns of tiles
  int side, per;       // the order of tiles: `side` sequences of `per` tiles each side by side
};

inline int groups_of(int nq) { return (nq + kGroup - 1) / kGroup; }
inline size_t round_up(size_t n) { return (n + 255) / 256 * 256; }
inline size_t map_bytes(int nq, int D) { return round_up((size_t)nq * D * 8); }
inline size_t chain_bytes(int nq, int D) {
  return nq <= 1 ? 0 : 256 + map_bytes(nq, D) + round_up((size_t)groups_of(nq) * D * 4);
}
// The chain in `workspace` (chain_bytes) over tiles of `tile` tokens.
inline Chain make_chain(const GlrArgs& a, void* workspace, int tile, int width) {
  Chain c{};
  c.nq = (int)(((int64_t)a.T + tile - 1) / tile), c.ncol = (a.D + width - 1) / width;
  c.side = 1, c.per = c.nq;
  if (c.nq <= 1) return c;
  // equal sequences of whole tiles do not depend on each other: side by side, each has the workgroups in
  // flight reach less far, and waits less
  if (!a.seqs.cu && a.seqs.len % tile == 0) c.side = a.N, c.per = c.nq / a.N;
  unsigned char* p = static_cast<unsigned char*>(workspace);
  c.ticket = reinterpret_cast<unsigned*>(p);
  c.map = reinterpret_cast<uint64_t*>(p + 256);
  c.state = reinterpret_cast<unsigned*>(p + 256 + map_bytes(c.nq, a.D));
  return c;
}
// Readies the chain, and passes the states of sequences without tokens through (from: init or dfinal, or
// null: zeros; to: final or dinit, or null).
hipError_t launch_ready(const GlrArgs& a, const Chain& c, const float* from, float* to, hipStream_t stream);

// Workgroups of a launch: one a CU, or one a tile if those are fewer or do not wait for each other.
inline unsigned chain_blocks(const Chain& c) {
  const int64_t tiles = (int64_t)c.nq * c.ncol;
  return (unsigned)(c.nq <= 1 || tiles < 256 ? tiles : 256);
}

__device__ __forceinline__ unsigned stored_bits(float x) { return x != x ? 0x7fc00000u : __float_as_uint(x); }

__device__ __forceinline__ void put_map(const Chain& c, int q, int D, int col, float A, float B) {
  const uint64_t w = (uint64_t)stored_bits(A) << 32 | __float_as_uint(B);
  __hip_atomic_store(c.map + (size_t)q * D + col, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void put_state(const Chain& c, int group, int D, int col, float h) {
  __hip_atomic_store(c.state + (size_t)group * D + col, stored_bits(h), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state in front of tile q, whose sequence reaches back to tile q0 < q: its own tile (q0) when that is
// in q's group, else the state behind the group in front; then the maps of the tiles between, in order.
template <int VEC>
__device__ __forceinline__ void wait_front(const Chain& c, int q, int q0, int D, int col, float (&front)[VEC]) {
  const int group = q / kGroup, group0 = group * kGroup, from = max(q0, group0), count = q - from;
  const bool far = q0 < group0;
  uint64_t w[kGroup - 1][VEC];
  unsigned s[VEC];
  // bit k: map k is awaited; bit kGroup - 1: the state is. Uniform over the wave.
  unsigned open = (1u << count) - 1 | (far ? 1u << (kGroup - 1) : 0u);
#pragma unroll
  for (int e = 0; e < VEC; ++e) s[e] = 0;
  for (int i = 0; i < kPolls && open; ++i) {
    if (open >> (kGroup - 1)) {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        s[e] = __hip_atomic_load(c.state + (size_t)(group - 1) * D + col + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
#pragma unroll
    for (int k = 0; k < kGroup - 1; ++k)
      if (open >> k & 1) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          w[k][e] = __hip_atomic_load(c.map + (size_t)(from + k) * D + col + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    unsigned left = 0;
    if (open >> (kGroup - 1)) {
      bool here = true;
#pragma unroll
      for (int e = 0; e < VEC; ++e) here = here && s[e] != kAbsent;
      if (wave_any(!here)) left |= 1u << (kGroup - 1);
    }
#pragma unroll
    for (int k = 0; k < kGroup - 1; ++k)
      if (open >> k & 1) {
        bool here = true;
#pragma unroll
        for (int e = 0; e < VEC; ++e) here = here && (unsigned)(w[k][e] >> 32) != kAbsent;
        if (wave_any(!here)) left |= 1u << k;
      }
    open = left;
    if (open) __builtin_amdgcn_s_sleep(1);
  }
  if (open && __lane_id() == 0) __hip_atomic_store(c.ticket + 1, kGaveUp, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
  for (int e = 0; e < VEC; ++e) front[e] = __uint_as_float(s[e]);  // still absent: all ones is a NaN
#pragma unroll
  for (int k = 0; k < kGroup - 1; ++k)
    if (k < count) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float A = __uint_as_float((unsigned)(w[k][e] >> 32)), B = __uint_as_float((unsigned)w[k][e]);
        // what was in front of the tile where the sequence began does not reach it
        front[e] = k == 0 && !far ? B : fmaf(A, front[e], B);
      }
    }
}

// A tile as the chain wave finds it for the other waves: its place along the tokens, its column, and the
// sequence [bos, eos] that its first (forward) or last (backward) token lies in (as `around`).
struct Tile {
  int q, column;  // q = nq: none is left
  int bos, eos;
};
// The chain wave's next tile: by the counter where tiles wait for each other, else by its index. ask() sends
// for it, and told() is uniform.
__device__ __forceinline__ int ask(const Chain& c, bool first) {
  if (c.nq <= 1) return first ? blockIdx.x : c.ncol;  // a workgroup a tile
  return __lane_id() == 0 ? (int)__hip_atomic_fetch_add(c.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
}
__device__ __forceinline__ int told(int answer) { return __builtin_amdgcn_readfirstlane(answer); }
// Place along the tokens (nq behind the last tile) and column of a tile.
__device__ __forceinline__ void place_of(const Chain& c, int tile, int& q, int& column) {
  const int i = tile / c.ncol;
  column = tile - i * c.ncol;
  q = i >= c.nq ? c.nq : c.side == 1 ? i : (i % c.side) * c.per + i / c.side;
}
// A tile through LDS, written by one lane.
__device__ __forceinline__ void publish(Tile* s, const Tile& t) {
  if (__lane_id() == 0) *s = t;
}
__device__ __forceinline__ Tile read(const Tile* s) {
  return {__builtin_amdgcn_readfirstlane(s->q), __builtin_amdgcn_readfirstlane(s->column),
          __builtin_amdgcn_readfirstlane(s->bos), __builtin_amdgcn_readfirstlane(s->eos)};
}

// VEC channels a lane in LDS.
template <int VEC> struct Lanes {
  typename RowVec<float, VEC>::type v[64];
  __device__ __forceinline__ void get(int lane, float (&f)[VEC]) const {
    const typename RowVec<float, VEC>::type t = v[lane];
    if constexpr (VEC == 1) f[0] = t;
    else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = t[e];
    }
  }
  __device__ __forceinline__ void set(int lane, const float (&f)[VEC]) {
    typename RowVec<float, VEC>::type t;
    if constexpr (VEC == 1) t = f[0];
    else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) t[e] = f[e];
    }
    v[lane] = t;
  }
};

// What a lane holds of a tensor over its wave's span of NT tokens.
template <typename T, int VEC, int NT, bool CK> struct Held {
  Piece<T, VEC> at[NT];
  static __device__ __forceinline__ Rows rows(const Source& s, int64_t t, int n, int D) { return Piece<T, VEC>::rows(s, t, n, D); }
  __device__ __forceinline__ void begin(const Rows&, int, int, int) {}
  __device__ __forceinline__ void load(const Rows& r, int j, int row, int col) { at[j].load(r, row, col); }
  __device__ __forceinline__ void get(int j, float (&v)[VEC]) const { at[j].get(v); }
};
// A checkpoint's: a span has 2 VEC scales a token, one load brings a scale to a lane, and they are passed
// between lanes where they are used (every lane takes part). With a load of each token's scales the backward
// pass took 166 us where it takes 144 (8192 x 2048).
template <typename T, int VEC, int NT> struct Held<T, VEC, NT, true> {
  static constexpr int kScales = 64 * VEC / kScaleBlock;
  static_assert(kScales * NT <= 64, "a scale a lane");
  unsigned word[NT], scale;
  static __device__ __forceinline__ Rows rows(const Source& s, int64_t t, int n, int D) { return PackedPiece<VEC>::rows(s, t, n, D); }
  // c0: the wave's first channel
  __device__ __forceinline__ void begin(const Rows& r, int n, int c0, int D) {
    const int lane = __lane_id(), j = min(lane / kScales, n - 1);
    const int block = min(c0 / kScaleBlock + lane % kScales, D / kScaleBlock - 1);
    scale = __builtin_amdgcn_raw_buffer_load_b8(r.scales, j * r.ld_scales + block, 0, 0);
  }
  __device__ __forceinline__ void load(const Rows& r, int j, int row, int col) { word[j] = PackedPiece<VEC>::codes(r, row, col); }
  __device__ __forceinline__ void get(int j, float (&v)[VEC]) const {
    PackedPiece<VEC> p;
    p.word[0] = word[j];
    p.byte = __builtin_amdgcn_ds_bpermute((j * kScales + (int)__lane_id() * VEC / kScaleBlock) * 4, scale);
    p.get(v);
  }
};

// Which tokens of a wave's span begin or end a sequence, or lie in one: bit j is token t0 + j.
struct Marks {
  unsigned start, end, valid;
  int first;     // a sequence at or in front of the first one that is met in the span
  int bos, eos;  // the first token of the sequence that the first token lies in (that token, if in none),
                 // and the last token of the one that the last token lies in (that token, if in none)
};
__device__ __forceinline__ unsigned bits_between(int lo, int hi) {  // [lo, hi), hi - lo >= 1, hi <= 32
  return (0xffffffffu >> (32 - (hi - lo))) << lo;
}
// The last sequence at or behind `i` whose first token is at or before t (i where there is none); empty ones in
// front of it are passed over. By halving, with scalar loads, which wait for no tile's loads in flight.
__device__ __forceinline__ int last_at(const Sequences& s, int i, int t) {
  if (!s.cu) return max(i, min(t / s.len, s.N - 1));
  for (int end = s.N; i + 1 < end;) {
    const int mid = (i + end) / 2;
    const bool here = s.span(mid).bos <= t;
    i = here ? mid : i;
    end = here ? end : mid;
  }
  return i;
}
// 1 <= n <= 32 tokens from t0, in [0, T).
__device__ __forceinline__ Marks marks_of(const Sequences& s, int t0, int n) {
  Marks m{0, 0, 0, last_at(s, 0, t0), t0, t0 + n - 1};
  for (int i = m.first;;) {
    const Span p = s.span(i);
    if (p.bos >= t0 + n) break;
    const int lo = max(p.bos, t0), hi = min(p.eos, t0 + n);
    if (lo < hi) {
      m.valid |= bits_between(lo - t0, hi - t0);
      if (p.bos >= t0) m.start |= 1u << (p.bos - t0);
      if (p.eos <= t0 + n) m.end |= 1u << (p.eos - 1 - t0);
      if (lo == t0) m.bos = p.bos;
      if (hi == t0 + n) m.eos = p.eos - 1;
    }
    if (i + 1 >= s.N) break;
    i = last_at(s, i + 1, p.eos);
  }
  return m;
}
// The sequence that token t lies in, as its first and last tokens; t itself where it lies in none.
__device__ __forceinline__ Span around(const Sequences& s, int t) {
  const Span p = s.span(last_at(s, 0, t));
  return p.bos <= t && p.eos > t ? Span{p.bos, p.eos - 1} : Span{t, t};
}
// The sequence at or behind `i` (which begins at or before t) whose first (last) token is t; N where there is none.
__device__ __forceinline__ int starting_at(const Sequences& s, int i, int t) {
  if (i >= s.N) return s.N;
  i = last_at(s, i, t);
  const Span p = s.span(i);
  return p.bos == t && p.eos > t ? i : s.N;
}
__device__ __forceinline__ int ending_at(const Sequences& s, int i, int t) {
  if (i >= s.N) return s.N;
  i = last_at(s, i, t);
  const Span p = s.span(i);
  return p.bos <= t && p.eos == t + 1 ? i : s.N;
}

// go(has an input gate, is normalised), as types.
template <class F> hipError_t with_gates(const GlrArgs& a, F&& go) {
  std::true_type yes;
  std::false_type no;
  if (a.in.p) return a.normalise ? go(yes, yes) : go(yes, no);
  return a.normalise ? go(no, yes) : go(no, no);
}

}  // namespace glr
}  // namespace kda
