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

// ---- Gates. Per channel: -exp(A_log) in units of log2 (an exp(A_log) above 2e38 counts as that, so
// that the product is finite), and the bias.
struct Channel {
  float neg_rate2, bias;
};
__device__ __forceinline__ Channel channel(const GlrArgs& a, int c) {
  const float rate = expf(a.A_log[c]);
  return {-(rate > 2.0e38f ? 2.0e38f : rate) * kLog2e, a.dt_bias ? a.dt_bias[c] : 0.f};
}

// log2 of the decay, g2 <= 0, for the gate's input; also what the softplus leaves for its slope, the
// logistic of z. Held above -1e30, so that products with it stay finite (the decay is 0 long before).
__device__ __forceinline__ float decay_log2(float x, const Channel& ch, float& slope) {
  float e, r;
  const float z = x + ch.bias, g2 = ch.neg_rate2 * softplus_f32(z, e, r);
  slope = logistic_from(z, e, r);
  return g2 < -1e30f ? -1e30f : g2;
}

// logistic(z), the input gate.
__device__ __forceinline__ float sigmoid_fast(float z) {
  return __builtin_amdgcn_rcpf(1.f + fast_exp2(-z * kLog2e));
}

// sqrt(1 - a^2) for a = 2^g2. Near a = 1 the difference would cancel: there 1 - e^-v, v = -2 g ln 2,
// by its series (relative error v^5 / 720 < 5e-8 at v = 1/8); elsewhere from a, whose last bit costs
// 1e-6 at most.
__device__ __forceinline__ float input_weight(float a, float g2) {
  const float v = -2.f * kLn2 * g2;
  const float p = v * fmaf(v, fmaf(v, fmaf(v, fmaf(v, 1.f / 120, -1.f / 24), 1.f / 6), -0.5f), 1.f);
  return __builtin_amdgcn_sqrtf(v < 0.125f ? p : fmaf(-a, a, 1.f));
}

// ---- Work. A workgroup's tile is kWaves consecutive spans of tokens (one a wave) by 64 VEC channels
// (VEC a lane). A tile's effect on the state is h -> A h + B per channel; tiles of one column follow
// each other along the tokens (backward: against them), `q` counting from the first.
//
// The token axis is scanned in one pass, every tensor read once: a tile leaves (A, B) for the tiles
// behind it as soon as it has them, the last tile of every kGroup leaves the state behind it, and a
// tile gathers the state in front of it from the state behind the previous group and the (A, B) of its
// own group's tiles in front of it, always folded in the same order: results do not depend on timing.
// Workgroups take their tiles from a counter, in the order of q. So a tile waits only for tiles whose
// workgroups have started before its own; (A, B) waits for nothing, and the state behind a group only
// for those and for the state behind the group in front: every wait ends.
//
// A word that is not there yet is all ones, which no value that is stored has (NaN is stored as
// 0x7fc00000 where it could be mistaken): value and presence arrive together, in one relaxed atomic
// access of the whole device (the XCDs' L2 caches are not coherent for plain ones).
constexpr int kGroup = 8;
constexpr unsigned kAbsent = 0xffffffffu;
constexpr int kPolls = 1 << 22;  // of one word at most (seconds): then NaN, so that every wave ends

struct Chain {
  unsigned* ticket;    // counter
  uint64_t* map;       // [nq][D]: A in the upper, B in the lower half
  unsigned* state;     // [groups][D]
  int nq, ncol;        // tiles along the tokens, columns of tiles
};

inline int groups_of(int nq) { return (nq + kGroup - 1) / kGroup; }
inline size_t round_up(size_t n) { return (n + 255) / 256 * 256; }
inline size_t map_bytes(int nq, int D) { return round_up((size_t)nq * D * 8); }
inline size_t chain_bytes(int nq, int D) {
  return nq <= 1 ? 0 : 256 + map_bytes(nq, D) + round_up((size_t)groups_of(nq) * D * 4);
}
// The chain in `workspace` (chain_bytes), and a launch that readies it.
Chain make_chain(void* workspace, int nq, int ncol, int D);
hipError_t launch_ready_chain(const Chain& c, int D, hipStream_t stream);

__device__ __forceinline__ unsigned stored_bits(float x) { return x != x ? 0x7fc00000u : __float_as_uint(x); }

__device__ __forceinline__ void put_map(const Chain& c, int q, int D, int col, float A, float B) {
  const uint64_t w = (uint64_t)stored_bits(A) << 32 | __float_as_uint(B);
  __hip_atomic_store(c.map + (size_t)q * D + col, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void put_state(const Chain& c, int group, int D, int col, float h) {
  __hip_atomic_store(c.state + (size_t)group * D + col, stored_bits(h), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void wait_map(const Chain& c, int q, int D, int col, float& A, float& B) {
  uint64_t w;
  for (int i = 0; i < kPolls; ++i) {
    w = __hip_atomic_load(c.map + (size_t)q * D + col, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if ((unsigned)(w >> 32) != kAbsent) break;
    __builtin_amdgcn_s_sleep(1);
  }
  A = __uint_as_float((unsigned)(w >> 32));  // still absent: all ones is a NaN
  B = __uint_as_float((unsigned)w);
}
__device__ __forceinline__ float wait_state(const Chain& c, int group, int D, int col) {
  unsigned w;
  for (int i = 0; i < kPolls; ++i) {
    w = __hip_atomic_load(c.state + (size_t)group * D + col, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (w != kAbsent) break;
    __builtin_amdgcn_s_sleep(1);
  }
  return __uint_as_float(w);
}

// This workgroup's tile: by the counter where tiles wait for each other, else by its index.
__device__ __forceinline__ int take_tile(const Chain& c, int* shared) {
  if (c.nq <= 1) return blockIdx.x;
  if (threadIdx.x == 0) *shared = (int)__hip_atomic_fetch_add(c.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  block_barrier();
  return __builtin_amdgcn_readfirstlane(*shared);
}

constexpr int kSeqs = 16;  // sequences a wave looks at for ones without tokens

// Which tokens of a wave's span begin or end a sequence, or lie in one: bit j is token t0 + j.
struct Marks {
  unsigned start, end, valid;
  int first;  // a sequence at or in front of the first one that is met in the span
};
__device__ __forceinline__ unsigned bits_between(int lo, int hi) {  // [lo, hi), hi - lo >= 1, hi <= 32
  return (0xffffffffu >> (32 - (hi - lo))) << lo;
}
// Every lane takes part. t0 < T.
__device__ __forceinline__ Marks marks_of(const Sequences& s, int t0, int n) {
  Marks m{0, 0, 0, s.find(t0)};
  for (int i = m.first; i < s.N; ++i) {
    const Span p = s.span(i);
    if (p.bos >= t0 + n) break;
    const int lo = max(p.bos, t0), hi = min(p.eos, t0 + n);
    if (lo >= hi) continue;
    m.valid |= bits_between(lo - t0, hi - t0);
    if (p.bos >= t0) m.start |= 1u << (p.bos - t0);
    if (p.eos <= t0 + n) m.end |= 1u << (p.eos - 1 - t0);
  }
  return m;
}
// The sequence at or behind `i` whose first (last) token is t; N where there is none.
__device__ __forceinline__ int starting_at(const Sequences& s, int i, int t) {
  for (; i < s.N; ++i) {
    const Span p = s.span(i);
    if (p.bos == t && p.eos > t) break;
  }
  return i;
}
__device__ __forceinline__ int ending_at(const Sequences& s, int i, int t) {
  for (; i < s.N; ++i) {
    const Span p = s.span(i);
    if (p.eos == t + 1 && p.bos <= t) break;
  }
  return i;
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
