// Gated linear recurrence with one state per channel, forward, and its one-token step.
//
//   g_t = -exp(A_log) softplus(gate_x_t + dt_bias),  a_t = exp(g_t)       (the standard decay gate)
//   h_t = a_t h_{t-1} + w_t logistic(in_gate_t) x_t,  w_t = sqrt(1 - a_t^2) or 1;   y_t = h_t
//
// About 30 operations an element, six of them transcendental (16 cycles a wave each, the others 4), and
// 8 bytes in bf16: the vector ALU needs about two thirds of the time that HBM does, so the gates are
// computed once and every tensor moves once. A wave holds a span of tokens for 64 VEC channels in
// registers: the states from zero, and the products of decays with which the state in front of the
// span enters them. That state comes through the waves of the workgroup and the chain of tiles
// (kda_glr.h).
#include <type_traits>

#include "kda_glr.h"

namespace kda {
namespace glr {

constexpr int kReadyThreads = 256;

__global__ __launch_bounds__(kReadyThreads) void ready_kernel(Chain c, int64_t words) {
  const int64_t i = (int64_t)blockIdx.x * kReadyThreads + threadIdx.x;
  if (i == 0) *c.ticket = 0;
  // the maps and the states lie behind each other: 16 bytes a thread
  if (i < words) reinterpret_cast<uint4*>(c.map)[i] = make_uint4(kAbsent, kAbsent, kAbsent, kAbsent);
}

Chain make_chain(void* workspace, int nq, int ncol, int D) {
  Chain c{};
  c.nq = nq, c.ncol = ncol;
  if (nq <= 1) return c;
  unsigned char* p = static_cast<unsigned char*>(workspace);
  c.ticket = reinterpret_cast<unsigned*>(p);
  c.map = reinterpret_cast<uint64_t*>(p + 256);
  c.state = reinterpret_cast<unsigned*>(p + 256 + map_bytes(nq, D));
  return c;
}

hipError_t launch_ready_chain(const Chain& c, int D, hipStream_t stream) {
  if (c.nq <= 1) return hipSuccess;
  const int64_t words = (int64_t)(chain_bytes(c.nq, D) - 256) / 16;
  hipLaunchKernelGGL(ready_kernel, dim3((unsigned)((words + kReadyThreads - 1) / kReadyThreads)),
                     dim3(kReadyThreads), 0, stream, c, words);
  return hipGetLastError();
}

// Sequences without tokens: a chunk of kSeqs a wave.
template <int VEC, int WAVES>
__device__ __forceinline__ void empty_sequences(const GlrArgs& a, int chunk, int col, const float* from, float* to) {
  const int wave = threadIdx.x / 64;
  for (int i = 0; i < kSeqs; ++i) {
    const int n = (chunk * kSeqs + i) * WAVES + wave;
    if (n >= a.N) return;
    const Span s = a.seqs.span(n);
    if (s.eos > s.bos) continue;
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (col + e < a.D) to[(int64_t)n * a.D + col + e] = from ? from[(int64_t)n * a.D + col + e] : 0.f;
  }
}

constexpr int kFwdTokens = 16, kFwdWaves = 8;  // a wave's span, waves of a workgroup
constexpr int kFwdTile = kFwdTokens * kFwdWaves;
static_assert(kGlrBlock % kFwdTokens == 0 && kFwdTile % kGlrBlock == 0, "a block's first token begins a span");

template <typename T, int VEC, bool CK, bool GATE, bool NORM>
__global__ __launch_bounds__(64 * kFwdWaves, 4) void fwd_kernel(GlrArgs a, Chain chain, int ntiles) {
  constexpr int NT = kFwdTokens, NW = kFwdWaves, C = 64 * VEC;
  constexpr unsigned kFull = 0xffffffffu >> (32 - NT);
  typedef typename KeptPiece<T, VEC, CK>::type piece;
  __shared__ float s_wave[NW][2][C];       // a span's map
  __shared__ float s_tile[kGroup][2][C];   // the maps of the group's tiles in front; slot kGroup - 1: the
                                           // state in front of the group in its first row
  __shared__ int s_index;
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  const int tile = take_tile(chain, &s_index);
  const bool extra = tile >= ntiles;
  const int index = extra ? tile - ntiles : tile;
  const int q = index / chain.ncol, k0 = (index - q * chain.ncol) * C + lane * VEC;
  if (extra) {
    empty_sequences<VEC, NW>(a, q, k0, a.init, a.final);
    return;
  }
  const bool active = k0 < a.D;            // D is a multiple of VEC
  const int col = active ? k0 : a.D - VEC;
  const int tile0 = q * kFwdTile, t0 = __builtin_amdgcn_readfirstlane(tile0 + wave * NT);
  const int count = min(max(a.T - t0, 0), NT);

  piece x[NT], r[NT], in[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t t = min(t0 + j, a.T - 1);
    r[j].load(a.r, t * a.r.ld + col);
    x[j].load(a.x, t * a.x.ld + col);
    if constexpr (GATE) in[j].load(a.in, t * a.in.ld + col);
  }
  Channel ch[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) ch[e] = channel(a, col + e);
  Marks m{0, 0, 0, 0};
  if (count > 0) m = marks_of(a.seqs, t0, count);

  float h[NT][VEC], p[NT][VEC];  // states from zero in front of the span; products of its decays
  {
    float hs[VEC], ps[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) hs[e] = 0.f, ps[e] = 1.f;
    auto token = [&](int j, float (&av)[VEC], float (&bv)[VEC]) {
      float xv[VEC], rv[VEC], iv[VEC];
      x[j].get(xv);
      r[j].get(rv);
      if constexpr (GATE) in[j].get(iv);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float slope, b = xv[e];
        const float g2 = decay_log2(rv[e], ch[e], slope);
        av[e] = fast_exp2(g2);
        if constexpr (GATE) b *= sigmoid_fast(iv[e]);
        if constexpr (NORM) b *= input_weight(av[e], g2);
        bv[e] = b;
      }
    };
    if (m.start == 0 && m.valid == kFull) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float av[VEC], bv[VEC];
        token(j, av, bv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          h[j][e] = hs[e] = fmaf(av[e], hs[e], bv[e]);
          p[j][e] = ps[e] = ps[e] * av[e];
        }
      }
    } else {
      int n = m.first;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float av[VEC], bv[VEC];
        token(j, av, bv);
        if (m.start >> j & 1) {
          n = starting_at(a.seqs, n, t0 + j);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float first = a.init && n < a.N ? a.init[(int64_t)n * a.D + col + e] : 0.f;
            hs[e] = fmaf(av[e], first, bv[e]);
          }
        } else if (m.valid >> j & 1) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            hs[e] = fmaf(av[e], hs[e], bv[e]);
            ps[e] *= av[e];
          }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[j][e] = hs[e], p[j][e] = ps[e];
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      s_wave[wave][0][lane * VEC + e] = ps[e];
      s_wave[wave][1][lane * VEC + e] = hs[e];
    }
  }
  lds_barrier();
  // The sequence that holds a token, if it began in front of it: where it began. Else the token.
  auto began = [&](int t) {
    const Span s = a.seqs.span(a.seqs.find(t));
    return s.bos < t && s.eos > t ? s.bos : t;
  };
  const bool whole = chain.nq > 1;
  const int tile_bos = began(tile0);
  // Folds the spans [from, to) of this tile behind the state c (to: wave-uniform).
  auto fold = [&](float (&c)[VEC], int from, int to) {
    for (int i = from; i < to; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) c[e] = fmaf(s_wave[i][0][lane * VEC + e], c[e], s_wave[i][1][lane * VEC + e]);
  };
  // The state in front of this wave's span, given the tile's.
  const int span_bos = count > 0 ? began(t0) : t0;
  auto span_state = [&](float (&c)[VEC], const float (&front)[VEC]) {
    if (span_bos >= t0) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) c[e] = 0.f;
    } else if (span_bos >= tile0) {
      const int i = (span_bos - tile0) / NT;
#pragma unroll
      for (int e = 0; e < VEC; ++e) c[e] = s_wave[i][1][lane * VEC + e];
      fold(c, i + 1, wave);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) c[e] = front[e];
      fold(c, 0, wave);
    }
  };
  // The last sequence that a token of this tile lies in: did it begin in the tile?
  const int last = min(tile0 + kFwdTile, a.T) - 1, last_bos = began(last);
  const bool resets = last_bos >= tile0;
  const int last_wave = (last - tile0) / NT;
  auto behind = [&](float (&c)[VEC], const float (&front)[VEC]) {  // the state behind the tile
    if (resets) {
      const int i = (last_bos - tile0) / NT;
#pragma unroll
      for (int e = 0; e < VEC; ++e) c[e] = s_wave[i][1][lane * VEC + e];
      fold(c, i + 1, last_wave + 1);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) c[e] = front[e];
      fold(c, 0, last_wave + 1);
    }
  };
  float front[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) front[e] = 0.f;
  const int group = q / kGroup, group0 = group * kGroup;
  if (whole) {
    if (wave == NW - 1 && active && q + 1 < chain.nq) {
      float A[VEC], B[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) A[e] = 1.f;
      for (int i = 0; i <= last_wave; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) A[e] *= s_wave[i][0][lane * VEC + e];
      behind(B, front);
#pragma unroll
      for (int e = 0; e < VEC; ++e) put_map(chain, q, a.D, col + e, A[e], B[e]);
    }
    if (tile_bos < tile0) {  // the state in front comes from other tiles
      const int q0 = tile_bos / kFwdTile, from = max(q0, group0);
      static_assert(NW >= kGroup, "a wave for every tile of a group");
      if (wave < q - from) {
        float A, B;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          wait_map(chain, from + wave, a.D, col + e, A, B);
          s_tile[wave][0][lane * VEC + e] = A;
          s_tile[wave][1][lane * VEC + e] = B;
        }
      } else if (wave == kGroup - 1 && q0 < group0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          s_tile[kGroup - 1][0][lane * VEC + e] = wait_state(chain, group - 1, a.D, col + e);
      }
      lds_barrier();
      int i = 0;
      if (q0 < group0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) front[e] = s_tile[kGroup - 1][0][lane * VEC + e];
      } else {  // the sequence began in this tile: its state does not depend on what was in front
#pragma unroll
        for (int e = 0; e < VEC; ++e) front[e] = s_tile[0][1][lane * VEC + e];
        i = 1;
      }
      for (; i < q - from; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) front[e] = fmaf(s_tile[i][0][lane * VEC + e], front[e], s_tile[i][1][lane * VEC + e]);
    }
    if (wave == NW - 1 && active && q + 1 < chain.nq && q - group0 == kGroup - 1) {
      float c[VEC];
      behind(c, front);
#pragma unroll
      for (int e = 0; e < VEC; ++e) put_state(chain, group, a.D, col + e, c[e]);
    }
  }
  if (count == 0 || !active) return;
  float c[VEC];
  span_state(c, front);
  if (a.states && t0 % kGlrBlock == 0) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) a.states[(int64_t)(t0 / kGlrBlock) * a.D + col + e] = c[e];
  }
  T* y = static_cast<T*>(a.y) + (int64_t)t0 * a.D + col;
  auto put = [&](int j, const float (&v)[VEC]) {
    Piece<T, VEC> o;
    o.set(v);
    o.store(y, (int64_t)j * a.D);
  };
  if (m.start == 0 && m.valid == kFull) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[j][e] = fmaf(p[j][e], c[e], h[j][e]);
      if (a.y) put(j, h[j]);
    }
  } else {
    unsigned begun = 0;  // a sequence has begun in the span
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      begun |= m.start >> j & 1;
      const bool lies = m.valid >> j & 1;
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[j][e] = !lies ? 0.f : begun ? h[j][e] : fmaf(p[j][e], c[e], h[j][e]);
      if (a.y && j < count && (lies || a.zero_rest)) put(j, h[j]);
    }
  }
  if (!a.final) return;
  int n = m.first;
  for (unsigned left = m.end; left; left &= left - 1) {
    const int at = __builtin_ctz(left);
    n = ending_at(a.seqs, n, t0 + at);
    if (n >= a.N) break;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      if (j == at) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) a.final[(int64_t)n * a.D + col + e] = h[j][e];
      }
  }
}

template <typename T, int VEC, bool CK, bool GATE, bool NORM>
hipError_t run_fwd(const GlrArgs& a, void* workspace, hipStream_t stream) {
  const int nq = (a.T + kFwdTile - 1) / kFwdTile, ncol = (a.D + 64 * VEC - 1) / (64 * VEC);
  const Chain c = make_chain(workspace, nq, ncol, a.D);
  hipError_t e = launch_ready_chain(c, a.D, stream);
  if (e != hipSuccess) return e;
  // sequences without tokens are looked for where there may be any
  const int chunks = a.final && (a.seqs.cu || a.T == 0) ? (a.N + kSeqs * kFwdWaves - 1) / (kSeqs * kFwdWaves) : 0;
  const int64_t blocks = (int64_t)(nq + chunks) * ncol;
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL((fwd_kernel<T, VEC, CK, GATE, NORM>), dim3((unsigned)blocks), dim3(64 * kFwdWaves), 0, stream, a, c,
                     nq * ncol);
  return hipGetLastError();
}

// One token of B requests on slots of a pool of states.
constexpr int kStepThreads = 256;

template <typename T, int VEC, bool GATE, bool NORM>
__global__ __launch_bounds__(kStepThreads) void step_kernel(GlrArgs a, int ncol) {
  const int n = blockIdx.x / ncol, col = ((blockIdx.x - n * ncol) * kStepThreads + threadIdx.x) * VEC;
  if (col >= a.D) return;
  Piece<T, VEC> x, r, in, o;
  const int64_t slot = a.slots ? a.slots[n] : n;
  float y[VEC];
  if (slot < 0 || slot >= a.nslots) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) y[e] = 0.f;
  } else {
    x.load(a.x, n * a.x.ld + col);
    r.load(a.r, n * a.r.ld + col);
    if constexpr (GATE) in.load(a.in, n * a.in.ld + col);
    float* st = a.pool + slot * a.D + col;
    float xv[VEC], rv[VEC], iv[VEC], h[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] = st[e];
    x.get(xv);
    r.get(rv);
    if constexpr (GATE) in.get(iv);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float slope, b = xv[e];
      const float g2 = decay_log2(rv[e], channel(a, col + e), slope), av = fast_exp2(g2);
      if constexpr (GATE) b *= sigmoid_fast(iv[e]);
      if constexpr (NORM) b *= input_weight(av, g2);
      y[e] = fmaf(av, h[e], b);
      st[e] = y[e];
    }
  }
  o.set(y);
  o.store(a.y, (int64_t)n * a.D + col);
}

template <typename T, int VEC, bool GATE, bool NORM>
hipError_t run_step(const GlrArgs& a, hipStream_t stream) {
  const int ncol = (a.D + VEC * kStepThreads - 1) / (VEC * kStepThreads);
  hipLaunchKernelGGL((step_kernel<T, VEC, GATE, NORM>), dim3((unsigned)((int64_t)a.B * ncol)), dim3(kStepThreads), 0, stream,
                     a, ncol);
  return hipGetLastError();
}

}  // namespace glr

size_t glr_fwd_workspace_bytes(int T, int D) {
  return glr::chain_bytes((int)(((int64_t)T + glr::kFwdTile - 1) / glr::kFwdTile), D);
}

hipError_t launch_glr_fwd(GlrArgs a, void* workspace, hipStream_t stream) {
  const void* ptrs[] = {a.x.p, a.r.p, a.in.p, a.y};
  return glr::with_gates(a, [&](auto gate, auto norm) {
    constexpr bool G = decltype(gate)::value, M = decltype(norm)::value;
    if (a.packed) {  // states in front of the blocks of a checkpointed call: no outputs of type T
      if (vector_width(2, 1, a.D, ptrs, 3) == 2) return glr::run_fwd<bf16, 2, true, G, M>(a, workspace, stream);
      return glr::run_fwd<bf16, 1, true, G, M>(a, workspace, stream);
    }
    if (!a.bf) return glr::run_fwd<float, 1, false, G, M>(a, workspace, stream);
    if (vector_width(2, 2, a.D | a.x.ld | a.r.ld | a.in.ld, ptrs, 4) == 2)
      return glr::run_fwd<bf16, 2, false, G, M>(a, workspace, stream);
    return glr::run_fwd<bf16, 1, false, G, M>(a, workspace, stream);
  });
}

hipError_t launch_glr_step(const GlrArgs& a, hipStream_t stream) {
  const void* ptrs[] = {a.x.p, a.r.p, a.in.p, a.y};
  return glr::with_gates(a, [&](auto gate, auto norm) {
    constexpr bool G = decltype(gate)::value, M = decltype(norm)::value;
    if (!a.bf) return glr::run_step<float, 1, G, M>(a, stream);
    if (vector_width(2, 2, a.D | a.x.ld | a.r.ld | a.in.ld, ptrs, 4) == 2) return glr::run_step<bf16, 2, G, M>(a, stream);
    return glr::run_step<bf16, 1, G, M>(a, stream);
  });
}

}  // namespace kda
