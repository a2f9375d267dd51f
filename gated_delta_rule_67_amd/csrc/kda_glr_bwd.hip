// Gated linear recurrence with one state per channel, backward.
//
// With G_t the gradient that reaches h_t and R_t its part from behind (a_{t+1} G_{t+1}, or the final
// state's gradient at a sequence's last token), s = logistic(in_gate), q = s x:
//   G_t = dy_t + R_t,   R_{t-1} = a_t G_t,   the initial state's gradient is a_1 G_1,
//   dx = G s w,   din_gate = G x w s (1 - s),
//   dg = G a h_{t-1} - G q a^2 / w   (the second term where w = sqrt(1 - a^2); 0 where w = 0),
//   dgate_x = -exp(A_log) logistic(gate_x + dt_bias) dg,   ddt_bias = sum of it,   dA_log = sum dg g.
// R is a scan against the tokens, by the chain of tiles (kda_glr.h) counted from the last one. h_{t-1}
// comes from the states in front of blocks that the forward pass kept (or, without them, from its
// kernel run for the states only), so every tensor moves once: 14 bytes an element in bf16. The gates
// are computed once and stay in registers: eight values an element, so a wave's span is 8 tokens.
#include <type_traits>

#include "kda_glr.h"

namespace kda {
namespace glr {

constexpr int kBwdTokens = 8, kBwdWaves = 8;
constexpr int kBwdTile = kBwdTokens * kBwdWaves;
static_assert(kBwdTile == kGlrBlock, "a tile begins at a kept state");

template <typename T, int VEC, bool CK, bool GATE, bool NORM>
__global__ __launch_bounds__(64 * kBwdWaves) void bwd_kernel(GlrArgs a, Chain chain, int ntiles) {
  constexpr int NT = kBwdTokens, NW = kBwdWaves, C = 64 * VEC;
  constexpr unsigned kFull = 0xffffffffu >> (32 - NT);
  typedef typename KeptPiece<T, VEC, CK>::type kept;
  typedef Piece<T, VEC> piece;
  __shared__ float s_wave[NW][3][C];      // a span's decays, its state and its gradient, each from zero
  __shared__ float s_tile[kGroup][2][C];  // as in the forward kernel
  __shared__ int s_index;
  const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
  const int tile = take_tile(chain, &s_index);
  const bool extra = tile >= ntiles;
  const int index = extra ? tile - ntiles : tile;
  const int q = index / chain.ncol, k0 = (index - q * chain.ncol) * C + lane * VEC;
  if (extra) {  // sequences without tokens: the final state's gradient passes through
    for (int i = 0; i < kSeqs; ++i) {
      const int n = (q * kSeqs + i) * NW + wave;
      if (n >= a.N) return;
      const Span s = a.seqs.span(n);
      if (s.eos > s.bos) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (k0 + e < a.D) a.dinit[(int64_t)n * a.D + k0 + e] = a.dfinal ? a.dfinal[(int64_t)n * a.D + k0 + e] : 0.f;
    }
    return;
  }
  const bool active = k0 < a.D;
  const int col = active ? k0 : a.D - VEC;
  const int block = chain.nq - 1 - q;  // of tokens
  const int tile0 = block * kBwdTile, t0 = __builtin_amdgcn_readfirstlane(tile0 + wave * NT);
  const int count = min(max(a.T - t0, 0), NT);

  kept xk[NT], rk[NT], ik[NT];
  piece gk[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t t = min(t0 + j, a.T - 1);
    rk[j].load(a.r, t * a.r.ld + col);
    xk[j].load(a.x, t * a.x.ld + col);
    if constexpr (GATE) ik[j].load(a.in, t * a.in.ld + col);
    gk[j].load(a.dy, t * a.dy.ld + col);
  }
  Channel ch[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) ch[e] = channel(a, col + e);
  Marks m{0, 0, 0, 0};
  if (count > 0) m = marks_of(a.seqs, t0, count);
  const bool whole = m.valid == kFull && !m.start && !m.end;  // inside one sequence

  // Per element: decay, its log2, input weight, input gate and one minus it, slope of the softplus
  float av[NT][VEC], g2[NT][VEC], w[NT][VEC], s[NT][VEC], rest[NT][VEC], slope[NT][VEC];
  float A[VEC], hs[VEC], rs[VEC];
  auto input = [&](int j, float (&b)[VEC]) {  // w s x
    xk[j].get(b);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if constexpr (GATE) b[e] *= s[j][e];
      if constexpr (NORM) b[e] *= w[j][e];
    }
  };
  auto first_state = [&](int n, int e) { return a.init && n < a.N ? a.init[(int64_t)n * a.D + col + e] : 0.f; };
  auto last_grad = [&](int n, int e) { return a.dfinal && n < a.N ? a.dfinal[(int64_t)n * a.D + col + e] : 0.f; };
  // The states of the span behind hs, one token at a time: each(j) comes before token j.
  auto states = [&](auto&& each) {
    if (whole) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        each(j);
        float b[VEC];
        input(j, b);
#pragma unroll
        for (int e = 0; e < VEC; ++e) hs[e] = fmaf(av[j][e], hs[e], b[e]);
      }
      return;
    }
    int n = m.first;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (m.start >> j & 1) {
        n = starting_at(a.seqs, n, t0 + j);
#pragma unroll
        for (int e = 0; e < VEC; ++e) hs[e] = first_state(n, e);
      }
      each(j);
      float b[VEC];
      input(j, b);
      if (m.valid >> j & 1) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) hs[e] = fmaf(av[j][e], hs[e], b[e]);
      }
    }
  };
  // The sequences whose last tokens lie in the span, from the last one on: one at a time, against the tokens.
  // (offsets do not decrease, so the walk begins at the span's first sequence each time)
  auto grads = [&](auto&& each) {
#pragma unroll
    for (int j = NT - 1; j >= 0; --j) {
      if (!whole && (m.end >> j & 1)) {
        const int n = ending_at(a.seqs, m.first, t0 + j);
#pragma unroll
        for (int e = 0; e < VEC; ++e) rs[e] = last_grad(n, e);
      }
      each(j);
    }
  };
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    float rv[VEC], iv[VEC];
    rk[j].get(rv);
    if constexpr (GATE) ik[j].get(iv);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      g2[j][e] = decay_log2(rv[e], ch[e], slope[j][e]);
      av[j][e] = fast_exp2(g2[j][e]);
      if constexpr (NORM) w[j][e] = input_weight(av[j][e], g2[j][e]);
      if constexpr (GATE) logistic_pair(iv[e], s[j][e], rest[j][e]);
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) A[e] = 1.f, hs[e] = rs[e] = 0.f;
#pragma unroll
  for (int j = 0; j < NT; ++j)
    if (whole || (m.valid >> j & 1)) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) A[e] *= av[j][e];
    }
  states([](int) {});
  grads([&](int j) {
    if (whole || (m.valid >> j & 1)) {
      float dy[VEC];
      gk[j].get(dy);
#pragma unroll
      for (int e = 0; e < VEC; ++e) rs[e] = av[j][e] * (dy[e] + rs[e]);
    }
  });
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    s_wave[wave][0][lane * VEC + e] = A[e];
    s_wave[wave][1][lane * VEC + e] = hs[e];
    s_wave[wave][2][lane * VEC + e] = rs[e];
  }
  lds_barrier();
  // Where the sequence that holds a token began, if in front of it, and its last token, if behind it;
  // else the token itself.
  auto around = [&](int t) {
    const Span p = a.seqs.span(a.seqs.find(t));
    return p.bos <= t && p.eos > t ? Span{p.bos, p.eos - 1} : Span{t, t};
  };
  const int last = min(tile0 + kBwdTile, a.T) - 1, last_wave = (last - tile0) / NT;
  const Span at_first = around(tile0), at_last = around(last);
  const int span_last = count > 0 ? t0 + count - 1 : t0;
  const int span_bos = count > 0 ? around(t0).bos : t0, span_end = count > 0 ? around(span_last).eos : t0;
  // ---- the state in front of the span
#pragma unroll
  for (int e = 0; e < VEC; ++e) hs[e] = 0.f;
  if (span_bos < t0) {
    int i = 0;
    if (span_bos >= tile0) {
      i = (span_bos - tile0) / NT;
#pragma unroll
      for (int e = 0; e < VEC; ++e) hs[e] = s_wave[i][1][lane * VEC + e];
      ++i;
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) hs[e] = a.states[(int64_t)block * a.D + col + e];
    }
    for (; i < wave; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) hs[e] = fmaf(s_wave[i][0][lane * VEC + e], hs[e], s_wave[i][1][lane * VEC + e]);
  }
  // ---- the gradient behind the tile, by the chain
  auto fold = [&](float (&c)[VEC], int from, int to) {  // spans from, from - 1, ..., to
    for (int i = from; i >= to; --i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) c[e] = fmaf(s_wave[i][0][lane * VEC + e], c[e], s_wave[i][2][lane * VEC + e]);
  };
  // From behind the last sequence that ends at token `end` of this tile, or from `front`, to span `to`.
  auto gather = [&](float (&c)[VEC], int end, int to, const float (&front)[VEC]) {
    int i = last_wave;
    if (end <= last) {
      i = (end - tile0) / NT;
#pragma unroll
      for (int e = 0; e < VEC; ++e) c[e] = s_wave[i][2][lane * VEC + e];
      --i;
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) c[e] = front[e];
    }
    fold(c, i, to);
  };
  float front[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) front[e] = 0.f;
  if (chain.nq > 1) {
    const int group = q / kGroup, group0 = group * kGroup;
    if (wave == NW - 1 && active && q + 1 < chain.nq) {
      float P[VEC], B[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) P[e] = 1.f;
      for (int i = 0; i <= last_wave; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) P[e] *= s_wave[i][0][lane * VEC + e];
      gather(B, at_first.eos, 0, front);
#pragma unroll
      for (int e = 0; e < VEC; ++e) put_map(chain, q, a.D, col + e, P[e], B[e]);
    }
    if (at_last.eos > last) {
      const int q0 = chain.nq - 1 - at_last.eos / kBwdTile, from = max(q0, group0);
      static_assert(NW >= kGroup, "a wave for every tile of a group");
      if (wave < q - from) {
        float P, B;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          wait_map(chain, from + wave, a.D, col + e, P, B);
          s_tile[wave][0][lane * VEC + e] = P;
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
      } else {  // the sequence ends in this tile
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
      gather(c, at_first.eos, 0, front);
#pragma unroll
      for (int e = 0; e < VEC; ++e) put_state(chain, group, a.D, col + e, c[e]);
    }
  }
  if (span_end > span_last) gather(rs, span_end, wave + 1, front);
  else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) rs[e] = 0.f;
  }
  // ---- the span's gradients
  float hp[NT][VEC], dA[VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) dA[e] = db[e] = 0.f;
  states([&](int j) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) hp[j][e] = hs[e];
  });
  grads([&](int j) {
    if (!whole && !(m.valid >> j & 1)) return;
    float x[VEC], dy[VEC], dx[VEC], dr[VEC], di[VEC];
    xk[j].get(x);
    gk[j].get(dy);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float G = dy[e] + rs[e], back = av[j][e] * G;
      float gs = G, qx = x[e];  // G s, s x
      if constexpr (GATE) gs *= s[j][e], qx *= s[j][e];
      float dg = back * hp[j][e];
      if constexpr (NORM) {
        const float ratio = w[j][e] > 0.f ? av[j][e] * __builtin_amdgcn_rcpf(w[j][e]) : 0.f;
        dg = fmaf(-back * qx, ratio, dg);
        gs *= w[j][e];
      }
      dx[e] = gs;
      if constexpr (GATE) di[e] = gs * x[e] * rest[j][e];
      dr[e] = ch[e].neg_rate2 * kLn2 * slope[j][e] * dg;
      dA[e] = fmaf(dg, g2[j][e], dA[e]);
      db[e] += dr[e];
      rs[e] = back;
    }
    if (active) {
      const int64_t off = (int64_t)(t0 + j) * a.D + col;
      piece o;
      o.set(dx);
      o.store(a.dx, off);
      o.set(dr);
      o.store(a.dr, off);
      if constexpr (GATE) {
        o.set(di);
        o.store(a.din, off);
      }
      if (a.dinit && (m.start >> j & 1)) {
        const int n = starting_at(a.seqs, m.first, t0 + j);
        if (n < a.N) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) a.dinit[(int64_t)n * a.D + col + e] = rs[e];
        }
      }
    }
  });
  if (a.zero_rest && !whole && active) {  // tokens in no sequence
    piece o;
    float zero[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) zero[e] = 0.f;
    o.set(zero);
    for (int j = 0; j < count; ++j) {
      if (m.valid >> j & 1) continue;
      const int64_t off = (int64_t)(t0 + j) * a.D + col;
      o.store(a.dx, off);
      o.store(a.dr, off);
      if constexpr (GATE) o.store(a.din, off);
    }
  }
  if (!a.part) return;
  // ---- the tile's sums, spans in order
  lds_barrier();  // the spans' maps have been read
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    s_wave[wave][0][lane * VEC + e] = dA[e] * kLn2;
    s_wave[wave][1][lane * VEC + e] = db[e];
  }
  lds_barrier();
  if (wave < 2 && active) {
    float* part = a.part + ((size_t)block * 2 + wave) * a.D + col;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) sum += s_wave[i][wave][lane * VEC + e];
      part[e] = sum;
    }
  }
}

template <typename T, int VEC, bool CK, bool GATE, bool NORM>
hipError_t run_bwd(const GlrArgs& a, void* workspace, hipStream_t stream) {
  const int nq = (a.T + kBwdTile - 1) / kBwdTile, ncol = (a.D + 64 * VEC - 1) / (64 * VEC);
  const Chain c = make_chain(workspace, nq, ncol, a.D);
  hipError_t e = launch_ready_chain(c, a.D, stream);
  if (e != hipSuccess) return e;
  const int chunks = a.dinit && (a.seqs.cu || a.T == 0) ? (a.N + kSeqs * kBwdWaves - 1) / (kSeqs * kBwdWaves) : 0;
  const int64_t blocks = (int64_t)(nq + chunks) * ncol;
  if (blocks > 0) {
    hipLaunchKernelGGL((bwd_kernel<T, VEC, CK, GATE, NORM>), dim3((unsigned)blocks), dim3(64 * kBwdWaves), 0, stream, a,
                       c, nq * ncol);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (!a.part && nq > 0) return e;
  if (!a.dA_log && !a.ddt_bias) return e;
  return launch_column_sums({a.part, {a.dA_log, a.ddt_bias}, nq, 2, a.D}, stream);
}

}  // namespace glr

// The chain, then the partial sums, then the states where none are given.
size_t glr_bwd_workspace_bytes(int T, int D, bool kept_states) {
  const int nq = (int)(((int64_t)T + glr::kBwdTile - 1) / glr::kBwdTile);
  const size_t states = kept_states ? 0 : glr::round_up((size_t)nq * D * 4);
  const size_t chain = glr::chain_bytes(nq, D), forward = kept_states ? 0 : glr_fwd_workspace_bytes(T, D);
  return (chain > forward ? chain : forward) + glr::round_up((size_t)nq * 2 * D * 4) + states;
}

hipError_t launch_glr_bwd(GlrArgs a, void* workspace, hipStream_t stream) {
  const int nq = (a.T + glr::kBwdTile - 1) / glr::kBwdTile;
  const bool kept = a.states != nullptr;
  const size_t chain = glr::chain_bytes(nq, a.D), forward = kept ? 0 : glr_fwd_workspace_bytes(a.T, a.D);
  unsigned char* p = static_cast<unsigned char*>(workspace) + (chain > forward ? chain : forward);
  a.part = a.dA_log || a.ddt_bias ? reinterpret_cast<float*>(p) : nullptr;
  if (!kept && a.T > 0) {
    a.states = reinterpret_cast<float*>(p + glr::round_up((size_t)nq * 2 * a.D * 4));
    GlrArgs f = a;
    f.y = nullptr, f.final = nullptr;
    const hipError_t e = launch_glr_fwd(f, workspace, stream);
    if (e != hipSuccess) return e;
  }
  const void* ptrs[] = {a.dy.p, a.dx, a.dr, a.din};
  const void* in[] = {a.x.p, a.r.p, a.in.p};
  return glr::with_gates(a, [&](auto gate, auto norm) {
    constexpr bool G = decltype(gate)::value, M = decltype(norm)::value;
    if (!a.bf)
      return a.packed ? glr::run_bwd<float, 1, true, G, M>(a, workspace, stream)
                      : glr::run_bwd<float, 1, false, G, M>(a, workspace, stream);
    const bool two = vector_width(2, 2, a.D | a.dy.ld, ptrs, 4) == 2 &&
                     vector_width(2, a.packed ? 1 : 2, a.x.ld | a.r.ld | a.in.ld, in, 3) == 2;
    if (a.packed)
      return two ? glr::run_bwd<bf16, 2, true, G, M>(a, workspace, stream)
                 : glr::run_bwd<bf16, 1, true, G, M>(a, workspace, stream);
    return two ? glr::run_bwd<bf16, 2, false, G, M>(a, workspace, stream)
               : glr::run_bwd<bf16, 1, false, G, M>(a, workspace, stream);
  });
}

}  // namespace kda
