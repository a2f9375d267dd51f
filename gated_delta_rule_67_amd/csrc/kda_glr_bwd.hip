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
// are computed once; what the outputs need of them and nothing in between waits in LDS, the rest in
// registers, of which a span of 8 tokens takes 156 (163 from checkpoints).
//
// Measured, calls back to back: 265 us at 4 x 8192 tokens of 2048 channels, bf16, with both gates and kept states
// (940 MB, 3.5 TB/s), 396 without those and 416 from checkpoints; 212, 312 and 320 at 4 x 8192 x 1024, float32; from
// checkpoints, 8192 x 2048 in nine sequences, 145 us, of them 52 and 5 for the states. The vector ALU is busy 57%,
// 75 instructions an element; beside the vector registers 39 to 81 scalar ones spill into lanes of others. At earlier
// steps, at the first size: without any waiting for the chain 10 us less; 4 tokens x 14 waves 310 us, 8 x 7 309, 8 x 11
// 272, against 270; the gradients, which the caches would not hold until they are read, stored past them 267 against
// 270, and from checkpoints 174 against 194.
#include <type_traits>

#include "kda_glr.h"

namespace kda {
namespace glr {

constexpr int kBwdTokens = 8, kBwdWaves = 8;
constexpr int kBwdTile = kBwdTokens * kBwdWaves;
static_assert(kBwdTile == kGlrBlock, "a tile begins at a kept state");

template <typename T, int VEC, bool CK, bool GATE, bool NORM>
__global__ __launch_bounds__(64 * (kBwdWaves + 1)) void bwd_kernel(GlrArgs a, Chain chain) {
  constexpr int NT = kBwdTokens, NW = kBwdWaves, C = 64 * VEC;
  constexpr unsigned kFull = 0xffffffffu >> (32 - NT);
  typedef Held<T, VEC, NT, CK> held;
  typedef Piece<T, VEC> piece;
  // A span's decays, its state and its gradient, each from zero, and whether a sequence ends in it; the map
  // (decays, gradient) from behind the tile to behind each span; the gradient that reaches the tile from
  // behind; a span's sums of dA_log and ddt_bias, of this turn and the one before.
  __shared__ Lanes<VEC> s_map[NW][3], s_behind[NW][2], s_front, s_sum[2][NW][2];
  __shared__ Lanes<VEC> s_held[NW][3][NT];  // what the outputs need and nothing in between (registers are scarce)
  __shared__ int s_ends[NW];
  __shared__ Tile s_next;  // the next turn's tile; first, this turn's
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, k0 = lane * VEC;
  // tiles are counted against the tokens
  auto first_token = [&](int q) { return (chain.nq - 1 - q) * kBwdTile; };

  if (wave == NW) {  // the chain wave: two barriers a turn, as in the other waves' loop
    auto find = [&](int answer) {
      Tile t;
      place_of(chain, told(answer), t.q, t.column);
      t.bos = t.eos = 0;
      if (t.q < chain.nq) {
        const Span s = around(a.seqs, min(first_token(t.q) + kBwdTile, a.T) - 1);
        t.bos = s.bos, t.eos = s.eos;
      }
      return t;
    };
    auto sums = [&](const Tile& t, int turn) {  // of a tile whose sums have been left, in order of the spans
      const int col = t.column * C + k0;
      float dA[VEC], db[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) dA[e] = db[e] = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        float u[VEC], v[VEC];
        s_sum[turn][i][0].get(lane, u);
        s_sum[turn][i][1].get(lane, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) dA[e] += u[e], db[e] += v[e];
      }
      float* out = a.part + (size_t)(chain.nq - 1 - t.q) * 2 * a.D + col;
      if (col < a.D) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) out[e] = dA[e] * kLn2, out[a.D + e] = db[e];
      }
    };
    Tile tile = find(ask(chain, true)), next = find(ask(chain, false)), before{};
    publish(&s_next, tile);
    lds_barrier();
    if (tile.q >= chain.nq) return;  // every tile is taken
    lds_barrier();
    bool later = false;
    for (int turn = 0;; turn ^= 1) {
      publish(&s_next, next);
      lds_barrier();
      const int answer = ask(chain, false);
      const int q = tile.q, last = min(first_token(q) + kBwdTile, a.T) - 1;
      const bool there = tile.column * C + k0 < a.D;
      const int col = there ? tile.column * C + k0 : a.D - VEC;
      float A[VEC], B[VEC], front[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) A[e] = 1.f, B[e] = front[e] = 0.f;
      bool ends = false;
#pragma unroll
      for (int i = NW - 1; i >= 0; --i) {
        float p[VEC], r[VEC];
        s_map[i][0].get(lane, p);
        s_map[i][2].get(lane, r);
        s_behind[i][0].set(lane, A);
        s_behind[i][1].set(lane, B);
        const bool here = s_ends[i];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          B[e] = here ? r[e] : fmaf(p[e], B[e], r[e]);
          A[e] *= p[e];
        }
        ends = ends || here;
      }
      if (chain.nq > 1) {
        if (there && q + 1 < chain.nq) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) put_map(chain, q, a.D, col + e, A[e], B[e]);
        }
        if (tile.eos > last) wait_front<VEC>(chain, q, chain.nq - 1 - tile.eos / kBwdTile, a.D, col, front);
        if (there && q + 1 < chain.nq && q % kGroup == kGroup - 1) {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            put_state(chain, q / kGroup, a.D, col + e, ends ? B[e] : fmaf(A[e], front[e], B[e]));
        }
      }
      s_front.set(lane, front);
      lds_barrier();
      const Tile after = find(answer);
      if (a.part && later) sums(before, turn ^ 1);
      before = tile;
      later = true;
      if (next.q >= chain.nq) {
        lds_barrier();
        if (a.part) sums(before, turn);
        return;
      }
      tile = next;
      next = after;
    }
  }

  struct Part {
    int t0, count, c0, col;  // c0: the wave's first channel
    bool there;
    Marks m;
  };
  auto part = [&](const Tile& t) {
    Part p;
    const int tile0 = first_token(t.q);
    p.t0 = tile0 + wave * NT;
    p.count = min(max(a.T - p.t0, 0), NT);
    p.c0 = t.column * C;
    p.col = p.c0 + k0;
    p.there = p.col < a.D;
    if (!p.there) p.col = a.D - VEC;
    if (t.bos < tile0 && t.eos >= tile0 + kBwdTile) p.m = Marks{0, 0, kFull, 0, t.bos, t.eos};
    else if (p.count > 0) p.m = marks_of(a.seqs, p.t0, p.count);
    else p.m = Marks{};
    return p;
  };
  held xk, rk, ik;
  piece gk[NT];
  float rate[VEC], bias[VEC];
  Part at;
  auto fetch = [&](const Part& p) {
    at = p;
    const float* db = a.dt_bias ? a.dt_bias : a.A_log;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      rate[e] = a.A_log[p.col + e];
      bias[e] = db[p.col + e];
    }
    const int rows = max(p.count, 1), t = min(p.t0, a.T - 1);
    const Rows rx = held::rows(a.x, t, rows, a.D), rr = held::rows(a.r, t, rows, a.D);
    const Rows ri = held::rows(GATE ? a.in : a.x, t, rows, a.D), rg = piece::rows(a.dy, t, rows, a.D);
    rk.begin(rr, rows, p.c0, a.D);
    xk.begin(rx, rows, p.c0, a.D);
    if constexpr (GATE) ik.begin(ri, rows, p.c0, a.D);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int row = min(j, rows - 1);
      rk.load(rr, j, row, p.col);
      xk.load(rx, j, row, p.col);
      if constexpr (GATE) ik.load(ri, j, row, p.col);
      gk[j].load(rg, row, p.col);
    }
  };
  lds_barrier();
  {
    const Tile first = read(&s_next);
    if (first.q >= chain.nq) return;
    lds_barrier();
    fetch(part(first));
  }
  for (int turn = 0;; turn ^= 1) {
    // Of every element: decay, and what makes the gradients from G, which the phases below complete:
    // dx = cx G, din_gate = ci G, dgate_x = cr G, dA_log's term ca G.
    float av[NT][VEC], cr[NT][VEC], ca[NT][VEC];
    float hs[VEC], rs[VEC];
    piece dy[NT];
    const Part now = at;
    const Marks& m = now.m;
    const bool whole = m.valid == kFull && !m.start && !m.end;  // inside one sequence
    // The state along the span, one token at a time: each(j) comes before token j, input(j) is w s x.
    // (inside, here and below: the span lies inside one sequence, known when compiled: no branches then)
    auto states = [&](auto inside, auto&& input, auto&& each) {
      constexpr bool W = decltype(inside)::value;
      int n = m.first;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (!W && (m.start >> j & 1)) {
          n = starting_at(a.seqs, n, now.t0 + j);
#pragma unroll
          for (int e = 0; e < VEC; ++e) hs[e] = a.init && n < a.N ? a.init[(int64_t)n * a.D + now.col + e] : 0.f;
        }
        each(j);
        if (W || (m.valid >> j & 1)) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) hs[e] = fmaf(av[j][e], hs[e], input(j, e));
        }
      }
    };
    // The gradient against the tokens: each(j) takes it over token j.
    auto grads = [&](auto inside, auto&& each) {
      constexpr bool W = decltype(inside)::value;
#pragma unroll
      for (int j = NT - 1; j >= 0; --j) {
        if (!W && (m.end >> j & 1)) {  // the walk begins at the span's first sequence each time
          const int n = ending_at(a.seqs, m.first, now.t0 + j);
#pragma unroll
          for (int e = 0; e < VEC; ++e) rs[e] = a.dfinal && n < a.N ? a.dfinal[(int64_t)n * a.D + now.col + e] : 0.f;
        }
        if (W || (m.valid >> j & 1)) each(j);
      }
    };
    // ---- the span's maps; ca holds log2 of the decay, cr the gate's slope, and:
    float b[NT][VEC], tw[NT][VEC];  // w s x; s x a / w
    auto gates = [&](auto inside) {
      constexpr bool W = decltype(inside)::value;
      Channel ch[VEC];
      float A[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) ch[e] = channel(rate[e], a.dt_bias ? bias[e] : 0.f), A[e] = 1.f, hs[e] = rs[e] = 0.f;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float rv[VEC], iv[VEC], xv[VEC], cx[VEC], ci[VEC], lg[VEC];
        dy[j] = gk[j];
        rk.get(j, rv);
        xk.get(j, xv);
        if constexpr (GATE) ik.get(j, iv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float slope, s = 1.f, rest = 0.f;
          const float g2 = decay_log2(rv[e], ch[e], slope), d = fast_exp2(g2);
          if constexpr (GATE) logistic_pair(iv[e], s, rest);
          float q = s * xv[e], w = 1.f;
          if constexpr (NORM) {
            float inv;
            w = input_weight(d, g2, inv);
            tw[j][e] = q * d * inv;
          }
          cx[e] = s * w;
          b[j][e] = q * w;
          ci[e] = b[j][e] * rest;
          cr[j][e] = ch[e].neg_rate * slope;
          lg[e] = g2;
          av[j][e] = d;
        }
        s_held[wave][2][j].set(lane, lg);
        if constexpr (GATE || NORM) s_held[wave][0][j].set(lane, cx);
        if constexpr (GATE) s_held[wave][1][j].set(lane, ci);
        if (W || (m.valid >> j & 1)) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) A[e] *= av[j][e];
        }
      }
      states(inside, [&](int j, int e) { return b[j][e]; }, [](int) {});
      grads(inside, [&](int j) {
        float d[VEC];
        dy[j].get(d);
#pragma unroll
        for (int e = 0; e < VEC; ++e) rs[e] = av[j][e] * (d[e] + rs[e]);
      });
      s_map[wave][0].set(lane, A);
      s_map[wave][1].set(lane, hs);
      s_map[wave][2].set(lane, rs);
      if (lane == 0) s_ends[wave] = m.end != 0;
    };
    whole ? gates(std::true_type{}) : gates(std::false_type{});
    lds_barrier();
    const Tile next = read(&s_next);
    // ---- the states in front of the tokens, while the chain wave waits: dg = G a (h_{t-1} - s x a / w)
    const int tile0 = now.t0 - wave * NT;
#pragma unroll
    for (int e = 0; e < VEC; ++e) hs[e] = 0.f;
    if (now.count > 0 && m.bos < now.t0) {
      const bool inside = m.bos >= tile0;
      int i = inside ? (m.bos - tile0) / NT : 0;
      if (inside) s_map[i][1].get(lane, hs);
      else
#pragma unroll
        for (int e = 0; e < VEC; ++e) hs[e] = a.states[(int64_t)(tile0 / kBwdTile) * a.D + now.col + e];
      for (i += inside; i < wave; ++i) {
        float p[VEC], h[VEC];
        s_map[i][0].get(lane, p);
        s_map[i][1].get(lane, h);
#pragma unroll
        for (int e = 0; e < VEC; ++e) hs[e] = fmaf(p[e], hs[e], h[e]);
      }
    }
    auto slopes = [&](auto inside) {
      states(inside, [&](int j, int e) { return b[j][e]; }, [&](int j) {
        float lg[VEC];
        s_held[wave][2][j].get(lane, lg);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float d = hs[e];
          if constexpr (NORM) d -= tw[j][e];
          d *= av[j][e];
          cr[j][e] *= d;
          ca[j][e] = lg[e] * d;
        }
      });
    };
    whole ? slopes(std::true_type{}) : slopes(std::false_type{});
    // (row 0 where no tile is left: the registers are then not the old values' any more)
    const bool more = next.q < chain.nq;
    Part p;
    p.t0 = 0, p.count = 1, p.c0 = 0, p.col = min(k0, a.D - VEC), p.there = false, p.m = Marks{};
    if (more) p = part(next);
    fetch(p);
    lds_barrier();
    // ---- gradients
    float dA[VEC], db[VEC];
    {
      float A[VEC], B[VEC], front[VEC];
      s_front.get(lane, front);
      s_behind[wave][0].get(lane, A);
      s_behind[wave][1].get(lane, B);
      const int span_last = now.t0 + now.count - 1, last = min(tile0 + kBwdTile, a.T) - 1;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        rs[e] = now.count == 0 || m.eos <= span_last ? 0.f : m.eos <= last ? B[e] : fmaf(A[e], front[e], B[e]);
        dA[e] = db[e] = 0.f;
      }
    }
    const Rows ox = piece::rows(a.dx, a.D, now.t0, now.count, a.D), orr = piece::rows(a.dr, a.D, now.t0, now.count, a.D);
    const Rows oi = piece::rows(GATE ? a.din : a.dx, a.D, now.t0, now.count, a.D);
    auto outputs = [&](auto inside) {
     grads(inside, [&](int j) {
      float d[VEC], dx[VEC], dr[VEC], di[VEC], cx[VEC], ci[VEC];
      dy[j].get(d);
      if constexpr (GATE || NORM) s_held[wave][0][j].get(lane, cx);
      if constexpr (GATE) s_held[wave][1][j].get(lane, ci);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float G = d[e] + rs[e];
        dx[e] = GATE || NORM ? cx[e] * G : G;
        if constexpr (GATE) di[e] = ci[e] * G;
        dr[e] = cr[j][e] * G;
        dA[e] = fmaf(ca[j][e], G, dA[e]);
        db[e] += dr[e];
        rs[e] = av[j][e] * G;
      }
      if (now.there) {
        piece o;
        o.set(dx);
        o.template store<true>(ox, j, now.col);
        o.set(dr);
        o.template store<true>(orr, j, now.col);
        if constexpr (GATE) {
          o.set(di);
          o.template store<true>(oi, j, now.col);
        }
        if (!decltype(inside)::value && a.dinit && (m.start >> j & 1)) {
          const int n = starting_at(a.seqs, m.first, now.t0 + j);
          if (n < a.N) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) a.dinit[(int64_t)n * a.D + now.col + e] = rs[e];
          }
        }
      }
     });
    };
    whole ? outputs(std::true_type{}) : outputs(std::false_type{});
    if (a.zero_rest && !whole && now.there) {  // tokens in no sequence
      piece o;
      float zero[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) zero[e] = 0.f;
      o.set(zero);
      for (int j = 0; j < now.count; ++j) {
        if (m.valid >> j & 1) continue;
        o.template store<true>(ox, j, now.col);
        o.template store<true>(orr, j, now.col);
        if constexpr (GATE) o.template store<true>(oi, j, now.col);
      }
    }
    s_sum[turn][wave][0].set(lane, dA);
    s_sum[turn][wave][1].set(lane, db);
    if (!more) break;
  }
  lds_barrier();
}

template <typename T, int VEC, bool CK, bool GATE, bool NORM>
hipError_t run_bwd(const GlrArgs& a, void* workspace, hipStream_t stream) {
  const Chain c = make_chain(a, workspace, kBwdTile, 64 * VEC);
  hipError_t e = launch_ready(a, c, a.dfinal, a.dinit, stream);
  if (e != hipSuccess) return e;
  if (c.nq > 0) {
    hipLaunchKernelGGL((bwd_kernel<T, VEC, CK, GATE, NORM>), dim3(chain_blocks(c)), dim3(64 * (kBwdWaves + 1)), 0, stream,
                       a, c);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (!a.dA_log && !a.ddt_bias) return e;
  return launch_column_sums({a.part, {a.dA_log, a.ddt_bias}, c.nq, 2, a.D}, stream);
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
