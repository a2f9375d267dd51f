// Gated linear recurrence with one state per channel, forward, and its one-token step.
//
//   g_t = -exp(A_log) softplus(gate_x_t + dt_bias),  a_t = exp(g_t)       (the standard decay gate)
//   h_t = a_t h_{t-1} + w_t logistic(in_gate_t) x_t,  w_t = sqrt(1 - a_t^2) or 1;   y_t = h_t
//
// 38 instructions of the vector ALU an element, six of them transcendental (which take twice the others'
// time), and 8 bytes in bf16: the vector ALU is busy 65% of the time, memory moves 4.2 TB/s, so the gates are
// computed once and every tensor moves once. A wave holds a span of tokens for 64 VEC channels: the states
// from zero in registers, and in LDS the products of decays with which the state in front of the span
// enters them. That state comes through the waves of the workgroup and the chain of tiles (kda_glr.h); the
// chain's waiting is covered by the next tile, whose loads are under way and whose states from zero are
// computed before the outputs of this one (without any waiting the kernel would take 3 us less).
//
// Measured, calls back to back: 127 us at 4 x 8192 tokens of 2048 channels, bf16, with both gates (537 MB; loads and
// stores alone, of the same sizes in the same order, take 100 us; with block_states 126 to 129). Traced, kernels
// apart, 139 and 5.4 for the one that readies the chain. 115 us at 4 x 8192 x 1024, 79 us at 16391 packed tokens of
// 1030 channels, float32: there rows are 4120 bytes apart, a wave's 256 bytes mostly straddle a third line, and 281 MB
// are read for 203; the vector ALU is busy 35%. Tiles loaded one ahead instead of two, at an earlier step: 139 us
// instead of 136 at the first size. y is stored through the caches: the layer's next operator reads it.
#include <type_traits>

#include "kda_glr.h"

namespace kda {
namespace glr {

constexpr int kReadyThreads = 256;

// A thread clears 16 bytes of the chain or copies a channel of a sequence without tokens.
__global__ __launch_bounds__(kReadyThreads) void ready_kernel(GlrArgs a, Chain c, int64_t words, const float* from, float* to,
                                                              int64_t channels) {
  int64_t i = (int64_t)blockIdx.x * kReadyThreads + threadIdx.x;
  if (c.nq > 1 && i == 0) *c.ticket = 0;
  // the maps and the states lie behind each other
  if (i < words) reinterpret_cast<uint4*>(c.map)[i] = make_uint4(kAbsent, kAbsent, kAbsent, kAbsent);
  if (i < channels) {
    const int n = (int)(i / a.D);
    int bos = 0, eos = 0;  // T = 0: none has tokens
    if (a.seqs.cu) {
      bos = min(max(a.seqs.cu[n], 0), a.T);
      eos = min(max(a.seqs.cu[n + 1], bos), a.T);
    }
    if (eos == bos) to[i] = from ? from[i] : 0.f;
  }
}

hipError_t launch_ready(const GlrArgs& a, const Chain& c, const float* from, float* to, hipStream_t stream) {
  const int64_t words = c.nq <= 1 ? 0 : (int64_t)(chain_bytes(c.nq, a.D) - 256) / 16;
  const int64_t channels = to && (a.seqs.cu || a.T == 0) ? (int64_t)a.N * a.D : 0;
  const int64_t n = words > channels ? words : channels;
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(ready_kernel, dim3((unsigned)((n + kReadyThreads - 1) / kReadyThreads)), dim3(kReadyThreads), 0,
                     stream, a, c, words, from, to, channels);
  return hipGetLastError();
}

// A wave's span and the spans of a tile, one workgroup a CU with the chain's wave as its sixteenth. At the
// first size above, with one tile ahead: 8 tokens x 15 waves 137 us, x 14 148, x 11 150, x 8 158; 16 x 7 153;
// four channels a lane, 4 x 15, 220. A checkpoint's codes are a byte each: four channels a lane there keep
// the loads 4 bytes wide (states of 8192 x 2048 for the backward pass, which takes 144 us with them and 147
// with two channels a lane; 20 bytes a lane go to scratch).
template <int VEC> struct FwdTile {
  static constexpr int kTokens = VEC == 4 ? 4 : 8, kWaves = 15, kTile = kTokens * kWaves;
  static_assert(kGlrBlock % kTokens == 0, "a block's first token begins a span");
};

template <typename T, int VEC, bool CK, bool GATE, bool NORM>
__global__ __launch_bounds__(64 * (FwdTile<VEC>::kWaves + 1)) void fwd_kernel(GlrArgs a, Chain chain) {
  constexpr int NT = FwdTile<VEC>::kTokens, NW = FwdTile<VEC>::kWaves, kFwdTile = NT * NW, C = 64 * VEC;
  typedef Held<T, VEC, NT, CK> held;
  // Of this turn's tile and of the one before: the spans' maps, which the chain wave replaces by the maps
  // from the tile's front to each span's, and whether a sequence begins in them; the state in front of the
  // tile; the products of decays (the last of a span is in registers too).
  __shared__ Lanes<VEC> s_map[2][NW][2], s_front[2], s_decay[2][NW][NT - 1];
  __shared__ int s_begins[2][NW];
  __shared__ Tile s_next[2];  // the tile of the turn after next; first, those of the first two
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, k0 = lane * VEC;

  if (wave == NW) {  // the chain wave: one barrier a turn, an even number of turns, as in the other waves' loop
    auto find = [&](int answer) {
      Tile t;
      place_of(chain, told(answer), t.q, t.column);
      const Span s = t.q < chain.nq ? around(a.seqs, t.q * kFwdTile) : Span{0, 0};
      t.bos = s.bos, t.eos = s.eos;
      return t;
    };
    Tile tile = find(ask(chain, true)), next = find(ask(chain, false)), later = find(ask(chain, false));
    publish(&s_next[0], tile);
    publish(&s_next[1], next);
    lds_barrier();
    if (tile.q >= chain.nq) return;  // every tile is taken
    lds_barrier();                   // both have been read
    for (int turn = 0;; turn ^= 1) {
      publish(&s_next[turn], later);
      lds_barrier();
      Tile after{chain.nq, 0, 0, 0};
      if (tile.q < chain.nq) {
        const int answer = ask(chain, false);
        const int q = tile.q, tile0 = q * kFwdTile;
        const bool there = tile.column * C + k0 < a.D;
        const int col = there ? tile.column * C + k0 : a.D - VEC;
        float A[VEC], B[VEC], front[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) A[e] = 1.f, B[e] = front[e] = 0.f;
        bool begins = false;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          float p[VEC], h[VEC];
          s_map[turn][i][0].get(lane, p);
          s_map[turn][i][1].get(lane, h);
          s_map[turn][i][0].set(lane, A);
          s_map[turn][i][1].set(lane, B);
          const bool here = s_begins[turn][i];
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            B[e] = here ? h[e] : fmaf(p[e], B[e], h[e]);
            A[e] *= p[e];
          }
          begins = begins || here;
        }
        if (chain.nq > 1) {
          if (there && q + 1 < chain.nq) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) put_map(chain, q, a.D, col + e, A[e], B[e]);
          }
          after = find(answer);  // while the other workgroups' maps are on their way
          if (tile.bos < tile0) wait_front<VEC>(chain, q, tile.bos / kFwdTile, a.D, col, front);
          if (there && q + 1 < chain.nq && q % kGroup == kGroup - 1) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
              put_state(chain, q / kGroup, a.D, col + e, begins ? B[e] : fmaf(A[e], front[e], B[e]));
          }
        }
        s_front[turn].set(lane, front);
      }
      if (turn && next.q >= chain.nq) break;
      tile = next;
      next = later;
      later = after;
    }
    lds_barrier();
    return;
  }

  // This wave's part of a tile: first token (-1: no tile), column, and whether the tile lies inside one sequence
  // that begins in front of it and ends behind it. The rest follows where it is needed: scalar registers are scarce.
  struct Part {
    int t0, column;
    bool whole;
  };
  auto part = [&](const Tile& t) {
    const int tile0 = t.q * kFwdTile;
    if (t.q >= chain.nq) return Part{-1, 0, true};
    return Part{tile0 + wave * NT, t.column, t.bos < tile0 && t.eos >= tile0 + kFwdTile};
  };
  auto tokens = [&](const Part& p) { return min(max(a.T - p.t0, 0), NT); };
  auto channel_of = [&](const Part& p) { return p.column * C + k0; };  // D and more: none (D is a multiple of VEC)
  auto marks = [&](const Part& p) {  // of a part that is not whole
    const int n = p.t0 < 0 ? 0 : tokens(p);
    return n > 0 ? marks_of(a.seqs, p.t0, n) : Marks{};
  };
  // A part's inputs: two of these take turns, so that a tile's loads are under way while the one in front
  // of it is worked on.
  struct Raw {
    held x, r, in;
    float rate[VEC], bias[VEC];  // A_log and dt_bias
    Part at;
  };
  // Loads are issued where no tile is left, too (of row 0): a wave waits for its loads by counting the ones behind
  // them, and where some might not be there, on any way through its loop, it would wait for all.
  auto fetch = [&](Raw& w, const Part& p) {
    w.at = p;
    const int col = min(channel_of(p), a.D - VEC);
    const float* bias = a.dt_bias ? a.dt_bias : a.A_log;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w.rate[e] = a.A_log[col + e];
      w.bias[e] = bias[col + e];
    }
    // rows that are there: the last one again behind the last token
    const int t = min(max(p.t0, 0), a.T - 1), rows = min(a.T - t, NT);
    const Rows rx = held::rows(a.x, t, rows, a.D), rr = held::rows(a.r, t, rows, a.D);
    const Rows ri = held::rows(GATE ? a.in : a.x, t, rows, a.D);
    w.r.begin(rr, rows, p.column * C, a.D);
    w.x.begin(rx, rows, p.column * C, a.D);
    if constexpr (GATE) w.in.begin(ri, rows, p.column * C, a.D);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int row = min(j, rows - 1);
      w.r.load(rr, j, row, col);
      w.x.load(rx, j, row, col);
      if constexpr (GATE) w.in.load(ri, j, row, col);
    }
  };
  // A span's states from zero in front of it, the product of its decays, and where it lies.
  struct Local {
    float h[NT][VEC], decay[VEC];
    Part at;
  };
  auto local = [&](const Raw& w, Local& l, int turn) {
    l.at = w.at;
    bool begins = false;
    Channel ch[VEC];
    float hs[VEC], ps[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) ch[e] = channel(w.rate[e], a.dt_bias ? w.bias[e] : 0.f), hs[e] = 0.f, ps[e] = 1.f;
    auto token = [&](int j, float (&av)[VEC], float (&bv)[VEC]) {
      float xv[VEC], rv[VEC], iv[VEC];
      w.x.get(j, xv);
      w.r.get(j, rv);
      if constexpr (GATE) w.in.get(j, iv);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float b = xv[e];
        const float g2 = decay_log2(rv[e], ch[e]);
        av[e] = fast_exp2(g2);
        if constexpr (GATE) b *= sigmoid_fast(iv[e]);
        if constexpr (NORM) b *= input_weight(av[e], g2);
        bv[e] = b;
      }
    };
    if (l.at.whole) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float av[VEC], bv[VEC];
        token(j, av, bv);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          l.h[j][e] = hs[e] = fmaf(av[e], hs[e], bv[e]);
          ps[e] *= av[e];
        }
        if (j < NT - 1) s_decay[turn][wave][j].set(lane, ps);
      }
    } else {
      const Marks m = marks(l.at);
      const int col = min(channel_of(l.at), a.D - VEC);
      begins = m.start != 0;
      int n = m.first;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float av[VEC], bv[VEC];
        token(j, av, bv);
        if (m.start >> j & 1) {
          n = starting_at(a.seqs, n, l.at.t0 + j);
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
        for (int e = 0; e < VEC; ++e) l.h[j][e] = hs[e];
        if (j < NT - 1) s_decay[turn][wave][j].set(lane, ps);
      }
    }
    s_map[turn][wave][0].set(lane, ps);
    s_map[turn][wave][1].set(lane, hs);
#pragma unroll
    for (int e = 0; e < VEC; ++e) l.decay[e] = ps[e];
    if (lane == 0) s_begins[turn][wave] = begins;
  };
  // Outputs of a tile, once the chain wave knows what is in front of it.
  auto finish = [&](Local& l, int turn) {
    const Part& at = l.at;
    const int col = channel_of(at);
    if (at.t0 < 0 || at.t0 >= a.T || col >= a.D) return;
    float c[VEC], A[VEC], B[VEC];
    s_front[turn].get(lane, c);
    s_map[turn][wave][0].get(lane, A);
    s_map[turn][wave][1].get(lane, B);
    const Rows y = Piece<T, VEC>::rows(a.y, a.D, at.t0, tokens(at), a.D);
    auto keep = [&] {
      if (a.states && at.t0 % kGlrBlock == 0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) a.states[(int64_t)(at.t0 / kGlrBlock) * a.D + col + e] = c[e];
      }
    };
    auto decays = [&](int j, float (&p)[VEC]) {
      if (j < NT - 1) s_decay[turn][wave][j].get(lane, p);
      else
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[e] = l.decay[e];
    };
    if (at.whole) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) c[e] = fmaf(A[e], c[e], B[e]);
      keep();
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float p[VEC];
        decays(j, p);
#pragma unroll
        for (int e = 0; e < VEC; ++e) l.h[j][e] = fmaf(p[e], c[e], l.h[j][e]);
      }
      if (a.y) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          Piece<T, VEC> o;
          o.set(l.h[j]);
          o.store(y, j, col);
        }
      }
      return;
    }
    const Marks m = marks(at);
    const bool inside = m.bos >= at.t0 - wave * NT;  // the sequence in front of the span began in this tile
#pragma unroll
    for (int e = 0; e < VEC; ++e) c[e] = m.bos >= at.t0 ? 0.f : inside ? B[e] : fmaf(A[e], c[e], B[e]);
    keep();
    const int count = tokens(at);
    unsigned begun = 0;  // a sequence has begun in the span
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      begun |= m.start >> j & 1;
      const bool lies = m.valid >> j & 1;
      float p[VEC];
      decays(j, p);
#pragma unroll
      for (int e = 0; e < VEC; ++e) l.h[j][e] = !lies ? 0.f : begun ? l.h[j][e] : fmaf(p[e], c[e], l.h[j][e]);
      if (a.y && j < count && (lies || a.zero_rest)) {
        Piece<T, VEC> o;
        o.set(l.h[j]);
        o.store(y, j, col);
      }
    }
    if (!a.final) return;
    int n = m.first;
    for (unsigned left = m.end; left; left &= left - 1) {
      const int last = __builtin_ctz(left);
      n = ending_at(a.seqs, n, at.t0 + last);
      if (n >= a.N) break;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (j == last) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) a.final[(int64_t)n * a.D + col + e] = l.h[j][e];
        }
    }
  };
  // A turn: the states of its tile from zero, then, behind the barrier, the outputs of the tile before and the loads
  // of the tile after next. Turns come in pairs (see fetch).
  Local before;
  before.at.t0 = -1;
  auto step = [&](Raw& w, int turn) {
    Local now;
    local(w, now, turn);
    lds_barrier();
    const Tile t = read(&s_next[turn]);
    finish(before, turn ^ 1);
    before = now;
    fetch(w, part(t));
  };
  lds_barrier();
  const Tile t0 = read(&s_next[0]), t1 = read(&s_next[1]);
  if (t0.q >= chain.nq) return;
  lds_barrier();
  Raw even, odd;
  fetch(even, part(t0));
  fetch(odd, part(t1));
  do {
    step(even, 0);
    step(odd, 1);
  } while (even.at.t0 >= 0);
  lds_barrier();
  finish(before, 1);
}

template <typename T, int VEC, bool CK, bool GATE, bool NORM>
hipError_t run_fwd(const GlrArgs& a, void* workspace, hipStream_t stream) {
  const Chain c = make_chain(a, workspace, FwdTile<VEC>::kTile, 64 * VEC);
  const hipError_t e = launch_ready(a, c, a.init, a.final, stream);
  if (e != hipSuccess || c.nq == 0) return e;
  hipLaunchKernelGGL((fwd_kernel<T, VEC, CK, GATE, NORM>), dim3(chain_blocks(c)), dim3(64 * (FwdTile<VEC>::kWaves + 1)), 0, stream, a, c);
  return hipGetLastError();
}

// One token of B requests on slots of a pool of states: 16 bytes an element in bf16, 1.4 us of HBM's time
// for 256 requests of 2048 channels. The kernel takes 4.1 us, 9.7 with its launch.
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
      float b = xv[e];
      const float g2 = decay_log2(rv[e], channel(a, col + e)), av = fast_exp2(g2);
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

size_t glr_fwd_workspace_bytes(int T, int D) {  // for the shortest tiles
  constexpr int tile = glr::FwdTile<4>::kTile;
  static_assert(tile <= glr::FwdTile<2>::kTile && tile <= glr::FwdTile<1>::kTile, "the shortest tiles");
  return glr::chain_bytes((int)(((int64_t)T + tile - 1) / tile), D);
}

hipError_t launch_glr_fwd(GlrArgs a, void* workspace, hipStream_t stream) {
  const void* ptrs[] = {a.x.p, a.r.p, a.in.p, a.y};
  return glr::with_gates(a, [&](auto gate, auto norm) {
    constexpr bool G = decltype(gate)::value, M = decltype(norm)::value;
    if (a.packed) {  // states in front of the blocks of a checkpointed call: no outputs of type T
      if (vector_width(4, 1, a.D, ptrs, 3) == 4) return glr::run_fwd<bf16, 4, true, G, M>(a, workspace, stream);
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
