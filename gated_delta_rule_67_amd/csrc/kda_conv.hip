// Short causal depthwise convolution over the tokens of each sequence, its backward, and its
// one-token step on a state.
//
// The layer in front of the recurrence (the KDA CUDA Trainer README's model paragraph: q, k and v
// pass a short convolution; the DM-KDAGQA-1.7B-SD model card's usage notes: generation keeps "the
// KDA recurrent and conv states"). Per channel d, width W, taps w, in float32:
//   pre_t = bias + sum_w weight[w] x_{t - (W-1) + w},    y_t = pre_t logistic(pre_t)  or  pre_t
// where the W - 1 rows before a sequence's first token are its initial state (or zeros). Backward,
// with s = logistic(pre) and dpre_t = dy_t s (1 + pre (1 - s)):
//   dx_r       = sum_k weight[W-1-k] dpre_{r+k}   over tokens r + k of the same sequence
//   dweight[w] = sum_t dpre_t x_{t - (W-1) + w},  dbias = sum_t dpre_t
// and the gradient of the initial state is dx of the rows before the first token.
//
// Both directions stream their tensors once (2W + 5 operations an element forward, about three
// times that backward) and are bound by HBM. A lane owns VEC channels (16 bytes where D, the row
// strides and the pointers allow) and walks consecutive rows with the last W - 1 rows in
// registers, so a row is read once, apart from the W - 1 rows in front of a wave's first one.
// Rows are split over waves and workgroups without regard to sequences: the branches at a
// sequence's ends are uniform over the wave.
#include "kda_sequence.h"

namespace kda {
namespace conv {

constexpr int kThreads = 256;
constexpr int kLanes = 64;                  // column vectors of a workgroup, one per lane
constexpr int kSlices = kThreads / kLanes;  // its waves take consecutive slices of the row block
constexpr int kMinRows = 4;                 // rows of a slice at least: fewer would mostly read its halo
constexpr int kRows = 4;                    // rows whose loads are issued before any is used

template <typename T, int VEC> struct Row {
  typedef T type __attribute__((ext_vector_type(VEC)));
};
template <typename T> struct Row<T, 1> { typedef T type; };

template <typename T, int VEC> using row_t = typename Row<T, VEC>::type;

template <typename T, int VEC>
__device__ __forceinline__ float at(const row_t<T, VEC>& v, int e) {
  if constexpr (VEC == 1) return to_f32(v);
  else return to_f32(v[e]);
}

template <typename T, int VEC>
__device__ __forceinline__ void put(row_t<T, VEC>& v, int e, float x) {
  if constexpr (VEC == 1) v = from_f32<T>(x);
  else v[e] = from_f32<T>(x);
}

struct Args {
  const void* x;
  int64_t ldx;         // elements between rows of x
  const float* weight; // [D, W]
  const float* bias;   // [D] or null
  const void* init;    // [N, W-1, D] or null
  Sequences seqs;
  int N, T, D;
  int silu, zero_rest;
  int64_t rpb;         // rows per row block
  int nrb;             // row blocks; the blocks behind them handle the sequences' states
  void* out_state;     // forward: final state, or null; backward: gradient of init, or null
  const void* dy;      // backward
  int64_t lddy;
  const void* dfinal;  // backward: gradient reaching the final state, or null
  void* out;           // y, or dx
  float* part;         // backward: partial sums [nrb][(W + 1) D]: taps, then bias
};

__device__ __forceinline__ float logistic(float x) {
  return __builtin_amdgcn_rcpf(1.f + fast_exp2(-x * kLog2e));
}

// This lane's VEC channels' taps and bias.
template <int VEC, int W>
__device__ __forceinline__ void load_taps(const Args& a, int col, float (&w)[W][VEC], float (&b)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][e] = a.weight[(size_t)(col + e) * W + k];
    b[e] = a.bias ? a.bias[col + e] : 0.f;
  }
}

// The row at place v of (state ; sequence): a row of the initial state, or token bos + v - (W-1).
template <typename T, int VEC, int W>
__device__ __forceinline__ row_t<T, VEC> state_or_token(const Args& a, int seq, int bos, int v, int col) {
  typedef row_t<T, VEC> vec_t;
  if (v >= W - 1)
    return *reinterpret_cast<const vec_t*>(static_cast<const T*>(a.x) + (int64_t)(bos + v - (W - 1)) * a.ldx + col);
  if (a.init)
    return *reinterpret_cast<const vec_t*>(static_cast<const T*>(a.init) + ((int64_t)seq * (W - 1) + v) * a.D + col);
  return vec_t{};
}

// Rows [r, end) lie in no sequence: zeros where the caller asks for them.
template <typename T, int VEC>
__device__ __forceinline__ void outside(const Args& a, int r, int end, int col) {
  if (!a.zero_rest) return;
  for (; r < end; ++r)
    *reinterpret_cast<row_t<T, VEC>*>(static_cast<T*>(a.out) + (int64_t)r * a.D + col) = row_t<T, VEC>{};
}

// Forward. grid.x: column blocks, grid.y: row blocks, then blocks of sequences (final states).
template <typename T, int VEC, int W, bool SILU>
__global__ __launch_bounds__(kThreads) void fwd_kernel(Args a) {
  typedef row_t<T, VEC> vec_t;
  const int lane = threadIdx.x % kLanes, slice = threadIdx.x / kLanes;
  const int col = (blockIdx.x * kLanes + lane) * VEC;
  const bool active = col < a.D;  // D % VEC == 0
  if ((int)blockIdx.y >= a.nrb) {  // final states: the last W - 1 rows of (state ; sequence)
    const int n = ((int)blockIdx.y - a.nrb) * kSlices + slice;
    if (n >= a.N || !active) return;
    const Span s = a.seqs.span(n);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      *reinterpret_cast<vec_t*>(static_cast<T*>(a.out_state) + ((int64_t)n * (W - 1) + j) * a.D + col) =
          state_or_token<T, VEC, W>(a, n, s.bos, s.eos - s.bos + j, col);
    return;
  }
  const int rb0 = (int)((int64_t)blockIdx.y * a.rpb);
  const int rb1 = (int)min((int64_t)rb0 + a.rpb, (int64_t)a.T);
  const int q = (rb1 - rb0 + kSlices - 1) / kSlices;
  int r = rb0 + slice * q;
  const int r1 = min(r + q, rb1);
  if (r >= r1) return;
  int seq = a.seqs.find(r);  // uses every lane of the wave
  if (!active) return;
  float w[W][VEC], b[VEC];
  load_taps<VEC, W>(a, col, w, b);
  const T* x = static_cast<const T*>(a.x) + col;
  T* y = static_cast<T*>(a.out) + col;
  while (r < r1 && seq < a.N) {
    const Span s = a.seqs.span(seq);
    if (s.eos <= r) { ++seq; continue; }
    if (s.bos > r) {  // rows in front of the first sequence
      outside<T, VEC>(a, r, min(s.bos, r1), col);
      r = s.bos;
      continue;
    }
    // the W - 1 rows in front of row r
    float win[W - 1][VEC];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const vec_t v = state_or_token<T, VEC, W>(a, seq, s.bos, r - s.bos + k, col);
#pragma unroll
      for (int e = 0; e < VEC; ++e) win[k][e] = at<T, VEC>(v, e);
    }
    auto row = [&](const vec_t& xv, T* out) {
      vec_t yv;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float xe = at<T, VEC>(xv, e);
        float pre = b[e];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) pre = fmaf(w[k][e], win[k][e], pre);
        pre = fmaf(w[W - 1][e], xe, pre);
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) win[k][e] = win[k + 1][e];
        win[W - 2][e] = xe;
        put<T, VEC>(yv, e, SILU ? pre * logistic(pre) : pre);
      }
      *reinterpret_cast<vec_t*>(out) = yv;  // cached: the recurrence reads it next
    };
    const int end = min(s.eos, r1);
    const T* xp = x + (int64_t)r * a.ldx;
    T* yp = y + (int64_t)r * a.D;
    for (; r + kRows <= end; r += kRows) {
      vec_t xv[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) xv[u] = *reinterpret_cast<const vec_t*>(xp + u * a.ldx);
#pragma unroll
      for (int u = 0; u < kRows; ++u) row(xv[u], yp + (int64_t)u * a.D);
      xp += kRows * a.ldx;
      yp += (int64_t)kRows * a.D;
    }
    for (; r < end; ++r, xp += a.ldx, yp += a.D) row(*reinterpret_cast<const vec_t*>(xp), yp);
    ++seq;
  }
  outside<T, VEC>(a, r, r1, col);
}

// Backward, stage 1: dx, the gradient of the initial states, and partial sums of dweight and
// dbias. A wave walks its rows t in order; with the W - 1 latest dpre in registers, the row
// W - 1 places before t gets its whole sum at t. A wave whose slice ends inside a sequence walks
// up to W - 1 rows further (recomputing their dpre, leaving them out of the sums), and one whose
// slice starts inside a sequence leaves the rows before its slice to the wave before it; a row is
// therefore written once, always by the wave whose slice holds it (rows of the initial state: by
// the wave that holds the sequence's first token).
template <typename T, int VEC, int W, bool SILU>
__global__ __launch_bounds__(kThreads) void bwd_kernel(Args a) {
  typedef row_t<T, VEC> vec_t;
  __shared__ float s_sum[kSlices][W + 1][VEC][kLanes];
  const int lane = threadIdx.x % kLanes, slice = threadIdx.x / kLanes;
  const int col = (blockIdx.x * kLanes + lane) * VEC;
  const bool active = col < a.D;
  if ((int)blockIdx.y >= a.nrb) {  // empty sequences: the state's gradient passes through
    const int n = ((int)blockIdx.y - a.nrb) * kSlices + slice;
    if (n >= a.N || !active) return;
    const Span s = a.seqs.span(n);
    if (s.eos > s.bos) return;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int64_t off = ((int64_t)n * (W - 1) + j) * a.D + col;
      *reinterpret_cast<vec_t*>(static_cast<T*>(a.out_state) + off) =
          a.dfinal ? *reinterpret_cast<const vec_t*>(static_cast<const T*>(a.dfinal) + off) : vec_t{};
    }
    return;
  }
  float dw[W][VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
#pragma unroll
    for (int k = 0; k < W; ++k) dw[k][e] = 0.f;
    db[e] = 0.f;
  }
  const int rb0 = (int)((int64_t)blockIdx.y * a.rpb);
  const int rb1 = (int)min((int64_t)rb0 + a.rpb, (int64_t)a.T);
  const int q = (rb1 - rb0 + kSlices - 1) / kSlices;
  int r = min(rb0 + slice * q, rb1);
  const int r1 = min(r + q, rb1);
  int seq = r < r1 ? a.seqs.find(r) : a.N;
  if (active && r < r1) {
    float w[W][VEC], b[VEC];
    load_taps<VEC, W>(a, col, w, b);
    const T* x = static_cast<const T*>(a.x) + col;
    const T* dy = static_cast<const T*>(a.dy) + col;
    while (r < r1 && seq < a.N) {
      const Span s = a.seqs.span(seq);
      if (s.eos <= r) { ++seq; continue; }
      if (s.bos > r) {
        outside<T, VEC>(a, r, min(s.bos, r1), col);
        r = s.bos;
        continue;
      }
      const int first = r == s.bos ? s.bos - (W - 1) : r;
      const int own = min(s.eos, r1);  // tokens [r, own) enter the sums, rows [first, own) are written
      float win[W - 1][VEC], dp[W - 1][VEC];  // x, and dpre, of the W - 1 rows before t
#pragma unroll
      for (int k = 0; k < W - 1; ++k) {
        const vec_t v = state_or_token<T, VEC, W>(a, seq, s.bos, r - s.bos + k, col);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          win[k][e] = at<T, VEC>(v, e);
          dp[k][e] = 0.f;
        }
      }
      // row `row` (a token, or a row of the initial state below s.bos) with its sum
      auto emit = [&](int row, const float (&sum)[VEC]) {
        vec_t o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) put<T, VEC>(o, e, sum[e]);
        if (row >= s.bos)
          __builtin_nontemporal_store(o, reinterpret_cast<vec_t*>(static_cast<T*>(a.out) + (int64_t)row * a.D + col));
        else if (a.out_state)
          *reinterpret_cast<vec_t*>(static_cast<T*>(a.out_state) + ((int64_t)seq * (W - 1) + row - s.bos + W - 1) * a.D + col) = o;
      };
      // dpre of a token (into the sums if it is this wave's); the sum of the row W - 1 places before it
      auto token = [&](const vec_t& xv, const vec_t& gv, bool mine, float (&sum)[VEC]) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xe = at<T, VEC>(xv, e);
          float d = at<T, VEC>(gv, e);
          if constexpr (SILU) {
            float pre = b[e];
#pragma unroll
            for (int k = 0; k < W - 1; ++k) pre = fmaf(w[k][e], win[k][e], pre);
            pre = fmaf(w[W - 1][e], xe, pre);
            const float sg = logistic(pre);
            d *= fmaf(pre * sg, 1.f - sg, sg);
          }
          if (mine) {
#pragma unroll
            for (int k = 0; k < W - 1; ++k) dw[k][e] = fmaf(d, win[k][e], dw[k][e]);
            dw[W - 1][e] = fmaf(d, xe, dw[W - 1][e]);
            db[e] += d;
          }
          float o = w[0][e] * d;
#pragma unroll
          for (int k = 0; k < W - 1; ++k) o = fmaf(w[W - 1 - k][e], dp[k][e], o);
          sum[e] = o;
#pragma unroll
          for (int k = 0; k + 1 < W - 1; ++k) {
            win[k][e] = win[k + 1][e];
            dp[k][e] = dp[k + 1][e];
          }
          win[W - 2][e] = xe;
          dp[W - 2][e] = d;
        }
      };
      const int stop = min(s.eos, own + (W - 1));
      const T* xp = x + (int64_t)r * a.ldx;
      const T* gp = dy + (int64_t)r * a.lddy;
      int t = r;
      auto single = [&] {
        float sum[VEC];
        token(*reinterpret_cast<const vec_t*>(xp), *reinterpret_cast<const vec_t*>(gp), t < own, sum);
        if (t - (W - 1) >= first) emit(t - (W - 1), sum);
        ++t, xp += a.ldx, gp += a.lddy;
      };
      const int head = min(r + W - 1, stop);  // tokens whose row is the state's, or the wave's before
      while (t < head) single();
      T* op = static_cast<T*>(a.out) + (int64_t)(t - (W - 1)) * a.D + col;
      for (; t + kRows <= own; t += kRows) {  // all of them this wave's, and their rows too
        vec_t xv[kRows], gv[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          xv[u] = __builtin_nontemporal_load(reinterpret_cast<const vec_t*>(xp + u * a.ldx));
          gv[u] = __builtin_nontemporal_load(reinterpret_cast<const vec_t*>(gp + u * a.lddy));
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          float sum[VEC];
          token(xv[u], gv[u], true, sum);
          vec_t o;
#pragma unroll
          for (int e = 0; e < VEC; ++e) put<T, VEC>(o, e, sum[e]);
          __builtin_nontemporal_store(o, reinterpret_cast<vec_t*>(op + (int64_t)u * a.D));
        }
        xp += kRows * a.ldx;
        gp += kRows * a.lddy;
        op += (int64_t)kRows * a.D;
      }
      while (t < stop) single();
      if (stop == s.eos) {  // the sequence's last rows: no token behind them
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
          const int row = s.eos - (W - 1) + j;
          if (row < first || row >= own) continue;
          float sum[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            float o = 0.f;
#pragma unroll
            for (int k = j; k < W - 1; ++k) o = fmaf(w[W - 1 - (k - j)][e], dp[k][e], o);
            sum[e] = o;
          }
          if (a.dfinal) {  // these rows are the final state's
            const vec_t fv = *reinterpret_cast<const vec_t*>(
                static_cast<const T*>(a.dfinal) + ((int64_t)seq * (W - 1) + j) * a.D + col);
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum[e] += at<T, VEC>(fv, e);
          }
          emit(row, sum);
        }
      }
      r = own;
      ++seq;
    }
    outside<T, VEC>(a, r, r1, col);
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
#pragma unroll
    for (int k = 0; k < W; ++k) s_sum[slice][k][e][lane] = dw[k][e];
    s_sum[slice][W][e][lane] = db[e];
  }
  block_barrier();
  float* part = a.part + (size_t)blockIdx.y * (W + 1) * a.D;
  const int c0 = blockIdx.x * kLanes * VEC;
  for (int i = threadIdx.x; i < (W + 1) * VEC * kLanes; i += kThreads) {
    const int k = i / (VEC * kLanes), c = i - k * (VEC * kLanes);
    if (c0 + c >= a.D) continue;
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < kSlices; ++j) s += s_sum[j][k][c % VEC][c / VEC];
    part[(size_t)k * a.D + c0 + c] = s;
  }
}

constexpr int kRedCols = 16;  // columns of a reducing workgroup, 16 row slices each
constexpr int kBatch = 8;     // loads a reducing thread issues before adding them

// Stage 2: sums part over the row blocks in a fixed order into dweight [D, W] and dbias [D].
__global__ __launch_bounds__(kThreads) void reduce_kernel(const float* __restrict__ part,
                                                          float* __restrict__ dweight,
                                                          float* __restrict__ dbias, int D, int W,
                                                          int nrb) {
  __shared__ float red[kThreads];
  constexpr int kParts = kThreads / kRedCols;
  const int c = threadIdx.x % kRedCols, p = threadIdx.x / kRedCols;
  const int64_t ld = (int64_t)(W + 1) * D, col = (int64_t)blockIdx.x * kRedCols + c;
  float s = 0.f;
  if (col < ld) {
    int j = p;
    for (; j + (kBatch - 1) * kParts < nrb; j += kBatch * kParts) {
      float v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) v[u] = part[(int64_t)(j + u * kParts) * ld + col];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) s += v[u];
    }
    for (; j < nrb; j += kParts) s += part[(int64_t)j * ld + col];
  }
  red[threadIdx.x] = s;
  block_barrier();
  if (p == 0 && col < ld) {
    float tot = 0.f;
    for (int i = 0; i < kParts; ++i) tot += red[i * kRedCols + c];
    const int k = (int)(col / D), d = (int)(col - (int64_t)k * D);
    if (k < W) {
      if (dweight) dweight[(size_t)d * W + k] = tot;
    } else if (dbias) {
      dbias[d] = tot;
    }
  }
}

// One token per request: the state's rows (the W - 1 inputs before it) and the token give y, and
// the state moves on by one row in place. slots: as kda_recurrent_step_slots. A lane takes its
// channels of REQ requests, so that their taps (float32: with W = 4 and a bias five times the bytes
// of a float32 row, ten times those of a bf16 row) are read once for all of them and all their loads
// are in flight together.
constexpr int kStepThreads = 64;

template <typename T, int VEC, int W, int REQ>
__global__ __launch_bounds__(kStepThreads) void step_kernel(const T* __restrict__ x, int64_t ldx,
                                                            const float* __restrict__ weight,
                                                            const float* __restrict__ bias,
                                                            T* __restrict__ pool,
                                                            const int* __restrict__ slots, int nslots,
                                                            T* __restrict__ y, int B, int D, int silu) {
  typedef row_t<T, VEC> vec_t;
  const int col = (blockIdx.x * kStepThreads + threadIdx.x) * VEC;
  if (col >= D) return;
  const int64_t n0 = (int64_t)blockIdx.y * REQ;
  vec_t v[REQ][W];
  int64_t slot[REQ];
#pragma unroll
  for (int u = 0; u < REQ; ++u) {
    const int64_t n = n0 + u;
    slot[u] = n >= B ? -1 : slots ? slots[n] : n;
    if (slot[u] >= nslots) slot[u] = -1;
    if (slot[u] < 0) continue;
    const T* st = pool + slot[u] * (W - 1) * D + col;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) v[u][k] = *reinterpret_cast<const vec_t*>(st + (int64_t)k * D);
    v[u][W - 1] = *reinterpret_cast<const vec_t*>(x + n * ldx + col);
  }
  float w[W][VEC], b[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][e] = weight[(size_t)(col + e) * W + k];
    b[e] = bias ? bias[col + e] : 0.f;
  }
#pragma unroll
  for (int u = 0; u < REQ; ++u) {
    if (n0 + u >= B) break;
    vec_t yv = vec_t{};
    if (slot[u] >= 0) {
      T* st = pool + slot[u] * (W - 1) * D + col;
#pragma unroll
      for (int k = 0; k < W - 1; ++k) *reinterpret_cast<vec_t*>(st + (int64_t)k * D) = v[u][k + 1];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float pre = b[e];
#pragma unroll
        for (int k = 0; k < W; ++k) pre = fmaf(w[k][e], at<T, VEC>(v[u][k], e), pre);
        put<T, VEC>(yv, e, silu ? pre * logistic(pre) : pre);
      }
    }
    *reinterpret_cast<vec_t*>(y + (n0 + u) * D + col) = yv;
  }
}

// ---- launchers

// Elements a lane takes: `vec` or the most that D, the strides and the pointers allow.
inline int vec_of(int vec, int esize, int D, int64_t strides, const void* const* ptrs, int nptrs) {
  uintptr_t bits = 0;
  for (int i = 0; i < nptrs; ++i) bits |= reinterpret_cast<uintptr_t>(ptrs[i]);
  while (vec > 1 && (D % vec || strides % vec || bits % ((size_t)vec * esize))) vec /= 2;
  return vec;
}

// Row blocks: enough workgroups to fill the GPU (target), kMinRows rows a slice at least.
struct Grid {
  int ncb, nrb;
  int64_t rpb;
};
inline Grid make_grid(int T, int D, int vec, int target) {
  Grid g;
  g.ncb = (D / vec + kLanes - 1) / kLanes;
  g.nrb = 0;
  g.rpb = 1;
  if (T == 0) return g;
  int64_t nrb = target / g.ncb;
  const int64_t most = ((int64_t)T + kSlices * kMinRows - 1) / (kSlices * kMinRows);
  nrb = nrb < 1 ? 1 : nrb > most ? most : nrb;
  g.rpb = ((int64_t)T + nrb - 1) / nrb;
  g.nrb = (int)((T + g.rpb - 1) / g.rpb);
  return g;
}

constexpr int kFwdBlocks = 4096, kBwdBlocks = 3 * 256;
// The backward holds 3 W - 1 floats a channel, so four channels a lane, not eight of bf16, and the
// resulting three workgroups a CU are launched in one round: 238 us at 32768 x 6144, bf16 (5.1
// TB/s), against 284 with eight channels and 277 with 1024 workgroups (a third of them in a second
// round). The forward (160 us, 5.0 TB/s) is fastest with several rounds of eight channels a lane.
constexpr int kBwdVec = 4;

template <typename T, int VEC, int W>
hipError_t run(int what, Args a, const ConvStep* st, float* dweight, float* dbias, hipStream_t stream) {
  if (what == 2) {
    const int ncb = (a.D / VEC + kStepThreads - 1) / kStepThreads;
    auto go = [&](auto kernel, int req) {
      hipLaunchKernelGGL(kernel, dim3(ncb, (st->B + req - 1) / req), dim3(kStepThreads), 0, stream,
                         static_cast<const T*>(a.x), a.ldx, a.weight, a.bias, static_cast<T*>(st->pool),
                         st->slots, st->nslots, static_cast<T*>(a.out), st->B, a.D, a.silu);
    };
    // several requests a lane where that leaves two waves a CU or more
    if ((int64_t)ncb * st->B >= 4 * 512) go(step_kernel<T, VEC, W, 4>, 4);
    else go(step_kernel<T, VEC, W, 1>, 1);
    return hipGetLastError();
  }
  const Grid g = make_grid(a.T, a.D, VEC, what == 0 ? kFwdBlocks : kBwdBlocks);
  a.rpb = g.rpb;
  a.nrb = g.nrb;
  const dim3 grid(g.ncb, g.nrb + (a.out_state ? (a.N + kSlices - 1) / kSlices : 0));
  hipError_t e = hipSuccess;
  if (grid.y > 0) {
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, a); };
    if (what == 0) a.silu ? go(fwd_kernel<T, VEC, W, true>) : go(fwd_kernel<T, VEC, W, false>);
    else if constexpr (VEC <= kBwdVec) a.silu ? go(bwd_kernel<T, VEC, W, true>) : go(bwd_kernel<T, VEC, W, false>);
    e = hipGetLastError();
  }
  if (what == 0) return e;
  if (e != hipSuccess || (!dweight && !dbias)) return e;
  const int64_t cols = (int64_t)(W + 1) * a.D;
  hipLaunchKernelGGL(reduce_kernel, dim3((unsigned)((cols + kRedCols - 1) / kRedCols)), dim3(kThreads), 0,
                     stream, a.part, dweight, dbias, a.D, W, g.nrb);
  return hipGetLastError();
}

template <typename T, int VEC>
hipError_t by_width(int what, const Args& a, int W, const ConvStep* st, float* dweight, float* dbias,
                    hipStream_t stream) {
  return W == 4 ? run<T, VEC, 4>(what, a, st, dweight, dbias, stream)
       : W == 3 ? run<T, VEC, 3>(what, a, st, dweight, dbias, stream)
                : run<T, VEC, 2>(what, a, st, dweight, dbias, stream);
}

inline hipError_t dispatch(int what, const Args& a, int W, bool bf, int vec, const ConvStep* st,
                           float* dweight, float* dbias, hipStream_t stream) {
  if (bf) {
    if (vec == 8) return by_width<bf16, 8>(what, a, W, st, dweight, dbias, stream);
    if (vec == 4) return by_width<bf16, 4>(what, a, W, st, dweight, dbias, stream);
    if (vec == 2) return by_width<bf16, 2>(what, a, W, st, dweight, dbias, stream);
    return by_width<bf16, 1>(what, a, W, st, dweight, dbias, stream);
  }
  if (vec == 4) return by_width<float, 4>(what, a, W, st, dweight, dbias, stream);
  if (vec == 2) return by_width<float, 2>(what, a, W, st, dweight, dbias, stream);
  return by_width<float, 1>(what, a, W, st, dweight, dbias, stream);
}

}  // namespace conv

// Partial sums of the backward: sized for the narrowest vector (the most row blocks).
size_t conv_bwd_workspace_bytes(int T, int D, int W) {
  int64_t nrb = 0;
  for (int vec = conv::kBwdVec; vec >= 1; vec /= 2) {
    if (D % vec) continue;
    const conv::Grid g = conv::make_grid(T, D, vec, conv::kBwdBlocks);
    nrb = nrb > g.nrb ? nrb : g.nrb;
  }
  return ((size_t)nrb * (W + 1) * D * 4 + 255) / 256 * 256;
}

hipError_t launch_conv_fwd(const ConvArgs& p, hipStream_t stream) {
  conv::Args a{};
  a.x = p.x, a.ldx = p.ldx, a.weight = p.weight, a.bias = p.bias, a.init = p.init, a.seqs = make_sequences(p.cu, p.N, p.T);
  a.N = p.N, a.T = p.T, a.D = p.D, a.silu = p.silu, a.zero_rest = p.zero_rest, a.out_state = p.out_state, a.out = p.out;
  const void* ptrs[] = {p.x, p.init, p.out_state, p.out};
  const int vec = conv::vec_of(p.bf ? 8 : 4, p.bf ? 2 : 4, p.D, p.ldx, ptrs, 4);
  return conv::dispatch(0, a, p.W, p.bf, vec, nullptr, nullptr, nullptr, stream);
}

hipError_t launch_conv_bwd(const ConvArgs& p, const void* dy, int64_t lddy, const void* dfinal,
                           float* dweight, float* dbias, void* workspace, hipStream_t stream) {
  conv::Args a{};
  a.x = p.x, a.ldx = p.ldx, a.weight = p.weight, a.bias = p.bias, a.init = p.init, a.seqs = make_sequences(p.cu, p.N, p.T);
  a.N = p.N, a.T = p.T, a.D = p.D, a.silu = p.silu, a.zero_rest = p.zero_rest, a.out_state = p.out_state, a.out = p.out;
  a.dy = dy, a.lddy = lddy, a.dfinal = dfinal, a.part = static_cast<float*>(workspace);
  const void* ptrs[] = {p.x, p.init, p.out_state, p.out, dy, dfinal};
  const int vec = conv::vec_of(conv::kBwdVec, p.bf ? 2 : 4, p.D, p.ldx | lddy, ptrs, 6);
  return conv::dispatch(1, a, p.W, p.bf, vec, nullptr, dweight, dbias, stream);
}

hipError_t launch_conv_step(const ConvArgs& p, const ConvStep& st, hipStream_t stream) {
  conv::Args a{};
  a.x = p.x, a.ldx = p.ldx, a.weight = p.weight, a.bias = p.bias;
  a.D = p.D, a.silu = p.silu, a.out = p.out;
  const void* ptrs[] = {p.x, st.pool, p.out};
  const int vec = conv::vec_of(p.bf ? 8 : 4, p.bf ? 2 : 4, p.D, p.ldx, ptrs, 3);
  return conv::dispatch(2, a, p.W, p.bf, vec, &st, nullptr, nullptr, stream);
}

}  // namespace kda
