// The norms around a block, forward (and the fixed-order column sums that backward passes share).
//
// In front of a block, with the residual addition behind the one before it: per row of D columns
//   h = residual + scale x,   y = weight h / sqrt(mean(h^2) + eps).
// Behind a block: y = residual + scale (weight act(gate) x / sqrt(mean(x^2) + eps)), act the logistic
// or silu; without gate, scale or residual their parts fall away.
// Sums and values are float32; y (and h) are rounded once, as they are stored, and in front of a block
// the norm is that of the unrounded h.
//
// A row is read once and held in registers between the sum of squares and the output, so the kernel
// moves what it must (8 bytes an element with a residual in bf16) and is bound by HBM. weight and
// scale are read once a thread: its columns stay the same over the rows that it works on.
//
// Measured in bf16, back to back: in front, 32768 rows of 2048 with the residual 102 us (537 MB, 5.3 TB/s; 85 where
// the outputs' memory is still in the last-level cache from the call before); behind, 524288 rows of 128 under a gate
// 66 us (403 MB, 6.1 TB/s) into memory that calls reuse, 73 otherwise; one row 3.1 us, 9.7 with its launch.
#include <type_traits>

#include "kda_norm_tile.h"

namespace kda {
namespace norm {

template <typename T, class TILE, int ROWS, bool BEHIND, bool ONCE>
__global__ __launch_bounds__(TILE::BLOCK) void fwd_kernel(NormArgs a) {
  constexpr int VEC = TILE::VEC, NC = TILE::NC;
  typedef Piece<T, VEC> piece;
  typedef RowSums<TILE, ROWS> sums;
  __shared__ typename sums::Shared lds;
  const int lane = threadIdx.x % TILE::THREADS, side = threadIdx.x / TILE::THREADS;
  int col[NC];
  bool in[NC];
  float w[NC][VEC], sc[NC][VEC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    col[c] = (c * TILE::THREADS + lane) * VEC;
    in[c] = col[c] < a.D;
    if (!in[c]) col[c] = a.D - VEC;  // reads stay inside the row
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[c][e] = a.weight[col[c] + e];
      sc[c][e] = a.scale ? a.scale[col[c] + e] : 1.f;
    }
  }
  const bool gated = BEHIND && a.gate.p, added = a.other.p;
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * (TILE::SIDE * ROWS);
  for (int64_t first = (int64_t)blockIdx.x * (TILE::SIDE * ROWS); first < a.rows; first += step, turn ^= 1) {
    piece v[ROWS][NC], z[ROWS][NC], r[ROWS][NC];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      const int64_t row = min(first + u * TILE::SIDE + side, a.rows - 1);
      const int64_t off = row_offset(a, a.v, row);
#pragma unroll
      for (int c = 0; c < NC; ++c) v[u][c].template load<ONCE>(a.v, off + col[c]);
      if (added) {
        const int64_t o = row_offset(a, a.other, row);
#pragma unroll
        for (int c = 0; c < NC; ++c) r[u][c].template load<ONCE>(a.other, o + col[c]);
      }
      if (gated) {
        const int64_t o = row_offset(a, a.gate, row);
#pragma unroll
        for (int c = 0; c < NC; ++c) z[u][c].template load<ONCE>(a.gate, o + col[c]);
      }
    }
    float x[ROWS][NC][VEC], sq[ROWS];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      sq[u] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        v[u][c].get(x[u][c]);
        if constexpr (!BEHIND) {
          if (a.scale) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[u][c][e] *= sc[c][e];
          }
          if (added) {
            float q[VEC];
            r[u][c].get(q);
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[u][c][e] += q[e];
          }
        }
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) s = fmaf(x[u][c][e], x[u][c][e], s);
        sq[u] += in[c] ? s : 0.f;
      }
    }
    sums::run(sq, lds, turn);
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      const int64_t row = first + u * TILE::SIDE + side;
      if (row >= a.rows) continue;
      const float inv = __builtin_amdgcn_rsqf(sq[u] / (float)a.D + a.eps);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (!in[c]) continue;
        const int64_t off = row * a.D + col[c];
        piece o;
        if constexpr (!BEHIND) {
          if (a.extra) {
            o.set(x[u][c]);
            o.store(a.extra, off);
          }
        }
        float y[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[e] = x[u][c][e] * inv * w[c][e];
        if constexpr (BEHIND) {
          if (gated) {
            float g[VEC];
            z[u][c].get(g);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              float s, rest;
              logistic_pair(g[e], s, rest);
              y[e] *= a.silu ? g[e] * s : s;
            }
          }
          if (a.scale) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] *= sc[c][e];
          }
          if (added) {
            float q[VEC];
            r[u][c].get(q);
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[e] += q[e];
          }
        }
        o.set(y);
        o.store(a.y, off);
      }
    }
  }
}

constexpr int kFwdThreads = 256 * 2048;  // threads of a launch: every CU full

template <typename T, int VEC, bool BEHIND, bool ONCE>
hipError_t run_fwd(const NormArgs& a, hipStream_t stream) {
  return with_tile<VEC>(a.D, [&](auto tile) {
    typedef decltype(tile) TILE;
    constexpr int ROWS = TILE::NC > 2 ? 1 : TILE::NC == 2 ? 2 : 4;
    const int64_t need = (a.rows + TILE::SIDE * ROWS - 1) / (TILE::SIDE * ROWS);
    const int64_t most = kFwdThreads / TILE::BLOCK;
    hipLaunchKernelGGL((fwd_kernel<T, TILE, ROWS, BEHIND, ONCE>), dim3((unsigned)(need < most ? need : most)),
                       dim3(TILE::BLOCK), 0, stream, a);
    return hipGetLastError();
  });
}

// 16 columns a workgroup, 16 row slices each.
constexpr int kRedCols = 16, kRedThreads = 256, kRedBatch = 8;

__global__ __launch_bounds__(kRedThreads) void column_sums_kernel(ColumnSums a) {
  __shared__ float red[kRedThreads];
  constexpr int kParts = kRedThreads / kRedCols;
  const int c = threadIdx.x % kRedCols, p = threadIdx.x / kRedCols;
  const int64_t ld = (int64_t)a.K * a.D, col = (int64_t)blockIdx.x * kRedCols + c;
  float s = 0.f;
  if (col < ld) {
    int j = p;
    for (; j + (kRedBatch - 1) * kParts < a.nb; j += kRedBatch * kParts) {
      float v[kRedBatch];
#pragma unroll
      for (int u = 0; u < kRedBatch; ++u) v[u] = a.part[(int64_t)(j + u * kParts) * ld + col];
#pragma unroll
      for (int u = 0; u < kRedBatch; ++u) s += v[u];
    }
    for (; j < a.nb; j += kParts) s += a.part[(int64_t)j * ld + col];
  }
  red[threadIdx.x] = s;
  block_barrier();
  if (p == 0 && col < ld) {
    float tot = 0.f;
    for (int i = 0; i < kParts; ++i) tot += red[i * kRedCols + c];
    const int k = (int)(col / a.D);
    if (a.out[k]) a.out[k][col - (int64_t)k * a.D] = tot;
  }
}

}  // namespace norm

hipError_t launch_column_sums(const ColumnSums& a, hipStream_t stream) {
  const int64_t cols = (int64_t)a.K * a.D;
  hipLaunchKernelGGL(norm::column_sums_kernel, dim3((unsigned)((cols + norm::kRedCols - 1) / norm::kRedCols)),
                     dim3(norm::kRedThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_norm_fwd(const NormArgs& a, bool behind, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  const void* ptrs[] = {a.v.p, a.gate.p, a.other.p, a.y, a.extra};
  const int vec = vector_width(a.bf ? 8 : 4, a.bf ? 2 : 4, a.D | a.v.ld | a.gate.ld | a.other.ld, ptrs, 5);
  const int tensors = 2 + (a.gate.p != nullptr) + (a.other.p != nullptr) + (a.extra != nullptr);
  const bool once = a.rows * a.D * (a.bf ? 2 : 4) * tensors > kCached;
  auto go = [&](auto b) {
    constexpr bool B = decltype(b)::value;
    if (a.bf) {
      if (vec == 8) return once ? norm::run_fwd<bf16, 8, B, true>(a, stream) : norm::run_fwd<bf16, 8, B, false>(a, stream);
      return vec >= 2 ? norm::run_fwd<bf16, 2, B, false>(a, stream) : norm::run_fwd<bf16, 1, B, false>(a, stream);
    }
    if (vec == 4) return once ? norm::run_fwd<float, 4, B, true>(a, stream) : norm::run_fwd<float, 4, B, false>(a, stream);
    return vec == 2 ? norm::run_fwd<float, 2, B, false>(a, stream) : norm::run_fwd<float, 1, B, false>(a, stream);
  };
  return behind ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace kda
