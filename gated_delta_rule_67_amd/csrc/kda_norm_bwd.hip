// The norms around a block, backward.
//
// With v the row under the norm (h in front of a block, x behind it), inv = 1 / sqrt(mean(v^2) + eps),
// n = v inv and u the gradient of n:
//   dv = inv (u - n mean(u n)),
// in front: u = weight dy, dresidual = dv + dh, dx = scale dresidual, dscale = sum_rows x dresidual;
// behind, with d = scale dy: u = weight act(gate) d, dx = dv, dgate = act'(gate) weight n d,
// dscale = sum_rows dy weight act(gate) n;
// and dweight = sum_rows of dy n, or d act(gate) n.
// Both means come from one pass over the row (sums of v^2 and of u v), which stays in registers, so
// that every tensor moves once and HBM bounds the kernel. A thread keeps its columns over all of its
// rows and adds dweight and dscale up in registers; workgroups leave partial sums, which a second
// kernel adds in a fixed order.
// Measured, back to back: behind, 524288 rows of 128 in bf16 under a gate 137 us (671 MB, 4.9 TB/s), 132 and 146 with
// outputs in the last-level cache and not; from checkpoints 131 and 136. In front, 32768 rows of 2048 in bf16 with
// residual and scale 156 and 165 us (805 MB), from checkpoints 145 and 153; 5003 rows of 1030 in float32 31 us
// (124 MB; its kernels, traced, 27 and 4.4). Behind, at an earlier step (139 us): the gate's activation kept in
// registers between its two uses 145 us; 1, 2, 3 and 4 rows at a time, before loads went past the caches, 149, 148,
// 168 and 170.
// v (and the gate, and x in front) may be 8-bit checkpoints: the gradients are those at the values
// that these stand for, and the tensor moves 33 bytes for every 32 elements.
#include <type_traits>

#include "kda_norm_tile.h"

namespace kda {
namespace norm {

template <typename T, class TILE, int ROWS, bool BEHIND, bool CK, bool ONCE>
__global__ __launch_bounds__(TILE::BLOCK) void bwd_kernel(NormArgs a) {
  constexpr int VEC = TILE::VEC, NC = TILE::NC;
  typedef Piece<T, VEC> piece;
  typedef typename KeptPiece<T, VEC, CK>::type kept;
  typedef RowSums<TILE, 2 * ROWS> sums;
  __shared__ typename sums::Shared lds;
  const int lane = threadIdx.x % TILE::THREADS, side = threadIdx.x / TILE::THREADS;
  int col[NC];
  bool in[NC];
  float w[NC][VEC], sc[NC][VEC], dw[NC][VEC], ds[NC][VEC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    col[c] = (c * TILE::THREADS + lane) * VEC;
    in[c] = col[c] < a.D;
    if (!in[c]) col[c] = a.D - VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[c][e] = a.weight[col[c] + e];
      sc[c][e] = a.scale ? a.scale[col[c] + e] : 1.f;
      dw[c][e] = ds[c][e] = 0.f;
    }
  }
  const bool gated = BEHIND && a.gate.p, scaled = a.scale, joined = !BEHIND && a.dh.p;
  const float inv_d = 1.f / (float)a.D;
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * (TILE::SIDE * ROWS);
  for (int64_t first = (int64_t)blockIdx.x * (TILE::SIDE * ROWS); first < a.rows; first += step, turn ^= 1) {
    kept v[ROWS][NC], k[ROWS][NC];  // k: the gate (behind), x (in front)
    piece g[ROWS][NC], r[ROWS][NC];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      const int64_t row = min(first + u * TILE::SIDE + side, a.rows - 1);
      const int64_t ov = row_offset(a, a.v, row), og = row_offset(a, a.dy, row);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        v[u][c].template load<ONCE>(a.v, ov + col[c]);
        g[u][c].template load<ONCE>(a.dy, og + col[c]);
      }
      if (BEHIND ? gated : scaled) {
        const Source& s = BEHIND ? a.gate : a.other;
        const int64_t o = row_offset(a, s, row);
#pragma unroll
        for (int c = 0; c < NC; ++c) k[u][c].template load<ONCE>(s, o + col[c]);
      }
      if (joined) {
        const int64_t o = row_offset(a, a.dh, row);
#pragma unroll
        for (int c = 0; c < NC; ++c) r[u][c].template load<ONCE>(a.dh, o + col[c]);
      }
    }
    // act(gate) of an element (its slope too): computed where it is needed, twice
    auto act = [&](float z, float& slope) {
      float s, rest;
      logistic_pair(z, s, rest);
      slope = a.silu ? s * fmaf(z, rest, 1.f) : s * rest;
      return a.silu ? z * s : s;
    };
    float sum[2 * ROWS];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      sum[2 * u] = sum[2 * u + 1] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float x[VEC], d[VEC], z[VEC], sq = 0.f, dot = 0.f;
        v[u][c].get(x);
        g[u][c].get(d);
        if (gated) k[u][c].get(z);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float t = d[e] * w[c][e], slope;
          if (BEHIND && scaled) t *= sc[c][e];
          if (gated) t *= act(z[e], slope);
          sq = fmaf(x[e], x[e], sq);
          dot = fmaf(t, x[e], dot);
        }
        sum[2 * u] += in[c] ? sq : 0.f;
        sum[2 * u + 1] += in[c] ? dot : 0.f;
      }
    }
    sums::run(sum, lds, turn);
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      const int64_t row = first + u * TILE::SIDE + side;
      if (row >= a.rows) continue;
      const float inv = __builtin_amdgcn_rsqf(fmaf(sum[2 * u], inv_d, a.eps));
      const float mean = sum[2 * u + 1] * inv * inv_d;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (!in[c]) continue;
        const int64_t off = row * a.D + col[c];
        float x[VEC], d[VEC], z[VEC], out[VEC], more[VEC];
        v[u][c].get(x);
        g[u][c].get(d);
        if (BEHIND ? gated : scaled) k[u][c].get(z);
        float q[VEC];
        if (joined) r[u][c].get(q);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float n = x[e] * inv;
          if constexpr (BEHIND) {
            float slope = 0.f, f = 1.f;
            if (gated) f = act(z[e], slope);
            const float dn = d[e] * n;  // dy n
            if (scaled) {
              ds[c][e] = fmaf(dn * f, w[c][e], ds[c][e]);
              f *= sc[c][e];
              slope *= sc[c][e];
            }
            dw[c][e] = fmaf(dn, f, dw[c][e]);
            more[e] = dn * w[c][e] * slope;
            out[e] = inv * fmaf(-n, mean, d[e] * w[c][e] * f);
          } else {
            dw[c][e] = fmaf(d[e], n, dw[c][e]);
            float t = inv * fmaf(-n, mean, d[e] * w[c][e]);
            if (joined) t += q[e];
            out[e] = t;
            if (scaled) {
              more[e] = t * sc[c][e];
              ds[c][e] = fmaf(z[e], t, ds[c][e]);
            }
          }
        }
        piece o;
        o.set(out);
        o.store(a.y, off);
        if (BEHIND ? gated : scaled) {
          o.set(more);
          o.store(a.extra, off);
        }
      }
    }
  }
  // partial sums of this workgroup's rows, the rows side by side added in order
  if (!a.part) return;
  float* part = a.part + (size_t)blockIdx.x * 2 * a.D;
  if constexpr (TILE::SIDE == 1) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (!in[c]) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        part[col[c] + e] = dw[c][e];
        part[a.D + col[c] + e] = ds[c][e];
      }
    }
  } else {
    static_assert(NC == 1, "rows side by side hold one vector a thread");
    constexpr int kCols = TILE::THREADS * VEC;
    __shared__ float acc[TILE::SIDE][kCols];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k) block_barrier();
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[side][lane * VEC + e] = k ? ds[0][e] : dw[0][e];
      block_barrier();
      for (int i = threadIdx.x; i < kCols && i < a.D; i += TILE::BLOCK) {
        float s = 0.f;
        for (int j = 0; j < TILE::SIDE; ++j) s += acc[j][i];
        part[(size_t)k * a.D + i] = s;
      }
    }
  }
}

// Workgroups of a launch at most: three of 256 threads a CU in one round (their partial sums are
// written and read once more, 8 bytes a column each). 2, 3, 4, 6 and 8 a CU: 28.5, 28.5, 29.7, 33 and
// 34.6 us for 5003 rows of 1030, on two sets of buffers in turn (31 us on more).
constexpr int kBwdBlocks = 3 * 256;

inline int bwd_blocks(int64_t rows, int batch) {
  const int64_t need = (rows + batch - 1) / batch;
  return (int)(need < kBwdBlocks ? need : kBwdBlocks);
}

template <typename T, int VEC, bool BEHIND, bool CK, bool ONCE>
hipError_t run_bwd(const NormArgs& a, hipStream_t stream) {
  return with_tile<VEC>(a.D, [&](auto tile) {
    typedef decltype(tile) TILE;
    constexpr int ROWS = TILE::NC > 1 ? 1 : 2;
    const int nb = bwd_blocks(a.rows, TILE::SIDE * ROWS);
    hipLaunchKernelGGL((bwd_kernel<T, TILE, ROWS, BEHIND, CK, ONCE>), dim3(nb), dim3(TILE::BLOCK), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.part) return e;
    return launch_column_sums({a.part, {a.dweight, a.dscale}, nb, 2, a.D}, stream);
  });
}

}  // namespace norm

size_t norm_bwd_workspace_bytes(int64_t rows, int D) {
  const int64_t nb = rows < norm::kBwdBlocks ? rows : norm::kBwdBlocks;
  return ((size_t)nb * 2 * D * 4 + 255) / 256 * 256;
}

hipError_t launch_norm_bwd(const NormArgs& a, bool behind, hipStream_t stream) {
  if (a.rows == 0)  // the sums of no rows
    return a.dweight || a.dscale ? launch_column_sums({nullptr, {a.dweight, a.dscale}, 0, 2, a.D}, stream) : hipSuccess;
  auto element = [&](const Source& s) { return a.packed ? nullptr : s.p; };
  const void* ptrs[] = {element(a.v), element(a.gate), element(a.other), a.dy.p, a.dh.p, a.y, a.extra};
  const int64_t widths = a.D | a.v.ld | a.gate.ld | a.other.ld | a.dy.ld | a.dh.ld;
  int vec = vector_width(a.bf ? 8 : 4, a.bf ? 2 : 4, widths, ptrs, 7);
  if (a.packed) {  // codes: a byte each
    const void* codes[] = {a.v.p, a.gate.p, a.other.p};
    const int most = vector_width(a.bf ? 8 : 4, 1, 0, codes, 3);
    vec = most < vec ? most : vec;
  }
  // 32 elements of a tensor move 32 elements' bytes, of a checkpoint 33
  const int whole = 32 * (a.bf ? 2 : 4), kept = a.packed ? kScaleBlock + 1 : whole;
  const int tensors = 2 + (a.dh.p != nullptr) + (a.extra != nullptr);
  const int read = 1 + (a.gate.p != nullptr) + (a.other.p != nullptr);
  const bool once = a.rows * a.D / 32 * (whole * tensors + kept * read) > kCached;
  auto go = [&](auto b, auto k) {
    constexpr bool B = decltype(b)::value, K = decltype(k)::value;
    if (a.bf) {
      if (vec == 8) return once ? norm::run_bwd<bf16, 8, B, K, true>(a, stream) : norm::run_bwd<bf16, 8, B, K, false>(a, stream);
      return vec >= 2 ? norm::run_bwd<bf16, 2, B, K, false>(a, stream) : norm::run_bwd<bf16, 1, B, K, false>(a, stream);
    }
    if (vec == 4) return once ? norm::run_bwd<float, 4, B, K, true>(a, stream) : norm::run_bwd<float, 4, B, K, false>(a, stream);
    return vec == 2 ? norm::run_bwd<float, 2, B, K, false>(a, stream) : norm::run_bwd<float, 1, B, K, false>(a, stream);
  };
  if (behind) return a.packed ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
  return a.packed ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
}

}  // namespace kda
