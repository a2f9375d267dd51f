// How the norms' kernels lay rows on threads. THREADS threads hold a row, NC vectors of VEC columns
// each; a workgroup of kNormThreads (or THREADS, if that is more) works on several rows at a time, and
// a thread on ROWS of them, so that the loads of ROWS rows are in flight together.
#pragma once

#include "kda_norm.h"

namespace kda {
namespace norm {

constexpr int kNormThreads = 256;

template <int VEC_, int THREADS_, int NC_> struct Tile {
  static constexpr int VEC = VEC_, THREADS = THREADS_, NC = NC_;
  static constexpr int BLOCK = THREADS > kNormThreads ? THREADS : kNormThreads;
  static constexpr int SIDE = BLOCK / THREADS;  // rows side by side
  static constexpr int WAVES = THREADS > 64 ? THREADS / 64 : 1;  // waves of a row
};

// Sums over the threads of a row of K values for each of ROWS rows: in registers inside a wave,
// through LDS where several waves hold a row. Every thread gets the sums; `turn` alternates between
// two LDS buffers, so that one barrier a call suffices.
template <class TILE, int K>
struct RowSums {
  static constexpr int kSlots = TILE::WAVES > 1 ? 2 * TILE::WAVES * K : 1;
  typedef float Shared[kSlots];

  static __device__ __forceinline__ void run(float (&v)[K], Shared& lds, int turn) {
    constexpr int W = TILE::THREADS < 64 ? TILE::THREADS : 64;
#pragma unroll
    for (int m = 1; m < W; m *= 2) {
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], m);
    }
    if constexpr (TILE::WAVES > 1) {
      float* buf = lds + turn * TILE::WAVES * K;
      const int wave = threadIdx.x / 64;
      if (threadIdx.x % 64 == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) buf[wave * K + k] = v[k];
      }
      lds_barrier();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < TILE::WAVES; ++w) s += buf[w * K + k];
        v[k] = s;
      }
    }
  }
};

// Element offset of a row's first column.
__device__ __forceinline__ int64_t row_offset(const NormArgs& a, const Source& s, int64_t row) {
  if (a.G == 1) return row * s.ld;
  const int64_t token = row / a.G;
  return token * s.ld + (row - token * a.G) * a.D;
}

// The tile of the fewest threads whose vectors hold a row, out of a list. Three vectors a thread for 1030
// columns of float32 (the backward pass 28.5 us over 5003 rows; with four, of which the last is empty, 34).
// Between the list's widths lanes or vectors stay empty. 134 MB a tensor, in front of a block, forward and backward
// (four tensors moved each), in us: bf16 512 columns 101 and 105, 520 126 and 324, 768 107 and 227, 1024 103 and 176,
// 1536 104 and 139, 2048 102 and 123, 4096 106 and 128, 5120 119 and 173, 6144 116 and 169, 8192 120 and 168; float32
// 512 to 2048 columns 97 to 109 and 102 to 110, 1030 116 and 103, 5120 to 8192 102 to 105 and 143 to 151.
template <int VEC, class F> inline hipError_t with_tile(int D, F&& go) {
  if constexpr (VEC >= 4) {
    if (D <= 8 * VEC) return go(Tile<VEC, 8, 1>{});
    if (D <= 16 * VEC) return go(Tile<VEC, 16, 1>{});
    if (D <= 32 * VEC) return go(Tile<VEC, 32, 1>{});
  }
  if (D <= 64 * VEC) return go(Tile<VEC, 64, 1>{});
  if (D <= 256 * VEC) return go(Tile<VEC, 256, 1>{});
  if (D <= 512 * VEC) return go(Tile<VEC, 256, 2>{});
  if constexpr (VEC < 4) {
    if (D <= 768 * VEC) return go(Tile<VEC, 256, 3>{});
  }
  if (D <= 1024 * VEC) return go(Tile<VEC, 256, 4>{});
  if constexpr (VEC < 8) return go(Tile<VEC, 1024, kNormMaxDim / (1024 * VEC)>{});
  else return hipErrorInvalidValue;  // 1024 VEC is the limit
}

}  // namespace norm
}  // namespace kda
