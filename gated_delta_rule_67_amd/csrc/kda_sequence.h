// Where the sequences of a batch lie on its token axis: N equal ones, or packed ones with offsets
// cu[0..N] in device memory. Shared by the convolution and the selective scan. Offsets are
// clamped into [0, T], so malformed ones give wrong results, never accesses out of range.
#pragma once

#include "kda_device.h"

namespace kda {

struct Span {
  int bos, eos;  // tokens bos .. eos - 1
};

__device__ __forceinline__ Span sequence_span(const int* cu, int N, int T, int n) {
  if (!cu) {
    const int len = T / N;
    return {n * len, (n + 1) * len};
  }
  const int bos = min(max(cu[n], 0), T);
  return {bos, min(max(cu[n + 1], bos), T)};
}

// The last sequence whose first token is at or before token t (0 if there is none); empty ones in
// front of it are passed over. Every lane of the wave takes part; offsets are read 64 at a time.
__device__ __forceinline__ int find_sequence(const int* cu, int N, int T, int t) {
  if (!cu) return t / (T / N);
  const int lane = __lane_id();
  int below = 0;
  for (int i = 0; i < N; i += 64) {
    const bool in = i + lane < N && cu[i + lane] <= t;
    below += __builtin_popcountll(__builtin_amdgcn_ballot_w64(in));
  }
  return __builtin_amdgcn_readfirstlane(below > 0 ? below - 1 : 0);
}

}  // namespace kda
