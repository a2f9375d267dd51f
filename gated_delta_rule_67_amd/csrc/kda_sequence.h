// Where the sequences of a batch lie on its token axis: N equal ones, or packed ones with offsets
// cu[0..N] in device memory. Shared by the convolution and the selective scan. Offsets are
// clamped into [0, T], so malformed ones give wrong results, never accesses out of range.
#pragma once

#include "kda_device.h"

namespace kda {

struct Span {
  int bos, eos;  // tokens bos .. eos - 1
};

struct Sequences {
  const int* cu;  // offsets, or null
  int N, T;       // sequences, tokens
  int len;        // tokens of each where cu is null

  // n is uniform over the wave: the offsets come by scalar loads (nothing writes them meanwhile),
  // which wait for no vector load or store in flight.
  __device__ __forceinline__ Span span(int n) const {
    if (!cu) return {n * len, (n + 1) * len};
    const int u = __builtin_amdgcn_readfirstlane(n);
    const auto* c = (const __attribute__((address_space(4))) int*)cu;
    const int bos = min(max(c[u], 0), T);
    return {bos, min(max(c[u + 1], bos), T)};
  }

  // The last sequence whose first token is at or before token t (0 if there is none); empty ones
  // in front of it are passed over. Every lane of the wave takes part; offsets are read 64 at a
  // time. T > 0.
  __device__ __forceinline__ int find(int t) const {
    if (!cu) return t / len;
    const int lane = __lane_id();
    int below = 0;
    for (int i = 0; i < N; i += 64) {
      const bool in = i + lane < N && cu[i + lane] <= t;
      below += __builtin_popcountll(__builtin_amdgcn_ballot_w64(in));
    }
    return __builtin_amdgcn_readfirstlane(below > 0 ? below - 1 : 0);
  }
};

inline Sequences make_sequences(const int* cu, int N, int T) { return {cu, N, T, T / N}; }

}  // namespace kda
