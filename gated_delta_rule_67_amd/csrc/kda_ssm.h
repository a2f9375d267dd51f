// Arguments of the selective scan's launches (validated by the C ABI).
#pragma once

#include "kda_sequence.h"

namespace kda {

// -exp(A_log), finite: an infinite rate times a step size that underflows to 0 would be NaN. (A
// NaN stays one.)
__device__ __forceinline__ float negative_rate(float A_log) {
  const float rate = -expf(A_log);
  return rate < -3.402823466e38f ? -3.402823466e38f : rate;
}

// max(v, least), but a NaN stays one.
__device__ __forceinline__ float at_least(float least, float v) { return v < least ? least : v; }

// 2^g, what a state keeps of itself: never 0, because an infinite state times 0 would be NaN. The
// smallest float (2^-149) adds less to a finite one than the error of an exponential that underflows.
__device__ __forceinline__ float decay_of(float g) { return at_least(0x1p-149f, fast_exp2(g)); }

struct SsmArgs {
  const void* x;   // [T, HV, V], ldx elements between tokens
  int64_t ldx;
  const void* dt;  // [T, HV]
  int64_t lddt;
  const float* A_log;  // [HV]
  const void* b;       // [T, H, K]
  int64_t ldb;
  const void* c;
  int64_t ldc;
  const float* D;        // [HV] or null
  const float* dt_bias;  // [HV] or null
  const float* s0;       // [N, HV, K, V] or null
  Sequences seqs;
  int N, T, H, HV, K, V;
  float* sT;             // [N, HV, K, V] or null
  void* y;               // [T, HV, V]
  bool bf, zero_rest;
  // the step
  float* pool;
  const int* slots;
  int nslots, B;
  // the prefill's segments of the token axis: seg tokens each, nseg of them; the state entering
  // segment k in seg_state[k - 1], the log2 of its decay since the segment before in seg_g
  int seg, nseg;
  int per;           // segments of each sequence where they divide it evenly, else 0
  bool crossed;      // whether a sequence may go on over a segment's end
  float* seg_state;  // [nseg - 1][HV][K][V]
  float* seg_g;      // [nseg - 1][HV]
  bool vec;          // rows of x, b, c and y are whole 16-byte pieces, aligned
};

// seg_g of a segment boundary at which no sequence goes on (decays have g <= 0).
constexpr float kNoCarry = 2.f;

}  // namespace kda
