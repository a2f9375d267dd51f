// Arguments of the norms in front of and behind a block (validated by the C ABI).
#pragma once

#include "kda_rows.h"

namespace kda {

struct NormArgs {
  int64_t rows;        // tokens x groups
  int G, D;            // rows of a token (at its start, D elements apart), columns
  float eps;
  const float* weight; // [D]
  const float* scale;  // [D] or null
  Source v;            // in front: x (backward: h); behind: x
  Source gate;         // behind: the gate, p null: none
  Source other;        // forward: the residual, p null: none; backward, in front: x, where scale is given
  Source dy, dh;       // backward; dh in front only, p null: zeros
  void* y;             // forward: out. Backward: dresidual (in front) or dx (behind)
  void* extra;         // forward, in front: h out, or null. Backward: dx (in front) or dgate (behind), or null
  float* part;         // backward: partial column sums [blocks][2][D]
  float* dweight;      // backward out, or null
  float* dscale;
  int silu;            // behind: the gate's activation is silu, else the logistic
  bool bf, packed;     // backward: v, gate and other are checkpoints
};

constexpr int kNormMaxDim = 8192;

hipError_t launch_norm_fwd(const NormArgs& a, bool behind, hipStream_t stream);
hipError_t launch_norm_bwd(const NormArgs& a, bool behind, hipStream_t stream);
size_t norm_bwd_workspace_bytes(int64_t rows, int D);

}  // namespace kda
