// One token of the selective scan per request, on a slot of a pool of K x V float32 states:
//   S <- a S + b (D_t x)^T,   y = S^T c + D x      (a, D_t as in the prefill)
//
// Bound by HBM: a state is read and written once, and a few operations are done on each of its
// values. One workgroup takes a head's state (or a quarter of its columns, where there are too
// few heads to fill the GPU); a lane owns VEC columns and every rgc-th row, updates its values as
// they arrive and adds its share of y, which the row groups then add up in LDS in a fixed order.
// 256 requests, 64 heads of 128 x 64: 199 us (5.4 TB/s; 204 us with 256 lanes a workgroup, 211 with
// cached stores, 376 with four workgroups a head).
#include "kda_ssm.h"

namespace kda {
namespace ssm_step {

constexpr int kThreads = 512;
constexpr int kRows = 4;     // rows whose loads a lane issues before using any
constexpr int kMaxK = 128;

template <typename T, int VEC>
__global__ __launch_bounds__(kThreads) void step_kernel(SsmArgs a, int nsplit) {
  typedef float vec_t __attribute__((ext_vector_type(VEC)));
  __shared__ float s_b[kMaxK], s_c[kMaxK];
  __shared__ float s_y[kThreads * VEC];
  const int K = a.K, V = a.V, t = threadIdx.x;
  const int part = blockIdx.x % nsplit, bh = blockIdx.x / nsplit;
  const int n = bh / a.HV, hv = bh - n * a.HV, h = hv / (a.HV / a.H);
  const int vw = V / nsplit, v0 = part * vw;  // this workgroup's columns, vw % VEC == 0
  const int nc = vw / VEC, rgc = kThreads / nc;
  const int c = t % nc, rg = t / nc, col = v0 + c * VEC;
  T* y = static_cast<T*>(a.y) + (int64_t)bh * V + v0;
  const int64_t slot = a.slots ? a.slots[n] : n;
  if (slot < 0 || slot >= a.nslots) {  // uniform over the workgroup, before any barrier
    for (int i = t; i < vw; i += kThreads) y[i] = from_f32<T>(0.f);
    return;
  }
  float* S = a.pool + (slot * a.HV + hv) * (int64_t)K * V + col;
  const T* xp = static_cast<const T*>(a.x) + n * a.ldx + (int64_t)hv * V;
  const bool active = rg < rgc;

  // the first rows of the state go out before anything is waited for
  vec_t s[kRows];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = r0 + u * rgc;
      if (active && r < K) s[u] = __builtin_nontemporal_load(reinterpret_cast<const vec_t*>(S + (int64_t)r * V));
    }
  };
  load(rg);
  const float raw = to_f32(static_cast<const T*>(a.dt)[n * a.lddt + hv]);
  if (t < K) {
    s_b[t] = to_f32(static_cast<const T*>(a.b)[n * a.ldb + (int64_t)h * K + t]);
    s_c[t] = to_f32(static_cast<const T*>(a.c)[n * a.ldc + (int64_t)h * K + t]);
  }
  float e, q;
  const float dt = softplus_f32(raw + (a.dt_bias ? a.dt_bias[hv] : 0.f), e, q);
  const float decay = decay_of(negative_rate(a.A_log[hv]) * dt * kLog2e);
  vec_t xd = {}, acc = {};
  if (active)
#pragma unroll
    for (int k = 0; k < VEC; ++k) xd[k] = dt * to_f32(xp[col + k]);
  block_barrier();
  for (int r0 = rg; r0 < K; r0 += kRows * rgc) {
    if (r0 != rg) load(r0);
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = r0 + u * rgc;
      if (active && r < K) {
        const vec_t v = decay * s[u] + s_b[r] * xd;
        acc += s_c[r] * v;
        __builtin_nontemporal_store(v, reinterpret_cast<vec_t*>(S + (int64_t)r * V));
      }
    }
  }
  if (active)
#pragma unroll
    for (int k = 0; k < VEC; ++k) s_y[(rg * nc + c) * VEC + k] = acc[k];
  block_barrier();
  const float skip = a.D ? a.D[hv] : 0.f;
  for (int i = t; i < vw; i += kThreads) {
    float sum = 0.f;
    for (int j = 0; j < min(rgc, K); ++j) sum += s_y[j * vw + i];
    y[i] = from_f32<T>(sum + skip * to_f32(xp[v0 + i]));
  }
}

template <typename T>
hipError_t run(const SsmArgs& a, hipStream_t stream) {
  const int heads = a.B * a.HV;
  const bool vec = a.V % 4 == 0 && reinterpret_cast<uintptr_t>(a.pool) % 16 == 0;
  const int nsplit = heads < 1024 && a.V % 16 == 0 ? 4 : 1;
  if (vec) hipLaunchKernelGGL((step_kernel<T, 4>), dim3(heads * nsplit), dim3(kThreads), 0, stream, a, nsplit);
  else hipLaunchKernelGGL((step_kernel<T, 1>), dim3(heads * nsplit), dim3(kThreads), 0, stream, a, nsplit);
  return hipGetLastError();
}

}  // namespace ssm_step

hipError_t launch_ssm_step(const SsmArgs& a, hipStream_t stream) {
  return a.bf ? ssm_step::run<bf16>(a, stream) : ssm_step::run<float>(a, stream);
}

}  // namespace kda
