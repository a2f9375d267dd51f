// Activation checkpoints in 8 bits: a tensor that the forward pass keeps for the backward pass, in
// e4m3 codes with one power of two for every 32 neighbours of a row (33 bytes instead of 64 of bf16).
//
// Of 32 neighbours with the largest finite magnitude m, the scale is the smallest power of two
// 2^(byte - 127), byte >= 0, with m <= 448 2^(byte - 127) (448: the largest code), and a code is the
// element divided by it, rounded to nearest even: off by at most 2^-4 of the element, or by 2^-10 of
// the scale where the code is below 2^-6. Dividing by a power of two is exact, so the code is rounded
// once and reading it back gives a float exactly. Infinities and NaN become the NaN code and leave
// their neighbours as they are.
//
// Both directions move every byte once and are bound by HBM: a lane holds 8 elements (16 bytes of
// bf16, 8 of codes), four lanes share a scale and find it with two lane swaps; a thread takes several
// such pieces at a time, so that their loads are in flight together. Measured at 32768 x 2048 bf16:
// writing 42 us (203 MB), reading back 30 us; 71 for both (5.7 TB/s).
#include "kda_rows.h"

namespace kda {
namespace checkpoint {

constexpr int kThreads = 256;
constexpr int kVec = 8;                     // elements of a lane; kScaleBlock / kVec lanes share a scale
constexpr int kPieces = 4;                  // of a thread

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// 8 elements at p[off], as vectors of VEC (8: 16 bytes of bf16 or twice 16 of float32; or one by one).
template <typename T, int VEC, bool ONCE> __device__ __forceinline__ void read8(const T* p, float (&v)[kVec]) {
#pragma unroll
  for (int i = 0; i < kVec; i += VEC) {
    Piece<T, VEC> q;
    q.template load<ONCE>(p, i);
    float f[VEC];
    q.get(f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[i + e] = f[e];
  }
}

// Row and column of piece i, of a row of `per` pieces.
struct Place {
  int64_t row;
  int col;
};
__device__ __forceinline__ Place place(int64_t i, int per) {
  // 2^31 scale blocks at most, so 2^33 pieces: 32-bit division by blocks, then the lane in the block
  const unsigned block = (unsigned)(i / (kScaleBlock / kVec)), blocks = per / (kScaleBlock / kVec);
  const unsigned row = block / blocks;
  return {(int64_t)row, (int)(block - row * blocks) * kScaleBlock + (int)(i % (kScaleBlock / kVec)) * kVec};
}

template <typename T, int VEC, bool ONCE>
__global__ __launch_bounds__(kThreads) void pack_kernel(const T* __restrict__ x, int64_t ldx, uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales, int64_t pieces, int per) {
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kPieces) + threadIdx.x;
  float v[kPieces][kVec];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const Place at = place(min(first + u * kThreads, pieces - 1), per);
    read8<T, VEC, ONCE>(x + at.row * ldx + at.col, v[u]);
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < kVec; ++e) m = fmaxf(m, finite(v[u][e]) ? fabsf(v[u][e]) : 0.f);
    m = fmaxf(m, __shfl_xor(m, 1));
    m = fmaxf(m, __shfl_xor(m, 2));
    // m = (1 + f) 2^(k - 127): the scale's exponent is k - 8, and one more where 1 + f > 448 / 256.
    // A denormal m (k = 0) is far below 448 2^-127 and gets the smallest scale.
    const unsigned bits = __float_as_uint(m), k = bits >> 23;
    const unsigned mant = bits & 0x7fffffu;
    int byte = (int)k - 8 + (mant > 0x600000u ? 1 : 0);
    byte = byte < 0 ? 0 : byte;
    const float inv = scale_of(254 - byte);  // 2^(127 - byte); byte <= 247
    const int64_t i = first + u * kThreads;
    if (i >= pieces) continue;  // whole scale blocks: pieces is a multiple of the lanes that share one
    int word[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float s = v[u][4 * h + e];
        q[e] = finite(s) ? s * inv : __builtin_nanf("");
      }
      int wd = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
      word[h] = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], wd, true);
    }
    *reinterpret_cast<int2*>(codes + i * kVec) = make_int2(word[0], word[1]);
    if (i % (kScaleBlock / kVec) == 0) scales[i / (kScaleBlock / kVec)] = (uint8_t)byte;
  }
}

template <typename T, int VEC>
__global__ __launch_bounds__(kThreads) void unpack_kernel(Source s, T* __restrict__ x, int64_t pieces) {
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kPieces) + threadIdx.x;
  PackedPiece<kVec> q[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) q[u].load(s, min(first + u * kThreads, pieces - 1) * kVec);
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int64_t i = first + u * kThreads;
    if (i >= pieces) continue;
    float v[kVec];
    q[u].get(v);
#pragma unroll
    for (int j = 0; j < kVec; j += VEC) {
      Piece<T, VEC> o;
      float f[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = v[j + e];
      o.set(f);
      o.store(x, i * kVec + j);
    }
  }
}

inline unsigned blocks_of(int64_t pieces) {
  return (unsigned)((pieces + kThreads * kPieces - 1) / (kThreads * kPieces));
}

}  // namespace checkpoint

hipError_t launch_checkpoint_pack(const void* x, int64_t ldx, uint8_t* codes, uint8_t* scales, int64_t rows, int D,
                                  bool bf, hipStream_t stream) {
  using namespace checkpoint;
  const int64_t pieces = rows * (D / kVec);
  if (pieces == 0) return hipSuccess;
  const dim3 grid(blocks_of(pieces)), block(kThreads);
  const int vec = vector_width(bf ? 8 : 4, bf ? 2 : 4, ldx, &x, 1);
  const bool once = rows * D * (bf ? 3 : 5) > kCached;
  auto go = [&](auto kernel, auto* p) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, p, ldx, codes, scales, pieces, D / kVec);
  };
  if (bf) {
    const bf16* p = static_cast<const bf16*>(x);
    vec < 8 ? go(pack_kernel<bf16, 1, false>, p) : once ? go(pack_kernel<bf16, 8, true>, p) : go(pack_kernel<bf16, 8, false>, p);
  } else {
    const float* p = static_cast<const float*>(x);
    vec < 4 ? go(pack_kernel<float, 1, false>, p) : once ? go(pack_kernel<float, 4, true>, p) : go(pack_kernel<float, 4, false>, p);
  }
  return hipGetLastError();
}

hipError_t launch_checkpoint_unpack(const uint8_t* codes, const uint8_t* scales, void* x, int64_t rows, int D,
                                    bool bf, hipStream_t stream) {
  using namespace checkpoint;
  const int64_t pieces = rows * (D / kVec);
  if (pieces == 0) return hipSuccess;
  const dim3 grid(blocks_of(pieces)), block(kThreads);
  const Source s{codes, scales, D};
  const void* p = x;
  const int vec = vector_width(bf ? 8 : 4, bf ? 2 : 4, 0, &p, 1);
  auto go = [&](auto kernel, auto* q) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, s, q, pieces); };
  if (bf) vec == 8 ? go(unpack_kernel<bf16, 8>, static_cast<bf16*>(x)) : go(unpack_kernel<bf16, 1>, static_cast<bf16*>(x));
  else vec == 4 ? go(unpack_kernel<float, 4>, static_cast<float*>(x)) : go(unpack_kernel<float, 1>, static_cast<float*>(x));
  return hipGetLastError();
}

}  // namespace kda
