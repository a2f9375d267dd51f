// Rows of channels as the layer operators read them: elements of float32 or bf16, a vector of them a
// lane, or an 8-bit checkpoint of such a tensor (e4m3 codes, a power of two for every 32 neighbours).
#pragma once

#include "kda_device.h"

namespace kda {

// A tensor of tokens, or its checkpoint.
struct Source {
  const void* p;          // elements, or codes
  const uint8_t* scales;  // exponents of the codes' powers of two, or null: p holds elements
  int64_t ld;             // elements between tokens
};

constexpr int kScaleBlock = 32;  // neighbours that share a scale

// Rows of a Source from some token on, for buffer accesses: a row's offset is scalar, a lane's column the
// vector part. Offsets stay below 2^31: no more rows than that are asked for.
struct Rows {
  __amdgpu_buffer_rsrc_t p, scales;
  int ld, ld_scales;  // bytes between rows
};
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_at(const void* p, int64_t first, int64_t bytes) {
  char* q = const_cast<char*>(static_cast<const char*>(p)) + first;
  return __builtin_amdgcn_make_buffer_rsrc(q, 0, (int)bytes, 0x00020000);
}

// 2^(byte - 127), the scale that a checkpoint's byte stands for (byte <= 254; 0 is 2^-127).
__device__ __forceinline__ float scale_of(unsigned byte) {
  return __uint_as_float(byte ? byte << 23 : 1u << 22);
}

template <typename T, int VEC> struct RowVec {
  typedef T type __attribute__((ext_vector_type(VEC)));
};
template <typename T> struct RowVec<T, 1> { typedef T type; };

// VEC elements in the memory's type, and their float32 values.
template <typename T, int VEC> struct Piece {
  typename RowVec<T, VEC>::type raw;

  // ONCE: past the caches (kCached).
  template <bool ONCE = false> __device__ __forceinline__ void load(const void* p, int64_t off) {
    const auto* q = reinterpret_cast<const typename RowVec<T, VEC>::type*>(static_cast<const T*>(p) + off);
    if constexpr (ONCE) raw = __builtin_nontemporal_load(q);
    else raw = *q;
  }
  template <bool ONCE = false> __device__ __forceinline__ void load(const Source& s, int64_t off) { load<ONCE>(s.p, off); }
  // `rows` rows of D columns from `token` on, and a lane's piece of one (row uniform over the wave).
  static __device__ __forceinline__ Rows rows(const void* p, int64_t ld, int64_t token, int rows, int D) {
    const int64_t step = ld * (int64_t)sizeof(T);
    Rows r;
    r.p = rows_at(p, token * step, (rows - 1) * step + D * (int64_t)sizeof(T));
    r.ld = (int)step;
    return r;
  }
  static __device__ __forceinline__ Rows rows(const Source& s, int64_t token, int n, int D) { return rows(s.p, s.ld, token, n, D); }
  __device__ __forceinline__ void load(const Rows& r, int row, int col) {
    const int off = col * (int)sizeof(T);
    if constexpr (sizeof(raw) == 8) raw = __builtin_bit_cast(decltype(raw), __builtin_amdgcn_raw_buffer_load_b64(r.p, off, row * r.ld, 0));
    else if constexpr (sizeof(raw) == 4) raw = __builtin_bit_cast(decltype(raw), __builtin_amdgcn_raw_buffer_load_b32(r.p, off, row * r.ld, 0));
    else raw = __builtin_bit_cast(decltype(raw), __builtin_amdgcn_raw_buffer_load_b16(r.p, off, row * r.ld, 0));
  }
  template <bool ONCE = false> __device__ __forceinline__ void store(const Rows& r, int row, int col) const {
    constexpr int kHow = ONCE ? 2 : 0;  // 2: non-temporal
    const int off = col * (int)sizeof(T);
    typedef unsigned two __attribute__((ext_vector_type(2)));
    if constexpr (sizeof(raw) == 8) __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(two, raw), r.p, off, row * r.ld, kHow);
    else if constexpr (sizeof(raw) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, raw), r.p, off, row * r.ld, kHow);
    else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, raw), r.p, off, row * r.ld, kHow);
  }
  __device__ __forceinline__ void get(float (&v)[VEC]) const {
    if constexpr (VEC == 1) v[0] = to_f32(raw);
    else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = to_f32(raw[e]);
    }
  }
  __device__ __forceinline__ void set(const float (&v)[VEC]) {
    if constexpr (VEC == 1) raw = from_f32<T>(v[0]);
    else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) raw[e] = from_f32<T>(v[e]);
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t off) const {
    *reinterpret_cast<typename RowVec<T, VEC>::type*>(static_cast<T*>(p) + off) = raw;
  }
};

// VEC codes of a checkpoint and their scale; off is a multiple of VEC, so that one scale serves them.
template <int VEC> struct PackedPiece {
  static constexpr int kWords = VEC > 4 ? VEC / 4 : 1;
  unsigned word[kWords];
  unsigned byte;

  template <bool ONCE = false> __device__ __forceinline__ void load(const Source& s, int64_t off) {
    const uint8_t* c = static_cast<const uint8_t*>(s.p) + off;
    typedef unsigned two __attribute__((ext_vector_type(2)));
    if constexpr (VEC == 8) {
      const two* q = reinterpret_cast<const two*>(c);
      const two v = ONCE ? __builtin_nontemporal_load(q) : *q;
      word[0] = v[0], word[1] = v[1];
    } else if constexpr (VEC == 4 && ONCE) word[0] = __builtin_nontemporal_load(reinterpret_cast<const unsigned*>(c));
    else if constexpr (VEC == 4) word[0] = *reinterpret_cast<const unsigned*>(c);
    else if constexpr (VEC == 2) word[0] = *reinterpret_cast<const unsigned short*>(c);
    else word[0] = *c;
    byte = s.scales[off / kScaleBlock];
  }
  static __device__ __forceinline__ Rows rows(const Source& s, int64_t token, int n, int D) {
    const int64_t few = s.ld / kScaleBlock;
    Rows r;
    r.p = rows_at(s.p, token * s.ld, (n - 1) * s.ld + D);
    r.scales = rows_at(s.scales, token * few, n * few);
    r.ld = (int)s.ld, r.ld_scales = (int)few;
    return r;
  }
  static __device__ __forceinline__ unsigned codes(const Rows& r, int row, int col) {
    static_assert(VEC <= 4, "a word of codes a lane");
    if constexpr (VEC == 4) return __builtin_amdgcn_raw_buffer_load_b32(r.p, col, row * r.ld, 0);
    else if constexpr (VEC == 2) return __builtin_amdgcn_raw_buffer_load_b16(r.p, col, row * r.ld, 0);
    else return __builtin_amdgcn_raw_buffer_load_b8(r.p, col, row * r.ld, 0);
  }
  __device__ __forceinline__ void get(float (&v)[VEC]) const {
    const float f = scale_of(byte);
    if constexpr (VEC == 1) v[0] = f * __builtin_amdgcn_cvt_f32_fp8(word[0], 0);
    else {
#pragma unroll
      for (int e = 0; e < VEC; e += 2) {
        const auto two = (e & 2) ? __builtin_amdgcn_cvt_pk_f32_fp8(word[e / 4], true)
                                 : __builtin_amdgcn_cvt_pk_f32_fp8(word[e / 4], false);
        v[e] = f * two[0];
        v[e + 1] = f * two[1];
      }
    }
  }
};

// Bytes that the last-level cache holds. A call that moves more reads its tensors past the caches, in its form of
// whole 16-byte pieces (the narrower forms read through them). What that gains depends on where the outputs are.
// Past the caches and through them, 32768 rows of 2048 channels in bf16, in us:
//                                            outputs last written long ago    by the call before
//   in front of a block                             102 and 102                    85 and 102
//   behind, under a gate                             74 and  77                    68 and  77
//   in front, backward                              167 and 168                   157 and 168
//   behind, backward                                148 and 140                   134 and 141
//   in front, backward, from checkpoints            154 and 154                   147 and 153
//   behind, backward, from checkpoints              136 and 133                   132 and 133
// 12288 rows, whose inputs may still be there, in front of a block 42 and 44, 40 and 40. The norms store through
// the caches; past them, too, the first case takes 96 us in both places.
constexpr int64_t kCached = (int64_t)256 << 20;

// What a backward pass reads of the forward's inputs: elements, or a checkpoint of them.
template <typename T, int VEC, bool CK> struct KeptPiece { typedef Piece<T, VEC> type; };
template <typename T, int VEC> struct KeptPiece<T, VEC, true> { typedef PackedPiece<VEC> type; };

// logistic(z) and 1 - logistic(z), each to float32 accuracy of its own.
__device__ __forceinline__ void logistic_pair(float z, float& s, float& rest) {
  const float e = fast_exp2(-fabsf(z) * kLog2e), r = __builtin_amdgcn_rcpf(1.f + e), l = e * r;
  s = z >= 0.f ? r : l;
  rest = z >= 0.f ? l : r;
}

// Column sums in a fixed order: out[k][c] = sum over the nb row blocks j of part[j][k][c], for K
// vectors of D columns (a null out is not wanted).
struct ColumnSums {
  const float* part;  // [nb][K][D]
  float* out[2];
  int nb, K, D;
};
hipError_t launch_column_sums(const ColumnSums& a, hipStream_t stream);

// The largest vector, of `most` elements or a half, a quarter ... of them, that the widths and strides
// (or-ed together) and the addresses allow.
inline int vector_width(int most, int esize, int64_t widths, const void* const* ptrs, int n) {
  uintptr_t bits = 0;
  for (int i = 0; i < n; ++i) bits |= reinterpret_cast<uintptr_t>(ptrs[i]);
  int vec = most;
  while (vec > 1 && (widths % vec || bits % ((size_t)vec * esize))) vec /= 2;
  return vec;
}

}  // namespace kda
