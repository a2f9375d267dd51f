// Selective state space scan over whole sequences: the recurrence with one scalar decay per
// head that hybrid stacks put beside the gated delta rule. Per value head, K x V float32 state S:
//   D_t = softplus(dt_t + dt_bias),  a_t = exp(-exp(A_log) D_t)      (the KDA decay gate's form)
//   S_t = a_t S_{t-1} + b_t (D_t x_t)^T,     y_t = S_t^T c_t + D x_t
// HV value heads share H pairs of b and c (value head hv reads pair hv / (HV / H)).
//
// Tiles of 64 tokens, with G the in-tile inclusive sum of log2 a (so every exponent below is of a
// difference <= 0):
//   M[i, j] = (c_i . b_j) 2^(G_i - G_j) D_j  for j <= i, else 0
//   y_i     = sum_j M[i, j] x_j + 2^(G_i) S^T c_i + D x_i
//   S      <- 2^(G_63) S + sum_j b_j (2^(G_63 - G_j) D_j x_j)^T
// The products run on the matrix cores (16x16x32 bf16, float32 accumulators). M and the S that y
// reads are rounded to bf16, as y is; the state itself keeps float32 accuracy: b is bf16 as given,
// and the weighted x of its update is split into three bf16 terms (8 bits each), three products.
//
// A workgroup of four waves owns 64 or 128 columns: one or two value heads of one b / c pair, whose
// b, c and c . b products they share, and carries the state in accumulators (16 PT columns a wave)
// over the tiles of one segment of the token axis. Segments have equal lengths whatever the
// sequences: a tile ends at the sequence's end. With more than one segment, a pass over the tiles
// of each boundary's sequence without outputs (OUT = false) gives the state that leaves the
// segment, a scan composes them, and the pass with outputs starts from the composed states.
// float32 inputs take the same steps with tiles of 32 tokens, 16x16x4 float32 products and nothing
// rounded.
//
// Such products multiply every x of a tile, also with zeros of M, so a sequence with an x that is not
// finite goes another way (by_token()). The passes find that out from the sum of the squares of all x,
// 16 dot products a lane and tile: 355 -> 358 us at the sizes below.
//
// Measured at 4 x 8192 tokens, 64 heads x 64, K = 128, 8 pairs, bf16: 358 us for 684 MB, 114 us at
// a copy's rate (traced: 254 pass with outputs, 117 without, 15 composition). Before the squares a tile
// of two heads took a workgroup about 14,300 cycles beside a second one on its CU: 2,050 for M, 3,500
// for y, 4,100 for the state, 2,000 until the next tile's loads are issued, 760 for LDS stores. No
// single pipeline is full (VALU 44%, matrix cores 31%, LDS 34% of the cycles). Tiles of 32 tokens were
// 5% slower, 256 or 768 workgroups 29% and 12%, each against the kernel of its day; eight waves of 16
// columns were the same. float32 at these sizes: 1,365 us (50 TFLOP/s of the recurrence's operations).
#include <type_traits>

#include "kda_ssm.h"

namespace kda {
namespace ssm {

// Tokens of a tile. float32 takes half as many: its products are 16 times as expensive, and those
// inside a tile grow with it.
template <typename T> constexpr int kTokens = sizeof(T) == 2 ? 64 : 32;
constexpr int kThreads = 256;
constexpr unsigned kOutOfRange = 0x80000000u;  // buffer loads there read zeros

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) unsigned char lds_u8;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, unsigned bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// Four bf16 by the LDS transpose load: in each 16-lane group, lane l receives element l % 4 of
// the 8-byte pieces addressed by lanes 4e + l / 4, e = 0 .. 3.
__device__ __forceinline__ bf16x4 load_tr4(const bf16* p) {
#if __HIP_DEVICE_COMPILE__
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                        (__attribute__((address_space(3))) s16x4*)(lds_u8*)p));
#else
  (void)p;
  return bf16x4{};
#endif
}

__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f32x4 mfma(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// A tile: tokens t0 .. t0 + rows - 1 of sequence seq; first / last: holds its first / last token.
struct Tile {
  int t0, rows, seq, eos;  // eos: the sequence's end
  bool first, last;
};

// A ROWS x COLS matrix on its way from memory to LDS: each thread holds pieces of 16 bytes.
// Columns are blocks of PAD, of which `width` are real. VEC: every real row of a block is whole
// 16-byte pieces, aligned in memory.
template <typename T, int ROWS, int COLS, int PAD, bool VEC>
struct Stage {
  static constexpr int kElem = 16 / sizeof(T), kRow = COLS / kElem;
  static constexpr int kPieces = (ROWS * kRow + kThreads - 1) / kThreads;
  static_assert(kPieces * kThreads == ROWS * kRow, "every thread holds as many");
  u32x4 v[kPieces];

  // base: column 0 of token 0; ld: elements between tokens (<= 2^24); tokens behind t0 + rows and
  // columns behind `width` of a block read zeros.
  __device__ __forceinline__ void load(const T* base, int ld, int t0, int rows, int width) {
    constexpr int kBlocks = COLS / PAD;
    // up to the last row's last column, without a branch; nothing for no rows
    const unsigned elems = (unsigned)(rows * ld) - (unsigned)(min(rows, 1) * (ld - kBlocks * width));
    const __amdgpu_buffer_rsrc_t r = make_rsrc(base + (int64_t)t0 * ld, elems * (unsigned)sizeof(T));
    const unsigned rowb = (unsigned)ld * (unsigned)sizeof(T);
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
      const int piece = threadIdx.x + kThreads * e, row = piece / kRow, c = piece % kRow * kElem;
      const int blk = c / PAD, p = c - blk * PAD;
      const unsigned off = (unsigned)row * rowb + (unsigned)(blk * width + p) * sizeof(T);
      auto in = [&](int k) { return p + k < width ? off + k * (unsigned)sizeof(T) : kOutOfRange; };
      if constexpr (VEC) {
        v[e] = __builtin_amdgcn_raw_buffer_load_b128(r, in(0), 0, 0);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (sizeof(T) == 4) {
            v[e][k] = __builtin_amdgcn_raw_buffer_load_b32(r, in(k), 0, 0);
          } else {
            const unsigned lo = __builtin_amdgcn_raw_buffer_load_b16(r, in(2 * k), 0, 0);
            const unsigned hi = __builtin_amdgcn_raw_buffer_load_b16(r, in(2 * k + 1), 0, 0);
            v[e][k] = lo | hi << 16;
          }
        }
      }
    }
  }
  __device__ __forceinline__ void store(T* dst, int ldd) const {
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
      const int piece = threadIdx.x + kThreads * e, row = piece / kRow, c = piece % kRow * kElem;
      *reinterpret_cast<u32x4*>(dst + row * ldd + c) = v[e];
    }
  }
  // Adds the squares of this thread's values: the sum is finite only if all of them are under 2^64.
  __device__ __forceinline__ void add_squares(float& sum) const {
#pragma unroll
    for (int e = 0; e < kPieces; ++e)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const unsigned u = v[e][k];
        if constexpr (sizeof(T) == 4) {
          sum = fmaf(__builtin_bit_cast(float, u), __builtin_bit_cast(float, u), sum);
        } else {
#if __HIP_DEVICE_COMPILE__
          sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, u), __builtin_bit_cast(bf16x2, u), sum, false);
#endif
        }
      }
  }
};

// Per token and head of a tile: what the state's products take, and what M takes. Exponents are of
// differences of G in float64.
struct Decay {
  float eg[64], w[64];  // 2^G, and D 2^(G_63 - G)
  float end, pad[3];    // G_63, the whole tile's
};
constexpr float kFactorSpan = 64.f;
struct Inner {
  float dt[64], hi[64], lo[64];  // D, and G as a sum of two floats (log2 units)
  // M between token i of a block of 16 tokens and token j at or in front of its end, over the last
  // token q in front of the block (G_q = 0 for the first): row[i] = 2^(G_i - G_q) <= 1, and
  // col[8 it (it + 1) + j] = D_j 2^(G_q - G_j) for block it. For j inside the block that factor is
  // at most 2^kFactorSpan D_j, unless `wide` says that some block decays further than that.
  float row[64], col[160];
  int wide, pad[3];
};

// v of the lane `OP` names (a DPP control); lanes without one, or masked out, get 0.
template <int OP, int ROWS>
__device__ __forceinline__ double dpp_or_zero(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)(unsigned)u, OP, ROWS, 0xf, false);
  const unsigned hi = __builtin_amdgcn_update_dpp(0, (int)(unsigned)(u >> 32), OP, ROWS, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double read_lane(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const unsigned lo = __builtin_amdgcn_readlane((int)(unsigned)u, lane);
  const unsigned hi = __builtin_amdgcn_readlane((int)(unsigned)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// A decay below e^-1e6 is 0 in any case; without the bound an infinite rate would leave no differences.
__device__ __forceinline__ float bounded_rate(float rate) { return at_least(-1e6f, rate); }

// One wave: lane = token (those behind the tile's rows have D = 0). G is summed in float64, so
// that differences of two of its values keep float32 accuracy however large both are.
// BLOCKS: also what joins blocks of 16 tokens.
template <bool OUT, bool BLOCKS>
__device__ __forceinline__ void make_decay(Decay& d, Inner& m, float raw, bool in, float bias, float neg_rate) {
  const int lane = __lane_id();
  float e, r;
  const float dt = in ? softplus_f32(raw + bias, e, r) : 0.f;
  const float rate = in ? bounded_rate(neg_rate * dt) : 0.f;
  double g = (double)rate * 1.4426950408889634;
  g += dpp_or_zero<0x111, 0xf>(g);  // inclusive sums within rows of 16 lanes: shifts by 1, 2, 4, 8
  g += dpp_or_zero<0x112, 0xf>(g);
  g += dpp_or_zero<0x114, 0xf>(g);
  g += dpp_or_zero<0x118, 0xf>(g);
  g += dpp_or_zero<0x142, 0xa>(g);  // lane 15 of rows 0 and 2 to rows 1 and 3
  g += dpp_or_zero<0x143, 0xc>(g);  // lane 31 to rows 2 and 3
  const double end = read_lane(g, 63);
  d.w[lane] = dt * fast_exp2((float)(end - g));
  if (lane == 0) d.end = (float)end;
  if constexpr (OUT) {
    const float hi = (float)g;
    d.eg[lane] = decay_of(hi);
    m.dt[lane] = dt;
    m.hi[lane] = hi;
    m.lo[lane] = (float)(g - (double)hi);
  }
  if constexpr (BLOCKS) {
    double before = 0.0;  // G of the token in front of this lane's block
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const double q = it ? read_lane(g, 16 * it - 1) : 0.0;
      if (lane >= 16 * it) before = q;
      if (lane < 16 * (it + 1)) m.col[8 * it * (it + 1) + lane] = dt * fast_exp2((float)(q - g));
    }
    const float f = (float)(g - before);
    m.row[lane] = fast_exp2(f);
    const bool wide = wave_any(!(f >= -kFactorSpan));
    if (lane == 0) m.wide = wide;
  }
}

// Two floats rounded to bf16 in one register, and back.
__device__ __forceinline__ unsigned pack2(float a, float b) {
  return __builtin_bit_cast(unsigned, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ float low(unsigned u) { return __builtin_bit_cast(float, u << 16); }
__device__ __forceinline__ float high(unsigned u) { return __builtin_bit_cast(float, u & 0xffff0000u); }

// The part of the work that a workgroup takes: a segment, and columns of HB heads that share b and c.
struct Place {
  int segk, seg0, end;   // the segment, and its tokens
  int h0, v0, width, grp;  // first head, first column in it, real columns of each head, pair of b and c
  int pos, seq;          // the first token to look at, and its sequence
  bool carry;            // without outputs: the state that enters the segment reaches its end
  bool any;              // without outputs: a sequence goes on over the segment's end
};

// Workgroups that have a segment: with outputs every one, without those whose end a sequence may go on over.
template <bool OUT>
__device__ __forceinline__ int main_blocks(const SsmArgs& a, int hblocks) {
  const int inner = a.per > 0 ? a.per - 1 : a.nseg - 1;
  return hblocks * (OUT ? a.nseg : a.per > 0 ? a.N * inner : inner);
}

template <int PP, int HB, bool OUT>
__device__ __forceinline__ Place place_of(const SsmArgs& a, int hblocks, int bid) {
  Place w;
  const int vblocks = (a.V + PP - 1) / PP, inner = a.per > 0 ? a.per - 1 : a.nseg - 1;
  const int blocks = main_blocks<OUT>(a, hblocks);
  // neighbouring head blocks (which share b and c) on one XCD: workgroups are dealt out
  // round-robin over the 8 of them
  if (blocks % 8 == 0) bid = (bid & 7) * (blocks / 8) + (bid >> 3);
  w.segk = bid / hblocks;
  const int hb = bid - w.segk * hblocks;
  if (!OUT && a.per > 0) w.segk = w.segk / inner * a.per + w.segk % inner;
  w.h0 = hb / vblocks * HB, w.v0 = hb % vblocks * PP;
  w.width = min(PP, a.V - w.v0);
  w.grp = w.h0 / (a.HV / a.H);
  w.seg0 = w.segk * a.seg;
  w.end = (int)min((int64_t)w.seg0 + a.seg, (int64_t)a.T);
  w.pos = w.seg0;
  w.carry = w.any = true;
  if constexpr (OUT) {
    w.seq = a.seqs.find(w.seg0);
  } else {
    // only the part of the sequence that goes on behind the segment's end
    w.seq = a.seqs.find(w.end - 1);
    const Span s = a.seqs.span(w.seq);
    w.any = s.eos > w.end && s.bos < w.end;
    w.carry = s.bos < w.seg0;
    w.pos = max(w.seg0, s.bos);
  }
  return w;
}

// The tile at or behind token t, looked for from sequence s on: rows == 0 if there is none in front of end.
template <int ROWS>
__device__ __forceinline__ Tile tile_at(const SsmArgs& a, int end, int t, int s) {
  while (t < end && s < a.N) {
    const Span sp = a.seqs.span(s);
    if (sp.eos <= t) { ++s; continue; }
    if (sp.bos > t) { t = sp.bos; continue; }
    const int rows = min(ROWS, min(sp.eos, end) - t);
    return Tile{t, rows, s, sp.eos, t == sp.bos, t + rows == sp.eos};
  }
  return Tile{end, 0, s, end, false, false};
}

// A value of x that the products of a tile do not take: not finite, or so large that D x may be past the
// largest bf16. Its square is infinite or NaN.
__device__ __forceinline__ bool odd_value(float v) { return !(fabsf(v) < 0x1p64f); }

// The sequences of a workgroup's segment that hold an odd x, as the recurrence is defined: token by
// token. Products of a whole tile are no form of it there: the zeros of M times an infinity are NaN in
// tokens in front of it, and an infinity less its own first term is NaN in the state. Runs behind the
// products and writes over what they left in these sequences. It is rare, so it is written for few
// registers, and not inlined, so that the products' loop is compiled as if it were not there (inlined:
// 378 us instead of 366 at 4 x 8192 tokens, 64 heads x 64, K = 128). One NaN there: 5.9 ms, 4096 tokens
// in each of the two passes.
// SPLIT threads share a column, each has R rows of the state. args: the kernel's SsmArgs.
typedef const __attribute__((address_space(4))) unsigned* arg_words;
template <typename X> using lds = __attribute__((address_space(3))) X;
template <typename T, int NP, int PP, int HB, bool OUT, int LDX, int LDB, int LDC>
__device__ __attribute__((noinline)) void by_token(arg_words args, int hblocks, int bid, int tid,
                                                    lds<T>* Xs, lds<T>* Bs, lds<T>* Cs,
                                                    lds<Decay>* dec, lds<int>* s_odd) {
  constexpr int XC = HB * PP, SPLIT = kThreads / XC, R = NP / SPLIT, kTok = kTokens<T>;
  static_assert(SPLIT * XC == kThreads && R * SPLIT == NP, "whole columns");
  static_assert(PP % (64 / SPLIT) == 0, "a wave's columns are of one head");
  // arguments of a function arrive in vector registers: uniform ones go back to scalar ones
  const uint64_t words = (uint64_t)args;
  args = (arg_words)((uint64_t)(unsigned)__builtin_amdgcn_readfirstlane((int)(words >> 32)) << 32 |
                     (unsigned)__builtin_amdgcn_readfirstlane((int)words));
  SsmArgs a;
#pragma unroll
  for (unsigned i = 0; i < sizeof(a) / 4; ++i) reinterpret_cast<unsigned*>(&a)[i] = args[i];
  const Place w = place_of<PP, HB, OUT>(a, __builtin_amdgcn_readfirstlane(hblocks), __builtin_amdgcn_readfirstlane(bid));
  const int K = a.K, V = a.V, k = tid % SPLIT, col = tid / SPLIT, p = col % PP;
  const int head = __builtin_amdgcn_readfirstlane(col / PP);
  const int hv = w.h0 + head;
  const bool real = p < w.width;
  const int64_t sz = (int64_t)K * V, ldy = (int64_t)a.HV * V;
  const int at = w.v0 + p;
  const T* x = static_cast<const T*>(a.x) + (int64_t)w.h0 * V + w.v0;
  const T* b = static_cast<const T*>(a.b) + (int64_t)w.grp * K;
  const T* c = static_cast<const T*>(a.c) + (int64_t)w.grp * K;
  float s[R], gsum = 0.f;  // gsum: log2 of the decay so far
  // as in the products' pass: elements outside of [K, V] read zeros and are not written
  const unsigned state_bytes = (unsigned)(K * V * 4);
  auto each_row = [&](auto f) {
    unsigned off = real ? (unsigned)(k * R * V + at) * 4u : kOutOfRange;
#pragma unroll
    for (int r = 0; r < R; ++r, off += (unsigned)(V * 4)) {
      f(r, off);
      asm volatile("" : "+v"(off));
    }
  };
  auto load_state = [&](const float* src) {
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(src, src ? state_bytes : 0u);
    each_row([&](int r, unsigned off) { s[r] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0)); });
  };
  auto store_state = [&](float* dst) {
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(dst, state_bytes);
    each_row([&](int r, unsigned off) {
      const float v = s[r];
      __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v), rs, off, 0, 0);
    });
  };
  load_state(OUT && w.segk > 0 && a.seqs.span(w.seq).bos < w.seg0 ? a.seg_state + ((int64_t)(w.segk - 1) * a.HV + hv) * sz
                                                                   : nullptr);
  const float skip = a.D ? a.D[hv] : 0.f;
  for (Tile t = tile_at<kTok>(a, w.end, w.pos, w.seq); t.rows > 0;) {
    const int stop = min(t.eos, w.end);  // of the sequence's part
    bool odd = false;
    // column tid % XC of every (kThreads / XC)-th token
    const int j = tid % XC / PP * V + tid % PP;
    if (tid % PP < w.width)
#pragma unroll 8
      for (int i = t.t0 + tid / XC; i < stop; i += SPLIT) odd |= odd_value(to_f32(x[i * a.ldx + j]));
    block_barrier();
    if (tid == 0) *s_odd = 0;
    block_barrier();
    if (odd) *s_odd = 1;  // any writer stores the same
    block_barrier();
    if (*s_odd == 0) {
      t = tile_at<kTok>(a, w.end, stop, t.seq);
      continue;
    }
    for (; t.t0 < stop && t.rows > 0; t = tile_at<kTok>(a, w.end, t.t0 + t.rows, t.seq)) {
      if (t.first) load_state(a.s0 ? a.s0 + ((int64_t)t.seq * a.HV + hv) * sz : nullptr);
      block_barrier();
      // rows of `width` elements, n of them for every token, to LDS
      auto stage = [&](lds<T>* dst, int ldd, const T* src, int64_t ld, auto n, int width) {
        constexpr int kCols = decltype(n)::value;
        const int e = tid % kCols;
        if (e % kCols < width)
#pragma unroll 8
          for (int i = tid / kCols; i < t.rows; i += kThreads / kCols) dst[i * ldd + e] = src[(t.t0 + i) * ld + e];
        else
          for (int i = tid / kCols; i < t.rows; i += kThreads / kCols) dst[i * ldd + e] = from_f32<T>(0.f);
      };
      for (int h = 0; h < HB; ++h) stage(Xs + h * PP, LDX, x + (int64_t)h * V, a.ldx, std::integral_constant<int, PP>{}, w.width);
      stage(Bs, LDB, b, a.ldb, std::integral_constant<int, NP>{}, K);
      if constexpr (OUT) stage(Cs, LDC, c, a.ldc, std::integral_constant<int, NP>{}, K);
      if (tid < t.rows)
        for (int h = 0; h < HB; ++h) {
          float e, q;
          const float raw = to_f32(static_cast<const T*>(a.dt)[(int64_t)(t.t0 + tid) * a.lddt + w.h0 + h]);
          const float dt = softplus_f32(raw + (a.dt_bias ? a.dt_bias[w.h0 + h] : 0.f), e, q);
          dec[h].w[tid] = dt;
          dec[h].eg[tid] = bounded_rate(negative_rate(a.A_log[w.h0 + h]) * dt) * kLog2e;
        }
      block_barrier();
#pragma unroll 1
      for (int i = 0; i < t.rows; ++i) {
        const float g = dec[head].eg[i], decay = decay_of(g), xv = to_f32(Xs[i * LDX + col]), dx = dec[head].w[i] * xv;
        float sum = 0.f;
        gsum += g;
        int left = K - k * R;  // rows of the state from this thread's first one on
        asm volatile("" : "+v"(left));  // compared anew for every token: masks would fill the registers
        const lds<T>* bi = Bs + i * LDB + k * R;
        const lds<T>* ci = Cs + (OUT ? i * LDC + k * R : 0);
        typedef T t4 __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int r = 0; r < R; r += 4) {
          const t4 b4 = *(const lds<t4>*)(bi + r);
          const t4 c4 = *(const lds<t4>*)(ci + (OUT ? r : 0));
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float xr = r + u < left ? dx : 0.f;  // rows behind K, which b and c do not have, stay zero
            s[r + u] = decay * s[r + u] + to_f32(b4[u]) * xr;
            if constexpr (OUT) sum += s[r + u] * to_f32(c4[u]);
          }
          if (r % 8 == 4) asm volatile("" : "+v"(left)::"memory");  // few registers rather than speed
        }
        if constexpr (OUT) {
#pragma unroll
          for (int off = 1; off < SPLIT; off *= 2) sum += __shfl_xor(sum, off);
          if (k == 0 && real) static_cast<T*>(a.y)[(t.t0 + i) * ldy + (int64_t)hv * V + at] = from_f32<T>(sum + skip * xv);
        }
      }
      if (OUT && t.last && a.sT) store_state(a.sT + ((int64_t)t.seq * a.HV + hv) * sz);
      if (!OUT && t.t0 + t.rows == w.end) {
        store_state(a.seg_state + ((int64_t)w.segk * a.HV + hv) * sz);
        if (at == 0 && k == 0) a.seg_g[(int64_t)w.segk * a.HV + hv] = w.carry ? gsum : -INFINITY;
      }
    }
  }
}

// NT: K in tiles of 16; HB heads of PP columns; PT tiles of 16 columns a wave.
template <typename T, int NT, int PP, int HB, int PT, bool OUT, bool VEC>
__global__ __launch_bounds__(kThreads, 2) void prefill_kernel(SsmArgs a, int hblocks) {
  constexpr int NW = kThreads / 64;
  constexpr bool BF = sizeof(T) == 2;
  constexpr int kTok = kTokens<T>, kPad = 16 / sizeof(T);
  constexpr int XC = HB * PP, NP = 16 * NT, LDX = XC + kPad, LDM = kTok + kPad, KS = NT / 2;
  // rows of b and c in LDS: c is read 16 bytes a lane along rows, b also four rows at a time; the
  // row lengths with the fewest bank conflicts for these (cycles of a 1 KB read: c 4 instead of 6
  // at 272 bytes a row, b 6 and, transposed, 3.4 instead of 6)
  constexpr int LDC = BF ? NP + 16 : NP + 4, LDB = BF ? (NT == 8 ? 160 : 104) : NP + 4;
  static_assert(BF || PT == 1, "float32 products take the wave's columns in order");
  static_assert(XC <= 16 * PT * NW && NT % 2 == 0 && PP % (16 * PT) == 0, "tile shape");
  __shared__ __attribute__((aligned(16))) T Xs[kTok * LDX];
  __shared__ __attribute__((aligned(16))) T Bs[kTok * LDB];
  __shared__ __attribute__((aligned(16))) T Cs[OUT ? kTok * LDC : 8];
  __shared__ __attribute__((aligned(16))) T Ms[OUT ? HB * kTok * LDM : 8];
  __shared__ __attribute__((aligned(16))) Decay s_dec[2][HB];
  __shared__ __attribute__((aligned(16))) Inner s_in[OUT ? HB : 1];  // read in front of a tile's second barrier only
  __shared__ int s_odd[NW];

  const int K = a.K, V = a.V;
  if (OUT && (int)blockIdx.x >= main_blocks<OUT>(a, hblocks)) {  // empty sequences: the state passes through
    const int n = blockIdx.x - main_blocks<OUT>(a, hblocks);
    const Span s = a.seqs.span(n);
    if (s.eos > s.bos) return;
    const int64_t sz = (int64_t)a.HV * K * V;
    for (int64_t i = threadIdx.x; i < sz; i += kThreads) a.sT[n * sz + i] = a.s0 ? a.s0[n * sz + i] : 0.f;
    return;
  }
  const Place w = place_of<PP, HB, OUT>(a, hblocks, blockIdx.x);
  const int segk = w.segk, h0 = w.h0, v0 = w.v0, width = w.width, grp = w.grp, end = w.end;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int lr = lane & 15, lq = lane >> 4;
  const int col0 = wv * 16 * PT, hh = col0 / PP, p0 = v0 + col0 - hh * PP;
  const bool active = XC == 16 * PT * NW || hh < HB;  // waves behind the last head only help with c . b
  const int hv = h0 + (active ? hh : 0);
  const int dw = wv - (NW - HB);  // the last HB waves prepare the decays of head dw
  if (!w.any) {
    if (wv == 0 && lane < HB && v0 == 0) a.seg_g[(int64_t)segk * a.HV + h0 + lane] = kNoCarry;
    return;
  }

  T* y = static_cast<T*>(a.y);
  const int64_t ldy = (int64_t)a.HV * V;
  // rows [t, to) lie in no sequence
  auto outside = [&](int t, int to) {
    if (!OUT || !a.zero_rest || t >= to) return;
    for (; t < to; ++t)
      for (int i = threadIdx.x; i < HB * width; i += kThreads)
        y[t * ldy + (int64_t)(h0 + i / width) * V + v0 + i % width] = from_f32<T>(0.f);
  };

  Stage<T, kTok, XC, PP, VEC> xr;
  Stage<T, kTok, NP, NP, VEC> br, cr;
  T dtr = from_f32<T>(0.f);
  const int ldx = (int)a.ldx, ldb = (int)a.ldb, ldc = (int)a.ldc, lddt = (int)a.lddt;
  auto load = [&](const Tile& t) {
    xr.load(static_cast<const T*>(a.x) + (int64_t)h0 * V + v0, ldx, t.t0, t.rows, width);
    br.load(static_cast<const T*>(a.b) + (int64_t)grp * K, ldb, t.t0, t.rows, K);
    if constexpr (OUT) cr.load(static_cast<const T*>(a.c) + (int64_t)grp * K, ldc, t.t0, t.rows, K);
    const __amdgpu_buffer_rsrc_t rd = make_rsrc(static_cast<const T*>(a.dt) + (int64_t)t.t0 * lddt + h0, 0x7fffffffu);
    const unsigned off = dw >= 0 && lane < t.rows ? (unsigned)(lane * lddt + dw) * (unsigned)sizeof(T) : kOutOfRange;
    if constexpr (BF) dtr = __builtin_bit_cast(T, (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(rd, off, 0, 0));
    else dtr = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(rd, off, 0, 0));
  };
  float bias = 0.f, neg_rate = 0.f;
  if (dw >= 0) {
    bias = a.dt_bias ? a.dt_bias[h0 + dw] : 0.f;
    neg_rate = negative_rate(a.A_log[h0 + dw]);
  }
  const float skip = a.D ? a.D[hv] : 0.f;

  // Columns of the wave's 16 PT: index 4 q + r of tile pt is column 4 PT q + 4 pt + r, so that the four
  // consecutive rows that a lane holds of each tile of y^T join to 4 PT consecutive columns.
  auto column = [](int pt, int q, int r) { return 4 * PT * q + 4 * pt + r; };
  // column index lr; rows 16 nt + 4 lq .. + 3, or, for bf16, in the order in which
  // two tiles make an operand of the next product: 32 (nt / 2) + 8 lq + 4 (nt % 2) .. + 3
  f32x4 S[PT][NT];
  // this wave's part of a [K, V] float32 state in memory; elements outside of it read zeros and
  // are not written
  auto each_state = [&](auto f) {
    if (!active) return;
    int n = (BF ? 8 : 4) * lq;
    asm volatile("" : "+v"(n));  // the offsets are made here, not kept over the tile loop
#pragma unroll
    for (int pt = 0; pt < PT; ++pt) {
      const int p = p0 + column(pt, lr >> 2, lr & 3);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          f(pt, nt, r, p < V ? (unsigned)(((BF ? nt / 2 * 32 + nt % 2 * 4 : 16 * nt) + n + r) * V + p) * 4u : kOutOfRange);
    }
  };
  const unsigned state_bytes = (unsigned)(K * V * 4);
  auto load_state = [&](const float* src) {
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(src, state_bytes);
    each_state([&](int pt, int nt, int r, unsigned off) {
      S[pt][nt][r] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0));
    });
  };
  auto store_state = [&](float* dst) {
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(dst, state_bytes);
    each_state([&](int pt, int nt, int r, unsigned off) {
      const float v = S[pt][nt][r];
      __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v), rs, off, 0, 0);
    });
  };
  auto zero_state = [&] {
#pragma unroll
    for (int pt = 0; pt < PT; ++pt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) S[pt][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  const int64_t sz = (int64_t)K * V;
  zero_state();
  if constexpr (OUT) {
    if (segk > 0 && a.seqs.span(w.seq).bos < w.seg0) {
      load_state(a.seg_state + ((int64_t)(segk - 1) * a.HV + hv) * sz);
    }
  }

  if constexpr (OUT && BF) {  // the blocks above the diagonal: (i, j) = (0, 1) and (2, 3)
    const int i = threadIdx.x / 16 % 16, j = threadIdx.x % 16;
    for (int h = 0; h < HB; ++h) {
      Ms[(h * kTok + i) * LDM + 16 + j] = from_f32<T>(0.f);
      Ms[(h * kTok + 32 + i) * LDM + 48 + j] = from_f32<T>(0.f);
    }
  }

  Tile cur = tile_at<kTok>(a, end, w.pos, w.seq);
  outside(w.pos, cur.t0);
  if (cur.rows == 0) return;
  load(cur);
  if (dw >= 0)
    make_decay<OUT, OUT && BF>(s_dec[0][dw], s_in[OUT ? dw : 0], to_f32(dtr), lane < cur.rows, bias, neg_rate);
  float gsum = 0.f, squares = 0.f;

  __builtin_amdgcn_s_waitcnt(0);  // the first tile's loads, so that the wait in the loop is that of later ones
  for (int buf = 0;; buf ^= 1) {
    xr.add_squares(squares);
    xr.store(Xs, LDX);
    br.store(Bs, LDB);
    if constexpr (OUT) cr.store(Cs, LDC);
    lds_barrier();
    const int done = cur.t0 + cur.rows;
    Tile nxt = {done, min(kTok, min(cur.eos, end) - done), cur.seq, cur.eos, false, false};
    if (nxt.rows > 0) {
      nxt.last = done + nxt.rows == cur.eos;
    } else {
      nxt = tile_at<kTok>(a, end, done, cur.seq);
      outside(done, nxt.t0);
    }
    if (cur.first) {  // the sequence's initial state
      zero_state();
      if (a.s0) {
        load_state(a.s0 + ((int64_t)cur.seq * a.HV + hv) * sz);
        // waited for here: a wait behind the branch would cover the loads of every next tile too
        __builtin_amdgcn_s_waitcnt(0);
      }
    }
    if constexpr (!OUT) load(nxt);

    const Decay* dec = s_dec[buf];
    // lane addresses are made anew in every tile: kept over the loop they would not fit the registers
    asm volatile("" : "+v"(lr), "+v"(lq));

    if constexpr (OUT) {
      // c . b transposed (rows j, columns i) in blocks of 16, then M of each head. The blocks at
      // and below the diagonal, dealt out evenly; those above are read as part of a product of 32
      // tokens only where they are zeros from the start.
      constexpr int kBlocks = BF ? 3 : 1;  // a wave's blocks: i and j, four bits each, lowest first
      int fresh = 0;
      asm volatile("" : "+v"(fresh));  // as above: made in every tile
      const int wv = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6) + fresh);
      unsigned its, jts;
      if constexpr (!BF) {
        its = wv == 0 ? 0x0 : wv < 3 ? 0x1 : 0xf;
        jts = wv == 2 ? 0x1 : 0x0;
      } else {
        its = wv == 0 ? 0x033 : wv == 1 ? 0x122 : wv == 2 ? 0xf33 : 0xf21;
        jts = wv == 0 ? 0x010 : wv == 1 ? 0x110 : wv == 2 ? 0xf32 : 0xf20;
      }
      // m of one block and head, rounded, to LDS
      auto put_m = [&](int h, int i, int j, const f32x4& m) {
        T* dst = Ms + (h * kTok + i) * LDM + j;
        if constexpr (BF) {
          typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
          *reinterpret_cast<u32x2*>(dst) = u32x2{pack2(m[0], m[1]), pack2(m[2], m[3])};
        } else {
          *reinterpret_cast<f32x4*>(dst) = m;
        }
      };
      bool wide = !BF;
      if constexpr (BF) {
#pragma unroll
        for (int h = 0; h < HB; ++h) wide |= __builtin_amdgcn_readfirstlane(s_in[h].wide) != 0;
      }
#pragma unroll
      for (int k = 0; k < kBlocks; ++k) {
        const int it = its >> 4 * k & 15, jt = jts >> 4 * k & 15;
        if (it == 15) continue;
        const int i = 16 * it + lr, j = 16 * jt + 4 * lq;
        f32x4 sc = {0.f, 0.f, 0.f, 0.f};
        if constexpr (BF) {
          bf16x8 bfr[KS], cfr[KS];
          f32x4 col[HB];
          float row[HB];
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            bfr[ks] = *reinterpret_cast<const bf16x8*>(Bs + (16 * jt + lr) * LDB + 32 * ks + 8 * lq);
            cfr[ks] = *reinterpret_cast<const bf16x8*>(Cs + i * LDC + 32 * ks + 8 * lq);
          }
#pragma unroll
          for (int h = 0; h < HB; ++h) {
            col[h] = *reinterpret_cast<const f32x4*>(&s_in[h].col[8 * it * (it + 1) + j]);
            row[h] = s_in[h].row[i];
          }
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) sc = mfma(bfr[ks], cfr[ks], sc);
          if (!wide || jt < it) {
#pragma unroll
            for (int h = 0; h < HB; ++h) {
              // the factors first: their product is at most D_j, a score times one of them may overflow
              f32x4 m = sc * (col[h] * row[h]);
#pragma unroll
              for (int r = 0; r < 4; ++r) m[r] = j + r <= i ? m[r] : 0.f;
              put_m(h, i, j, m);
            }
            continue;
          }
        } else {
#pragma unroll 4
          for (int n = lq; n < NP; n += 4) sc = mfma(Bs[(16 * jt + lr) * LDB + n], Cs[i * LDC + n], sc);
        }
        // every pair's decay as one exponential
#pragma unroll
        for (int h = 0; h < HB; ++h) {
          f32x4 m;
          const f32x4 hj = *reinterpret_cast<const f32x4*>(s_in[h].hi + j), lj = *reinterpret_cast<const f32x4*>(s_in[h].lo + j);
          const f32x4 dj = *reinterpret_cast<const f32x4*>(s_in[h].dt + j);
          const float hi = s_in[h].hi[i], lo = s_in[h].lo[i];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            // j > i gives a positive exponent, possibly inf: not taken
            const float v = sc[r] * dj[r] * fast_exp2((hi - hj[r]) + (lo - lj[r]));
            m[r] = j + r <= i ? v : 0.f;
          }
          put_m(h, i, j, m);
        }
      }
      lds_barrier();
    }

    if (active) {
      // y of 16 tokens and this wave's columns (rows p), from accumulators that hold it transposed
      const unsigned yrow = (unsigned)ldy * (unsigned)sizeof(T);
      // the buffer ends with the tile's last row; columns behind V lie out of its range
      const __amdgpu_buffer_rsrc_t yb = make_rsrc(y + (int64_t)cur.t0 * ldy + (int64_t)hv * V,
                                                  (unsigned)(cur.rows - 1) * yrow + (unsigned)V * (unsigned)sizeof(T));
      const int py = p0 + column(0, lq, 0);  // the first of this lane's columns of y
      const unsigned yoff = (unsigned)lr * yrow + (py < V ? (unsigned)py * (unsigned)sizeof(T) : kOutOfRange);
      auto store_y = [&](int it, const f32x4 (&acc)[PT]) {
        const unsigned at = yoff + (unsigned)(16 * it) * yrow;
        if constexpr (VEC && BF && PT == 2) {
          const u32x4 o = {pack2(acc[0][0], acc[0][1]), pack2(acc[0][2], acc[0][3]),
                           pack2(acc[PT - 1][0], acc[PT - 1][1]), pack2(acc[PT - 1][2], acc[PT - 1][3])};
          __builtin_amdgcn_raw_buffer_store_b128(o, yb, at, 0, 0);
        } else if constexpr (VEC && BF) {
          typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
          const u32x2 o = {pack2(acc[0][0], acc[0][1]), pack2(acc[0][2], acc[0][3])};
          __builtin_amdgcn_raw_buffer_store_b64(o, yb, at, 0, 0);
        } else if constexpr (VEC) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[0]), yb, at, 0, 0);
        } else {
#pragma unroll
          for (int pt = 0; pt < PT; ++pt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const unsigned off = py + 4 * pt + r < V ? at + (4 * pt + r) * (unsigned)sizeof(T) : kOutOfRange;
              const T o = from_f32<T>(acc[pt][r]);
              if constexpr (BF) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, o), yb, off, 0, 0);
              else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, o), yb, off, 0, 0);
            }
        }
      };
      // 2^(G_i) (S^T c_i) + D x_i, ahead of the products inside the tile
      auto decay_y = [&](int i, f32x4 (&acc)[PT]) {
        const float eg = dec[hh].eg[i];
#pragma unroll
        for (int pt = 0; pt < PT; ++pt)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[pt][r] = acc[pt][r] * eg + skip * to_f32(Xs[i * LDX + col0 + column(pt, lq, r)]);
      };
      const float ga = decay_of(dec[hh].end);
      if constexpr (BF) {
        // x of this wave's columns, transposed: rows p, 8 tokens a lane
        bf16x8 xf[PT][2];
#pragma unroll
        for (int pt = 0; pt < PT; ++pt)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            const bf16* src = Xs + (32 * ks + 8 * lq + (lr >> 2)) * LDX + col0 + column(pt, lr & 3, 0);
            xf[pt][ks] = join(load_tr4(src), load_tr4(src + 4 * LDX));
          }
        if constexpr (OUT) {
          bf16x8 sf[PT][KS];  // S^T as an operand
#pragma unroll
          for (int pt = 0; pt < PT; ++pt)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              const f32x4 a0 = S[pt][2 * ks], a1 = S[pt][2 * ks + 1];
              sf[pt][ks] = __builtin_bit_cast(bf16x8, u32x4{pack2(a0[0], a0[1]), pack2(a0[2], a0[3]),
                                                            pack2(a1[0], a1[1]), pack2(a1[2], a1[3])});
            }
#pragma unroll
          for (int it = 0; it < kTok / 16; ++it) {
            const int i = 16 * it + lr;
            f32x4 acc[PT];
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) acc[pt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              const bf16x8 cv = *reinterpret_cast<const bf16x8*>(Cs + i * LDC + 32 * ks + 8 * lq);
#pragma unroll
              for (int pt = 0; pt < PT; ++pt) acc[pt] = mfma(sf[pt][ks], cv, acc[pt]);
            }
            decay_y(i, acc);
#pragma unroll
            for (int ks = 0; ks <= it / 2; ++ks) {
              const bf16x8 mv = *reinterpret_cast<const bf16x8*>(Ms + (hh * kTok + i) * LDM + 32 * ks + 8 * lq);
#pragma unroll
              for (int pt = 0; pt < PT; ++pt) acc[pt] = mfma(xf[pt][ks], mv, acc[pt]);
            }
            store_y(it, acc);
          }
        }
        // the next tile's loads go out here: their registers are free only now (loads of single elements
        // take twice as many: behind the state's products, 8192 tokens, 16 heads x 60, K 100: 192 -> 124 us)
        if constexpr (OUT) {
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (VEC) load(nxt);
          __builtin_amdgcn_sched_barrier(0);  // not behind the products of the state
        }
        // the state's update
#pragma unroll
        for (int pt = 0; pt < PT; ++pt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) S[pt][nt] *= ga;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          u32x4 w0[PT], w1[PT], w2[PT];
          const f32x4 wa = *reinterpret_cast<const f32x4*>(dec[hh].w + 32 * ks + 8 * lq);
          const f32x4 wb = *reinterpret_cast<const f32x4*>(dec[hh].w + 32 * ks + 8 * lq + 4);
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) {
            const u32x4 xu = __builtin_bit_cast(u32x4, xf[pt][ks]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float a0 = low(xu[e]) * (e < 2 ? wa[2 * e] : wb[2 * e - 4]);
              float a1 = high(xu[e]) * (e < 2 ? wa[2 * e + 1] : wb[2 * e - 3]);
              const unsigned u0 = pack2(a0, a1);
              a0 = a0 - low(u0), a1 = a1 - high(u0);
              const unsigned u1 = pack2(a0, a1);
              w0[pt][e] = u0;
              w1[pt][e] = u1;
              w2[pt][e] = pack2(a0 - low(u1), a1 - high(u1));
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const bf16* src = Bs + (32 * ks + 8 * lq + (lr >> 2)) * LDB + nt / 2 * 32 + nt % 2 * 4 + 8 * (lr & 3);
            const bf16x8 bt = join(load_tr4(src), load_tr4(src + 4 * LDB));
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) {
              S[pt][nt] = mfma(bt, __builtin_bit_cast(bf16x8, w0[pt]), S[pt][nt]);
              S[pt][nt] = mfma(bt, __builtin_bit_cast(bf16x8, w1[pt]), S[pt][nt]);
              S[pt][nt] = mfma(bt, __builtin_bit_cast(bf16x8, w2[pt]), S[pt][nt]);
            }
          }
        }
      } else {
        // float32: 16x16x4 products, one operand value a lane; slot lq of step r of a state tile
        // holds its row 4 lq + r
        if constexpr (OUT) {
#pragma unroll
          for (int it = 0; it < kTok / 16; ++it) {
            const int i = 16 * it + lr;
            f32x4 acc[PT];
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) acc[pt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const f32x4 cv = *reinterpret_cast<const f32x4*>(Cs + i * LDC + 16 * nt + 4 * lq);
#pragma unroll
              for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int pt = 0; pt < PT; ++pt) acc[pt] = mfma(S[pt][nt][r], cv[r], acc[pt]);
            }
            decay_y(i, acc);
#pragma unroll
            for (int j = 0; j < 16 * (it + 1); j += 4)
#pragma unroll
              for (int pt = 0; pt < PT; ++pt)
                acc[pt] = mfma(Xs[(j + lq) * LDX + col0 + 16 * pt + lr], Ms[i * LDM + j + lq], acc[pt]);
            store_y(it, acc);
          }
          load(nxt);
        }
#pragma unroll
        for (int pt = 0; pt < PT; ++pt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) S[pt][nt] *= ga;
#pragma unroll 2
        for (int j = lq; j < kTok; j += 4) {
          const float w = dec[hh].w[j];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float bt = Bs[j * LDB + 16 * nt + lr];
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) S[pt][nt] = mfma(bt, w * Xs[j * LDX + col0 + 16 * pt + lr], S[pt][nt]);
          }
        }
      }
      if (OUT && cur.last && a.sT) store_state(a.sT + ((int64_t)cur.seq * a.HV + hv) * sz);
      if constexpr (OUT && BF && !VEC) load(nxt);
      gsum += dec[hh].end;
    } else if constexpr (OUT) {
      load(nxt);
    }
    if (nxt.rows == 0) break;
    if (dw >= 0)
      make_decay<OUT, OUT && BF>(s_dec[buf ^ 1][dw], s_in[OUT ? dw : 0], to_f32(dtr), lane < nxt.rows, bias, neg_rate);
    lds_barrier();
    cur = nxt;
  }
  if constexpr (!OUT) {
    store_state(a.seg_state + ((int64_t)segk * a.HV + hv) * sz);
    // a sequence that starts in the segment takes nothing from the segment before
    if (active && p0 == 0 && lane == 0) a.seg_g[(int64_t)segk * a.HV + hv] = w.carry ? gsum : -INFINITY;
  }
  // a sum of squares that is not finite: some x may be odd (which by_token() finds out)
  if (lane == 0) s_odd[wv] = 0;
  if (!(squares < INFINITY)) s_odd[wv] = 1;  // any writer stores the same
  block_barrier();
  if (__builtin_amdgcn_readfirstlane(s_odd[0] | s_odd[1] | s_odd[2] | s_odd[3]) != 0) {
    __builtin_amdgcn_s_waitcnt(0);  // what by_token() writes over is written
    by_token<T, NP, PP, HB, OUT, LDX, LDB, LDC>((arg_words)__builtin_amdgcn_kernarg_segment_ptr(), hblocks, blockIdx.x,
                                                threadIdx.x, (lds<T>*)Xs, (lds<T>*)Bs, (lds<T>*)Cs,
                                                (lds<Decay>*)s_dec[0], (lds<int>*)s_odd);
  }
}

constexpr int kAhead = 8;  // boundaries whose loads are issued before any is used

// Composes the segments' states in order, in place: seg_state[k] becomes the state that enters
// segment k + 1. One thread an element of [HV, K, V].
__global__ __launch_bounds__(kThreads) void compose_kernel(float* __restrict__ seg_state,
                                                           const float* __restrict__ seg_g, int nb, int per,
                                                           int HV, int64_t sz) {
  const int64_t n = (int64_t)HV * sz, i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  const int hv = (int)(i / sz);
  float s = 0.f;
  for (int k0 = 0; k0 < nb; k0 += kAhead) {
    float g[kAhead], v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {  // loads behind the last boundary read it again
      const int k = min(k0 + u, nb - 1);
      g[u] = seg_g[(int64_t)k * HV + hv];
      v[u] = seg_state[(int64_t)k * n + i];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (k0 + u >= nb) break;
      // nothing was made of a sequence's last segment; where nothing is carried the product is left
      // out: s may be infinite
      const bool none = g[u] == kNoCarry || (per > 0 && (k0 + u + 1) % per == 0);
      s = none ? 0.f : g[u] > -INFINITY ? v[u] + decay_of(g[u]) * s : v[u];
      if (!none) seg_state[(int64_t)(k0 + u) * n + i] = s;
    }
  }
}

// ---- launchers

template <typename T, int NT, int PP, int HB, int PT, bool VEC>
hipError_t run(const SsmArgs& a, hipStream_t stream) {
  const int hblocks = a.HV / HB * ((a.V + PP - 1) / PP);
  if (((int64_t)hblocks * a.nseg + a.N) * kThreads > UINT32_MAX) return hipErrorNotSupported;
  if (a.crossed) {
    hipLaunchKernelGGL((prefill_kernel<T, NT, PP, HB, PT, false, VEC>), dim3(hblocks * (a.per > 0 ? a.N * (a.per - 1) : a.nseg - 1)),
                       dim3(kThreads), 0, stream, a, hblocks);
    const int64_t n = (int64_t)a.HV * a.K * a.V;
    hipLaunchKernelGGL(compose_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream,
                       a.seg_state, a.seg_g, a.nseg - 1, a.per, a.HV, (int64_t)a.K * a.V);
  }
  const int empties = (a.seqs.cu || a.T == 0) && a.sT ? a.N : 0;
  if (hblocks * a.nseg + empties == 0) return hipSuccess;
  hipLaunchKernelGGL((prefill_kernel<T, NT, PP, HB, PT, true, VEC>), dim3(hblocks * a.nseg + empties),
                     dim3(kThreads), 0, stream, a, hblocks);
  return hipGetLastError();
}

// Heads and columns of a workgroup.
struct Shape {
  int heads, cols;
};
inline Shape shape_of(bool bf, int H, int HV, int V) {
  if (!bf) return {1, 64};
  const int pair = (HV / H) % 2 == 0 ? 2 : 1;  // two heads that share b and c, where V leaves room
  return V > 64 ? Shape{1, 128} : V > 32 ? Shape{pair, 64} : Shape{pair, 32};
}

template <typename T, int NT, bool VEC>
hipError_t by_heads(const SsmArgs& a, hipStream_t stream) {
  if constexpr (sizeof(T) == 4) return run<T, NT, 64, 1, 1, VEC>(a, stream);
  else {
    const Shape s = shape_of(true, a.H, a.HV, a.V);
    if (s.cols == 128) return run<T, NT, 128, 1, 2, VEC>(a, stream);
    if (s.cols == 64) return s.heads == 2 ? run<T, NT, 64, 2, 2, VEC>(a, stream) : run<T, NT, 64, 1, 1, VEC>(a, stream);
    return s.heads == 2 ? run<T, NT, 32, 2, 1, VEC>(a, stream) : run<T, NT, 32, 1, 1, VEC>(a, stream);
  }
}

template <typename T>
hipError_t by_state(const SsmArgs& a, hipStream_t stream) {
  if (a.K > 64) return a.vec ? by_heads<T, 8, true>(a, stream) : by_heads<T, 8, false>(a, stream);
  return a.vec ? by_heads<T, 4, true>(a, stream) : by_heads<T, 4, false>(a, stream);
}

}  // namespace ssm

// Segments of the token axis for these arguments.
struct Segments {
  int len, n;
  bool crossed;  // a sequence may go on over a boundary
};
static Segments ssm_segments(int T, int N, bool packed, int H, int HV, int V, bool bf) {
  if (T == 0) return {1, 0, false};
  const ssm::Shape s = ssm::shape_of(bf, H, HV, V);
  const int64_t hblocks = (int64_t)HV / s.heads * ((V + s.cols - 1) / s.cols);
  const int64_t want = (512 + hblocks - 1) / hblocks;  // two workgroups a CU
  int64_t len = (((int64_t)T + want - 1) / want + 63) / 64 * 64;
  if (len < 256) len = 256;
  if (!packed && len >= T / N) len = T / N;  // whole sequences
  const int n = (int)((T + len - 1) / len);
  return {(int)len, n, n > 1 && (packed || len % (T / N) != 0)};
}

size_t ssm_prefill_workspace_bytes(int T, int N, bool packed, int H, int HV, int K, int V, bool bf) {
  const Segments g = ssm_segments(T, N, packed, H, HV, V, bf);
  if (!g.crossed) return 0;
  const size_t n = (size_t)(g.n - 1) * HV * ((size_t)K * V + 1) * 4;
  return (n + 255) / 256 * 256;
}

hipError_t launch_ssm_prefill(SsmArgs a, void* workspace, hipStream_t stream) {
  const Segments g = ssm_segments(a.T, a.N, a.seqs.cu != nullptr, a.H, a.HV, a.V, a.bf);
  a.seg = g.len;
  a.nseg = g.n;
  a.crossed = g.crossed;
  a.per = g.crossed && !a.seqs.cu && a.seqs.len % g.len == 0 ? a.seqs.len / g.len : 0;
  if (g.crossed) {
    a.seg_state = static_cast<float*>(workspace);
    a.seg_g = a.seg_state + (size_t)(g.n - 1) * a.HV * a.K * a.V;
  }
  // 16-byte pieces: whole ones in every row, at aligned addresses (y rows are whole ones too then)
  const int per = a.bf ? 8 : 4;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.b) |
                         reinterpret_cast<uintptr_t>(a.c) | reinterpret_cast<uintptr_t>(a.y);
  a.vec = (a.K | a.V | a.ldx | a.ldb | a.ldc) % per == 0 && bits % 16 == 0;
  return a.bf ? ssm::by_state<bf16>(a, stream) : ssm::by_state<float>(a, stream);
}

}  // namespace kda
