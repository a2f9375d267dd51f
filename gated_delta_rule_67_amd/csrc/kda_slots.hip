// Copies, forks, clears and compaction of slots in state pools: the caches whose slots
// kda_recurrent_step_slots, kda_conv_step and kda_ssm_step read and update (the
// DM-KDAGQA-1.7B-SD model card's usage notes: generation keeps recurrent and conv states). A pool
// is [num_slots] slots of slot_bytes bytes; one call moves the same slots of many pools (a
// model's layers), in one launch per kMaxPools of them.
//
// The work is one read and one write of what moves, so HBM bounds it: 24 slots of 1 MB in each of
// 18 pools take 150 to 156 us (5.8 to 6.0 TB/s). Its items (pool, pair, piece of a slot) are dealt out to at most
// kBlocks workgroups of 256 lanes, each lane with up to eight 16-byte loads in flight before its
// stores; pieces are 32 KB, or smaller where there would be too few items for the GPU.
//
// The pairs of one call apply in order. Where no destination is named twice or is another pair's
// source, the order does not matter and all items run side by side. Every workgroup finds that
// out for itself, once, with a bitmap of the destinations in LDS; where it does matter, each
// piece of a slot is taken through all pairs, in order, by the same lanes of one workgroup.
#include <type_traits>

#include "kda_device.h"

namespace kda {
namespace slots {

constexpr int kThreads = 256;
constexpr int kBlocks = 2048;       // eight workgroups a CU
constexpr int kPiece = 32 << 10;    // bytes of an item at most: eight 16-byte accesses a lane
constexpr int kSmallPiece = 4 << 10;
constexpr int kMaxPools = 64;       // pools of a launch (their table is a kernel argument)

struct Pools {
  char* base[kMaxPools];
  int64_t bytes[kMaxPools];  // of a slot
};

// One lane's part of a piece: copies (or clears, from == null) [0, len) in units of U.
template <typename U>
__device__ __forceinline__ void move_piece(char* to, const char* from, int len) {
  constexpr int kStep = kThreads * (int)sizeof(U);
  int i = threadIdx.x * (int)sizeof(U);
  auto batch = [&](auto count) {
    constexpr int kCount = decltype(count)::value;
    for (; i + (kCount - 1) * kStep < len; i += kCount * kStep) {
      U v[kCount];
#pragma unroll
      for (int u = 0; u < kCount; ++u)
        v[u] = from ? __builtin_nontemporal_load(reinterpret_cast<const U*>(from + i + u * kStep)) : U{};
#pragma unroll
      for (int u = 0; u < kCount; ++u) __builtin_nontemporal_store(v[u], reinterpret_cast<U*>(to + i + u * kStep));
    }
  };
  batch(std::integral_constant<int, 8>{});
  batch(std::integral_constant<int, 4>{});
  batch(std::integral_constant<int, 1>{});
}

__device__ __forceinline__ void move_item(char* base, int64_t bytes, int size, int piece, int from, int to) {
  const int64_t off = (int64_t)piece * size;
  const int len = (int)(bytes - off < size ? bytes - off : size);
  char* d = base + (int64_t)to * bytes + off;
  const char* s = from < 0 ? nullptr : base + (int64_t)from * bytes + off;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(base) | (uintptr_t)bytes;
  if (bits % 16 == 0) move_piece<f32x4>(d, s, len);
  else if (bits % 4 == 0) move_piece<uint32_t>(d, s, len);
  else if (bits % 2 == 0) move_piece<uint16_t>(d, s, len);
  else move_piece<uint8_t>(d, s, len);
}

// moves: device count of pairs that are known to be independent (compaction), or null: n pairs.
__global__ __launch_bounds__(kThreads) void copy_kernel(Pools pools, int npools, int pieces, int size,
                                                        const int* __restrict__ src,
                                                        const int* __restrict__ dst, int n,
                                                        const int* __restrict__ moves, int nslots) {
  extern __shared__ unsigned s_dst[];  // a bit per slot: a destination (pairs given by the caller)
  __shared__ int s_order;
  // pair i moves something: a valid destination, and a source in the pool or a clear
  auto valid = [&](int i) { return dst[i] >= 0 && dst[i] < nslots && src[i] < nslots && src[i] != dst[i]; };
  bool order = false;
  if (moves) {
    n = min(*moves, n);
  } else if (n > 1) {
    const int words = (nslots + 31) / 32;
    for (int i = threadIdx.x; i < words; i += kThreads) s_dst[i] = 0;
    if (threadIdx.x == 0) s_order = 0;
    block_barrier();
    for (int i = threadIdx.x; i < n; i += kThreads)
      if (valid(i)) {
        const unsigned bit = 1u << (dst[i] & 31);
        if (atomicOr(&s_dst[dst[i] >> 5], bit) & bit) s_order = 1;  // any writer stores the same
      }
    block_barrier();
    for (int i = threadIdx.x; i < n; i += kThreads)
      if (valid(i) && src[i] >= 0 && (s_dst[src[i] >> 5] >> (src[i] & 31) & 1)) s_order = 1;
    block_barrier();
    order = s_order != 0;
  }
  const int64_t items = (int64_t)npools * pieces * (order ? 1 : n);
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int piece = (int)(it % pieces);
    const int64_t rest = it / pieces;
    const int pool = (int)(rest % npools);
    const int64_t bytes = pools.bytes[pool];
    if ((int64_t)piece * size >= bytes) continue;
    if (!order) {
      const int i = (int)(rest / npools);
      if (valid(i)) move_item(pools.base[pool], bytes, size, piece, src[i], dst[i]);
    } else {
      for (int i = 0; i < n; ++i)
        if (valid(i)) {
          move_item(pools.base[pool], bytes, size, piece, src[i], dst[i]);
          // a lane reads back only what it wrote itself; the fence keeps its accesses in order
          __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
        }
    }
  }
}

constexpr int kPlanThreads = 1024;

// The moves of a compaction, by one workgroup: with c live slots, the live slots at or behind
// slot c, in order, go to the free slots in front of it, in order (as many of the one as of the
// other). list: {count, src[nslots], dst[nslots]}; new_slot[s]: where s lives now, -1 for a free
// slot; *count = c.
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(const uint8_t* __restrict__ live,
                                                            int nslots, int* __restrict__ new_slot,
                                                            int* __restrict__ count, int* list) {
  constexpr int kWaves = kPlanThreads / 64;
  __shared__ int s_part[2][kWaves];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int c = 0;
  for (int i = t; i < nslots; i += kPlanThreads) c += live[i] != 0;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) c += __shfl_xor(c, off);
  if (lane == 0) s_part[0][wave] = c;
  block_barrier();
  c = 0;
  for (int w = 0; w < kWaves; ++w) c += s_part[0][w];
  block_barrier();
  int* src = list + 1;
  int* dst = list + 1 + nslots;
  int holes = 0, movers = 0;  // found so far
  for (int base = 0; base < nslots; base += kPlanThreads) {
    const int i = base + t;
    const bool l = i < nslots && live[i] != 0;
    const bool hole = i < nslots && !l && i < c, mover = l && i >= c;
    const uint64_t hm = __builtin_amdgcn_ballot_w64(hole), mm = __builtin_amdgcn_ballot_w64(mover);
    if (lane == 0) {
      s_part[0][wave] = __builtin_popcountll(hm);
      s_part[1][wave] = __builtin_popcountll(mm);
    }
    block_barrier();
    int h0 = holes, m0 = movers;
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) h0 += s_part[0][w], m0 += s_part[1][w];
      holes += s_part[0][w];
      movers += s_part[1][w];
    }
    const uint64_t below = (1ull << lane) - 1;
    if (hole) dst[h0 + __builtin_popcountll(hm & below)] = i;
    if (mover) src[m0 + __builtin_popcountll(mm & below)] = i;
    if (i < nslots && !mover) new_slot[i] = l ? i : -1;
    block_barrier();
  }
  for (int i = t; i < movers; i += kPlanThreads) new_slot[src[i]] = dst[i];
  if (t == 0) {
    list[0] = movers;
    *count = c;
  }
}

hipError_t launch_copy(void* const* base, const size_t* bytes, int npools, int nslots, const int* src,
                       const int* dst, int n, const int* moves, hipStream_t stream) {
  for (int p0 = 0; p0 < npools; p0 += kMaxPools) {
    Pools pools{};
    const int np = npools - p0 < kMaxPools ? npools - p0 : kMaxPools;
    int64_t most = 0, total = 0;
    for (int i = 0; i < np; ++i) {
      pools.base[i] = static_cast<char*>(base[p0 + i]);
      pools.bytes[i] = (int64_t)bytes[p0 + i];
      most = most > pools.bytes[i] ? most : pools.bytes[i];
      total += pools.bytes[i];
    }
    // an item for every workgroup, if pieces of 4 KB or more can do that
    const int64_t each = total / kBlocks > kPiece / n ? kPiece : total * n / kBlocks;
    const int size = each >= kPiece ? kPiece : each <= kSmallPiece ? kSmallPiece : (int)(each / kSmallPiece * kSmallPiece);
    const int64_t pieces = (most + size - 1) / size;
    const int64_t items = pieces * np * n;
    const int lds = moves || n < 2 ? 0 : (nslots + 31) / 32 * 4;
    hipLaunchKernelGGL(copy_kernel, dim3((unsigned)(items < kBlocks ? items : kBlocks)), dim3(kThreads), lds,
                       stream, pools, np, (int)pieces, size, src, dst, n, moves, nslots);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace slots

hipError_t launch_slots_copy(void* const* pools, const size_t* slot_bytes, int npools, int nslots,
                             const int* src, const int* dst, int n, hipStream_t stream) {
  return slots::launch_copy(pools, slot_bytes, npools, nslots, src, dst, n, nullptr, stream);
}

size_t slots_compact_workspace_bytes(int nslots) {
  return ((2 * (size_t)nslots + 1) * 4 + 255) / 256 * 256;
}

hipError_t launch_slots_compact(void* const* pools, const size_t* slot_bytes, int npools, int nslots,
                                const uint8_t* live, int* new_slot, int* count, void* workspace,
                                hipStream_t stream) {
  int* list = static_cast<int*>(workspace);
  hipLaunchKernelGGL(slots::plan_kernel, dim3(1), dim3(slots::kPlanThreads), 0, stream, live, nslots,
                     new_slot, count, list);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || npools == 0) return e;
  // at most half of the slots move
  const int most = nslots / 2 > 0 ? nslots / 2 : 1;
  return slots::launch_copy(pools, slot_bytes, npools, nslots, list + 1, list + 1 + nslots, most, list, stream);
}

}  // namespace kda
