// Block mass: what the attention kernels and block_mass.cu share.
#pragma once

#include "common.cuh"

namespace sparda {

// The blocks in the slots of a (sequence, group), slots lane and lane + 32 in each lane of a warp: its list
// of n blocks, or (idx == nullptr) slot s is block s.
static_assert(kMaxTopk + 2 <= 64, "a list in two registers per lane");
struct SlotBlocks {
  bool listed;
  int lo, hi;
};
__device__ __forceinline__ SlotBlocks slot_blocks(const int32_t* idx, int n) {
  const int lane = threadIdx.x & 31;
  return {idx != nullptr, idx && lane < n ? idx[lane] : -1, idx && lane + 32 < n ? idx[lane + 32] : -1};
}

// Adds the weight of the attended block in slot s to the group's mass, by one warp: l exp2(m - M) / L over
// the block's parts and heads (M, L: the final maximum and sum of head lane % 16; st: the group's
// statistics), if it is one of blocks 0 .. last. Of the slots that name the same block the first adds
// all their weights, in order, and the others nothing: no sum depends on which warp comes first.
__device__ __forceinline__ void add_block_mass(const float2* st, int parts, int H, float M, float L, const SlotBlocks& list,
                                               int s, int last, float* mass) {
  const int lane = threadIdx.x & 31;
  const int j = list.listed ? __shfl_sync(0xffffffffu, s < 32 ? list.lo : list.hi, s & 31) : s;
  if (j < 0 || j > last) return;                   // reported by the attention
  const auto weight = [&](int slot) {
    const float2* p = st + (size_t)slot * parts * kHeads + lane;
    const float2 x = p[0], y = parts == 4 ? p[32] : make_float2(0.f, 0.f);
    float w = 0.f;                                 // a part without tokens has l = 0
    if (x.y != 0.f) w += x.y * exp2f(x.x - M);
    if (y.y != 0.f) w += y.y * exp2f(y.x - M);
    w = (lane & 15) < H && L != 0.f ? w / L : 0.f;
#pragma unroll
    for (int d = 16; d; d >>= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
    return w;
  };
  unsigned long long same = 0;                     // later slots of the same block
  if (list.listed) {
    same = __ballot_sync(0xffffffffu, list.lo == j) | (unsigned long long)__ballot_sync(0xffffffffu, list.hi == j) << 32;
    if (same & ((1ull << s) - 1ull)) return;
    same &= same - 1;
  }
  float sum = weight(s);
  for (; same; same &= same - 1) sum += weight(__ffsll((long long)same) - 1);
  if (lane == 0) atomicAdd(mass + j, sum);         // the only one to this block; nothing waits for the old value
}

}  // namespace sparda
