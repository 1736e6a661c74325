// What the forms of the decode attention over the 4-bit cache share: the plan that cuts the blocks of
// all (sequence, group)s into one contiguous range per CTA, and the numbers of the softmax.
#pragma once

#include "kernels.h"
#include "kv4.cuh"

namespace sparda {
namespace kv4 {

constexpr int kPlanMax = 1024;                              // (sequence, group)s the balanced plan holds
constexpr int kMinUnits = 2;                                // blocks per CTA below which fewer CTAs work
constexpr float kPShift = 6.f;                              // weights are scaled by 2^kPShift
constexpr float kRise = 8.f;                                // rise of a maximum (base 2) that is let pass
constexpr uint32_t kProducerPolls = 1u << 25;               // bounds a lane's wait to seconds
constexpr float kNegInf = -INFINITY;
// The reference before any token: finite, so that no difference of references is a NaN.
constexpr float kLowest = -3.0e38f;
constexpr float kScale2 = 1.4426950408889634f * 0.08838834764831845f;   // log2(e) / sqrt(128)

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// Blocks of (sequence, group) bg.
__device__ __forceinline__ int group_blocks(const Kv4AttnArgs& a, int bg, int T) {
  if (T < 1 || T > a.max_ctx) return 0;
  const int tb = (T - 1) / kBlock;
  return a.idx ? min(max(a.cnt[bg], 0), a.kslots) : tb + 1;
}

// Shared-memory loads by 32-bit address: through pointers into the aligned ring the compiler
// would make them generic loads.
__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t p) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(p) : "memory");
  return v;
}

// The pieces of the unit range that a CTA owns, one (sequence, group) at a time.
struct Piece {
  int bg, s0, s1;       // slots s0 .. s1-1 of group bg
  int first, n_cta;     // the group's first CTA and how many share it
};

// The balanced plan. U blocks in all, cut into one range [u0, u1) for each of the first `ctas` CTAs.
struct Plan {
  const int* pre;       // prefix sums of the groups' blocks, in shared memory
  int bg_count, U, ctas, u0, u1;

  // CTA whose range holds a block.
  __device__ __forceinline__ int cta_of(long long unit) const { return (int)(((unit + 1) * ctas - 1) / U); }
  __device__ __forceinline__ int start_of(int cta) const { return (int)((long long)U * cta / ctas); }
  // The group with pre[bg] <= unit < pre[bg + 1].
  __device__ __forceinline__ int group_of(int unit) const {
    int lo = 0, hi = bg_count - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid + 1] > unit) hi = mid;
      else lo = mid + 1;
    }
    return lo;
  }
  // The piece of [u, u1) that lies in one group, from group bg on; moves both behind it.
  __device__ __forceinline__ bool next(Piece& p, int& u, int& bg) const {
    if (u >= u1) return false;
    while (pre[bg + 1] <= u) ++bg;
    const int g0 = pre[bg], g1 = pre[bg + 1];
    p.bg = bg;
    p.s0 = u - g0;
    p.s1 = min(u1, g1) - g0;
    p.first = cta_of(g0);
    p.n_cta = cta_of(g1 - 1) - p.first + 1;
    u = min(u1, g1);
    return true;
  }
  // Where a CTA leaves its partial result of a piece (two places per CTA): its first piece in the first,
  // its last in the second; a piece that is neither covers its group alone.
  __device__ __forceinline__ int own_place(int cta, bool first_piece) const { return cta * 2 + (first_piece ? 0 : 1); }
  // The place of part q of a piece's group: the group's first CTA used its second unless the group
  // begins that CTA's range, the others their first.
  __device__ __forceinline__ int place_of(const Piece& p, int q) const {
    return q == 0 ? p.first * 2 + (start_of(p.first) == pre[p.bg] ? 0 : 1) : (p.first + q) * 2;
  }
};

// Every thread of the CTA; s_pre holds bg_count + 1 numbers, bg_count <= kPlanMax.
__device__ __forceinline__ Plan make_plan(const Kv4AttnArgs& a, int* s_pre) {
  const int tid = threadIdx.x, lane = tid & 31;
  for (int bg = tid; bg < a.bg_count; bg += blockDim.x) {
    const int T = a.seq_len[bg / a.G];
    if ((T < 1 || T > a.max_ctx) && blockIdx.x == 0) atomicOr(a.err, SPARDA_DEV_BAD_SEQ_LEN);
    s_pre[bg + 1] = group_blocks(a, bg, T);
  }
  __syncthreads();
  if (tid < 32) {
    if (lane == 0) s_pre[0] = 0;
    int carry = 0;
    for (int base = 0; base < a.bg_count; base += 32) {
      int v = base + lane < a.bg_count ? s_pre[base + lane + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
      }
      v += carry;
      if (base + lane < a.bg_count) s_pre[base + lane + 1] = v;
      carry = __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  Plan p;
  p.pre = s_pre;
  p.bg_count = a.bg_count;
  p.U = s_pre[a.bg_count];
  p.ctas = min((int)gridDim.x, max(1, (p.U + kMinUnits - 1) / kMinUnits));
  const bool works = (int)blockIdx.x < p.ctas;
  p.u0 = works ? p.start_of(blockIdx.x) : p.U;
  p.u1 = works ? p.start_of(blockIdx.x + 1) : p.U;
  return p;
}

// Zeros for the groups without a block, which belong to no range: threads 0 .. n-1 of the first CTAs.
__device__ __forceinline__ void zero_empty_groups(const Kv4AttnArgs& a, const Plan& p, int thread, int n) {
  for (int bg = blockIdx.x; bg < a.bg_count; bg += p.ctas) {
    if (p.pre[bg + 1] != p.pre[bg]) continue;
    uint32_t* out = reinterpret_cast<uint32_t*>(a.out + (size_t)bg * a.H * kHeadDim);
    for (int i = thread; i < a.H * kHeadDim / 2; i += n) out[i] = 0u;
  }
}

}  // namespace kv4
}  // namespace sparda
