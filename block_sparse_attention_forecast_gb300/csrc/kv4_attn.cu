// Decode attention over the 4-bit cache: o = sum_t softmax_t(q . k_t / sqrt(d)) v_t for the H <= 16
// query heads of each (sequence, group), over the tokens of the selected blocks or of all blocks.
//
// What bounds it: a token is 160 bytes of cache for 4 * 16 * 128 multiply-adds and 256 codes to
// expand, so at the memory's rate one SM has about 7 cycles per token. The expansion (1.4
// instructions per code, kv4.cuh) and the tensor instructions (two m16n8k16 per token) both have
// to fit under that. The heads are the M dimension of warp-level MMAs: the cache is the B operand,
// expanded in registers straight into B fragments. A tcgen05 form would have to write the
// expanded 512 bytes per token to shared or tensor memory first, as much traffic again as the
// tensor cores then read.
//
// Work: the blocks of all (sequence, group)s in a row, U of them, are cut into one contiguous
// range per CTA, balanced to one block, whatever the lengths; every CTA finds its range itself
// from seq_len or cnt (a prefix sum over the groups), since the lengths live on the device. One
// producer thread brings whole blocks (10 KiB, one bulk copy each) into a shared-memory ring; the
// consumer warps form groups of four that take blocks in turn, a warp 16 tokens of each.
//
// Numbers: S in float32 from exact products (keys and queries are bf16); softmax in float32, base
// 2; weights are rounded to fp16 against the running maximum, scaled by 2^14 so that everything
// down to 2^-28 of the largest weight keeps fp16's 11 bits; sums in float32. The accumulator is
// rescaled only when a warp's running maximum moves.
#include <cuda_fp16.h>

#include "kernels.h"
#include "kv4.cuh"

namespace sparda {
using namespace kv4;

namespace {

constexpr int kWarpsPerBlock = 4;
constexpr int kBlockGroups = 2;                             // groups of four consumer warps
constexpr int kCWarps = kBlockGroups * kWarpsPerBlock;
constexpr int kCThreads = kCWarps * 32;
constexpr int kThreads4 = kCThreads + 32;
constexpr int kRing = 12;
static_assert(kRing % kBlockGroups == 0, "each ring stage must belong to one consumer group");
constexpr int kPlanMax = 1024;                              // (sequence, group)s the balanced plan holds
constexpr int kRow = 144;                                   // merge-buffer row: 128 + 4 per 32, no bank conflicts
constexpr int kMergeFloats4 = kCWarps * (kHeads * kRow + 2 * kHeads);
constexpr int kHeader4 = 1024 + (kPlanMax + 32) * 4;
constexpr int kSmem4 = 128 + kHeader4 + kRing * kBlockBytes4 + kMergeFloats4 * 4;
constexpr int kMinUnits = 2;                                // blocks per CTA below which fewer CTAs work
constexpr float kPShift = 14.f;                             // weights are scaled by 2^kPShift
constexpr float kNegInf = -INFINITY;

__device__ __forceinline__ void sync_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(kCThreads) : "memory"); }
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// Channel c of a merge-buffer row.
__device__ __forceinline__ int mcol(int c) { return c + 4 * (c >> 5); }

// Blocks of (sequence, group) bg.
__device__ __forceinline__ int group_blocks(const Kv4AttnArgs& a, int bg, int T) {
  if (T < 1 || T > a.max_ctx) return 0;
  const int tb = (T - 1) / kBlock;
  return a.idx ? min(max(a.cnt[bg], 0), a.kslots) : tb + 1;
}

__device__ __forceinline__ uint4 lds128(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

// The pieces of the unit range that a CTA owns, one (sequence, group) at a time.
struct Piece {
  int bg, s0, s1;       // slots s0 .. s1-1 of group bg
  int first, n_cta;     // the group's first CTA and how many share it
};

}  // namespace

// kStats: also store every quarter block's softmax statistics (max, sum of each head) and the
// final ones, for the block mass.
template <bool kStats>
__global__ void __launch_bounds__(kThreads4, 1) kv4_attn_kernel(const Kv4AttnArgs a) {
  extern __shared__ uint8_t smem_raw4[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw4) + 127) & ~static_cast<uintptr_t>(127));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + kRing;
  int* stage_live = reinterpret_cast<int*>(empty + kRing);   // tokens of the staged block that exist
  int* s_flag = stage_live + kRing;
  int* s_pre = reinterpret_cast<int*>(smem + 1024);
  uint8_t* ring = smem + kHeader4;
  float* mO = reinterpret_cast<float*>(ring + kRing * kBlockBytes4);
  float* mM = mO + kCWarps * kHeads * kRow;
  float* mL = mM + kCWarps * kHeads;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarpsPerBlock);
    }
    fence_mbar_init();
  }
  grid_dep_wait();
  grid_dep_launch();

  // ------------------------------------------------------------ the plan
  const bool balanced = a.bg_count <= kPlanMax;
  int U = 0, ctas = gridDim.x, u0 = 0, u1 = 0;
  if (balanced) {
    for (int bg = tid; bg < a.bg_count; bg += kThreads4) {
      const int T = a.seq_len[bg / a.G];
      if ((T < 1 || T > a.max_ctx) && blockIdx.x == 0) atomicOr(a.err, SPARDA_DEV_BAD_SEQ_LEN);
      s_pre[bg + 1] = group_blocks(a, bg, T);
    }
    __syncthreads();
    if (warp == 0) {
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
    U = s_pre[a.bg_count];
    ctas = min((int)gridDim.x, max(1, (U + kMinUnits - 1) / kMinUnits));
    if ((int)blockIdx.x >= ctas) return;
    u0 = (int)((long long)U * blockIdx.x / ctas);
    u1 = (int)((long long)U * (blockIdx.x + 1) / ctas);
  } else {
    __syncthreads();
  }
  const int c = blockIdx.x;
  const auto cta_of = [&](long long unit) { return (int)(((unit + 1) * ctas - 1) / U); };

  // Walks the CTA's pieces: balanced, the groups its unit range meets; else whole groups c, c + grid, ...
  int w_u = u0, w_bg = 0;
  if (balanced && u0 < u1) {
    int lo = 0, hi = a.bg_count - 1;                 // the group with pre[bg] <= u0 < pre[bg + 1]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_pre[mid + 1] > u0) hi = mid;
      else lo = mid + 1;
    }
    w_bg = lo;
  } else if (!balanced) {
    w_bg = c;
  }
  const auto next_piece = [&](Piece& p) -> bool {
    if (balanced) {
      if (w_u >= u1) return false;
      while (s_pre[w_bg + 1] <= w_u) ++w_bg;
      const int g0 = s_pre[w_bg], g1 = s_pre[w_bg + 1];
      p.bg = w_bg;
      p.s0 = w_u - g0;
      p.s1 = min(u1, g1) - g0;
      p.first = cta_of(g0);
      p.n_cta = cta_of(g1 - 1) - p.first + 1;
      w_u = min(u1, g1);
      return true;
    }
    if (w_bg >= a.bg_count) return false;
    p.bg = w_bg;
    p.s0 = 0;
    const int T = a.seq_len[w_bg / a.G];
    if ((T < 1 || T > a.max_ctx) && tid == 0) atomicOr(a.err, SPARDA_DEV_BAD_SEQ_LEN);
    p.s1 = group_blocks(a, w_bg, T);
    p.first = c;
    p.n_cta = 1;
    w_bg += gridDim.x;
    return true;
  };

  if (warp == kCWarps) {
    // ------------------------------------------------------------ producer
    int it = 0;
    Piece p;
    while (next_piece(p)) {
      const int T = a.seq_len[p.bg / a.G];
      const int tb = (T - 1) / kBlock;
      for (int base = p.s0; base < p.s1; base += 32) {
        const int s = base + lane;
        int j = s, live = 0;
        if (s < p.s1) {
          if (a.idx) j = a.idx[(size_t)p.bg * a.kslots + s];
          if (j < 0 || j > tb) {
            atomicOr(a.err, SPARDA_DEV_BAD_INDEX);   // skipped: block 0 is staged with no live token
            j = 0;
          } else {
            live = min(kBlock, T - j * kBlock);
          }
        }
        const int n = min(32, p.s1 - base);
        for (int i = 0; i < n; ++i, ++it) {
          const int jj = __shfl_sync(0xffffffffu, j, i), ll = __shfl_sync(0xffffffffu, live, i);
          const int stage = it % kRing;
          int ok = 1;
          if (lane == 0) {
            if (it >= kRing) ok = mbar_wait(&empty[stage], ((it / kRing) & 1) ^ 1, a.err);
            if (ok) {
              stage_live[stage] = ll;
              mbar_arrive_expect_tx(&full[stage], kBlockBytes4);
              bulk_load(ring + stage * kBlockBytes4, a.kv + ((size_t)p.bg * a.nb_cap + jj) * kBlockBytes4, kBlockBytes4,
                        &full[stage]);
            }
          }
          if (!__shfl_sync(0xffffffffu, ok, 0)) return;
        }
      }
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int grp = warp / kWarpsPerBlock, wq = warp % kWarpsPerBlock;
  const int g = lane >> 2, cq = lane & 3;
  const float sl2 = 1.4426950408889634f * 0.08838834764831845f;   // log2(e) / sqrt(128)
  int it = 0;
  bool ok = true;             // a wait that ran out: no further compute, the barriers stay matched
  bool first_piece = true;
  Piece p;
  while (next_piece(p)) {
    float m0 = kNegInf, m1 = kNegInf, l0 = 0.f, l1 = 0.f;
    float o[16][4];
#pragma unroll
    for (int n = 0; n < 16; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    uint4 qa[4], qb[4];       // rows g and g + 8, channels 32 cq + 8 w ..
    {
      const uint4* q0 = reinterpret_cast<const uint4*>(a.q + ((size_t)p.bg * a.H + g) * kHeadDim + 32 * cq);
      const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        qa[w] = g < a.H ? q0[w] : none;
        qb[w] = g + 8 < a.H ? q0[w + 8 * (kHeadDim / 8)] : none;
      }
    }
    for (int s = p.s0; s < p.s1; ++s, ++it) {
      if (it % kBlockGroups != grp) continue;
      const int stage = it % kRing;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&full[stage], (it / kRing) & 1, a.err));
      if (!ok) continue;
      const uint8_t* blk = ring + stage * kBlockBytes4;
      const int live = stage_live[stage] - 16 * wq;              // tokens of this warp's 16 that exist

      float sc[2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4 kw = lds128(blk + kKCodes + wq * 1024 + r * 512 + lane * 16);
        const uint32_t sz = *reinterpret_cast<const uint32_t*>(blk + kKScales + wq * 256 + r * 128 + lane * 4);
        const __nv_bfloat162 s2 = as_bf2(dup_lo(sz)), z2 = as_bf2(dup_hi(sz));
        float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t word = w == 0 ? kw.x : w == 1 ? kw.y : w == 2 ? kw.z : kw.w;
          mma_16816(x, qa[w].x, qb[w].x, qa[w].y, qb[w].y, key_pair(word, 0, s2, z2), key_pair(word, 1, s2, z2));
          mma_16816(y, qa[w].z, qb[w].z, qa[w].w, qb[w].w, key_pair(word, 2, s2, z2), key_pair(word, 3, s2, z2));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[r][e] = (x[e] + y[e]) * sl2;
      }
      if (live < 16) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (8 * r + 2 * cq + (e & 1) >= live) sc[r][e] = kNegInf;
      }
      float mx0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
      float mx1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
      if (__any_sync(0xffffffffu, mx0 > m0 || mx1 > m1)) {
        const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
        const float al0 = m0 == kNegInf ? 0.f : fast_exp2(m0 - n0), al1 = m1 == kNegInf ? 0.f : fast_exp2(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= al0;
        l1 *= al1;
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          o[n][0] *= al0;
          o[n][1] *= al0;
          o[n][2] *= al1;
          o[n][3] *= al1;
        }
      }
      const float base0 = (m0 == kNegInf ? 0.f : m0) - kPShift, base1 = (m1 == kNegInf ? 0.f : m1) - kPShift;
      float pr[2][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        pr[r][0] = fast_exp2(sc[r][0] - base0);
        pr[r][1] = fast_exp2(sc[r][1] - base0);
        pr[r][2] = fast_exp2(sc[r][2] - base1);
        pr[r][3] = fast_exp2(sc[r][3] - base1);
      }
      float ps0 = (pr[0][0] + pr[0][1]) + (pr[1][0] + pr[1][1]);
      float ps1 = (pr[0][2] + pr[0][3]) + (pr[1][2] + pr[1][3]);
      if constexpr (kStats) {
        ps0 += __shfl_xor_sync(0xffffffffu, ps0, 1);
        ps1 += __shfl_xor_sync(0xffffffffu, ps1, 1);
        ps0 += __shfl_xor_sync(0xffffffffu, ps0, 2);
        ps1 += __shfl_xor_sync(0xffffffffu, ps1, 2);
        if (cq == 0) {
          const int slots = a.idx ? a.kslots : a.nb_cap;
          float2* st = a.stats + (((size_t)p.bg * slots + s) * kWarpsPerBlock + wq) * kHeads;
          st[g] = make_float2(m0, ps0);
          st[g + 8] = make_float2(m1, ps1);
        }
      }
      l0 += ps0;              // without kStats: this lane's share, summed over the four lanes at the end
      l1 += ps1;
      const __half2 h0 = __floats2half2_rn(pr[0][0], pr[0][1]), h1 = __floats2half2_rn(pr[0][2], pr[0][3]);
      const __half2 h2 = __floats2half2_rn(pr[1][0], pr[1][1]), h3 = __floats2half2_rn(pr[1][2], pr[1][3]);
      const uint32_t pa0 = *reinterpret_cast<const uint32_t*>(&h0), pa1 = *reinterpret_cast<const uint32_t*>(&h1);
      const uint32_t pa2 = *reinterpret_cast<const uint32_t*>(&h2), pa3 = *reinterpret_cast<const uint32_t*>(&h3);
      const uint4 v0 = lds128(blk + kVCodes + wq * 1024 + lane * 16), v1 = lds128(blk + kVCodes + wq * 1024 + 512 + lane * 16);
      uint2 z0 = *reinterpret_cast<const uint2*>(blk + kVScales + ((wq * 2) * 4 + cq) * 32 + (g >> 1) * 8);
      uint2 z1 = *reinterpret_cast<const uint2*>(blk + kVScales + ((wq * 2 + 1) * 4 + cq) * 32 + (g >> 1) * 8);
      if (live < 16) {        // tokens that do not exist hold anything: their values become 0
        const uint32_t k0 = (2 * cq < live ? 0xffffu : 0u) | (2 * cq + 1 < live ? 0xffff0000u : 0u);
        const uint32_t k1 = (8 + 2 * cq < live ? 0xffffu : 0u) | (9 + 2 * cq < live ? 0xffff0000u : 0u);
        z0.x &= k0;
        z0.y &= k0;
        z1.x &= k1;
        z1.y &= k1;
      }
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        const uint32_t wa = n < 4 ? v0.x : n < 8 ? v0.y : n < 12 ? v0.z : v0.w;
        const uint32_t wb = n < 4 ? v1.x : n < 8 ? v1.y : n < 12 ? v1.z : v1.w;
        mma_16816_f16(o[n], pa0, pa1, pa2, pa3, value_pair(wa, n & 3, as_h2(z0.x), as_h2(z0.y)),
                      value_pair(wb, n & 3, as_h2(z1.x), as_h2(z1.y)));
      }
      __syncwarp();
      if (lane == 0) arrive(&empty[stage]);
    }
    if constexpr (!kStats) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    }

    // ---------------------------------------------------------- merge the warps
    sync_consumers();                          // the merge buffer is free again
    {
      float* r0 = mO + (warp * kHeads + g) * kRow;
      float* r1 = r0 + 8 * kRow;
#pragma unroll
      for (int i = 0; i < 4; ++i) {            // o[n][0]: channel 32 cq + n; o[n][1]: 32 cq + 16 + n
        *reinterpret_cast<float4*>(r0 + 36 * cq + 4 * i) = make_float4(o[4 * i][0], o[4 * i + 1][0], o[4 * i + 2][0], o[4 * i + 3][0]);
        *reinterpret_cast<float4*>(r0 + 36 * cq + 16 + 4 * i) = make_float4(o[4 * i][1], o[4 * i + 1][1], o[4 * i + 2][1], o[4 * i + 3][1]);
        *reinterpret_cast<float4*>(r1 + 36 * cq + 4 * i) = make_float4(o[4 * i][2], o[4 * i + 1][2], o[4 * i + 2][2], o[4 * i + 3][2]);
        *reinterpret_cast<float4*>(r1 + 36 * cq + 16 + 4 * i) = make_float4(o[4 * i][3], o[4 * i + 1][3], o[4 * i + 2][3], o[4 * i + 3][3]);
      }
      if (cq == 0) {
        mM[warp * kHeads + g] = m0;
        mM[warp * kHeads + g + 8] = m1;
        mL[warp * kHeads + g] = l0;
        mL[warp * kHeads + g + 8] = l1;
      }
    }
    sync_consumers();
    // thread t < 256: head h = t / 16, channels d0 .. d0 + 7
    const int t = tid, h = (t >> 4) & 15, d0 = (t & 15) * 8;
    float M = kNegInf, L = 0.f, acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    const bool active = t < 256;
    if (active) {
#pragma unroll
      for (int w = 0; w < kCWarps; ++w) M = fmaxf(M, mM[w * kHeads + h]);
      const float base = M == kNegInf ? 0.f : M;
#pragma unroll
      for (int w = 0; w < kCWarps; ++w) {
        const float wt = fast_exp2(mM[w * kHeads + h] - base);
        L += wt * mL[w * kHeads + h];
        const float* row = mO + (w * kHeads + h) * kRow + mcol(d0);
        const float4 x = *reinterpret_cast<const float4*>(row), y = *reinterpret_cast<const float4*>(row + 4);
        acc[0] += wt * x.x; acc[1] += wt * x.y; acc[2] += wt * x.z; acc[3] += wt * x.w;
        acc[4] += wt * y.x; acc[5] += wt * y.y; acc[6] += wt * y.z; acc[7] += wt * y.w;
      }
    }
    bool write = active;
    if (p.n_cta > 1) {
      // a CTA's partial of its first piece lies in slot 0, of its last in slot 1; a piece that is
      // neither covers its group alone
      const int slot = c * 2 + (first_piece ? 0 : 1);
      if (active) {
        float4* po = reinterpret_cast<float4*>(a.part_o + ((size_t)slot * kHeads + h) * kHeadDim + d0);
        po[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        po[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if ((t & 15) == 0) {
          a.part_ml[slot * 2 * kHeads + h] = M;
          a.part_ml[slot * 2 * kHeads + kHeads + h] = L;
        }
      }
      sync_consumers();                        // every consumer's partial stores are issued
      if (t == 0) {
        unsigned prev;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(prev) : "l"(a.counters + p.bg) : "memory");
        *s_flag = prev == (unsigned)(p.n_cta - 1);
        if (*s_flag) a.counters[p.bg] = 0u;
      }
      sync_consumers();
      write = write && *s_flag != 0;
      if (write) {
        // the last CTA of the group joins the partials. The group's first CTA left its partial in
        // slot 1 unless the group begins that CTA's range; all others in slot 0.
        const int g0 = s_pre[p.bg];
        const int first_slot = p.first * 2 + ((int)((long long)U * p.first / ctas) == g0 ? 0 : 1);
        M = kNegInf;
        L = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        constexpr int kFlight = 8;
        for (int q0 = 0; q0 < p.n_cta; q0 += kFlight) {
          float pm[kFlight], pl[kFlight];
          float4 px[kFlight][2];
#pragma unroll
          for (int q = 0; q < kFlight; ++q) {
            const bool in = q0 + q < p.n_cta;
            const int sl = q0 + q == 0 || !in ? first_slot : (p.first + q0 + q) * 2;
            pm[q] = in ? __ldcg(a.part_ml + sl * 2 * kHeads + h) : kNegInf;
            pl[q] = __ldcg(a.part_ml + sl * 2 * kHeads + kHeads + h);
            const float4* src = reinterpret_cast<const float4*>(a.part_o + ((size_t)sl * kHeads + h) * kHeadDim + d0);
            px[q][0] = __ldcg(src);
            px[q][1] = __ldcg(src + 1);
          }
          float Mn = M;
#pragma unroll
          for (int q = 0; q < kFlight; ++q) Mn = fmaxf(Mn, pm[q]);
          const float base = Mn == kNegInf ? 0.f : Mn;
          const float old = fast_exp2(M - base);
          L *= old;
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] *= old;
#pragma unroll
          for (int q = 0; q < kFlight; ++q) {
            const float wt = fast_exp2(pm[q] - base);
            if (q0 + q < p.n_cta) {
              L += wt * pl[q];
              acc[0] += wt * px[q][0].x; acc[1] += wt * px[q][0].y; acc[2] += wt * px[q][0].z; acc[3] += wt * px[q][0].w;
              acc[4] += wt * px[q][1].x; acc[5] += wt * px[q][1].y; acc[6] += wt * px[q][1].z; acc[7] += wt * px[q][1].w;
            }
          }
          M = Mn;
        }
      }
    }
    if (write) {
      if constexpr (kStats) {
        if ((t & 15) == 0) {
          a.ml[p.bg * 2 * kHeads + h] = M;
          a.ml[p.bg * 2 * kHeads + kHeads + h] = L;
        }
      }
      if (h < a.H) {
        uint32_t pk[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) pk[e] = L == 0.f ? 0u : pack_bf16(acc[2 * e] / L, acc[2 * e + 1] / L);
        *reinterpret_cast<uint4*>(a.out + ((size_t)p.bg * a.H + h) * kHeadDim + d0) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
      }
    }
    first_piece = false;
  }
  // groups without a block belong to no range: their output is zero
  if (balanced) {
    for (int bg = c; bg < a.bg_count; bg += ctas) {
      if (s_pre[bg + 1] != s_pre[bg]) continue;
      uint32_t* out = reinterpret_cast<uint32_t*>(a.out + (size_t)bg * a.H * kHeadDim);
      for (int i = tid; i < a.H * kHeadDim / 2; i += kCThreads) out[i] = 0u;
    }
  }
}

void launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t s) {
  const long long bound = (long long)a.bg_count * (a.idx ? a.kslots : a.nb_cap);
  int grid = sm_count() < kKv4MaxCtas ? sm_count() : kKv4MaxCtas;
  const long long want = a.bg_count <= kPlanMax ? (bound + kMinUnits - 1) / kMinUnits : a.bg_count;
  if (want < grid) grid = (int)want;
  auto kern = a.stats ? kv4_attn_kernel<true> : kv4_attn_kernel<false>;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem4);
  launch_pdl(kern, dim3(grid), dim3(kThreads4), kSmem4, s, a);
}

}  // namespace sparda
