// Decode attention over the 4-bit cache: o = sum_t softmax_t(q . k_t / sqrt(d)) v_t for the H <= 16
// query heads of each (sequence, group), over the tokens of the selected blocks or of all blocks.
//
// What bounds it: a token is 160 bytes of cache for 4 * 16 * 128 multiply-adds and 256 codes to
// expand. The heads are the M dimension of warp-level MMAs (m16n8k16), and the cache is the B operand,
// expanded in registers straight into B fragments (1.4 instructions per code, kv4.cuh). Batch 16 of 131072
// tokens (671 MB) takes 139.5 us, and 137 us when every copy hits the same blocks in L2, so not the
// memory bounds a long cache. At the 2070 MHz sampled meanwhile a scheduler spends 670 cycles on 16 tokens
// of a group. 293 instructions are issued for them, 32 of them products; in a loop of nothing else a product
// with the expansion of its operands took 13.5 cycles (8.2 and 8.7 apart: the two only half overlap), which
// makes 430. The other 240 belong to neither: a scheduler has two of these warps, and the rest of a step, the
// maximum, the vote, the exponentials and their packing, has only the other warp's products to hide
// behind. A tcgen05 form, whose expanded operands go through tensor memory, took 240 us. With at most 8 heads (kEight) the roles
// change: the cache is the A operand, 16 tokens or 16 channels of it, the heads are the N dimension,
// and half the products do: the same batch with 8 heads takes 116 us, 0.85 of the memory's rate
// (147 with the heads as M; 113 without the memory's part). A score tile's 8 x 8 weights are transposed
// between lanes on the way.
//
// Work, three forms chosen by launch_kv4_attn:
//   - few blocks per (sequence, group): one thread-block cluster each (of one CTA where there are more
//     groups than SMs), the blocks split evenly over its CTAs, results joined in distributed shared
//     memory; no plan, no workspace;
//   - else the blocks of all (sequence, group)s in a row, U of them, cut into one contiguous range
//     per CTA, of equal cost whatever the lengths. Every CTA finds its range itself from seq_len
//     or cnt (a prefix sum over the groups), since the lengths live on the device. A group's CTAs
//     leave partial results in a workspace, and the last to arrive joins them, always in the same order;
//   - with more (sequence, group)s than the prefix sums hold, whole groups per CTA, in turn.
// Whole blocks (10 KiB, one bulk copy each) go through a ring of 16 stages in shared memory: lane l of the
// producer warp fills stage l whenever it is free, so all stages are polled at once and no free one
// waits for another. The consumer warps take blocks in turn, kW warps per block.
//
// Numbers: S in float32 from exact products (keys and queries are bf16); softmax in float32, base
// 2; sums in float32. A weight is a power of two of its score's distance to a reference, which
// follows the running maximum of its head only when that has risen by more than 2^8: with 16 heads
// some maximum rises in most steps of 16 tokens, and the rescaling (64 multiplications) with it
// (batch 16 of 131072 tokens: 192 us with a rescaling at every rise, 186 us at that stage without). The
// weights are operands in fp16, scaled by 2^6: at most 2^14, at full precision (2^-11) down to 2^-20 of
// the reference, and below that off by at most 2^-31 of it each.
#include <cuda_fp16.h>

#include "block_mass.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace sparda {
using namespace kv4;

namespace {

constexpr int kCWarps = 8;
constexpr int kCThreads = kCWarps * 32;
// The producer has a warpgroup to itself, of which one warp works: registers are moved from it to the
// consumers, which would otherwise be held to 168 each and spill (162 us instead of 147 for batch 16 of
// 131072 tokens when it was tried; twelve consumer warps of fewer registers also 162; now 143.0 at 208,
// with a few spilled, and 139.6 at 232).
constexpr int kThreads4 = kCThreads + 128;
constexpr int kLaunchRegs = 168, kProducerRegs = 40, kConsumerRegs = 232;
static_assert(128 * kProducerRegs + kCThreads * kConsumerRegs <= kThreads4 * kLaunchRegs, "registers the launch holds");
constexpr int kRing = 16;                                   // at most a warp's lanes
constexpr int kPlanMax = 1024;
static_assert(kPlanMax <= 32 * 32, "two steps of a warp find a group");
constexpr int kRow = 144;                                   // merge-buffer row: 128 + 4 per 32, no bank conflicts
constexpr int kMergeWarps = kCWarps / 2;                    // the others' results are folded in first
constexpr int kMergeFloats4 = kMergeWarps * (kHeads * kRow + 2 * kHeads);
constexpr int kQBytes = 8 * 512;                            // the queries as A fragments
constexpr int kHeader4 = 1024 + (kPlanMax + 32) * 4;
constexpr int kSmem4 = 128 + kHeader4 + kRing * kBlockBytes4 + kQBytes + kMergeFloats4 * 4;
// The cluster form's receive area: of each head that a CTA owns (rank h % cluster), the partial
// result of every CTA at entry (h / cluster) * cluster + source rank.
constexpr int kMaxCluster4 = 8;
constexpr int kRecv4 = kHeads + kMaxCluster4 - 1;
constexpr int kClusterSmem4 = kSmem4 + kRecv4 * (kHeadDim + 2) * 4;
constexpr int kMassSmem4 = kClusterSmem4 + kMaxCluster4 * 2 * kHeads * 4;      // and every CTA's references and sums
// The rules' limits, with both sides measured (kW = warps that share a block):
//   kWholeBlocks    blocks per warp from which a warp takes whole ones. Batch 16 of 131072 tokens (431
//                   blocks per CTA), 16 heads: kW 1 148 us, 2 151, 4 177; 8 heads: 117, 121, 144. A ragged
//                   batch of 8 x 8 groups of 4096 to 8191 tokens (41 per CTA), 4 heads: 24.6, 24.3, 25.6.
//   kPairBlocks     blocks per CTA of a cluster above which two warps share a block, not four. 34 blocks in
//                   clusters of 4 (8.5 per CTA): kW 2 8.45 us, 4 8.8, with 8 heads 7.4, 7.57; clusters
//                   of 8 (4.25 per CTA): 7.04, 6.95.
//   kCtaCost        what a CTA of the cluster form costs beside its blocks, and the planned form beside its
//   kPlanCost       share of blocks and beginnings, in blocks. With them the cheaper form is the one measured
//                   faster at (groups, blocks, clusters vs plan in us, 16 heads): (2, 34) 6.8, 12.5; (32, 34)
//                   8.4, 14.8; (140, 34) 17.5, 26.2; (160, 16) 17.9, 19.0; (160, 34) 30.2, 27.8; (200, 24)
//                   24.6, 27.5; (200, 34) 31.2, 31.3; (200, 64) 49, 44; (400, 6) 18.7, 20.8; (600, 34) 64, 71;
//                   (600, 64) 95, 104. The rule counts SMs, but a cluster lies inside one GPC, where some
//                   sizes leave SMs over and take a second wave that it does not expect: 34 blocks of 16 to 21,
//                   24, 25, 30 or 38 groups take 11.8 to 13.4 us, of 22, 26, 28 or 32 groups 6.9 to 7.7.
//   kClusterBlocks  blocks per CTA up to which groups get clusters where no list bounds them: above, the
//                   plan's balance over ragged lengths counts for more.
//   kMinUnits       blocks per CTA below which fewer CTAs work; 1, 2 and 4 measured alike, and 2 halves
//                   the CTAs that a small call occupies.
//   kPiece          what beginning a group costs a CTA of the planned form (its warps drain, join and start
//                   again), in blocks. 8 x 8 groups of 64 to 128 blocks, 4 heads: 24.5 us at 0, 22.6 at 14
//                   (22.9 now), 23.5 at 28; 200 groups of 34 blocks: 34.5, 30.6, 31.8.
//   kJoin           CTAs that join their results at once; those of a longer group join in two levels. One sequence
//                   of 131072 tokens (76 CTAs per group): 24.3 us at 4, 23.7 at 8, 24.2 at 16, 32.4 at once.
//   kPlanMax        (sequence, group)s of the balanced plan, held in 4 KiB of shared memory; beyond it there
//                   are at least six per SM, and whole groups balance well enough.
constexpr int kWholeBlocks = 2;
constexpr int kPiece = 14;
constexpr int kJoin = 8;
constexpr int kPairBlocks = 6;
constexpr int kCtaCost = 8, kPlanCost = 20;
constexpr int kClusterBlocks = 24;
constexpr int kMinUnits = 2;
constexpr float kPShift = 6.f;                              // weights are scaled by 2^kPShift
constexpr float kRise = 8.f;                                // rise of a maximum (base 2) that is let pass
constexpr uint32_t kProducerPolls = 1u << 25;               // bounds a lane's wait to seconds
constexpr float kNegInf = -INFINITY;
// The running maximum before any token: finite, so that no difference of maxima is a NaN.
constexpr float kLowest = -3.0e38f;

__device__ __forceinline__ void sync_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(kCThreads) : "memory"); }
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// D += A B (m16n8k16, fp16 or bf16 operands). Not volatile: the compiler may interleave products with
// the unpacking of later operands.
template <bool kHalf>
__device__ __forceinline__ void product(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  if constexpr (kHalf) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}
// x of all the lanes that hold the same heads: the four of a quad, or with kEight one of each quad.
template <bool kEight, typename Op>
__device__ __forceinline__ float over_lanes(float x, Op op) {
#pragma unroll
  for (int d = kEight ? 4 : 1; d <= (kEight ? 16 : 2); d <<= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}
// An 8 x 8 matrix of 16-bit values, two per lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Channel c of a merge-buffer row.
__device__ __forceinline__ int mcol(int c) { return c + 4 * (c >> 5); }

// Blocks of (sequence, group) bg.
__device__ __forceinline__ int group_blocks(const Kv4AttnArgs& a, int bg, int T) {
  const int n = a.idx ? min(max(a.cnt[bg], 0), a.kslots) : (T - 1) / kBlock + 1;    // loaded beside T
  return T < 1 || T > a.max_ctx ? 0 : n;
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

}  // namespace

// kStats: also store every quarter block's softmax statistics (max, sum of each head) and the
// final ones, for the block mass.
//
// kW: warps that share a block. 1: a warp takes whole blocks, 32 tokens at a time; 2 and 4: a warp takes
// 32 or 16 tokens of each block, for short ranges, where the time to the first result counts.
// kCluster: the n_cta CTAs of a (sequence, group) form a thread-block cluster, one piece each, and
// join their results in distributed shared memory; no plan, no workspace.
// kEight: at most 8 heads.
template <int kW, bool kStats, bool kCluster, bool kEight>
__global__ void __launch_bounds__(kThreads4, 1) kv4_attn_kernel(const Kv4AttnArgs a, int cluster) {
  extern __shared__ uint8_t smem_raw4[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw4) + 127) & ~static_cast<uintptr_t>(127));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + kRing;
  int* stage_live = reinterpret_cast<int*>(empty + kRing);   // tokens of the staged block that exist
  int* s_flag = stage_live + kRing;
  int* s_pre = reinterpret_cast<int*>(smem + 1024);
  uint8_t* ring = smem + kHeader4;
  uint4* s_q = reinterpret_cast<uint4*>(ring + kRing * kBlockBytes4);
  float* mO = reinterpret_cast<float*>(ring + kRing * kBlockBytes4 + kQBytes);
  float* mM = mO + kMergeWarps * kHeads * kRow;
  float* mL = mM + kMergeWarps * kHeads;
  constexpr int kBlockGroups = kCWarps / kW;     // blocks in the consumers' hands at a time
  constexpr int kTiles = kW == 4 ? 2 : 4;        // 8-token tiles of a step
  constexpr int kSteps = 8 / kW / kTiles;        // steps of a warp per block
  constexpr int kAcc = kEight ? 8 : 16;          // accumulators of 16 heads x 8 channels, or of 16 channels x 8 heads
  static_assert(kRing % kBlockGroups == 0, "each ring stage must belong to one group of consumers");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kW);
    }
    fence_mbar_init();
    const Masks m;
    s_flag[1] = (int)m.key;
    s_flag[2] = (int)m.lo;
    s_flag[3] = (int)m.hi;
  }
  // A group's queries as A fragments, rows g and g + 8: K step 2 w + i takes channels 32 cq + 8 w + 4 i ..
  // They are put together in shared memory and loaded as quadruples: built in registers, they would be
  // moved into place again in every step.
  const auto stage_queries = [&](int bg, int w) {
    const int g = lane >> 2, cq = lane & 3;
    const uint4* q0 = reinterpret_cast<const uint4*>(a.q + ((size_t)bg * a.H + g) * kHeadDim + 32 * cq);
    const uint4 none = make_uint4(0, 0, 0, 0);
    const uint4 x = g < a.H ? q0[w] : none, y = g + 8 < a.H ? q0[w + 8 * (kHeadDim / 8)] : none;
    s_q[(2 * w) * 32 + lane] = make_uint4(x.x, y.x, x.y, y.y);
    s_q[(2 * w + 1) * 32 + lane] = make_uint4(x.z, y.z, x.w, y.w);
  };
  if constexpr (kCluster) cluster_arrive();       // waited for before the first write to another CTA's memory
  grid_dep_wait();
  grid_dep_launch();

  // ------------------------------------------------------------ the plan
  const bool balanced = !kCluster && a.bg_count <= kPlanMax;
  // The CTAs' ranges are equal in cost: a block counts 1, a group's beginning kPiece more. Block u of the
  // row, of group bg, then begins at cost u + kPiece (bg + 1).
  int U = 0, V = 0, ctas = gridDim.x, u0 = 0, u1 = 0, n0 = 0, w_bg = 0, T0 = 0;
  // the first block of CTA i's range, and (bg) a group at or before its
  const auto cut = [&](int i, int& bg) {
    const int v = (int)((long long)V * i / ctas);
    // the last group that begins at or before cost v, by a warp, in two steps of 32 candidates
    const int stride = (a.bg_count + 31) >> 5;
    int at = lane * stride;
    unsigned m = __ballot_sync(0xffffffffu, at < a.bg_count && s_pre[at] + kPiece * at <= v);
    int lo = (31 - __clz(m)) * stride;
    at = lo + lane;
    m = __ballot_sync(0xffffffffu, lane < stride && at < a.bg_count && s_pre[at] + kPiece * at <= v);
    lo += 31 - __clz(m);
    bg = lo;
    return min(s_pre[lo] + max(v - (s_pre[lo] + kPiece * (lo + 1)), 0), s_pre[lo + 1]);
  };
  const auto cta_of = [&](int unit, int bg) {
    return (int)(((long long)(unit + kPiece * (bg + 1) + 1) * ctas - 1) / V);
  };
  if constexpr (kCluster) {
    const int bg = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    // the length, the list and the queries at once: one round trip to memory
    const int T = a.seq_len[bg / a.G];
    const int j = a.idx && tid < a.kslots ? a.idx[(size_t)bg * a.kslots + tid] : 0;
    if (warp < 4) stage_queries(bg, warp);
    n0 = group_blocks(a, bg, T);
    s_pre[tid] = j;
    u0 = n0 * rank / cluster;
    u1 = n0 * (rank + 1) / cluster;
    T0 = T;
    if ((T < 1 || T > a.max_ctx) && rank == 0 && tid == 0) atomicOr(a.err, SPARDA_DEV_BAD_SEQ_LEN);
    __syncthreads();                               // the barriers are initialised
  } else if (balanced) {
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
    V = U + kPiece * a.bg_count;
    u0 = cut(blockIdx.x, w_bg);
    int end_bg;
    u1 = cut(blockIdx.x + 1, end_bg);
  } else {
    __syncthreads();
  }
  const int c = blockIdx.x;

  // Walks the CTA's pieces: balanced, the groups its unit range meets; in a cluster, its share of the
  // one group; else whole groups c, c + grid, ...
  int w_u = u0;
  if (!balanced) w_bg = kCluster ? c / cluster : c;
  const auto next_piece = [&](Piece& p) -> bool {
    if (balanced) {
      if (w_u >= u1) return false;
      while (s_pre[w_bg + 1] <= w_u) ++w_bg;
      const int g0 = s_pre[w_bg], g1 = s_pre[w_bg + 1];
      p.bg = w_bg;
      p.s0 = w_u - g0;
      p.s1 = min(u1, g1) - g0;
      p.first = cta_of(g0, w_bg);
      p.n_cta = cta_of(g1 - 1, w_bg) - p.first + 1;
      w_u = min(u1, g1);
      return true;
    }
    if (w_bg >= a.bg_count) return false;
    p.bg = w_bg;
    if constexpr (kCluster) {
      p.s0 = u0;
      p.s1 = u1;
      p.first = c;
      p.n_cta = 1;
      w_bg = a.bg_count;
      return true;
    }
    p.s0 = 0;
    const int T = a.seq_len[w_bg / a.G];
    if ((T < 1 || T > a.max_ctx) && tid == 0) atomicOr(a.err, SPARDA_DEV_BAD_SEQ_LEN);
    p.s1 = group_blocks(a, w_bg, T);
    p.first = c;
    p.n_cta = 1;
    w_bg += gridDim.x;
    return true;
  };

  if (warp >= kCWarps) {
    // ------------------------------------------------------------ producer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    // Lane l < kRing fills ring stage l: the CTA's units l, l + kRing, ... Each pass over the lanes
    // polls every stage at once and refills those that are free.
    if (warp == kCWarps && lane < kRing) {
      int left = u1 - u0 - lane;                     // balanced or cluster: units from this lane's next on
      int bg = w_bg, n = 0, s = lane;                // its next unit: slot s of the n of group bg
      if (kCluster) {
        s += u0;
        n = n0;
      } else if (balanced) {
        if (left > 0) {
          s += u0 - s_pre[bg];
          n = s_pre[bg + 1] - s_pre[bg];
        }
      } else if (bg < a.bg_count) {
        n = group_blocks(a, bg, a.seq_len[bg / a.G]);
      }
      uint32_t round = 0, polls = 0;
      const uint8_t* src = nullptr;
      int live = 0;
      // the lane's next unit, looked up ahead of the wait for its stage; false behind the last
      const auto look_up = [&]() -> bool {
        if (kCluster || balanced ? left <= 0 : bg >= a.bg_count) return false;
        while (s >= n) {
          s -= n;
          bg += balanced ? 1 : (int)gridDim.x;
          if (!balanced && bg >= a.bg_count) return false;
          n = balanced ? s_pre[bg + 1] - s_pre[bg] : group_blocks(a, bg, a.seq_len[bg / a.G]);
        }
        int j = !a.idx ? s : kCluster ? s_pre[s] : a.idx[(size_t)bg * a.kslots + s];
        const int T = kCluster ? T0 : a.seq_len[bg / a.G];
        if ((unsigned)j > (unsigned)((T - 1) / kBlock)) {
          atomicOr(a.err, SPARDA_DEV_BAD_INDEX);     // skipped: block 0 is staged with no live token
          j = 0;
          live = 0;
        } else {
          live = min(kBlock, T - j * kBlock);
        }
        src = a.kv + ((size_t)bg * a.nb_cap + j) * kBlockBytes4;
        s += kRing;
        left -= kRing;
        return true;
      };
      bool more = look_up();
      while (more) {
        if (round == 0 || mbar_test_wait(&empty[lane], (round & 1) ^ 1)) {
          stage_live[lane] = live;
          mbar_arrive_expect_tx(&full[lane], kBlockBytes4);
          bulk_load(ring + lane * kBlockBytes4, src, kBlockBytes4, &full[lane]);
          ++round;
          polls = 0;
          more = look_up();
        } else if (++polls > kProducerPolls) {
          atomicOr(a.err, SPARDA_DEV_WAIT_TIMEOUT);
          more = false;
        }
      }
    }
    if constexpr (kCluster) {                        // the consumers' barriers
      cluster_wait();
      cluster_sync();
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
  const int grp = warp / kW, wq = warp % kW;
  const int g = lane >> 2, cq = lane & 3;
  const float sl2 = 1.4426950408889634f * 0.08838834764831845f;   // log2(e) / sqrt(128)
  int it = 0;
  bool ok = true;             // a wait that ran out: no further compute, the barriers stay matched
  const uint32_t masks_at = smem_addr(s_flag) + 4;
  const Masks mk{lds32(masks_at), lds32(masks_at + 4), lds32(masks_at + 8)};
  const uint32_t ring_at = smem_addr(ring), live_at = smem_addr(stage_live);
  Piece p;
  while (next_piece(p)) {
    // the references, raw scores, and the exponents' offsets: p = 2^(sl2 (s - m) + kPShift)
    float m0 = kLowest, m1 = kLowest, l0 = 0.f, l1 = 0.f;
    float nb0 = kPShift - m0 * sl2, nb1 = kPShift - m1 * sl2;
    float up0 = kLowest, up1 = kLowest;        // a score above it moves the reference
    float o[kAcc][4];
#pragma unroll
    for (int n = 0; n < kAcc; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    uint4 qf[8];
    if constexpr (!kCluster) {                     // every warp writes the same values before it reads them
#pragma unroll
      for (int w = 0; w < 4; ++w) stage_queries(p.bg, w);
    }
#pragma unroll
    for (int w = 0; w < 8; ++w) qf[w] = lds128(smem_addr(s_q + w * 32 + lane));
    // this group's blocks of the piece: its ring stages come round every kBlockGroups
    int skip = grp - it % kBlockGroups;
    if (skip < 0) skip += kBlockGroups;
    int stage = (it + skip) % kRing, phase = ((it + skip) / kRing) & 1;
    it += p.s1 - p.s0;
    for (int s = p.s0 + skip; ok && s < p.s1; s += kBlockGroups) {
      ok = __all_sync(0xffffffffu, mbar_wait(&full[stage], phase, a.err));
      if (!ok) break;
      const int block_live = (int)lds32(live_at + 4 * stage);
#pragma unroll 1
      for (int step = 0; step < kSteps; ++step) {
        const int tile0 = (wq * kSteps + step) * kTiles;         // the step's first 8-token tile of the block
        const int live = block_live - 8 * tile0;                 // tokens of the step that exist
        const uint32_t blk = ring_at + stage * kBlockBytes4;
        const uint32_t kc = blk + kKCodes + tile0 * 512 + lane * 16, ks = blk + kKScales + tile0 * 128 + lane * 4;
        const uint32_t vc = blk + kVCodes + tile0 * 512 + lane * 16;
        const uint32_t vs = blk + kVScales + (tile0 * 4 + cq) * 32 + (g >> 1) * 8;
        // raw scores: tokens 2 cq and 2 cq + 1 of tile r, heads g and g + 8; kEight: of a pair of tiles,
        // token g of either, heads 2 cq and 2 cq + 1
        constexpr int kScores = kEight ? kTiles / 2 : kTiles;
        float sc[kScores][4];
        uint4 kw[kTiles];
        uint32_t s2[kTiles], z2[kTiles];
#pragma unroll
        for (int r = 0; r < kTiles; ++r) {
          kw[r] = lds128(kc + r * 512);
          const uint32_t sz = lds32(ks + r * 128);
          s2[r] = dup_lo(sz);
          z2[r] = dup_hi(sz);
        }
#pragma unroll
        for (int r = 0; r < kScores; ++r) sc[r][0] = sc[r][1] = sc[r][2] = sc[r][3] = 0.f;
        // the tiles side by side, so that consecutive products do not wait for one another
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const auto keys = [&](int r, int half) {
            const uint32_t word = k < 2 ? kw[r].x : k < 4 ? kw[r].y : k < 6 ? kw[r].z : kw[r].w;
            return key_pair(word, 2 * (k & 1) + half, s2[r], z2[r], mk);
          };
#pragma unroll
          for (int r = 0; r < kScores; ++r) {
            if constexpr (kEight)
              product<false>(sc[r], keys(2 * r, 0), keys(2 * r + 1, 0), keys(2 * r, 1), keys(2 * r + 1, 1), qf[k].x, qf[k].z);
            else
              product<false>(sc[r], qf[k].x, qf[k].y, qf[k].z, qf[k].w, keys(r, 0), keys(r, 1));
          }
        }
        // scales and offsets of the value tiles
        uint2 z[kTiles];
#pragma unroll
        for (int r = 0; r < kTiles; ++r) z[r] = lds64(vs + r * 128);
        if (live < 8 * kTiles) {
          // tokens that do not exist hold anything: no weight, and values of 0
#pragma unroll
          for (int r = 0; r < kTiles; ++r) {
            const bool in0 = 8 * r + 2 * cq < live, in1 = 8 * r + 2 * cq + 1 < live;
            if constexpr (kEight) {
              if (8 * r + g >= live) sc[r / 2][2 * (r & 1)] = sc[r / 2][2 * (r & 1) + 1] = kNegInf;
            } else {
              sc[r][0] = in0 ? sc[r][0] : kNegInf;
              sc[r][1] = in1 ? sc[r][1] : kNegInf;
              sc[r][2] = in0 ? sc[r][2] : kNegInf;
              sc[r][3] = in1 ? sc[r][3] : kNegInf;
            }
            const uint32_t keep = (in0 ? 0xffffu : 0u) | (in1 ? 0xffff0000u : 0u);
            z[r].x &= keep;
            z[r].y &= keep;
          }
        }
        // a lane's two heads are its scores 0, 1 and 2, 3; kEight: 0, 2 and 1, 3
        float mx0 = fmaxf(sc[0][0], sc[0][kEight ? 2 : 1]), mx1 = fmaxf(sc[0][kEight ? 1 : 2], sc[0][3]);
#pragma unroll
        for (int r = 1; r < kScores; ++r) {
          mx0 = fmaxf(mx0, fmaxf(sc[r][0], sc[r][kEight ? 2 : 1]));
          mx1 = fmaxf(mx1, fmaxf(sc[r][kEight ? 1 : 2], sc[r][3]));
        }
        if (__any_sync(0xffffffffu, mx0 > up0 || mx1 > up1)) {     // move the references
          mx0 = over_lanes<kEight>(mx0, [](float x, float y) { return fmaxf(x, y); });
          mx1 = over_lanes<kEight>(mx1, [](float x, float y) { return fmaxf(x, y); });
          const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
          const float al0 = fast_exp2((m0 - n0) * sl2), al1 = fast_exp2((m1 - n1) * sl2);
          m0 = n0;
          m1 = n1;
          nb0 = kPShift - m0 * sl2;
          nb1 = kPShift - m1 * sl2;
          up0 = m0 + kRise / sl2;
          up1 = m1 + kRise / sl2;
          l0 *= al0;
          l1 *= al1;
#pragma unroll
          for (int n = 0; n < kAcc; ++n) {
            o[n][0] *= al0;
            o[n][1] *= kEight ? al1 : al0;
            o[n][2] *= kEight ? al0 : al1;
            o[n][3] *= al1;
          }
        }
        // weights, as A fragments of 16 tokens; kEight: as B fragments, a tile's 8 x 8 transposed
        uint32_t pa[kTiles][2];
        float ps0 = 0.f, ps1 = 0.f;
#pragma unroll
        for (int r = 0; r < kScores; ++r) {
          const float nb01 = kEight ? nb1 : nb0, nb10 = kEight ? nb0 : nb1;
          const float p0 = fast_exp2(fmaf(sc[r][0], sl2, nb0)), p1 = fast_exp2(fmaf(sc[r][1], sl2, nb01));
          const float p2 = fast_exp2(fmaf(sc[r][2], sl2, nb10)), p3 = fast_exp2(fmaf(sc[r][3], sl2, nb1));
          ps0 += p0 + (kEight ? p2 : p1);
          ps1 += (kEight ? p1 : p2) + p3;
          const __half2 x = __floats2half2_rn(p0, p1), y = __floats2half2_rn(p2, p3);
          const uint32_t xb = *reinterpret_cast<const uint32_t*>(&x), yb = *reinterpret_cast<const uint32_t*>(&y);
          if constexpr (kEight) {
            pa[2 * r][0] = transposed(xb);
            pa[2 * r + 1][0] = transposed(yb);
          } else {
            pa[r][0] = xb;
            pa[r][1] = yb;
          }
        }
        if constexpr (kStats) {
          ps0 = over_lanes<kEight>(ps0, [](float x, float y) { return x + y; });
          ps1 = over_lanes<kEight>(ps1, [](float x, float y) { return x + y; });
          const int slots = a.idx ? a.kslots : a.nb_cap;
          float2* st = a.stats + (((size_t)p.bg * slots + s) * (8 / kTiles) + tile0 / kTiles) * kHeads;
          if (kEight ? g == 0 : cq == 0) {
            st[kEight ? 2 * cq : g] = make_float2(m0 * sl2, ps0);
            st[kEight ? 2 * cq + 1 : g + 8] = make_float2(m1 * sl2, ps1);
          }
        }
        l0 += ps0;            // without kStats: this lane's share, summed over the lanes at the end
        l1 += ps1;
        // o += weights . values
#pragma unroll
        for (int r = 0; r < kTiles; r += 2) {
          const uint4 v0 = lds128(vc + r * 512), v1 = lds128(vc + r * 512 + 512);
          const auto values = [&](const uint4& v, int n, const uint2& sz) {
            return value_pair(n < 4 ? v.x : n < 8 ? v.y : n < 12 ? v.z : v.w, n & 3, sz.x, sz.y, mk);
          };
#pragma unroll
          for (int n = 0; n < kAcc; ++n) {
            if constexpr (kEight)
              product<true>(o[n], values(v0, 2 * n, z[r]), values(v0, 2 * n + 1, z[r]), values(v1, 2 * n, z[r + 1]),
                            values(v1, 2 * n + 1, z[r + 1]), pa[r][0], pa[r + 1][0]);
            else
              product<true>(o[n], pa[r][0], pa[r][1], pa[r + 1][0], pa[r + 1][1], values(v0, n, z[r]), values(v1, n, z[r + 1]));
          }
        }
      }
      __syncwarp();
      if (lane == 0) arrive(&empty[stage]);
      stage += kBlockGroups;
      if (stage >= kRing) {
        stage -= kRing;
        phase ^= 1;
      }
    }
    m0 *= sl2;
    m1 *= sl2;
    if constexpr (!kStats) {
      l0 = over_lanes<kEight>(l0, [](float x, float y) { return x + y; });
      l1 = over_lanes<kEight>(l1, [](float x, float y) { return x + y; });
    }
    // ---------------------------------------------------------- merge the warps
    // The upper half of the warps hand their results to the lower half, lane for lane.
    if (warp >= kMergeWarps) {
      float4* give = reinterpret_cast<float4*>(mO + (warp - kMergeWarps) * kHeads * kRow) + lane;
#pragma unroll
      for (int n = 0; n < kAcc; ++n) give[n * 32] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
      give[kAcc * 32] = make_float4(m0, m1, l0, l1);
    }
    sync_consumers();
    if (warp < kMergeWarps) {
      float* mine = mO + warp * kHeads * kRow;
      const float4* take = reinterpret_cast<const float4*>(mine) + lane;
      const float4 ml = take[kAcc * 32];
      const float n0 = fmaxf(m0, ml.x), n1 = fmaxf(m1, ml.y);
      const float wa0 = fast_exp2(m0 - n0), wa1 = fast_exp2(m1 - n1), wb0 = fast_exp2(ml.x - n0), wb1 = fast_exp2(ml.y - n1);
      l0 = l0 * wa0 + ml.z * wb0;
      l1 = l1 * wa1 + ml.w * wb1;
#pragma unroll
      for (int n = 0; n < kAcc; ++n) {
        const float4 x = take[n * 32];
        o[n][0] = o[n][0] * wa0 + x.x * wb0;
        o[n][1] = o[n][1] * (kEight ? wa1 : wa0) + x.y * (kEight ? wb1 : wb0);
        o[n][2] = o[n][2] * (kEight ? wa0 : wa1) + x.z * (kEight ? wb0 : wb1);
        o[n][3] = o[n][3] * wa1 + x.w * wb1;
      }
      __syncwarp();
      const int h0 = kEight ? 2 * cq : g, h1 = kEight ? 2 * cq + 1 : g + 8;      // the lane's heads
      float* r0 = mine + h0 * kRow;
      float* r1 = mine + h1 * kRow;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kEight) {                // o[n][0]: channel 16 g + 2 n; o[n][2]: 16 g + 2 n + 1
          const int at = mcol(16 * g) + 4 * i;
          *reinterpret_cast<float4*>(r0 + at) = make_float4(o[2 * i][0], o[2 * i][2], o[2 * i + 1][0], o[2 * i + 1][2]);
          *reinterpret_cast<float4*>(r1 + at) = make_float4(o[2 * i][1], o[2 * i][3], o[2 * i + 1][1], o[2 * i + 1][3]);
        } else {                               // o[n][0]: channel 32 cq + n; o[n][1]: 32 cq + 16 + n
          const int at = mcol(32 * cq) + 4 * i;
          *reinterpret_cast<float4*>(r0 + at) = make_float4(o[4 * i][0], o[4 * i + 1][0], o[4 * i + 2][0], o[4 * i + 3][0]);
          *reinterpret_cast<float4*>(r0 + at + 16) = make_float4(o[4 * i][1], o[4 * i + 1][1], o[4 * i + 2][1], o[4 * i + 3][1]);
          *reinterpret_cast<float4*>(r1 + at) = make_float4(o[4 * i][2], o[4 * i + 1][2], o[4 * i + 2][2], o[4 * i + 3][2]);
          *reinterpret_cast<float4*>(r1 + at + 16) = make_float4(o[4 * i][3], o[4 * i + 1][3], o[4 * i + 2][3], o[4 * i + 3][3]);
        }
      }
      if (kEight ? g == 0 : cq == 0) {
        mM[warp * kHeads + h0] = n0;
        mM[warp * kHeads + h1] = n1;
        mL[warp * kHeads + h0] = l0;
        mL[warp * kHeads + h1] = l1;
      }
    }
    sync_consumers();
    // thread t: head h = t / 16, channels d0 .. d0 + 7
    const int t = tid, h = t >> 4, d0 = (t & 15) * 8;
    float M = kLowest, L = 0.f, acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    {
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) M = fmaxf(M, mM[w * kHeads + h]);
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
        const float wt = fast_exp2(mM[w * kHeads + h] - M);
        L += wt * mL[w * kHeads + h];
        const float* row = mO + (w * kHeads + h) * kRow + mcol(d0);
        const float4 x = *reinterpret_cast<const float4*>(row), y = *reinterpret_cast<const float4*>(row + 4);
        acc[0] += wt * x.x; acc[1] += wt * x.y; acc[2] += wt * x.z; acc[3] += wt * x.w;
        acc[4] += wt * y.x; acc[5] += wt * y.y; acc[6] += wt * y.z; acc[7] += wt * y.w;
      }
    }
    bool write = true;
    if constexpr (kCluster) {
      // pushed to the CTA that owns the head; behind the one cluster barrier no CTA reads another's
      // memory, so none has to stay for the others
      float* rO = mL + kMergeWarps * kHeads;
      float* rM = rO + kRecv4 * kHeadDim;
      float* rL = rM + kRecv4;
      const uint32_t rank = cluster_rank(), owner = (uint32_t)(h % cluster);
      const int e0 = (h / cluster) * cluster, entry = e0 + (int)rank;
      cluster_wait();                          // every CTA of the cluster has started
      st_cluster_f4(rO + entry * kHeadDim + d0, owner, make_float4(acc[0], acc[1], acc[2], acc[3]));
      st_cluster_f4(rO + entry * kHeadDim + d0 + 4, owner, make_float4(acc[4], acc[5], acc[6], acc[7]));
      if ((t & 15) == 0) {
        st_cluster_f(rM + entry, owner, M);
        st_cluster_f(rL + entry, owner, L);
        if constexpr (kStats) {
          // for the block mass every CTA learns everyone's: it then needs no second barrier
          for (int q = 0; q < cluster; ++q) {
            st_cluster_f(rL + kRecv4 + (rank * 2) * kHeads + h, (uint32_t)q, M);
            st_cluster_f(rL + kRecv4 + (rank * 2 + 1) * kHeads + h, (uint32_t)q, L);
          }
        }
      }
      cluster_sync();
      write = owner == rank;
      if (write) {
        for (int q = 0; q < cluster; ++q) M = fmaxf(M, rM[e0 + q]);
        L = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        for (int q = 0; q < cluster; ++q) {
          const float wt = fast_exp2(rM[e0 + q] - M);
          L += wt * rL[e0 + q];
          const float4* src = reinterpret_cast<const float4*>(rO + (e0 + q) * kHeadDim + d0);
          const float4 x = src[0], y = src[1];
          acc[0] += wt * x.x; acc[1] += wt * x.y; acc[2] += wt * x.z; acc[3] += wt * x.w;
          acc[4] += wt * y.x; acc[5] += wt * y.y; acc[6] += wt * y.z; acc[7] += wt * y.w;
        }
      }
    } else if (p.n_cta > 1) {
      // A CTA's partial of its first piece lies in slot 0, of its last in slot 1; a piece that is
      // neither covers its group alone. The group's first CTA left its partial in slot 1 unless the
      // group begins that CTA's range; all others in slot 0.
      const auto store_partial = [&](int slot) {
        float4* po = reinterpret_cast<float4*>(a.part_o + ((size_t)slot * kHeads + h) * kHeadDim + d0);
        po[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        po[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if ((t & 15) == 0) {
          a.part_ml[slot * 2 * kHeads + h] = M;
          a.part_ml[slot * 2 * kHeads + kHeads + h] = L;
        }
      };
      int at;
      const int first_slot = p.first * 2 + (cut(p.first, at) == s_pre[p.bg] ? 0 : 1);
      const auto slot_of = [&](int k) { return k == 0 ? first_slot : (p.first + k) * 2; };
      // Counts this CTA in; the last of n joins the partials of the group's CTAs k0, k0 + step, ... (n of
      // them, always in this order) into (M, L, acc) and returns true.
      const auto join = [&](unsigned* counter, int n, int k0, int step) -> bool {
        sync_consumers();                      // every consumer's partial stores are issued
        if (t == 0) {
          unsigned prev;
          asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(prev) : "l"(counter) : "memory");
          *s_flag = prev == (unsigned)(n - 1);
          if (*s_flag) *counter = 0u;
        }
        sync_consumers();
        if (*s_flag == 0) return false;
        M = kLowest;
        L = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        constexpr int kFlight = 4;
        for (int q0 = 0; q0 < n; q0 += kFlight) {
          float pm[kFlight], pl[kFlight];
          float4 px[kFlight][2];
#pragma unroll
          for (int q = 0; q < kFlight; ++q) {
            const bool in = q0 + q < n;
            const int sl = slot_of(in ? k0 + (q0 + q) * step : k0);
            pm[q] = in ? __ldcg(a.part_ml + sl * 2 * kHeads + h) : kLowest;
            pl[q] = __ldcg(a.part_ml + sl * 2 * kHeads + kHeads + h);
            const float4* src = reinterpret_cast<const float4*>(a.part_o + ((size_t)sl * kHeads + h) * kHeadDim + d0);
            px[q][0] = __ldcg(src);
            px[q][1] = __ldcg(src + 1);
          }
          float Mn = M;
#pragma unroll
          for (int q = 0; q < kFlight; ++q) Mn = fmaxf(Mn, pm[q]);
          const float old = fast_exp2(M - Mn);
          L *= old;
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] *= old;
#pragma unroll
          for (int q = 0; q < kFlight; ++q) {
            const float wt = fast_exp2(pm[q] - Mn);
            if (q0 + q < n) {
              L += wt * pl[q];
              acc[0] += wt * px[q][0].x; acc[1] += wt * px[q][0].y; acc[2] += wt * px[q][0].z; acc[3] += wt * px[q][0].w;
              acc[4] += wt * px[q][1].x; acc[5] += wt * px[q][1].y; acc[6] += wt * px[q][1].z; acc[7] += wt * px[q][1].w;
            }
          }
          M = Mn;
        }
        return true;
      };
      // Up to kJoin CTAs join at once; a group of more in two levels, kJoin neighbours first, whose result takes
      // the first one's slot.
      const int k = c - p.first, lead = k - k % kJoin;
      store_partial(slot_of(k));
      write = join(a.join_counters + slot_of(lead), min(kJoin, p.n_cta - lead), lead, 1);
      if (write && p.n_cta > kJoin) {
        __syncwarp();                          // the head's M and L have been read by its 16 threads
        store_partial(slot_of(lead));
        write = join(a.counters + p.bg, (p.n_cta + kJoin - 1) / kJoin, 0, kJoin);
      }
    }
    if (write) {
      if constexpr (kStats && !kCluster) {
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
    if constexpr (kCluster && kStats) {
      const SlotBlocks list = slot_blocks(a.idx ? s_pre : nullptr, n0);
      const int tb = (T0 - 1) / kBlock;
      const int slots = a.idx ? a.kslots : a.nb_cap;
      const float* every = mL + kMergeWarps * kHeads + kRecv4 * (kHeadDim + 2) + (lane & 15);
      float Mh = kLowest, Lh = 0.f;
      for (int q = 0; q < cluster; ++q) Mh = fmaxf(Mh, every[2 * q * kHeads]);
      for (int q = 0; q < cluster; ++q) Lh += fast_exp2(every[2 * q * kHeads] - Mh) * every[(2 * q + 1) * kHeads];
      for (int s = p.s0 + warp; s < p.s1; s += kCWarps)
        add_block_mass(a.stats + (size_t)p.bg * slots * (8 / kTiles) * kHeads, 8 / kTiles, a.H, Mh, Lh, list, s, tb,
                       a.mass + (size_t)p.bg * a.nb_cap);
    }
    if constexpr (kCluster) return;
    sync_consumers();                          // the merge buffer is free again
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

namespace {

template <int kW, bool kStats, bool kCluster, bool kEight>
cudaError_t launch_form(const Kv4AttnArgs& a, int grid, int cluster, cudaStream_t s, int* parts) {
  auto kern = kv4_attn_kernel<kW, kStats, kCluster, kEight>;
  constexpr int smem = !kCluster ? kSmem4 : kStats ? kMassSmem4 : kClusterSmem4;
  static_assert(smem <= 232448, "shared memory of a CTA");
  // the register split needs the registers that it counts on; a build with fewer must not run
  static std::atomic<bool> fits{false};
  if (!fits.load(std::memory_order_relaxed)) {
    cudaFuncAttributes at;
    const cudaError_t err = cudaFuncGetAttributes(&at, kern);
    if (err != cudaSuccess) return err;
    fits.store(at.numRegs * kThreads4 >= 128 * kProducerRegs + kCThreads * kConsumerRegs, std::memory_order_relaxed);
  }
  static SmemOptIn opt_in;
  if (!fits || !opt_in.set(kern, smem)) return cudaErrorLaunchOutOfResources;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads4);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 2 : 1;
  *parts = !kStats || kCluster ? 0 : kW == 4 ? 4 : 2;
  return cudaLaunchKernelEx(&cfg, kern, a, cluster);
}

template <int kW, bool kCluster>
cudaError_t launch_form(const Kv4AttnArgs& a, int grid, int cluster, cudaStream_t s, int* parts) {
  if (a.H <= 8)
    return a.stats ? launch_form<kW, true, kCluster, true>(a, grid, cluster, s, parts)
                   : launch_form<kW, false, kCluster, true>(a, grid, cluster, s, parts);
  return a.stats ? launch_form<kW, true, kCluster, false>(a, grid, cluster, s, parts)
                 : launch_form<kW, false, kCluster, false>(a, grid, cluster, s, parts);
}

}  // namespace

cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t s, int* parts) {
  const int sms = sm_count() < kKv4MaxCtas ? sm_count() : kKv4MaxCtas;
  const int slots = a.idx ? a.kslots : a.nb_cap;
  const long long bound = (long long)a.bg_count * slots;
  // One cluster per (sequence, group), or the plan: whichever the costs below favour. Clusters fill the SMs
  // at most once, or are single CTAs that come in waves.
  int cluster = a.bg_count <= sms ? sms / a.bg_count : 1;
  if (cluster > kMaxCluster4) cluster = kMaxCluster4;
  const int useful = (slots + kMinUnits - 1) / kMinUnits;
  if (cluster > useful) cluster = useful;
  const int share = (slots + cluster - 1) / cluster;
  const long long waves = ((long long)a.bg_count * cluster + sms - 1) / sms;
  const long long planned = (long long)a.bg_count * (slots + kPiece) / sms + kPlanCost;
  // Without a list, slots is the capacity: sequences may be far shorter, which the plan takes into account.
  if ((a.idx || share <= kClusterBlocks) && waves * (share + kCtaCost) <= planned) {
    const int ctas = cluster * a.bg_count;
    return share > kWholeBlocks * kCWarps ? launch_form<1, true>(a, ctas, cluster, s, parts)
           : share > kPairBlocks          ? launch_form<2, true>(a, ctas, cluster, s, parts)
                                          : launch_form<4, true>(a, ctas, cluster, s, parts);
  }
  int grid = sms;
  const long long want = a.bg_count <= kPlanMax ? (bound + kMinUnits - 1) / kMinUnits : a.bg_count;
  if (want < grid) grid = (int)want;
  // whole blocks per warp once a warp has several
  return bound >= (long long)kWholeBlocks * kCWarps * grid ? launch_form<1, false>(a, grid, 1, s, parts)
                                                           : launch_form<4, false>(a, grid, 1, s, parts);
}

}  // namespace sparda
