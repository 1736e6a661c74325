// The decode attention over the 4-bit cache on the fifth-generation tensor cores, for ranges of many
// blocks. (kv4_attn.cu has the form for few blocks, on warp-level MMAs.)
//
// Why: there, the products and the unpacking share the register file's ports, and one step of 16 tokens
// takes as long as both together (about 560 cycles of an SM's quarter; 147 us for batch 16 at 131072
// tokens, where the cache alone takes 99). Here the unpacked operands go to tensor memory, and the
// products run beside the unpacking without touching registers.
//
// A tile is 128 tokens, two blocks of one (sequence, group):
//   S^T [128 tokens x 16 heads]   = K [128 x 128, tensor memory] . Q^T [shared memory]      (bf16)
//   O^T [128 channels x 16 heads] += V^T [128 x 128 tokens, tensor memory] . P^T [shared]   (fp16)
// so the cache is the operand with 128 rows and no row is wasted on padding heads. tcgen05.st's
// 16x128b form writes the same register fragments that a warp-level MMA would take: lane (g, cq) of a
// warp holds token g (or channel octet g) and channel pairs (or token pairs) of cq, and the columns'
// order within a contraction is free as long as both operands agree.
//
// Roles: warps 0-3 unpack keys and do the softmax (a thread has a token: its 16 scores are one tensor
// memory load, and the sums need no shuffles until the end), warps 4-7 unpack values, warp 8 feeds the
// ring of blocks, one thread of warp 9 issues the products. K, V, S and P are double-buffered, and the
// keys of tile i+1 are unpacked before the softmax of tile i, so the tensor cores always have the next
// product's operands under way. O stays in tensor memory for a whole piece.
//
// The softmax reference of a head is common to the CTA and moves only when a score exceeds it by more
// than 2^8 (a barrier with a vote per tile); then O is rescaled in tensor memory, behind the products
// issued so far.
#include "kv4_attn.cuh"
#include "tc05.cuh"

namespace sparda {
using namespace kv4;

namespace {

constexpr int kThreadsTc = 320;
constexpr int kRingTc = 16;
// shared memory, from a 1024-byte boundary
constexpr int kTcPlan = 1024;                                // prefix sums
constexpr int kTcQ = 6144;                                   // Q: 16 heads x 128 channels, two halves of 64
constexpr int kTcP = kTcQ + 4096;                            // P: two buffers of 16 heads x 128 tokens
constexpr int kTcRed = kTcP + 2 * 4096;                      // reductions over the four warps
constexpr int kTcOut = kTcRed + 1024;                        // O [16 heads][136]
constexpr int kOutRow = 136;                                 // channel c at c + c / 16: no bank conflicts
constexpr int kTcRing = kTcOut + kHeads * kOutRow * 4 + 256; // 28160
constexpr int kSmemTc = 1024 + kTcRing + kRingTc * kBlockBytes4;
static_assert(kTcPlan + (kPlanMax + 1) * 4 <= kTcQ && kTcRing % 128 == 0 && kSmemTc <= 232448, "shared memory");
// tensor memory columns
constexpr int kColK = 0, kColV = 128, kColS = 256, kColO = 288, kCols = 512;
constexpr uint32_t kIdQk = tc05::idesc_bf16(128, 16, 0, 0);
constexpr uint32_t kIdPv = (1u << 4) | ((16u >> 3) << 17) | ((128u >> 4) << 24);   // the same with fp16 operands
constexpr int kEmptyArrivals = 2 + 4;                        // warps that read a block: two for keys, four for values

__device__ __forceinline__ void sync_softmax() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// Whether any of the 128 softmax threads says so.
__device__ __forceinline__ bool any_softmax(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// 16 rows x 64 (32) columns from register fragments: r[2i] is row lane/4, r[2i+1] row lane/4 + 8 of
// column 4i + lane%4.
__device__ __forceinline__ void st_fragments(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void st_fragments(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 columns of the thread's lane.
__device__ __forceinline__ void ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
  tc05::wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    asm volatile("" : "+r"(r[i]));               // not before the wait
    v[i] = __uint_as_float(r[i]);
  }
}

__device__ __forceinline__ void sts16(uint32_t p, uint16_t x) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(p), "h"(x) : "memory");
}

struct Bars {
  uint64_t full[kRingTc], empty[kRingTc];
  uint64_t kready[2], sready[2], vready[2], pready[2], pvdone[2];
  int live[kRingTc];               // tokens of the staged block that exist
  uint32_t masks[3];
  uint32_t tmem;
  int last;
};
static_assert(sizeof(Bars) <= 1024, "header");

}  // namespace

__global__ void __launch_bounds__(kThreadsTc, 1) kv4_attn_tc_kernel(const Kv4AttnArgs a) {
  extern __shared__ uint8_t smem_raw_tc[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw_tc) + 1023) & ~static_cast<uintptr_t>(1023));
  Bars& bar = *reinterpret_cast<Bars*>(smem);
  const uint32_t at = smem_addr(smem), ring_at = at + kTcRing, live_at = smem_addr(bar.live);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kRingTc; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], kEmptyArrivals);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.kready[i], 4);
      mbar_init(&bar.sready[i], 1);
      mbar_init(&bar.vready[i], 4);
      mbar_init(&bar.pready[i], 4);
      mbar_init(&bar.pvdone[i], 1);
    }
    fence_mbar_init();
    const Masks m;
    bar.masks[0] = m.key;
    bar.masks[1] = m.lo;
    bar.masks[2] = m.hi;
  }
  grid_dep_wait();
  grid_dep_launch();
  const Plan plan = make_plan(a, reinterpret_cast<int*>(smem + kTcPlan));
  if ((int)blockIdx.x >= plan.ctas) return;
  if (warp == 9) {
    tc05::alloc(&bar.tmem, kCols);
    tc05::relinquish();
  }
  tc05::fence_before();
  __syncthreads();
  tc05::fence_after();
  const uint32_t tmem = bar.tmem;
  const uint32_t masks_at = smem_addr(bar.masks);
  const Masks mk{lds32(masks_at), lds32(masks_at + 4), lds32(masks_at + 8)};
  int u = plan.u0, bg = plan.u0 < plan.u1 ? plan.group_of(plan.u0) : 0;
  Piece p;
  // A wait that runs out sets the device error word; its warp then waits no more but takes every step,
  // so that all barriers stay matched.
  bool ok = true;
  const auto wait = [&](uint64_t* b, uint32_t parity) {
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(b, parity, a.err));
  };
  const int g = lane >> 2, cq = lane & 3;
  int unit = 0, tc = 0;                        // the CTA's units and tiles so far

  if (warp == 8) {
    // ------------------------------------------------------------ blocks into the ring
    // lane l fills stage l with the CTA's units l, l + kRingTc, ...
    if (lane < kRingTc) {
      int mine = plan.u0 + lane, n_bg = bg;
      uint32_t round = 0, polls = 0;
      const uint8_t* src = nullptr;
      int live = 0;
      const auto look_up = [&]() -> bool {
        if (mine >= plan.u1) return false;
        while (plan.pre[n_bg + 1] <= mine) ++n_bg;
        const int s = mine - plan.pre[n_bg], T = a.seq_len[n_bg / a.G];
        int j = a.idx ? a.idx[(size_t)n_bg * a.kslots + s] : s;
        if ((unsigned)j > (unsigned)((T - 1) / kBlock)) {
          atomicOr(a.err, SPARDA_DEV_BAD_INDEX);   // skipped: block 0 is staged with no live token
          j = 0;
          live = 0;
        } else {
          live = min(kBlock, T - j * kBlock);
        }
        src = a.kv + ((size_t)n_bg * a.nb_cap + j) * kBlockBytes4;
        mine += kRingTc;
        return true;
      };
      bool more = look_up();
      while (more) {
        if (round == 0 || mbar_test_wait(&bar.empty[lane], (round & 1) ^ 1)) {
          bar.live[lane] = live;
          mbar_arrive_expect_tx(&bar.full[lane], kBlockBytes4);
          bulk_load(smem + kTcRing + lane * kBlockBytes4, src, kBlockBytes4, &bar.full[lane]);
          ++round;
          polls = 0;
          more = look_up();
        } else if (++polls > kProducerPolls) {
          atomicOr(a.err, SPARDA_DEV_WAIT_TIMEOUT);
          more = false;
        }
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ the products
    const uint32_t q_at = at + kTcQ;
    const auto issue_qk = [&](int t) {
      wait(&bar.kready[t & 1], (t >> 1) & 1);
      tc05::fence_after();
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          tc05::mma_bf16_ts(tmem + kColS + 16 * (t & 1), tmem + kColK + 64 * (t & 1) + 8 * k,
                            tc05::smem_desc(q_at + (k >> 2) * 2048 + (k & 3) * 32, 16, 1024), kIdQk, k > 0);
        tc05::commit(&bar.sready[t & 1]);
      }
      __syncwarp();
    };
    while (plan.next(p, u, bg)) {
      const int tiles = (p.s1 - p.s0 + 1) / 2;
      issue_qk(tc);
      for (int i = 0; i < tiles; ++i, ++tc) {
        if (i + 1 < tiles) issue_qk(tc + 1);
        wait(&bar.vready[tc & 1], (tc >> 1) & 1);
        wait(&bar.pready[tc & 1], (tc >> 1) & 1);
        tc05::fence_after();
        if (lane == 0) {
          const uint32_t p_at = at + kTcP + 4096 * (tc & 1);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc05::mma_bf16_ts(tmem + kColO, tmem + kColV + 64 * (tc & 1) + 8 * k,
                              tc05::smem_desc(p_at + (k >> 2) * 2048 + (k & 3) * 32, 16, 1024), kIdPv, i > 0 || k > 0);
          tc05::commit(&bar.pvdone[tc & 1]);
        }
        __syncwarp();
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ values
    // warp w owns the tensor memory lanes 32 w ..: channels n and n + 8 of every octet for n = 2 w, 2 w + 1,
    // which lie in words w / 2 and w / 2 + 2
    const int w = warp - 4;
    while (plan.next(p, u, bg)) {
      const int n = p.s1 - p.s0;
      for (int i = 0; i < n; i += 2, ++tc) {
        if (tc >= 2) wait(&bar.pvdone[tc & 1], ((tc - 2) >> 1) & 1);   // this buffer's last products
        tc05::fence_after();
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {
          const uint32_t col = tmem + kColV + 64 * (tc & 1) + 32 * b;
          uint32_t r0[16], r1[16];
          if (i + b < n) {
            const int stage = (unit + i + b) % kRingTc;
            wait(&bar.full[stage], ((unit + i + b) / kRingTc) & 1);
            const uint32_t blk = ring_at + stage * kBlockBytes4;
            const int live = (int)lds32(live_at + 4 * stage);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              const uint2 v = lds64(blk + kVCodes + r * 512 + (w >> 1) * 256 + lane * 8);
              uint2 z = lds64(blk + kVScales + (r * 4 + cq) * 32 + (g >> 1) * 8);
              if (live < kBlock) {             // tokens that do not exist hold anything: their values become 0
                const uint32_t keep = (8 * r + 2 * cq < live ? 0xffffu : 0u) | (8 * r + 2 * cq + 1 < live ? 0xffff0000u : 0u);
                z.x &= keep;
                z.y &= keep;
              }
              const uint32_t x = ror(v.x, 8 * (w & 1)), y = ror(v.y, 8 * (w & 1));
              r0[2 * r] = value_pair(x, 0, z.x, z.y, mk);
              r0[2 * r + 1] = value_pair(y, 0, z.x, z.y, mk);
              r1[2 * r] = value_pair(x, 1, z.x, z.y, mk);
              r1[2 * r + 1] = value_pair(y, 1, z.x, z.y, mk);
            }
            __syncwarp();
            if (lane == 0) arrive(&bar.empty[stage]);
          } else {
#pragma unroll
            for (int r = 0; r < 16; ++r) r0[r] = r1[r] = 0u;
          }
          st_fragments(tc05::taddr_at(col, 32 * w, 0), r0);
          st_fragments(tc05::taddr_at(col, 32 * w + 16, 0), r1);
        }
        tc05::wait_st();
        tc05::fence_before();
        __syncwarp();
        if (lane == 0) arrive(&bar.vready[tc & 1]);
      }
      unit += n;
    }
  } else {
    // ------------------------------------------------------------ keys and the softmax
    float* s_max = reinterpret_cast<float*>(smem + kTcRed);    // [4 warps][16 heads]
    float* s_sum = s_max + 64;                                 // [4][16]
    float* s_m = s_sum + 64;                                   // [16]
    float* s_l = s_m + 16;                                     // [16]
    float* s_o = reinterpret_cast<float*>(smem + kTcOut);
    const uint32_t lanes = (uint32_t)(32 * warp);
    const int token = tid, half = token >> 6;                  // of the tile
    bool first_piece = true;
    while (plan.next(p, u, bg)) {
      const int n = p.s1 - p.s0, tiles = (n + 1) / 2;
      // Q, with the contraction's order of the key fragments: position 8 r + 2 cq + e is channel 32 cq + 2 r + e
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = (tid >> 4) + 8 * i, r = tid & 15;
        const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q + ((size_t)p.bg * a.H + h) * kHeadDim);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (h < a.H) x = make_uint4(q[r], q[16 + r], q[32 + r], q[48 + r]);
        *reinterpret_cast<uint4*>(smem + kTcQ + (r >> 3) * 2048 + h * 128 + (((r & 7) ^ (h & 7)) << 4)) = x;
      }
      fence_proxy_async_shared();
      sync_softmax();
      float m[16], l[16];
#pragma unroll
      for (int h = 0; h < 16; ++h) {
        m[h] = kLowest;
        l[h] = 0.f;
      }
      // Keys of the piece's tile i (tile t of the CTA) to tensor memory; whether this thread's token exists.
      const auto keys = [&](int i, int t) -> bool {
        const int ui = 2 * i + (warp >> 1);                    // this warp's block of the piece
        bool exists = false;
        if (ui < n) {
          const int stage = (unit + ui) % kRingTc;
          wait(&bar.full[stage], ((unit + ui) / kRingTc) & 1);
          const uint32_t blk = ring_at + stage * kBlockBytes4;
          exists = (token & 63) < (int)lds32(live_at + 4 * stage);
#pragma unroll 1
          for (int j = 0; j < 2; ++j) {
            const int r = (warp & 1) * 4 + 2 * j;              // 8-token tiles r and r + 1 of the block
            uint32_t out[32];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint4 kw = lds128(blk + kKCodes + (r + e) * 512 + lane * 16);
              const uint32_t sz = lds32(blk + kKScales + (r + e) * 128 + lane * 4);
              const uint32_t s2 = dup_lo(sz), z2 = dup_hi(sz);
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t word = w == 0 ? kw.x : w == 1 ? kw.y : w == 2 ? kw.z : kw.w;
#pragma unroll
                for (int c = 0; c < 4; ++c) out[2 * (4 * w + c) + e] = key_pair(word, c, s2, z2, mk);
              }
            }
            st_fragments(tc05::taddr_at(tmem + kColK + 64 * (t & 1), lanes + 16 * j, 0), out);
          }
          __syncwarp();
          if (lane == 0) arrive(&bar.empty[stage]);
          tc05::wait_st();
        }
        tc05::fence_before();
        __syncwarp();
        if (lane == 0) arrive(&bar.kready[t & 1]);
        return exists;
      };
      bool exists = keys(0, tc);
      for (int i = 0; i < tiles; ++i, ++tc) {
        const bool next_exists = i + 1 < tiles ? keys(i + 1, tc + 1) : false;
        wait(&bar.sready[tc & 1], (tc >> 1) & 1);
        tc05::fence_after();
        float s[16];
        ld16(tc05::taddr_at(tmem + kColS + 16 * (tc & 1), lanes, 0), s);
        bool rise = false;
#pragma unroll
        for (int h = 0; h < 16; ++h) {
          if (!exists) s[h] = kNegInf;
          rise = rise || s[h] - m[h] > kRise / kScale2;
        }
        if (any_softmax(rise)) {
          // the references of all heads move to the largest score so far
#pragma unroll
          for (int h = 0; h < 16; ++h) {
            float x = s[h];
#pragma unroll
            for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            if (lane == 0) s_max[warp * 16 + h] = x;
          }
          sync_softmax();
          float al[16];
#pragma unroll
          for (int h = 0; h < 16; ++h) {
            const float top = fmaxf(m[h], fmaxf(fmaxf(s_max[h], s_max[16 + h]), fmaxf(s_max[32 + h], s_max[48 + h])));
            al[h] = fast_exp2((m[h] - top) * kScale2);
            m[h] = top;
            l[h] *= al[h];
          }
          if (i > 0) {
            wait(&bar.pvdone[(tc - 1) & 1], ((tc - 1) >> 1) & 1);
            tc05::fence_after();
            float o[16];
            ld16(tc05::taddr_at(tmem + kColO, lanes, 0), o);
            uint32_t r[16];
#pragma unroll
            for (int h = 0; h < 16; ++h) r[h] = __float_as_uint(o[h] * al[h]);
            tc05::st16(tc05::taddr_at(tmem + kColO, lanes, 0), r);
            tc05::wait_st();
          }
          sync_softmax();                          // s_max may be written again
        }
        if (tc >= 2) wait(&bar.pvdone[tc & 1], ((tc - 2) >> 1) & 1);   // this P buffer's last products
        const uint32_t p_at = at + kTcP + 4096 * (tc & 1) + half * 2048 + (token & 7) * 2;
        const uint32_t chunk = (uint32_t)((token & 63) >> 3);
#pragma unroll
        for (int h = 0; h < 16; ++h) {
          const float w = fast_exp2(fmaf(s[h] - m[h], kScale2, kPShift));
          l[h] += w;
          sts16(p_at + h * 128 + ((chunk ^ (h & 7)) << 4), __half_as_ushort(__float2half_rn(w)));
        }
        fence_proxy_async_shared();
        tc05::fence_before();
        __syncwarp();
        if (lane == 0) arrive(&bar.pready[tc & 1]);
        exists = next_exists;
      }
      unit += n;

      // ---------------------------------------------------------- the piece's result
      wait(&bar.pvdone[(tc - 1) & 1], ((tc - 1) >> 1) & 1);
      tc05::fence_after();
      float o[16];
      ld16(tc05::taddr_at(tmem + kColO, lanes, 0), o);
      tc05::fence_before();
      // lane 16 n + 8 b + g of tensor memory: channel 16 g + n + 8 b
      const int channel = 16 * (tid & 7) + (tid >> 4) + (tid & 8);
#pragma unroll
      for (int h = 0; h < 16; ++h) {
        s_o[h * kOutRow + channel + (channel >> 4)] = o[h];
        float x = l[h];
#pragma unroll
        for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        if (lane == 0) s_sum[warp * 16 + h] = x;
      }
      if (tid == 0) {
#pragma unroll
        for (int h = 0; h < 16; ++h) s_m[h] = m[h] * kScale2;
      }
      sync_softmax();
      if (tid < 16) s_l[tid] = (s_sum[tid] + s_sum[16 + tid]) + (s_sum[32 + tid] + s_sum[48 + tid]);
      sync_softmax();
      // thread: head h, channels 16 part ..
      const int h = tid >> 3, part = tid & 7;
      float M = s_m[h], L = s_l[h], acc[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[e] = s_o[h * kOutRow + 17 * part + e];
      bool write = true;
      if (p.n_cta > 1) {
        const int place = plan.own_place(blockIdx.x, first_piece);
        float4* po = reinterpret_cast<float4*>(a.part_o + ((size_t)place * kHeads + h) * kHeadDim + 16 * part);
#pragma unroll
        for (int e = 0; e < 4; ++e) po[e] = make_float4(acc[4 * e], acc[4 * e + 1], acc[4 * e + 2], acc[4 * e + 3]);
        if (part == 0) {
          a.part_ml[place * 2 * kHeads + h] = M;
          a.part_ml[place * 2 * kHeads + kHeads + h] = L;
        }
        sync_softmax();                            // every thread's stores are issued
        if (tid == 0) {
          unsigned prev;
          asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(prev) : "l"(a.counters + p.bg) : "memory");
          bar.last = prev == (unsigned)(p.n_cta - 1);
          if (bar.last) a.counters[p.bg] = 0u;
        }
        sync_softmax();
        write = *reinterpret_cast<volatile int*>(&bar.last) != 0;
        if (write) {
          // the last CTA of the group to get here joins the partial results
          M = kLowest;
          L = 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[e] = 0.f;
          constexpr int kFlight = 4;
          for (int q0 = 0; q0 < p.n_cta; q0 += kFlight) {
            float pm[kFlight], pl[kFlight];
            float4 px[kFlight][4];
#pragma unroll
            for (int q = 0; q < kFlight; ++q) {
              const bool in = q0 + q < p.n_cta;
              const int pl_at = plan.place_of(p, in ? q0 + q : 0);
              pm[q] = in ? __ldcg(a.part_ml + pl_at * 2 * kHeads + h) : kLowest;
              pl[q] = __ldcg(a.part_ml + pl_at * 2 * kHeads + kHeads + h);
              const float4* src = reinterpret_cast<const float4*>(a.part_o + ((size_t)pl_at * kHeads + h) * kHeadDim + 16 * part);
#pragma unroll
              for (int e = 0; e < 4; ++e) px[q][e] = __ldcg(src + e);
            }
            float top = M;
#pragma unroll
            for (int q = 0; q < kFlight; ++q) top = fmaxf(top, pm[q]);
            const float old = fast_exp2(M - top);
            L *= old;
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e] *= old;
#pragma unroll
            for (int q = 0; q < kFlight; ++q) {
              if (q0 + q >= p.n_cta) continue;
              const float wt = fast_exp2(pm[q] - top);
              L += wt * pl[q];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                acc[4 * e] += wt * px[q][e].x;
                acc[4 * e + 1] += wt * px[q][e].y;
                acc[4 * e + 2] += wt * px[q][e].z;
                acc[4 * e + 3] += wt * px[q][e].w;
              }
            }
            M = top;
          }
        }
      }
      if (write && h < a.H) {
        uint32_t pk[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) pk[e] = L == 0.f ? 0u : pack_bf16(acc[2 * e] / L, acc[2 * e + 1] / L);
        uint4* out = reinterpret_cast<uint4*>(a.out + ((size_t)p.bg * a.H + h) * kHeadDim + 16 * part);
        out[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        out[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
      }
      first_piece = false;
      sync_softmax();                              // s_o and the reductions are free again
    }
    zero_empty_groups(a, plan, tid, 128);
  }
  tc05::fence_before();
  __syncthreads();
  tc05::fence_after();
  if (warp == 9) tc05::dealloc(tmem, kCols);
}

bool launch_kv4_attn_tc(const Kv4AttnArgs& a, int grid, cudaStream_t s) {
  static SmemOptIn opt_in;
  if (!opt_in.set(kv4_attn_tc_kernel, kSmemTc)) return false;
  launch_pdl(kv4_attn_tc_kernel, dim3(grid), dim3(kThreadsTc), kSmemTc, s, a);
  return true;
}

}  // namespace sparda
