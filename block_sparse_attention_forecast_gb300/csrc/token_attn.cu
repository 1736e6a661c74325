// Attention of many new tokens per sequence over a bf16 cache, on the fifth-generation tensor cores:
// packed prompts (causal, on top of what the cache holds) and trees of drafted tokens.
//
// For token i of a sequence and head h of group g, over the keys u it attends (cached tokens, and the new
// tokens up to i, or i's ancestors and itself):
//   out = sum_u p_u v_u / sum_u p_u,   p_u = 2^((q . k_u - m) log2(e) / sqrt(128)),   m a running maximum
//
// A CTA holds the query rows of an item, row (token - first) * H + h of one KV group: two tiles of 128 rows
// that share every key tile (128 keys: two 64-token blocks) it loads, or, where the rows of a sequence's group fit one
// tile, that tile, and two CTAs run on an SM (kSolo). Either keeps two softmaxes and two accumulators under way for
// the one tensor pipe:
//   warp 0, one lane: TMA loads of the query tiles and of each key tile's K and V into a ring of 32 KiB stages;
//   warp 1: tensor-memory allocation; zeroes the value rows past a sequence's end (0 * NaN is NaN) and
//       issues S_t = Q_t K^T (M 128, N 128) and O_t += P_t V, P read from tensor memory, where it
//       overwrites S; one thread's MMAs run in issue order, so S of a tile's next step is issued behind the
//       O that reads the P it overwrites, and the completion of S tells that of that O;
//   warp 2: hands out the segments (token_attn.cuh), through shared memory;
//   warps 4-19 (kSolo: 4-11), two threads per row (each 64 of a key tile's 128 keys): online softmax. The two agree on a
//       reference that only moves, and O is only rescaled, when a score passes it by more than 8 (log2); any
//       reference serves that keeps P in range, since P and its sum are divided by one another. P goes to tensor
//       memory as bf16 (rounded once; the sum is taken before that, in float32), 32 keys of each half at a
//       time, so that their O += P V runs while the others are formed.
// S and P never leave the SM, K and V are read once per item, and nothing is written but the output (or a partial
// result where an item is cut). A long prompt is bound by the tensor pipe and what stands between its MMAs: 32768
// tokens, 32 heads over 2 groups, 5.4 ms, 1.63 PFLOP/s (0.85 of the measured GEMM rate; 4.9 ms with a softmax that
// does nothing). A decode step over 16 x 131072 tokens is bound by memory: 0.317 ms, 6.8 TB/s (1.01 of the measured
// copy rate). What was measured on the way there, for the 32768-token prompt: one thread per row, all S in registers,
// MMAs issued from a divergent branch 11.0 ms; the issuing warp kept together (uniform registers) 7.5; a look
// at each barrier before the suspended wait 6.3; a step's bookkeeping cut to counters 5.65; two threads per row
// 5.65 (and 0.91 of the time for packed prompts); P handed on in two parts 5.4. Slower: two issuing warps (7.2), a
// watcher of the loads for the issuer (6.9), waits that poll (7.0), P formed ahead of the reference (6.4), no
// maximum at all (5.9), S fetched in pieces of 16 keys ahead of their use (5.6).
// Every wait is bounded. A phase of a barrier is only followed by the next one after the thread that
// waits for it has arrived somewhere.
#include <algorithm>

#include "tc05.cuh"
#include "token_attn.cuh"

namespace sparda {

namespace {
using tok::Item;
using tok::Segments;
using tok::u64;

// Two forms: two query tiles per CTA and a CTA per SM, or (kSolo) one tile per CTA and two CTAs per SM.
template <bool kSolo>
struct Form {
  static constexpr int kTiles = kSolo ? 1 : 2;
  static constexpr int kSoftmaxWarps = 8 * kTiles;
  static constexpr int kThreads = 128 + 32 * kSoftmaxWarps;
  static constexpr int kPerSm = kSolo ? 2 : 1;
  static constexpr int kStages = kSolo ? 2 : 5;              // of the ring
  // Blocks of the join per CTA: 256 rows of few parts each to 64 warps (16 trees over 34 blocks 27 us, to 16 warps 31);
  // 128 rows at most, and twice the CTAs, to 16 (64 trees over 500 tokens 41 us, to 64 warps 43).
  static constexpr int kJoinSplit = kSolo ? 2 : 8;
  // registers per thread: the softmax warps take what the first warpgroup gives of those at launch
  static constexpr int kRegsLaunch = kSolo ? 80 : 96, kRegsMain = 64, kRegsSoftmax = kSolo ? 88 : 104;
  static constexpr uint32_t kCols = 256 * kTiles;            // tensor memory: per tile 128 columns of S (then P), 128 of O
  static_assert(128 * kRegsMain + 32 * kSoftmaxWarps * kRegsSoftmax <= kThreads * kRegsLaunch, "the registers of the launch");
};
constexpr int kTileRows = 128;
constexpr int kQTile = kTileRows * kRowBytes;              // 32 KiB: columns 0..63 of 128 rows, then 64..127
constexpr int kStage = 2 * kBlockBytes;                    // 32 KiB: the same of 128 keys or values
constexpr int kHalfCols = kStage / 2;
constexpr int kPage = 1024;                                // barriers
constexpr float kGrow = 8.f;                               // the reference moves when a score passes it by this (log2)
constexpr float kScaleLog2 = 1.4426950408889634f * 0.08838834764831845f;   // log2(e) / sqrt(128)
// The exponent of a probability is one fused operation, score * kScaleLog2 - reference, so it carries the rounding of the
// reference: the same factor for all keys of a row, which the division by the sum takes out while it is in range (2^16 at
// most below 2^29; twice the exponent with every bit more). Beyond, float32 scores are equal or 2^8 and more apart (2^32 as
// probabilities), and any scale tells which: a power of two, with which products and references are exact. This one
// keeps the references in the order of the scores. (8 packed prompts 583 us, with one scale for all rows 575; the scale chosen
// again in every step 581, and the 32768-token prompt 1 % slower; far rows in a loop of their own 613.)
constexpr float kFar = 536870912.f, kScaleFar = 0.25f;
__device__ __forceinline__ float reference(float score) {
  const float r = __fmul_rn(score, kScaleLog2);
  return fabsf(r) < kFar ? r : score * kScaleFar;
}

// [barriers][query tiles][ring][two floats per row]
template <bool kSolo>
constexpr int smem_bytes() {
  return kPage + Form<kSolo>::kTiles * (kQTile + 8 * kTileRows) + Form<kSolo>::kStages * kStage;
}
static_assert(smem_bytes<false>() <= 227 * 1024 && 2 * (smem_bytes<true>() + 1024) <= 228 * 1024,
              "the token attention fits shared memory");

__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, int v,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// two float32 operations in one instruction
__device__ __forceinline__ u64 pack2(float lo, float hi) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(u64 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 32 bytes of global memory (32-byte aligned) in one store: a whole sector, where each thread writes a row of its own
__device__ __forceinline__ void store32(void* dst, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// A segment as the scheduling warp hands it to the other warps, through a ring in shared memory.
struct Work {
  int b, g, n, P, nctx, row0, tok0, nblk, k0, k1, slot, tiles;   // k0 == k1: no more
};
constexpr int kWorkRing = 1;   // an item is taken when all warps have begun the one before, not earlier

// The blocks of an item. Block s < nctx is a block of the cache, the others are blocks of the new tokens.
struct Blocks {
  int j0, j1;        // lane l: the selection's entries l and 32 + l (selected blocks)
  bool sel;
  __device__ __forceinline__ int rows_of(const Work& it, int j) const {
    return j < 0 || j > it.P / kBlock ? 0 : min(kBlock, it.P - j * kBlock);
  }
  __device__ __forceinline__ void load(const TokenAttnArgs& a, const Work& it, int lane) {
    sel = a.idx != nullptr;
    if (sel) {
      const int32_t* p = a.idx + (size_t)(it.b * a.G + it.g) * a.kslots;
      j0 = lane < it.nctx ? p[lane] : 0;
      j1 = lane + 32 < it.nctx ? p[lane + 32] : 0;
    }
  }
  // the cache's block number (every lane calls); -1: outside the sequence
  __device__ __forceinline__ int block(const Work& it, int s) const {
    if (!sel) return s;
    const int j = __shfl_sync(0xffffffffu, s < 32 ? j0 : j1, s & 31);
    return j >= 0 && j <= it.P / kBlock ? j : -1;
  }
  // rows of block s that hold tokens: 0 .. 64 (every lane calls)
  __device__ __forceinline__ int rows(const Work& it, int s) const {
    return s >= it.nctx ? min(kBlock, it.n - (s - it.nctx) * kBlock) : rows_of(it, block(it, s));
  }
};

// The bounded wait of a whole warp: true in every lane or in none, and the warp is converged behind it. One look
// first: a phase that is complete costs no suspended wait (32768-token prompt 7.5 -> 6.3 ms; more looks, 7.0).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* err) {
  if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
  const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, err));
  __syncwarp();
  return ok;
}

// The two warps that share rows: a barrier of their own, and one that tells whether any of their threads says so.
__device__ __forceinline__ void pair_sync(int id) {
  __syncwarp();
  asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool pair_any(int id, bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}

// 64-bit mask of the first n keys, 0 <= n <= 64
__device__ __forceinline__ u64 first_bits(int n) { return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1ull); }

}  // namespace

template <bool kSolo>
__global__ void __launch_bounds__(Form<kSolo>::kThreads, Form<kSolo>::kPerSm) token_attn_kernel(const TokenAttnArgs a, const __grid_constant__ CUtensorMap mq,
                                                                const __grid_constant__ CUtensorMap mkc,
                                                                const __grid_constant__ CUtensorMap mvc,
                                                                const __grid_constant__ CUtensorMap mkn,
                                                                const __grid_constant__ CUtensorMap mvn) {
  using F = Form<kSolo>;
  constexpr int kTiles = F::kTiles, kSoftmaxWarps = F::kSoftmaxWarps, kThreads = F::kThreads, kStages = F::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* q_empty = q_full + 1;
  uint64_t* drain = q_empty + 1;
  uint64_t* kv_full = drain + 1;                             // [stages]
  uint64_t* kv_empty = kv_full + kStages;                    // [stages]
  uint64_t* s_full = kv_empty + kStages;                     // [tile]
  uint64_t* p_full = s_full + 2;                             // [tile][32 keys of each half]
  uint64_t* o_full = p_full + 4;                             // [tile]
  uint64_t* w_full = o_full + 2;                             // [work ring]
  uint64_t* w_empty = w_full + kWorkRing;
  uint32_t* tmem_sh = reinterpret_cast<uint32_t*>(w_empty + kWorkRing);
  volatile uint32_t* fail_sh = tmem_sh + 1;                  // [row pairs]: a wait of one of the two warps ran out
  volatile Work* work = reinterpret_cast<volatile Work*>(smem + 512);
  uint8_t* qs = smem + kPage;
  uint8_t* ring = qs + kTiles * kQTile;
  float* row_sh = reinterpret_cast<float*>(ring + kStages * kStage);  // [tile][2][128]: between a row's two threads

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = a.H, tp = a.tp, tpi = kTiles * tp;
  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(drain, 1);
    for (int i = 0; i < kSoftmaxWarps / 2; ++i) fail_sh[i] = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int t = 0; t < kTiles; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[2 * t], 8);
      mbar_init(&p_full[2 * t + 1], 8);
      mbar_init(&o_full[t], 1);
    }
    for (int i = 0; i < kWorkRing; ++i) {
      mbar_init(&w_full[i], 1);
      mbar_init(&w_empty[i], 2 + kSoftmaxWarps);             // producer, issuer, softmax warps
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tc05::alloc(tmem_sh, F::kCols);
    tc05::relinquish();
  }
  grid_dep_wait();
  grid_dep_launch();                                         // (only now: what runs next may not wait for the launch before)
  Segments seg(a, tpi, lane, blockIdx.x);
  if (warp == 2) seg.init(blockIdx.x == 0);
  // query rows that no load fills: zero, once
  for (int i = tid; i < (kTileRows - tp * H) * 8; i += kThreads)
#pragma unroll
    for (int part = 0; part < 2 * kTiles; ++part)
      *reinterpret_cast<uint4*>(qs + part * (kQTile / 2) + tp * H * 128 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_shared();
  tc05::fence_before();
  __syncthreads();
  tc05::fence_after();
  const uint32_t tmem = *tmem_sh;
  bool ok = true;
  unsigned n_work = 0;
  Work it;
  Blocks bl;
  // the next segment; false: none is left
  auto next = [&]() {
    const int i = n_work % kWorkRing;
    ok = warp_wait(&w_full[i], (n_work / kWorkRing) & 1, a.err);
    if (!ok) return false;
    it.b = work[i].b;
    it.g = work[i].g;
    it.n = work[i].n;
    it.P = work[i].P;
    it.nctx = work[i].nctx;
    it.row0 = work[i].row0;
    it.tok0 = work[i].tok0;
    it.nblk = work[i].nblk;
    it.k0 = work[i].k0;
    it.k1 = work[i].k1;
    it.slot = work[i].slot;
    it.tiles = work[i].tiles;
    __syncwarp();
    if (lane == 0) bar_arrive(&w_empty[i]);
    ++n_work;
    if (it.k0 == it.k1) return false;
    bl.load(a, it, lane);
    return true;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(F::kRegsMain));
  if (warp == 2) {
    // ------------------------------------------------------------ scheduler
    Item im;
    int n_join = 0;
    for (bool more = true; more;) {                          // (to the end, though a wait ran out: see take())
      more = seg.next(im);
      const int i = n_work % kWorkRing;
      if (ok && n_work >= (unsigned)kWorkRing) ok = warp_wait(&w_empty[i], ((n_work / kWorkRing) & 1) ^ 1, a.err);
      if (ok && lane == 0) {
        if (more) {
          const int b = a.by_G.div(im.e);
          work[i].b = b;
          work[i].g = im.e - b * a.G;
          work[i].n = im.en.n;
          work[i].P = im.en.P;
          work[i].nctx = im.en.nctx;
          work[i].row0 = im.en.row0;
          work[i].tok0 = im.tok0;
          work[i].nblk = im.nblk;
          work[i].k0 = im.k0;
          work[i].k1 = im.k1;
          work[i].slot = im.slot;
          work[i].tiles = kSolo || im.tok0 + tp >= im.en.n ? 1 : 2;
        } else {
          work[i].k0 = work[i].k1 = 0;
        }
        bar_arrive(&w_full[i]);
      }
      __syncwarp();
      ++n_work;
      TokenJoin j;
      if (more && seg.join(im, j)) {
        if (lane == 0) a.joins[2 * blockIdx.x + n_join] = j;
        ++n_join;
      }
    }
    if (lane == 0)
      for (; n_join < 2; ++n_join) a.joins[2 * blockIdx.x + n_join] = TokenJoin{};
  } else if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      prefetch_tensormap(&mq);
      prefetch_tensormap(&mkn);
      prefetch_tensormap(&mvn);
      if (a.ctx_len) {
        prefetch_tensormap(&mkc);
        prefetch_tensormap(&mvc);
      }
    }
    unsigned n_ld = 0, n_item = 0;
    auto load = [&](const CUtensorMap* mc, const CUtensorMap* mn, int p) {
      const int s0 = 2 * p, two = s0 + 1 < it.nblk ? 2 : 1;
      int j[2];
      for (int h = 0; h < two; ++h) j[h] = s0 + h < it.nctx ? bl.block(it, s0 + h) : 0;
      const int stage = n_ld % kStages;
      if (lane == 0) {
        if (n_ld >= (unsigned)kStages) ok = mbar_wait(&kv_empty[stage], ((n_ld / kStages) & 1) ^ 1, a.err);
        if (ok) {
          uint8_t* dst = ring + stage * kStage;
          uint64_t* bar = &kv_full[stage];
          mbar_arrive_expect_tx(bar, two * kBlockBytes);
          for (int h = 0; h < two; ++h) {
            uint8_t* d = dst + h * (kBlockBytes / 2);
            if (s0 + h < it.nctx) {
              if (j[h] < 0) atomicOr(a.err, SPARDA_DEV_BAD_INDEX);
              const int rr = (it.b * a.G + it.g) * a.max_ctx + max(j[h], 0) * kBlock;
              tma_load_2d(d, mc, 0, rr, bar);
              tma_load_2d(d + kHalfCols, mc, 64, rr, bar);
            } else {
              const int t0 = it.row0 + (s0 + h - it.nctx) * kBlock, bb = a.cu ? 0 : it.b;
              tma_load_4d(d, mn, 0, it.g, t0, bb, bar);
              tma_load_4d(d + kHalfCols, mn, 64, it.g, t0, bb, bar);
            }
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (ok) ++n_ld;
    };
    while (ok && next()) {
      if (lane == 0) {
        if (n_item > 0) ok = mbar_wait(q_empty, (n_item - 1) & 1, a.err);
        if (ok) {
          mbar_arrive_expect_tx(q_full, it.tiles * tp * H * kRowBytes);
          for (int t = 0; t < it.tiles; ++t) {
            uint8_t* d = qs + t * kQTile;
            const int t0 = it.row0 + it.tok0 + t * tp, bb = a.cu ? 0 : it.b;
            tma_load_5d(d, &mq, 0, 0, it.g, t0, bb, q_full);
            tma_load_5d(d + kQTile / 2, &mq, 64, 0, it.g, t0, bb, q_full);
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      ++n_item;
      const int n = it.k1 - it.k0;
      for (int p = 0; ok && p < n; ++p) {
        load(&mkc, &mkn, it.k0 + p);
        if (ok) load(&mvc, &mvn, it.k0 + p);
      }
    }
    // a wait ran out: no copy may still be under way when the CTA ends
    if (!ok && lane == 0)
      for (unsigned i = n_ld > (unsigned)kStages ? n_ld - kStages : 0; i < n_ld; ++i)
        mbar_wait(&kv_full[i % kStages], (i / kStages) & 1, a.err);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp stays together (uniform arithmetic), one lane issues. What stands between two MMAs is the
    // tensor pipe's idle time, so a step's bookkeeping is a few counters: the ring is read in the order of loading.
    constexpr uint32_t id_qk = tc05::idesc_bf16(128, 128, 0, 0);
    constexpr uint32_t id_pv = tc05::idesc_bf16(128, 128, 0, 1);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), qs_at = __shfl_sync(0xffffffffu, smem_addr(qs), 0);
    const uint32_t ring_at = __shfl_sync(0xffffffffu, smem_addr(ring), 0);
    const u64 dq = tc05::smem_desc(qs_at, 16, 1024);
    const u64 dk = tc05::smem_desc(ring_at, 16, 1024);
    const u64 dv = tc05::smem_desc(ring_at, kHalfCols, 1024);
    const uint32_t leader = tc05::elect_leader();
    unsigned stage = 0, full_parity = 0, q_parity = 0, p_parity = 0;   // (p_parity: bit t)
    // the next load of the ring, once it is there
    auto take = [&]() {
      const unsigned at = stage;
      ok = ok && warp_wait(&kv_full[at], full_parity, a.err);
      if (++stage == kStages) {
        stage = 0;
        full_parity ^= 1;
      }
      tc05::fence_after();
      return at;
    };
    auto issue_qk = [&](int t, unsigned at) {                // S_t = Q_t K^T
      const u64 da = dq + t * (kQTile >> 4), db = dk + at * (kStage >> 4);
      const uint32_t d = tm + 256 * t;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint32_t off = (kk >> 2) * (kHalfCols >> 4) + (kk & 3) * 2;
        tc05::mma_bf16_ss_by(leader, d, da + off, db + off, id_qk, kk > 0 ? 1u : 0u);
      }
      tc05::commit_by(leader, &s_full[t]);
    };
    auto issue_pv = [&](int t, unsigned at, bool first, bool two) {   // O_t += P_t V
      u64 db = dv + at * (kStage >> 4);
      const uint32_t d = tm + 256 * t + 128;
      uint32_t pa = tm + 256 * t;
      // 32 keys of each half at a time: the products of the first run beside the softmax of the others
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        ok = ok && warp_wait(&p_full[2 * t + c], (p_parity >> t) & 1, a.err);
        if (ok) {
          tc05::fence_after();
#pragma unroll
          for (int i = 0; i < 4; ++i) {                      // P of the second half lies 64 columns behind the first's
            const int kk = 2 * c + (i & 1) + (i < 2 ? 0 : 4);
            if (i < 2 || two)
              tc05::mma_bf16_ts_by(leader, d, pa + 8 * kk + (i < 2 ? 0 : 32), db + kk * 128, id_pv, c > 0 || i > 0 || !first ? 1u : 0u);
          }
        }
      }
      p_parity ^= 1u << t;
    };
    // value rows without a token, of a key tile whose blocks hold rows0 and rows1 tokens: zeroed
    auto clear_rows = [&](unsigned at, int rows0, int rows1) {
      uint8_t* vs = ring + at * kStage;
      for (int h = 0; h < 2; ++h)
        for (int e = (h ? rows1 : rows0) * 8 + lane; e < kBlock * 8; e += 32) {
          uint8_t* d = vs + h * (kBlockBytes / 2) + e * 16;
          *reinterpret_cast<uint4*>(d) = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(d + kHalfCols) = make_uint4(0u, 0u, 0u, 0u);
        }
      fence_proxy_async_shared();
      __syncwarp();
    };
    while (ok && next()) {
      const int n = __shfl_sync(0xffffffffu, it.k1 - it.k0, 0), tiles = kSolo ? 1 : __shfl_sync(0xffffffffu, it.tiles, 0);
      // the segment's key tiles with fewer than 128 tokens: all before the last new block's tile are whole, but
      // for the one at the cache's end (and selected blocks)
      const int nblk = __shfl_sync(0xffffffffu, it.nblk, 0), k0 = __shfl_sync(0xffffffffu, it.k0, 0);
      const int ragged0 = bl.sel ? 0 : __shfl_sync(0xffffffffu, it.P % kBlock ? (it.nctx - 1) / 2 : it.nblk, 0) - k0;
      const int ragged1 = __shfl_sync(0xffffffffu, (it.nctx + it.n / kBlock) / 2, 0) - k0;
      ok = warp_wait(q_full, q_parity, a.err);
      q_parity ^= 1;
      unsigned ks = take();
      if (!ok) break;
      issue_qk(0, ks);
      if (!kSolo && tiles == 2) issue_qk(1, ks);
      tc05::commit_by(leader, &kv_empty[ks]);
      if (n == 1) tc05::commit_by(leader, q_empty);
      // per key tile: O += P V (V in stage vs) and S of the next key tile (K in ks), tile by tile
      for (int p = 0; ok && p < n; ++p) {
        const bool two = 2 * (k0 + p) + 1 < nblk;
        const unsigned vs = take();
        if (!ok) break;
        if (p == ragged0 || p >= ragged1 || bl.sel) {
          const int blk = 2 * (k0 + p);
          const int rows0 = bl.rows(it, blk), rows1 = two ? bl.rows(it, blk + 1) : kBlock;
          if (rows0 < kBlock || rows1 < kBlock) clear_rows(vs, rows0, rows1);
        }
        const bool more = p + 1 < n;
        issue_pv(0, vs, p == 0, two);
        if (!ok) break;
        if (kSolo || tiles == 1) tc05::commit_by(leader, &kv_empty[vs]);
        if (more) {
          ks = take();
          if (!ok) break;
          issue_qk(0, ks);
        } else {
          tc05::commit_by(leader, &o_full[0]);
        }
        if (!kSolo && tiles == 2) {
          issue_pv(1, vs, p == 0, two);
          if (!ok) break;
          tc05::commit_by(leader, &kv_empty[vs]);
          if (more)
            issue_qk(1, ks);
          else
            tc05::commit_by(leader, &o_full[1]);
        }
        if (more) tc05::commit_by(leader, &kv_empty[ks]);
        if (p + 2 == n) tc05::commit_by(leader, q_empty);
      }
    }
    if (!ok) {                                               // a wait ran out: let the MMAs under way end
      tc05::commit_by(leader, drain);
      mbar_wait(drain, 0, a.err);
      __syncwarp();
    }
    }
    // every tensor-memory access of this CTA is done before the allocating warp frees it
    asm volatile("bar.sync 15, %0;" ::"n"(kThreads) : "memory");
    if (warp == 1) {
      tc05::fence_after();
      tc05::dealloc(tmem, F::kCols);
    }
  } else {
    // ------------------------------------------------------------ softmax, two threads per row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(F::kRegsSoftmax));
    const int t = kSolo ? 0 : ((warp - 4) >> 2) & 1, h = (warp - 4) >> (kSolo ? 2 : 3);   // tile, half of the key tile
    const int quarter = warp & 3;                            // tensor-memory lanes 32q .. 32q+31
    const int r = quarter * 32 + lane;
    const int rt = a.by_H.div(r);                                 // the row's token in its tile
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t t_s = tmem + 256 * t + lane_off, t_o = t_s + 128;
    const int pair = 1 + 4 * t + quarter;                    // named barrier of the rows' two warps
    // Between the row's two threads: the maximum that moves a reference, and the row's sum. A word each: the reference is
    // read behind the last barrier of a step, and the segment's end may follow at once with no barrier before its sum.
    // (Every word is written behind a barrier that follows its last read: the vote of a later step.)
    float* other = row_sh + 256 * t + r;
    float* row_sum = other + 128;
    bool met = false;                                        // both warps of the rows know that a wait ran out
    unsigned n_s = 0, n_o = 0;
    int tree_b = -1;
    u64 anc0 = 0, anc1 = 0;                                  // tree: this row's ancestors and itself
    while (ok && next()) {
      if (t >= it.tiles) continue;
      const int n = it.k1 - it.k0;
      const int tile_tok = it.tok0 + t * tp;
      const int tok = tile_tok + rt;                         // in the sequence
      if (a.parent && (it.b != tree_b || !kSolo)) {
        // the chain of parents, from a table that the warp holds in registers
        tree_b = it.b;
        int par[4];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int node = 32 * i + lane;
          par[i] = node < it.n ? a.parent[(size_t)it.b * a.n_rows + node] : -1;
          if (par[i] < -1 || par[i] >= node) {
            par[i] = -1;
            bad = true;
          }
        }
        if (bad) atomicOr(a.err, SPARDA_DEV_BAD_INDEX);
        anc0 = anc1 = 0;
        int j = rt < tp && tok < it.n ? tok : -1;
        while (__any_sync(0xffffffffu, j >= 0)) {
          const int src = max(j, 0);
          const int p0 = __shfl_sync(0xffffffffu, par[0], src & 31), p1 = __shfl_sync(0xffffffffu, par[1], src & 31);
          const int p2 = __shfl_sync(0xffffffffu, par[2], src & 31), p3 = __shfl_sync(0xffffffffu, par[3], src & 31);
          if (j >= 0) {
            if (j < 64) anc0 |= 1ull << j;
            else anc1 |= 1ull << (j - 64);
            const int w = j >> 5;
            j = w == 0 ? p0 : (w == 1 ? p1 : (w == 2 ? p2 : p3));
          }
        }
      }
      // key tiles before this one are attended whole by every row of the tile (selected blocks: looked at one by one)
      const int whole = bl.sel ? 0 : (it.P % kBlock ? it.nctx - 1 : it.nctx + (a.parent ? 0 : (tile_tok + 1) / kBlock)) / 2;
      float m_used = -INFINITY, l = 0.f;                     // the reference (log2), the sum
      float scale = kScaleFar;                               // the reference's (that of -inf is far)
      bool any = false;                                      // this tile has had a step
      for (int p = 0; p < n; ++p) {
        const int blk = 2 * (it.k0 + p) + h;
        const bool there = blk < it.nblk;                    // an odd number of blocks: the last tile has one
        u64 see = ~0ull;                                     // the keys of the block that this row attends
        if (it.k0 + p >= whole && there)
          see = blk < it.nctx ? first_bits(bl.rows(it, blk))
                              : a.parent ? (blk == it.nctx ? anc0 : anc1) : first_bits(tok + 1 - (blk - it.nctx) * kBlock);
        const bool masked = __any_sync(0xffffffffu, see != ~0ull);
        ok = warp_wait(&s_full[t], n_s & 1, a.err);
        ++n_s;
        // 32 keys of S, -inf where the row does not attend the key
        float x[32];
        auto load = [&](int c) {
          tc05::ld32(t_s + 64 * h + 32 * c, x);
          tc05::wait_ld();
          if (masked) {
            const uint32_t bits = (uint32_t)(see >> (32 * c));
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = (bits >> e) & 1u ? x[e] : -INFINITY;
          }
        };
        float mb = -INFINITY;
        if (ok && there) {
          tc05::fence_after();
#pragma unroll(kSolo ? 1 : 2)
          for (int c = 0; c < 2; ++c) {
            load(c);
            float m4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) m4[k] = max3(x[k], x[k + 4], x[k + 8]);
#pragma unroll
            for (int e = 12; e < 28; e += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) m4[k] = max3(m4[k], x[e + k], x[e + 4 + k]);
#pragma unroll
            for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], x[28 + k]);
            mb = max3(mb, fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          }
        }
        // does a maximum move (also at the first key a row sees)?
        if (!ok) fail_sh[pair - 1] = 1;
        if (pair_any(pair, mb * scale > m_used + kGrow || !ok)) {
          if (fail_sh[pair - 1]) {                           // in one of the two: both leave
            ok = false;
            met = true;
            break;
          }
          if (h == 1) *other = mb;
          pair_sync(pair);
          if (h == 0) {
            mb = fmaxf(mb, *other);
            *other = mb * scale > m_used + kGrow ? reference(mb) : m_used;
          }
          pair_sync(pair);
          const float mn = *other;
          const float alpha = mn > m_used ? fast_exp2(m_used - mn) : 1.f;
          if (any) {                                         // S is there, so the O before it is
            tc05::fence_after();
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
              tc05::ld32(t_o + 64 * h + 32 * i, x);
              tc05::wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] *= alpha;
              tc05::st32(t_o + 64 * h + 32 * i, x);
            }
          }
          l *= alpha;
          m_used = mn;
          scale = fabsf(mn) < kFar ? kScaleLog2 : kScaleFar;
        }
        any = true;
        if (there) {
          const float neg = m_used == -INFINITY ? 0.f : -m_used;
          const u64 scale2 = pack2(scale, scale), neg2 = pack2(neg, neg);
          u64 sum2[2] = {0ull, 0ull};
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            // P lies over S of this half's first 32 keys, which are read by then
            load(c);
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float p0, p1;
              unpack2(fma2(pack2(x[2 * e], x[2 * e + 1]), scale2, neg2), p0, p1);
              p0 = fast_exp2(p0);
              p1 = fast_exp2(p1);
              sum2[e & 1] = add2(sum2[e & 1], pack2(p0, p1));
              pk[e] = pack_bf16(p0, p1);
            }
            tc05::st16(t_s + 64 * h + 16 * c, pk);
            tc05::wait_st();
            tc05::fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&p_full[2 * t + c]);
          }
          float s0, s1;
          unpack2(add2(sum2[0], sum2[1]), s0, s1);
          l += s0 + s1;
        }
        if (!there) {
          tc05::wait_st();                                   // (O that was rescaled)
          tc05::fence_before();
          __syncwarp();
          if (lane == 0) {
            bar_arrive(&p_full[2 * t]);
            bar_arrive(&p_full[2 * t + 1]);
          }
        }
      }
      if (!ok) break;
      // ---- the segment's end: the row's sum, and O complete
      if (h == 1) *row_sum = l;
      pair_sync(pair);
      if (h == 0) *row_sum = l += *row_sum;
      pair_sync(pair);
      l = *row_sum;
      ok = warp_wait(&o_full[t], n_o & 1, a.err);
      ++n_o;
      if (ok) {
        tc05::fence_after();
        const bool live = rt < tp && tok < it.n;
        const size_t row = a.cu ? (size_t)it.row0 + tok : (size_t)it.b * a.n_rows + tok;
        const float inv = 1.f / l;                           // (every token attends itself; l is 0 if all its scores are -inf: NaN)
        __nv_bfloat16* dst = a.out + ((row * a.G + it.g) * H + (r - rt * H)) * kHeadDim;
        const int prow = t * kTileRows + r;
        float* part = a.part + (size_t)max(it.slot, 0) * kTiles * kTokenPartFloats;
        const int c0 = 2 * h, c1 = c0 + 2;                   // a warp's columns: half of the tile's
#pragma unroll
        for (int c = c0; c < c1; ++c) {
          float o[32];
          __syncwarp();
          tc05::ld32(t_o + 32 * c, o);
          tc05::wait_ld();
          if (live && it.slot < 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = pack_bf16(o[16 * e + 2 * i] * inv, o[16 * e + 2 * i + 1] * inv);
              if (a.wide_out) {
                store32(dst + 32 * c + 16 * e, w);
              } else {
                reinterpret_cast<uint4*>(dst + 32 * c + 16 * e)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4*>(dst + 32 * c + 16 * e)[1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          } else if (live) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              store32(part + prow * kHeadDim + 32 * c + 8 * e, reinterpret_cast<const uint32_t*>(o + 8 * e));
          }
        }
        if (live && it.slot >= 0 && h == 0) {
          float* ml = part + kTiles * kTileRows * kHeadDim;
          ml[prow] = m_used;
          ml[kTiles * kTileRows + prow] = l;
        }
        tc05::fence_before();
      }
    }
    // a warp whose wait ran out outside of a step leaves by way of the barrier that the other one is at, or comes to
    if (!met) {
      if (!ok) fail_sh[pair - 1] = 1;
      pair_any(pair, !ok);
    }
    tc05::fence_before();
    asm volatile("bar.sync 15, %0;" ::"n"(kThreads) : "memory");
  }
}

// Joins the partial results of the items that the key-tile division cut: out = sum_i w_i O_i / sum_i w_i l_i
// with w_i = 2^(m_i - max m). joins[c] holds what CTA c of the attention is to join: its shares of the rows of at most two
// items (the one its range began in and the one it ended in). Form::kJoinSplit blocks take a share together: what
// joining costs is the latency of a few dependent reads, so each thread has as few as may be, and kJoinLoads parts are under
// way at a time (in turn 16 trees over 34 blocks take 29 us, two at a time 27, eight 31: fewer blocks on an SM). A
// block holds 8 rows of 32 column quads at a time or, for items of many parts, one row whose parts are dealt out to the
// 8 warps.
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinLoads = 2;      // parts under way

struct JoinSum {
  float m, l;
  float4 o;
  // mi is -inf where a row attends no key of a part (or every score is a NaN: then li is one too)
  __device__ __forceinline__ void add(float mi, float li, float4 oi) {
    const float mn = fmaxf(m, mi), ref = mn == -INFINITY ? 0.f : mn;
    const float w = fast_exp2(m - ref), wi = mi == -INFINITY ? 1.f : fast_exp2(mi - ref);
    o.x = o.x * w + oi.x * wi;
    o.y = o.y * w + oi.y * wi;
    o.z = o.z * w + oi.z * wi;
    o.w = o.w * w + oi.w * wi;
    l = l * w + li * wi;
    m = mn;
  }
};

template <bool kSolo>
__global__ void __launch_bounds__(kJoinThreads) token_attn_join_kernel(const TokenAttnArgs a) {
  constexpr int kTiles = Form<kSolo>::kTiles, kJoinSplit = Form<kSolo>::kJoinSplit;
  __shared__ float ml_sh[kJoinWarps][2];
  __shared__ float4 o_sh[kJoinWarps][32];
  grid_dep_wait();
  const int tp = a.tp, H = a.H, warp = threadIdx.x >> 5, quad = threadIdx.x & 31, rows = kTiles * kTileRows;
  // the rows of both joins, one after the other
  const int at = blockIdx.x % kJoinSplit;
  const TokenJoin* js = a.joins + 2 * (blockIdx.x / kJoinSplit);
  const TokenJoin j0 = js[0], j1 = js[1];
  const int n0 = j0.r1 - j0.r0, n = n0 + j1.r1 - j1.r0;
  const bool many = max(j0.k, j1.k) > 2 * kJoinWarps;        // the parts of a row to all warps
  const int end = n * (at + 1) / kJoinSplit, step = many ? kJoinWarps : 1;
  for (int r = n * at / kJoinSplit + (many ? 0 : warp); r < end; r += many ? 1 : kJoinWarps) {
    const TokenJoin& j = r < n0 ? j0 : j1;
    const int v = r < n0 ? j0.r0 + r : j1.r0 + r - n0;
    const int tk = a.by_H.div(v), h = v - tk * H;
    const int prow = (tk >= tp ? kTileRows + (tk - tp) * H : tk * H) + h;
    JoinSum s{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int q0 = many ? warp : 0; q0 < j.k; q0 += kJoinLoads * step) {
      float mi[kJoinLoads], li[kJoinLoads];
      float4 oi[kJoinLoads];
#pragma unroll
      for (int i = 0; i < kJoinLoads; ++i) {                 // (the last part again: no branch between the loads)
        const int q = min(q0 + i * step, j.k - 1);
        const float* part = a.part + (size_t)(q == 0 ? j.first_slot : 2 * (j.c1 + q)) * kTiles * kTokenPartFloats;
        mi[i] = part[rows * kHeadDim + prow];
        li[i] = part[rows * (kHeadDim + 1) + prow];
        oi[i] = reinterpret_cast<const float4*>(part + prow * kHeadDim)[quad];
      }
#pragma unroll
      for (int i = 0; i < kJoinLoads; ++i)
        if (q0 + i * step < j.k) s.add(mi[i], li[i], oi[i]);
    }
    if (many) {
      o_sh[warp][quad] = s.o;
      if (quad == 0) {
        ml_sh[warp][0] = s.m;
        ml_sh[warp][1] = s.l;
      }
      __syncthreads();
      if (warp == 0)
        for (int w = 1; w < kJoinWarps; ++w) s.add(ml_sh[w][0], ml_sh[w][1], o_sh[w][quad]);
      __syncthreads();
    }
    if (!many || warp == 0) {
      const float inv = 1.f / s.l;
      uint2* dst = reinterpret_cast<uint2*>(a.out + (((size_t)(j.out_row + tk) * a.G + j.g) * H + h) * kHeadDim);
      dst[quad] = make_uint2(pack_bf16(s.o.x * inv, s.o.y * inv), pack_bf16(s.o.z * inv, s.o.w * inv));
    }
  }
}

template <bool kSolo>
static cudaError_t launch(const TokenAttnArgs& a, const CUtensorMap* m, bool joined, cudaStream_t s) {
  using F = Form<kSolo>;
  static SmemOptIn opt;
  if (!opt.set(token_attn_kernel<kSolo>, smem_bytes<kSolo>())) return cudaErrorInvalidValue;
  const cudaError_t e = launch_pdl(token_attn_kernel<kSolo>, dim3(a.n_ctas), dim3(F::kThreads), smem_bytes<kSolo>(), s, a, m[0], m[1],
                             m[2], m[3], m[4]);
  if (e != cudaSuccess || !joined) return e;
  return launch_pdl(token_attn_join_kernel<kSolo>, dim3(a.n_ctas * F::kJoinSplit), dim3(kJoinThreads), 0, s, a);
}

cudaError_t launch_token_attn(const TokenAttnArgs& args, const CUtensorMap* maps, cudaStream_t s) {
  TokenAttnArgs a = args;
  // One tile per CTA where the rows of a sequence's group fit it (of packed prompts, whose lengths only the device knows, the
  // average): 64 trees of 4 nodes over 500 tokens 41 us, in the two-tile form, with its second tile empty, 48; 64
  // sequences of one packed token over 32768 317 us and 331. Items of more rows read each key tile once for two
  // query tiles: 32768 tokens 5.4 ms (a tile per CTA 6.3), 64 nodes over 16 x 32768 tokens 379 us (480). The average is
  // that of the rows the call is given: a captured call whose buffers its batches do not fill may take the two-tile form
  // for short sequences, the second of those times.
  const bool solo = a.n_rows <= (a.cu ? (int64_t)a.tp * (a.n_entries / a.G) : a.tp);
  // Costs in key tiles (about 1.5 us each).
  //   item_tiles: an item's start, first step and output; without them a causal prompt's ranges of many short items
  //     end late (8192 tokens of 16 single heads 241 us, with them 224);
  //   join_tiles, cut_tiles: a partial result written and read, and a second kernel that waits for the last CTA
  //     (337 tokens with every item cut 22.6 us, with none 16.4; 4096 tokens, 512 items of up to 32 key tiles, cut 142,
  //     whole 134; 512 items of up to 64, one head a group, cut 224, whole 300);
  //   seg_tiles: a range's second segment (16 trees over 34 blocks in ranges 29 us, in equal parts 27);
  //   split_items: items in 4 rounds are dealt out whole, which leaves no partial results (8192 tokens, 1024 items: whole
  //     408 to 430 us from run to run, cut 404).
  a.n_ctas *= solo ? 2 : 1;
  a.split_items = 4 * a.n_ctas;
  a.min_tiles = 2;
  a.item_tiles = 3;
  a.join_tiles = 4;
  a.cut_tiles = 20;
  a.seg_tiles = 3;
  a.by_G = FastDiv(a.G);
  a.by_H = FastDiv(a.H);
  a.by_item = FastDiv(solo ? a.tp : 2 * a.tp);
  // What no call with these arguments can cut needs no second kernel (337 tokens 16.4 us, with it 18.6).
  const int64_t blocks = (a.idx ? a.kslots : a.ctx_len ? (a.max_ctx + kBlock - 1) / kBlock : 0) + (a.n_rows + kBlock - 1) / kBlock;
  const bool joined = (blocks + 1) / 2 > std::min(a.join_tiles, a.cut_tiles / 2);
  return solo ? launch<true>(a, maps, joined, s) : launch<false>(a, maps, joined, s);
}

}  // namespace sparda
