// Eviction: every (sequence, group) keeps block 0, its `recent` newest blocks and, of the others,
// the ones with the largest accumulated attention weight, `keep` blocks in all; kept blocks move
// together to the front in their order, with their compressed keys and weights, in the cache itself
// or into another (smaller) one, and the sequence's length drops by the blocks lost.
//
//   evict_select_kernel   one CTA per (sequence, group): the kept list. The weights stay in
//                         registers as order-preserving integers; the (keep - forced)-th largest
//                         is found digit by digit, three histograms at most, whatever the
//                         weights' spread; of the keys tied there the lowest blocks are taken.
//   evict_move_kernel     into another cache: bytes in, bytes out.
//   evict_shift_kernel    in the cache itself: block n moves from kept[n] >= n, so its place may be
//                         written only once the block that lay there, if it is kept, has been read.
//                         That block is kept[m] == n for an m < n: the kept list carries a mark on
//                         every block still to be read, whoever has read it clears the mark, and
//                         block n's write waits for m's. One cooperative launch, blocks in the order
//                         of n: the lowest one in flight never waits, so every wait ends.
//   evict_join_kernel     after the shift: the compressed keys of windows that span two blocks
//                         which were not neighbours before (the move kernel does its own), and the
//                         weights, which must not move unless the blocks do.
//   evict_length_kernel   after the shift: the new lengths, once nothing reads the old ones.
//
// A moved block's windows 4n .. 4n+2 lie inside it and move with it; window 4n+3 takes its last 16
// keys and the first 16 of the next block.
#include "append_body.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace sparda {

namespace {

constexpr int kSelThreads = 512;
static_assert(kSelThreads / 32 <= 32, "a warp's lanes hold the warps' totals");
constexpr int kSelPer = kMaxCtx / kBlock / kSelThreads;         // weights per thread: 8
constexpr int kBins = 2048;
constexpr int kMoveThreads = 256;
// The move's ring slots per CTA, and the bytes of all CTAs' slots on an SM. Twice 32 KiB (bf16) or three times
// 20 (4 bits) per SM is the fastest of rings from 16 to 192 KiB: more or fewer bytes in flight cost up to a
// quarter, as DRAM switches between reading and writing.
//   4096 blocks of bf16 keys and values, with the selection: 49.1 us; 54.4 with twice 96 KiB, 63 with once 32
//   4096 blocks in 4 bits, with the selection and the reading back: 43.6 us; 45.1 with twice 32, 49.3 with twice 96
constexpr int kMoveSlots = 2;
constexpr int kMoveBytes = 64 * 1024;
constexpr uint32_t kMovePolls = 1u << 25;                       // bounds a lane's wait to seconds
// The same, each a round trip to L2. (A test builds this file with a limit that runs out.)
#ifndef SPARDA_SHIFT_POLLS
#define SPARDA_SHIFT_POLLS (1u << 22)
#endif
constexpr uint32_t kShiftPolls = SPARDA_SHIFT_POLLS;
// Shared memory of the shift's CTAs on an SM, a block each. With the selection, 4 sequences of bf16 blocks to 512:
// 81 us at 72 KiB, 70 at 140, 68 at 175, 67 at 210; 16 sequences in 4 bits to 512: 129, 112, 110, 108. (A cluster
// per group that reads a round of blocks before it writes it: 125 and 146; of one sequence 103, this 23.)
constexpr int kShiftBytes = 175 * 1024;
// In the kept list while a cache is cut in place: a block that moves and has not been read. On the first
// entry of a sequence's first group, block 0, which never moves: a wait ran out and blocks of the sequence
// were left.
constexpr int kUnread = 1 << 30;
constexpr int kCkRow = kHeadDim * 2;                            // bytes of a compressed key

__device__ __forceinline__ bool valid_len(int T, int nb) { return T >= 1 && T <= nb * kBlock; }
__device__ __forceinline__ int blocks_of(int T) { return (T - 1) / kBlock + 1; }
// The length after the eviction of a sequence of T tokens.
__device__ __forceinline__ int kept_len(int T, int keep) {
  const int n = blocks_of(T);
  return T - kBlock * (n - min(n, keep));
}

// Weight -> integer in the weights' order: a NaN above every number, -0 equal to +0, 0 unused.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  return ordered_key(w == 0.f ? 0.f : w);
}

// Two channels of the key of token `tok` of block j of (sequence, group) bg.
__device__ __forceinline__ uint32_t cache_key2(const uint8_t* plane, int kv4, size_t block, int tok, int t) {
  if (!kv4) return reinterpret_cast<const uint32_t*>(plane + block * kBlockBytes + tok * kRowBytes)[t];
  const uint8_t* b = plane + block * kv4::kBlockBytes4;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(b + kv4::kKCodes + tok * 64 + (t >> 2) * 4);
  const uint32_t sz = *reinterpret_cast<const uint32_t*>(b + kv4::kKScales + tok * 16 + (t >> 4) * 4);
  return kv4::key_pair(w, t & 3, kv4::dup_lo(sz), kv4::dup_hi(sz));
}

// The compressed key of a window made of the last 16 keys of block ja and the first 16 of jb, by 64 threads.
__device__ __forceinline__ uint32_t joined_window(const uint8_t* plane, int kv4, size_t ja, size_t jb, int t) {
  uint32_t xs[kWinKernel];
#pragma unroll
  for (int u = 0; u < kWinKernel / 2; ++u) {
    xs[u] = cache_key2(plane, kv4, ja, kBlock - kWinKernel / 2 + u, t);
    xs[u + kWinKernel / 2] = cache_key2(plane, kv4, jb, u, t);
  }
  return window_mean(xs);
}

// Bytes of compressed keys that move with kept block n of `count` (T tokens afterwards): its windows
// that are complete, its last only beside its old neighbour.
__device__ __forceinline__ int window_bytes(int n, int count, int T, bool neighbour) {
  const int complete = num_windows(T) - 4 * n;
  const int own = n + 1 < count && neighbour ? 4 : 3;
  return min(max(complete, 0), own) * kCkRow;
}
// Whether the shift left blocks of sequence b (of a valid length) where they were.
__device__ __forceinline__ bool left_blocks(const EvictArgs& a, int b) {
  return (a.kept[(size_t)b * a.G * a.keep] & kUnread) != 0;
}
// Whether window 4n+3 has to be formed anew.
__device__ __forceinline__ bool joins(int n, int count, int T, bool neighbour) {
  return n + 1 < count && !neighbour && num_windows(T) > 4 * n + 3;
}

}  // namespace

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ int s_bin[kBins], s_found[3];
  __shared__ int s_warp[3][kSelThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int bg = blockIdx.x, b = bg / a.G, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float* src = a.src_mass + (size_t)bg * a.src_nb;
  float w[kSelPer];
  uint32_t key[kSelPer];
#pragma unroll
  for (int i = 0; i < kSelPer; ++i) {              // beside the length's load, not behind it
    const int j = tid * kSelPer + i;
    w[i] = j < a.src_nb ? src[j] : 0.f;
  }
  const int T = a.src_len[b];
  const bool valid = valid_len(T, a.src_nb);
  const int n = valid ? blocks_of(T) : 0, count = min(n, a.keep);
  if (!valid && tid == 0) atomicOr(a.err, SPARDA_DEV_BAD_SEQ_LEN);
  // the sum of the earlier warps' totals
  const auto earlier = [&](const int (&totals)[kSelThreads / 32]) {
    return (int)__reduce_add_sync(0xffffffffu, lane < warp ? totals[lane] : 0);
  };
#pragma unroll
  for (int i = 0; i < kSelPer; ++i) {
    const int j = tid * kSelPer + i;
    key[i] = j >= 1 && j < n - a.recent ? weight_key(w[i]) : 0u;     // candidates only
  }
  uint32_t sel = 0;                                // bit i: block tid * kSelPer + i is kept
  if (n <= a.keep) {
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) sel |= (tid * kSelPer + i < n ? 1u : 0u) << i;
  } else {
    const int want = a.keep - 1 - a.recent;        // candidates to keep; more of them exist
    uint32_t thr = 0xffffffffu;                    // the want-th largest key (its leading bits)
    int share = 0, low = 0;                        // of the keys whose bits above `low` are thr's, the share kept
    if (want > 0) {
      // digits of 11, 11 and 10 bits: a histogram of the keys that agree so far, and the digit at
      // which the counts from the top reach the share
      thr = 0u;
      share = want;
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass < 2 ? 11 : 10, above = pass == 0 ? 32 : pass == 1 ? 21 : 10;
        low = above - bits;
        for (int i = tid; i < kBins; i += kSelThreads) s_bin[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSelPer; ++i)
          if (key[i] != 0u && (pass == 0 || (key[i] ^ thr) >> above == 0u))
            atomicAdd(&s_bin[(key[i] >> low) & ((1u << bits) - 1u)], 1);
        __syncthreads();
        // this thread's bins are the highest kBins / kSelThreads not yet taken: thread 0 the top ones
        constexpr int kPer = kBins / kSelThreads;
        int n_bin[kPer], mine = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          n_bin[i] = s_bin[kBins - 1 - tid * kPer - i];
          mine += n_bin[i];
        }
        int sum = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, sum, d);
          if (lane >= d) sum += o;
        }
        if (lane == 31) s_warp[0][warp] = sum;
        __syncthreads();
        int before = sum - mine + earlier(s_warp[0]);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (before < share && before + n_bin[i] >= share) {
            s_found[0] = kBins - 1 - tid * kPer - i;
            s_found[1] = share - before;
            s_found[2] = n_bin[i];
          }
          before += n_bin[i];
        }
        __syncthreads();
        thr |= (uint32_t)s_found[0] << low;
        share = s_found[1];
        if (s_found[2] == share) break;            // all of them are kept
      }
    }
    const uint32_t lead = thr >> low;              // keys are ranked by their bits from `low` on
    // ties go to the lowest blocks: the rank of each key equal to thr
    int ties = 0;
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) ties += want > 0 && key[i] != 0u && key[i] >> low == lead;
    int scan = ties;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, scan, d);
      if (lane >= d) scan += o;
    }
    if (lane == 31) s_warp[1][warp] = scan;
    __syncthreads();
    int rank = scan - ties + earlier(s_warp[1]);
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      const int j = tid * kSelPer + i;
      bool in = j == 0 || (j >= n - a.recent && j < n);
      if (want > 0 && key[i] != 0u) {
        in = in || key[i] >> low > lead;
        if (key[i] >> low == lead) in = in || rank++ < share;
      }
      sel |= (in ? 1u : 0u) << i;
    }
  }
  // places: an exclusive scan of the kept flags in block order
  const int mine = __popc(sel);
  int scan = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, scan, d);
    if (lane >= d) scan += o;
  }
  if (lane == 31) s_warp[2][warp] = scan;
  __syncthreads();
  int at = scan - mine + earlier(s_warp[2]);
  int32_t* kept = a.kept + (size_t)bg * a.keep;
  float* dst = a.dst_mass + (size_t)bg * a.dst_nb;
#pragma unroll
  for (int i = 0; i < kSelPer; ++i)
    if (sel >> i & 1u) {
      const int j = tid * kSelPer + i;
      kept[at] = a.in_place && j != at ? j | kUnread : j;
      if (!a.in_place) dst[at] = w[i];             // in place the weights move when the blocks have
      ++at;
    }
  for (int i = count + tid; i < a.keep; i += kSelThreads) kept[i] = -1;
  if (valid && !a.in_place)
    for (int i = count + tid; i < a.dst_nb; i += kSelThreads) dst[i] = 0.f;
  if (!a.in_place && tid == 0 && bg % a.G == 0) a.dst_len[b] = valid ? kept_len(T, a.keep) : T;
}

// A fixed grid. Warp 0 moves whole blocks by bulk copies through a ring in shared memory: lane l owns a
// slot of it and every (slots x CTAs)-th block, so the reads in flight do not depend on registers. The
// other warps, 64 threads per kept block, move the compressed keys and form those of windows that join blocks.
__global__ void __launch_bounds__(kMoveThreads + 32) evict_move_kernel(const EvictArgs a) {
  extern __shared__ uint8_t smem_move[];
  __shared__ alignas(8) uint64_t full[kMoveSlots];
  const int tid = threadIdx.x, lane = tid & 31;
  const int n_kept = a.B * a.G * a.keep;
  if (tid < 32) {
    if (lane < kMoveSlots) mbar_init(&full[lane], 1);
    fence_mbar_init();
    __syncwarp();
  }
  grid_dep_wait();
  grid_dep_launch();
  if (tid < 32) {
    if (lane >= kMoveSlots) return;
    uint8_t* slot = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_move) + 127) & ~static_cast<uintptr_t>(127)) +
                    (size_t)lane * a.block_bytes;
    int item = (int)blockIdx.x * kMoveSlots + lane;     // one plane's kept blocks, then the other's
    const int step = (int)gridDim.x * kMoveSlots, items = n_kept * a.planes;
    uint8_t* dst = nullptr;
    // issues the read of the lane's next block, if there is one
    const auto read_next = [&]() -> bool {
      for (; item < items; item += step) {
        const int k = item % n_kept, p = item / n_kept, bg = k / a.keep, n = k % a.keep;
        const int j = a.kept[k];
        if (j < 0) continue;
        dst = a.dst[p] + ((size_t)bg * a.dst_nb + n) * a.block_bytes;
        mbar_arrive_expect_tx(&full[lane], a.block_bytes);
        bulk_load(slot, a.src[p] + ((size_t)bg * a.src_nb + j) * a.block_bytes, a.block_bytes, &full[lane]);
        item += step;
        return true;
      }
      return false;
    };
    uint32_t phase = 0, polls = 0;
    bool reading = read_next();
    while (reading) {
      if (mbar_test_wait(&full[lane], phase)) {
        bulk_store(dst, slot, a.block_bytes);
        bulk_commit();
        bulk_wait_read<0>();                       // the slot may be filled again
        phase ^= 1;
        polls = 0;
        reading = read_next();
      } else if (++polls > kMovePolls) {
        atomicOr(a.err, SPARDA_DEV_WAIT_TIMEOUT);
        reading = false;
      }
    }
    bulk_wait_all();
    return;
  }
  const int t = (tid - 32) % 64;
  for (int k = (int)blockIdx.x * (kMoveThreads / 64) + (tid - 32) / 64; k < n_kept; k += (int)gridDim.x * (kMoveThreads / 64)) {
    const int bg = k / a.keep, n = k % a.keep;
    const int j = a.kept[k], nxt = n + 1 < a.keep ? a.kept[k + 1] : -1;
    if (j < 0) continue;
    const int T0 = a.src_len[bg / a.G];
    const int T = kept_len(T0, a.keep), count = min(blocks_of(T0), a.keep);
    const size_t from = (size_t)bg * a.src_nb + j;
    const size_t src_row = (size_t)bg * (4 * a.src_nb - 1) + 4 * j, dst_row = (size_t)bg * (4 * a.dst_nb - 1) + 4 * n;
    const bool neighbour = nxt == j + 1;
    if (t < window_bytes(n, count, T, neighbour) / 16)
      reinterpret_cast<uint4*>(a.dst_ck + dst_row * kHeadDim)[t] = reinterpret_cast<const uint4*>(a.src_ck + src_row * kHeadDim)[t];
    if (joins(n, count, T, neighbour))
      reinterpret_cast<uint32_t*>(a.dst_ck + (dst_row + 3) * kHeadDim)[t] =
          joined_window(a.src[0], a.kv4, from, (size_t)bg * a.src_nb + nxt, t);
  }
}

// One warp per CTA, whose first lane moves one block at a time, with its compressed keys: its read, the mark, the
// wait, its write. All CTAs are resident (a cooperative launch). Reads and writes of a block are each
// whole before the next thing happens to its place, so no write meets a read of the same bytes.
__global__ void __launch_bounds__(32) evict_shift_kernel(const EvictArgs a) {
  extern __shared__ uint8_t smem_shift[];
  __shared__ alignas(8) uint64_t full;
  if (threadIdx.x) return;
  mbar_init(&full, 1);
  fence_mbar_init();
  uint8_t* slot = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_shift) + 127) & ~static_cast<uintptr_t>(127));
  const int groups = a.B * a.G, items = groups * a.keep;
  uint32_t phase = 0;
  bool ok = true;                                  // until a wait runs out: then nothing more is moved
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int bg = item % groups, n = item / groups;
    int32_t* kept = a.kept + (size_t)bg * a.keep;
    const int v = kept[n], j = v & ~kUnread;
    if (v < 0 || !(v & kUnread) || j == n) continue;     // behind the last block, or already in place with its windows
    // a block is left: its sequence is marked, its own mark cleared, so that nobody waits for it
    const auto leave = [&]() {
      atomicOr(a.kept + (size_t)(bg / a.G) * a.G * a.keep, kUnread);
      asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(kept + n), "r"(j) : "memory");
    };
    if (!ok) {
      leave();
      continue;
    }
    const int T0 = a.src_len[bg / a.G];
    const int T = kept_len(T0, a.keep), count = min(blocks_of(T0), a.keep);
    const bool neighbour = n + 1 < count && (kept[n + 1] & ~kUnread) == j + 1;
    const int ck = window_bytes(n, count, T, neighbour);
    const size_t row = (size_t)bg * (4 * a.dst_nb - 1);
    mbar_arrive_expect_tx(&full, a.planes * a.block_bytes + ck);
    for (int p = 0; p < a.planes; ++p)
      bulk_load(slot + p * a.block_bytes, a.dst[p] + ((size_t)bg * a.dst_nb + j) * a.block_bytes, a.block_bytes, &full);
    if (ck) bulk_load(slot + a.planes * a.block_bytes, a.dst_ck + (row + 4 * j) * kHeadDim, ck, &full);
    // meanwhile: the kept block that lies at n, kept[m] for an m < n (the list ascends, and kept[i] >= i)
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if ((kept[mid] & ~kUnread) < n) lo = mid + 1;
      else hi = mid;
    }
    ok = mbar_wait(&full, phase, a.err);
    phase ^= 1;
    if (ok) asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(kept + n), "r"(j) : "memory");
    if (ok && lo < n && (kept[lo] & ~kUnread) == n) {
      uint32_t polls = 0;
      for (;;) {
        int at;
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(at) : "l"(kept + lo) : "memory");
        if (!(at & kUnread)) break;
        if (++polls > kShiftPolls) {
          atomicOr(a.err, SPARDA_DEV_WAIT_TIMEOUT);
          ok = false;
          break;
        }
      }
    }
    if (!ok) {
      leave();
      continue;
    }
    for (int p = 0; p < a.planes; ++p)
      bulk_store(a.dst[p] + ((size_t)bg * a.dst_nb + n) * a.block_bytes, slot + p * a.block_bytes, a.block_bytes);
    if (ck) bulk_store(a.dst_ck + (row + 4 * n) * kHeadDim, slot + a.planes * a.block_bytes, ck);
    bulk_commit();
    bulk_wait_read<0>();                           // the slot may be filled again
  }
  bulk_wait_all();
}

// Grid: (sequence, group) x groups of kept blocks, 64 threads per kept block. A group's first CTA also moves
// its weights, each read before one is written.
__global__ void __launch_bounds__(kMoveThreads) evict_join_kernel(const EvictArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int per = kMoveThreads / 64;
  const int pieces = (a.keep + per - 1) / per;
  const int bg = blockIdx.x / pieces, n = (blockIdx.x % pieces) * per + (int)threadIdx.x / 64, t = threadIdx.x % 64;
  const int T0 = a.src_len[bg / a.G];
  if (!valid_len(T0, a.src_nb)) return;
  const int32_t* kept = a.kept + (size_t)bg * a.keep;
  const int count = min(blocks_of(T0), a.keep);
  if (left_blocks(a, bg / a.G)) return;
  if (blockIdx.x % pieces == 0) {
    float* mass = a.dst_mass + (size_t)bg * a.dst_nb;
    float w[kMaxCtx / kBlock / kMoveThreads];
#pragma unroll
    for (int i = 0; i < kMaxCtx / kBlock / kMoveThreads; ++i) {
      const int at = i * kMoveThreads + (int)threadIdx.x;
      w[i] = at < count ? mass[kept[at]] : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMaxCtx / kBlock / kMoveThreads; ++i) {
      const int at = i * kMoveThreads + (int)threadIdx.x;
      if (at < a.dst_nb) mass[at] = w[i];
    }
  }
  if (n + 1 >= a.keep || !joins(n, count, kept_len(T0, a.keep), kept[n + 1] == kept[n] + 1)) return;
  const size_t block = (size_t)bg * a.dst_nb + n;
  reinterpret_cast<uint32_t*>(a.dst_ck + ((size_t)bg * (4 * a.dst_nb - 1) + 4 * n + 3) * kHeadDim)[t] =
      joined_window(a.dst[0], a.kv4, block, block + 1, t);
}

__global__ void evict_length_kernel(const EvictArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    const int T = a.src_len[b];
    if (!valid_len(T, a.src_nb)) continue;
    if (left_blocks(a, b))
      a.kept[(size_t)b * a.G * a.keep] = 0;        // block 0, without the mark
    else
      a.dst_len[b] = kept_len(T, a.keep);
  }
}

namespace {

// CTAs of the shift that an SM holds at once, found once per device and size of a block.
int shift_ctas_per_sm(const EvictArgs& a, int smem) {
  static std::atomic<int> known[64][2] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::atomic<int>& n = known[dev][a.kv4 ? 1 : 0];
  int ctas = n.load(std::memory_order_relaxed);
  if (ctas == 0 && cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, evict_shift_kernel, 32, smem) == cudaSuccess)
    n.store(ctas, std::memory_order_relaxed);
  return ctas;
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  const unsigned bg = (unsigned)a.B * a.G;
  const int smem = 128 + a.planes * a.block_bytes + 4 * kCkRow;       // of the shift
  long long most = 0;
  if (a.in_place) {
    const int fit = shift_ctas_per_sm(a, smem);    // the cooperative launch needs all its CTAs resident
    if (fit < 1) return cudaErrorCooperativeLaunchTooLarge;
    most = (long long)min(fit, kShiftBytes / smem) * sm_count();
  }
  cudaError_t err = launch_pdl(evict_select_kernel, dim3(bg), dim3(kSelThreads), 0, s, a);
  if (err != cudaSuccess) return err;
  if (!a.in_place) {
    const int ring = kMoveSlots * a.block_bytes;
    const long long items = (long long)bg * a.keep * a.planes, ctas = (items + kMoveSlots - 1) / kMoveSlots;
    const int all = kMoveBytes / ring * sm_count(), grid = (int)(ctas < all ? ctas : all);
    return launch_pdl(evict_move_kernel, dim3(grid), dim3(kMoveThreads + 32), (size_t)ring + 128, s, a);
  }
  const long long items = (long long)bg * a.keep;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items < most ? items : most));
  cfg.blockDim = dim3(32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, evict_shift_kernel, a);
  if (err != cudaSuccess) return err;
  err = launch_pdl(evict_join_kernel, dim3(bg * (unsigned)((a.keep + 3) / 4)), dim3(kMoveThreads), 0, s, a);
  if (err != cudaSuccess) return err;
  return launch_pdl(evict_length_kernel, dim3(1), dim3(256), 0, s, a);
}

}  // namespace sparda
