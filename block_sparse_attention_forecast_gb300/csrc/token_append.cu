// Many new tokens into a bf16 cache: packed prompts, or the accepted paths of trees of drafted tokens, with
// the compressed keys of the windows that they complete (the exact mean of 32 keys, rounded once to bf16).
//
// A CTA takes the new tokens of one 64-token block of one sequence's cache, for one KV group: their keys
// go through shared memory together with the 16 keys before the block and the block's cached ones that their
// windows reach back to (from the cache, or from the new rows), values straight through; then 64 threads per
// window, two channels each, form the four windows that end in the block. Bound by memory, and so by the bytes under
// way: every load of a thread is issued before its first store, keys go to shared memory without a register in
// between, and the 48 registers that the windows need let 5 CTAs run on an SM (4 x up to 131072 tokens, 2 groups: 145 us,
// 6.1 TB/s, 0.91 of the measured copy rate; keys through registers and 4 CTAs 152 us; 6 CTAs, with the windows'
// values spilled, 149; each load stored before the next 252).
#include "append_body.cuh"

namespace sparda {

namespace {
constexpr int kThreads = 256;
constexpr int kHalo = kWinKernel - kWinStride;               // windows begin at multiples of 16
constexpr int kCommitBlocks = kTokenMaxNodes / kBlock + 1;   // cache blocks that a path reaches into, at most

// What sequence b appends: n rows behind its S cached tokens; false: nothing may be written.
__device__ __forceinline__ bool append_range(const TokenAppendArgs& a, int b, int& S, int& n, int& row0) {
  S = a.seq_len ? a.seq_len[b] : 0;
  bool good = S >= 0 && S <= a.max_ctx;
  if (a.cu) {
    const int lo = a.cu[b], hi = a.cu[b + 1];
    good = good && lo >= 0 && hi >= lo && hi <= a.n_rows && hi - lo <= a.max_ctx - S;
    row0 = lo;
    n = hi - lo;
  } else {
    n = a.n_path[b];
    good = good && n >= 0 && n <= a.n_rows && n <= a.max_ctx - S;
    row0 = b * a.n_rows;
  }
  if (!good) n = 0;
  return good;
}

// 16 bytes of global memory, or zeros, to shared memory, without a register in between
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}

__device__ __forceinline__ int blocks_touched(int S, int n) { return n == 0 ? 0 : (S + n - 1) / kBlock - S / kBlock + 1; }

struct AppendShared {
  __align__(16) uint32_t ks[kHalo + kBlock][kHeadDim / 2];
  int path[kTokenMaxNodes];
  int bad_path;
};

// Block `at` of the call, for group g (all threads of the CTA). False if there is none, or if none can be behind the grid.
//
// Prompts: the blocks are counted off sequence by sequence, and the grid holds as many as ascending rows can make. Where
// cu descends somewhere (that sequence is refused), the sequences behind it may name rows again and have more blocks than
// that: `falls`, which the barrier before the windows gathers. It is looked up behind the values' stores, where their
// registers are free and the copies are still waited for.
__device__ __forceinline__ bool append_block(const TokenAppendArgs& a, unsigned at, int g, AppendShared& sh) {
  auto& ks = sh.ks;
  const int tid = threadIdx.x, lane = tid & 31;
  int b, blk, S, n, row0;
  bool good;
  if (a.cu) {
    // every warp looks the block up: blocks before 32 sequences at a time
    int left = at;
    b = -1;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      int s_ = 0, n_ = 0, r_ = 0;
      bool good_ = true;
      if (b0 + lane < a.B) {
        good_ = append_range(a, b0 + lane, s_, n_, r_);
        if (at == 0 && g == 0 && tid < 32) {
          if (!good_) atomicOr(a.err, SPARDA_DEV_BAD_SEQ_LEN);
          if (a.new_len) a.new_len[b0 + lane] = s_ + n_;
        }
      }
      int incl = blocks_touched(s_, n_);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const int sum = __shfl_sync(0xffffffffu, incl, 31);
      if (b < 0 && left < sum) {
        const int l = __ffs(__ballot_sync(0xffffffffu, incl > left)) - 1;
        blk = left - (l == 0 ? 0 : __shfl_sync(0xffffffffu, incl, (l + 31) & 31));
        b = b0 + l;
        if (at != 0) break;
      }
      left -= sum;
    }
    if (b < 0) return false;
    good = append_range(a, b, S, n, row0);
  } else {
    b = blockIdx.x / kCommitBlocks;
    blk = blockIdx.x % kCommitBlocks;
    good = append_range(a, b, S, n, row0);
    if (tid == 0) sh.bad_path = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const int r = a.path[(size_t)b * a.n_rows + i];
      sh.path[i] = r;
      if (r < 0 || r >= a.n_rows) sh.bad_path = 1;
    }
    __syncthreads();
    if (sh.bad_path) n = 0;
    if (blk == 0 && g == 0 && tid == 0) {
      if (!good) atomicOr(a.err, SPARDA_DEV_BAD_SEQ_LEN);
      if (sh.bad_path) atomicOr(a.err, SPARDA_DEV_BAD_INDEX);
      if (a.new_len) a.new_len[b] = S + n;
    }
    if (blk >= blocks_touched(S, n)) return false;
  }
  // cache positions lo .. hi-1 of this block
  const size_t bg = (size_t)b * a.G + g;
  const int base = (S / kBlock + blk) * kBlock;
  const int lo = max(S, base), hi = min(S + n, base + kBlock);
  const __nv_bfloat16* kc = a.k + bg * a.max_ctx * kHeadDim;
  auto new_row = [&](int pos) {
    const int i = pos - S;
    return (size_t)(row0 + (a.cu ? i : sh.path[i])) * a.kv_stride + g * kHeadDim;
  };
  // thread: 16 bytes of the rows r, r + 16, ..; the first 16 rows are those before the block
  constexpr int kRows = kThreads / 16, kParts = (kHalo + kBlock) / kRows;
  static_assert(kHalo == kRows && kBlock % kRows == 0, "the rows before the block are the first part");
  const int c = tid & 15, r = tid >> 4;
  uint4 y[kParts];
#pragma unroll
  for (int j = 0; j < kParts; ++j) {
    const int pos = base - kHalo + r + kRows * j;
    const __nv_bfloat16* src = nullptr;
    if (pos >= S && pos < hi) {
      const size_t row = new_row(pos) + 8 * c;
      src = a.k_new + row;
      if (j > 0) y[j] = *reinterpret_cast<const uint4*>(a.v_new + row);
    } else if (pos >= 0 && pos < S) {
      src = kc + (size_t)pos * kHeadDim + 8 * c;
    }
    cp_async16_or_zero(&ks[r + kRows * j][4 * c], src ? src : kc, src != nullptr);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
  for (int j = 1; j < kParts; ++j) {
    const int pos = base - kHalo + r + kRows * j;
    if (pos >= S && pos < hi) *reinterpret_cast<uint4*>(a.v + (bg * a.max_ctx + pos) * kHeadDim + 8 * c) = y[j];
  }
  bool falls = false;
  if (a.cu)
    for (int i = tid; i < a.B; i += kThreads) falls = falls || a.cu[i + 1] < a.cu[i];
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int j = 1; j < kParts; ++j) {
    const int pos = base - kHalo + r + kRows * j;
    if (pos >= S && pos < hi)
      *reinterpret_cast<uint4*>(a.k + (bg * a.max_ctx + pos) * kHeadDim + 8 * c) =
          *reinterpret_cast<const uint4*>(&ks[r + kRows * j][4 * c]);   // (what this thread copied itself)
  }
  const bool more = __syncthreads_or(falls);
  // the windows that end in lo+1 .. hi: window w ends at 16 w + 32
  const int w = base / kWinStride - 1 + (tid >> 6), end = w * kWinStride + kWinKernel, pair = tid & 63;
  if (w >= 0 && end > lo && end <= hi) {
    uint32_t xs[kWinKernel];
#pragma unroll
    for (int u = 0; u < kWinKernel; ++u) xs[u] = ks[end - kWinKernel + u - (base - kHalo)][pair];
    reinterpret_cast<uint32_t*>(a.ck + (bg * a.W_cap + w) * kHeadDim)[pair] = window_mean(xs);
  }
  return more;
}

// The blocks behind the grid's, a grid further at a time. A function of its own: with this loop around the block in the kernel
// the windows spill (4 x up to 131072 tokens 194 us; this way 145, and 143.5 with no look at cu).
__device__ __noinline__ void append_rest(const TokenAppendArgs& a, int g, AppendShared& sh) {
  for (unsigned at = blockIdx.x + gridDim.x;; at += gridDim.x) {
    __syncthreads();                                           // the block before is read
    if (!append_block(a, at, g, sh)) return;
  }
}
}  // namespace

// grid (blocks of all sequences, G)
__global__ void __launch_bounds__(kThreads, 5) token_append_kernel(const __grid_constant__ TokenAppendArgs a) {
  __shared__ AppendShared sh;
  if (append_block(a, blockIdx.x, blockIdx.y, sh)) append_rest(a, blockIdx.y, sh);
}

cudaError_t launch_token_append(const TokenAppendArgs& a, cudaStream_t s) {
  // a prompt of n tokens reaches into at most n / 64 + 2 blocks of its cache
  const long long blocks = a.cu ? (long long)a.n_rows / kBlock + 2ll * a.B : (long long)a.B * kCommitBlocks;
  token_append_kernel<<<dim3((unsigned)blocks, a.G), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace sparda
