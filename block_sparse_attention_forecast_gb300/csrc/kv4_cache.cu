// Writing and reading back the 4-bit KV cache (layout and grid: kv4.cuh): a prompt's keys and
// values at once, one decode token, and blocks back to bf16. All three move bytes: a prompt token
// is 512 bytes read and 160 written per KV group, or the reverse. Storing a prompt, some 9 instructions
// per value, hides behind that; read back, a value is one and a half.
#include "append_body.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace sparda {
using namespace kv4;

constexpr int kQThreads = 256;
constexpr int kQRounds = kBlock * 16 / kQThreads;      // (token, 8 channels) items per thread: 4

// (smallest, -largest) of packed bf16 pairs; a NaN takes over.
__device__ __forceinline__ uint32_t min_bf2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t max_bf2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// The grid of a 32-channel group spread over kLanes neighbouring lanes; x: the lane's values, in pairs.
template <bool kKey, int kLanes>
__device__ __forceinline__ Grid group_grid(const uint32_t (&x)[16 / kLanes]) {
  uint32_t lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 16 / kLanes; ++i) {
    lo = min_bf2(lo, x[i]);
    hi = max_bf2(hi, x[i]);
  }
  lo = min_bf2(lo, dup_hi(lo));                    // the low half is the smaller of the pair
  hi = max_bf2(hi, dup_hi(hi));
  uint32_t v = __byte_perm(lo, hi ^ 0x8000u, 0x5410);    // (lo, -hi): one minimum for both
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) v = min_bf2(v, __shfl_xor_sync(0xffffffffu, v, d));
  return make_grid<kKey>(bf16_lo(v), -bf16_hi(v));
}
// The codes of four pairs of values, as codes_of leaves them.
__device__ __forceinline__ void codes8(uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3, const Grid& g, uint32_t (&c)[8]) {
  const float f[8] = {bf16_lo(x0), bf16_hi(x0), bf16_lo(x1), bf16_hi(x1), bf16_lo(x2), bf16_hi(x2), bf16_lo(x3), bf16_hi(x3)};
  codes_of(f, g, c);
}

// 16 bytes into shared memory, zeros beyond the first `bytes` of them.
__device__ __forceinline__ void copy16(uint4* dst, const uint4* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
// Where 16-byte chunk q of a warp's 8 rows lies: neither its 32 lanes' consecutive chunks nor every fourth
// one meet in a bank.
__device__ __forceinline__ int swizzled(int q) { return q ^ ((q >> 3) & 3); }

// One CTA per (sequence-group, block), one thread per (token, group of 32 channels) of the keys and of
// the values: a group's extremes and grid are found once, by the thread that needs them. A warp
// fetches its own 8 tokens, whole lines at a time, through shared memory: loaded straight into registers, a
// group's 64 bytes are four loads that share lines with the neighbours', and the cache they share them in
// is too small for the CTAs in flight (a round trip that moves 1.0 GB takes 184 us that way with four CTAs per
// SM and 213 with five, 179.5 like this). The layout of a block puts every warp's codes side by side, so they
// are stored from registers, without a barrier.
__global__ void __launch_bounds__(kQThreads, 5) kv4_quantize_kernel(const Kv4CacheArgs a) {
  __shared__ uint4 rows[kQThreads / 32 * 256];
  grid_dep_wait();
  grid_dep_launch();
  const int j = blockIdx.x % a.nb_cap, bg = blockIdx.x / a.nb_cap, b = bg / a.G;
  const int T = a.seq_len[b];
  if (T < 1 || T > a.max_ctx) {
    if (threadIdx.x == 0 && j == 0) atomicOr(a.err, SPARDA_DEV_BAD_SEQ_LEN);
    return;
  }
  if (j * kBlock >= T) return;
  uint8_t* blk = a.kv + ((size_t)bg * a.nb_cap + j) * kBlockBytes4;
  // the warp's 8 tokens of the keys, then of the values
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t row = (size_t)bg * a.max_ctx + (size_t)j * kBlock + warp * 8;
  uint4* mine = rows + warp * 256;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const uint4* src = reinterpret_cast<const uint4*>(m ? a.v : a.k) + row * 16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int q = r * 32 + lane;
      // rows past the prompt are stored as zeros
      const uint32_t bytes = j * kBlock + warp * 8 + (q >> 4) < T ? 16u : 0u;
      copy16(mine + m * 128 + swizzled(q), bytes ? src + q : src, bytes);
    }
    copy_commit();
  }
  const int t = threadIdx.x >> 2, grp = threadIdx.x & 3;
  uint32_t x[16];
  const auto take_group = [&](int m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 y = mine[m * 128 + swizzled(lane * 4 + i)];
      x[4 * i] = y.x, x[4 * i + 1] = y.y, x[4 * i + 2] = y.z, x[4 * i + 3] = y.w;
    }
  };
  copy_wait<1>();
  __syncwarp();
  take_group(0);
  {
    const Grid g = group_grid<true, 1>(x);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t c[8];
      codes8(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3], g, c);
      w[i] = rol(__byte_perm(nibbles(c[0], c[2], c[4], c[6]), nibbles(c[1], c[3], c[5], c[7]), 0x5410), 3);
    }
    *reinterpret_cast<uint4*>(blk + kKCodes + threadIdx.x * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint32_t*>(blk + kKScales + threadIdx.x * 4) = g.s16 | (g.z16 << 16);
  }
  copy_wait<0>();
  __syncwarp();
  take_group(1);
  {
    const Grid g = group_grid<false, 1>(x);
    uint32_t h[8];                                 // four channels each, in the low half
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t c[8];
      codes8(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3], g, c);
      h[2 * i] = nibbles(c[0], c[1], c[2], c[3]);
      h[2 * i + 1] = nibbles(c[4], c[5], c[6], c[7]);
    }
    // the even token's thread takes the first octet of 16 channels of both tokens, the odd one's the other
    const bool odd = t & 1;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint32_t give = __byte_perm(odd ? h[i] : h[4 + i], odd ? h[i + 1] : h[5 + i], 0x5410);
      const uint32_t take = __shfl_xor_sync(0xffffffffu, give, 4);
      const uint32_t own0 = odd ? h[4 + i] : h[i], own1 = odd ? h[5 + i] : h[i + 1];
      w[i] = rol(odd ? __byte_perm(take, own0, 0x5410) : __byte_perm(own0, take, 0x5410), 2);
      w[i + 1] = rol(odd ? __byte_perm(take, own1, 0x5432) : __byte_perm(own1, take, 0x7610), 2);
    }
    *reinterpret_cast<uint4*>(blk + value_chunk(t >> 1, 2 * grp + (t & 1))) = make_uint4(w[0], w[1], w[2], w[3]);
    const uint32_t sz = g.s16 | (g.z16 << 16), so = __shfl_xor_sync(0xffffffffu, sz, 4);
    if (!odd)
      *reinterpret_cast<uint2*>(blk + value_scale(t >> 1, grp)) =
          make_uint2(__byte_perm(sz, so, 0x5410), __byte_perm(sz, so, 0x7632));
  }
}

// One CTA per (sequence-group, slot): the block's values back as bf16, rows of the sequence only.
// idx == nullptr: slot j is block j and rows go to a cache [.., max_ctx, 128]; otherwise the slot's
// block is idx[slot] and rows go to a staging buffer [.., kslots, 64, 128]. The rows, 3.2 times the
// bytes read, are stored to be evicted first, so that they do not push out a cache that was just
// written (128 blocks of 32 groups after their eviction: 49.0 us instead of 52.1, both calls).
__global__ void __launch_bounds__(kQThreads) kv4_dequantize_kernel(const Kv4CacheArgs a) {
  __shared__ alignas(16) uint8_t blk[kBlockBytes4];
  grid_dep_wait();
  grid_dep_launch();
  const int n_slots = a.idx ? a.kslots : a.nb_cap;
  const int s = blockIdx.x % n_slots, bg = blockIdx.x / n_slots, b = bg / a.G;
  const int T = a.seq_len[b];
  if (T < 1 || T > a.max_ctx) {
    if (threadIdx.x == 0 && s == 0) atomicOr(a.err, SPARDA_DEV_BAD_SEQ_LEN);
    return;
  }
  int j = s;
  if (a.idx) {
    if (s >= a.cnt[bg]) return;
    j = a.idx[(size_t)bg * a.kslots + s];
    if (j < 0 || j > (T - 1) / kBlock) {
      if (threadIdx.x == 0) atomicOr(a.err, SPARDA_DEV_BAD_INDEX);
      return;
    }
  } else if (j * kBlock >= T) {
    return;
  }
  const uint4* src = reinterpret_cast<const uint4*>(a.kv + ((size_t)bg * a.nb_cap + j) * kBlockBytes4);
  for (int i = threadIdx.x; i < kBlockBytes4 / 16; i += kQThreads) reinterpret_cast<uint4*>(blk)[i] = __ldcs(src + i);
  __syncthreads();
  const size_t row = a.idx ? ((size_t)bg * a.kslots + s) * kBlock : (size_t)bg * a.max_ctx + (size_t)j * kBlock;
  uint4* k = reinterpret_cast<uint4*>(a.k_out) + row * 16;
  uint4* v = reinterpret_cast<uint4*>(a.v_out) + row * 16;
  const int live = min(kBlock, T - j * kBlock);
  const int l16 = threadIdx.x & 15;
#pragma unroll
  for (int r = 0; r < kQRounds; ++r) {
    const int t = (threadIdx.x >> 4) + r * (kQThreads / 16);
    if (t >= live) break;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(blk + kKCodes + t * 64 + l16 * 4);
    const uint32_t sz = *reinterpret_cast<const uint32_t*>(blk + kKScales + t * 16 + (l16 >> 2) * 4);
    const uint32_t s2 = dup_lo(sz), z2 = dup_hi(sz);
    __stcs(k + t * 16 + l16, make_uint4(key_pair(w, 0, s2, z2), key_pair(w, 1, s2, z2), key_pair(w, 2, s2, z2),
                                        key_pair(w, 3, s2, z2)));
  }
#pragma unroll
  for (int r = 0; r < kQRounds / 2; ++r) {         // a token pair of 8 channels per thread
    const int pair = (threadIdx.x >> 4) + r * (kQThreads / 16);
    if (2 * pair >= live) break;
    const uint2 w = *reinterpret_cast<const uint2*>(blk + value_chunk(pair, l16 >> 1) + (l16 & 1) * 8);
    const uint2 sz = *reinterpret_cast<const uint2*>(blk + value_scale(pair, l16 >> 2));
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t word = i < 2 ? w.x : w.y;
      const float2 c0 = floats_h2(value_pair(word, (2 * i) & 3, sz.x, sz.y));
      const float2 c1 = floats_h2(value_pair(word, (2 * i + 1) & 3, sz.x, sz.y));
      lo[i] = pack_bf16(c0.x, c1.x);
      hi[i] = pack_bf16(c0.y, c1.y);
    }
    __stcs(v + (2 * pair) * 16 + l16, make_uint4(lo[0], lo[1], lo[2], lo[3]));
    if (2 * pair + 1 < live) __stcs(v + (2 * pair + 1) * 16 + l16, make_uint4(hi[0], hi[1], hi[2], hi[3]));
  }
}

// One decode token: 64 threads per (sequence, group), thread t owns channels 2t and 2t+1 of the
// key and of the value. When the token completes a compression window the same threads form the exact
// mean of the window's 32 stored keys (window_mean).
constexpr int kAppendPerCta4 = 4;

__global__ void __launch_bounds__(64 * kAppendPerCta4) kv4_append_kernel(const Kv4CacheArgs a, int bg_count) {
  grid_dep_wait();
  grid_dep_launch();
  const int bg = blockIdx.x * kAppendPerCta4 + (int)threadIdx.x / 64, t = threadIdx.x % 64;
  if (bg >= bg_count) return;                      // whole warps
  const int b = bg / a.G;
  const int T = a.seq_len[b];
  if (T < 1 || T > a.max_ctx) {
    if (t == 0) atomicOr(a.err, SPARDA_DEV_BAD_SEQ_LEN);
    return;
  }
  const int p = T - 1, tok = p % kBlock;
  uint8_t* blk = a.kv + ((size_t)bg * a.nb_cap + p / kBlock) * kBlockBytes4;
  const bool window = T >= kWinKernel && (T - kWinKernel) % kWinStride == 0;
  // the window's 31 older keys: their words and scales, issued before anything waits
  uint32_t ww[kWinKernel - 1], ws[kWinKernel - 1];
  if (window) {
#pragma unroll
    for (int u = 0; u < kWinKernel - 1; ++u) {
      const int pos = T - kWinKernel + u;
      const uint8_t* src = a.kv + ((size_t)bg * a.nb_cap + pos / kBlock) * kBlockBytes4;
      ww[u] = *reinterpret_cast<const uint32_t*>(src + kKCodes + (pos % kBlock) * 64 + (t >> 2) * 4);
      ws[u] = *reinterpret_cast<const uint32_t*>(src + kKScales + (pos % kBlock) * 16 + (t >> 4) * 4);
    }
  }
  const uint32_t kn = reinterpret_cast<const uint32_t*>(a.k + (size_t)bg * kHeadDim)[t];
  const uint32_t vn = reinterpret_cast<const uint32_t*>(a.v + (size_t)bg * kHeadDim)[t];
  const Grid gk = group_grid<true, 16>({kn}), gv = group_grid<false, 16>({vn});
  uint32_t ck[2], cv[2];
  codes_of({bf16_lo(kn), bf16_hi(kn)}, gk, ck);
  codes_of({bf16_lo(vn), bf16_hi(vn)}, gv, cv);
  // key: four threads make a word
  uint32_t w = ((ck[0] & 15u) | ((ck[1] & 15u) << 16)) << (4 * (t & 3));
  w |= __shfl_xor_sync(0xffffffffu, w, 1);
  w |= __shfl_xor_sync(0xffffffffu, w, 2);
  w = rol(w, 3);
  if ((t & 3) == 0) *reinterpret_cast<uint32_t*>(blk + kKCodes + tok * 64 + (t >> 2) * 4) = w;
  if ((t & 15) == 0) *reinterpret_cast<uint32_t*>(blk + kKScales + tok * 16 + (t >> 4) * 4) = gk.s16 | (gk.z16 << 16);
  // value: two threads make the half-word of four channels; the other half belongs to the pair's
  // other token and is kept
  uint32_t hw = ((cv[0] & 15u) | ((cv[1] & 15u) << 4)) << (8 * (t & 1));
  hw |= __shfl_xor_sync(0xffffffffu, hw, 1);
  const int pair = tok >> 1;
  if ((t & 1) == 0) {
    uint32_t* word = reinterpret_cast<uint32_t*>(blk + value_chunk(pair, t >> 3) + ((t >> 1) & 3) * 4);
    *word = rol((tok & 1) ? ((ror(*word, 2) & 0xffffu) | (hw << 16)) : hw, 2);
  }
  if ((t & 15) == 0) {
    uint16_t* sz = reinterpret_cast<uint16_t*>(blk + value_scale(pair, t >> 4)) + (tok & 1);
    sz[0] = (uint16_t)gv.s16;
    sz[2] = (uint16_t)gv.z16;
    if (!(tok & 1)) sz[1] = sz[3] = 0;             // the pair's other token is not there yet
  }
  if (!window) return;
  uint32_t xs[kWinKernel];
#pragma unroll
  for (int u = 0; u < kWinKernel - 1; ++u)
    xs[u] = key_pair(ww[u], t & 3, dup_lo(ws[u]), dup_hi(ws[u]));
  const uint32_t sz = gk.s16 | (gk.z16 << 16);
  xs[kWinKernel - 1] = key_pair(w, t & 3, dup_lo(sz), dup_hi(sz));
  reinterpret_cast<uint32_t*>(a.ck + ((size_t)bg * a.W_cap + (T - kWinKernel) / kWinStride) * kHeadDim)[t] =
      window_mean(xs);
}

void launch_kv4_quantize(const Kv4CacheArgs& a, int bg_count, cudaStream_t s) {
  launch_pdl(kv4_quantize_kernel, dim3((unsigned)bg_count * a.nb_cap), dim3(kQThreads), 0, s, a);
}
void launch_kv4_dequantize(const Kv4CacheArgs& a, int bg_count, cudaStream_t s) {
  launch_pdl(kv4_dequantize_kernel, dim3((unsigned)bg_count * (a.idx ? a.kslots : a.nb_cap)), dim3(kQThreads), 0, s, a);
}
void launch_kv4_append(const Kv4CacheArgs& a, int bg_count, cudaStream_t s) {
  launch_pdl(kv4_append_kernel, dim3((bg_count + kAppendPerCta4 - 1) / kAppendPerCta4), dim3(64 * kAppendPerCta4), 0, s, a,
             bg_count);
}

}  // namespace sparda
