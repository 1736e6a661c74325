// The 4-bit KV cache: its block layout and the conversion between bf16 rows and 4-bit codes.
//
// A row (one token's key or value of one KV group) is 128 channels in four groups of 32. Each
// group has its own grid of 16 levels, given by a scale s and an offset z of 16 bits each:
//   s = T((hi - lo) / 15),  z = T(lo - 16 s),  code = clamp(rint((x - z) / s - 16), 0, 15)
//   value(code) = T(s * (16 + code) + z)
// with lo / hi the group's smallest and largest value and T the storage type, bf16 for keys and
// fp16 for values; every operation before T is one float32 operation, s * (16 + code) + z is
// rounded once. A group of equal values has s = 0 and stands for z = lo. A group with a
// non-finite value, or whose s or z overflows T, has z = NaN and stands for NaN.
//
// Why this form: 16 + code is a bit pattern. The upper mantissa bits of 16.0 (bf16 0x4180, fp16
// 0x4c00) count units, so a code placed there is 16 + code with one AND-OR, and one packed fused
// multiply-add turns two codes into two values in the type the tensor cores read: 11
// instructions for 8 values. z carries the rounding of 24 s at most (half of 0.125 s in bf16),
// which only moves the grid, since codes are taken against the rounded z. Keys are bf16 because
// the queries are; values are fp16 so that the attention weights, its other operand, keep 11
// bits instead of 8.
//
// One block (64 tokens, keys and values) is kKv4BlockBytes contiguous bytes, one bulk copy:
//   [0, 4096)      key codes    [token 64][word 16] u32, word w = channels 8w .. 8w+7
//   [4096, 8192)   value codes  [token pair 32 as (step 4, half 2, cq 4)] interleaved, below
//   [8192, 9216)   key scales   [token 64][group 4] u32: s low, z high
//   [9216, 10240)  value scales [pair 32][group 4] 2 x u32: s of both tokens, z of both tokens
// They are laid out as the attention's tensor-core fragments need them, so that a warp's
// 16-byte shared-memory loads are contiguous and nothing is moved between lanes:
//   * key word w: channel pair p (8w+2p, 8w+2p+1) in nibble p of the low / high half-word, then
//     the word rotated left by 3, which puts pair 0 where the bf16 pattern wants it; a right
//     rotation by 4p brings pair p there.
//   * value pair (tokens t0 = 16 step + 8 half + 2 cq and t0 + 1): 16 bytes for each octet g of
//     16 channels, at ((step * 2 + half) * 32 + 4 g + cq) * 16; word w of it holds channels
//     16 g + 4 w + p in nibble p, t0 in the low half-word and t0 + 1 in the high one, rotated
//     left by 6.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace sparda {
namespace kv4 {

constexpr int kGroup = 32;                         // channels that share a scale
constexpr int kGroups = kHeadDim / kGroup;         // 4
constexpr int kKCodes = 0;
constexpr int kVCodes = 4096;
constexpr int kKScales = 8192;
constexpr int kVScales = 9216;
constexpr int kBlockBytes4 = SPARDA_KV4_BLOCK_BYTES;
static_assert(kBlockBytes4 == 10240, "block layout");

__device__ __forceinline__ uint32_t ror(uint32_t x, int n) { return __funnelshift_r(x, x, n); }
__device__ __forceinline__ uint32_t rol(uint32_t x, int n) { return __funnelshift_l(x, x, n); }

// Channel pair p of a key word -> two bf16 values (s2, z2: the group's scale and offset twice).
__device__ __forceinline__ uint32_t key_pair(uint32_t word, int p, __nv_bfloat162 s2, __nv_bfloat162 z2) {
  const uint32_t u = (ror(word, 4 * p) & 0x00780078u) | 0x41804180u;
  const __nv_bfloat162 v = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u), s2, z2);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Channel p of a value word -> the values of its two tokens as fp16 (s2, z2: per token).
__device__ __forceinline__ uint32_t value_pair(uint32_t word, int p, __half2 s2, __half2 z2) {
  const uint32_t u = (ror(word, 4 * p) & 0x03c003c0u) | 0x4c004c00u;
  const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&u), s2, z2);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ __nv_bfloat162 as_bf2(uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
// The low / high half-word of u in both halves.
__device__ __forceinline__ uint32_t dup_lo(uint32_t u) { return __byte_perm(u, u, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t u) { return __byte_perm(u, u, 0x3232); }

// A group's grid. s and z as stored (16 bits each) and as float.
struct Grid {
  uint32_t s16, z16;
  float s, z;
};

template <bool kKey>
__device__ __forceinline__ Grid make_grid(float lo, float hi, bool finite) {
  Grid r;
  const float range = __fdiv_rn(__fsub_rn(hi, lo), 15.0f);
  if (kKey) {
    const __nv_bfloat16 s = __float2bfloat16_rn(range);
    r.s = __bfloat162float(s);
    __nv_bfloat16 z = __float2bfloat16_rn(__fsub_rn(lo, 16.0f * r.s));
    r.z = __bfloat162float(z);
    r.s16 = __bfloat16_as_ushort(s);
    r.z16 = __bfloat16_as_ushort(z);
  } else {
    const __half s = __float2half_rn(range);
    r.s = __half2float(s);
    __half z = __float2half_rn(__fsub_rn(lo, 16.0f * r.s));
    r.z = __half2float(z);
    r.s16 = __half_as_ushort(s);
    r.z16 = __half_as_ushort(z);
  }
  if (!finite || !(fabsf(r.z) < INFINITY) || !(r.s < INFINITY)) {
    r.s = r.z = 0.f;                               // codes 0; the offset makes every value NaN
    r.s16 = 0u;
    r.z16 = 0x7fffu;                               // NaN in bf16 and in fp16
  }
  return r;
}

__device__ __forceinline__ uint32_t code_of(float x, const Grid& g) {
  if (!(g.s > 0.f)) return 0u;
  const float c = rintf(__fsub_rn(__fdiv_rn(__fsub_rn(x, g.z), g.s), 16.0f));
  return (uint32_t)fminf(fmaxf(c, 0.f), 15.f);
}

// Byte offset in a block of the 16 bytes of value codes of token pair `pair` (token / 2) and
// channel octet g (channels 16 g ..): pairs are numbered (step, half, cq) = (bits 3.., 2, 1..0).
__device__ __forceinline__ int value_chunk(int pair, int g) {
  return kVCodes + ((pair >> 2) * 32 + 4 * g + (pair & 3)) * 16;
}
// Byte offset of the (s pair, z pair) of token pair `pair` and channel group `grp`.
__device__ __forceinline__ int value_scale(int pair, int grp) { return kVScales + (pair * 4 + grp) * 8; }

}  // namespace kv4
}  // namespace sparda
