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
// instructions for 8 values, 5 to 7 of them on the half-rate logic pipe. z carries one rounding, of at most
// 2^-8 |z| in bf16 and 2^-11 |z| in fp16 (|z| is about 24 s for a group around zero, and without bound beside
// s for values with a common offset). It only moves the grid, since codes are taken against the rounded z. Keys are bf16 because
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
//     left by 2: channels 0 and 1 (and, after a rotation by 8, 2 and 3) can then be taken where they
//     lie, as 256 + code and as 16 + code; the 240 too many come off in one addition, on the
//     multiply-add pipe, which has room where the logic pipe has none.
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

// Two values at a time, packed in 32 bits; each result is rounded once.
__device__ __forceinline__ uint32_t fma_bf2(uint32_t x, uint32_t y, uint32_t z) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
  return r;
}
__device__ __forceinline__ uint32_t fma_h2(uint32_t x, uint32_t y, uint32_t z) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
  return r;
}
__device__ __forceinline__ uint32_t add_h2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ float2 floats_h2(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

// The code masks. A kernel in which the unpacking counts holds them in vector registers (read from
// shared memory): an AND-OR with the mask and the pattern both constants, or both uniform
// registers, costs a second instruction, a move.
struct Masks {
  uint32_t key = 0x00780078u;       // bits 3..6 of each half
  uint32_t lo = 0x003c003cu;        // bits 2..5
  uint32_t hi = 0x03c003c0u;        // bits 6..9
};

template <uint32_t kPattern>
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "r"(mask), "n"(kPattern));
  return r;
}

// Channel pair p of a key word -> two bf16 values (s2, z2: the group's scale and offset twice).
__device__ __forceinline__ uint32_t key_pair(uint32_t word, int p, uint32_t s2, uint32_t z2, const Masks& m = Masks()) {
  return fma_bf2(and_or<0x41804180u>(ror(word, 4 * p), m.key), s2, z2);
}

// Channel p of a value word -> the values of its two tokens as fp16 (s2, z2: per token).
__device__ __forceinline__ uint32_t value_pair(uint32_t word, int p, uint32_t s2, uint32_t z2, const Masks& m = Masks()) {
  const uint32_t u = p < 2 ? word : ror(word, 8);
  // 16 + code, from 256 + code for even p
  const uint32_t c = p & 1 ? and_or<0x4c004c00u>(u, m.hi) : add_h2(and_or<0x5c005c00u>(u, m.lo), 0xdb80db80u);
  return fma_h2(c, s2, z2);
}

// The low / high half-word of u in both halves.
__device__ __forceinline__ uint32_t dup_lo(uint32_t u) { return __byte_perm(u, u, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t u) { return __byte_perm(u, u, 0x3232); }

// A group's grid: s and z as stored (16 bits each), and what the codes are found with, in units of
// 2^-64, 1 or 2^64 so that neither s nor 1 / s leaves float32's range.
struct Grid {
  uint32_t s16, z16;
  float unit, s, z, r;          // s and z times the unit, and 1 / s, approximately
  bool clamp;                   // whether a code may leave 0 .. 15
};

// x / 15 rounded to float32 and then to the storage type, given as float: by a multiplication, except
// beside the storage type's rounding borders (the dropped bits within 2 units of halfway), where the
// division decides.
template <bool kKey>
__device__ __forceinline__ float fifteenth(float x) {
  float q = x * (1.0f / 15.0f);
  constexpr uint32_t kDropped = kKey ? 0xffffu : 0x1fffu, kHalf = (kDropped + 1) / 2;
  const bool plain = kKey ? q >= 1e-30f : q >= 6.2e-5f;      // above the storage type's subnormals
  if (!plain || (__float_as_uint(q) & kDropped) - (kHalf - 3u) <= 6u) q = __fdiv_rn(x, 15.0f);
  return q;
}

// lo or hi is a NaN or an infinity if the group holds one.
template <bool kKey>
__device__ __forceinline__ Grid make_grid(float lo, float hi) {
  Grid g;
  const float step = fifteenth<kKey>(__fsub_rn(hi, lo));
  if (kKey) {
    const __nv_bfloat16 s = __float2bfloat16_rn(step);
    g.s = __bfloat162float(s);
    const __nv_bfloat16 z = __float2bfloat16_rn(__fsub_rn(lo, 16.0f * g.s));
    g.z = __bfloat162float(z);
    g.s16 = __bfloat16_as_ushort(s);
    g.z16 = __bfloat16_as_ushort(z);
  } else {
    const __half s = __float2half_rn(step);
    g.s = __half2float(s);
    const __half z = __float2half_rn(__fsub_rn(lo, 16.0f * g.s));
    g.z = __half2float(z);
    g.s16 = __half_as_ushort(s);
    g.z16 = __half_as_ushort(z);
  }
  g.unit = 1.f;
  if (!(fabsf(g.z) < INFINITY && g.s >= 1e-30f && g.s <= 1e30f)) {
    if (!(fabsf(g.z) < INFINITY) || !(g.s < INFINITY)) {
      g.s = g.z = 0.f;                             // the offset makes every value NaN
      g.s16 = 0u;
      g.z16 = 0x7fffu;                             // NaN in bf16 and in fp16
    }
    if (g.s > 0.f) g.unit = g.s > 1.f ? 5.421010862427522e-20f : 18446744073709551616.f;
    g.s *= g.unit;
    g.z *= g.unit;
  }
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(g.r) : "f"(g.s));
  // only where the offset's rounding moved the grid past lo or hi; s = 0 (a NaN here) and huge s too
  g.clamp = !(g.unit >= 1.f && fmaf(lo, g.unit, -g.z) * g.r > 15.6f && fmaf(hi, g.unit, -g.z) * g.r < 31.4f);
  return g;
}

// Two float32 operations at a time, each rounded once.
struct Pair {
  float x, y;
};
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair d;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Low 16 bits of c[i]: the code of x[i], clamp(rint((x[i] - z) / s - 16), 0, 15), for finite x; the upper
// bits are constant. Without a division and without a branch on a border between two codes. With
// d = x - z (one rounding) and n the even number nearest to d / s, or the other one when d / s is
// nearly odd, e = d - n s is exact: n s has at most 16 bits, d and n s are multiples of d's last bit, and
// |e| < 2 s. The quotient is n + e / s, and since n is even a tie goes to n: it is n + rint(e r') with
// r' = (1 - 2^-21) / s up to 2^-22.4 of it. At a tie e r' is below 1/2; past a tie |e| is at least s / 2 plus one
// last bit of d, more than 2^-20.1 s as d >= 15.5 s, and e r' above 1/2. (Below 15.5 s, or above 31.5 s, the
// code is clamped.) Both sums with a large constant round to whole numbers, the first to even ones.
template <int kN>
__device__ __forceinline__ void codes_of(const float (&x)[kN], const Grid& g, uint32_t (&c)[kN]) {
  static_assert(kN % 2 == 0, "pairs of values");
  constexpr float kEven = 25165824.f;              // 1.5 * 2^24
  constexpr float kWhole = 12582912.f;             // 1.5 * 2^23
  constexpr float kBack = -(kEven - kWhole + 16.f);
  const float r1 = g.r * (1.f - 1.f / 2097152.f);
#pragma unroll
  for (int i = 0; i < kN; i += 2) {
    const Pair d = fma2({x[i], x[i + 1]}, {g.unit, g.unit}, {-g.z, -g.z});
    const Pair w = fma2(d, {g.r, g.r}, {kEven, kEven});
    const Pair n = add2(w, {-kEven, -kEven});
    const Pair e = fma2(n, {-g.s, -g.s}, d);
    const Pair q = fma2(e, {r1, r1}, add2(w, {kBack, kBack}));
    c[i] = __float_as_uint(q.x);
    c[i + 1] = __float_as_uint(q.y);
  }
  if (g.clamp) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      c[i] = __float_as_uint(fminf(fmaxf(__uint_as_float(c[i]), kWhole), kWhole + 15.f));
    if (g.unit < 1.f) {                            // x - z may be infinite: the last code
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (__fsub_rn(x[i], g.z / g.unit) == INFINITY) c[i] = __float_as_uint(kWhole + 15.f);
    }
  }
}

// Four results of codes_of as four nibbles in the low half, the first lowest; the high half is anything.
__device__ __forceinline__ uint32_t nibbles(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3) {
  return (c0 + (c1 << 4)) + ((c2 + (c3 << 4)) << 8);
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
