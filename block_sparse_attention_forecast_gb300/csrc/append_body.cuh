// Compressed-key maintenance: storing a decode token's key/value and the mean-pooled keys of
// windows of kernel 32 / stride 16 (the inference-time key compression window of the
// techwalker article, section 四), one token at a time (decode).
//
// A window mean is the exact mean of 32 bf16 keys rounded once to bf16 (nearest, ties to
// even). The decode append sums each dimension exactly in a 64-bit fixed-point integer with
// 47 fractional bits and rounds that integer directly: every bf16 of magnitude in
// [2^-40, 2^11), and zero, converts without loss, and 32 of them cannot overflow. GB300
// issues float64 arithmetic at a small fraction of its integer rate, so the integer sum keeps
// the append short. A window holding any other value (a subnormal, a magnitude of 2^11 or
// more, a non-finite value) is summed in float64 instead, which is exact while its nonzero keys lie within a
// factor of 2^40 of one another, and rounded to bf16 without double rounding. (window_mean below, for the
// 4-bit cache and the eviction, is exact for every window.)
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace sparda {

// Key `tok` of sequence-group `bg`, for the resident cache or an offloaded layer (where
// block 0 and the two newest blocks live in the hot ring, older blocks in host memory).
__device__ __forceinline__ uint32_t load_key2(const __nv_bfloat16* k, const __nv_bfloat16* hot_k,
                                              int on_host, size_t bg, int max_ctx, int tb,
                                              int tok, int dim2) {
  const __nv_bfloat16* row;
  const int j = tok / kBlock;
  if (!on_host || !(j == 0 || j == tb || j == tb - 1)) {
    row = k + ((bg * max_ctx) + tok) * kHeadDim;
  } else {
    row = hot_k + ((bg * kHotSlots + hot_slot(j)) * kBlock + (tok % kBlock)) * kHeadDim;
  }
  return reinterpret_cast<const uint32_t*>(row)[dim2];
}

constexpr int kFixFrac = 47;          // fractional bits of the fixed-point window sums

// bf16 (given as its 16 bits) -> the integer x * 2^kFixFrac. Clears *in_range unless x is zero
// or of magnitude in [2^-40, 2^11) (biased exponent 87 .. 137), where the conversion is exact
// and the sum of 32 values stays below 2^63 in magnitude.
__device__ __forceinline__ long long bf16_to_fixed(uint32_t h, bool& in_range) {
  const int e = (int)((h >> 7) & 0xffu);
  const uint32_t m = h & 0x7fu;
  if (e == 0) {
    in_range = in_range && m == 0u;
    return 0;
  }
  in_range = in_range && e >= 87 && e <= 137;
  const int sh = min(max(e - 87, 0), 50);   // x = (128 + m) * 2^(e - 134)
  const long long v = (long long)(0x80u | m) << sh;
  return (h & 0x8000u) ? -v : v;
}

// bf16 bits of S * 2^-(kFixFrac + 5), rounded to nearest even: the mean of 32 values whose
// exact sum is S * 2^-kFixFrac (an exactly zero mean is +0).
__device__ __forceinline__ uint16_t fixed_mean_to_bf16(long long S) {
  if (S == 0) return 0u;
  const uint32_t sign = S < 0 ? 0x8000u : 0u;
  const unsigned long long A = S < 0 ? 0ull - (unsigned long long)S : (unsigned long long)S;
  const int p = 63 - __clzll((long long)A);      // A in [2^p, 2^(p+1))
  uint32_t m;                                    // the 8 leading bits, rounded: 128 .. 256
  if (p <= 7) {
    m = (uint32_t)(A << (7 - p));
  } else {
    const int sh = p - 7;
    m = (uint32_t)(A >> sh);
    const unsigned long long rem = A & ((1ull << sh) - 1ull), half = 1ull << (sh - 1);
    if (rem > half || (rem == half && (m & 1u))) ++m;
  }
  // the mean is (m / 128) * 2^(p - 52); its biased exponent p - 52 + 127 lies in 75 .. 137.
  // m = 256 (rounded up to the next power of two) carries into the exponent.
  return (uint16_t)(sign + ((uint32_t)(p + 75) << 7) + (m - 128u));
}

// The mean of 32 bf16 values of any magnitudes, exact, rounded once to bf16 (nearest, ties to even); with an
// infinity or a NaN among them what their sum is. The sum is an integer of 2^-133, the last bit of the smallest
// subnormal, in words of 32 bits that take 42 before they are carried. For the rare window: `half` 0 or 1
// of the 32 pairs at xs, in a loop over local memory.
inline __device__ __noinline__ uint32_t any_mean(const uint32_t* xs, int half) {
  constexpr int kWords = 9;                        // 254 + 8 + 5 bits
  long long acc[kWords] = {};
  float special = 0.f;
#pragma unroll 1
  for (int u = 0; u < kWinKernel; ++u) {
    const uint32_t h = half ? xs[u] >> 16 : xs[u] & 0xffffu;
    const int e = (int)((h >> 7) & 0xffu);
    if (e == 255) special += __uint_as_float(h << 16);
    const int at = max(e, 1) - 1;                  // x = m * 2^(at - 133)
    const long long v = (long long)((h & 0x7fu) | (e ? 0x80u : 0u)) << (at & 31);
    acc[at >> 5] += (h & 0x8000u) ? -v : v;
  }
  if (special != 0.f) return __bfloat16_as_ushort(__float2bfloat16_rn(special));
  // carried: the words are the sum modulo 2^288, whose sign is the last carry's
  long long carry = 0;
#pragma unroll 1
  for (int i = 0; i < kWords; ++i) {
    acc[i] += carry;
    carry = acc[i] >> 32;
    acc[i] &= 0xffffffffll;
  }
  const uint32_t sign = carry < 0 ? 0x8000u : 0u;
  if (sign) {
    carry = 1;
#pragma unroll 1
    for (int i = 0; i < kWords; ++i) {
      acc[i] = (~acc[i] & 0xffffffffll) + carry;
      carry = acc[i] >> 32;
      acc[i] &= 0xffffffffll;
    }
  }
  int top = kWords - 1;
  while (top > 0 && acc[top] == 0) --top;
  if (acc[top] == 0) return 0u;                    // an exactly zero mean is +0
  const int p = 32 * top + 31 - __clz((int)acc[top]);         // the sum is in [2^p, 2^(p+1)) times 2^-133
  // The mean is the sum times 2^-138. It keeps 8 leading bits, or (subnormal) what lies above 2^-133.
  const int cut = max(p - 7, 5);
  const auto bit = [&](int i) { return (uint32_t)(acc[i >> 5] >> (i & 31)) & 1u; };
  uint32_t m = 0u;
  for (int i = p; i >= cut; --i) m = 2u * m + bit(i);
  bool below = false;
#pragma unroll 1
  for (int i = 0; i < cut - 1 && !below; ++i) below = bit(i) != 0u;
  if (bit(cut - 1) && (below || (m & 1u))) ++m;
  // m = 256 carries into the exponent, and so does the subnormals' m = 128
  return sign + (p >= 12 ? ((uint32_t)(p - 11) << 7) + m - 128u : m);
}

// The exact sum of 32 bf16 values, as two float32 numbers hi + lo. amax: their largest magnitude,
// in [2^-64, 2^64). Each value is cut at u = 2^-12 of amax's power of two (adding and taking off 1.5 * 2^23 u
// rounds to multiples of u): the upper parts are multiples of u below 2^19 u in sum, the lower parts
// multiples of the smallest value's last bit and below 16 u in sum, so neither sum is ever rounded
// while no nonzero value is below 2^-24 amax.
__device__ __forceinline__ float2 exact_sum(const float (&x)[kWinKernel], float amax) {
  const float u = __uint_as_float((__float_as_uint(amax) & 0x7f800000u) - (12u << 23)), cut = 12582912.f * u;
  float hi = 0.f, lo = 0.f;
#pragma unroll
  for (int i = 0; i < kWinKernel; ++i) {
    const float h = __fsub_rn(__fadd_rn(x[i], cut), cut);
    hi += h;
    lo += __fsub_rn(x[i], h);
  }
  return make_float2(hi, lo);
}

// The mean of 32 bf16 pairs, per half-word, rounded once to bf16: a compression window's
// compressed key for two channels. A window of ordinary values is summed in float32 (exact_sum), at
// 8 instructions per value; one of the append's wide range in fixed point; any other by any_mean.
__device__ __forceinline__ uint32_t window_mean(const uint32_t (&xs)[kWinKernel]) {
  uint32_t top = 0u, low = 0xffffffffu;            // per half: largest magnitude, smallest nonzero one less 1
#pragma unroll
  for (int u = 0; u < kWinKernel; ++u) {
    const uint32_t m = xs[u] & 0x7fff7fffu;
    top = __vmaxu2(top, m);
    low = __vminu2(low, __vsub2(m, 0x00010001u));
  }
  const uint32_t t0 = top & 0xffffu, t1 = top >> 16, l0 = low & 0xffffu, l1 = low >> 16;
  // bf16 codes of 2^-64 and 2^64; a magnitude 24 powers of two down is a code 24 * 128 down
  const auto plain = [](uint32_t t, uint32_t l) { return t >= 0x1f80u && t < 0x5f80u && l + 24u * 128u >= t; };
  if (plain(t0, l0) && plain(t1, l1)) {
    uint32_t r[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float x[kWinKernel];
#pragma unroll
      for (int u = 0; u < kWinKernel; ++u) x[u] = half ? bf16_hi(xs[u]) : bf16_lo(xs[u]);
      const float2 s = exact_sum(x, __uint_as_float((half ? t1 : t0) << 16));
      // hi + lo rounded to odd, then to bf16: one rounding in all
      const float f = __fadd_rn(s.x, s.y);
      const float e = __fadd_rn(__fsub_rn(s.x, __fsub_rn(f, __fsub_rn(f, s.x))), __fsub_rn(s.y, __fsub_rn(f, s.x)));
      uint32_t bits = __float_as_uint(f);
      if (e != 0.f) {
        if ((e < 0.f) == (f > 0.f)) --bits;        // towards zero
        bits |= 1u;
      }
      r[half] = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(bits) * (1.f / kWinKernel)));
      if (f == 0.f && e == 0.f) r[half] = 0u;
    }
    return r[0] | (r[1] << 16);
  }
  bool in_range = true;
  long long S0 = 0, S1 = 0;
#pragma unroll
  for (int u = 0; u < kWinKernel; ++u) {
    S0 += bf16_to_fixed(xs[u] & 0xffffu, in_range);
    S1 += bf16_to_fixed(xs[u] >> 16, in_range);
  }
  if (in_range) return (uint32_t)fixed_mean_to_bf16(S0) | ((uint32_t)fixed_mean_to_bf16(S1) << 16);
  uint32_t ys[kWinKernel];                         // a copy, so that xs stays in registers
#pragma unroll
  for (int u = 0; u < kWinKernel; ++u) ys[u] = xs[u];
  return any_mean(ys, 0) | (any_mean(ys, 1) << 16);
}

// The append of sequence-group `bg` by 64 threads; thread t (0..63) owns dims 2t and 2t+1.
__device__ __forceinline__ void append_token(const AppendArgs& a, int bg, int t) {
  const int b = bg / a.G;
  const int T = a.seq_len[b];
  if (T < 1 || T > a.max_ctx) {
    if (t == 0) atomicOr(a.err, SPARDA_DEV_BAD_SEQ_LEN);
    return;
  }
  const int p = T - 1;
  const int tb = p / kBlock;
  const uint32_t kn = reinterpret_cast<const uint32_t*>(a.k_new + (size_t)bg * kHeadDim)[t];
  const uint32_t vn = reinterpret_cast<const uint32_t*>(a.v_new + (size_t)bg * kHeadDim)[t];
  if (!a.on_host) {
    const size_t off = ((size_t)bg * a.max_ctx + p) * kHeadDim;
    reinterpret_cast<uint32_t*>(a.k + off)[t] = kn;
    reinterpret_cast<uint32_t*>(a.v + off)[t] = vn;
  } else {
    const size_t off = (((size_t)bg * kHotSlots + hot_slot(tb)) * kBlock + p % kBlock) * kHeadDim;
    reinterpret_cast<uint32_t*>(a.hot_k + off)[t] = kn;
    reinterpret_cast<uint32_t*>(a.hot_v + off)[t] = vn;
  }
  if (T >= kWinKernel && (T - kWinKernel) % kWinStride == 0) {
    const int i = (T - kWinKernel) / kWinStride;
    uint32_t xs[kWinKernel - 1];           // all loads in flight before the sums
#pragma unroll
    for (int u = 0; u < kWinKernel - 1; ++u)
      xs[u] = load_key2(a.k, a.hot_k, a.on_host, bg, a.max_ctx, tb, T - kWinKernel + u, t);
    bool in_range = true;
    long long S0 = bf16_to_fixed(kn & 0xffffu, in_range), S1 = bf16_to_fixed(kn >> 16, in_range);
#pragma unroll
    for (int u = 0; u < kWinKernel - 1; ++u) {
      S0 += bf16_to_fixed(xs[u] & 0xffffu, in_range);
      S1 += bf16_to_fixed(xs[u] >> 16, in_range);
    }
    uint32_t packed;
    if (in_range) {
      packed = (uint32_t)fixed_mean_to_bf16(S0) | ((uint32_t)fixed_mean_to_bf16(S1) << 16);
    } else {
      double s0 = 0.0 + bf16_lo(kn), s1 = 0.0 + bf16_hi(kn);    // an all-zero window gives +0
#pragma unroll
      for (int u = 0; u < kWinKernel - 1; ++u) {
        s0 += bf16_lo(xs[u]);
        s1 += bf16_hi(xs[u]);
      }
      const __nv_bfloat16 b0 = f64_to_bf16_rn(s0 / kWinKernel), b1 = f64_to_bf16_rn(s1 / kWinKernel);
      packed = (uint32_t)__bfloat16_as_ushort(b0) | ((uint32_t)__bfloat16_as_ushort(b1) << 16);
    }
    reinterpret_cast<uint32_t*>(a.ck + ((size_t)bg * a.W_cap + i) * kHeadDim)[t] = packed;
  }
  // Offloaded layer: a block that just filled is written to the host cache, so that a
  // gather issued at a later step finds it there. Each thread copies its own two dims of
  // the 64 rows, which it wrote itself at earlier steps or just now.
  if (a.on_host && T % kBlock == 0) {
    const size_t src = ((size_t)bg * kHotSlots + hot_slot(tb)) * kBlock * kHeadDim;
    const size_t dst = ((size_t)bg * a.max_ctx + (size_t)tb * kBlock) * kHeadDim;
    const uint32_t* hk = reinterpret_cast<const uint32_t*>(a.hot_k + src);
    const uint32_t* hv = reinterpret_cast<const uint32_t*>(a.hot_v + src);
    uint32_t* ck = reinterpret_cast<uint32_t*>(a.k + dst);
    uint32_t* cv = reinterpret_cast<uint32_t*>(a.v + dst);
    for (int r = 0; r < kBlock; ++r) {
      ck[r * (kHeadDim / 2) + t] = hk[r * (kHeadDim / 2) + t];
      cv[r * (kHeadDim / 2) + t] = hv[r * (kHeadDim / 2) + t];
    }
  }
}

}  // namespace sparda
