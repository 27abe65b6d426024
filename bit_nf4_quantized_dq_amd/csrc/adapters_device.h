// Device helpers of the operators with many adapters and with dropout: the counter-based
// generator, its masks, and FP32 values as pairs of BF16.
#pragma once

#include "qlora_adapters_host.h"
#include "qlora_device.h"

namespace qlora {

// ---- Philox4x32, ten rounds (Salmon et al. 2011): each round multiplies two of the four counter
// words by constants and mixes the halves of the 64-bit products with the others and the key,
// whose words step by the golden ratio and sqrt(3) - 1.
struct RngKey {
  uint32_t k0, k1, c2, c3;  // seed, offset
};
__device__ __forceinline__ RngKey load_rng(const uint64_t* __restrict__ rng) {
  const uint64_t seed = rng[0], offset = rng[1];
  const auto scalar = [](uint64_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v); };
  return RngKey{scalar(seed), scalar(seed >> 32), scalar(offset), scalar(offset >> 32)};
}
__device__ __forceinline__ uint4 philox(const RngKey& key, uint64_t block) {
  uint32_t a = (uint32_t)block, b = (uint32_t)(block >> 32), c = key.c2, d = key.c3;
  uint32_t k0 = key.k0, k1 = key.k1;
  // the round keys are scalar additions: formed anew, they take no registers between calls
  asm volatile("" : "+s"(k0), "+s"(k1));
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t x = (uint64_t)a * 0xD2511F53u, y = (uint64_t)c * 0xCD9E8D57u;
    a = (uint32_t)(y >> 32) ^ b ^ k0;
    b = (uint32_t)y;
    c = (uint32_t)(x >> 32) ^ d ^ k1;
    d = (uint32_t)x;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(a, b, c, d);
}
// 0xFFFF in each 16-bit half of w that is at least the threshold t (1..65535, in both halves of
// t2): the saturated difference to t - 1 is zero below it, then one or more.
__device__ __forceinline__ uint32_t keep_halves(uint32_t w, uint32_t t2) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  const u16x2 one = {1, 1}, zero = {0, 0};
  const u16x2 over = __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, w), __builtin_bit_cast(u16x2, t2));
  return __builtin_bit_cast(uint32_t, (u16x2)(zero - __builtin_elementwise_min(over, one)));
}
// t2 of keep_halves for threshold t
__device__ __forceinline__ uint32_t threshold_halves(uint32_t t) { return (t - 1u) * 0x00010001u; }

// Eight BF16 elements 8 block .. 8 block + 7 with the dropped ones zero.
__device__ __forceinline__ uint4 drop8(uint4 v, const RngKey& key, uint64_t block, uint32_t t2) {
  const uint4 w = philox(key, block);
  return make_uint4(v.x & keep_halves(w.x, t2), v.y & keep_halves(w.y, t2), v.z & keep_halves(w.z, t2),
                    v.w & keep_halves(w.w, t2));
}

// ---- FP32 values as hi + lo of BF16: sixteen bits of significand, so that a product on the
// matrix cores loses 2^-17 of the value instead of 2^-9.  An infinite value has lo = 0.
__device__ __forceinline__ void split_bf16(const float f[8], uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    float a = f[2 * i] - bf16lo_to_f32(h[i]), b = f[2 * i + 1] - bf16hi_to_f32(h[i]);
    a = fabsf(a) <= 3.4e38f ? a : 0.f;
    b = fabsf(b) <= 3.4e38f ? b : 0.f;
    l[i] = pack_bf16x2(a, b);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Row m's adapter, -1 for none (also past the rows).
__device__ __forceinline__ int adapter_of(const AdapterRows& rows, int64_t m) {
  if (m >= rows.M) return -1;
  const int id = rows.ids ? rows.ids[m] : 0;
  return (uint32_t)id < (uint32_t)rows.count ? id : -1;
}

}  // namespace qlora
