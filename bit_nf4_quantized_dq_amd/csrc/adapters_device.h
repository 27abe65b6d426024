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

// ---- FP32 values as hi + lo of BF16, so that a product on the matrix cores loses little of them: hi is
// off by at most half a step, 2^-8 of the value, and lo, which is that difference, by half a step
// of its own, 2^-17 of the value.  An infinite value has lo = 0, and one that rounds past BF16's
// largest (3.39e38) counts as infinite.
//
// Times an infinite operand, hi gives the infinity (or NaN) of the whole product, and lo, whose sign
// is its own, must not: lo meets an operand without its infinities and NaN (finite_only()).
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

// The larger of each half of `most` and of the magnitudes of the BF16 values of w.
__device__ __forceinline__ uint32_t most_halves(uint32_t most, uint32_t w) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, most), __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu)));
}
__device__ __forceinline__ uint32_t most_halves(uint32_t most, const uint4& v) {
  return most_halves(most_halves(most_halves(most_halves(most, v.x), v.y), v.z), v.w);
}
// Whether some lane's magnitudes reach infinity (or NaN); the same for the whole wavefront.
__device__ __forceinline__ bool some_not_finite(uint32_t most) {
  return __ballot(most >= 0x7F800000u || (most & 0xFFFFu) >= 0x7F80u) != 0;
}
// Eight BF16 values, zeros for those that are not finite.
__device__ __forceinline__ bf16x8_t finite_only(const bf16x8_t& v) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  const u16x2 one = {1, 1}, most = {0x7F7F, 0x7F7F};
  const uint4 u = __builtin_bit_cast(uint4, v);
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u16x2 over = __builtin_elementwise_sub_sat(__builtin_bit_cast(u16x2, w[i] & 0x7FFF7FFFu), most);
    w[i] = __builtin_bit_cast(uint32_t, (u16x2)(__builtin_bit_cast(u16x2, w[i]) * __builtin_elementwise_sub_sat(one, over)));
  }
  return as_bf16x8(make_uint4(w[0], w[1], w[2], w[3]));
}

// ---- operands
// block_scale() by the chip's own conversion of OCP E4M3 (exact, and no branch): stored codes hold no
// NaN.
__device__ __forceinline__ float stored_scale(uint32_t code8, float c2s, float mu) {
  return __fadd_rn(__fmul_rn(__builtin_amdgcn_cvt_f32_fp8((int)code8, 0), c2s), mu);
}

typedef short lds_i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) lds_i16x4 lds_i16x4_t;

// 8 consecutive rows k .. k + 7 of column i (0..15) of an LDS tile of BF16 rows of 32 bytes, by two
// transposing reads (as in lora.hip: within 16 lanes, lane i receives element i % 4 of the 8
// bytes that lanes i/4, i/4 + 4, i/4 + 8, i/4 + 12 address).
__device__ __forceinline__ bf16x8_t tr_operand(const char* tile, int i, int k) {
  const char* p0 = tile + (k + (i >> 2)) * 32 + 8 * (i & 3);
  const lds_i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(p0));
  const lds_i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(p0 + 4 * 32));
  bf16x8_t r;
  r[0] = lo[0]; r[1] = lo[1]; r[2] = lo[2]; r[3] = lo[3];
  r[4] = hi[0]; r[5] = hi[1]; r[6] = hi[2]; r[7] = hi[3];
  return r;
}

__device__ __forceinline__ uint64_t readlane64(uint64_t v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
  return ((uint64_t)hi << 32) | lo;
}

// Elements at .. at + 7 of a row that starts at `row` of a matrix of `total` BF16 (at least 8) and
// has n: zeros from n on.  Rows of any width, so the vector may start at any element; near the
// matrix's end it starts early enough to stay inside and is shifted.
__device__ __forceinline__ uint4 load_row8(const uint16_t* __restrict__ p, int64_t total, int64_t row, int at, int n) {
  typedef uint32_t u32x4_e2 __attribute__((ext_vector_type(4), aligned(2)));
  const int left = n - at;  // elements of the row
  const int64_t first = row + (left > 0 ? at : 0), start = first < total - 8 ? first : total - 8;
  u32x4_e2 v = *reinterpret_cast<const u32x4_e2*>(p + start);
  const int shift = (int)(first - start);
  if (__ballot(shift)) {
    uint64_t a = ((uint64_t)v.y << 32) | v.x, b = ((uint64_t)v.w << 32) | v.z;
    const int bits = 16 * shift;
    if (bits >= 64) a = b >> (bits - 64), b = 0;
    else if (bits) a = (a >> bits) | (b << (64 - bits)), b >>= bits;
    v.x = (uint32_t)a, v.y = (uint32_t)(a >> 32), v.z = (uint32_t)b, v.w = (uint32_t)(b >> 32);
  }
  const auto keep = [&](int i) { return left >= 2 * i + 2 ? ~0u : (left == 2 * i + 1 ? 0xFFFFu : 0u); };
  return make_uint4(v.x & keep(0), v.y & keep(1), v.z & keep(2), v.w & keep(3));
}

// ---- partial sums between workgroups: stores and loads that pass the caches, 8 bytes each
__device__ __forceinline__ void store_partial(float* to, const f32x4_t& v) {
  uint64_t* p = reinterpret_cast<uint64_t*>(to);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    __hip_atomic_store(p + i, ((uint64_t)__float_as_uint(v[2 * i + 1]) << 32) | __float_as_uint(v[2 * i]), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_SYSTEM);
}
__device__ __forceinline__ f32x4_t load_partial(const float* from) {
  const uint64_t* p = reinterpret_cast<const uint64_t*>(from);
  const uint64_t a = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
  const uint64_t b = __hip_atomic_load(p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
  return f32x4_t{__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)(a >> 32)), __uint_as_float((uint32_t)b),
                 __uint_as_float((uint32_t)(b >> 32))};
}

// Row m's adapter, -1 for none (also past the rows).
__device__ __forceinline__ int adapter_of(const AdapterRows& rows, int64_t m) {
  if (m >= rows.M) return -1;
  const int id = rows.ids ? rows.ids[m] : 0;
  return (uint32_t)id < (uint32_t)rows.count ? id : -1;
}

}  // namespace qlora
