// Device helpers of the training-step operators (norms, losses, gradients): eight consecutive
// elements of a row as FP32, at any element alignment, and sums over a workgroup in a fixed
// order.
#pragma once

#include "qlora_device.h"

namespace qlora {

// A row of odd width starts at any multiple of its element size.  gfx950 loads and stores
// 16 bytes from any address, so the types below only lower the alignment that the compiler
// may assume; the instructions are the same ones.
typedef uint32_t u32x4_e2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_e4 __attribute__((ext_vector_type(4), aligned(4)));

// ---- eight BF16 (uint16_t bit patterns) or eight FP32 elements, as loaded
template <class E>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  uint32_t w[4];
  __device__ __forceinline__ float get(int i) const {
    return (i & 1) ? bf16hi_to_f32(w[i >> 1]) : bf16lo_to_f32(w[i >> 1]);
  }
};
template <>
struct Raw8<float> {
  float f[8];
  __device__ __forceinline__ float get(int i) const { return f[i]; }
};

// The full vector at p.
__device__ __forceinline__ void load_all8(Raw8<uint16_t>& r, const uint16_t* __restrict__ p) {
  const u32x4_e2 v = *reinterpret_cast<const u32x4_e2*>(p);
  r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
}
__device__ __forceinline__ void load_all8(Raw8<float>& r, const float* __restrict__ p) {
  const f32x4_e4 a = *reinterpret_cast<const f32x4_e4*>(p), b = *reinterpret_cast<const f32x4_e4*>(p + 4);
  r.f[0] = a.x, r.f[1] = a.y, r.f[2] = a.z, r.f[3] = a.w;
  r.f[4] = b.x, r.f[5] = b.y, r.f[6] = b.z, r.f[7] = b.w;
}
// The same for an operand that is not read again soon.
__device__ __forceinline__ void stream_all8(Raw8<uint16_t>& r, const uint16_t* __restrict__ p) {
  const u32x4_e2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_e2*>(p));
  r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
}
__device__ __forceinline__ void stream_all8(Raw8<float>& r, const float* __restrict__ p) {
  const f32x4_e4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4_e4*>(p));
  const f32x4_e4 b = __builtin_nontemporal_load(reinterpret_cast<const f32x4_e4*>(p + 4));
  r.f[0] = a.x, r.f[1] = a.y, r.f[2] = a.z, r.f[3] = a.w;
  r.f[4] = b.x, r.f[5] = b.y, r.f[6] = b.z, r.f[7] = b.w;
}
__device__ __forceinline__ void zero8(Raw8<uint16_t>& r) { r.w[0] = r.w[1] = r.w[2] = r.w[3] = 0u; }
__device__ __forceinline__ void zero8(Raw8<float>& r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) r.f[i] = 0.f;
}
// Drops the first s (1..7) elements and appends zeros.
__device__ __forceinline__ void shift8(Raw8<uint16_t>& r, int s) {
  if (s & 4) r.w[0] = r.w[2], r.w[1] = r.w[3], r.w[2] = r.w[3] = 0u;
  if (s & 2) r.w[0] = r.w[1], r.w[1] = r.w[2], r.w[2] = r.w[3], r.w[3] = 0u;
  if (s & 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = (r.w[i] >> 16) | (i < 3 ? r.w[i + 1] << 16 : 0u);
  }
}
__device__ __forceinline__ void shift8(Raw8<float>& r, int s) {
#pragma unroll
  for (int k = 4; k >= 1; k >>= 1)
    if (s & k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r.f[i] = i + k < 8 ? r.f[i + k] : 0.f;
    }
}
__device__ __forceinline__ void set8(Raw8<uint16_t>& r, int i, uint16_t v) { r.w[i >> 1] |= (uint32_t)v << (16 * (i & 1)); }
__device__ __forceinline__ void set8(Raw8<float>& r, int i, float v) { r.f[i] = v; }

// Elements [0, n) of p, n in 0..8, zeros beyond them.  `wide`: the eight elements that end at
// p + n belong to the same row; a short vector is then one load of those and a shift (a load
// under a condition for each element would be waited for before the next one).
template <class E>
__device__ __forceinline__ void load8(Raw8<E>& r, const E* __restrict__ p, int n, bool wide) {
  if (n >= 8) {
    load_all8(r, p);
  } else {
    zero8(r);
    if (n > 0) {
      if (wide) {
        load_all8(r, p + (n - 8));
        shift8(r, 8 - n);
      } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
          if (i < n) set8(r, i, p[i]);
      }
    }
  }
}
// The first n (0..8) of f, rounded to the element type (nearest, ties to even).
__device__ __forceinline__ void store8(uint16_t* __restrict__ p, const float f[8], int n) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  if (n >= 8) {
    *reinterpret_cast<u32x4_e2*>(p) = u32x4_e2{w[0], w[1], w[2], w[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint16_t)((i & 1) ? (w[i >> 1] >> 16) : (w[i >> 1] & 0xFFFFu));
  }
}
__device__ __forceinline__ void store8(float* __restrict__ p, const float f[8], int n) {
  if (n >= 8) {
    *reinterpret_cast<f32x4_e4*>(p) = f32x4_e4{f[0], f[1], f[2], f[3]};
    *reinterpret_cast<f32x4_e4*>(p + 4) = f32x4_e4{f[4], f[5], f[6], f[7]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = f[i];
  }
}

// store8 for results that are not read again soon.
__device__ __forceinline__ void stream8(uint16_t* __restrict__ p, const float f[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  __builtin_nontemporal_store(u32x4_e2{w[0], w[1], w[2], w[3]}, reinterpret_cast<u32x4_e2*>(p));
}
__device__ __forceinline__ void stream8(float* __restrict__ p, const float f[8]) {
  __builtin_nontemporal_store(f32x4_e4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f32x4_e4*>(p));
  __builtin_nontemporal_store(f32x4_e4{f[4], f[5], f[6], f[7]}, reinterpret_cast<f32x4_e4*>(p + 4));
}

// ---- a lane's eight columns of a row of d >= 8: [8 lane, 8 lane + 8), and from the row's end on
// the row's last eight columns.  Every load and store is then a whole vector of the row without
// a branch, which lets the compiler count what is in flight (behind a branch it waits for all
// of it).  Columns that several lanes hold count once in sums (own()); each of the lanes stores
// them, with the same bits.
// SHORT: d < 8, in the first lane, element by element.
template <bool SHORT>
struct Columns {
  uint32_t at;  // first column of the vector
  int n;        // the lane's own columns: the last n of the eight (SHORT: the first n)
  __device__ __forceinline__ Columns(int d, uint32_t e) {
    const int left = d - (int)e;
    n = left < 0 ? 0 : (left > 8 ? 8 : left);
    at = SHORT || n == 8 ? e : (uint32_t)(d - 8);
  }
  // The vector's place in a row; asked for anew at each use, so that no address of a later use
  // is held in registers.
  __device__ __forceinline__ uint32_t place() const {
    uint32_t o = at;
    asm volatile("" : "+v"(o));
    return o;
  }
  template <class E>
  __device__ __forceinline__ void load(Raw8<E>& r, const E* __restrict__ row) const {
    if constexpr (SHORT) load8(r, row + at, n, false);
    else load_all8(r, row + place());
  }
  template <class E>
  __device__ __forceinline__ void store(E* __restrict__ row, const float f[8]) const {
    store8(row + place(), f, SHORT ? n : 8);
  }
  // Zeros where the column is another lane's.
  __device__ __forceinline__ Raw8<uint16_t> own(Raw8<uint16_t> r) const {
    if (!SHORT && n < 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (2 * i < 8 - n) r.w[i] &= 0xFFFF0000u;
        if (2 * i + 1 < 8 - n) r.w[i] &= 0x0000FFFFu;
      }
    }
    return r;
  }
  __device__ __forceinline__ Raw8<float> own(Raw8<float> r) const {
    if (!SHORT && n < 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < 8 - n) r.f[i] = 0.f;
    }
    return r;
  }
};

// The columns of an operand that (STREAM) is not read again soon.
template <bool STREAM, bool SHORT, class E>
__device__ __forceinline__ void load_in(const Columns<SHORT>& col, Raw8<E>& r, const E* __restrict__ row) {
  if constexpr (SHORT || !STREAM) col.load(r, row);
  else stream_all8(r, row + col.place());
}

__device__ __forceinline__ void and8(Raw8<uint16_t>& r, uint32_t bits) {
#pragma unroll
  for (int i = 0; i < 4; ++i) r.w[i] &= bits;
}
__device__ __forceinline__ void and8(Raw8<float>& r, uint32_t bits) {
#pragma unroll
  for (int i = 0; i < 8; ++i) r.f[i] = __uint_as_float(__float_as_uint(r.f[i]) & bits);
}

// Eight ones, for a weight that is not given.
__device__ __forceinline__ void ones8(Raw8<uint16_t>& r) { r.w[0] = r.w[1] = r.w[2] = r.w[3] = 0x3F803F80u; }

// Hides from the compiler that r keeps its value, so that nothing derived from it is held in
// registers across the point.
__device__ __forceinline__ void opaque(Raw8<uint16_t>& r) {
  asm volatile("" : "+v"(r.w[0]), "+v"(r.w[1]), "+v"(r.w[2]), "+v"(r.w[3]));
}
__device__ __forceinline__ void opaque(Raw8<float>& r) {
  asm volatile("" : "+v"(r.f[0]), "+v"(r.f[1]), "+v"(r.f[2]), "+v"(r.f[3]), "+v"(r.f[4]), "+v"(r.f[5]), "+v"(r.f[6]),
               "+v"(r.f[7]));
}

__device__ __forceinline__ float to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float to_f32(float f) { return f; }
__device__ __forceinline__ uint16_t bf16_of(float f) { return (uint16_t)(pack_bf16x2(f, 0.f) & 0xFFFFu); }

// Clipping coefficient of a global gradient norm; a norm that is NaN gives NaN.
__device__ __forceinline__ float clip_coefficient(float norm, float max_norm) {
  const float c = max_norm / (norm + 1e-6f);
  return c >= 1.f ? 1.f : c;
}

// Sum over each row of 16 lanes, the same in them all.
__device__ __forceinline__ float row_sum(float v) {
  v += dpp_partner<0xB1>(v);   // quad_perm [1, 0, 3, 2]
  v += dpp_partner<0x4E>(v);   // quad_perm [2, 3, 0, 1]
  v += dpp_partner<0x141>(v);  // row_half_mirror
  v += dpp_partner<0x140>(v);  // row_mirror
  return v;
}

// ---- sums of N values over a workgroup of up to 16 wavefronts (ONE: a single one), the same in
// every thread: each wavefront, then the wavefronts' sums as a row of lanes.  `lds` holds 16 N
// floats; a caller that sums again without a barrier of its own in between gives the next call
// another array.
template <bool ONE, int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* lds) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (!ONE) {
    const int slot = threadIdx.x & 15, waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) lds[i * 16 + (threadIdx.x >> 6)] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = row_sum(slot < waves ? lds[i * 16 + slot] : 0.f);
  }
}

// The same for one FP64 value; `lds` holds T / 64 doubles, and the caller separates two calls
// on one array by a barrier.
template <int T>
__device__ __forceinline__ double block_sum_f64(double v, double* lds) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  if constexpr (T > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[wave] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < T / 64; ++w) v += lds[w];
  }
  return v;
}

}  // namespace qlora
