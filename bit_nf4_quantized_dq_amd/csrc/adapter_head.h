// The adapters' term of a GEMM whose rows each name their adapter, as the start of its
// accumulators: shared by the GEMMs whose wavefronts hold 32 TI features x 32 TJ tokens as tiles of
// MFMA 32x32x16 (gemm_nt.hip, adapters_gemm.hip).
#pragma once

#include "adapters_device.h"

namespace qlora {

typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16_t;

__device__ __forceinline__ f32x16_t mfma32(const bf16x8_t& a, const bf16x8_t& b, const f32x16_t& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// A tile of 16 ranks x 16 features in LDS, padded so that the tiles start at different banks; for
// W_a = A_a^T a wavefront needs 2 TI of them.
constexpr int kHeadTile = 16 * 32 + 32;

// acc[f][m] += sum_j W_a(f, j) scale s_a U[m][j],   a the adapter of token m,
// over the distinct adapters of the wavefront's tokens (features f0 .., tokens m0 ..), of which
// this call takes every nz-th from the z-th on.  Returns whether it took any.
//
// A step is 16 ranks of one adapter.  Its W rows come from memory as MFMA operands (B_a) or
// through the wavefront's own LDS with transposing reads (A_a [r, F]); U as hi and lo BF16 parts,
// zeros for tokens of other adapters.  Zero times an infinite weight would be NaN in their rows,
// so a step sums its products apart and adds them for its own tokens only.  The next step's loads
// are in flight during a step's MFMAs.
template <bool WT, int TI, int TJ>
__device__ __forceinline__ bool adapter_rows(const AdapterHead& h, int64_t F, int64_t f0, int64_t m0, int lane, char* lds,
                                             uint32_t z, uint32_t nz, f32x16_t (&acc)[TI][TJ]) {
  const int l32 = lane & 31, h32 = lane >> 5;
  const int width = h.rows.width;
  const rsrc_t ru = make_rsrc(h.U + m0 * width, (h.rows.M - m0) * width * 4);
  // each lane its tokens' adapters and what their table entries hold
  int id[TJ], rank[TJ];
  uint64_t base[TJ], pending[TJ];
  float scale[TJ];
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    id[j] = adapter_of(h.rows, m0 + 32 * j + l32);
    pending[j] = __ballot(id[j] >= 0);
    base[j] = 0, rank[j] = 0, scale[j] = 0.f;
    if (id[j] >= 0) {
      const AdapterEntry* e = h.rows.table + id[j];
      base[j] = reinterpret_cast<uint64_t>(WT ? e->A : e->B);
      rank[j] = e->r;
      scale[j] = e->s * h.scale;
    }
  }
  // the adapter at hand
  int cur = -1, r = 0, r0 = 0;
  uint64_t w_base = 0;
  float s = 0.f;
  uint32_t skip = z;
  const auto next_adapter = [&] {
    cur = -1;
    while (pending[0] | pending[TJ - 1]) {
      const bool second = !pending[0];
      const int from = __builtin_ctzll(second ? pending[TJ - 1] : pending[0]);
      const int a = __builtin_amdgcn_readlane(second ? id[TJ - 1] : id[0], from);
#pragma unroll
      for (int j = 0; j < TJ; ++j) pending[j] &= ~__ballot(id[j] == a);
      if (skip) {
        --skip;
        continue;
      }
      skip = nz - 1;
      cur = a;
      r0 = 0;
      r = __builtin_amdgcn_readlane(second ? rank[TJ - 1] : rank[0], from);
      w_base = readlane64(second ? base[TJ - 1] : base[0], from);
      s = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(second ? scale[TJ - 1] : scale[0]), from));
      return;
    }
  };
  uint4 w[TI], u[TJ][2];
  const auto load = [&] {
    // formed anew at each step, so that no tile's offsets are held in registers
    uint32_t lane_ = (uint32_t)lane;
    asm volatile("" : "+v"(lane_));
    const uint32_t l = lane_ & 31, hh = lane_ >> 5;
    const uint32_t at = (uint32_t)r0 + 8 * hh;
    if (WT) {
      const rsrc_t rw = make_rsrc(reinterpret_cast<const void*>(w_base), F * r * 2);
      // 4 TI lanes to a rank's features
      const uint32_t f = (uint32_t)f0 + 8 * (lane_ % (4 * TI));
#pragma unroll
      for (int q = 0; q < TI; ++q)
        w[q] = bload16(rw, f < F ? (((uint32_t)r0 + 16 / TI * q + lane_ / (4 * TI)) * (uint32_t)F + f) * 2 : kOOB);
    } else if (h.rows.whole) {
      const rsrc_t rw = make_rsrc(reinterpret_cast<const void*>(w_base), F * r * 2);
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const uint32_t f = (uint32_t)f0 + 32 * i + l;
        w[i] = bload16(rw, (f < F && (int)at < r) ? (f * r + at) * 2 : kOOB);
      }
    } else {
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const int64_t f = f0 + 32 * i + l;
        w[i] = load_row8(reinterpret_cast<const uint16_t*>(w_base), F * r, (f < F ? f : F - 1) * r, (int)at, r);
      }
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const uint32_t off = (id[j] == cur && (int)at < width) ? ((32 * j + l) * width + at) * 4 : kOOB;
      u[j][0] = bload16(ru, off);
      u[j][1] = bload16(ru, off == kOOB ? kOOB : off + 16);
    }
  };
  next_adapter();
  const bool any = cur >= 0;
  if (any) load();
  while (cur >= 0) {
    bf16x8_t wo[TI], hi[TJ], lo[TJ];
    bool mine[TJ];
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      mine[j] = id[j] == cur;
      const uint4 x = u[j][0], y = u[j][1];
      const float v[8] = {__uint_as_float(x.x) * s, __uint_as_float(x.y) * s, __uint_as_float(x.z) * s,
                          __uint_as_float(x.w) * s, __uint_as_float(y.x) * s, __uint_as_float(y.y) * s,
                          __uint_as_float(y.z) * s, __uint_as_float(y.w) * s};
      uint4 a, b;
      split_bf16(v, a, b);
      hi[j] = as_bf16x8(a), lo[j] = as_bf16x8(b);
    }
    if (WT) {
      // the wavefront's LDS accesses run in order
      asm volatile("" ::: "memory");
#pragma unroll
      for (int q = 0; q < TI; ++q)
        *reinterpret_cast<uint4*>(lds + (lane % (4 * TI) >> 1) * kHeadTile + (16 / TI * q + lane / (4 * TI)) * 32 +
                                  16 * (lane & 1)) = w[q];
      asm volatile("" ::: "memory");
#pragma unroll
      for (int i = 0; i < TI; ++i)
        wo[i] = tr_operand(lds + (2 * i + ((lane >> 4) & 1)) * kHeadTile, lane & 15, 8 * h32);
      asm volatile("" ::: "memory");
    } else {
#pragma unroll
      for (int i = 0; i < TI; ++i) wo[i] = as_bf16x8(w[i]);
    }
    r0 += 16;
    if (r0 >= r) next_adapter();
    if (cur >= 0) load();
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const bf16x8_t wl = finite_only(wo[i]);
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const f32x16_t t = mfma32(wl, lo[j], mfma32(wo[i], hi[j], f32x16_t{}));
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] += mine[j] ? t[q] : 0.f;
        __builtin_amdgcn_sched_barrier(0);  // one tile's temporaries at a time
      }
    }
  }
  return any;
}

// The mask over acc (the adapters' term): register 4q + v of tile (i, j) is element (m0 + 32 j +
// l32, f0 + 32 i + 8 q + 4 h32 + v), so the lanes l and l + 32 share the generator's blocks of
// eight: lane half h computes the block of q = 2p + h and the halves swap two of its four words.
template <int TI, int TJ>
__device__ __forceinline__ void drop_acc(const DropMask& drop, int64_t F, int64_t f0, int64_t m0, int l32, int h32,
                                         f32x16_t (&acc)[TI][TJ]) {
  const RngKey key = load_rng(drop.rng);
  const uint32_t t2 = threshold_halves(drop.threshold);
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    const uint64_t row = (uint64_t)(m0 + 32 * j + l32) * (uint64_t)(F / 8) + (uint64_t)(f0 / 8);
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint4 w = philox(key, row + (uint64_t)(4 * i + 2 * p + h32));
        // the upper half's first and the lower half's second argument change places
        const auto s0 = __builtin_amdgcn_permlane32_swap(w.x, w.z, false, false);
        const auto s1 = __builtin_amdgcn_permlane32_swap(w.y, w.w, false, false);
        const uint32_t k[4] = {keep_halves(s0[0], t2), keep_halves(s1[0], t2), keep_halves(s0[1], t2), keep_halves(s1[1], t2)};
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const uint32_t bits = (v & 1) ? k[2 * q + (v >> 1)] >> 16 : k[2 * q + (v >> 1)] & 0xFFFFu;
            const int at = 4 * (2 * p + q) + v;
            acc[i][j][at] = bits ? acc[i][j][at] : 0.f;
          }
        __builtin_amdgcn_sched_barrier(0);  // one block's words at a time
      }
  }
}

}  // namespace qlora
