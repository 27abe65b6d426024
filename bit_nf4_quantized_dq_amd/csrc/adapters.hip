// The kernels of a frozen linear with many adapters ("QLoRA -- Fine-Tuning a 65B Model on One
// GPU", "Prerequisite: LoRA's low-rank update": one shared frozen base, small pairs A, B beside
// it): each row m of a batch names its adapter a = ids[m].
//
// shrink : T[m] = drop(X[m]) A_a^T  and  G[m] = dY[m] B_a           (FP32 [M, width])
// stream : Y = X w_hat^T + s_a T B_a^T for few rows, the weight decoded as it is read
// grads  : dA_a = s_a sum of G[m]^T drop(X[m]),  dB_a = s_a sum of dY[m]^T T[m]
// (more rows' Y, and dX: adapters_gemm.hip and gemm_nt.hip)
//
// Rows come in any order.  A workgroup finds the distinct adapters of its rows by ballots, loads
// each one's operand once and takes the result for the rows that name it: a select, not a
// multiplication by zero, so that an adapter with infinite values reaches its own rows only.
#include "adapters_device.h"
#include "decode_tiles.h"

namespace qlora {
namespace {

__device__ __forceinline__ int lowest(uint64_t mask) { return __builtin_ctzll(mask); }

// ---------------------------------------------------------------- the table
__global__ __launch_bounds__(128) void k_adapter_table(AdapterBatch batch, int count, AdapterEntry* __restrict__ table) {
  const int i = threadIdx.x;
  if (i < count) table[i] = batch.e[i];
}

// ---------------------------------------------------------------- T and G
constexpr int kShrinkThreads = 512;
constexpr int kShrinkWaves = kShrinkThreads / 64;
constexpr int kRowTile = 16;

struct ShrinkArgs {
  AdapterRows rows;
  const uint16_t* P;  // X [M, Kd] or dY
  int64_t Kd;
  DropMask drop;
  float* out;  // [M, width]
  float* part;
  unsigned int* counters;
  int32_t split;
};

// One workgroup per 16 rows and slice of the reduction.  An item is 64 columns (or rows of B) of the
// slice for one of the rows' adapters; the wavefronts take the items in turn, D in flight each.
// JT: 16-rank tiles.  QT: the operand is B_a [Kd, r], else A_a [r, Kd].  Rows of X (dY) and A come in
// whole cache lines and pass through the wavefront's own LDS into operand order, chunks laid as in
// the stream below (straight into operand order, where neighbouring lanes are in 16 rows, the
// address unit bounds the loads: 8192 rows over 14336 columns 91 us, so 76).  Bound by HBM for many rows
// (those 76 us: 235 MB of dY, and 147 MB of the decode beside it), by A's rows through the L2 where a
// tile's rows name many adapters or ranks (256 rows of 48 adapters over 14336 columns 20 us for 103 MB).
template <int JT>
struct ShrinkLds {
  uint4 tiles[kShrinkWaves][(1 + JT) * 128];  // (no byte more: two of 80 KB, JT = 4, fill a compute unit)
};
template <int JT, bool QT, bool DROP, bool VEC, int D>
__device__ __forceinline__ void shrink_body(const ShrinkArgs& a, uint32_t wg, ShrinkLds<JT>& lds) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const uint32_t split = (uint32_t)a.split, tile = wg / split, slice = wg - tile * split;
  const int64_t m0 = (int64_t)tile * kRowTile, M = a.rows.M, Kd = a.Kd, width = a.rows.width;
  // each lane its row's adapter; the four groups of 16 lanes hold the same rows
  const int id = adapter_of(a.rows, m0 + l16);
  uint64_t base = 0;
  int rank = 0;
  if (id >= 0) {
    const AdapterEntry* e = a.rows.table + id;
    base = reinterpret_cast<uint64_t>(QT ? e->B : e->A);
    rank = e->r;
  }
  RngKey key{};
  uint32_t t2 = 0;
  if (DROP) key = load_rng(a.drop.rng), t2 = threshold_halves(a.drop.threshold);
  const rsrc_t rp = make_rsrc(a.P + m0 * Kd, (M - m0) * Kd * 2);
  const uint64_t block0 = (uint64_t)(m0 + l16) * (uint64_t)(Kd / 8);

  const int nblk = (int)((Kd + 63) / 64), per = (nblk + (int)split - 1) / (int)split;
  const int sbeg = (int)slice * per, send = sbeg + per < nblk ? sbeg + per : nblk, len = send - sbeg;
  f32x4_t acc[JT];
#pragma unroll
  for (int t = 0; t < JT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  uint4* xs = lds.tiles[wave];
  uint4* qs = xs + 128;

  uint64_t pending = __ballot(id >= 0);
  int cur = -1, at = wave;  // the adapter's lane, the block within the slice
  if (len > 0 && pending) {
    cur = lowest(pending);
    const auto step = [&](int by) {  // to the item `by` further on
      at += by;
      while (cur >= 0 && at >= len) {
        at -= len;
        pending &= ~__ballot(id == __builtin_amdgcn_readlane(id, cur));
        cur = pending ? lowest(pending) : -1;
      }
    };
    step(0);
    while (cur >= 0) {
      uint4 pv[D][2], qv[D][JT][2];
      int which[D], blk[D];
#pragma unroll
      for (int d = 0; d < D; ++d) {
        which[d] = -2;
        if (cur < 0) continue;
        which[d] = __builtin_amdgcn_readlane(id, cur);
        blk[d] = sbeg + at;
        const int r = __builtin_amdgcn_readlane(rank, cur);
        const uint64_t rows_mine = __ballot(id == which[d]);  // bit m: row m of the tile
        const rsrc_t rq = make_rsrc(reinterpret_cast<const void*>(readlane64(base, cur)), (int64_t)r * Kd * 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 8 * i + (lane >> 3), chunk = (lane & 7) ^ ((4 * i + (lane >> 4)) & 7);
          const int64_t k = 64 * (int64_t)blk[d] + 8 * chunk;
          pv[d][i] = bload16(rp, (k < Kd && ((rows_mine >> row) & 1)) ? (uint32_t)((row * Kd + k) * 2) : kOOB);
          if (!QT) {
#pragma unroll
            for (int t = 0; t < JT; ++t) {
              const int j = 16 * t + row;
              qv[d][t][i] = bload16(rq, (k < Kd && j < r) ? (uint32_t)((j * Kd + k) * 2) : kOOB);
            }
          } else {
            // rows 64 blk + 32 i + (lane >> 1), columns 8 (lane & 1) .. +7 of every tile
            const int64_t kr = 64 * (int64_t)blk[d] + 32 * i + (lane >> 1);
#pragma unroll
            for (int t = 0; t < JT; ++t) {
              const int j = 16 * t + 8 * (lane & 1);
              if (VEC)
                qv[d][t][i] = bload16(rq, (kr < Kd && j < r) ? (uint32_t)((kr * r + j) * 2) : kOOB);
              else  // zeros past the rows (in the reduction, dY's zeros there would not do beside an infinity)
                qv[d][t][i] = load_row8(reinterpret_cast<const uint16_t*>(readlane64(base, cur)), Kd * r, (kr < Kd ? kr : Kd - 1) * r, j,
                                        kr < Kd ? r : 0);
            }
          }
        }
        step(kShrinkWaves);
      }
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (which[d] == -2) break;  // no more items
        const bool mine = id == which[d];
        // the wavefront's LDS tiles are reused item after item; its LDS accesses run in order
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          xs[64 * i + lane] = pv[d][i];
#pragma unroll
          for (int t = 0; t < JT; ++t) qs[128 * t + 64 * i + lane] = qv[d][t][i];
        }
        asm volatile("" ::: "memory");
        f32x4_t v[JT];
#pragma unroll
        for (int t = 0; t < JT; ++t) v[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int chunk = 8 * l16 + ((4 * h + g) ^ (l16 >> 1));
          uint4 p = xs[chunk];
          if (DROP) p = drop8(p, key, block0 + (uint64_t)(8 * blk[d] + 4 * h + g), t2);
#pragma unroll
          for (int t = 0; t < JT; ++t)
            v[t] = mfma16x16x32(QT ? tr_operand(reinterpret_cast<const char*>(qs + 128 * t + 64 * h), l16, 8 * g)
                                   : as_bf16x8(qs[128 * t + chunk]),
                                as_bf16x8(p), v[t]);
        }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int t = 0; t < JT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][i] += mine ? v[t][i] : 0.f;
      }
    }
  }
  // fixed-order sum over the wavefronts; D[j][m]: lane l holds ranks 4 (l >> 4) + v of row l & 15
  __syncthreads();
  f32x4_t* red = reinterpret_cast<f32x4_t*>(&lds.tiles[0][0]);
#pragma unroll
  for (int t = 0; t < JT; ++t) red[(wave * JT + t) * 64 + lane] = acc[t];
  __syncthreads();
  const int64_t m = m0 + l16;
  const float keep = DROP ? a.drop.scale : 1.f;
  for (int t = wave; t < JT; t += kShrinkWaves) {
    f32x4_t sum = red[t * 64 + lane];
    for (int w = 1; w < kShrinkWaves; ++w) {
      const f32x4_t v = red[(w * JT + t) * 64 + lane];
      sum[0] += v[0]; sum[1] += v[1]; sum[2] += v[2]; sum[3] += v[3];
    }
    const int j = 16 * t + 4 * g;
    if (m >= M || j >= width) continue;
    if (split == 1) {
#pragma unroll
      for (int v = 0; v < 4; ++v) sum[v] = j + v < rank ? sum[v] * keep : 0.f;
      *reinterpret_cast<f32x4_t*>(a.out + m * width + j) = sum;
    } else {
      store_partial(a.part + ((int64_t)slice * M + m) * width + j, sum);
    }
  }
  if (split == 1) return;
  // every partial store of this workgroup has completed before its counter increment
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned int old = __hip_atomic_fetch_add(&a.counters[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    lds.tiles[0][0].x = old + 1u == split;  // (the sums are read)
    if (old + 1u == split) __hip_atomic_store(&a.counters[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!lds.tiles[0][0].x) return;
  for (int t = wave; t < JT; t += kShrinkWaves) {
    const int j = 16 * t + 4 * g;
    if (m >= M || j >= width) continue;
    f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
    for (uint32_t s0 = 0; s0 < split; s0 += 8) {
      f32x4_t v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = s0 + u < split ? load_partial(a.part + ((int64_t)(s0 + u) * M + m) * width + j) : f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += v[u][i];
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) sum[v] = j + v < rank ? sum[v] * keep : 0.f;
    *reinterpret_cast<f32x4_t*>(a.out + m * width + j) = sum;
  }
}

// T or G; workgroups from n_shrink on decode the weight beside it (w_hat, or w_hat^T beside G).
template <int JT, bool QT, bool DROP, bool VEC, int D>
__global__ __launch_bounds__(kShrinkThreads) void k_adapter_shrink(ShrinkArgs a, ShrinkDecode dec, uint32_t n_shrink,
                                                                   Nf4Tables tab) {
  __shared__ ShrinkLds<JT> lds;
  if (blockIdx.x < n_shrink) {
    shrink_body<JT, QT, DROP, VEC, D>(a, blockIdx.x, lds);
  } else if (!QT) {
    decode_words<kDqE4M3, kShrinkThreads>(dec.codes, dec.code8, dec.c2s, dec.mu, reinterpret_cast<uint4*>(dec.out),
                                          (int64_t)(blockIdx.x - n_shrink), threadIdx.x, dec.N * dec.K / 8, tab);
  } else {
    const uint32_t groups_k = (uint32_t)((dec.K / 64 + kShrinkWaves - 1) / kShrinkWaves);
    const uint32_t grp = blockIdx.x - n_shrink, gn = grp / groups_k;
    decode_pairs_t<kDqE4M3, kShrinkThreads>(dec.codes, dec.code8, dec.c2s, dec.mu, dec.out, dec.N, dec.K, tab, (int64_t)gn,
                                            (int64_t)(grp - gn * groups_k), threadIdx.x);
  }
}
// T and G in one launch: they are independent, and few rows fill the chip with neither (555 rows of 6
// adapters at 1040 x 4096: 13 us together).
template <int JT, bool DROP, bool VEC, int D>
__global__ __launch_bounds__(kShrinkThreads) void k_adapter_shrink2(ShrinkArgs t, ShrinkArgs g, uint32_t n_t) {
  __shared__ ShrinkLds<JT> lds;
  if (blockIdx.x < n_t) shrink_body<JT, false, DROP, true, D>(t, blockIdx.x, lds);
  else shrink_body<JT, true, false, VEC, D>(g, blockIdx.x - n_t, lds);
}

template <int JT, bool QT, bool DROP, bool VEC>
hipError_t shrink_as(const ShrinkArgs& a, const ShrinkDecode* dec, const Nf4Tables& tab, hipStream_t st) {
  constexpr int kMost = JT == 1 ? 4 : (JT <= 4 ? 2 : 1);
  const int64_t tiles = (a.rows.M + kRowTile - 1) / kRowTile;
  const int64_t n = tiles * a.split;
  int64_t n_dec = 0;
  if (dec)
    n_dec = QT ? ((dec->K / 64 + kShrinkWaves - 1) / kShrinkWaves) * ((dec->N + kTRows - 1) / kTRows)
               : (dec->N * dec->K / 8 + kShrinkThreads * kDecWords - 1) / (kShrinkThreads * kDecWords);
  const ShrinkDecode d = dec ? *dec : ShrinkDecode{};
  hipLaunchKernelGGL((k_adapter_shrink<JT, QT, DROP, VEC, kMost>), dim3((unsigned)(n + n_dec)), dim3(kShrinkThreads), 0, st, a,
                     d, (uint32_t)n, tab);
  return hipGetLastError();
}
template <int JT, bool DROP, bool VEC>
hipError_t shrink2_as(const ShrinkArgs& t, const ShrinkArgs& g, hipStream_t st) {
  constexpr int kMost = JT == 1 ? 4 : (JT <= 4 ? 2 : 1);
  const int64_t tiles = (t.rows.M + kRowTile - 1) / kRowTile, n_t = tiles * t.split;
  hipLaunchKernelGGL((k_adapter_shrink2<JT, DROP, VEC, kMost>), dim3((unsigned)(n_t + tiles * g.split)), dim3(kShrinkThreads), 0,
                     st, t, g, (uint32_t)n_t);
  return hipGetLastError();
}
template <bool DROP, bool VEC>
hipError_t shrink2_by_rank(const ShrinkArgs& t, const ShrinkArgs& g, hipStream_t st) {
  if (t.rows.max_rank <= 16) return shrink2_as<1, DROP, VEC>(t, g, st);
  if (t.rows.max_rank <= 32) return shrink2_as<2, DROP, VEC>(t, g, st);
  if (t.rows.max_rank <= 64) return shrink2_as<4, DROP, VEC>(t, g, st);
  return shrink2_as<8, DROP, VEC>(t, g, st);
}
template <bool QT, bool DROP, bool VEC>
hipError_t shrink_by_rank(const ShrinkArgs& a, const ShrinkDecode* dec, const Nf4Tables& tab, hipStream_t st) {
  if (a.rows.max_rank <= 16) return shrink_as<1, QT, DROP, VEC>(a, dec, tab, st);
  if (a.rows.max_rank <= 32) return shrink_as<2, QT, DROP, VEC>(a, dec, tab, st);
  if (a.rows.max_rank <= 64) return shrink_as<4, QT, DROP, VEC>(a, dec, tab, st);
  return shrink_as<8, QT, DROP, VEC>(a, dec, tab, st);
}

// ---------------------------------------------------------------- few rows: the weight's stream
// Rows of 16 lanes 1 and 3 of a change places with rows 0 and 2 of b; the upper 32 lanes of a with
// the lower 32 of b.
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto s = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = s[0], b = s[1];
}
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto s = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = s[0], b = s[1];
}

constexpr int kStreamThreads = 512;
constexpr int kStreamWaves = kStreamThreads / 64;
constexpr int kStreamRows = 16;  // weight rows of a tile
constexpr int kStreamMaxRows = 128;

struct StreamArgs {
  const uint8_t *codes, *code8;
  const float *c2s, *mu;
  int64_t N, K;
  const uint16_t* X;
  AdapterRows rows;
  DropMask drop;
  float* T;  // read; where the stream forms T itself, written (null: not wanted)
  uint16_t* Y;
  int32_t lists;
  uint64_t* words;  // [workgroup][row][width], zero before and after
  int32_t polls;    // how often a word that is not there yet is looked for
};

// T for the stream: 16 rows, 16 ranks and every `lists`-th of the rows' distinct adapters, over the
// whole reduction.  No partial sums cross workgroups (with the reduction split over 16 workgroups
// and added up by the last of them, 37 rows of 24 adapters took 20 us).  Zeros past a row's rank;
// list 0 also writes the zeros of rows without an adapter.
template <bool DROP>
__global__ __launch_bounds__(kStreamThreads) void k_adapter_t(StreamArgs a) {
  constexpr int D = 4;  // blocks of 64 columns in flight
  __shared__ uint4 smem[kStreamWaves * 256];
  f32x4_t* red = reinterpret_cast<f32x4_t*>(smem);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int width = a.rows.width, ranks = (width + 15) / 16;
  const int list = (int)blockIdx.x % a.lists, rest = (int)blockIdx.x / a.lists, jt = rest % ranks, m0 = rest / ranks * kRowTile;
  const int64_t K = a.K;
  const int id = adapter_of(a.rows, m0 + l16);
  uint64_t base = 0;
  int rank = 0;
  if (id >= 0) {
    const AdapterEntry* e = a.rows.table + id;
    base = reinterpret_cast<uint64_t>(e->A);
    rank = e->r;
  }
  RngKey key{};
  if (DROP) key = load_rng(a.drop.rng);
  const uint32_t t2 = threshold_halves(a.drop.threshold);
  const rsrc_t rp = make_rsrc(a.X + (int64_t)m0 * K, (a.rows.M - m0) * K * 2);
  const int nb = (int)(K / 64);
  uint4* xs = smem + wave * 256;  // this wavefront's tiles of X and A (as in the stream below)
  f32x4_t out = {0.f, 0.f, 0.f, 0.f};
  bool write = id < 0 && list == 0;
  uint64_t pending = __ballot(id >= 0);
  int skip = list;
  while (pending) {
    const int from = lowest(pending), one = __builtin_amdgcn_readlane(id, from), r = __builtin_amdgcn_readlane(rank, from);
    const bool mine = id == one;
    pending &= ~__ballot(mine);
    if (skip) {
      --skip;
      continue;
    }
    skip = a.lists - 1;
    write |= mine;
    if (16 * jt >= r) continue;
    const rsrc_t rq = make_rsrc(reinterpret_cast<const void*>(readlane64(base, from)), (int64_t)r * K * 2);
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    const uint64_t rows_mine = __ballot(mine);  // bit m: row m of the tile (in every group of 16 lanes)
    uint4 x[D][2], q[D][2];
    const auto load = [&](int d, int blk) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 8 * i + (lane >> 3), chunk = (lane & 7) ^ ((4 * i + (lane >> 4)) & 7);
        const uint32_t off = (uint32_t)(row * K + 64 * (int64_t)blk + 8 * chunk) * 2;
        x[d][i] = bload16(rp, (blk < nb && ((rows_mine >> row) & 1)) ? off : kOOB);
        q[d][i] = bload16(rq, (blk < nb && 16 * jt + row < r) ? off + (uint32_t)(32 * jt * K) : kOOB);
      }
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(d, wave + kStreamWaves * d);
    for (int b0 = wave; b0 < nb; b0 += kStreamWaves * D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const int blk = b0 + kStreamWaves * d;
        if (blk >= nb) break;
        // the wavefront's LDS accesses run in order
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < 2; ++i) xs[64 * i + lane] = x[d][i], xs[128 + 64 * i + lane] = q[d][i];
        asm volatile("" ::: "memory");
        load(d, blk + kStreamWaves * D);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int at = 8 * l16 + ((4 * h + g) ^ (l16 >> 1));
          uint4 p = xs[at];
          if (DROP) p = drop8(p, key, (uint64_t)(m0 + l16) * (uint64_t)(K / 8) + (uint64_t)(8 * blk + 4 * h + g), t2);
          acc = mfma16x16x32(as_bf16x8(xs[128 + at]), as_bf16x8(p), acc);
        }
        asm volatile("" ::: "memory");
      }
    }
    __syncthreads();  // the sums take the place of the tiles
    // the wavefronts' sums in order; D[j][m]: ranks 4 g + v of row l16
    red[wave * 64 + lane] = acc;
    __syncthreads();
    if (wave == 0) {
      f32x4_t sum = red[lane];
#pragma unroll
      for (int w = 1; w < kStreamWaves; ++w) {
        const f32x4_t v = red[w * 64 + lane];
        sum[0] += v[0]; sum[1] += v[1]; sum[2] += v[2]; sum[3] += v[3];
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) out[v] = mine ? sum[v] : out[v];
    }
    __syncthreads();  // before the next adapter's tiles
  }
  const int j = 16 * jt + 4 * g;
  if (wave != 0 || !write || m0 + l16 >= a.rows.M || j >= width) return;
#pragma unroll
  for (int v = 0; v < 4; ++v) out[v] = j + v < rank ? out[v] * a.drop.scale : 0.f;
  *reinterpret_cast<f32x4_t*>(a.T + (int64_t)(m0 + l16) * width + j) = out;
}

// ---- T of a row or a few, formed by the stream's own workgroups.  Workgroup j takes element j of T
// [M][width] (and every gridDim.x-th from there), a dot product of two rows of K, and posts it, with a
// bit that marks it as there, to a word of its own in each workgroup's block, in the workspace's
// head.  A workgroup reads its words after its share of the weight and clears them.  (A launch for T
// before the stream costs 1 to 8 us: stream_forms_t().)
//
// Nothing says that the posting workgroups run while others wait: each XCD starts its workgroups on
// its own, and launches on several streams share the chip.  So no wait depends on it.  A reader looks
// a.polls times, then forms the elements that are missing itself, by the same sums in the same
// order, so to the same bits.  Posts are additions to a word that is zero, and such a reader subtracts
// from the word what it formed: whichever of the two comes first, both leave zero, and a late post
// finds no word to spoil.  The head is zero after every call.
constexpr uint64_t kPosted = uint64_t(1) << 32;  // beside the value's 32 bits
constexpr int64_t kPostedWords = 32768;

// The word of a value: all NaN are one, so that two ways to form it agree.
__device__ __forceinline__ uint64_t posted_word(float t) { return kPosted | (t == t ? __float_as_uint(t) : 0x7FC00000u); }

// Thread tid's share of row m of X (its dropout applied) times a row of A, summed over its wavefront.
template <int W>
__device__ __forceinline__ float dot_share(const StreamArgs& a, const RngKey& key, uint32_t t2, uint32_t m,
                                           const uint16_t* A_row, int tid) {
  const uint32_t chunks = (uint32_t)(a.K / 8);
  const uint4* p = reinterpret_cast<const uint4*>(A_row);
  const uint4* x = reinterpret_cast<const uint4*>(a.X + (int64_t)m * a.K);
  float sum = 0.f;
  for (uint32_t c = (uint32_t)tid; c < chunks; c += 64 * W) {
    const uint4 u = p[c];
    uint4 v = x[c];
    if (a.drop.threshold) v = drop8(v, key, (uint64_t)m * chunks + c, t2);
    const uint32_t pu[4] = {u.x, u.y, u.z, u.w}, pv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum = fmaf(bf16lo_to_f32(pu[i]), bf16lo_to_f32(pv[i]), sum);
      sum = fmaf(bf16hi_to_f32(pu[i]), bf16hi_to_f32(pv[i]), sum);
    }
  }
#pragma unroll
  for (int by = 32; by; by >>= 1) sum += __shfl_xor(sum, by);
  return sum;
}

template <int W>
__device__ __forceinline__ void post_t(const StreamArgs& a, int tid) {
  __shared__ float dots[W];
  const uint32_t width = (uint32_t)a.rows.width, slots = (uint32_t)a.rows.M * width, groups = gridDim.x;
  if (blockIdx.x >= slots) return;
  const uint32_t t2 = threshold_halves(a.drop.threshold);
  RngKey key{};
  if (a.drop.threshold) key = load_rng(a.drop.rng);
  for (uint32_t slot = blockIdx.x; slot < slots; slot += groups) {
    const uint32_t m = slot / width, j = slot - m * width;
    const int one = adapter_of(a.rows, m);
    const bool has = one >= 0 && (int)j < a.rows.table[one].r;
    float t = 0.f;
    if (has) {
      const float sum = dot_share<W>(a, key, t2, m, a.rows.table[one].A + (int64_t)j * a.K, tid);
      if ((tid & 63) == 0) dots[tid >> 6] = sum;
      __syncthreads();
      t = dots[0];
#pragma unroll
      for (int w = 1; w < W; ++w) t += dots[w];
      t *= a.drop.scale;
      const uint64_t word = posted_word(t);
      for (uint32_t to = (uint32_t)tid; to < groups; to += 64 * W)
        __hip_atomic_fetch_add(a.words + (uint64_t)to * slots + slot, word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
      __syncthreads();  // dots is free again
    }
    if (a.T && tid == 0) a.T[slot] = t;
  }
}

// The words of row k that did not arrive (bit i of a lane's `missing`: word i of its eight ranks), formed
// by this wavefront and taken out of the memory that they would have come to.
template <int W>
__device__ __forceinline__ void form_missing(const StreamArgs& a, uint64_t* words, int k, int r0, uint32_t missing, int lane,
                                             uint64_t (&t)[8]) {
  const uint32_t t2 = threshold_halves(a.drop.threshold);
  RngKey key{};
  if (a.drop.threshold) key = load_rng(a.drop.rng);
  const uint16_t* A = a.rows.table[adapter_of(a.rows, k)].A;
#pragma unroll 1
  for (int q = 0; q < 32; ++q) {
    const int from = 16 * (q >> 3) + k;  // the lane that reads rank r0 + q
    if (!(((uint32_t)__builtin_amdgcn_readlane((int)missing, from) >> (q & 7)) & 1u)) continue;
    float sum = 0.f;
#pragma unroll 1
    for (int w = 0; w < W; ++w) {
      const float d = dot_share<W>(a, key, t2, (uint32_t)k, A + (int64_t)(r0 + q) * a.K, 64 * w + lane);
      sum = w ? sum + d : d;
    }
    const uint64_t word = posted_word(sum * a.drop.scale);
    if (lane != from) continue;
    __hip_atomic_fetch_add(words + r0 + q, 0 - word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = i == (q & 7) ? word : t[i];
  }
}

// acc += B's 16 rows times hi + lo (eight ranks for each lane's row of X) where `has`: the products of
// other rows are not taken.
__device__ __forceinline__ void add_term(f32x4_t& acc, const uint4& w, const uint4& hi, const uint4& lo, bool has) {
  const f32x4_t p = mfma16x16x32(finite_only(as_bf16x8(w)), as_bf16x8(lo),
                                 mfma16x16x32(as_bf16x8(w), as_bf16x8(hi), f32x4_t{0.f, 0.f, 0.f, 0.f}));
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] += has ? p[i] : 0.f;
}

// 16 RT weight rows over the whole reduction.  A wavefront takes groups of four 64-weight blocks;
// lane (l16, g) decodes block 4 group + g of row l16 (32 bytes of codes, one level table scaled by
// the block's constant: exactly w_hat).  The four lanes of a row then exchange their words (a 4 x 4
// transpose by lane swaps), so that an MFMA 16x16x32 operand holds 32 consecutive columns.  X comes
// block by block in whole cache lines (eight lanes to a row's 128 bytes), PD blocks ahead in
// registers, and through LDS of the wavefront's own into operand order; 16-byte chunk c of row r
// lies at c ^ (r / 2 % 8), so that reads and writes meet all banks.  (Operands straight from memory
// have neighbouring lanes in 16 rows: 37 rows at 14336 x 4096 91 us in the blocks' order, 56 in
// 64-byte pieces.)
//
// The adapters' term is more of the same sum.  Without POST, T is there; the wavefronts deal the
// distinct adapters of all rows among themselves, and each multiplies its ones' 16 rows of B with T
// (hi and lo BF16 parts) into its accumulators.  With POST (a row or a few), workgroups form T while
// they stream, one element each, and post it to every workgroup (below); the wavefronts deal the rows
// among themselves.
//
// Every workgroup reads all of X, by way of the L2 (at 14336 x 4096 and RT = 1, 940 MB for 64 rows), so
// wide weights are taken two tiles of rows at a time, RT = 2 (64 rows there 44 us with RT = 1, 35 with 2;
// 4096 x 4096, where that leaves half of the compute units without work, 16 and 20).  W: wavefronts;
// four where more workgroups of eight are started than fit at once (longer runs of blocks for each:
// 64 rows at 14336 x 4096 35 -> 32 us; at 4096 x 4096 16 -> 19).
template <int W, int RT, int MT, bool POST, int PD, bool WHOLE>
__global__ __launch_bounds__(64 * W, !POST && RT == 1 && MT <= 3 ? 4 : 2) void k_adapter_stream(StreamArgs a, Nf4Tables tab) {
  static_assert(!POST || RT * MT == 1, "few rows");
  static_assert(RT <= 2, "the sums take the place of the tiles");
  __shared__ uint4 smem[W * MT * 128];  // a wavefront's tiles of X; then the sums
  f32x4_t(*red)[RT * MT][64] = reinterpret_cast<f32x4_t(*)[RT * MT][64]>(smem);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int64_t K = a.K, N = a.N, row0 = (int64_t)blockIdx.x * (kStreamRows * RT);
  const int M = (int)a.rows.M, width = a.rows.width;
  const uint32_t nb = (uint32_t)(K / 64), ng = (nb + 3) / 4;
  const rsrc_t rx = make_rsrc(a.X, (int64_t)M * K * 2);
  const int64_t rows_here = N - row0 < kStreamRows * RT ? N - row0 : kStreamRows * RT;
  const rsrc_t rc = make_rsrc(a.codes + row0 * (K / 2), rows_here * (K / 2));
  const rsrc_t r8 = make_rsrc(a.code8 + row0 * nb, rows_here * nb);
  const rsrc_t r2 = make_rsrc(a.c2s, ((N * nb + 255) / 256) * 4);
  const uint32_t blk_row = (uint32_t)(row0 + l16) * nb;
  struct Codes {
    uint4 c0[RT], c1[RT];
    uint32_t c8[RT], c2[RT];
  };
  const auto load = [&](uint32_t group) {
    const uint32_t b = 4 * group + g;
    const bool ok = group < ng && b < nb;
    Codes c;
#pragma unroll
    for (int u = 0; u < RT; ++u) {
      const uint32_t off = (uint32_t)((16 * u + l16) * (K / 2)) + 32 * b;
      c.c0[u] = bload16(rc, ok ? off : kOOB);
      c.c1[u] = bload16(rc, ok ? off + 16 : kOOB);
      c.c8[u] = bload1(r8, ok ? (16 * u + l16) * nb + b : kOOB);
      c.c2[u] = bload4(r2, ok ? ((blk_row + 16 * u * nb + b) >> 8) * 4 : kOOB);
    }
    return c;
  };
  // each lane its rows' adapters (asked for first: what follows depends on them)
  int id[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) id[t] = adapter_of(a.rows, 16 * t + l16);
  Codes cur = load(wave), next = load(wave + W);
  const float mu = a.mu[0];
  f32x4_t acc[RT][MT];
#pragma unroll
  for (int u = 0; u < RT; ++u)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[u][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  uint4* xs = smem + wave * MT * 128;
  uint4 xr[PD][MT][2];
  const auto load_x = [&](uint4 (&x)[MT][2], uint32_t blk) {
    // lane p takes chunk (p & 7) ^ (row / 2 % 8) of rows p >> 3 and 8 + (p >> 3) of a tile
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int m = 16 * t + 8 * i + (lane >> 3), chunk = (lane & 7) ^ ((4 * i + (lane >> 4)) & 7);
        x[t][i] = bload16(rx, (m < M && blk < nb) ? (uint32_t)((m * K + 64 * (int64_t)blk + 8 * chunk) * 2) : kOOB);
      }
  };
#pragma unroll
  for (int d = 0; d < PD; ++d) load_x(xr[d], 4 * wave + d);

  if (POST) post_t<W>(a, tid);
  // this wavefront's adapters, every W-th distinct one, lane k holding the k-th; with POST, lane m
  // holds row m's
  int mine = 0, count = 0;
  if (!POST) {
    uint64_t pending[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) pending[t] = __ballot(id[t] >= 0);
    uint32_t skip = wave;
#pragma unroll
    for (int t = 0; t < MT; ++t)
      while (pending[t]) {
        const int one = __builtin_amdgcn_readlane(id[t], lowest(pending[t]));
#pragma unroll
        for (int u = t; u < MT; ++u) pending[u] &= ~__ballot(id[u] == one);
        if (skip) {
          --skip;
        } else {
          mine = lane == count ? one : mine;
          ++count;
          skip = W - 1;
        }
      }
  } else {
    mine = id[0] < 0 ? 0 : id[0];
    count = M;
  }
  uint64_t base_b = 0;
  int rank_l = 0;
  float scale_l = 0.f;
  if (count) {
    const AdapterEntry* e = a.rows.table + mine;
    base_b = reinterpret_cast<uint64_t>(e->B);
    rank_l = POST && id[0] < 0 ? 0 : e->r;
    scale_l = e->s;
  }
  // ranks r0 + 8 g .. +7 of B's row row0 + 16 u + l16, for the adapter that lane k holds
  const auto load_b = [&](int k, int r0, int u) {
    const int r = __builtin_amdgcn_readlane(rank_l, k), at = r0 + 8 * g;
    const uint16_t* B = reinterpret_cast<const uint16_t*>(readlane64(base_b, k));
    if (WHOLE)
      return bload16(make_rsrc(B + row0 * r, rows_here * r * 2), at < r ? (uint32_t)(((16 * u + l16) * r + at) * 2) : kOOB);
    const int64_t row = row0 + 16 * u + l16;
    return load_row8(B, N * (r ? r : 1), (row < N ? row : N - 1) * r, at, r);
  };
  uint4 ahead_b = make_uint4(0, 0, 0, 0);
  if (POST && wave < M) ahead_b = load_b(wave, 0, 0);

  // ---- the base product
  for (uint32_t group = wave; group < ng; group += W) {
    const Codes c = cur;
    cur = next;
    next = load(group + 2 * W);
    uint32_t w[RT][8][4];  // word i of this lane's block; then, of block i % 4, word 4 (i / 4) + g
#pragma unroll
    for (int u = 0; u < RT; ++u) {
      Lut L;
      build_scaled_lut(tab, stored_scale(c.c8[u], __uint_as_float(c.c2[u]), mu), L);
      const uint32_t words[8] = {c.c0[u].x, c.c0[u].y, c.c0[u].z, c.c0[u].w, c.c1[u].x, c.c1[u].y, c.c1[u].z, c.c1[u].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) decode8(words[i], L, w[u][i]);
#pragma unroll
      for (int h = 0; h < 8; h += 4)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          swap16(w[u][h][q], w[u][h + 1][q]);
          swap16(w[u][h + 2][q], w[u][h + 3][q]);
          swap32(w[u][h][q], w[u][h + 2][q]);
          swap32(w[u][h + 1][q], w[u][h + 3][q]);
        }
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      // the wavefront's LDS accesses run in order
      asm volatile("" ::: "memory");
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) xs[128 * t + 64 * i + lane] = xr[b % PD][t][i];
      asm volatile("" ::: "memory");
      const uint32_t ahead = 4 * (group + W * ((b + PD) / 4)) + (b + PD) % 4;
      load_x(xr[b % PD], ahead);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = 8 * l16 + ((4 * h + g) ^ (l16 >> 1));
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const bf16x8_t x = as_bf16x8(xs[128 * t + at]);
#pragma unroll
          for (int u = 0; u < RT; ++u) acc[u][t] = mfma16x16x32(as_bf16x8(w[u][b + 4 * h]), x, acc[u][t]);
        }
      }
      asm volatile("" ::: "memory");
    }
  }

  if (!POST) {
    // ---- this wavefront's adapters, 32 ranks an item
    const rsrc_t rt = make_rsrc(a.T, (int64_t)M * width * 4);
    const auto load_t = [&](int t, int one, int at, uint4& x, uint4& y) {
      const uint32_t off = (id[t] == one && at < width) ? (uint32_t)(((16 * t + l16) * width + at) * 4) : kOOB;
      x = bload16(rt, off), y = bload16(rt, off == kOOB ? kOOB : off + 16);
    };
    const auto take = [&](int t, const uint4 (&w)[RT], const uint4& x, const uint4& y, float s, bool has) {
      const float v[8] = {__uint_as_float(x.x) * s, __uint_as_float(x.y) * s, __uint_as_float(x.z) * s,
                          __uint_as_float(x.w) * s, __uint_as_float(y.x) * s, __uint_as_float(y.y) * s,
                          __uint_as_float(y.z) * s, __uint_as_float(y.w) * s};
      uint4 hi, lo;
      split_bf16(v, hi, lo);
#pragma unroll
      for (int q = 0; q < RT; ++q) add_term(acc[q][t], w[q], hi, lo, has);
    };
    const auto scale_of = [&](int k) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scale_l), k)); };
    // D items' loads in flight, as registers allow (37 rows of 24 adapters at 14336 x 4096 36.5 us one
    // by one, 35.0 so)
    if constexpr (MT <= 4) {
      constexpr int D = RT == 1 && MT <= 3 ? 5 - MT : (MT <= 3 ? 4 : 3);
      uint4 w[D][RT], u[D][MT][2];
      int k = 0, r0 = 0, which[D], lane_of[D];
      const auto fetch = [&](int d) {
        which[d] = -2;
        if (k >= count) return;
        lane_of[d] = k;
        which[d] = __builtin_amdgcn_readlane(mine, k);
#pragma unroll
        for (int v = 0; v < RT; ++v) w[d][v] = load_b(k, r0, v);
#pragma unroll
        for (int t = 0; t < MT; ++t) load_t(t, which[d], r0 + 8 * g, u[d][t][0], u[d][t][1]);
        r0 += 32;
        if (r0 >= __builtin_amdgcn_readlane(rank_l, k)) r0 = 0, ++k;
      };
#pragma unroll
      for (int d = 0; d < D; ++d) fetch(d);
      while (which[0] != -2) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
          if (which[d] == -2) continue;
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            const bool has = id[t] == which[d];
            if (__ballot(has)) take(t, w[d], u[d][t][0], u[d][t][1], scale_of(lane_of[d]), has);
          }
          fetch(d);
        }
      }
    } else {
      for (int k = 0; k < count; ++k) {
        const int one = __builtin_amdgcn_readlane(mine, k), r = __builtin_amdgcn_readlane(rank_l, k);
        for (int r0 = 0; r0 < r; r0 += 32) {
          uint4 w[RT];
#pragma unroll
          for (int u = 0; u < RT; ++u) w[u] = load_b(k, r0, u);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            const bool has = id[t] == one;
            if (!__ballot(has)) continue;
            uint4 x, y;
            load_t(t, one, r0 + 8 * g, x, y);
            take(t, w, x, y, scale_of(k), has);
          }
        }
      }
    }
  } else {
    // ---- this wavefront's rows: their words of T, taken as they arrive and cleared
    uint64_t* mine_t = a.words + (int64_t)blockIdx.x * M * width;
    for (int k = wave; k < M; k += W) {
      const int r = __builtin_amdgcn_readlane(rank_l, k);
      const float s = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scale_l), k));
      for (int r0 = 0; r0 < r; r0 += 32) {
        const int at = r0 + 8 * g, have = l16 == k && at < r ? r - at : 0;
        const uint4 w = k == wave && r0 == 0 ? ahead_b : load_b(k, r0, 0);
        uint64_t t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = i < have ? 0 : kPosted;
        bool ready = false;
        for (int it = 0; !ready && it < a.polls; ++it) {
          if (it) __builtin_amdgcn_s_sleep(1);
          ready = true;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (i < have) t[i] = __hip_atomic_load(mine_t + k * width + at + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
            ready = ready && (t[i] & kPosted);
          }
        }
        uint32_t missing = 0;
        if (__builtin_expect(__ballot(!ready) != 0, 0)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) missing |= (t[i] & kPosted) ? 0u : 1u << i;
          form_missing<W>(a, mine_t + k * width, k, r0, missing, lane, t);
        }
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = __uint_as_float((uint32_t)t[i]) * s;
          if (i < have && !((missing >> i) & 1u))
            __hip_atomic_store(mine_t + k * width + at + i, (uint64_t)0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
        }
        uint4 hi, lo;
        split_bf16(v, hi, lo);
        add_term(acc[0][0], w, hi, lo, l16 == k);
      }
    }
  }
  __syncthreads();  // the sums take the place of every wavefront's tiles
#pragma unroll
  for (int u = 0; u < RT; ++u)
#pragma unroll
    for (int t = 0; t < MT; ++t) red[wave][RT * t + u][lane] = acc[u][t];
  __syncthreads();
  // the wavefronts' sums in order; lane l of tile RT t + u: row 16 t + (l & 15) of X, weight rows
  // 16 u + 4 (l >> 4) + v
  for (int i = wave; i < RT * MT; i += W) {
    const int m = 16 * (i / RT) + l16;
    const int64_t n = row0 + 16 * (i % RT) + 4 * g;
    if (m >= M || n >= N) continue;
    f32x4_t y = red[0][i][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const f32x4_t v = red[w][i][lane];
      y[0] += v[0]; y[1] += v[1]; y[2] += v[2]; y[3] += v[3];
    }
    *reinterpret_cast<uint2*>(a.Y + (int64_t)m * N + n) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
  }
}

// ---------------------------------------------------------------- dA and dB
constexpr int kGradThreads = 256;
constexpr int kGradWaves = kGradThreads / 64;
constexpr int kGradCols = 64;         // columns per workgroup
constexpr int kGradRanks = 64;        // ranks per workgroup
constexpr int kSpan = 256;            // rows that a wavefront looks through at once, at most
constexpr int kVTile = 32 * 32 + 64;  // bytes of a staged [32][16] BF16 tile, padded (bank offset)
constexpr int kSumU = 4;              // partials loaded together before they are added

struct GradsArgs {
  AdapterRows rows;
  const uint16_t *X, *dY;
  const float *T, *G;
  int64_t K, N;
  DropMask drop;
  float* part;
  unsigned int* counters;
  uint32_t tiles_a;
  int32_t blocks, split;
  int64_t mps;  // rows per slice
};

// Workgroup (x, y, z): 64 columns of dA (or of dB), a slice of the rows, an adapter and up to 64 of
// its ranks.  The workgroup looks through 1024 rows at a time, lists those of its adapter (ballots
// over ids) and deals them to its wavefronts 32 by 32, so that runs of one adapter's rows are
// shared like rows that lie apart (555 rows of 6 adapters in runs 19.4 us when each wavefront kept to
// 256 rows, so 11): U [32 rows][ranks] as hi and lo BF16 parts and V [32 rows][64
// columns], both transposed through LDS.  Bound by HBM at low ranks (8192 rows of 4 adapters of rank 16
// at 14336 x 4096 84 us for 303 MB), by U at high ones, which every tile of columns reads anew (4096
// rows of rank 64 at 4096 x 4096 40 us: 134 MB of U through the L2 beside 67 MB of V).
template <int JT>
struct GradsLds {
  static constexpr int kWaveBytes = (4 + 2 * JT) * kVTile;
  static constexpr int kRedBytes = kGradWaves * JT * 4 * 64 * 16;
  __attribute__((aligned(16))) char tiles[kGradWaves * kWaveBytes > kRedBytes ? kGradWaves * kWaveBytes : kRedBytes];
  uint16_t list[kGradWaves * kSpan];
  int counts[kGradWaves];
  bool last;
};
template <int JT, int D, bool DROP, bool IS_B>
__device__ __forceinline__ void grads_body(const GradsArgs& a, GradsLds<JT>& lds) {
  constexpr int kWaveBytes = GradsLds<JT>::kWaveBytes;
  char* smem = lds.tiles;
  const int adapter = (int)(blockIdx.z / (unsigned)a.blocks), block = (int)blockIdx.z - adapter * a.blocks;
  const AdapterEntry e = a.rows.table[adapter];
  const int j_first = block * kGradRanks;
  if (j_first >= e.r) return;  // all slices alike: no counter is touched
  const uint16_t* __restrict__ V = IS_B ? a.dY : a.X;
  const float* __restrict__ U = IS_B ? a.T : a.G;
  const int64_t C = IS_B ? a.N : a.K, width = a.rows.width;
  const int64_t c0 = (int64_t)(IS_B ? blockIdx.x - a.tiles_a : blockIdx.x) * kGradCols;
  const int64_t mbeg = (int64_t)blockIdx.y * a.mps, mend = mbeg + a.mps < a.rows.M ? mbeg + a.mps : a.rows.M;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RngKey key{};
  uint32_t t2 = 0;
  if (DROP) key = load_rng(a.drop.rng), t2 = threshold_halves(a.drop.threshold);
  char* vt = smem + wave * kWaveBytes;  // 4 V tiles, JT hi tiles, JT lo tiles
  char* ut = vt + 4 * kVTile;
  uint16_t* list = lds.list;
  const int span = C <= (int64_t(1) << 20) ? kSpan : 64;  // the rows looked through stay below 2^31 bytes
  const int32_t* __restrict__ ids = a.rows.ids;
  const uint64_t below = lane ? ~0ull >> (64 - lane) : 0ull;
  f32x4_t acc[JT][4];
#pragma unroll
  for (int t = 0; t < JT; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[t][q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int64_t first = mbeg; first < mend; first += (int64_t)span * kGradWaves) {
    const int n = (int)(mend - first < span * kGradWaves ? mend - first : span * kGradWaves);
    int own = 0, id[kSpan / 64];
    uint64_t hits[kSpan / 64];
#pragma unroll
    for (int q = 0; q < kSpan / 64; ++q) {
      const int at = span * wave + 64 * q + lane;
      id[q] = 64 * q < span && at < n ? (ids ? ids[first + at] : 0) : -1;
    }
#pragma unroll
    for (int q = 0; q < kSpan / 64; ++q) hits[q] = __ballot(id[q] == adapter), own += __popcll(hits[q]);
    __syncthreads();  // the last rows' list is read
    if (lane == 0) lds.counts[wave] = own;
    __syncthreads();
    int to = 0, count = 0;
#pragma unroll
    for (int w = 0; w < kGradWaves; ++w) {
      const int c = __builtin_amdgcn_readfirstlane(lds.counts[w]);
      to += w < wave ? c : 0;
      count += c;
    }
#pragma unroll
    for (int q = 0; q < kSpan / 64; ++q) {
      if (id[q] == adapter) list[to + __popcll(hits[q] & below)] = (uint16_t)(span * wave + 64 * q + lane);
      to += __popcll(hits[q]);
    }
    __syncthreads();
    const rsrc_t rv = make_rsrc(V + first * C, n * C * 2);
    const rsrc_t ru = make_rsrc(U + first * width, n * width * 4);
    const auto row = [&](int i) { return i < count ? (int)list[i] : -1; };
    constexpr int kStep = 32 * kGradWaves;  // from one of a wavefront's groups to its next
    for (int i0 = 32 * wave; i0 < count; i0 += kStep * D) {
      uint4 vv[D][4], uw[D][JT][2];
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (i0 + kStep * d >= count) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = row(i0 + kStep * d + 8 * i + (lane >> 3));
          const int64_t c = c0 + 8 * (lane & 7);
          vv[d][i] = bload16(rv, (m >= 0 && c < C) ? (uint32_t)((m * C + c) * 2) : kOOB);
        }
        const int m = row(i0 + kStep * d + (lane >> 1));
#pragma unroll
        for (int t = 0; t < JT; ++t) {
          const int j = j_first + 16 * t + 8 * (lane & 1);
          const uint32_t off = (m >= 0 && j < width) ? (uint32_t)((m * width + j) * 4) : kOOB;
          uw[d][t][0] = bload16(ru, off);
          uw[d][t][1] = bload16(ru, off == kOOB ? kOOB : off + 16);
        }
      }
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (i0 + kStep * d >= count) break;
        // the wavefront's LDS tiles are reused chunk after chunk; its LDS accesses run in order
        asm volatile("" ::: "memory");
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int in = 8 * i + (lane >> 3), ct = (lane & 7) >> 1, half = lane & 1;
          uint4 v = vv[d][i];
          if (DROP) {
            const int m = row(i0 + kStep * d + in);
            v = drop8(v, key, (uint64_t)((first + (m < 0 ? 0 : m)) * (C / 8) + c0 / 8 + (lane & 7)), t2);
          }
          most = most_halves(most, v);
          *reinterpret_cast<uint4*>(vt + ct * kVTile + in * 32 + 16 * half) = v;
        }
#pragma unroll
        for (int t = 0; t < JT; ++t) {
          const uint4 x = uw[d][t][0], y = uw[d][t][1];
          const float f[8] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w),
                              __uint_as_float(y.x), __uint_as_float(y.y), __uint_as_float(y.z), __uint_as_float(y.w)};
          uint4 hi, lo;
          split_bf16(f, hi, lo);
          *reinterpret_cast<uint4*>(ut + t * kVTile + (lane >> 1) * 32 + 16 * (lane & 1)) = hi;
          *reinterpret_cast<uint4*>(ut + (JT + t) * kVTile + (lane >> 1) * 32 + 16 * (lane & 1)) = lo;
        }
        asm volatile("" ::: "memory");
        bf16x8_t b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) b[q] = tr_operand(vt + q * kVTile, lane & 15, 8 * (lane >> 4));
        const auto add = [&](const char* u) {
#pragma unroll
          for (int t = 0; t < JT; ++t) {
            const bf16x8_t v = tr_operand(u + t * kVTile, lane & 15, 8 * (lane >> 4));
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[t][q] = mfma16x16x32(v, b[q], acc[t][q]);
          }
        };
        add(ut);
        if (some_not_finite(most)) {
#pragma unroll
          for (int q = 0; q < 4; ++q) b[q] = finite_only(b[q]);
        }
        add(ut + JT * kVTile);
        asm volatile("" ::: "memory");
      }
    }
  }
  // fixed-order sum over the wavefronts: D[j][c], lane l holds j = 4 (l >> 4) + v, c = l & 15
  __syncthreads();
  f32x4_t* red = reinterpret_cast<f32x4_t*>(smem);
#pragma unroll
  for (int t = 0; t < JT; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) red[((wave * JT + t) * 4 + q) * 64 + lane] = acc[t][q];
  __syncthreads();
  const float scale = DROP ? e.s * a.drop.scale : e.s;
  const int32_t split = a.split;
  constexpr int kItems = JT * 4 * 64;  // of four ranks each
  float* part = a.part + ((int64_t)(blockIdx.z * gridDim.x + blockIdx.x) * split) * kItems * 4;
  uint16_t* out = IS_B ? e.dB : e.dA;
  // item i: ranks j_first + 16 (i / 256) + 4 (i % 64 / 16) .. +3 of column c0 + 16 (i / 64 % 4) + i % 16
  const auto store = [&](int i, const f32x4_t& sum) {
    const int l = i & 63;
    const int64_t c = c0 + 16 * ((i >> 6) & 3) + (l & 15);
    const int j = j_first + 16 * (i >> 8) + 4 * (l >> 4);
    if (c >= C) return;
    const uint32_t lo = pack_bf16x2(sum[0] * scale, sum[1] * scale), hi = pack_bf16x2(sum[2] * scale, sum[3] * scale);
    const uint32_t h[4] = {lo & 0xFFFFu, lo >> 16, hi & 0xFFFFu, hi >> 16};
    if (IS_B && (e.r & 3) == 0 && (reinterpret_cast<uintptr_t>(out) & 7u) == 0) {
      if (j < e.r) *reinterpret_cast<uint2*>(out + c * e.r + j) = make_uint2(lo, hi);
      return;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (j + v < e.r) out[IS_B ? c * e.r + j + v : (int64_t)(j + v) * C + c] = (uint16_t)h[v];
  };
  for (int i = threadIdx.x; i < kItems; i += kGradThreads) {
    const int l = i & 63, q = (i >> 6) & 3, t = i >> 8;
    f32x4_t sum = red[(t * 4 + q) * 64 + l];
    for (int w = 1; w < kGradWaves; ++w) {
      const f32x4_t v = red[((w * JT + t) * 4 + q) * 64 + l];
      sum[0] += v[0]; sum[1] += v[1]; sum[2] += v[2]; sum[3] += v[3];
    }
    if (split == 1) store(i, sum);
    else if (j_first + 16 * t < e.r) store_partial(part + ((int64_t)blockIdx.y * kItems + i) * 4, sum);
  }
  if (split == 1) return;
  // every partial store of this workgroup has completed before its counter increment
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned int* counter = a.counters + (uint32_t)blockIdx.z * gridDim.x + blockIdx.x;
    const unsigned int old = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    lds.last = old + 1u == (unsigned int)split;
    if (lds.last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!lds.last) return;
  for (int i = threadIdx.x; i < kItems && j_first + 16 * (i >> 8) < e.r; i += kGradThreads) {
    f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
    for (int32_t k0 = 0; k0 < split; k0 += kSumU) {
      f32x4_t v[kSumU];
#pragma unroll
      for (int u = 0; u < kSumU; ++u)
        v[u] = k0 + u < split ? load_partial(part + ((int64_t)(k0 + u) * kItems + i) * 4) : f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < kSumU; ++u)
#pragma unroll
        for (int n = 0; n < 4; ++n) sum[n] += v[u][n];
    }
    store(i, sum);
  }
}

template <int JT, int D, bool DROP>
__global__ __launch_bounds__(kGradThreads) void k_adapter_grads(GradsArgs a) {
  __shared__ GradsLds<JT> lds;
  if (blockIdx.x < a.tiles_a) grads_body<JT, D, DROP, false>(a, lds);
  else grads_body<JT, D, false, true>(a, lds);
}

template <int W, int RT, int MT, bool POST, int PD>
hipError_t stream_go(const StreamArgs& a, const Nf4Tables& tab, hipStream_t st) {
  const dim3 grid((unsigned)((a.N + kStreamRows * RT - 1) / (kStreamRows * RT)));
  if (a.rows.whole) hipLaunchKernelGGL((k_adapter_stream<W, RT, MT, POST, PD, true>), grid, dim3(64 * W), 0, st, a, tab);
  else hipLaunchKernelGGL((k_adapter_stream<W, RT, MT, POST, PD, false>), grid, dim3(64 * W), 0, st, a, tab);
  return hipGetLastError();
}
// 17 to 96 rows
template <int W, int RT>
hipError_t stream_as(const StreamArgs& a, const Nf4Tables& tab, hipStream_t st) {
  if (a.rows.M <= 32) return stream_go<W, RT, 2, false, 2>(a, tab, st);
  if (a.rows.M <= 48) return stream_go<W, RT, 3, false, 1>(a, tab, st);
  if (a.rows.M <= 64) return stream_go<W, RT, 4, false, 1>(a, tab, st);
  return stream_go<W, RT, 6, false, 1>(a, tab, st);
}

template <int JT>
hipError_t grads_as(const GradsArgs& a, const GradPlan& plan, hipStream_t st) {
  constexpr int D = JT <= 2 ? 4 : 2;
  const dim3 grid((unsigned)(plan.tiles_a + plan.tiles_b), (unsigned)plan.split, (unsigned)(a.rows.count * plan.blocks));
  if (a.drop.threshold) hipLaunchKernelGGL((k_adapter_grads<JT, D, true>), grid, dim3(kGradThreads), 0, st, a);
  else hipLaunchKernelGGL((k_adapter_grads<JT, D, false>), grid, dim3(kGradThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adapter_table(const AdapterBatch& batch, int count, AdapterEntry* table, hipStream_t st) {
  hipLaunchKernelGGL(k_adapter_table, dim3(1), dim3(128), 0, st, batch, count, table);
  return hipGetLastError();
}

int32_t shrink_split(int64_t M, int64_t Kd) {
  const int64_t tiles = (M + kRowTile - 1) / kRowTile, blocks = (Kd + 63) / 64;
  const int64_t split = std::min<int64_t>({int64_t(32), 512 / tiles, blocks / kShrinkWaves});
  return (int32_t)std::max<int64_t>(split, 1);
}

hipError_t launch_shrink_a(const AdapterRows& rows, const uint16_t* X, int64_t K, const DropMask& drop, float* T,
                           float* part, unsigned int* counters, const ShrinkDecode* decode, const Nf4Tables& tab,
                           hipStream_t st) {
  const ShrinkArgs a{rows, X, K, drop, T, part, counters, shrink_split(rows.M, K)};
  return drop.threshold ? shrink_by_rank<false, true, true>(a, decode, tab, st)
                        : shrink_by_rank<false, false, true>(a, decode, tab, st);
}

hipError_t launch_shrink_b(const AdapterRows& rows, const uint16_t* dY, int64_t N, float* G, float* part,
                           unsigned int* counters, const ShrinkDecode* decode, const Nf4Tables& tab, hipStream_t st) {
  const ShrinkArgs a{rows, dY, N, DropMask{}, G, part, counters, shrink_split(rows.M, N)};
  return rows.whole ? shrink_by_rank<true, false, true>(a, decode, tab, st)
                    : shrink_by_rank<true, false, false>(a, decode, tab, st);
}

hipError_t launch_shrink_both(const AdapterRows& rows, const uint16_t* X, int64_t K, const DropMask& drop, float* T,
                              const uint16_t* dY, int64_t N, float* G, float* part_t, float* part_g,
                              unsigned int* counters, hipStream_t st) {
  const int64_t tiles = (rows.M + kRowTile - 1) / kRowTile;
  const ShrinkArgs t{rows, X, K, drop, T, part_t, counters, shrink_split(rows.M, K)};
  const ShrinkArgs g{rows, dY, N, DropMask{}, G, part_g, counters + tiles, shrink_split(rows.M, N)};
  if (drop.threshold) return rows.whole ? shrink2_by_rank<true, true>(t, g, st) : shrink2_by_rank<true, false>(t, g, st);
  return rows.whole ? shrink2_by_rank<false, true>(t, g, st) : shrink2_by_rank<false, false>(t, g, st);
}

// Up to 64 rows, and up to 128 of a smaller weight: the stream's workgroups read all of X in each, which
// a product over tiles of 128 x 128 does not (128 rows: 4096 x 4096 23 us here and 28 by tiles, 14336 x
// 4096 64 and 41, 4096 x 14336 60 and 42; 64 rows: 14336 x 4096 33 and 36, 4096 x 14336 41 and 37, where
// the rule, which does not go by the reduction's length, loses).
bool adapter_stream_fits(int64_t M, int64_t N, int64_t K) { return M <= 64 || (M <= kStreamMaxRows && N * K < (int64_t(1) << 25)); }

// Where the stream's workgroups form T and post it: one tile of rows, few enough elements that no
// workgroup forms more than two and that the posted words (elements times workgroups) cost less
// than the launch that they save (replayed, here and in two launches: 4096 x 4096: one row of 16 ranks
// 9.3 us and 12.4, of 64 10.7 and 12.6, 8 rows of 16 11.3 and 12.9; 14336 x 4096: one row of 16 19.9 and
// 22.7; 4096 x 14336: 18.4 and 26.9.  At the rule's edges little is left of it: 4096 x 4096, one row of
// 128 ranks 13.6 and 13.3, 16 rows of 8 13.6 and 13.3; 64 x 64 7.4 and 7.1.  Past them: 14336 x 4096,
// 8 rows of 8 ranks, 57000 words, 33 and 24; 64 x 64, four elements each, 8.6 and 7.0).
bool stream_forms_t(int64_t M, int64_t N, int32_t width) {
  const int64_t slots = M * width, groups = N / kStreamRows;
  static_assert(kPostedWords * sizeof(uint64_t) <= QLORA_WS_COUNTER_BYTES, "in the workspace's head");
  return M <= 16 && slots <= 2 * groups && slots * groups <= kPostedWords;
}

hipError_t launch_adapter_stream(const uint32_t* codes, const uint8_t* code8, const float* c2s, const float* mu,
                                 int64_t N, int64_t K, const uint16_t* X, const AdapterRows& rows, const DropMask& drop,
                                 float* T, uint16_t* Y, void* head, int32_t polls, const Nf4Tables& tab, hipStream_t st) {
  if (rows.M > kStreamMaxRows) return hipErrorInvalidValue;
  const int tiles = (int)((rows.M + kRowTile - 1) / kRowTile), ranks = (rows.width + 15) / 16;
  const StreamArgs a{reinterpret_cast<const uint8_t*>(codes), code8, c2s, mu, N, K, X, rows, drop, T, Y,
                     std::min((int)rows.count, kRowTile), static_cast<uint64_t*>(head), polls};
  const bool wide = N / kStreamRows > 512;  // more single tiles than workgroups of eight wavefronts fit at once
  if (stream_forms_t(rows.M, N, rows.width))
    return wide ? stream_go<4, 1, 1, true, 4>(a, tab, st) : stream_go<8, 1, 1, true, 4>(a, tab, st);
  const dim3 grid_t((unsigned)(tiles * ranks * a.lists));
  if (drop.threshold) hipLaunchKernelGGL(k_adapter_t<true>, grid_t, dim3(kStreamThreads), 0, st, a);
  else hipLaunchKernelGGL(k_adapter_t<false>, grid_t, dim3(kStreamThreads), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (rows.M <= 16) return wide ? stream_go<4, 1, 1, false, 4>(a, tab, st) : stream_go<8, 1, 1, false, 4>(a, tab, st);
  if (rows.M > 96) return wide ? stream_go<4, 1, 8, false, 1>(a, tab, st) : stream_go<8, 1, 8, false, 1>(a, tab, st);
  // two weight tiles to a workgroup where that leaves one for each compute unit (and registers last), by
  // four wavefronts, and by eight at the narrowest of these weights, whose 256 workgroups are one each
  if (N < 8192) return stream_as<8, 1>(a, tab, st);
  return wide ? stream_as<4, 2>(a, tab, st) : stream_as<8, 2>(a, tab, st);
}

GradPlan adapter_grad_plan(int64_t M, int64_t N, int64_t K, int32_t count, int32_t max_rank) {
  GradPlan p{};
  p.tiles_a = (K + kGradCols - 1) / kGradCols;
  p.tiles_b = (N + kGradCols - 1) / kGradCols;
  p.blocks = (max_rank + kGradRanks - 1) / kGradRanks;
  p.split = 1;
  const int64_t groups = (p.tiles_a + p.tiles_b) * count * p.blocks;
  while (groups * p.split < 512 && (int64_t)p.split * 2 * 512 <= M && p.split < 64) p.split *= 2;
  if (p.split > 1) p.part_bytes = sizeof(float) * (size_t)groups * p.split * kGradRanks * kGradCols;
  return p;
}

hipError_t launch_adapter_grads(const AdapterRows& rows, const uint16_t* X, int64_t K, const uint16_t* dY, int64_t N,
                                const float* T, const float* G, const DropMask& drop, float* part,
                                unsigned int* counters, hipStream_t st) {
  const GradPlan plan = adapter_grad_plan(rows.M, N, K, rows.count, rows.max_rank);
  GradsArgs a{rows, X, dY, T, G, K, N, drop, part, counters, (uint32_t)plan.tiles_a, plan.blocks, plan.split, 0};
  a.mps = ((rows.M + plan.split - 1) / plan.split + 31) / 32 * 32;
  if (rows.max_rank <= 16) return grads_as<1>(a, plan, st);
  if (rows.max_rank <= 32) return grads_as<2>(a, plan, st);
  return grads_as<4>(a, plan, st);
}

}  // namespace qlora
