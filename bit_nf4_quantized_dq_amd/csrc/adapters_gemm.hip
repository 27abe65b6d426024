// Products with the stored weight for tens to about two thousand rows, each row with its own
// adapter: the weight is decoded tile by tile on chip (exactly w_hat), so no decoded copy is written
// and read back.
//
//   forward : Y[m][n]  = sum_k w_hat[n][k] X[m][k]    + adapters     features n, reduction k
//   dX      : dX[m][k] = sum_n w_hat[n][k] dY[m][n]   + adapters     features k, reduction n
//
// Tile: 128 features x 128 TJ tokens per workgroup of eight wavefronts (2 x 4, each 64 features x
// 32 TJ tokens of MFMA 32x32x16), reduction step 64.  A step decodes 128 blocks of 64 weights, two
// threads to a block and its level table, so four wavefronts decode in one step and the other
// four in the next: each SIMD holds one of either kind, and one's decode (vector units) meets the
// other's products (matrix units).  A step of 128 x 256 takes 0.95 us, as long as the GEMM over a
// decoded copy takes for its share: both read 32 KB of activations a step through the L2.  (Four
// wavefronts that all decode, two workgroups to a compute unit: 1.1 us for 128 x 128; 1024 rows of
// 4096 x 4096 backward 96 us, here 76.)  Few tiles split the reduction over several workgroups (FP32
// partials, added in order by launch_sum_parts).
//
// Pipeline: step kb issues the activations' direct loads to LDS for step kb + 2 (ring of three); half
// of the wavefronts load their codes for it (registers) and the other half decodes step kb + 1
// into the other weight buffer while both multiply step kb; then the activations of step kb + 1 are
// waited for and one barrier passed.  Every buffer is a __shared__ array of its own, known at
// compile time in a loop unrolled six times, so that the compiler waits only for the loads an
// access needs.
//
// LDS.  Activations and the forward's weight: rows of 128 bytes, 16-byte chunk c of row r at c ^
// (r / 2 % 8).  The transposed weight: rows n of 128 features in 64-byte units, unit u at u ^ (n % 4),
// read with transposing reads (8 consecutive n of one feature); the four rows of a read then meet
// all banks.
#include "adapter_head.h"

namespace qlora {
namespace {

constexpr int kThreads = 512;
constexpr int BF = 128;   // features per workgroup
constexpr int BK = 64;    // reduction step
constexpr int TI = 2;     // 32 x 32 tiles per wavefront: TI of features, TJ of tokens
template <int TJ> constexpr int kTokens = 128 * TJ;  // tokens per workgroup
typedef __attribute__((address_space(3))) void lds_void;

// An offset past every operand (tiles are below 2^31 bytes, the scalar offsets of steps below 2^24):
// reads zeros however a step's offset adds to it.
constexpr uint32_t kFar = 0xF0000000u;

template <int N> __device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}
// Own LDS accesses done, then the workgroup barrier (also a compiler memory barrier).
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  asm volatile("s_barrier" ::: "memory");
}

// (sized for TJ = 2; a workgroup has a compute unit to itself with TJ = 1 too)
__shared__ uint4 s_w0[1024], s_w1[1024];              // decoded weights, 16 KB each
__shared__ uint4 s_x0[2048], s_x1[2048], s_x2[2048];  // activations, 32 KB each
template <int I> __device__ __forceinline__ uint4* wbuf() { return I == 0 ? s_w0 : s_w1; }
template <int I> __device__ __forceinline__ uint4* xbuf() { return I == 0 ? s_x0 : (I == 1 ? s_x1 : s_x2); }

struct MidArgs {
  const uint8_t *codes, *code8;
  const float *c2s, *mu;
  int64_t N, K;
  const uint16_t* X;  // [M, Kr]
  int64_t M, F, Kr;   // features and reduction: (N, K), or (K, N) for dX
  AdapterHead head;
  uint16_t* C;
  float* part;
  uint32_t kb_per;
};

// Activation ring: 128 TJ rows from m0.  Wavefront w fills rows 16 TJ w .. of a slot, eight rows
// of 128 bytes a load; lane p writes slot chunk p & 7 and fetches the chunk that belongs there.
template <int TJ>
struct Ring {
  static constexpr int kLoads = 2 * TJ;
  rsrc_t r;
  uint32_t base[kLoads], col[kLoads], Kr;
  int wave;
  __device__ __forceinline__ void init(const MidArgs& a, int64_t m0, int w, int lane) {
    const int64_t rows = a.M - m0 < kTokens<TJ> ? a.M - m0 : kTokens<TJ>;
    r = make_rsrc(a.X + m0 * a.Kr, rows * a.Kr * 2);
    Kr = (uint32_t)a.Kr;
    wave = w;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int row = 8 * (kLoads * w + j) + (lane >> 3), chunk = (lane & 7) ^ ((row >> 1) & 7);
      col[j] = 8 * chunk;
      base[j] = row < rows ? (uint32_t)(row * a.Kr * 2 + 16 * chunk) : kFar;
    }
  }
  template <int SLOT> __device__ __forceinline__ void issue(uint32_t kb) const {
    const uint32_t k0 = kb * BK;
    const bool whole = k0 + BK <= Kr;  // uniform: else the step is the product's last, or past it
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const uint32_t off = whole || k0 + col[j] < Kr ? base[j] : kFar;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(xbuf<SLOT>() + (kLoads * wave + j) * 64), 16, off, 2 * k0, 0, 0);
    }
  }
};

// The weight of a step: thread t decodes half a block, 32 weights.  Forward: row f0 + t / 2, block kb,
// half t % 2.  dX: row 64 kb + t / 4, block f0 / 64 + (t / 2) % 2, half t % 2.
template <bool WT>
struct Decoder {
  static constexpr int kLoads = 3;
  struct Regs {
    uint4 c;
    uint32_t c8, c2;
  };
  const uint8_t* codes;
  rsrc_t rc, r8, r2;
  int64_t codes_bytes;
  uint32_t row_bytes, nb, off, blk, to, chunk[4];
  float mu;
  int t;
  __device__ __forceinline__ void init(const MidArgs& a, int64_t f0, int tid) {
    t = tid;
    nb = (uint32_t)(a.K / 64);
    row_bytes = (uint32_t)(a.K / 2);
    codes = a.codes;
    codes_bytes = a.N * (a.K / 2);
    r8 = make_rsrc(a.code8, a.N * nb);
    r2 = make_rsrc(a.c2s, ((a.N * nb + 255) / 256) * 4);
    mu = a.mu[0];
    if (!WT) {
      const uint32_t row = (uint32_t)f0 + (t >> 1);
      rc = make_rsrc(codes + f0 * row_bytes, (a.N - f0) * row_bytes);
      off = row < a.N ? (t >> 1) * row_bytes + 16 * (t & 1) : kFar;
      blk = row < a.N ? row * nb : 0;
      const int s = ((t >> 2) & 7) ^ (4 * (t & 1));
      to = 8 * (t >> 1);
#pragma unroll
      for (int c = 0; c < 4; ++c) chunk[c] = to + (s ^ c);
    } else {
      const uint32_t b = (uint32_t)(f0 / 64) + ((t >> 1) & 1);
      off = b < nb ? (t >> 2) * row_bytes + 32 * b + 16 * (t & 1) : kFar;
      blk = (t >> 2) * nb + (b < nb ? b : 0);
      to = 16 * (t >> 2) + 4 * ((t & 3) ^ ((t >> 2) & 3));  // features 32 (t & 3) ..
#pragma unroll
      for (int c = 0; c < 4; ++c) chunk[c] = to + c;
    }
  }
  // Steps past the product load its last one again (into registers that nothing uses); rows past the
  // weight read as zero codes, whose products meet rows of the activations that are zero.
  __device__ __forceinline__ void load(Regs& R, uint32_t kb) const {
    if (!WT) {
      const uint32_t k = kb < nb ? kb : nb - 1;
      R.c = load16(rc, off, 32 * k);
      const uint32_t at = blk + k;
      R.c8 = bload1(r8, at);
      R.c2 = bload4(r2, (at >> 8) * 4);
    } else {
      const int64_t step = (int64_t)kb * BK * row_bytes;
      R.c = load16(make_rsrc(codes + step, codes_bytes - step), off, 0);
      const uint32_t at = blk + kb * BK * nb;
      R.c8 = bload1(r8, at);
      R.c2 = bload4(r2, (at >> 8) * 4);
    }
  }
  static __device__ __forceinline__ uint4 load16(rsrc_t r, uint32_t off, uint32_t scalar) {
    const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, (int)scalar, 0);
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
  // The level table of the thread's block, then its words one by one.
  __device__ __forceinline__ void table(const Regs& R, const Nf4Tables& tab, Lut& L) const {
    build_scaled_lut(tab, stored_scale(R.c8, __uint_as_float(R.c2), mu), L);
  }
  __device__ __forceinline__ void store(uint4* __restrict__ w, const Regs& R, const Lut& L, int c) const {
    const uint32_t words[4] = {R.c.x, R.c.y, R.c.z, R.c.w};
    uint32_t o[4];
    decode8(words[c], L, o);
    w[chunk[c]] = make_uint4(o[0], o[1], o[2], o[3]);
  }
};

// Operand of features 32 u .. 32 u + 31, reduction indices 16 ks + 8 (lane >> 5) .. +7 of a step.
template <bool WT>
__device__ __forceinline__ bf16x8_t w_operand(const uint4* __restrict__ w, int u, int ks, int lane) {
  const int l32 = lane & 31, h32 = lane >> 5;
  if (!WT) {
    const int row = 32 * u + l32;
    return as_bf16x8(w[8 * row + ((2 * ks + h32) ^ ((row >> 1) & 7))]);
  }
  const int j = lane & 15, n = 16 * ks + 8 * h32 + (j >> 2);
  const char* p = reinterpret_cast<const char*>(w) + 256 * n + 64 * (u ^ (n & 3)) + 32 * ((lane >> 4) & 1) + 8 * (j & 3);
  const lds_i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(p));
  const lds_i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(p + 4 * 256));
  bf16x8_t r;
  r[0] = lo[0]; r[1] = lo[1]; r[2] = lo[2]; r[3] = lo[3];
  r[4] = hi[0]; r[5] = hi[1]; r[6] = hi[2]; r[7] = hi[3];
  return r;
}

// Step kb of a wavefront.  The group whose turn it is (DEC) decodes step kb + 1 from R; the other
// loads R for step kb + 2.  `live`: the wavefront has tokens (uniform).
template <bool WT, int TJ, bool DEC, int XS, int WB>
__device__ __forceinline__ void mid_step(const Decoder<WT>& dec, const Ring<TJ>& ring, const Nf4Tables& tab, uint32_t kb,
                                         uint32_t last, typename Decoder<WT>::Regs& R, int wf, int wm, int lane, bool live,
                                         f32x16_t (&acc)[TI][TJ]) {
  // loads past the range go into buffers that nothing reads
  const uint32_t k2 = kb + 2 < last ? kb + 2 : last;
  if (!DEC) dec.load(R, k2);
  ring.template issue<(XS + 2) % 3>(k2);
  const int l32 = lane & 31, h32 = lane >> 5;
  Lut L;
  if (DEC) dec.table(R, tab, L);
  if (live) {
    bf16x8_t x[2][TI], y[2][TJ];
    const auto read = [&](int ks) {
#pragma unroll
      for (int i = 0; i < TI; ++i) x[ks & 1][i] = w_operand<WT>(wbuf<WB>(), wf / 32 + i, ks, lane);
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const int row = wm + 32 * j + l32;
        y[ks & 1][j] = as_bf16x8(xbuf<XS>()[8 * row + ((2 * ks + h32) ^ ((row >> 1) & 7))]);
      }
    };
    read(0);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks < 3) read(ks + 1);
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = mfma32(x[ks & 1][i], y[ks & 1][j], acc[i][j]);
      if (DEC) dec.store(wbuf<WB ^ 1>(), R, L, ks);
    }
    // operands one 16-wide step ahead; the decode's vector instructions between the products, each of
    // which holds the matrix unit for 32 clocks
    constexpr int kReads = WT ? 2 * TI + TJ : TI + TJ;
    __builtin_amdgcn_sched_group_barrier(0x100, 2 * kReads, 0);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
#pragma unroll
      for (int q = 0; q < TI * TJ; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (DEC) __builtin_amdgcn_sched_group_barrier(0x002, 40 / (TI * TJ), 0);
      }
      if (ks < 2) __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
    }
  } else if (DEC) {
#pragma unroll
    for (int c = 0; c < 4; ++c) dec.store(wbuf<WB ^ 1>(), R, L, c);
  }
  // the activations of step kb + 1 have landed
  wait_vm<DEC ? Ring<TJ>::kLoads : Ring<TJ>::kLoads + Decoder<WT>::kLoads>();
  lds_barrier();
}

// The steps of the wavefronts of group G: those with kb - kb0 of G's parity load, the others decode.
template <bool WT, int TJ, int G>
__device__ __forceinline__ void mid_loop(const Decoder<WT>& dec, const Ring<TJ>& ring, const Nf4Tables& tab, uint32_t kb0,
                                         uint32_t kb1, uint32_t nk, typename Decoder<WT>::Regs& R, int wf, int wm, int lane,
                                         bool live, f32x16_t (&acc)[TI][TJ]) {
  for (uint32_t kb = kb0; kb < kb1; kb += 6) {
    mid_step<WT, TJ, G == 1, 0, 0>(dec, ring, tab, kb + 0, nk, R, wf, wm, lane, live, acc);
    if (kb + 1 >= kb1) break;
    mid_step<WT, TJ, G == 0, 1, 1>(dec, ring, tab, kb + 1, nk, R, wf, wm, lane, live, acc);
    if (kb + 2 >= kb1) break;
    mid_step<WT, TJ, G == 1, 2, 0>(dec, ring, tab, kb + 2, nk, R, wf, wm, lane, live, acc);
    if (kb + 3 >= kb1) break;
    mid_step<WT, TJ, G == 0, 0, 1>(dec, ring, tab, kb + 3, nk, R, wf, wm, lane, live, acc);
    if (kb + 4 >= kb1) break;
    mid_step<WT, TJ, G == 1, 1, 0>(dec, ring, tab, kb + 4, nk, R, wf, wm, lane, live, acc);
    if (kb + 5 >= kb1) break;
    mid_step<WT, TJ, G == 0, 2, 1>(dec, ring, tab, kb + 5, nk, R, wf, wm, lane, live, acc);
  }
}

template <bool WT, int TJ>
__global__ __launch_bounds__(kThreads, 2) void k_adapter_gemm(MidArgs a, Nf4Tables tab) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wf = (wave & 1) * 64, wm = (wave >> 1) * 32 * TJ;
  const int64_t f0 = (int64_t)blockIdx.x * BF, m0 = (int64_t)blockIdx.y * kTokens<TJ>;
  const uint32_t nk = (uint32_t)((a.Kr + BK - 1) / BK);
  const uint32_t kb0 = blockIdx.z * a.kb_per, kb1 = kb0 + a.kb_per < nk ? kb0 + a.kb_per : nk;
  Ring<TJ> ring;
  ring.init(a, m0, wave, lane);
  Decoder<WT> dec;
  dec.init(a, f0, tid & 255);
  // group 0 decodes the first step here, group 1 the second in the loop
  const int group = wave >> 2;
  const bool live = m0 + wm < a.M;
  typename Decoder<WT>::Regs R;
  ring.template issue<0>(kb0);
  dec.load(R, kb0 + group < nk ? kb0 + group : nk);
  ring.template issue<1>(kb0 + 1 < nk ? kb0 + 1 : nk);
  f32x16_t acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f32x16_t{};
  // (s_x2 is free until the barrier)
  const bool any = live && adapter_rows<WT>(a.head, a.F, f0 + wf, m0 + wm, lane, reinterpret_cast<char*>(s_x2) + wave * 4096,
                                            blockIdx.z, gridDim.z, acc);
  if (WT && any && a.head.drop.threshold) drop_acc(a.head.drop, a.F, f0 + wf, m0 + wm, lane & 31, lane >> 5, acc);
  if (group == 0) {
    Lut L;
    dec.table(R, tab, L);
#pragma unroll
    for (int c = 0; c < 4; ++c) dec.store(s_w0, R, L, c);
  }
  wait_vm<0>();
  lds_barrier();
  if (group == 0) mid_loop<WT, TJ, 0>(dec, ring, tab, kb0, kb1, nk, R, wf, wm, lane, live, acc);
  else mid_loop<WT, TJ, 1>(dec, ring, tab, kb0, kb1, nk, R, wf, wm, lane, live, acc);
  wait_vm<0>();   // the loads issued past the range have landed
  lds_barrier();  // every wavefront is done with the buffers, which now stage the result
  // 32 tokens x 64 features of FP32 at a time (8 KB of the wavefront's own): 16-byte unit u of row m at
  // u ^ (m % 16); read back so that each row leaves in whole
  uint4* stage = (wave < 4 ? s_x0 : s_x1) + (wave & 3) * 512;
  const int l32 = lane & 31, h32 = lane >> 5;
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int u = 8 * i + 2 * q + h32;
        stage[16 * l32 + (u ^ (l32 & 15))] = make_uint4(__float_as_uint(acc[i][j][4 * q]), __float_as_uint(acc[i][j][4 * q + 1]),
                                                        __float_as_uint(acc[i][j][4 * q + 2]), __float_as_uint(acc[i][j][4 * q + 3]));
      }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // its own writes are done (it reads only its own region)
    asm volatile("" ::: "memory");
    if (a.part) {
      float* part = a.part + (int64_t)blockIdx.z * a.M * a.F;
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        const int m = 4 * it + (lane >> 4), c = lane & 15;
        const uint4 v = stage[16 * m + (c ^ (m & 15))];
        const int64_t gm = m0 + wm + 32 * j + m, gf = f0 + wf + 4 * c;
        if (gm < a.M && gf < a.F) *reinterpret_cast<uint4*>(part + gm * a.F + gf) = v;
      }
    } else {
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int m = 8 * it + (lane >> 3), c = lane & 7;
        const uint4 v = stage[16 * m + ((2 * c) ^ (m & 15))], w = stage[16 * m + ((2 * c + 1) ^ (m & 15))];
        const int64_t gm = m0 + wm + 32 * j + m, gf = f0 + wf + 8 * c;
        if (gm < a.M && gf < a.F)
          *reinterpret_cast<uint4*>(a.C + gm * a.F + gf) =
              make_uint4(pack_bf16x2(__uint_as_float(v.x), __uint_as_float(v.y)), pack_bf16x2(__uint_as_float(v.z), __uint_as_float(v.w)),
                         pack_bf16x2(__uint_as_float(w.x), __uint_as_float(w.y)), pack_bf16x2(__uint_as_float(w.z), __uint_as_float(w.w)));
      }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // reads done before the next rows
    asm volatile("" ::: "memory");
  }
}

int64_t mid_tiles(int64_t M, int64_t F, int tj) { return ((F + BF - 1) / BF) * ((M + 128 * tj - 1) / (128 * tj)); }

// Tiles of 256 tokens (TJ = 2) read the weight and the activations less often; of 128 where there are no
// more rows, and for short reductions, whose time goes into the tiles' start and end (555 rows over
// 1040 to 4096: 53 us in tiles of 128 and 58 in tiles of 256; 1024 rows over 4096 to 4096: 87 and 76).
int mid_tj(int64_t M, int64_t F, int64_t Kr) { return M <= 128 || (Kr < 32 * BK && mid_tiles(M, F, 1) <= 256) ? 1 : 2; }

}  // namespace

// From about one tile for each compute unit on, the weight decoded once and the larger tiles of the
// GEMM over the copy are faster (400 rows of 14336 x 4096, 224 tiles: 85 us here and 103 there;
// 8192 rows of 1024 x 4096, 256 tiles: 101 and 95; 1024 rows of 14336 x 4096, 448: 157 and 136).
bool adapter_gemm_fits(int64_t M, int64_t F, int64_t Kr) { return M <= 128 || mid_tj(M, F, Kr) == 1 || mid_tiles(M, F, 2) <= 224; }

int32_t adapter_gemm_split(int64_t M, int64_t F, int64_t Kr) {
  // a workgroup to a compute unit, and four steps at least to a split (1999 rows of 1024 x 4096: 80 us
  // whole, 58 in two, 50 in four, 62 in eight)
  const int64_t nk = (Kr + BK - 1) / BK, tiles = mid_tiles(M, F, mid_tj(M, F, Kr));
  return (int32_t)std::max<int64_t>(1, std::min<int64_t>(256 / tiles, nk / 4));
}

hipError_t launch_adapter_gemm(const uint32_t* codes, const uint8_t* code8, const float* c2s, const float* mu, int64_t N,
                               int64_t K, const uint16_t* X, int64_t M, const AdapterHead& head, uint16_t* C, float* part,
                               int32_t split, const Nf4Tables& tab, int kernel_id, hipStream_t st) {
  const int64_t F = head.transposed ? K : N, Kr = head.transposed ? N : K;
  if (split > 1 && !part) return hipErrorInvalidValue;
  const uint32_t nk = (uint32_t)((Kr + BK - 1) / BK), kb_per = (nk + split - 1) / split;
  const uint32_t splits = (nk + kb_per - 1) / kb_per;  // no split is empty
  const MidArgs a{reinterpret_cast<const uint8_t*>(codes), code8, c2s, mu, N, K, X, M, F, Kr, head, C, splits > 1 ? part : nullptr, kb_per};
  const int tj = mid_tj(M, F, Kr);
  const dim3 grid((unsigned)((F + BF - 1) / BF), (unsigned)((M + 128 * tj - 1) / (128 * tj)), splits);
  {
    LaunchTimer t(kernel_id, st);
    const auto go = [&](auto kernel) { hipExtLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, st, t.start, t.stop, 0, a, tab); };
    if (tj == 1) head.transposed ? go(k_adapter_gemm<true, 1>) : go(k_adapter_gemm<false, 1>);
    else head.transposed ? go(k_adapter_gemm<true, 2>) : go(k_adapter_gemm<false, 2>);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits <= 1) return e;
  return launch_sum_parts(part, (int32_t)splits, M, F, C, st);
}

}  // namespace qlora
