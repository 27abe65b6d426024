// Block norms: the root-mean-square norm after a block, its gate and residual scale, and the
// norm before the next block, as one pass over the rows, with the backward.
//
//   n  = y                                   (or y r_y w_post,  r_y = (mean(y^2) + eps)^-1/2)
//   x' = s x + g n
//   h  = x' r_x w_pre,                        r_x = (mean(x'^2) + eps)^-1/2
//
// and, given dh and the gradient dx' that reaches x' from later blocks, with a = dh w_pre:
//   t    = dx' + r_x a - x' r_x^3 mean(a x')
//   dx   = s t,     dw_pre = sum_rows dh x' r_x,     dgate = sum_rows t n
//   b    = t g w_post,   dy = r_y b - y r_y^3 mean(b y),   dw_post = sum_rows t g y r_y
// (without the norm after the block dy = t g).
//
// A row is read once and held in registers, eight columns to a thread, and its sums cross the
// workgroup through LDS, so the forward moves 8 and the backward 12 bytes an element (BF16
// stream).  HBM bounds the forward: a simple copy reaches 6.3 TB/s on this card.  The backward
// is bound by HBM and by the issue of vector instructions at once: 579 a wavefront and row, four
// cycles each, are 62 of the 77 us that its kernel takes at 4096 x 8192 (its bytes, partials
// included, 68 us), and 24 of 36 us at 8192 x 1280 (bytes 23 us), where 17% of the lanes hold no
// columns.  What it takes to
// come near the copy is to keep loads in flight during the exchanges: the next row's are issued
// before this row's sums (without it 114 us for 4096 x 8192 backward, with it 80), and every
// load and store is unconditional, so that the compiler's counters tell loads from stores.
// Measured (MI355X, BF16, post-norm and one gate): forward 8192 x 4096 45 - 50 us (5.4 - 6.0
// TB/s), 4096 x 8192 46 us, 1 x 4096 2.9 us on the device; backward with every gradient 4096 x
// 8192 77 - 82 us (5.0 TB/s), 8192 x 4096 77 - 82 us, 8192 x 1280 38 us; without post-norm and gate
// and with frozen weights 8192 x 4096 42 us forward and 68 us backward, 4096 x 8192 42 and 66,
// 8192 x 1280 13 and 29.  FP32 sums and statistics; each output is rounded once.
#include "qlora_train_host.h"
#include "train_device.h"

namespace qlora {
namespace {

// The gate of a row: none or one gate row for a run of rows (loaded where a run begins), or loaded
// with each row.
enum GateKind { kGateRuns, kGateRows };
// Which outputs: any of them, or both large ones (stored without a branch); in the backward the
// latter also with operands larger than the cache, which are read past it.
enum Outputs { kAny, kBoth, kBothStream };

template <class S>
struct FwdArgs {
  const S* x;
  const uint16_t *y, *w_post, *gate, *w_pre;  // y is never null here: see y_bits
  S* x_out;
  uint16_t* h;
  int64_t M, d, gate_rows;
  uint32_t y_bits;                // zeros where the block adds nothing
  float scale, eps, inv_d;
  int post;
};

// One workgroup of d / 8 threads (in whole wavefronts; ONE: one) for every gridDim.x-th row, one row at a time and eight columns to
// a thread: every operand is read once and kept in registers, the weights for all rows, and
// the next row is loaded while this one's two sums cross the workgroup.  (Rows that are worked
// on at the same time lie together in memory.)
template <class S, bool ONE, bool SHORT, GateKind KIND, Outputs OUT>
__global__ __launch_bounds__(ONE ? 64 : 1024) void k_norm_fwd(FwdArgs<S> a) {
  __shared__ float lds[2][2][16];
  const int64_t d = a.d;
  const uint32_t rows = (uint32_t)a.M, run = (uint32_t)a.gate_rows;  // below 2^24
  const Columns<SHORT> col((int)d, 8 * threadIdx.x);
  Raw8<S> x, x_next;
  Raw8<uint16_t> y, y_next, g, g_next, w_post, w_pre;
  col.load(x, a.x + blockIdx.x * d);
  col.load(y, a.y + blockIdx.x * d);
  if (a.gate) col.load(g, a.gate + (KIND == kGateRows ? blockIdx.x / run * d : 0));
  else ones8(g);
  if (a.w_post) col.load(w_post, a.w_post);
  else ones8(w_post);
  if (a.w_pre) col.load(w_pre, a.w_pre);
  else ones8(w_pre);
  // all of it waited for here: a load that may still be under way where the loop is entered
  // would make each row wait for the stores of the row before
  opaque(w_post), opaque(w_pre), opaque(g), opaque(x), opaque(y);
  bool odd = false;
  for (uint32_t row = blockIdx.x; row < rows; row += gridDim.x, odd = !odd) {
    // past the last row: once more the last one, so that the loop's loads need no condition
    const uint32_t ahead = row + gridDim.x < rows ? row + gridDim.x : row;
    col.load(x_next, a.x + ahead * d);
    col.load(y_next, a.y + ahead * d);
    if constexpr (KIND == kGateRows) col.load(g_next, a.gate + ahead / run * d);
    and8(y, a.y_bits);
    float r_y = 1.f;
    if (a.post) {
      const Raw8<uint16_t> own = col.own(y);
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] = fmaf(own.get(i), own.get(i), s[0]);
      block_sum<ONE>(s, lds[odd][0]);
      r_y = 1.f / sqrtf(s[0] * a.inv_d + a.eps);
    }
    Raw8<float> xo;
#pragma unroll
    for (int i = 0; i < 8; ++i) xo.f[i] = a.scale * x.get(i) + y.get(i) * r_y * w_post.get(i) * g.get(i);
    const Raw8<float> own = col.own(xo);
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] = fmaf(own.f[i], own.f[i], s[0]);
    // (also where h is not wanted: the exchange lies between the loads of a row and the stores
    // that may replace it)
    block_sum<ONE>(s, lds[odd][1]);
    if (OUT != kAny || a.x_out) col.store(a.x_out + row * d, xo.f);
    if (OUT != kAny || a.h) {
      const float r_x = 1.f / sqrtf(s[0] * a.inv_d + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) xo.f[i] *= r_x * w_pre.get(i);
      col.store(a.h + row * d, xo.f);
    }
    x = x_next, y = y_next;
    if constexpr (KIND == kGateRows) g = g_next;
  }
}

template <class S>
struct BwdArgs {
  // an operand that is not given points at another of the call (read, and made zeros by its bits)
  const S* x;  // x', as the forward stored it
  const uint16_t *y, *dh;
  const S* dx_out;
  const uint16_t *w_post, *gate, *w_pre;
  S* dx;
  uint16_t* dy;
  uint16_t* dgate;                 // for gate rows whole in a segment, else null
  float *p_pre, *p_post, *p_gate;  // [segment][d] FP32 partials, null where not wanted
  unsigned int* counter;           // for few partials, which the last workgroup adds (else null)
  uint16_t *sum_pre, *sum_post, *sum_gate;  // where it writes the sums
  int64_t M, d, gate_rows;
  NormSegments seg;
  uint32_t y_bits, h_bits, o_bits;  // y; x and dh; dx_out
  float scale, eps, inv_d;
  int post;
};

// What one row gives a lane's columns.
template <class S, bool SHORT, GateKind KIND, bool STREAM>
struct RowVec {
  Raw8<S> x, dxo;
  Raw8<uint16_t> y, dh, g;
  __device__ __forceinline__ void load(const BwdArgs<S>& a, const Columns<SHORT>& col, int64_t at) {
    load_in<STREAM>(col, x, a.x + at);
    load_in<STREAM>(col, dh, a.dh + at);
    load_in<STREAM>(col, dxo, a.dx_out + at);
    load_in<STREAM>(col, y, a.y + at);
    if constexpr (KIND == kGateRows) col.load(g, a.gate + at);
  }
  __device__ __forceinline__ void pack() { opaque(x), opaque(dxo), opaque(y), opaque(dh), opaque(g); }
};

// Few partials: the last workgroup to finish adds them in the segments' order.  (A second launch
// takes 3 us of the host and 4 of the device; here each workgroup writes its L2 back once, and
// one of them reads all partials, which is as long at about 256 KB.)
constexpr int64_t kFewSegments = 32;
constexpr size_t kFewBytes = 256 * 1024;
template <class S, bool SHORT>
__device__ void add_segments(const BwdArgs<S>& a, const Columns<SHORT>& col) {
  __shared__ bool last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const unsigned int old = __hip_atomic_fetch_add(a.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = old + 1u == gridDim.x;
    if (last) __hip_atomic_store(a.counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  const auto add = [&](const float* p, int64_t first, int64_t count, uint16_t* out) {
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int64_t s = first; s < first + count; ++s) {
      Raw8<float> r;
      col.load(r, p + s * a.d);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += r.f[i];
    }
    col.store(out, sum);
  };
  if (a.p_pre) add(a.p_pre, 0, gridDim.x, a.sum_pre);
  if (a.p_post) add(a.p_post, 0, gridDim.x, a.sum_post);
  if (a.p_gate)
    for (int64_t g = 0; g * a.seg.per_group < gridDim.x; ++g)
      add(a.p_gate, g * a.seg.per_group, a.seg.per_group, a.sum_gate + g * a.d);
}

// One workgroup per segment of rows.  Its threads own columns, so the column sums (weights, gate)
// stay in registers over the segment; the sums over a row are one exchange: with q = g w_post y,
// sum(b y) = sum(dx' q) + r_x sum(a q) - k r_x sum(x' q),  k = r_x^2 mean(a x').  The third factor
// r_x goes to x' itself (and r_y's to y): u = r_x x' is of order one, and no cube of a row's
// norm leaves FP32's range before what it multiplies brings it back.
// An operand that is not given is zeros, a weight or gate that is not given is ones, so the
// arithmetic has no cases.
// What keeps it below the forward's rate: the instructions (operands are unpacked on both sides
// of the exchange, each thread takes two square roots and two reciprocals a row, and the next
// row is copied into this one's registers), four wavefronts a SIMD to hide a row's latency
// behind (24 sums, two rows and the weights take 103 - 127 registers), and the partials, 12 bytes
// a column and segment (25 MB written and read again beside 403 MB at 4096 x 8192).
template <class S, bool ONE, bool SHORT, GateKind KIND, Outputs OUT>
__global__ __launch_bounds__(ONE ? 64 : 1024, SHORT ? 1 : 4) void k_norm_bwd(BwdArgs<S> a) {
  __shared__ float lds[2][6 * 16];
  const int64_t d = a.d, seg = blockIdx.x;
  // a segment of whole gate rows, or one of per_group segments that share a gate row's rows
  int64_t r0 = seg * a.seg.rows, r1 = r0 + a.seg.rows < a.M ? r0 + a.seg.rows : a.M, group;
  int64_t step = 1;
  if (a.seg.per_group) {
    // (rows that are worked on at the same time lie together in memory)
    group = seg / a.seg.per_group;
    step = a.seg.per_group;
    r0 = group * a.gate_rows + (seg - group * step);
    r1 = (group + 1) * a.gate_rows < a.M ? (group + 1) * a.gate_rows : a.M;
  } else {
    group = r0 / a.gate_rows;
  }
  int64_t group_end = (group + 1) * a.gate_rows;
  const Columns<SHORT> col((int)d, 8 * threadIdx.x);
  // s_tu: sum of t u over the rows of one gate row; times the gate it goes into dw_post, times
  // w_post it is the gate's gradient
  float s_pre[8], s_post[8], s_tu[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s_pre[i] = s_post[i] = s_tu[i] = 0.f;
  if (r0 >= r1) {  // a segment past the rows of a short last gate row
    if (a.p_pre) col.store(a.p_pre + seg * d, s_pre);
    if (a.p_post) col.store(a.p_post + seg * d, s_post);
    if (a.p_gate) col.store(a.p_gate + seg * d, s_tu);
    if (a.counter) add_segments(a, col);
    return;
  }
  RowVec<S, SHORT, KIND, OUT == kBothStream> r, next;
  r.load(a, col, r0 * d);
  Raw8<uint16_t> w_pre, w_post;
  if (a.w_pre) col.load(w_pre, a.w_pre);
  else ones8(w_pre);
  if (a.w_post) col.load(w_post, a.w_post);
  else ones8(w_post);
  if constexpr (KIND == kGateRuns) {
    if (a.gate) col.load(r.g, a.gate + group * d);
    else ones8(r.g);
  }
  // all of it waited for here: a load that may still be under way where the loop is entered
  // would make each row wait for the stores of the row before
  opaque(w_pre), opaque(w_post), r.pack();
  const bool post = a.post != 0;
  const uint32_t post_bits = post ? 0xFFFFFFFFu : 0u;
  const bool all = (a.y_bits & a.h_bits & a.o_bits) != 0u;
  bool odd = false;
  for (int64_t row = r0; row < r1; row += step, odd = !odd) {
    const int64_t at = row * d;
    // the next row's loads run under this row's exchange (past the last row: that one again)
    next.load(a, col, (row + step < r1 ? row + step : row) * d);
    // what is held across the exchange stays packed (unpacked once for both uses it would take
    // 56 registers more)
    opaque(w_pre), opaque(w_post), r.pack();
    if (!all) and8(r.x, a.h_bits), and8(r.dh, a.h_bits), and8(r.dxo, a.o_bits), and8(r.y, a.y_bits);
    const Raw8<S> x_own = col.own(r.x);
    const Raw8<uint16_t> y_own = col.own(r.y);
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float xi = x_own.get(i), yi = y_own.get(i), ai = r.dh.get(i) * w_pre.get(i);
      const float q = yi * w_post.get(i) * r.g.get(i);
      s[0] = fmaf(xi, xi, s[0]);
      s[1] = fmaf(ai, xi, s[1]);
      s[2] = fmaf(yi, yi, s[2]);
      s[3] = fmaf(r.dxo.get(i), q, s[3]);
      s[4] = fmaf(ai, q, s[4]);
      s[5] = fmaf(xi, q, s[5]);
    }
    block_sum<ONE>(s, lds[odd]);
    opaque(w_pre), opaque(w_post), r.pack();
    const float r_x = a.h_bits ? 1.f / sqrtf(s[0] * a.inv_d + a.eps) : 0.f;
    const float k = a.h_bits ? r_x * (r_x * (s[1] * a.inv_d)) : 0.f;
    const float r_y = post ? 1.f / sqrtf(s[2] * a.inv_d + a.eps) : 1.f;
    const float c = post ? r_y * (r_y * ((s[3] + r_x * s[4] - k * (r_x * s[5])) * a.inv_d)) : 0.f;
    float t[8], o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float ui = r.x.get(i) * r_x, dhi = r.dh.get(i);
      t[i] = r.dxo.get(i) + (r_x * (dhi * w_pre.get(i)) - ui * k);
      s_pre[i] = fmaf(dhi, ui, s_pre[i]);
      o[i] = a.scale * t[i];
    }
    if (OUT != kAny || a.dx) col.store(a.dx + at, o);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float vi = r.y.get(i) * r_y;
      s_tu[i] = fmaf(t[i], vi, s_tu[i]);
      o[i] = r_y * (t[i] * r.g.get(i) * w_post.get(i)) - __uint_as_float(__float_as_uint(vi) & post_bits) * c;
    }
    if (OUT != kAny || a.dy) col.store(a.dy + at, o);
    const Raw8<uint16_t> g = r.g;
    r = next;
    if constexpr (KIND == kGateRuns) r.g = g;
    if (KIND == kGateRows || row + 1 == group_end || row + step >= r1) {
      float dg[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s_post[i] = fmaf(s_tu[i], g.get(i), s_post[i]);
        dg[i] = s_tu[i] * w_post.get(i);
        s_tu[i] = 0.f;
      }
      if (a.dgate) col.store(a.dgate + group * d, dg);
      if (a.p_gate) col.store(a.p_gate + seg * d, dg);
      if (row + step < r1) {
        ++group, group_end += a.gate_rows;
        if constexpr (KIND == kGateRuns) {
          col.load(r.g, a.gate + group * d);
          opaque(r.g);  // waited for here, not in every row
        }
      }
    }
  }
  if (a.p_pre) col.store(a.p_pre + seg * d, s_pre);
  if (a.p_post) col.store(a.p_post + seg * d, s_post);
  if (a.counter) add_segments(a, col);
}

// Column sums of the segments' partials, in the segments' order within each of the 16 slices and
// the slices in order: job 0 dw_pre, job 1 dw_post over all segments, job 2 + g the gate's row
// g over its segments.  (256 segments of 8192 columns, three jobs: 5 us.)
constexpr int kColThreads = 1024, kCols = 64, kSlices = kColThreads / kCols;

__global__ __launch_bounds__(kColThreads) void k_norm_cols(const float* __restrict__ p_pre,
                                                           const float* __restrict__ p_post,
                                                           const float* __restrict__ p_gate, uint16_t* dw_pre,
                                                           uint16_t* dw_post, uint16_t* dgate, int64_t d,
                                                           int64_t nseg, int64_t per_group, int64_t job0) {
  __shared__ float lds[kSlices][kCols];
  const int64_t job = job0 + blockIdx.y;
  const float* p = job == 0 ? p_pre : (job == 1 ? p_post : p_gate);
  if (!p) return;
  uint16_t* out = job == 0 ? dw_pre : (job == 1 ? dw_post : dgate + (job - 2) * d);
  const int64_t first = job < 2 ? 0 : (job - 2) * per_group, count = job < 2 ? nseg : per_group;
  const int64_t col = (int64_t)blockIdx.x * kCols + threadIdx.x % kCols;
  const int slice = threadIdx.x / kCols;
  const int64_t each = (count + kSlices - 1) / kSlices;
  const int64_t s0 = slice * each, s1 = s0 + each < count ? s0 + each : count;
  float sum = 0.f;
  if (col < d) {
    const float* q = p + (first + s0) * d + col;
#pragma unroll 8
    for (int64_t s = s0; s < s1; ++s, q += d) sum += *q;
  }
  lds[slice][threadIdx.x % kCols] = sum;
  __syncthreads();
  if (slice == 0 && col < d) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kSlices; ++i) t += lds[i][threadIdx.x];
    out[col] = bf16_of(t);
  }
}

template <class S, bool ONE, bool SHORT>
hipError_t fwd_as(const NormFwd& p, hipStream_t st) {
  // as many workgroups as the 32 wavefronts of each of the 256 compute units hold at once
  const unsigned threads = norm_threads(p.d);
  const int64_t slots = 256 * (32 / (threads / 64));
  const unsigned grid = (unsigned)(p.M < slots ? p.M : slots);
  const FwdArgs<S> a{static_cast<const S*>(p.x),
                     p.y ? p.y : static_cast<const uint16_t*>(p.x),
                     p.w_post,
                     p.gate,
                     p.w_pre,
                     static_cast<S*>(p.x_out),
                     p.h,
                     p.M,
                     p.d,
                     p.gate && p.gate_rows < p.M ? p.gate_rows : p.M,
                     p.y ? 0xFFFFFFFFu : 0u,
                     p.scale,
                     p.eps,
                     (float)(1.0 / (double)p.d),
                     p.post};
  const bool both = a.x_out && a.h;
  const auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads), 0, st, a); };
  if (a.gate && a.gate_rows < a.M) {
    if (both) launch(k_norm_fwd<S, ONE, SHORT, kGateRows, kBoth>);
    else launch(k_norm_fwd<S, ONE, SHORT, kGateRows, kAny>);
  } else {
    if (both) launch(k_norm_fwd<S, ONE, SHORT, kGateRuns, kBoth>);
    else launch(k_norm_fwd<S, ONE, SHORT, kGateRuns, kAny>);
  }
  return hipGetLastError();
}

template <class S, bool ONE, bool SHORT>
hipError_t bwd_rows(const BwdArgs<S>& a, GateKind kind, hipStream_t st) {
  // Operands that the 256 MB cache could hold may be there already.  Reading past it, with 4096
  // columns: 1024 rows (48 MB) 22.4 us for 19.8, 2048 (96 MB) 34 for 31, 4096 (192 MB) 48 for
  // 50, 8192 82 for 89, 16384 158 for 171.
  const bool large = a.M * a.d * (int64_t)(3 * sizeof(S) + 6) > (int64_t)160 << 20;
  const Outputs out = !a.dx || !a.dy ? kAny : (large ? kBothStream : kBoth);
  const dim3 grid((unsigned)a.seg.count), block(norm_threads(a.d));
  const auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, st, a); };
  if (kind == kGateRows) {
    if (out == kAny) launch(k_norm_bwd<S, ONE, SHORT, kGateRows, kAny>);
    else if (out == kBoth) launch(k_norm_bwd<S, ONE, SHORT, kGateRows, kBoth>);
    else launch(k_norm_bwd<S, ONE, SHORT, kGateRows, kBothStream>);
  } else {
    if (out == kAny) launch(k_norm_bwd<S, ONE, SHORT, kGateRuns, kAny>);
    else if (out == kBoth) launch(k_norm_bwd<S, ONE, SHORT, kGateRuns, kBoth>);
    else launch(k_norm_bwd<S, ONE, SHORT, kGateRuns, kBothStream>);
  }
  return hipGetLastError();
}

template <class S, bool ONE, bool SHORT>
hipError_t bwd_as(const NormBwd& p, hipStream_t st) {
  const NormSegments seg = norm_segments(p.M, p.d, p.gate ? p.gate_rows : 0);
  const int64_t per = seg.count * p.d;
  float* part = p.part;
  const S *x = static_cast<const S*>(p.x), *o = static_cast<const S*>(p.dx_out);
  // any tensor of the call with as many elements of the type or wider
  const S* any = x && p.dh ? x : o;
  const uint16_t* any16 = p.dh ? p.dh : reinterpret_cast<const uint16_t*>(any);
  BwdArgs<S> a{};
  a.x = p.dh ? x : any, a.dh = p.dh ? p.dh : any16, a.dx_out = o ? o : any, a.y = p.y ? p.y : any16;
  a.h_bits = p.dh ? ~0u : 0u, a.o_bits = o ? ~0u : 0u, a.y_bits = p.y ? ~0u : 0u;
  a.w_post = p.w_post, a.gate = p.gate, a.w_pre = p.w_pre;
  a.dx = static_cast<S*>(p.dx), a.dy = p.dy;
  if (!seg.per_group) a.dgate = p.dgate;
  a.M = p.M, a.d = p.d, a.gate_rows = p.gate ? p.gate_rows : p.M, a.seg = seg;
  a.scale = p.scale, a.eps = p.eps, a.inv_d = (float)(1.0 / (double)p.d), a.post = p.post;
  if (p.dw_pre) a.p_pre = part, part += per;
  if (p.dw_post) a.p_post = part, part += per;
  if (p.dgate && seg.per_group) a.p_gate = part;
  const bool partials = a.p_pre || a.p_post || a.p_gate;
  if (partials && seg.count <= kFewSegments && 3 * sizeof(float) * (size_t)per <= kFewBytes) {
    a.counter = p.counter;
    a.sum_pre = p.dw_pre, a.sum_post = p.dw_post, a.sum_gate = p.dgate;
  }
  const hipError_t e = bwd_rows<S, ONE, SHORT>(a, p.gate && p.gate_rows == 1 ? kGateRows : kGateRuns, st);
  if (e != hipSuccess || !partials || a.counter) return e;
  const int64_t groups = a.p_gate ? (p.M + p.gate_rows - 1) / p.gate_rows : 0;
  const int64_t job0 = a.p_pre ? 0 : (a.p_post ? 1 : 2), jobs = (groups ? 2 + groups : (a.p_post ? 2 : 1)) - job0;
  hipLaunchKernelGGL(k_norm_cols, dim3((unsigned)((p.d + kCols - 1) / kCols), (unsigned)jobs), dim3(kColThreads), 0,
                     st, a.p_pre, a.p_post, a.p_gate, p.dw_pre, p.dw_post, p.dgate, p.d, seg.count, seg.per_group,
                     job0);
  return hipGetLastError();
}

template <class S>
hipError_t fwd(const NormFwd& p, hipStream_t st) {
  if (p.d < 8) return fwd_as<S, true, true>(p, st);
  return norm_threads(p.d) == 64 ? fwd_as<S, true, false>(p, st) : fwd_as<S, false, false>(p, st);
}
template <class S>
hipError_t bwd(const NormBwd& p, hipStream_t st) {
  if (p.d < 8) return bwd_as<S, true, true>(p, st);
  return norm_threads(p.d) == 64 ? bwd_as<S, true, false>(p, st) : bwd_as<S, false, false>(p, st);
}

}  // namespace

hipError_t launch_norm_fwd(const NormFwd& p, hipStream_t st) { return p.f32 ? fwd<float>(p, st) : fwd<uint16_t>(p, st); }
hipError_t launch_norm_bwd(const NormBwd& p, hipStream_t st) { return p.f32 ? bwd<float>(p, st) : bwd<uint16_t>(p, st); }

}  // namespace qlora
