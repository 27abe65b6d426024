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
#include "qlora_train_host.h"
#include "train_device.h"

namespace qlora {
namespace {

template <class S>
struct FwdArgs {
  const S* x;
  const uint16_t *y, *w_post, *gate, *w_pre;
  S* x_out;
  uint16_t* h;
  int64_t d, gate_rows;
  float scale, eps, inv_d;
  int post;
};

// One workgroup of T threads per row, eight columns to a thread: every operand is read once and
// kept in registers.
template <class S, int T, bool SHORT>
__global__ __launch_bounds__(T) void k_norm_fwd(FwdArgs<S> a) {
  __shared__ float lds[2][T / 64];
  const int64_t row = blockIdx.x, d = a.d;
  const Columns<SHORT> col((int)d, 8 * threadIdx.x);
  Raw8<S> x;
  Raw8<uint16_t> y, w;
  col.load(x, a.x + row * d);
  col.drop(x);
  if (a.y) {
    col.load(y, a.y + row * d);
    col.drop(y);
  }
  float r_y = 1.f;
  if (a.post) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] = fmaf(y.get(i), y.get(i), s[0]);
    block_sum<T>(s, lds[0]);
    r_y = 1.f / sqrtf(s[0] * a.inv_d + a.eps);
  }
  float xo[8], s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < 8; ++i) xo[i] = a.scale * x.get(i);
  if (a.y) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = y.get(i) * r_y;
    if (a.w_post) {
      col.load(w, a.w_post);
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] *= w.get(i);
    }
    if (a.gate) {
      col.load(w, a.gate + row / a.gate_rows * d);
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] *= w.get(i);
    }
    // (a column that is not the lane's own gives 0 times a weight: an infinite one would reach
    // the sum)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= 8 - col.n || SHORT) xo[i] += q[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) s[0] = fmaf(xo[i], xo[i], s[0]);
  if (a.x_out) col.store(a.x_out + row * d, xo);
  if (!a.h) return;
  block_sum<T>(s, lds[1]);
  const float r_x = 1.f / sqrtf(s[0] * a.inv_d + a.eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) xo[i] *= r_x;
  if (a.w_pre) {
    col.load(w, a.w_pre);
#pragma unroll
    for (int i = 0; i < 8; ++i) xo[i] *= w.get(i);
  }
  col.store(a.h + row * d, xo);
}

template <class S>
struct BwdArgs {
  const S* x;  // x', as the forward stored it
  const uint16_t *y, *dh;
  const S* dx_out;
  const uint16_t *w_post, *gate, *w_pre;
  S* dx;
  uint16_t* dy;
  uint16_t* dgate;                 // for gate rows whole in a segment, else null
  float *p_pre, *p_post, *p_gate;  // [segment][d] FP32 partials, null where not wanted
  int64_t M, d, gate_rows;
  NormSegments seg;
  float scale, eps, inv_d;
  int post;
};

// What one row gives a lane's columns.  An operand that is not given is zeros, a weight or gate
// that is not given is ones, so the arithmetic has no cases.
template <class S, bool SHORT>
struct RowVec {
  Raw8<S> x, dxo;
  Raw8<uint16_t> y, dh;
  __device__ __forceinline__ void load(const BwdArgs<S>& a, const Columns<SHORT>& col, int64_t at) {
    if (a.dh) {
      col.load(x, a.x + at);
      col.load(dh, a.dh + at);
    } else {
      zero8(x), zero8(dh);
    }
    if (a.dx_out) col.load(dxo, a.dx_out + at);
    else zero8(dxo);
    if (a.y) col.load(y, a.y + at);
    else zero8(y);
  }
  __device__ __forceinline__ void pack() { opaque(x), opaque(dxo), opaque(y), opaque(dh); }
};

// One workgroup per segment of consecutive rows.  Its threads own columns, so the column sums
// (weights, gate) stay in registers over the segment; the sums over a row are one exchange:
// with q = g w_post y,  sum(b y) = sum(dx' q) + r_x sum(a q) - k sum(x' q),  k = r_x^3 mean(a x').
template <class S, int T, bool SHORT>
__global__ __launch_bounds__(T, SHORT ? 1 : 4) void k_norm_bwd(BwdArgs<S> a) {
  __shared__ float lds[2][6 * (T / 64)];
  const int64_t d = a.d, seg = blockIdx.x;
  // segments inside a gate row's rows (per_group of them), or of whole gate rows
  int64_t r0 = seg * a.seg.rows, end = a.M, group;
  if (a.seg.per_group) {
    group = seg / a.seg.per_group;
    r0 = group * a.gate_rows + (seg - group * a.seg.per_group) * a.seg.rows;
    end = (group + 1) * a.gate_rows < a.M ? (group + 1) * a.gate_rows : a.M;
  } else {
    group = r0 / a.gate_rows;
  }
  const int64_t r1 = r0 + a.seg.rows < end ? r0 + a.seg.rows : end;
  int64_t group_end = (group + 1) * a.gate_rows < a.M ? (group + 1) * a.gate_rows : a.M;
  const Columns<SHORT> col((int)d, 8 * threadIdx.x);
  Raw8<uint16_t> w_pre, w_post, g;
  if (a.w_pre) col.load(w_pre, a.w_pre);
  else ones8(w_pre);
  if (a.w_post) col.load(w_post, a.w_post);
  else ones8(w_post);
  const auto load_gate = [&] {
    if (a.gate) col.load(g, a.gate + group * d);
    else ones8(g);
  };
  // s_tu: sum of t u over the rows of one gate row; times the gate it goes into dw_post, times
  // w_post it is the gate's gradient
  float s_pre[8], s_post[8], s_tu[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s_pre[i] = s_post[i] = s_tu[i] = 0.f;
  const bool post = a.post != 0;
  const uint32_t post_bits = post ? 0xFFFFFFFFu : 0u;
  // sixteen wavefronts to a compute unit have 128 registers each: with an FP32 stream the next
  // row does not fit
  constexpr bool kAhead = sizeof(S) == 2 && !SHORT;
  RowVec<S, SHORT> r, next;
  if (r0 < r1) r.load(a, col, r0 * d), load_gate();
  else if (a.p_gate) col.store(a.p_gate + seg * d, s_tu);
  for (int64_t row = r0; row < r1; ++row) {
    const int64_t at = row * d;
    // the next row's loads run under this row's exchange
    if (kAhead && row + 1 < r1) next.load(a, col, at + d);
    // what is held across the exchange stays packed (unpacked once for both uses it would take
    // 56 registers more)
    opaque(w_pre), opaque(w_post), opaque(g), r.pack();
    col.drop(r.x), col.drop(r.y);
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float xi = r.x.get(i), yi = r.y.get(i), ai = r.dh.get(i) * w_pre.get(i);
      const float q = yi * w_post.get(i) * g.get(i);
      s[0] = fmaf(xi, xi, s[0]);
      s[1] = fmaf(ai, xi, s[1]);
      s[2] = fmaf(yi, yi, s[2]);
      s[3] = fmaf(r.dxo.get(i), q, s[3]);
      s[4] = fmaf(ai, q, s[4]);
      s[5] = fmaf(xi, q, s[5]);
    }
    block_sum<T>(s, lds[(row - r0) & 1]);
    opaque(w_pre), opaque(w_post), opaque(g), r.pack();
    const float r_x = a.dh ? 1.f / sqrtf(s[0] * a.inv_d + a.eps) : 0.f;
    const float k = a.dh ? r_x * r_x * r_x * (s[1] * a.inv_d) : 0.f;
    const float r_y = post ? 1.f / sqrtf(s[2] * a.inv_d + a.eps) : 1.f;
    const float c = post ? r_y * r_y * r_y * ((s[3] + r_x * s[4] - k * s[5]) * a.inv_d) : 0.f;
    float t[8], o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float xi = r.x.get(i), dhi = r.dh.get(i);
      t[i] = r.dxo.get(i) + (r_x * (dhi * w_pre.get(i)) - xi * k);
      s_pre[i] = fmaf(dhi, xi * r_x, s_pre[i]);
      o[i] = a.scale * t[i];
    }
    if (a.dx) col.store(a.dx + at, o);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float yi = r.y.get(i);
      s_tu[i] = fmaf(t[i], yi * r_y, s_tu[i]);
      o[i] = r_y * (t[i] * g.get(i) * w_post.get(i)) - __uint_as_float(__float_as_uint(yi) & post_bits) * c;
    }
    if (a.dy) col.store(a.dy + at, o);
    if (row + 1 == group_end || row + 1 == r1) {
      float dg[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s_post[i] = fmaf(s_tu[i], g.get(i), s_post[i]);
        dg[i] = s_tu[i] * w_post.get(i);
        s_tu[i] = 0.f;
      }
      if (a.dgate) col.store(a.dgate + group * d, dg);
      if (a.p_gate) col.store(a.p_gate + seg * d, dg);
      if (row + 1 < r1) {
        ++group;
        group_end = group_end + a.gate_rows < a.M ? group_end + a.gate_rows : a.M;
        load_gate();
      }
    }
    if (kAhead) r = next;
    else if (row + 1 < r1) r.load(a, col, at + d);
  }
  if (a.p_pre) col.store(a.p_pre + seg * d, s_pre);
  if (a.p_post) col.store(a.p_post + seg * d, s_post);
}

// Column sums of the segments' partials, in the segments' order within each of the 16 slices
// and the slices in order: job 0 dw_pre, job 1 dw_post over all segments, job 2 + g the gate's
// row g over its segments.
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

template <class S, int T, bool SHORT = false>
hipError_t fwd_as(const NormFwd& p, hipStream_t st) {
  FwdArgs<S> a{static_cast<const S*>(p.x), p.y, p.w_post, p.gate, p.w_pre, static_cast<S*>(p.x_out), p.h, p.d,
               p.gate_rows, p.scale, p.eps, (float)(1.0 / (double)p.d), p.post};
  hipLaunchKernelGGL((k_norm_fwd<S, T, SHORT>), dim3((unsigned)p.M), dim3(T), 0, st, a);
  return hipGetLastError();
}

template <class S>
hipError_t fwd(const NormFwd& p, hipStream_t st) {
  const int64_t n8 = (p.d + 7) / 8;
  if (p.d < 8) return fwd_as<S, 64, true>(p, st);
  if (n8 <= 64) return fwd_as<S, 64>(p, st);
  if (n8 <= 128) return fwd_as<S, 128>(p, st);
  if (n8 <= 256) return fwd_as<S, 256>(p, st);
  if (n8 <= 512) return fwd_as<S, 512>(p, st);
  return fwd_as<S, 1024>(p, st);
}

template <class S, int T, bool SHORT = false>
hipError_t bwd_as(const NormBwd& p, hipStream_t st) {
  const NormSegments seg = norm_segments(p.M, p.d, p.gate ? p.gate_rows : 0);
  const int64_t per = seg.count * p.d;
  float* part = p.part;
  BwdArgs<S> a{};
  a.x = static_cast<const S*>(p.x), a.y = p.y, a.dh = p.dh, a.dx_out = static_cast<const S*>(p.dx_out);
  a.w_post = p.w_post, a.gate = p.gate, a.w_pre = p.w_pre;
  a.dx = static_cast<S*>(p.dx), a.dy = p.dy;
  a.M = p.M, a.d = p.d, a.gate_rows = p.gate ? p.gate_rows : p.M, a.seg = seg;
  a.scale = p.scale, a.eps = p.eps, a.inv_d = (float)(1.0 / (double)p.d), a.post = p.post;
  if (!seg.per_group) a.dgate = p.dgate;
  if (p.dw_pre) a.p_pre = part, part += per;
  if (p.dw_post) a.p_post = part, part += per;
  if (p.dgate && seg.per_group) a.p_gate = part;
  hipLaunchKernelGGL((k_norm_bwd<S, T, SHORT>), dim3((unsigned)seg.count), dim3(T), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t groups = a.p_gate ? (p.M + p.gate_rows - 1) / p.gate_rows : 0;
  const int64_t job0 = a.p_pre ? 0 : (a.p_post ? 1 : 2), jobs = (groups ? 2 + groups : (a.p_post ? 2 : 1)) - job0;
  if (!a.p_pre && !a.p_post && !groups) return hipSuccess;
  hipLaunchKernelGGL(k_norm_cols, dim3((unsigned)((p.d + kCols - 1) / kCols), (unsigned)jobs), dim3(kColThreads), 0,
                     st, a.p_pre, a.p_post, a.p_gate, p.dw_pre, p.dw_post, p.dgate, p.d, seg.count, seg.per_group,
                     job0);
  return hipGetLastError();
}

template <class S>
hipError_t bwd(const NormBwd& p, hipStream_t st) {
  const int64_t n8 = (p.d + 7) / 8;
  if (p.d < 8) return bwd_as<S, 64, true>(p, st);
  if (n8 <= 64) return bwd_as<S, 64>(p, st);
  if (n8 <= 128) return bwd_as<S, 128>(p, st);
  if (n8 <= 256) return bwd_as<S, 256>(p, st);
  if (n8 <= 512) return bwd_as<S, 512>(p, st);
  return bwd_as<S, 1024>(p, st);
}

}  // namespace

hipError_t launch_norm_fwd(const NormFwd& p, hipStream_t st) { return p.f32 ? fwd<float>(p, st) : fwd<uint16_t>(p, st); }
hipError_t launch_norm_bwd(const NormBwd& p, hipStream_t st) { return p.f32 ? bwd<float>(p, st) : bwd<uint16_t>(p, st); }

}  // namespace qlora
