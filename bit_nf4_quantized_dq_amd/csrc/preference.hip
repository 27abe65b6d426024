// Token log-probabilities over a vocabulary, and the preference loss of answer pairs.
//
//   logp_t = x_t[label_t] - log sum_v exp(x_t[v])          (0 for a token that is not counted)
//   D_i = sum_t (logp_t - ref_t) over sequence i,   z_p = beta (D_chosen(p) - D_rejected(p))
//   loss = mean_p ((1 - e) softplus(-z_p) + e softplus(z_p))
//   dloss/dx_t[v] = c_i ([v = label_t] - exp(x_t[v] - lse_t)),
//   c_chosen = -c_rejected = grad_scale (beta / P) (sigmoid(z_p) + e - 1)
//
// Two passes over the logits: a row's maximum and sum, then its gradient, since a row's c needs
// every row of its pair.  HBM bounds both (a copy reaches 6.3 TB/s here, a plain read 7.0), and
// rows that are not counted are never read.  The first pass leaves the end of what it read in
// the 256 MB cache: the second goes from the last row to the first (4 x 1024 rows of 131072:
// 417 us in the first pass's order, 397 in reverse) and writes past the cache (446 us without
// that; 4096 rows of 32768 122 us, 96 with it; both also with a product that reads the gradient
// next).  Measured (MI355X, BF16, about 60% of the tokens counted): log-probabilities of 4096 x
// 32768 33 us (4.9 TB/s), of 4096 x 131072 112 us (5.8 TB/s); loss and gradient 98 us and 395 us
// (the gradient pass alone 66 us, 6.4 TB/s, and 288 us, 6.0 TB/s); 66 rows of 1003 in FP32 4.4 +
// 5.2 us on the device.
//
// Precision: a row's exponentials are summed in FP32, a thread at a time and then by wavefronts;
// the logarithm, a token's log ratio and a pair's sums are FP64, because hundreds of tokens
// cancel in z; probabilities and gradients are FP32, rounded once.
#include <type_traits>

#include "qlora_train_host.h"
#include "train_device.h"

namespace qlora {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kRowThreads = 256, kUnroll = 4;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Running maximum m and sum s of exp(x - m).  An empty or all -inf set is (-inf, 0); a maximum
// of -inf is never subtracted from itself.
__device__ __forceinline__ void merge(float& m, float& s, float m2, float s2) {
  const float t = fmaxf(m, m2);
  const float ref = t == -INFINITY ? 0.f : t;
  s = s * exp2_hw((m - ref) * kLog2e) + s2 * exp2_hw((m2 - ref) * kLog2e);
  m = t;
}

// What one pass over a row gives, rounded to FP32 only at the end: the label's log-probability
// from the exact difference to the maximum and an FP64 logarithm.
__device__ __forceinline__ double label_logp(float xl, float m, float s) {
  return (double)xl - (double)m - log((double)s);
}

// A row or part of `count` elements in whole vectors from its first 16-byte boundary on (`at`
// decides), and what is left over before them and after.  (Rows of an odd width otherwise have
// every vector across a boundary: log-probabilities of 4096 rows of 50257 58 us, so 48.)
struct Span {
  int head, tail;
  int32_t full;
  bool wide;
  template <class E>
  __device__ __forceinline__ Span(const E* at, int64_t count) {
    const int to = (int)((16 - (reinterpret_cast<uintptr_t>(at) & 15)) & 15) / (int)sizeof(E);
    head = to < count ? to : (int)count;
    full = (int32_t)((count - head) >> 3);
    tail = (int)((count - head) & 7);
    wide = count >= 8;
  }
  // the first `head` elements (the rest of the vector is to be dropped)
  template <class E>
  __device__ __forceinline__ void load_head(Raw8<E>& r, const E* x) const {
    if (wide) load_all8(r, x);
    else load8(r, x, head, false);
  }
  template <class E>
  __device__ __forceinline__ void load_tail(Raw8<E>& r, const E* x) const {
    load8(r, x + head + 8 * full, tail, wide);
  }
};

// One workgroup per row and part: one pass with the running maximum and sum of each thread.  A
// whole row (parts == 1) is finished here, a split one by its readers.
template <class E, int T>
__global__ __launch_bounds__(T) void k_row_stats(const E* __restrict__ logits,
                                                           const int64_t* __restrict__ labels,
                                                           const float* __restrict__ ref, int64_t V, int64_t parts,
                                                           int64_t len, RowStats ws, float* __restrict__ logps) {
  __shared__ float lm[T / 64], ls[T / 64];
  const int64_t row = blockIdx.x / parts, p = blockIdx.x - row * parts;
  const int64_t label = labels[row];
  if (label < 0 || label >= V) {
    if (parts == 1 && threadIdx.x == 0) {
      logps[row] = 0.f;
      if (ws.ratio) ws.ratio[row] = 0.0;
    }
    return;
  }
  const E* x = logits + row * V;
  const int64_t v0 = p * len, v1 = v0 + len < V ? v0 + len : V;
  float xl = 0.f;
  if (threadIdx.x == 0) xl = to_f32(x[label]);
  float m = -INFINITY, s = 0.f;
  const auto take = [&](const Raw8<E>& r, int n) {
    float f[8], t = m;
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j < n ? r.get(j) : -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j) t = fmaxf(t, f[j]);
    const float base = t == -INFINITY ? 0.f : t;
    s *= exp2_hw((m - base) * kLog2e);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += exp2_hw((f[j] - base) * kLog2e);
    m = t;
  };
  const Span span(x + v0, v1 - v0);
  const int32_t full = span.full, batches = full / (kUnroll * T);
  const E* xp = x + v0 + span.head;
  // Batches of 32 elements a thread.  The exponentials are 2^(x log2 e - n) with a whole number n:
  // the product is not rounded before n leaves it, so this is one operation for the difference
  // and the factor, and changes of n scale exactly.  n is taken from the rounded product of the
  // maximum, which below 2^23 is off by at most 1/4: n is the maximum's x log2 e or just above
  // it.  (From 2^32 on the rounding passes the range of exp2.)  n stays above kLow: elements below
  // it (masked by a large negative number, -inf or the type's lowest value) add zero.
  constexpr float kLow = -8388608.f;
  float n = kLow;
  for (int32_t i = 0; i < batches; ++i) {
    Raw8<E> r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) load_all8(r[u], xp + 8 * ((i * kUnroll + u) * T + (int)threadIdx.x));
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, r[u].get(j));
    const float to = ceilf(fmaxf(m * kLog2e, kLow));
    s *= exp2_hw(n - to);
    n = to;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += exp2_hw(fmaf(r[u].get(j), kLog2e, -n));
  }
  // From n to the maximum itself.  A thread whose maximum is not within kHuge (times log2 e that
  // stays below 2^23) keeps only a NaN: beside a row's maximum above -kHuge / 2 it adds zero.
  constexpr float kHuge = 4194304.f;
  if (batches) s = fabsf(m) < kHuge ? s * exp2_hw(fmaf(-m, kLog2e, n)) : (s != s ? s : 0.f);
  // Any other maximum (large, infinite, or of a row that is masked throughout): the batches once
  // more, each difference before its factor.
  if (__syncthreads_or(batches && !(fabsf(m) < kHuge))) {
    float top = m;
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1) top = fmaxf(top, __shfl_xor(top, k, 64));
    if ((threadIdx.x & 63) == 0) lm[threadIdx.x >> 6] = top;
    __syncthreads();
    for (int w = 0; w < T / 64; ++w) top = fmaxf(top, lm[w]);
    __syncthreads();
    if (!(top > -0.5f * kHuge && top < kHuge)) {
      m = -INFINITY, s = 0.f;
      for (int32_t i = threadIdx.x; i < batches * kUnroll * T; i += T) {
        Raw8<E> r;
        load_all8(r, xp + 8 * i);
        take(r, 8);
      }
    }
  }
  for (int32_t i = batches * kUnroll * T + (int)threadIdx.x; i < full; i += T) {
    Raw8<E> r;
    load_all8(r, xp + 8 * i);
    take(r, 8);
  }
  if (threadIdx.x == 0 && span.head) {
    Raw8<E> r;
    span.load_head(r, x + v0);
    take(r, span.head);
  }
  if (threadIdx.x == T - 1 && span.tail) {
    Raw8<E> r;
    span.load_tail(r, x + v0);
    take(r, span.tail);
  }
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) merge(m, s, __shfl_xor(m, k, 64), __shfl_xor(s, k, 64));
  if ((threadIdx.x & 63) == 0) lm[threadIdx.x >> 6] = m, ls[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    m = lm[0], s = ls[0];
    for (int w = 1; w < T / 64; ++w) merge(m, s, lm[w], ls[w]);
    ws.part[row * parts + p] = MaxSum{m, s};
    if (parts == 1) {
      const double lp = label_logp(xl, m, s);
      logps[row] = (float)lp;
      if (ws.ratio) ws.ratio[row] = lp - (ref ? (double)ref[row] : 0.0);
    } else if (p == 0) {
      ws.label_logit[row] = xl;
    }
  }
}

// The parts of one row, joined in their order.
__device__ __forceinline__ MaxSum join_row(const MaxSum* part, int64_t parts) {
  MaxSum r = part[0];
  for (int64_t p = 1; p < parts; ++p) merge(r.m, r.s, part[p].m, part[p].s);
  return r;
}

__global__ __launch_bounds__(kRowThreads) void k_row_join(const int64_t* __restrict__ labels, int64_t V, int64_t rows,
                                                          int64_t parts, RowStats ws, float* __restrict__ logps) {
  const int64_t row = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  if (row >= rows) return;
  float lp = 0.f;
  if (labels[row] >= 0 && labels[row] < V) {
    const MaxSum r = join_row(ws.part + row * parts, parts);
    lp = (float)label_logp(ws.label_logit[row], r.m, r.s);
  }
  logps[row] = lp;
}

struct PairArgs {
  const int64_t* labels;
  const float* ref;
  int64_t pairs, S, V, parts;
  float beta, smoothing, grad_scale;
  RowStats ws;
  float *logps, *log_ratios, *loss;
};
struct PairLds {
  double sum[2][16];  // one for each wavefront of a workgroup
  double mean[16];
  bool last;
};

// The pair's log ratios, summed in FP64 in one order by whichever workgroup asks: for whole rows
// two short sums of what the first pass left, for split rows after joining their parts.
template <int T>
__device__ __forceinline__ void pair_sums(const PairArgs& a, int64_t pair, bool write, PairLds& lds, double out[2]) {
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int64_t r0 = (pair + side * a.pairs) * a.S;
    double sum = 0.0;
    if (a.parts == 1) {
#pragma unroll 4
      for (int64_t t = threadIdx.x; t < a.S; t += T) sum += a.ws.ratio[r0 + t];
    } else {
      for (int64_t t = threadIdx.x; t < a.S; t += T) {
        const int64_t row = r0 + t, label = a.labels[row];
        double lp = 0.0;
        if (label >= 0 && label < a.V) {
          const MaxSum r = join_row(a.ws.part + row * a.parts, a.parts);
          lp = label_logp(a.ws.label_logit[row], r.m, r.s);
          sum += lp - (a.ref ? (double)a.ref[row] : 0.0);
        }
        if (write) a.logps[row] = (float)lp;
      }
    }
    out[side] = block_sum_f64<T>(sum, lds.sum[side]);
  }
}

// d loss / d (chosen log ratio) of a pair, times grad_scale.
__device__ __forceinline__ float pair_slope(const PairArgs& a, const double d[2]) {
  const double z = (double)a.beta * (d[0] - d[1]);
  const double t = exp(-fabs(z)), sig = (z >= 0.0 ? 1.0 : t) / (1.0 + t);
  return (float)((double)a.grad_scale * ((double)a.beta / (double)a.pairs) * (sig + (double)a.smoothing - 1.0));
}

// One workgroup of each pair writes its log ratios and its loss; the last of them to arrive adds
// the losses in the pairs' order.  The losses travel by system-scope (cache-bypassing) stores
// and loads, and a store has completed before its workgroup is counted: the wait between them
// is what orders the two on this chip.  (No rule of the language does; a release would write
// back the L2 too, which took 65 ns a workgroup in the norm backward.)
template <int T>
__device__ void finish_pair(const PairArgs& a, int64_t pair, const double d[2], PairLds& lds) {
  if (threadIdx.x == 0) {
    a.log_ratios[pair] = (float)d[0];
    a.log_ratios[pair + a.pairs] = (float)d[1];
    const double z = (double)a.beta * (d[0] - d[1]), e = a.smoothing;
    const double tail = log1p(exp(-fabs(z)));
    double loss = z;  // NaN stays NaN
    if (z == z) {
      // a factor of exactly 0 leaves an infinite term out
      loss = (e == 1.0 ? 0.0 : (1.0 - e) * (tail + fmax(-z, 0.0))) + (e == 0.0 ? 0.0 : e * (tail + fmax(z, 0.0)));
    }
    __hip_atomic_store(a.ws.pair_loss + pair, loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
    __builtin_amdgcn_s_waitcnt(0);
    const unsigned int old =
        __hip_atomic_fetch_add(a.ws.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    lds.last = old + 1u == (unsigned int)a.pairs;
    if (lds.last) __hip_atomic_store(a.ws.counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!lds.last) return;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < a.pairs; i += T)
    s += __hip_atomic_load(a.ws.pair_loss + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
  s = block_sum_f64<T>(s, lds.mean);
  if (threadIdx.x == 0) *a.loss = (float)(s / (double)a.pairs);
}

// The loss alone: one workgroup per pair.
__global__ __launch_bounds__(kRowThreads) void k_pref_loss(PairArgs a) {
  __shared__ PairLds lds;
  double d[2];
  pair_sums<kRowThreads>(a, blockIdx.x, true, lds, d);
  finish_pair<kRowThreads>(a, blockIdx.x, d, lds);
}

// The gradient: one workgroup per row and part, each element read and written once.  Each takes
// its pair's slope from the pair's sums itself, so nothing runs between the two passes.  That is
// 16 S bytes of FP64 ratios a counted row, mostly from L2, before the row's first load: little
// beside a wide row (V = 32768, all tokens counted: the gradient adds 80 us to the loss of 4096
// rows at S = 512, 171 to 8192 at S = 4096, 410 to 16384 at S = 8192), most of the time of a
// narrow one (V = 1000: 114 us for 16384 rows at S = 8192, whose bytes take about 10).  Rows go
// from the last to the first: the end of what the first pass read is still in the cache.
template <class E, int T>
__global__ __launch_bounds__(T) void k_pref_grad(const E* logits, E* dlogits, PairArgs a, int64_t len) {
  __shared__ PairLds lds;
  const int64_t block = (int64_t)gridDim.x - 1 - blockIdx.x;
  const int64_t row = block / a.parts, p = block - row * a.parts;
  const int64_t seq = row / a.S, pair = seq < a.pairs ? seq : seq - a.pairs;
  const int64_t label = a.labels[row], V = a.V;
  const bool counted = label >= 0 && label < V;
  // the workgroup that writes the pair's results: among the first to run
  const bool lead = p == 0 && seq >= a.pairs && row == (seq + 1) * a.S - 1;
  double d[2];
  if (counted || lead) pair_sums<T>(a, pair, lead, lds, d);
  if (lead) finish_pair<T>(a, pair, d, lds);
  float c = 0.f, scale = 0.f, m = 0.f;
  if (counted) {
    c = pair_slope(a, d);
    if (seq >= a.pairs) c = -c;
    const MaxSum r = join_row(a.ws.part + row * a.parts, a.parts);
    m = r.m;
    scale = -c / r.s;
  }
  const int64_t v0 = p * len, v1 = v0 + len < V ? v0 + len : V;
  const E* x = logits + row * V + v0;
  E* out = dlogits + row * V + v0;
  const auto give = [&](const Raw8<E>& r, int64_t at, int n) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = scale * exp2_hw((r.get(j) - m) * kLog2e);
    const int64_t j0 = label - v0 - at;
    if (j0 >= 0 && j0 < 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j == j0) f[j] += c;
    }
    if (n == 8) stream8(out + at, f);
    else store8(out + at, f, n);
  };
  const Span span(out, v1 - v0);
  const int32_t full = span.full;
  if (!counted) {
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int32_t i = threadIdx.x; i < full; i += T) stream8(out + span.head + 8 * i, zero);
    if (threadIdx.x == 0) store8(out, zero, span.head);
    if (threadIdx.x == T - 1) store8(out + span.head + 8 * full, zero, span.tail);
    return;
  }
  for (int32_t i = threadIdx.x; i < full; i += kUnroll * T) {
    Raw8<E> r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i + u * T < full) load_all8(r[u], x + span.head + 8 * (i + u * T));
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i + u * T < full) give(r[u], span.head + 8 * (i + u * T), 8);
  }
  // (in place, a neighbour may have replaced the elements that these two drop)
  if (threadIdx.x == 0 && span.head) {
    Raw8<E> r;
    span.load_head(r, x);
    give(r, 0, span.head);
  }
  if (threadIdx.x == T - 1 && span.tail) {
    Raw8<E> r;
    span.load_tail(r, x);
    give(r, span.head + 8 * full, span.tail);
  }
}

// The threads of each of `blocks` rows or parts of `len` elements (a launch has fewer than 2^32
// threads in all).  Short rows take few, so that many rows are under way; 8192 rows of 1000: 10.5 us
// by 64 threads, 20 by 256; 16384 of 8192: 33 by 128, 37 by 256; 4096 of 32768: 33 by 256, 38 by
// 128 or 1024; 4096 of 131072: 112 by 1024, 121 by 256 (all of these the statistics).  The gradient
// (`writes`), which keeps loads and stores in flight, has 256 from 2048 elements on (1600 rows of
// 16384: 28 us, 29.6 by 128); from 48 K on it follows the statistics, which is not measured for it
// by itself (by 1024 threads its 88 registers leave one workgroup to a compute unit).
template <bool writes, class F>
void by_threads(int64_t blocks, int64_t len, F launch) {
  if (len >= 128 * 1024 && blocks < int64_t(1) << 22) launch(std::integral_constant<int, 1024>());
  else if (len >= 48 * 1024 && blocks < int64_t(1) << 23) launch(std::integral_constant<int, 512>());
  else if (len >= (writes ? 2 * 1024 : 24 * 1024)) launch(std::integral_constant<int, 256>());
  else if constexpr (writes) launch(std::integral_constant<int, 64>());
  else if (len >= 4 * 1024) launch(std::integral_constant<int, 128>());
  else launch(std::integral_constant<int, 64>());
}

template <class E>
hipError_t stats(const E* logits, const int64_t* labels, const float* ref, int64_t rows, int64_t V, const RowSplit& sp,
                 float* logps, const RowStats& ws, hipStream_t st) {
  by_threads<false>(rows * sp.parts, sp.len, [&](auto t) {
    constexpr int T = decltype(t)::value;
    hipLaunchKernelGGL((k_row_stats<E, T>), dim3((unsigned)(rows * sp.parts)), dim3(T), 0, st, logits, labels, ref, V,
                       sp.parts, sp.len, ws, logps);
  });
  return hipGetLastError();
}

template <class E>
hipError_t logps_as(const E* logits, const int64_t* labels, int64_t rows, int64_t V, float* logps, const RowStats& ws,
                    hipStream_t st) {
  const RowSplit sp = row_split(rows, V);
  const hipError_t e = stats(logits, labels, nullptr, rows, V, sp, logps, ws, st);
  if (e != hipSuccess || sp.parts == 1) return e;
  hipLaunchKernelGGL(k_row_join, dim3((unsigned)((rows + kRowThreads - 1) / kRowThreads)), dim3(kRowThreads), 0, st,
                     labels, V, rows, sp.parts, ws, logps);
  return hipGetLastError();
}

template <class E>
hipError_t preference_as(const Preference& p, const RowStats& ws, hipStream_t st) {
  const int64_t rows = 2 * p.pairs * p.S;
  const RowSplit sp = row_split(rows, p.V);
  const E* logits = static_cast<const E*>(p.logits);
  const hipError_t e = stats(logits, p.labels, p.ref_logps, rows, p.V, sp, p.logps, ws, st);
  if (e != hipSuccess) return e;
  const PairArgs a{p.labels,    p.ref_logps,  p.pairs, p.S,     p.V,          sp.parts, p.beta,
                   p.smoothing, p.grad_scale, ws,      p.logps, p.log_ratios, p.loss};
  if (p.dlogits) {
    by_threads<true>(rows * sp.parts, sp.len, [&](auto t) {
      constexpr int T = decltype(t)::value;
      hipLaunchKernelGGL((k_pref_grad<E, T>), dim3((unsigned)(rows * sp.parts)), dim3(T), 0, st, logits,
                         static_cast<E*>(p.dlogits), a, sp.len);
    });
  } else {
    hipLaunchKernelGGL(k_pref_loss, dim3((unsigned)p.pairs), dim3(kRowThreads), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_token_logps(const void* logits, const int64_t* labels, int64_t rows, int64_t V, int f32,
                              float* logps, const RowStats& ws, hipStream_t st) {
  return f32 ? logps_as(static_cast<const float*>(logits), labels, rows, V, logps, ws, st)
             : logps_as(static_cast<const uint16_t*>(logits), labels, rows, V, logps, ws, st);
}
hipError_t launch_preference(const Preference& p, const RowStats& ws, hipStream_t st) {
  return p.f32 ? preference_as<float>(p, ws, st) : preference_as<uint16_t>(p, ws, st);
}

}  // namespace qlora
