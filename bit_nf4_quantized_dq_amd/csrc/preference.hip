// Token log-probabilities over a vocabulary, and the preference loss of answer pairs.
//
//   logp_t = x_t[label_t] - log sum_v exp(x_t[v])          (0 for a token that is not counted)
//   D_i = sum_t (logp_t - ref_t) over sequence i,   z_p = beta (D_chosen(p) - D_rejected(p))
//   loss = mean_p ((1 - e) softplus(-z_p) + e softplus(z_p))
//   dloss/dx_t[v] = c_i ([v = label_t] - exp(x_t[v] - lse_t)),
//   c_chosen = -c_rejected = grad_scale (beta / P) (sigmoid(z_p) + e - 1)
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

// Rows of a launch: `half` rows of chosen answers from row `first`, then as many of rejected
// ones from row first + offset (or, with offset 0, simply the rows from `first`).
struct Rows {
  int64_t first, half, offset;
  __device__ __forceinline__ int64_t at(int64_t i) const { return first + (i < half ? i : i - half + offset); }
};

// One workgroup per row and part: one pass with the running maximum and sum of each thread.
template <class E>
__global__ __launch_bounds__(kRowThreads) void k_row_stats(const E* __restrict__ logits,
                                                           const int64_t* __restrict__ labels, Rows rows, int64_t V,
                                                           int64_t parts, int64_t len, MaxSum* part, MaxSum* row_stat,
                                                           float* label_logit, float* logps) {
  __shared__ float lm[kRowThreads / 64], ls[kRowThreads / 64];
  const int64_t i = blockIdx.x / parts, p = blockIdx.x - i * parts;
  const int64_t row = rows.at(i);
  const int64_t label = labels[row];
  if (label < 0 || label >= V) {
    if (parts == 1 && threadIdx.x == 0) logps[row] = 0.f;
    return;
  }
  const E* x = logits + row * V;
  const int64_t v0 = p * len, v1 = v0 + len < V ? v0 + len : V;
  float xl = 0.f;
  if (threadIdx.x == 0) xl = to_f32(x[label]);
  float m = -INFINITY, s = 0.f;
  constexpr int64_t kStep = 8 * kRowThreads;
  for (int64_t v = v0 + 8 * threadIdx.x; v < v1; v += kUnroll * kStep) {
    Raw8<E> r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t left = v1 - (v + u * kStep);
      if (left >= 8) load8(r[u], x + v + u * kStep, 8);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t left = v1 - (v + u * kStep);
      if (left <= 0) break;
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = r[u].get(j);
      if (left < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = j < left ? to_f32(x[v + u * kStep + j]) : -INFINITY;
      }
      float t = m;
#pragma unroll
      for (int j = 0; j < 8; ++j) t = fmaxf(t, f[j]);
      const float ref = t == -INFINITY ? 0.f : t;
      s *= exp2_hw((m - ref) * kLog2e);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += exp2_hw((f[j] - ref) * kLog2e);
      m = t;
    }
  }
#pragma unroll
  for (int k = 32; k >= 1; k >>= 1) merge(m, s, __shfl_xor(m, k, 64), __shfl_xor(s, k, 64));
  if ((threadIdx.x & 63) == 0) lm[threadIdx.x >> 6] = m, ls[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    m = lm[0], s = ls[0];
    for (int w = 1; w < kRowThreads / 64; ++w) merge(m, s, lm[w], ls[w]);
    if (parts == 1) {
      logps[row] = (xl - m) - logf(s);
      row_stat[row] = MaxSum{m, 1.f / s};
    } else {
      part[row * parts + p] = MaxSum{m, s};
      if (p == 0) label_logit[row] = xl;
    }
  }
}

// The parts of one row, joined in their order.
__device__ __forceinline__ float join_row(const MaxSum* part, int64_t parts, float xl, MaxSum* stat) {
  float m = part[0].m, s = part[0].s;
  for (int64_t p = 1; p < parts; ++p) merge(m, s, part[p].m, part[p].s);
  *stat = MaxSum{m, 1.f / s};
  return (xl - m) - logf(s);
}

__global__ __launch_bounds__(kRowThreads) void k_row_join(const MaxSum* __restrict__ part, int64_t parts,
                                                          const float* __restrict__ label_logit,
                                                          const int64_t* __restrict__ labels, int64_t V, int64_t rows,
                                                          MaxSum* row_stat, float* logps) {
  const int64_t row = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
  if (row >= rows) return;
  const bool counted = labels[row] >= 0 && labels[row] < V;
  logps[row] = counted ? join_row(part + row * parts, parts, label_logit[row], row_stat + row) : 0.f;
}

// One workgroup per pair: joins split rows, sums the log ratios in FP64 and forms the pair's
// loss and the coefficient of its gradient.
constexpr int kPairThreads = 1024;
struct PairArgs {
  const int64_t* labels;
  const float* ref;
  int64_t pairs, S, V, parts, first;
  float beta, smoothing, grad_scale;
  RowStats ws;
  float *logps, *log_ratios;
};
__global__ __launch_bounds__(kPairThreads) void k_pairs(PairArgs a) {
  __shared__ double lds[2][kPairThreads / 64];
  const int64_t pair = a.first + blockIdx.x;
  double sum[2] = {0.0, 0.0};
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int64_t r0 = (pair + side * a.pairs) * a.S;
    for (int64_t t = threadIdx.x; t < a.S; t += kPairThreads) {
      const int64_t row = r0 + t, label = a.labels[row];
      if (label < 0 || label >= a.V) {
        if (a.parts > 1) a.logps[row] = 0.f;
        continue;
      }
      float lp;
      if (a.parts > 1) {
        lp = join_row(a.ws.part + row * a.parts, a.parts, a.ws.label_logit[row], a.ws.row + row);
        a.logps[row] = lp;
      } else {
        lp = a.logps[row];
      }
      sum[side] += (double)lp - (a.ref ? (double)a.ref[row] : 0.0);
    }
    sum[side] = block_sum_f64<kPairThreads>(sum[side], lds[side]);
  }
  if (threadIdx.x == 0) {
    a.log_ratios[pair] = (float)sum[0];
    a.log_ratios[pair + a.pairs] = (float)sum[1];
    const double z = (double)a.beta * (sum[0] - sum[1]), e = a.smoothing;
    const double tail = log1p(exp(-fabs(z)));
    // a product with a smoothing of exactly 0 or 1 leaves out an infinite softplus
    const double win = tail + fmax(-z, 0.0), lose = tail + fmax(z, 0.0);
    a.ws.pair_loss[pair] = (e == 1.0 ? 0.0 : (1.0 - e) * (z != z ? z : win)) + (e == 0.0 ? 0.0 : e * (z != z ? z : lose));
    const double sig = z >= 0.0 ? 1.0 / (1.0 + exp(-z)) : exp(z) / (1.0 + exp(z));
    const double c = (double)a.grad_scale * ((double)a.beta / (double)a.pairs) * (z != z ? z : sig + e - 1.0);
    a.ws.coef[pair] = (float)c;
    a.ws.coef[pair + a.pairs] = (float)-c;
  }
}

__device__ __forceinline__ void mean_loss(const double* pair_loss, int64_t pairs, float* loss, double* lds) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < pairs; i += kRowThreads) s += pair_loss[i];
  s = block_sum_f64<kRowThreads>(s, lds);
  if (threadIdx.x == 0) *loss = (float)(s / (double)pairs);
}
__global__ __launch_bounds__(kRowThreads) void k_loss(const double* pair_loss, int64_t pairs, float* loss) {
  __shared__ double lds[kRowThreads / 64];
  mean_loss(pair_loss, pairs, loss, lds);
}

// The gradient: one workgroup per row and part, each element read and written once.
template <class E>
__global__ __launch_bounds__(kRowThreads) void k_pref_grad(const E* logits, E* dlogits,
                                                           const int64_t* __restrict__ labels, Rows rows, int64_t S,
                                                           int64_t V, int64_t parts, int64_t len,
                                                           const MaxSum* __restrict__ row_stat,
                                                           const float* __restrict__ coef,
                                                           const double* __restrict__ pair_loss, int64_t pairs,
                                                           float* loss) {
  __shared__ double lds[kRowThreads / 64];
  if (loss && blockIdx.x == 0) mean_loss(pair_loss, pairs, loss, lds);
  const int64_t i = blockIdx.x / parts, p = blockIdx.x - i * parts;
  const int64_t row = rows.at(i);
  const int64_t label = labels[row];
  const bool counted = label >= 0 && label < V;
  const float c = counted ? coef[row / S] : 0.f;
  const MaxSum stat = counted ? row_stat[row] : MaxSum{0.f, 0.f};
  const float scale = -c * stat.s;
  const int64_t v0 = p * len, v1 = v0 + len < V ? v0 + len : V;
  const E* x = logits + row * V;
  E* out = dlogits + row * V;
  constexpr int64_t kStep = 8 * kRowThreads;
  for (int64_t v = v0 + 8 * threadIdx.x; v < v1; v += kUnroll * kStep) {
    Raw8<E> r[kUnroll];
    if (counted) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t left = v1 - (v + u * kStep);
        if (left > 0) load8(r[u], x + v + u * kStep, left < 8 ? (int)left : 8);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t at = v + u * kStep, left = v1 - at;
      if (left <= 0) break;
      float f[8];
      if (counted) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = scale * exp2_hw((r[u].get(j) - stat.m) * kLog2e);
        if (label >= at && label < at + 8) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (at + j == label) f[j] += c;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = 0.f;
      }
      store8(out + at, f, left < 8 ? (int)left : 8);
    }
  }
}

template <class E>
hipError_t logps_as(const E* logits, const int64_t* labels, int64_t rows, int64_t V, float* logps, const RowStats& ws,
                    hipStream_t st) {
  const RowSplit sp = row_split(rows, V);
  hipLaunchKernelGGL((k_row_stats<E>), dim3((unsigned)(rows * sp.parts)), dim3(kRowThreads), 0, st, logits, labels,
                     (Rows{0, rows, 0}), V, sp.parts, sp.len, ws.part, ws.row, ws.label_logit, logps);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || sp.parts == 1) return e;
  hipLaunchKernelGGL(k_row_join, dim3((unsigned)((rows + kRowThreads - 1) / kRowThreads)), dim3(kRowThreads), 0, st,
                     ws.part, sp.parts, ws.label_logit, labels, V, rows, ws.row, logps);
  return hipGetLastError();
}

template <class E>
hipError_t preference_as(const Preference& p, const RowStats& ws, hipStream_t st) {
  const int64_t rows = 2 * p.pairs * p.S;
  const RowSplit sp = row_split(rows, p.V);
  const E* logits = static_cast<const E*>(p.logits);
  const Rows all{0, p.pairs * p.S, p.pairs * p.S};
  hipLaunchKernelGGL((k_row_stats<E>), dim3((unsigned)(rows * sp.parts)), dim3(kRowThreads), 0, st, logits, p.labels,
                     all, p.V, sp.parts, sp.len, ws.part, ws.row, ws.label_logit, p.logps);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const PairArgs pa{p.labels, p.ref_logps, p.pairs, p.S, p.V, sp.parts, 0, p.beta, p.smoothing, p.grad_scale, ws,
                    p.logps, p.log_ratios};
  hipLaunchKernelGGL(k_pairs, dim3((unsigned)p.pairs), dim3(kPairThreads), 0, st, pa);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (!p.dlogits) {
    hipLaunchKernelGGL(k_loss, dim3(1), dim3(kRowThreads), 0, st, ws.pair_loss, p.pairs, p.loss);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((k_pref_grad<E>), dim3((unsigned)(rows * sp.parts)), dim3(kRowThreads), 0, st, logits,
                     static_cast<E*>(p.dlogits), p.labels, all, p.S, p.V, sp.parts, sp.len, ws.row, ws.coef,
                     ws.pair_loss, p.pairs, p.loss);
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
