// Global norm of a list of gradient tensors, and clipping:
//   norm = sqrt(sum over all tensors of sum g^2),   c = min(1, max_norm / (norm + 1e-6)),
//   out = c g.
// The list is a table in device memory with one entry per 16384 elements of a tensor, so one
// launch covers any number of tensors and no workgroup searches for its own.
//
// HBM bounds both kernels.  Measured (MI355X): the norm of 448 tensors, 41.9M elements, 17 us
// in BF16 (84 MB; 23 - 29 right after an optimizer step) and 32 us in FP32 (168 MB, 5.3 TB/s; a
// plain read reaches 7.0), of 14 tensors (2.6 MB) 4.7 us on the device; clipping the FP32 list into BF16 37 us more (6.8 TB/s: the
// cache still holds what the norm has read; results are written past it, 70 us for both
// kernels instead of 80, and 8 us less also with the optimizer step that reads them).
// Squares and sums are FP64: a conversion and a multiply-add an element stay below the load's
// time, and no square overflows or vanishes.
#include "qlora_train_host.h"
#include "train_device.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = (int)(kGradChunk / (8 * kThreads));  // vectors of eight per thread of a full chunk

__global__ __launch_bounds__(kThreads) void k_grad_table(GradTensors batch, GradChunk* __restrict__ table) {
  const GradTensor t = batch.t[blockIdx.x];
  const int64_t chunks = (t.n + kGradChunk - 1) / kGradChunk;
  for (int64_t c = threadIdx.x; c < chunks; c += kThreads) {
    const int64_t at = c * kGradChunk, left = t.n - at;
    GradChunk e;
    e.in = static_cast<const char*>(t.in) + at * (t.in_f32 ? 4 : 2);
    e.out = static_cast<char*>(t.out) + at * (t.out_f32 ? 4 : 2);
    e.n = (int32_t)(left < kGradChunk ? left : kGradChunk);
    e.in_f32 = (int16_t)t.in_f32;
    e.out_f32 = (int16_t)t.out_f32;
    table[t.first + c] = e;
  }
}

// Sum of the squares of a wavefront's piece [p, p + n): 32 elements a lane, all in flight at once.
constexpr int kPiece = 2048, kPieces = (int)(kGradChunk / kPiece), kPieceVecs = kPiece / (8 * 64);

template <class E>
__device__ __forceinline__ double piece_sum(const E* __restrict__ p, int32_t n, bool wide, double sum) {
  const int lane = threadIdx.x & 63;
  if (n >= kPiece) {
    Raw8<E> r[kPieceVecs];
#pragma unroll
    for (int v = 0; v < kPieceVecs; ++v) load_all8(r[v], p + 8 * (v * 64 + lane));
#pragma unroll
    for (int v = 0; v < kPieceVecs; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double g = (double)r[v].get(i);
        sum = fma(g, g, sum);
      }
  } else {
    for (int e = 8 * lane; e < n; e += 8 * 64) {
      Raw8<E> r;
      load8(r, p + e, n - e, wide);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double g = (double)r.get(i);
        sum = fma(g, g, sum);
      }
    }
  }
  return sum;
}

// Wavefronts take the pieces in turn.  The partials travel by system-scope (cache-bypassing)
// stores and loads, and a store has completed before its workgroup is counted (the wait orders
// the two on this chip; no rule of the language does); the last workgroup adds them in the
// workgroups' order.
template <int T>
__global__ __launch_bounds__(T) void k_grad_norm(const GradChunk* __restrict__ table, int64_t chunks, float* norm,
                                                 double* part, unsigned int* counter) {
  __shared__ double lds[2][T / 64];
  __shared__ bool s_last;
  double sum = 0.0;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  for (int64_t u = (int64_t)blockIdx.x * (T / 64) + wave; u < chunks * kPieces; u += (int64_t)gridDim.x * (T / 64)) {
    const GradChunk e = table[u / kPieces];
    const int32_t at = (int32_t)(u % kPieces) * kPiece, n = e.n - at;
    if (n <= 0) continue;
    // a short last vector may reach back into the piece, or the chunk, before it
    const bool wide = e.n >= 8;
    sum = e.in_f32 ? piece_sum(static_cast<const float*>(e.in) + at, n, wide, sum)
                   : piece_sum(static_cast<const uint16_t*>(e.in) + at, n, wide, sum);
  }
  sum = block_sum_f64<T>(sum, lds[0]);
  if (threadIdx.x == 0) {
    __hip_atomic_store(part + blockIdx.x, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
    __builtin_amdgcn_s_waitcnt(0);
    const unsigned int old = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s_last = old + 1u == gridDim.x;
  }
  __syncthreads();
  if (!s_last) return;
  sum = 0.0;
  for (unsigned int i = threadIdx.x; i < gridDim.x; i += T)
    sum += __hip_atomic_load(part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
  sum = block_sum_f64<T>(sum, lds[1]);
  if (threadIdx.x == 0) {
    *norm = (float)sqrt(sum);
    __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

template <class A, class B>
__device__ __forceinline__ void chunk_scale(const A* p, B* q, int32_t n, float c) {
  if (n == kGradChunk) {
    Raw8<A> r[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) load_all8(r[v], p + 8 * (v * kThreads + (int)threadIdx.x));
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = r[v].get(i) * c;
      stream8(q + 8 * (v * kThreads + (int)threadIdx.x), f);
    }
  } else {
    for (int e = 8 * (int)threadIdx.x; e < n; e += 8 * kThreads) {
      Raw8<A> r;
      load8(r, p + e, n - e, n >= 8);
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = r.get(i) * c;
      store8(q + e, f, n - e);
    }
  }
}

__global__ __launch_bounds__(kThreads) void k_grad_clip(const GradChunk* __restrict__ table, const float* norm,
                                                        float max_norm) {
  const float c = clip_coefficient(*norm, max_norm);
  const GradChunk e = table[blockIdx.x];
  if (e.in == e.out && e.in_f32 == e.out_f32 && c == 1.f) return;
  if (e.in_f32) {
    if (e.out_f32) chunk_scale(static_cast<const float*>(e.in), static_cast<float*>(e.out), e.n, c);
    else chunk_scale(static_cast<const float*>(e.in), static_cast<uint16_t*>(e.out), e.n, c);
  } else {
    if (e.out_f32) chunk_scale(static_cast<const uint16_t*>(e.in), static_cast<float*>(e.out), e.n, c);
    else chunk_scale(static_cast<const uint16_t*>(e.in), static_cast<uint16_t*>(e.out), e.n, c);
  }
}

}  // namespace

// At most one workgroup for each compute unit: each adds one to the counter, and additions to
// one address take about 8 ns each, one after the other.
int64_t grad_norm_parts(int64_t chunks) {
  const int64_t pieces = chunks * kPieces;
  if (pieces <= 256 * 4) return pieces < 4 ? 1 : (pieces + 3) / 4;  // four wavefronts each
  return pieces < 256 * 16 ? (pieces + 15) / 16 : 256;              // sixteen
}

hipError_t launch_grad_table(const GradTensors& batch, int count, GradChunk* table, hipStream_t st) {
  hipLaunchKernelGGL(k_grad_table, dim3((unsigned)count), dim3(kThreads), 0, st, batch, table);
  return hipGetLastError();
}

hipError_t launch_grad_norm(const GradChunk* table, int64_t chunks, float* norm, double* part, unsigned int* counter,
                            hipStream_t st) {
  const dim3 grid((unsigned)grad_norm_parts(chunks));
  if (chunks * kPieces <= 256 * 4) {
    hipLaunchKernelGGL(k_grad_norm<256>, grid, dim3(256), 0, st, table, chunks, norm, part, counter);
  } else {
    hipLaunchKernelGGL(k_grad_norm<1024>, grid, dim3(1024), 0, st, table, chunks, norm, part, counter);
  }
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradChunk* table, int64_t chunks, const float* norm, float max_norm,
                            hipStream_t st) {
  hipLaunchKernelGGL(k_grad_clip, dim3((unsigned)chunks), dim3(kThreads), 0, st, table, norm, max_norm);
  return hipGetLastError();
}

}  // namespace qlora
