// AdamW step over the flat trainable adapter parameters.
//
// State per parameter, as the pages account for it: an FP32 master weight, an FP32 first
// moment and an FP32 second moment (12 bytes), beside the BF16 working weight and the BF16
// gradient ("QLoRA: Quantize Base Weights to 4-Bit", Section 1 and the optimizer term of
// Section 4; "QLoRA -- Fine-Tuning a 65B Model on One GPU", "Paged optimizers").  The update
// is the published AdamW (Loshchilov and Hutter, "Decoupled Weight Decay Regularization",
// 2019; bias correction of Kingma and Ba, "Adam", 2015), decay scaled by the learning rate:
//   theta *= 1 - lr wd;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2;
//   theta -= (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps);  param = bf16(theta).
// The step-dependent scalars are formed on the host in FP64 and rounded once to FP32.
//
// The kernel is a pure stream: 14 bytes read and 14 written per parameter (28 B), so it is
// bound by HBM.  Each lane takes 4 consecutive parameters (16-byte state loads, 8-byte
// gradient loads and parameter stores); a tail of n % 4 parameters runs element by element.
//
// With clipping (kClip) each gradient is multiplied by min(1, max_norm / (norm + 1e-6)) as it
// is read, in FP32 and without a rounding to BF16: the clipped gradients are never written, so
// the step still moves 28 B per parameter.  A norm that is not finite leaves every state as it
// is.  41.9M parameters with their norm: 219 us, 5.4 TB/s of the step's 1.17 GB (239 us when the
// states go through the cache and push the gradients out).
#include "qlora_train_host.h"
#include "train_device.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void adamw1(float& th, float& m, float& v, float g, const AdamWScalars& a) {
  th = __fmul_rn(th, a.decay);
  m = __fadd_rn(__fmul_rn(a.b1, m), __fmul_rn(a.omb1, g));
  v = __fadd_rn(__fmul_rn(a.b2, v), __fmul_rn(a.omb2, __fmul_rn(g, g)));
  const float den = __fadd_rn(__fmul_rn(__fsqrt_rn(v), a.inv_bc2_sqrt), a.eps);
  th = __fsub_rn(th, __fdiv_rn(__fmul_rn(a.step_size, m), den));
}

// Four values of a state.  kPast: read and written past the cache, which then still holds the
// gradients that the norm has just read.
template <bool kPast>
__device__ __forceinline__ float4 state_load(const float* p, int64_t i) {
  typedef float f4 __attribute__((ext_vector_type(4)));
  if (!kPast) return reinterpret_cast<const float4*>(p)[i];
  const f4 v = __builtin_nontemporal_load(reinterpret_cast<const f4*>(p) + i);
  return make_float4(v.x, v.y, v.z, v.w);
}
template <bool kPast>
__device__ __forceinline__ void state_store(float* p, int64_t i, const float4& v) {
  typedef float f4 __attribute__((ext_vector_type(4)));
  if (kPast) __builtin_nontemporal_store(f4{v.x, v.y, v.z, v.w}, reinterpret_cast<f4*>(p) + i);
  else reinterpret_cast<float4*>(p)[i] = v;
}

template <bool kClip>
__device__ __forceinline__ float clipped(float g, float c) {
  return kClip ? __fmul_rn(g, c) : g;
}

template <bool kClip>
__global__ __launch_bounds__(kThreads) void k_adamw(float* __restrict__ master, float* __restrict__ mom1,
                                                    float* __restrict__ mom2, const uint16_t* __restrict__ grad,
                                                    uint16_t* __restrict__ param, int64_t n, AdamWScalars a,
                                                    const float* __restrict__ norm, float max_norm) {
  float c = 1.f;
  if (kClip) {
    if (!(fabsf(*norm) < INFINITY)) return;
    c = clip_coefficient(*norm, max_norm);
  }
  const int64_t n4 = n >> 2;
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n4; i += stride) {
    float4 th = state_load<kClip>(master, i);
    float4 m = state_load<kClip>(mom1, i);
    float4 v = state_load<kClip>(mom2, i);
    const uint2 gb = reinterpret_cast<const uint2*>(grad)[i];
    adamw1(th.x, m.x, v.x, clipped<kClip>(bf16lo_to_f32(gb.x), c), a);
    adamw1(th.y, m.y, v.y, clipped<kClip>(bf16hi_to_f32(gb.x), c), a);
    adamw1(th.z, m.z, v.z, clipped<kClip>(bf16lo_to_f32(gb.y), c), a);
    adamw1(th.w, m.w, v.w, clipped<kClip>(bf16hi_to_f32(gb.y), c), a);
    state_store<kClip>(master, i, th);
    state_store<kClip>(mom1, i, m);
    state_store<kClip>(mom2, i, v);
    if (param) reinterpret_cast<uint2*>(param)[i] = make_uint2(pack_bf16x2(th.x, th.y), pack_bf16x2(th.z, th.w));
  }
  // tail: the last n % 4 parameters, one per lane of the first workgroup
  if (blockIdx.x == 0 && threadIdx.x < (n & 3)) {
    const int64_t j = 4 * n4 + threadIdx.x;
    float th = master[j], m = mom1[j], v = mom2[j];
    adamw1(th, m, v, clipped<kClip>(__uint_as_float((uint32_t)grad[j] << 16), c), a);
    master[j] = th;
    mom1[j] = m;
    mom2[j] = v;
    if (param) param[j] = (uint16_t)(pack_bf16x2(th, 0.f) & 0xFFFFu);
  }
}

unsigned grid_for(int64_t n) {
  const int64_t want = ((n >> 2) + kThreads - 1) / kThreads;
  return (unsigned)(want < 1 ? 1 : (want > 65536 ? 65536 : want));
}

}  // namespace

hipError_t launch_adamw(float* master, float* m, float* v, const uint16_t* grad, uint16_t* param, int64_t n,
                        const AdamWScalars& a, hipStream_t s) {
  LaunchTimer t(10, s);
  hipExtLaunchKernelGGL(k_adamw<false>, dim3(grid_for(n)), dim3(kThreads), 0, s, t.start, t.stop, 0, master, m, v, grad,
                        param, n, a, (const float*)nullptr, 0.f);
  return hipGetLastError();
}

hipError_t launch_adamw_clipped(float* master, float* m, float* v, const uint16_t* grad, uint16_t* param, int64_t n,
                                const AdamWScalars& a, const float* norm, float max_norm, hipStream_t s) {
  LaunchTimer t(10, s);
  hipExtLaunchKernelGGL(k_adamw<true>, dim3(grid_for(n)), dim3(kThreads), 0, s, t.start, t.stop, 0, master, m, v, grad,
                        param, n, a, norm, max_norm);
  return hipGetLastError();
}

}  // namespace qlora
