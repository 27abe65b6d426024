// out = residual + drop(x): eight elements per generator block, one fused multiply-add each.  A thread
// makes the mask of the eight elements that it loads, so nothing but the operands moves.  Bound by
// HBM for long tensors (8192 x 4096 BF16 and a residual 30.6 us, 6.6 TB/s), by the launch for short ones
// (4096 elements 2 us).
#include "adapters_device.h"
#include "train_device.h"

namespace qlora {
namespace {

constexpr int kThreads = 256;

template <class X, class O, bool RES>
__global__ __launch_bounds__(kThreads) void k_dropout(const X* x, int64_t n, DropMask drop, const O* residual, O* out) {
  RngKey key{};
  if (drop.threshold) key = load_rng(drop.rng);
  const uint32_t t2 = threshold_halves(drop.threshold);
  const int64_t blocks = (n + 7) / 8, stride = (int64_t)gridDim.x * kThreads;
  for (int64_t b = (int64_t)blockIdx.x * kThreads + threadIdx.x; b < blocks; b += stride) {
    const int left = (int)(n - 8 * b < 8 ? n - 8 * b : 8);
    Raw8<X> v;
    load8(v, x + 8 * b, left, false);
    Raw8<O> r;
    if (RES) load8(r, residual + 8 * b, left, false);
    const uint4 w = drop.threshold ? philox(key, (uint64_t)b) : make_uint4(0, 0, 0, 0);
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t keep = drop.threshold ? keep_halves(words[i], t2) : 0xFFFFFFFFu;
      const float a = (keep & 0xFFFFu) ? v.get(2 * i) : 0.f, c = (keep >> 16) ? v.get(2 * i + 1) : 0.f;
      f[2 * i] = RES ? fmaf(a, drop.scale, r.get(2 * i)) : a * drop.scale;
      f[2 * i + 1] = RES ? fmaf(c, drop.scale, r.get(2 * i + 1)) : c * drop.scale;
    }
    store8(out + 8 * b, f, left);
  }
}

template <class X, class O>
hipError_t dropout_as(const void* x, int64_t n, const DropMask& drop, const void* residual, void* out, hipStream_t st) {
  const int64_t blocks = (n + 7) / 8;
  const dim3 grid((unsigned)std::min<int64_t>((blocks + kThreads - 1) / kThreads, 256 * 16));
  if (residual)
    hipLaunchKernelGGL((k_dropout<X, O, true>), grid, dim3(kThreads), 0, st, static_cast<const X*>(x), n, drop,
                       static_cast<const O*>(residual), static_cast<O*>(out));
  else
    hipLaunchKernelGGL((k_dropout<X, O, false>), grid, dim3(kThreads), 0, st, static_cast<const X*>(x), n, drop,
                       static_cast<const O*>(nullptr), static_cast<O*>(out));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const void* x, int x_f32, int64_t n, const DropMask& drop, const void* residual, void* out,
                          int out_f32, hipStream_t st) {
  if (x_f32) return out_f32 ? dropout_as<float, float>(x, n, drop, residual, out, st)
                            : dropout_as<float, uint16_t>(x, n, drop, residual, out, st);
  return out_f32 ? dropout_as<uint16_t, float>(x, n, drop, residual, out, st)
                 : dropout_as<uint16_t, uint16_t>(x, n, drop, residual, out, st);
}

}  // namespace qlora
