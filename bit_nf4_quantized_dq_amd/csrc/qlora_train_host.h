// Internal host-side declarations of the training-step operators (include/qlora_train.h):
// their launchers, defined next to their kernels, and the plans that the entry points and the
// launchers share.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "qlora.h"
#include "qlora_host.h"
#include "qlora_train.h"

namespace qlora {

// ---- block norms (norm.hip)
constexpr int64_t kNormMaxWidth = QLORA_NORM_MAX_WIDTH;  // 1024 threads of one vector of eight

struct NormFwd {
  const void* x;
  const uint16_t *y, *w_post, *gate, *w_pre;
  void* x_out;
  uint16_t* h;
  int64_t M, d, gate_rows;
  float scale, eps;
  int f32, post;
};
struct NormBwd {
  const void* x;
  const uint16_t *y, *dh;
  const void* dx_out;
  const uint16_t *w_post, *gate, *w_pre;
  void* dx;
  uint16_t *dy, *dw_post, *dgate, *dw_pre;
  float* part;
  unsigned int* counter;
  int64_t M, d, gate_rows;
  float scale, eps;
  int f32, post;
};
// The backward's rows in `count` segments of at most `rows` rows, one workgroup each.  A gate
// row's rows (without a gate all rows) are either split into per_group segments, each taking
// every per_group-th row (per_group > 0), or lie whole in one segment of consecutive rows
// (per_group == 0: rows is a multiple of gate_rows).
struct NormSegments {
  int64_t rows, count, per_group;
};
// The threads of a row: one for each eight columns, in whole wavefronts.
inline unsigned norm_threads(int64_t d) { return (unsigned)((d + 511) / 512 * 64); }
NormSegments norm_segments(int64_t M, int64_t d, int64_t gate_rows);
hipError_t launch_norm_fwd(const NormFwd& p, hipStream_t st);
hipError_t launch_norm_bwd(const NormBwd& p, hipStream_t st);

// ---- token log-probabilities and the preference loss (preference.hip)
struct RowSplit {
  int64_t parts, len;  // vocabulary parts of a row and their length
};
RowSplit row_split(int64_t rows, int64_t V);
struct MaxSum {  // a maximum, and the sum of the exponentials of the differences to it
  float m, s;
};
struct RowStats {       // carved from the workspace
  MaxSum* part;         // [rows][parts]
  float* label_logit;   // [rows], for split rows
  double* ratio;        // [rows] log ratios of whole rows (null without a loss)
  double* pair_loss;    // [pairs]
  unsigned int* counter;
};
struct Preference {
  const void* logits;
  const int64_t* labels;
  const float* ref_logps;
  int64_t pairs, S, V;
  float beta, smoothing, grad_scale;
  float *loss, *log_ratios, *logps;
  void* dlogits;
  int f32;
};
hipError_t launch_token_logps(const void* logits, const int64_t* labels, int64_t rows, int64_t V, int f32,
                              float* logps, const RowStats& ws, hipStream_t st);
hipError_t launch_preference(const Preference& p, const RowStats& ws, hipStream_t st);

// ---- gradient lists (gradients.hip)
constexpr int64_t kGradChunk = 16384;  // elements of one table entry
struct GradChunk {
  const void* in;
  void* out;
  int32_t n;
  int16_t in_f32, out_f32;
};
static_assert(sizeof(GradChunk) == 24, "one table entry");
struct GradTensor {
  const void* in;
  void* out;
  int64_t n, first;  // elements, first chunk
  int32_t in_f32, out_f32;
};
constexpr int kGradBatch = 96;  // tensors described by one launch's arguments (under 4 KB)
struct GradTensors {
  GradTensor t[kGradBatch];
};
hipError_t launch_grad_table(const GradTensors& batch, int count, GradChunk* table, hipStream_t st);
hipError_t launch_grad_norm(const GradChunk* table, int64_t chunks, float* norm, double* part, unsigned int* counter,
                            hipStream_t st);
hipError_t launch_grad_clip(const GradChunk* table, int64_t chunks, const float* norm, float max_norm, hipStream_t st);
int64_t grad_norm_parts(int64_t chunks);

// ---- the optimizer step with clipping folded in (adamw.hip), and the checks and scalars that
// both steps share (api.cpp)
hipError_t launch_adamw_clipped(float* master, float* m, float* v, const uint16_t* grad, uint16_t* param, int64_t n,
                                const AdamWScalars& a, const float* norm, float max_norm, hipStream_t s);

}  // namespace qlora
