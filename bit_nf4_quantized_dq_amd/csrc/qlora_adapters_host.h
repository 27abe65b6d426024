// Internal host-side declarations of the operators of include/qlora_adapters.h: the table
// entry, the plans that entry points and launchers share, and the launchers.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "qlora_adapters.h"
#include "qlora_host.h"

namespace qlora {

// One adapter of the device table.
struct AdapterEntry {
  const uint16_t *A, *B;
  uint16_t *dA, *dB;
  int32_t r;
  float s;  // alpha / r
};
static_assert(sizeof(AdapterEntry) == 40, "one table entry");
constexpr int kAdapterBatch = 96;  // adapters described by one launch's arguments (under 4 KB)
struct AdapterBatch {
  AdapterEntry e[kAdapterBatch];
};
hipError_t launch_adapter_table(const AdapterBatch& batch, int count, AdapterEntry* table, hipStream_t st);

// A mask: the generator's seed and offset in device memory, the 16-bit threshold below which an
// element is dropped (0: nothing is, rng is not read) and the scale of what is kept.
struct DropMask {
  const uint64_t* rng;
  uint32_t threshold;
  float scale;
};

// Rows and their adapters.
struct AdapterRows {
  const AdapterEntry* table;
  const int32_t* ids;  // null: adapter 0 for all
  int64_t M;
  int32_t count, max_rank, width;  // width: FP32 columns of T and G
  int32_t whole;                   // every rank is a multiple of 8
};

// ---- T = drop(X) A_a^T or G = dY B_a, FP32 [M, width] (adapters.hip), with the decode of the
// weight in the same launch when `decode` is given (E4M3 constants; into w_hat for T, w_hat^T
// for G).  The reduction is split over shrink_split() workgroups per 16 rows; the last of them
// adds the others' partials (part: FP32 [split][M][width]; one counter per 16 rows).
struct ShrinkDecode {
  const uint32_t* codes;
  const uint8_t* code8;
  const float *c2s, *mu;
  uint16_t* out;
  int64_t N, K;
};
int32_t shrink_split(int64_t M, int64_t Kd);
hipError_t launch_shrink_a(const AdapterRows& rows, const uint16_t* X, int64_t K, const DropMask& drop, float* T,
                           float* part, unsigned int* counters, const ShrinkDecode* decode, const Nf4Tables& tab,
                           hipStream_t st);
hipError_t launch_shrink_b(const AdapterRows& rows, const uint16_t* dY, int64_t N, float* G, float* part,
                           unsigned int* counters, const ShrinkDecode* decode, const Nf4Tables& tab, hipStream_t st);
// T and G in one launch (no decode); counters: two per 16 rows.
hipError_t launch_shrink_both(const AdapterRows& rows, const uint16_t* X, int64_t K, const DropMask& drop, float* T,
                              const uint16_t* dY, int64_t N, float* G, float* part_t, float* part_g,
                              unsigned int* counters, hipStream_t st);

// ---- few rows: Y by a launch that streams the weight once (E4M3 constants).  T (FP32 [M, width]) is
// written by a launch before it, or, where stream_forms_t(), by the same one (T may then be NULL),
// by way of the workspace's head, where a workgroup looks `polls` times for an element before it forms
// it itself.
bool adapter_stream_fits(int64_t M, int64_t N, int64_t K);
bool stream_forms_t(int64_t M, int64_t N, int32_t width);
hipError_t launch_adapter_stream(const uint32_t* codes, const uint8_t* code8, const float* c2s, const float* mu,
                                 int64_t N, int64_t K, const uint16_t* X, const AdapterRows& rows, const DropMask& drop,
                                 float* T, uint16_t* Y, void* head, int32_t polls, const Nf4Tables& tab, hipStream_t st);

// ---- many rows: the GEMM over the decoded copy (gemm_nt.hip), its accumulators started from the
// adapters' term, scale s_a U W_a^T (fwd: U = T, W_a = B_a [F, r]; else U = G, W_a = A_a^T of
// A_a [r, F]), under the mask `drop` over C's elements where its threshold is not 0.
struct AdapterHead {
  AdapterRows rows;
  const float* U;
  int32_t transposed;  // W_a = A_a^T
  float scale;
  DropMask drop;
};
hipError_t launch_gemm_nt_adapters(const uint16_t* A, int64_t F, const uint16_t* B, int64_t M, int64_t Kr,
                                   const AdapterHead& head, uint16_t* C, int kernel_id, hipStream_t st, float* part,
                                   int32_t ksplit);

// ---- a moderate number of rows: the same product over the codes, decoded on chip (adapters_gemm.hip,
// E4M3 constants), where adapter_gemm_fits(); part: FP32 [split][M][F] when split > 1.
bool adapter_gemm_fits(int64_t M, int64_t F, int64_t Kr);
int32_t adapter_gemm_split(int64_t M, int64_t F, int64_t Kr);
hipError_t launch_adapter_gemm(const uint32_t* codes, const uint8_t* code8, const float* c2s, const float* mu, int64_t N,
                               int64_t K, const uint16_t* X, int64_t M, const AdapterHead& head, uint16_t* C, float* part,
                               int32_t split, const Nf4Tables& tab, int kernel_id, hipStream_t st);

// ---- dA_a and dB_a of every adapter in one launch.  Rows in `split` slices; with more than one,
// FP32 partials [adapter][rank block][column tile][split][64 x 64] and one counter per
// (adapter, rank block, column tile).
struct GradPlan {
  int64_t tiles_a, tiles_b;  // 64-column tiles of dA and dB
  int32_t blocks, split;     // blocks of up to 64 ranks
  size_t part_bytes;
};
GradPlan adapter_grad_plan(int64_t M, int64_t N, int64_t K, int32_t count, int32_t max_rank);
hipError_t launch_adapter_grads(const AdapterRows& rows, const uint16_t* X, int64_t K, const uint16_t* dY, int64_t N,
                                const float* T, const float* G, const DropMask& drop, float* part,
                                unsigned int* counters, hipStream_t st);

// ---- dropout.hip
hipError_t launch_dropout(const void* x, int x_f32, int64_t n, const DropMask& drop, const void* residual, void* out,
                          int out_f32, hipStream_t st);

}  // namespace qlora
