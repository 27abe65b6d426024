// C ABI of the training-step operators (declared in include/qlora_train.h): argument checks,
// workspace layouts and plans; the kernels and their launches are in norm.hip, preference.hip,
// gradients.hip and adamw.hip.
#include <algorithm>
#include <cmath>

#include "qlora_train.h"
#include "qlora_train_host.h"

using namespace qlora;

namespace {

constexpr size_t kHead = QLORA_WS_COUNTER_BYTES;
constexpr int64_t kMaxRows = int64_t(1) << 24;   // a grid dimension's threads stay below 2^32
constexpr int64_t kMaxVocab = int64_t(1) << 22;  // the widest weight's d_out

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP; }
inline bool type_ok(int type) { return type == QLORA_BF16 || type == QLORA_F32; }
inline size_t type_bytes(int type) { return type == QLORA_F32 ? 4 : 2; }

int check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws || ws_bytes < need) return QLORA_ERR_WORKSPACE;
  return aligned(ws, 16) ? QLORA_OK : QLORA_ERR_INVALID_ARG;
}

int check_norm(int64_t M, int64_t d) {
  if (M < 1 || M >= kMaxRows) return QLORA_ERR_INVALID_ARG;
  if (d < 1 || d > kNormMaxWidth) return QLORA_ERR_BAD_SHAPE;
  return QLORA_OK;
}
int check_norm_operands(const uint16_t* y, int64_t M, int64_t d, int type, int post_norm, const uint16_t* w_post,
                        const uint16_t* gate, int64_t gate_rows, const uint16_t* w_pre, float res_scale, float eps) {
  const int st = check_norm(M, d);
  if (st) return st;
  if (!type_ok(type)) return QLORA_ERR_UNSUPPORTED;
  if (!std::isfinite(res_scale) || !std::isfinite(eps) || eps < 0.f) return QLORA_ERR_INVALID_ARG;
  if ((post_norm != 0 || gate) && !y) return QLORA_ERR_INVALID_ARG;
  if (w_post && !post_norm) return QLORA_ERR_INVALID_ARG;
  if (gate && gate_rows < 1) return QLORA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)y, (const void*)w_post, (const void*)gate, (const void*)w_pre})
    if (!aligned(p, 2)) return QLORA_ERR_INVALID_ARG;
  return QLORA_OK;
}

int check_logits(const void* logits, const int64_t* labels, int64_t rows, int64_t V, int type) {
  if (rows < 1 || rows >= kMaxRows) return QLORA_ERR_INVALID_ARG;
  if (V < 1 || V > kMaxVocab) return QLORA_ERR_BAD_SHAPE;
  if (!type_ok(type)) return QLORA_ERR_UNSUPPORTED;
  if (!logits || !labels || !aligned(logits, type_bytes(type)) || !aligned(labels, 8)) return QLORA_ERR_INVALID_ARG;
  return QLORA_OK;
}

// The statistics of `rows` rows, and for the loss what belongs to `pairs` pairs.
size_t carve_stats(void* ws, int64_t rows, int64_t V, int64_t pairs, RowStats* out) {
  const RowSplit sp = row_split(rows, V);
  size_t off = kHead;
  const auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return static_cast<char*>(ws) + at;
  };
  RowStats s{};
  s.counter = static_cast<unsigned int*>(ws);
  s.part = reinterpret_cast<MaxSum*>(take(sizeof(MaxSum) * (size_t)(rows * sp.parts)));
  if (sp.parts > 1) s.label_logit = reinterpret_cast<float*>(take(sizeof(float) * (size_t)rows));
  if (pairs) {
    if (sp.parts == 1) s.ratio = reinterpret_cast<double*>(take(sizeof(double) * (size_t)rows));
    s.pair_loss = reinterpret_cast<double*>(take(sizeof(double) * (size_t)pairs));
  }
  if (out) *out = s;
  return off;
}

int check_list(const qlora_gradlist_t* list) {
  if (!list || list->chunks < 0 || list->chunks >= kMaxRows) return QLORA_ERR_INVALID_ARG;
  if (list->chunks && (!list->table || !aligned(list->table, 16))) return QLORA_ERR_INVALID_ARG;
  return QLORA_OK;
}
int count_chunks(int count, const int64_t* numel, int64_t* chunks) {
  if (count < 0 || (count && !numel)) return QLORA_ERR_INVALID_ARG;
  int64_t n = 0;
  for (int i = 0; i < count; ++i) {
    if (numel[i] < 0) return QLORA_ERR_INVALID_ARG;
    if (numel[i] > kMaxRows * kGradChunk) return QLORA_ERR_BAD_SHAPE;
    n += (numel[i] + kGradChunk - 1) / kGradChunk;
    if (n >= kMaxRows) return QLORA_ERR_BAD_SHAPE;
  }
  *chunks = n;
  return QLORA_OK;
}
size_t grad_ws_bytes(int64_t chunks) { return kHead + sizeof(double) * (size_t)grad_norm_parts(chunks); }

}  // namespace

namespace qlora {

NormSegments norm_segments(int64_t M, int64_t d, int64_t gate_rows) {
  // As many segments as the sixteen wavefronts (of 128 registers) of each of the 256 compute units
  // hold at once, but at least four rows a segment, and eight where that leaves two segments
  // to a compute unit: their partials then cost an eighth of what the rows do (4096 x 2560:
  // 43 us with six rows, 38 with eight, 47 with twelve).
  const int64_t slots = 256 * (16 / (norm_threads(d) / 64));
  int64_t rows = std::max((M + slots - 1) / slots, std::min<int64_t>(8, std::max<int64_t>(4, M / 512)));
  NormSegments s{};
  gate_rows = gate_rows ? std::min(gate_rows, M) : M;
  if (gate_rows <= rows) {
    if (gate_rows > 1) rows = rows / gate_rows * gate_rows;
    s.rows = rows;
    s.count = (M + rows - 1) / rows;
  } else {
    s.per_group = (gate_rows + rows - 1) / rows;
    s.rows = (gate_rows + s.per_group - 1) / s.per_group;
    s.count = (M + gate_rows - 1) / gate_rows * s.per_group;
  }
  return s;
}

RowSplit row_split(int64_t rows, int64_t V) {
  // Whole rows from 128 rows on: 160 of 131072 entries 24 us with the gradient, 27.6 in parts, 400
  // of 32768 18.8 and 22.  Fewer leave compute units idle and are split into parts of at least
  // 8192 elements.
  const int64_t want = rows >= 128 ? 1 : (2048 + rows - 1) / rows;
  const int64_t parts = std::max<int64_t>(1, std::min(want, V / 8192));
  const int64_t len = ((V + parts - 1) / parts + 7) / 8 * 8;
  return RowSplit{(V + len - 1) / len, len};
}

}  // namespace qlora

extern "C" {

int qlora_norm_residual_fwd(const void* x, const uint16_t* y, int64_t M, int64_t d, int type, int post_norm,
                            const uint16_t* w_post, const uint16_t* gate, int64_t gate_rows, const uint16_t* w_pre,
                            float res_scale, float eps, void* x_out, uint16_t* h, hipStream_t stream) {
  const int st =
      check_norm_operands(y, M, d, type, post_norm, w_post, gate, gate_rows, w_pre, res_scale, eps);
  if (st) return st;
  if (!x || (!x_out && !h) || (w_pre && !h)) return QLORA_ERR_INVALID_ARG;
  if (!aligned(x, type_bytes(type)) || !aligned(x_out, type_bytes(type)) || !aligned(h, 2))
    return QLORA_ERR_INVALID_ARG;
  return hip_status(launch_norm_fwd(
      NormFwd{x, y, w_post, gate, w_pre, x_out, h, M, d, gate ? gate_rows : 1, res_scale, eps, type == QLORA_F32,
              post_norm != 0},
      stream));
}

int qlora_norm_residual_workspace_size(int64_t M, int64_t d, int64_t gate_rows, size_t* ws_bytes) {
  if (!ws_bytes || gate_rows < 0) return QLORA_ERR_INVALID_ARG;
  const int st = check_norm(M, d);
  if (st) return st;
  *ws_bytes = kHead + 3 * sizeof(float) * (size_t)(norm_segments(M, d, gate_rows).count * d);
  return QLORA_OK;
}

int qlora_norm_residual_bwd(const void* x_out, const uint16_t* y, const uint16_t* dh, const void* dx_out, int64_t M,
                            int64_t d, int type, int post_norm, const uint16_t* w_post, const uint16_t* gate,
                            int64_t gate_rows, const uint16_t* w_pre, float res_scale, float eps, void* dx,
                            uint16_t* dy, uint16_t* dw_post, uint16_t* dgate, uint16_t* dw_pre, void* ws,
                            size_t ws_bytes, hipStream_t stream) {
  int st = check_norm_operands(y, M, d, type, post_norm, w_post, gate, gate_rows, w_pre, res_scale, eps);
  if (st) return st;
  if ((!dh && !dx_out) || (dh && !x_out) || (w_pre && !dh)) return QLORA_ERR_INVALID_ARG;
  if (!dx && !dy && !dw_post && !dgate && !dw_pre) return QLORA_ERR_INVALID_ARG;
  if (((dy || dw_post || dgate) && !y) || (dw_post && !post_norm) || (dgate && !gate) || (dw_pre && !dh))
    return QLORA_ERR_INVALID_ARG;
  for (const void* p : {x_out, dx_out, (const void*)dx})
    if (!aligned(p, type_bytes(type))) return QLORA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)dh, (const void*)dy, (const void*)dw_post, (const void*)dgate, (const void*)dw_pre})
    if (!aligned(p, 2)) return QLORA_ERR_INVALID_ARG;
  const NormSegments seg = norm_segments(M, d, gate ? gate_rows : 0);
  if ((st = check_ws(ws, ws_bytes, kHead + 3 * sizeof(float) * (size_t)(seg.count * d)))) return st;
  NormBwd p{};
  p.x = x_out, p.y = y, p.dh = dh, p.dx_out = dx_out;
  p.w_post = w_post, p.gate = gate, p.w_pre = w_pre;
  p.dx = dx, p.dy = dy, p.dw_post = dw_post, p.dgate = dgate, p.dw_pre = dw_pre;
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + kHead);
  p.counter = static_cast<unsigned int*>(ws);
  p.M = M, p.d = d, p.gate_rows = gate ? std::min(gate_rows, M) : 1;
  p.scale = res_scale, p.eps = eps, p.f32 = type == QLORA_F32, p.post = post_norm != 0;
  return hip_status(launch_norm_bwd(p, stream));
}

int qlora_logps_workspace_size(int64_t rows, int64_t V, size_t* ws_bytes) {
  if (!ws_bytes || rows < 1 || rows >= kMaxRows) return QLORA_ERR_INVALID_ARG;
  if (V < 1 || V > kMaxVocab) return QLORA_ERR_BAD_SHAPE;
  *ws_bytes = carve_stats(nullptr, rows, V, 0, nullptr);
  return QLORA_OK;
}

int qlora_token_logps(const void* logits, const int64_t* labels, int64_t rows, int64_t V, int type, float* logps,
                      void* ws, size_t ws_bytes, hipStream_t stream) {
  int st = check_logits(logits, labels, rows, V, type);
  if (st) return st;
  if (!logps || !aligned(logps, 4)) return QLORA_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, carve_stats(nullptr, rows, V, 0, nullptr)))) return st;
  RowStats s;
  carve_stats(ws, rows, V, 0, &s);
  return hip_status(launch_token_logps(logits, labels, rows, V, type == QLORA_F32, logps, s, stream));
}

int qlora_preference_workspace_size(int64_t pairs, int64_t S, int64_t V, size_t* ws_bytes) {
  if (!ws_bytes || pairs < 1 || S < 1 || pairs >= kMaxRows / 4 || S >= kMaxRows || 2 * pairs * S >= kMaxRows)
    return QLORA_ERR_INVALID_ARG;
  if (V < 1 || V > kMaxVocab) return QLORA_ERR_BAD_SHAPE;
  *ws_bytes = carve_stats(nullptr, 2 * pairs * S, V, pairs, nullptr);
  return QLORA_OK;
}

int qlora_preference_loss(const void* logits, const int64_t* labels, const float* ref_logps, int64_t pairs,
                          int64_t S, int64_t V, int type, float beta, float label_smoothing, float grad_scale,
                          float* loss, float* log_ratios, float* logps, void* dlogits, void* ws, size_t ws_bytes,
                          hipStream_t stream) {
  if (pairs < 1 || S < 1 || pairs >= kMaxRows / 4 || S >= kMaxRows) return QLORA_ERR_INVALID_ARG;
  const int64_t rows = 2 * pairs * S;
  int st = check_logits(logits, labels, rows, V, type);
  if (st) return st;
  if (!std::isfinite(beta) || !std::isfinite(grad_scale) || !(label_smoothing >= 0.f && label_smoothing <= 1.f))
    return QLORA_ERR_INVALID_ARG;
  if (!loss || !log_ratios || !logps) return QLORA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)ref_logps, (const void*)loss, (const void*)log_ratios, (const void*)logps})
    if (!aligned(p, 4)) return QLORA_ERR_INVALID_ARG;
  if (dlogits && dlogits != logits) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(logits), b = reinterpret_cast<uintptr_t>(dlogits);
    const uintptr_t bytes = (uintptr_t)rows * (uintptr_t)V * type_bytes(type);
    if (!aligned(dlogits, type_bytes(type)) || (a < b ? b - a : a - b) < bytes) return QLORA_ERR_INVALID_ARG;
  }
  if ((st = check_ws(ws, ws_bytes, carve_stats(nullptr, rows, V, pairs, nullptr)))) return st;
  RowStats s;
  carve_stats(ws, rows, V, pairs, &s);
  return hip_status(launch_preference(Preference{logits, labels, ref_logps, pairs, S, V, beta, label_smoothing,
                                                 grad_scale, loss, log_ratios, logps, dlogits, type == QLORA_F32},
                                      s, stream));
}

int qlora_gradlist_size(int count, const int64_t* numel, size_t* table_bytes) {
  if (!table_bytes) return QLORA_ERR_INVALID_ARG;
  int64_t chunks = 0;
  const int st = count_chunks(count, numel, &chunks);
  if (st) return st;
  *table_bytes = sizeof(GradChunk) * (size_t)chunks;
  return QLORA_OK;
}

int qlora_gradlist_init(int count, const void* const* grads, const int32_t* types, const int64_t* numel,
                        void* const* out, const int32_t* out_types, void* table, size_t table_bytes,
                        qlora_gradlist_t* list, hipStream_t stream) {
  int64_t chunks = 0;
  const int st = count_chunks(count, numel, &chunks);
  if (st) return st;
  if (!list || (count && (!grads || !types || (out && !out_types)))) return QLORA_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    const int32_t to = out ? out_types[i] : types[i];
    if (!type_ok(types[i]) || !type_ok(to)) return QLORA_ERR_UNSUPPORTED;
    if (!numel[i]) continue;
    const void* o = out ? out[i] : grads[i];
    if (!grads[i] || !o || !aligned(grads[i], type_bytes(types[i])) || !aligned(o, type_bytes(to)) ||
        (o == grads[i] && to != types[i]))
      return QLORA_ERR_INVALID_ARG;
  }
  if (chunks && (!table || table_bytes < sizeof(GradChunk) * (size_t)chunks)) return QLORA_ERR_WORKSPACE;
  if (!aligned(table, 16)) return QLORA_ERR_INVALID_ARG;
  int64_t first = 0;
  GradTensors batch;
  int n = 0;
  for (int i = 0; i < count; ++i) {
    if (numel[i]) {
      batch.t[n++] = GradTensor{grads[i], out ? out[i] : const_cast<void*>(grads[i]), numel[i], first,
                                types[i] == QLORA_F32, (out ? out_types[i] : types[i]) == QLORA_F32};
      first += (numel[i] + kGradChunk - 1) / kGradChunk;
    }
    if (n && (n == kGradBatch || i + 1 == count)) {
      if (launch_grad_table(batch, n, static_cast<GradChunk*>(table), stream) != hipSuccess) return QLORA_ERR_HIP;
      n = 0;
    }
  }
  list->table = table;
  list->chunks = chunks;
  return QLORA_OK;
}

int qlora_grad_workspace_size(const qlora_gradlist_t* list, size_t* ws_bytes) {
  const int st = check_list(list);
  if (st || !ws_bytes) return QLORA_ERR_INVALID_ARG;
  *ws_bytes = grad_ws_bytes(list->chunks);
  return QLORA_OK;
}

int qlora_grad_norm(const qlora_gradlist_t* list, float* norm, void* ws, size_t ws_bytes, hipStream_t stream) {
  int st = check_list(list);
  if (st) return st;
  if (!norm || !aligned(norm, 4)) return QLORA_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, grad_ws_bytes(list->chunks)))) return st;
  return hip_status(launch_grad_norm(static_cast<const GradChunk*>(list->table), list->chunks, norm,
                                     reinterpret_cast<double*>(static_cast<char*>(ws) + kHead),
                                     static_cast<unsigned int*>(ws), stream));
}

int qlora_grad_clip(const qlora_gradlist_t* list, float max_norm, float* norm, void* ws, size_t ws_bytes,
                    hipStream_t stream) {
  if (!std::isfinite(max_norm) || max_norm < 0.f) return QLORA_ERR_INVALID_ARG;
  const int st = qlora_grad_norm(list, norm, ws, ws_bytes, stream);
  if (st || !list->chunks) return st;
  return hip_status(
      launch_grad_clip(static_cast<const GradChunk*>(list->table), list->chunks, norm, max_norm, stream));
}

int qlora_adamw_step_clipped(float* master, float* m, float* v, const uint16_t* grad, uint16_t* param, int64_t n,
                             int64_t step, float lr, float beta1, float beta2, float eps, float weight_decay,
                             const float* norm, float max_norm, hipStream_t stream) {
  if (!std::isfinite(max_norm) || max_norm < 0.f) return QLORA_ERR_INVALID_ARG;
  AdamWScalars a;
  const int st = adamw_prepare(master, m, v, grad, param, n, step, lr, beta1, beta2, eps, weight_decay, &a);
  if (st || n == 0) return st;
  if (!norm || !aligned(norm, 4)) return QLORA_ERR_INVALID_ARG;
  return hip_status(launch_adamw_clipped(master, m, v, grad, param, n, a, norm, max_norm, stream));
}

}  // extern "C"
