// C ABI of the frozen linear with many adapters and of dropout (declared in
// include/qlora_adapters.h): argument checks, workspace layouts and plans; the kernels and their
// launches are in adapters.hip, adapters_gemm.hip, gemm_nt.hip and dropout.hip.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "qlora_adapters_host.h"

using namespace qlora;

namespace {

constexpr size_t kHead = QLORA_WS_COUNTER_BYTES;
constexpr int64_t kMaxRows = int64_t(1) << 23;
constexpr int64_t kMaxDropout = int64_t(1) << 40;

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
// Two ranges of memory that share no byte.
inline bool apart(const void* p, size_t bytes, const void* q, size_t other) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a + bytes <= b || b + other <= a;
}
struct Range {
  const void* p;
  size_t bytes;
};
// `out` shares no byte with any of `with` (null ranges are none).
inline bool apart_from(const Range& out, std::initializer_list<Range> with) {
  for (const Range& r : with)
    if (out.p && r.p && !apart(out.p, out.bytes, r.p, r.bytes)) return false;
  return true;
}
int hip_status(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP; }
inline bool type_ok(int type) { return type == QLORA_BF16 || type == QLORA_F32; }
inline size_t type_bytes(int type) { return type == QLORA_F32 ? 4 : 2; }
inline int32_t width_of(const qlora_adapters_t* set) { return (set->max_rank + 7) / 8 * 8; }

int check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws || ws_bytes < need) return QLORA_ERR_WORKSPACE;
  return aligned(ws, 16) ? QLORA_OK : QLORA_ERR_INVALID_ARG;
}

int check_set(const qlora_adapters_t* set) {
  if (!set || set->count < 1 || set->count > QLORA_MAX_ADAPTERS || set->max_rank < 1 || set->max_rank > 128)
    return QLORA_ERR_INVALID_ARG;
  return linear_shape_ok(set->d_out, set->d_in) ? QLORA_OK : QLORA_ERR_BAD_SHAPE;
}

int check_dropout(float p, const uint64_t* rng, DropMask* mask) {
  if (!(p >= 0.f && p < 1.f)) return QLORA_ERR_INVALID_ARG;
  const uint32_t threshold = (uint32_t)std::floor((double)p * 65536.0 + 0.5);
  if (threshold > 65535u) return QLORA_ERR_INVALID_ARG;
  if (p > 0.f && (!rng || !aligned(rng, 8))) return QLORA_ERR_INVALID_ARG;
  *mask = DropMask{rng, threshold, (float)(65536.0 / (65536.0 - (double)threshold))};
  return QLORA_OK;
}

int check_call(const qlora_nf4dq_t* Wq, const qlora_adapters_t* set, int64_t M, const int32_t* ids, float dropout,
               const uint64_t* rng, DropMask* mask) {
  int st;
  if ((st = check_weight(Wq)) || (st = check_set(set))) return st;
  if (!set->table || !aligned(set->table, 16)) return QLORA_ERR_INVALID_ARG;
  if (Wq->d_out != set->d_out || Wq->d_in != set->d_in) return QLORA_ERR_BAD_SHAPE;
  if (M < 1 || M > kMaxRows || !aligned(ids, 4)) return QLORA_ERR_INVALID_ARG;
  return check_dropout(dropout, rng, mask);
}

AdapterRows rows_of(const qlora_adapters_t* set, const int32_t* ids, int64_t M) {
  return AdapterRows{static_cast<const AdapterEntry*>(set->table), ids, M, set->count, set->max_rank, width_of(set), set->whole};
}

// Few rows read the weight's codes as they are; more (and formats that only the decode kernels
// read) go through the decoded copy.
bool stream_path(int64_t M, int64_t N, int64_t K, int dq) { return dq == QLORA_DQ_E4M3 && adapter_stream_fits(M, N, K); }
// The product over the codes, for the rows between few and many.
bool codes_path(int64_t M, int64_t F, int64_t Kr, int dq) { return dq == QLORA_DQ_E4M3 && adapter_gemm_fits(M, F, Kr); }

// ---- workspaces: the counter head, then T and G, then what the steps need in turn
struct Layout {
  size_t t, g, spart, gspart, wcopy, gpart, grads, total;
  int32_t gsplit;
};
Layout layout(bool bwd, int64_t M, const qlora_adapters_t* set, int dq) {
  const int64_t N = set->d_out, K = set->d_in, width = width_of(set);
  Layout w{};
  size_t off = kHead;
  const auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  const size_t t_bytes = sizeof(float) * (size_t)M * width;
  w.t = take(t_bytes);
  if (bwd) w.g = take(t_bytes);
  if (bwd || !stream_path(M, N, K, dq)) {
    const int32_t t_split = shrink_split(M, K), g_split = shrink_split(M, N);
    w.spart = take(t_split > 1 ? t_bytes * t_split : 0);
    if (bwd) w.gspart = take(g_split > 1 ? t_bytes * g_split : 0);
    const int64_t F = bwd ? K : N, Kr = bwd ? N : K;
    if (!codes_path(M, F, Kr, dq)) w.wcopy = take(2 * (size_t)N * K);
    w.gsplit = codes_path(M, F, Kr, dq) ? adapter_gemm_split(M, F, Kr) : gemm_nt_ksplit(F, M, Kr);
    w.gpart = take(w.gsplit > 1 ? sizeof(float) * (size_t)w.gsplit * M * F : 0);
  }
  if (bwd) w.grads = take(adapter_grad_plan(M, N, K, set->count, set->max_rank).part_bytes);
  w.total = off;
  return w;
}

// The weight's decode joins the launch of T or G where its kernels read the format.
ShrinkDecode decode_args(const qlora_nf4dq_t* Wq, uint16_t* out) {
  return ShrinkDecode{reinterpret_cast<const uint32_t*>(Wq->codes), Wq->code8, Wq->c2s, Wq->mu, out, Wq->d_out, Wq->d_in};
}

}  // namespace

extern "C" {

int qlora_adapters_size(int count, size_t* table_bytes) {
  if (!table_bytes || count < 1 || count > QLORA_MAX_ADAPTERS) return QLORA_ERR_INVALID_ARG;
  *table_bytes = sizeof(AdapterEntry) * (size_t)count;
  return QLORA_OK;
}

int qlora_adapters_init(int count, const uint16_t* const* A, const uint16_t* const* B, const int32_t* r,
                        const float* alpha, uint16_t* const* dA, uint16_t* const* dB, int64_t d_out, int64_t d_in,
                        void* table, size_t table_bytes, qlora_adapters_t* set, hipStream_t stream) {
  size_t need = 0;
  int st = qlora_adapters_size(count, &need);
  if (st) return st;
  if (!A || !B || !r || !alpha || !set || (dA == nullptr) != (dB == nullptr)) return QLORA_ERR_INVALID_ARG;
  if (!linear_shape_ok(d_out, d_in)) return QLORA_ERR_BAD_SHAPE;
  qlora_adapters_t out{table, d_out, d_in, count, 0, 1, dA != nullptr};
  for (int i = 0; i < count; ++i) {
    if (r[i] < 1 || r[i] > 128 || !std::isfinite(alpha[i])) return QLORA_ERR_INVALID_ARG;
    if (!A[i] || !B[i] || !aligned(A[i], 16) || !aligned(B[i], r[i] % 8 ? 2 : 16)) return QLORA_ERR_INVALID_ARG;
    if (dA && (!dA[i] || !dB[i] || !aligned(dA[i], 2) || !aligned(dB[i], 2))) return QLORA_ERR_INVALID_ARG;
    out.max_rank = std::max(out.max_rank, r[i]);
    if (r[i] % 8) out.whole = 0;
  }
  if ((st = check_ws(table, table_bytes, need))) return st;
  AdapterBatch batch;
  for (int first = 0; first < count; first += kAdapterBatch) {
    const int n = std::min(count - first, kAdapterBatch);
    for (int i = 0; i < n; ++i) {
      const int k = first + i;
      batch.e[i] = AdapterEntry{A[k], B[k], dA ? dA[k] : nullptr, dB ? dB[k] : nullptr, r[k], alpha[k] / (float)r[k]};
    }
    if (launch_adapter_table(batch, n, static_cast<AdapterEntry*>(table) + first, stream) != hipSuccess) return QLORA_ERR_HIP;
  }
  *set = out;
  return QLORA_OK;
}

int qlora_adapters_t_width(const qlora_adapters_t* set, int64_t* width) {
  const int st = check_set(set);
  if (st) return st;
  if (!width) return QLORA_ERR_INVALID_ARG;
  *width = width_of(set);
  return QLORA_OK;
}

int qlora_adapters_workspace_size(int op, int64_t M, const qlora_adapters_t* set, int dq_format, size_t* ws_bytes) {
  if (!ws_bytes || (op != QLORA_OP_FWD && op != QLORA_OP_BWD)) return QLORA_ERR_INVALID_ARG;
  const int st = check_set(set);
  if (st) return st;
  if (M < 1 || M > kMaxRows) return QLORA_ERR_INVALID_ARG;
  if (dq_format < QLORA_DQ_E4M3 || dq_format > QLORA_DQ_NONE) return QLORA_ERR_UNSUPPORTED;
  *ws_bytes = layout(op == QLORA_OP_BWD, M, set, dq_format).total;
  return QLORA_OK;
}

int qlora_adapters_fwd(const qlora_nf4dq_t* Wq, const qlora_adapters_t* set, const uint16_t* X, int64_t M,
                       const int32_t* ids, float dropout, const uint64_t* rng, uint16_t* Y, float* T_save, void* ws,
                       size_t ws_bytes, hipStream_t stream) {
  DropMask drop;
  int st = check_call(Wq, set, M, ids, dropout, rng, &drop);
  if (st) return st;
  if (!X || !Y || !aligned(X, 16) || !aligned(Y, 16) || !aligned(T_save, 16)) return QLORA_ERR_INVALID_ARG;
  const Range x{X, 2 * (size_t)M * Wq->d_in}, y{Y, 2 * (size_t)M * Wq->d_out}, t{T_save, sizeof(float) * (size_t)M * width_of(set)};
  const Range id{ids, sizeof(int32_t) * (size_t)M}, words{drop.threshold ? rng : nullptr, 2 * sizeof(uint64_t)};
  if (!apart_from(y, {x, id, words}) || !apart_from(t, {x, y, id, words})) return QLORA_ERR_INVALID_ARG;
  const int dq = Wq->dq_format;
  const Layout L = layout(false, M, set, dq);
  if ((st = check_ws(ws, ws_bytes, L.total))) return st;
  char* base = static_cast<char*>(ws);
  const int64_t N = Wq->d_out, K = Wq->d_in;
  const AdapterRows rows = rows_of(set, ids, M);
  const Nf4Tables& tab = weight_tables(Wq);
  float* T = T_save ? T_save : reinterpret_cast<float*>(base + L.t);
  float* part = reinterpret_cast<float*>(base + L.spart);
  unsigned int* counters = static_cast<unsigned int*>(ws);
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(Wq->codes);
  if (stream_path(M, N, K, dq))
    return hip_status(launch_adapter_stream(codes, Wq->code8, Wq->c2s, Wq->mu, N, K, X, rows, drop,
                                            stream_forms_t(M, N, rows.width) ? T_save : T, Y, ws, posted_polls(), tab, stream));
  const AdapterHead head{rows, T, 0, 1.f, DropMask{}};
  float* gpart = reinterpret_cast<float*>(base + L.gpart);
  if (codes_path(M, N, K, dq)) {
    if (launch_shrink_a(rows, X, K, drop, T, part, counters, nullptr, tab, stream) != hipSuccess) return QLORA_ERR_HIP;
    return hip_status(launch_adapter_gemm(codes, Wq->code8, Wq->c2s, Wq->mu, N, K, X, M, head, Y, gpart, L.gsplit, tab,
                                          QLORA_K_GEMM_FWD, stream));
  }
  uint16_t* wcopy = reinterpret_cast<uint16_t*>(base + L.wcopy);
  const ShrinkDecode dec = decode_args(Wq, wcopy);
  if (launch_shrink_a(rows, X, K, drop, T, part, counters, dq == QLORA_DQ_E4M3 ? &dec : nullptr, tab, stream) != hipSuccess)
    return QLORA_ERR_HIP;
  if (dq != QLORA_DQ_E4M3 &&
      launch_dequant(codes, Wq->code8, Wq->c2s, Wq->mu, wcopy, N * K / 8, tab, dq, stream) != hipSuccess)
    return QLORA_ERR_HIP;
  return hip_status(launch_gemm_nt_adapters(wcopy, N, X, M, K, head, Y, QLORA_K_GEMM_FWD, stream, gpart, L.gsplit));
}

int qlora_adapters_bwd(const qlora_nf4dq_t* Wq, const qlora_adapters_t* set, const uint16_t* X, const uint16_t* dY,
                       int64_t M, const int32_t* ids, float dropout, const uint64_t* rng, const float* T_saved,
                       uint16_t* dX, void* ws, size_t ws_bytes, hipStream_t stream) {
  DropMask drop;
  int st = check_call(Wq, set, M, ids, dropout, rng, &drop);
  if (st) return st;
  if (!set->grads) return QLORA_ERR_INVALID_ARG;
  if (!X || !dY || !aligned(X, 16) || !aligned(dY, 16) || !aligned(dX, 16) || !aligned(T_saved, 16))
    return QLORA_ERR_INVALID_ARG;
  const size_t x_bytes = 2 * (size_t)M * Wq->d_in;
  if (!apart_from({dX, x_bytes}, {{X, x_bytes}, {dY, 2 * (size_t)M * Wq->d_out}, {T_saved, sizeof(float) * (size_t)M * width_of(set)},
                                  {ids, sizeof(int32_t) * (size_t)M}, {drop.threshold ? rng : nullptr, 2 * sizeof(uint64_t)}}))
    return QLORA_ERR_INVALID_ARG;
  const int dq = Wq->dq_format;
  const Layout L = layout(true, M, set, dq);
  if ((st = check_ws(ws, ws_bytes, L.total))) return st;
  char* base = static_cast<char*>(ws);
  const int64_t N = Wq->d_out, K = Wq->d_in;
  const AdapterRows rows = rows_of(set, ids, M);
  const Nf4Tables& tab = weight_tables(Wq);
  float* G = reinterpret_cast<float*>(base + L.g);
  float* part = reinterpret_cast<float*>(base + L.spart);
  unsigned int* counters = static_cast<unsigned int*>(ws);
  float* g_part = reinterpret_cast<float*>(base + L.gspart);
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(Wq->codes);
  uint16_t* wcopy = reinterpret_cast<uint16_t*>(base + L.wcopy);
  const bool copied = dX && !codes_path(M, K, N, dq);
  const bool beside = copied && dq == QLORA_DQ_E4M3;  // the decode joins G's launch
  const ShrinkDecode dec = decode_args(Wq, wcopy);
  const float* T = T_saved;
  hipError_t e;
  if (!T && !beside) {
    float* t = reinterpret_cast<float*>(base + L.t);
    e = launch_shrink_both(rows, X, K, drop, t, dY, N, G, part, g_part, counters, stream);
    T = t;
  } else {
    if (!T) {
      float* t = reinterpret_cast<float*>(base + L.t);
      if (launch_shrink_a(rows, X, K, drop, t, part, counters, nullptr, tab, stream) != hipSuccess) return QLORA_ERR_HIP;
      T = t;
    }
    e = launch_shrink_b(rows, dY, N, G, g_part, counters, beside ? &dec : nullptr, tab, stream);
  }
  if (e != hipSuccess) return QLORA_ERR_HIP;
  if (dX) {
    if (copied && dq != QLORA_DQ_E4M3 &&
        launch_dequant_t(codes, Wq->code8, Wq->c2s, Wq->mu, N, K, wcopy, tab, dq, stream) != hipSuccess)
      return QLORA_ERR_HIP;
    const AdapterHead head{rows, G, 1, drop.scale, drop};
    float* gpart = reinterpret_cast<float*>(base + L.gpart);
    e = copied ? launch_gemm_nt_adapters(wcopy, K, dY, M, N, head, dX, QLORA_K_GEMM_DX, stream, gpart, L.gsplit)
               : launch_adapter_gemm(codes, Wq->code8, Wq->c2s, Wq->mu, N, K, dY, M, head, dX, gpart, L.gsplit, tab,
                                     QLORA_K_GEMM_DX, stream);
    if (e != hipSuccess) return QLORA_ERR_HIP;
  }
  return hip_status(launch_adapter_grads(rows, X, K, dY, N, T, G, drop, reinterpret_cast<float*>(base + L.grads), counters,
                                         stream));
}

int qlora_dropout(const void* x, int x_type, int64_t n, float dropout, const uint64_t* rng, const void* residual,
                  void* out, int out_type, hipStream_t stream) {
  if (!type_ok(x_type) || !type_ok(out_type)) return QLORA_ERR_UNSUPPORTED;
  DropMask drop;
  const int st = check_dropout(dropout, rng, &drop);
  if (st) return st;
  if (n < 0 || n > kMaxDropout) return QLORA_ERR_INVALID_ARG;
  if (n == 0) return QLORA_OK;
  const size_t xb = type_bytes(x_type), ob = type_bytes(out_type);
  if (!x || !out || !aligned(x, xb) || !aligned(out, ob) || !aligned(residual, ob)) return QLORA_ERR_INVALID_ARG;
  // an operand is out itself, element for element, or shares no byte with it
  const auto separate = [&](const void* p, size_t bytes) {
    return (p == out && bytes == ob) || apart(p, (size_t)n * bytes, out, (size_t)n * ob);
  };
  if (!separate(x, xb) || (residual && !separate(residual, ob))) return QLORA_ERR_INVALID_ARG;
  if (drop.threshold && !apart(rng, 2 * sizeof(uint64_t), out, (size_t)n * ob)) return QLORA_ERR_INVALID_ARG;
  return hip_status(launch_dropout(x, x_type == QLORA_F32, n, drop, residual, out, out_type == QLORA_F32, stream));
}

}  // extern "C"
