// Drives the host code of the training-step entry points (include/qlora_train.h) under
// AddressSanitizer and UndefinedBehaviorSanitizer, against the host-only runtime stand-in: no
// kernel runs, every launch is checked against the hardware's limits.  Device pointers are
// addresses that nothing here reads.  The last line of output is "OK <checks>".
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "qlora_train.h"
#include "sim_runtime.h"

namespace {

int g_checks = 0;
#define CHECK(cond, ...)                                  \
  do {                                                    \
    ++g_checks;                                           \
    if (!(cond)) {                                        \
      std::printf("FAIL line %d: %s: ", __LINE__, #cond); \
      std::printf(__VA_ARGS__);                           \
      std::printf("\n");                                  \
      std::exit(1);                                       \
    }                                                     \
  } while (0)

template <class T>
T* at(uintptr_t slot) { return reinterpret_cast<T*>((uintptr_t(1) << 46) + (slot << 42)); }

// Runs `call` and checks its status, its launches' limits and their number.
template <class F>
void run(F call, size_t launches, const char* what, long long a, long long b) {
  const size_t before = sim::launches();
  const int st = call();
  CHECK(st == QLORA_OK, "%s %lld %lld -> %d", what, a, b, st);
  CHECK(sim::bad_launches() == 0, "%s %lld %lld: launch limits", what, a, b);
  CHECK(sim::launches() - before == launches, "%s %lld %lld: %zu launches", what, a, b, sim::launches() - before);
}

void norms() {
  const int64_t most = (int64_t(1) << 24) - 1;
  for (int64_t M : {int64_t(1), int64_t(3), int64_t(777), int64_t(8192), most})
    for (int64_t d : {int64_t(1), int64_t(9), int64_t(513), int64_t(4096), int64_t(8192)})
      for (int64_t rows : {int64_t(0), int64_t(1), int64_t(5), int64_t(300), M, int64_t(1) << 40})
        for (int type : {QLORA_BF16, QLORA_F32}) {
          const uint16_t* gate = rows ? at<uint16_t>(1) : nullptr;
          uint16_t* dgate = rows ? at<uint16_t>(2) : nullptr;
          run([&] {
            return qlora_norm_residual_fwd(at<void>(3), at<uint16_t>(4), M, d, type, 1, at<uint16_t>(5), gate, rows,
                                           at<uint16_t>(6), 1.f, 1e-5f, at<void>(7), at<uint16_t>(8), nullptr);
          }, 1, "norm fwd", M, d);
          size_t need = 0;
          CHECK(qlora_norm_residual_workspace_size(M, d, rows, &need) == QLORA_OK, "size %lld %lld", (long long)M, (long long)d);
          const auto bwd = [&](size_t bytes) {
            return qlora_norm_residual_bwd(at<void>(3), at<uint16_t>(4), at<uint16_t>(9), at<void>(10), M, d, type, 1,
                                           at<uint16_t>(5), gate, rows, at<uint16_t>(6), 1.f, 1e-5f, at<void>(11),
                                           at<uint16_t>(12), at<uint16_t>(13), dgate, at<uint16_t>(14), at<void>(15), bytes,
                                           nullptr);
          };
          // few partials are added by the first launch itself
          const size_t partials = need - QLORA_WS_COUNTER_BYTES, segments = partials / (12 * d);
          run([&] { return bwd(need); }, segments <= 32 && partials <= 262144 ? 1 : 2, "norm bwd", M, d);
          CHECK(bwd(need - 1) == QLORA_ERR_WORKSPACE, "short workspace");
        }
}

void losses() {
  const int64_t most = (int64_t(1) << 23) - 1;
  struct { int64_t pairs, S; } shapes[] = {{1, 1}, {1, 33}, {4, 512}, {1, most}, {most / 2, 1}};
  for (auto [pairs, S] : shapes)
    for (int64_t V : {int64_t(1), int64_t(7), int64_t(1003), int64_t(131072), int64_t(1) << 22})
      for (int type : {QLORA_BF16, QLORA_F32}) {
        if (pairs >= int64_t(1) << 22) continue;
        size_t need = 0;
        CHECK(qlora_preference_workspace_size(pairs, S, V, &need) == QLORA_OK, "size");
        for (int grad = 0; grad < 2; ++grad) {
          const auto call = [&](size_t bytes) {
            return qlora_preference_loss(at<void>(1), at<int64_t>(2), at<float>(3), pairs, S, V, type, 0.1f, 0.f, 1.f,
                                         at<float>(4), at<float>(5), at<float>(6), grad ? at<void>(100) : nullptr,
                                         at<void>(8), bytes, nullptr);
          };
          run([&] { return call(need); }, 2, "preference", pairs * S, V);
          CHECK(call(need - 256) == QLORA_ERR_WORKSPACE, "short workspace");
        }
        const int64_t rows = 2 * pairs * S;
        CHECK(qlora_logps_workspace_size(rows, V, &need) == QLORA_OK, "size");
        const size_t launches = rows >= 128 || V < 2 * 8192 ? 1 : 2;
        run([&] {
          return qlora_token_logps(at<void>(1), at<int64_t>(2), rows, V, type, at<float>(3), at<void>(8), need, nullptr);
        }, launches, "logps", rows, V);
      }
}

void gradients() {
  for (int count : {0, 1, 95, 96, 97, 112, 448}) {
    std::vector<const void*> in(count);
    std::vector<void*> out(count);
    std::vector<int32_t> types(count), out_types(count);
    std::vector<int64_t> numel(count);
    int full = 0;
    for (int i = 0; i < count; ++i) {
      in[i] = at<void>(1 + i);
      out[i] = at<void>(1000 + i);
      types[i] = i % 2;
      out_types[i] = i % 3 == 0;
      numel[i] = i % 7 == 3 ? 0 : int64_t(1) << (i % 30);
      full += numel[i] != 0;
      if (!numel[i]) in[i] = out[i] = nullptr;
    }
    size_t bytes = 0;
    CHECK(qlora_gradlist_size(count, numel.data(), &bytes) == QLORA_OK, "size of %d", count);
    qlora_gradlist_t list{};
    for (int place = 0; place < 2; ++place) {
      run([&] {
        return qlora_gradlist_init(count, in.data(), types.data(), numel.data(), place ? nullptr : out.data(),
                                   place ? nullptr : out_types.data(), at<void>(3000), bytes, &list, nullptr);
      }, (size_t)(full + 95) / 96, "list", count, place);
      CHECK((size_t)list.chunks * 24 == bytes, "chunks");
      size_t ws = 0;
      CHECK(qlora_grad_workspace_size(&list, &ws) == QLORA_OK, "workspace");
      run([&] { return qlora_grad_norm(&list, at<float>(1), at<void>(2), ws, nullptr); }, 1, "norm", count, place);
      run([&] { return qlora_grad_clip(&list, 1.f, at<float>(1), at<void>(2), ws, nullptr); }, count ? 2 : 1, "clip", count,
          place);
      CHECK(qlora_grad_norm(&list, at<float>(1), at<void>(2), ws - 1, nullptr) == QLORA_ERR_WORKSPACE, "short");
    }
  }
  qlora_gradlist_t most{at<void>(1), (int64_t(1) << 24) - 1};
  size_t ws = 0;
  CHECK(qlora_grad_workspace_size(&most, &ws) == QLORA_OK, "workspace");
  run([&] { return qlora_grad_clip(&most, 1.f, at<float>(1), at<void>(2), ws, nullptr); }, 2, "clip", 0, 0);
  for (int64_t n : {int64_t(1), int64_t(1000003), int64_t(1) << 36})
    run([&] {
      return qlora_adamw_step_clipped(at<float>(1), at<float>(2), at<float>(3), at<uint16_t>(4), at<uint16_t>(5), n, 3, 1e-3f,
                                      0.9f, 0.999f, 1e-8f, 0.f, at<float>(6), 1.f, nullptr);
    }, 1, "adamw", n, 0);
}

}  // namespace

int main() {
  norms();
  losses();
  gradients();
  std::printf("OK %d\n", g_checks);
  return 0;
}
