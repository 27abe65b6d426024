// Drives the host code of the adapters' and dropout's entry points (include/qlora_adapters.h)
// under AddressSanitizer and UndefinedBehaviorSanitizer, against the host-only runtime stand-in:
// no kernel runs, every launch is checked against the hardware's limits.  Device pointers are
// addresses that nothing here reads.  The last line of output is "OK <checks>".
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "qlora_adapters.h"
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

// Runs `call` and checks its status, its launches' limits and that their number is in [least, most].
template <class F>
void run(F call, size_t least, size_t most, const char* what, long long a, long long b, long long c) {
  const size_t before = sim::launches();
  const int st = call();
  const size_t n = sim::launches() - before;
  CHECK(st == QLORA_OK, "%s %lld %lld %lld -> %d", what, a, b, c, st);
  CHECK(sim::bad_launches() == 0, "%s %lld %lld %lld: launch limits", what, a, b, c);
  CHECK(n >= least && n <= most, "%s %lld %lld %lld: %zu launches", what, a, b, c, n);
}

void tables() {
  for (int count : {1, 2, 95, 96, 97, 192, 193, 4096}) {
    std::vector<uint16_t*> a(count), b(count), da(count), db(count);
    std::vector<int32_t> r(count);
    std::vector<float> alpha(count);
    int most = 0, whole = 1;
    for (int i = 0; i < count; ++i) {
      a[i] = at<uint16_t>(1) + 8 * i, b[i] = at<uint16_t>(2) + 8 * i;
      da[i] = at<uint16_t>(3) + i, db[i] = at<uint16_t>(4) + i;
      r[i] = count < 3 ? 8 : 1 + (i * 37) % 128;
      alpha[i] = 1.f + i;
      most = std::max(most, r[i]), whole &= r[i] % 8 == 0;
    }
    size_t bytes = 0;
    CHECK(qlora_adapters_size(count, &bytes) == QLORA_OK, "size of %d", count);
    for (int grads = 0; grads < 2; ++grads) {
      qlora_adapters_t set{};
      const auto init = [&](size_t given) {
        return qlora_adapters_init(count, a.data(), b.data(), r.data(), alpha.data(), grads ? da.data() : nullptr,
                                   grads ? db.data() : nullptr, 64, 128, at<void>(5), given, &set, nullptr);
      };
      CHECK(init(bytes - 1) == QLORA_ERR_WORKSPACE, "short table");
      run([&] { return init(bytes); }, (count + 95) / 96, (count + 95) / 96, "init", count, grads, 0);
      CHECK(set.count == count && set.max_rank == most && set.whole == whole && set.grads == grads, "set of %d", count);
    }
  }
}

void linears() {
  const int64_t top = int64_t(1) << 23;
  struct { int64_t N, K; } shapes[] = {{16, 64}, {48, 4160}, {4096, 4096}, {8208, 192}, {14336, 4096}, {4096, 14336}, {131072, 8192}};
  struct { int32_t count, rank; } sets[] = {{1, 1}, {1, 16}, {2, 32}, {48, 16}, {300, 128}, {4096, 128}};
  for (auto [N, K] : shapes)
    for (auto [count, rank] : sets)
      for (int64_t M : {int64_t(1), int64_t(2), int64_t(16), int64_t(17), int64_t(128), int64_t(129), int64_t(520), int64_t(4096),
                        int64_t(4097), int64_t(100000), top})
        for (int dq = 0; dq < 4; ++dq)
          for (float p : {0.f, 0.1f}) {
            // operands lie 4 TiB apart here; the larger ones would reach the next
            if (2 * M * std::max(N, K) > int64_t(1) << 41) continue;
            const qlora_nf4dq_t q{at<uint8_t>(1), at<uint8_t>(2), at<float>(3), at<float>(4), N, K, 64, 256, 0, dq};
            const qlora_adapters_t set{at<void>(5), N, K, count, rank, rank % 8 == 0, 1};
            size_t fw = 0, bw = 0;
            CHECK(qlora_adapters_workspace_size(QLORA_OP_FWD, M, &set, dq, &fw) == QLORA_OK, "size");
            CHECK(qlora_adapters_workspace_size(QLORA_OP_BWD, M, &set, dq, &bw) == QLORA_OK, "size");
            const auto fwd = [&](size_t bytes, bool save) {
              return qlora_adapters_fwd(&q, &set, at<uint16_t>(6), M, at<int32_t>(7), p, at<uint64_t>(8), at<uint16_t>(9),
                                        save ? at<float>(10) : nullptr, at<void>(11), bytes, nullptr);
            };
            const auto bwd = [&](size_t bytes, bool saved, bool dx) {
              return qlora_adapters_bwd(&q, &set, at<uint16_t>(6), at<uint16_t>(9), M, at<int32_t>(7), p, at<uint64_t>(8),
                                        saved ? at<float>(10) : nullptr, dx ? at<uint16_t>(12) : nullptr, at<void>(11), bytes,
                                        nullptr);
            };
            const bool stream = (M <= 64 || (M <= 128 && N * K < int64_t(1) << 25)) && dq == QLORA_DQ_E4M3;
            for (int save = 0; save < 2; ++save) {
              // T and the stream, or T (with the decode, or before it), the product, its parts' sum
              run([&] { return fwd(fw, save); }, stream ? 1 : 2, stream ? 2 : 4, "fwd", M, N, K);
              run([&] { return bwd(bw, save, false); }, 2, 2, "bwd without dX", M, N, K);
              run([&] { return bwd(bw, save, true); }, 3, 5, "bwd", M, N, K);
            }
            CHECK(fwd(fw - 256, false) == QLORA_ERR_WORKSPACE && bwd(bw - 256, false, true) == QLORA_ERR_WORKSPACE, "short");
          }
}

void dropouts() {
  for (int64_t n : {int64_t(1), int64_t(7), int64_t(8), int64_t(2049), int64_t(1) << 31, int64_t(1) << 38})
    for (int xt : {QLORA_BF16, QLORA_F32})
      for (int ot : {QLORA_BF16, QLORA_F32})
        for (int odd = 0; odd < 2; ++odd)
          for (void* res : {static_cast<void*>(nullptr), at<void>(3)})
            run([&] {
              return qlora_dropout(at<char>(1) + 4 * odd, xt, n, 0.1f, at<uint64_t>(2), res, at<char>(5) + 4 * odd, ot, nullptr);
            }, 1, 1, "dropout", n, xt, ot);
}

}  // namespace

int main() {
  tables();
  linears();
  dropouts();
  std::printf("OK %d\n", g_checks);
  return 0;
}
