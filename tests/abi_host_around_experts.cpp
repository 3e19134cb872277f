// Drives the host code of the calls around the experts over sizes up to the largest
// ints: workspaces, and calls that end at the last argument check (an output on top of
// an input), so nothing is launched.  Built with the library under AddressSanitizer and
// with traps on undefined behaviour (signed overflow among it).
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "moe_decode.h"

static int failures = 0, calls = 0;

static void expect(const char* what, int rc, int late) {
  ++calls;
  if (rc == late || rc == MOE_ERR_SHAPE || rc == MOE_ERR_ARG) return;
  std::printf("%s: %d\n", what, rc);
  ++failures;
}

int main() {
  const int most = 2147483647;
  const int big[] = {0, 1, 2, 8, 17, 128, 513, 4096, 4097, 16385, 32768, 1 << 20, (1 << 22) - 1, 1 << 22, (1 << 24) - 1, 1 << 24,
                     (1 << 26) - 1, 1 << 26, 1 << 28, 1 << 30, most - 7, most};
  const int few[] = {1, 7, 8, 16, 64, 256, 1023, 1024, 1025, most};
  // stand-ins for device memory, never touched; outputs lie at the first input
  char* base = reinterpret_cast<char*>(uintptr_t(1) << 44);
  void* x = base;
  auto other = [&](int i) { return static_cast<void*>(base + (uint64_t(i) << 52)); };
  auto ints = [&](int i) { return static_cast<int32_t*>(other(i)); };
  auto floats = [&](int i) { return static_cast<float*>(other(i)); };

  for (int T : big)
    for (int E : few)
      for (int k : {1, 8, 64, 65}) {
        size_t n = 0;
        const int late = T == 0 ? MOE_OK : MOE_ERR_ALIAS;
        for (int G : {1, 2, 8, 64, most})
          for (long long ld : {(long long)E, 1LL << 30, 1LL << 62})
            expect("route", moe_decode_route_experts(x, ld, MOE_F32, nullptr, static_cast<int32_t*>(x), floats(1), T, E, k, G,
                                                     G > 1 ? G - 1 : 1, 7, 1.0f, nullptr), late);
        expect("route_backward", moe_decode_route_experts_backward(x, E, MOE_BF16, ints(1), floats(2), x, E, T, E, k, 0, 1.0f, nullptr), late);
        expect("sort workspace", moe_decode_sort_slots_workspace(T, E, k, &n), MOE_OK);
        expect("sort", moe_decode_sort_slots(static_cast<int32_t*>(x), nullptr, ints(1), ints(2), static_cast<int32_t*>(x), other(3), n,
                                             T, E, k, nullptr), late);
        for (int M : big)
          for (int N : {1, 2048, 1 << 28, most}) {
            expect("combine", moe_decode_combine(other(1), N, MOE_F32, static_cast<int32_t*>(x), floats(2), nullptr, 0, x, N, M, T, N, k,
                                                 nullptr), late);
            expect("combine_backward", moe_decode_combine_backward(other(1), N, other(2), N, MOE_BF16, static_cast<int32_t*>(x), floats(3),
                                                                   other(4), N, static_cast<float*>(x), M, T, N, k, nullptr), late);
          }
      }

  for (int M : big)
    for (int H : big)
      for (long long ld : {(long long)H, 1LL << 30, 1LL << 62}) {
        const int late = M == 0 ? MOE_OK : MOE_ERR_ALIAS;
        size_t n = 0;
        expect("norm", moe_decode_rms_norm(x, ld, nullptr, 0, MOE_F16, other(1), MOE_F32, 1e-6f, x, ld, nullptr, nullptr, nullptr, 0,
                                           nullptr, M, H, 0, nullptr), late);
        expect("norm workspace", moe_decode_rms_norm_backward_workspace(M, H, &n), MOE_OK);
        expect("norm_backward", moe_decode_rms_norm_backward(x, ld, other(1), ld, MOE_F32, other(2), MOE_F32, floats(3), nullptr, 0, x, ld,
                                                             floats(4), other(5), n, M, H, nullptr), late);
      }

  for (int M : big)
    for (int K : big)
      for (int N : big)
        for (int R : {8, 16, 256, 264, most - 7})
          for (int L : {1, 1023, 1024, most}) {
            size_t n = 0;
            expect("adapters workspace", moe_decode_adapters_workspace(M, K, N, R, L, &n), MOE_OK);
            expect("adapters", moe_decode_adapters(x, K, MOE_BF16, ints(1), other(2), other(3), floats(4), nullptr, 0, x, N, other(5), n, M,
                                                   K, N, R, L, nullptr), M == 0 ? MOE_OK : MOE_ERR_ALIAS);
          }
  std::printf("%d calls, %d failures\n", calls, failures);
  return failures != 0;
}
