// Drives the host code of the router's training pass and of the block-scaled
// 8-bit operators over sizes up to the largest ints: workspaces, plans, and
// calls that end at the last argument check (an output on top of an input), so
// nothing is launched.  Built with the library under AddressSanitizer and with
// traps on undefined behaviour (signed overflow among it).
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "moe_decode.h"

static int failures = 0, calls = 0;

static void expect(const char* what, int rc, bool refused_early, int late) {
  ++calls;
  const bool early = rc == MOE_ERR_SHAPE || rc == MOE_ERR_ARG;
  if (rc == late || (refused_early && early)) return;
  std::printf("%s: %d\n", what, rc);
  ++failures;
}

int main() {
  const int most = 2147483647;
  const int big[] = {0, 1, 2, 16, 17, 127, 128, 129, 300, 2048, 4096, 65536, (1 << 20) + 16, 1 << 24, (1 << 24) - 1,
                     1 << 28, 1 << 30, (1 << 30) + 16, most - 15, most};
  const int experts[] = {1, 2, 100, 128, 1024, 1025, most};
  // stand-ins for device memory, never touched; outputs lie inside the first input
  char* base = reinterpret_cast<char*>(uintptr_t(1) << 44);
  void* x = base;
  auto other = [&](int i) { return static_cast<void*>(base + (uint64_t(i) << 45)); };

  for (int T : big)
    for (int E : experts)
      for (int k : {1, 8, 64, 65})
        for (int G : {1, 2, 64, 1 << 19, (1 << 19) + 1}) {
          size_t n = 0;
          const int rc = moe_decode_balance_workspace(T, E, k, G, &n);
          expect("workspace", rc, true, MOE_OK);
          const int late = T == 0 ? MOE_OK : MOE_ERR_ALIAS;
          for (int dt : {MOE_F32, MOE_BF16}) {
            const int r = moe_decode_balance(x, E, dt, static_cast<int32_t*>(other(1)), nullptr, static_cast<float*>(other(2)),
                                             static_cast<int32_t*>(x), static_cast<int32_t*>(other(3)), other(4), n, T, E, k, G,
                                             nullptr);
            expect("balance", r, rc != MOE_OK, late);
            const int b = moe_decode_balance_backward(x, E, dt, nullptr, static_cast<int32_t*>(other(1)),
                                                      static_cast<int32_t*>(other(2)), static_cast<float*>(other(3)), x, E, T, E,
                                                      k, G, nullptr);
            expect("balance_backward", b, rc != MOE_OK, late);
          }
        }

  for (int M : big)
    for (int K : big)
      for (int flags : {0, 1, 2, 3})
        for (long long ld : {0LL, (long long)K, 2LL * K, 1LL << 30, (1LL << 62)}) {
          const int r = moe_decode_quantize_fp8(x, ld, MOE_BF16, static_cast<uint8_t*>(x), static_cast<float*>(other(1)), M, K,
                                                flags, nullptr);
          expect("quantize", r, true, M == 0 ? MOE_OK : MOE_ERR_ALIAS);
        }

  for (int M : big)
    for (int N : big)
      for (int K : big)
        for (int E : {0, 1, 128, 1024, 1025, most}) {
          int v = 0, g = 0;
          const int rc = moe_decode_matmul_fp8_plan(M, N, K, E, &v, &g);
          expect("plan", rc, true, MOE_OK);
          if (rc == MOE_OK && (v < MOE_MATMUL_ROWS_16 || v > MOE_MATMUL_FAR_ROWS || g < 0 || (M > 0 && g == 0))) {
            std::printf("plan %d %d %d %d: %d %d\n", M, N, K, E, v, g);
            ++failures;
          }
          const uint8_t* xb = static_cast<const uint8_t*>(x);
          const float* sx = static_cast<float*>(other(1));
          const uint8_t* w = static_cast<uint8_t*>(other(2));
          const float* sw = static_cast<float*>(other(3));
          for (long long ld : {(long long)K, 1LL << 30, 1LL << 62}) {
            const int late = M == 0 ? MOE_OK : MOE_ERR_ALIAS;
            if (E == 0)
              expect("matmul", moe_decode_matmul_fp8(xb, ld, sx, w, sw, x, ld > N ? ld : N, MOE_BF16, M, N, K, nullptr), true, late);
            else
              expect("experts", moe_decode_matmul_fp8_experts(xb, ld, sx, nullptr, static_cast<int32_t*>(other(4)), w, sw, x,
                                                              ld > N ? ld : N, MOE_F32, M, M, N, K, E, nullptr), true, late);
          }
        }
  std::printf("%d calls, %d failures\n", calls, failures);
  return failures != 0;
}
