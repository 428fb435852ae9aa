// Driver for a host-only build of csrc/adapter_ops.hpp: what the adapters' kernels
// address with 32 bits stays below the limits that their launchers rely on.
// Nothing touches a GPU.
#include <stdint.h>
#include <stdio.h>

#include "../../bitlinear_absmean_ternarise_bit_amd/csrc/adapter_ops.hpp"

int main() {
  using namespace bitlinear;
  const int64_t past = int64_t(1) << 31;  // an offset that the kernels take as behind every resource
  int run = 0, failed = 0;
  for (int64_t R = 1; R <= kAdapterMaxR; ++R)
    for (int64_t N : {int64_t(8), int64_t(2048), int64_t(11008), past / (4 * R) - 1, past / (4 * R), past / (4 * R) + 1,
                      (int64_t(1) << 23) + 1, (int64_t(1) << 24) - 1, int64_t(1) << 24})
      for (int64_t M : {int64_t(256), int64_t(2048), int64_t(1) << 20}) {
        ++run;
        // the epilogue holds an adapter's R rows of N float32 in one resource
        if (N >= 1 && adapted_gemm_takes(M, N, R) && 4 * R * N >= past) {
          ++failed;
          printf("M=%lld N=%lld R=%lld: %lld bytes of weights in one resource\n", (long long)M, (long long)N, (long long)R,
                 (long long)(4 * R * N));
        }
      }
  // and is taken where it fits
  for (int64_t N : {int64_t(2048), int64_t(11008), (past / 256) - 1}) {
    ++run;
    if (!adapted_gemm_takes(2048, N, 64)) ++failed, printf("N=%lld: not taken\n", (long long)N);
  }
  printf("%d checks, %d failed\n", run, failed);
  return failed != 0;
}
