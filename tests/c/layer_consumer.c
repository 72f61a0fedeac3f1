/* A plain C consumer of the operators around the recurrences: compiled with a C
 * compiler against include/osdn.h alone, it checks workspace queries and argument
 * validation without launching any GPU work. Exit status 0 = all checks passed;
 * otherwise the number of failed checks. */
#include <limits.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "osdn.h"

static int failures = 0;

#define CHECK(cond)                                                     \
  do {                                                                  \
    if (!(cond)) {                                                      \
      fprintf(stderr, "check failed (line %d): %s\n", __LINE__, #cond); \
      ++failures;                                                       \
    }                                                                   \
  } while (0)

#define P(x) ((void*)(uintptr_t)((uint64_t)(x) << 44))
#define F(x) ((float*)P(x))

int main(void) {
  static const int dims[3] = {32, 64, 128};
  static const int lens[8] = {0, 1, 31, 64, 65, 1000, 4096, 1 << 20};
  CHECK(strcmp(osdn_strerror(OSDN_ERR_MISALIGNED), "unknown status") != 0);

  /* every supported size has a workspace of whole 256-byte pieces that holds at
   * least what the header says it holds, and grows with T */
  for (int a = 0; a < 3; ++a)
    for (int b = 0; b < 3; ++b)
      for (int dt = 0; dt < 2; ++dt) {
        size_t last_f = 0, last_b = 0;
        for (int t = 0; t < 8; ++t) {
          const int T = lens[t], Q = dt ? 64 : 32;
          const size_t nch = ((size_t)T + Q - 1) / Q;
          const size_t f = ssm_forward_workspace_bytes(2, 6, 3, T, dims[a], dims[b], dt);
          const size_t w = ssm_backward_workspace_bytes(2, 6, 3, T, dims[a], dims[b], dt);
          CHECK(f % 256 == 0 && w % 256 == 0);
          CHECK(f >= last_f && w >= last_b);
          CHECK(w >= 12 * nch * 2 * dims[a] * dims[b] * 4);
          CHECK(T == 0 || f > 0);
          last_f = f;
          last_b = w;
        }
      }
  for (int c = 1; c < 2000; c += 37)
    for (int t = 0; t < 8; ++t) {
      const size_t w = short_conv_backward_workspace_bytes(2, lens[t], 1, c, 4);
      CHECK(w % 256 == 0 && w >= (size_t)5 * c * 4);
    }
  CHECK(gated_norm_backward_workspace_bytes(2, 0, 3, 64) == 0);
  CHECK(gated_norm_backward_workspace_bytes(2, 4, 0, 64) == 0);
  CHECK(gated_norm_backward_workspace_bytes(2, 4, 5, 64) > 0);
  CHECK(residual_norm_backward_workspace_bytes(0, 64) == 0);
  CHECK(residual_norm_backward_workspace_bytes(5, OSDN_RESIDUAL_NORM_MAX_WIDTH) > 0);
  CHECK(residual_norm_backward_workspace_bytes(5, OSDN_RESIDUAL_NORM_MAX_WIDTH + 1) == 0);

  /* sizes out of range never reach a size computation */
  CHECK(ssm_forward_workspace_bytes(INT_MAX, INT_MAX, 1, 1, 64, 64, 1) == 0);
  CHECK(ssm_forward_workspace_bytes(1, 1, 1, INT_MAX, 64, 64, 1) == 0);
  CHECK(ssm_backward_workspace_bytes(1, 4, 3, 8, 64, 64, 1) == 0);
  CHECK(ssm_backward_workspace_bytes(INT_MIN, 4, 2, 8, 64, 64, 1) == 0);
  CHECK(short_conv_backward_workspace_bytes(1, 8, INT_MAX, INT_MAX, 4) == 0);
  CHECK(short_conv_backward_workspace_bytes(1, 8, 2, 64, 9) == 0);
  CHECK(gated_norm_backward_workspace_bytes(1, INT_MAX, 8, 128) == 0);
  CHECK(residual_norm_backward_workspace_bytes(LLONG_MAX, 8) == 0);

  /* refusals before any launch */
  CHECK(short_conv_forward(1, 4, 2, 64, 4, OSDN_BF16, P(1), 0, 128, F(2), NULL, NULL,
                           NULL, 1, 0, 1e-6f, P(1), NULL, NULL) == OSDN_ERR_ALIASING);
  CHECK(short_conv_decode(1, 1, 2, 64, 4, OSDN_BF16, P(1), 0, 128, F(2), NULL, NULL, 1, 0,
                          1e-6f, P(3), NULL, NULL) == OSDN_ERR_NULL_ARG);
  CHECK(gated_norm_forward(1, 2, 4, 48, OSDN_BF16, P(1), P(2), 0, 96, F(3), 0, 1e-6f, 0,
                           P(4), NULL) == OSDN_ERR_UNSUPPORTED);
  CHECK(gated_norm_forward(1, 2, 4, 64, OSDN_BF16, P(1), P(2), 0, -1, F(3), 0, 1e-6f, 0,
                           P(4), NULL) == OSDN_ERR_BAD_DIMS);
  CHECK(residual_norm_forward(4, 64, OSDN_F32, OSDN_BF16, P(1), P(2), 1.f, F(3), 1e-6f,
                              P(4), P(5), NULL) == OSDN_ERR_UNSUPPORTED);
  CHECK(residual_norm_backward(4, 64, OSDN_F32, OSDN_F32, P(1), P(2), NULL, 1.f, F(3), 1e-6f,
                               P(4), P(5), F(6), NULL, 0, NULL) == OSDN_ERR_WORKSPACE);
  CHECK(ssm_forward(1, 2, 1, 4, 64, 64, OSDN_BF16, P(1), F(2), F(3), P(4), P(5), NULL, NULL,
                    1, NULL, NULL, P(6), F(7), NULL, 0, NULL) == OSDN_ERR_WORKSPACE);
  CHECK(ssm_decode(1, 2, 1, 1, 64, 64, OSDN_BF16, P(1), F(2), F(3), P(4), P(5), NULL, NULL,
                   1, F(6), P(6), F(6), NULL) == OSDN_ERR_ALIASING);

  /* nothing to do: returns before any launch */
  CHECK(ssm_forward(0, 2, 1, 4, 64, 64, OSDN_BF16, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 1,
                    NULL, NULL, NULL, NULL, NULL, 0, NULL) == OSDN_OK);
  CHECK(residual_norm_forward(0, 64, OSDN_F32, OSDN_F32, NULL, NULL, 1.f, NULL, 1e-6f, NULL,
                              NULL, NULL) == OSDN_OK);

  if (failures == 0) printf("all checks passed\n");
  return failures;
}
