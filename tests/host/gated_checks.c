/* Argument checks of the gated blocks and of dropout, driven from C without a GPU: every call
 * here is refused, or has nothing to do, before anything is enqueued. */
#include <limits.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "w4a16_moe.h"

static int failures = 0;
#define EXPECT(status, call)                                                               \
  do {                                                                                     \
    const int rc_ = (call);                                                                \
    if (rc_ != (status)) {                                                                 \
      ++failures;                                                                          \
      printf("line %d: %d, expected %d (%s)\n", __LINE__, rc_, (status), moe_last_error()); \
    }                                                                                      \
  } while (0)

static const int sizes[] = {INT_MIN, -1, 0, 1, 7, 8, 1024, 65536, 65544, 1 << 24, (1 << 24) + 1, INT_MAX};
#define NUM_SIZES ((int)(sizeof(sizes) / sizeof(sizes[0])))

int main(void) {
  /* never dereferenced: a valid address for the alignment checks only */
  void* p = aligned_alloc(256, 256);
  int calls = 0;
  for (int i = 0; i < NUM_SIZES; ++i)
    for (int j = 0; j < NUM_SIZES; ++j)
      for (int k = 0; k < NUM_SIZES; ++k) {
        const int R = sizes[i], d = sizes[j], n = sizes[k];
        /* a missing pointer: refused whatever the sizes are, or no rows */
        if (moe_dropout(NULL, n, p, n, MOE_BF16, R, d, 0.5, (const int64_t*)p, n, p, n, NULL) == MOE_OK && R != 0) {
          ++failures;
          printf("dropout accepted T=%d d=%d\n", R, d);
        }
        moe_gated_ffn_args a;
        memset(&a, 0, sizeof(a));
        a.num_rows = R;
        a.d = d;
        a.I = n;
        a.E = 1;
        a.rows_stride = n;
        a.w13 = a.w2 = p;
        moe_gated_ffn_grads g;
        memset(&g, 0, sizeof(g));
        g.dw2 = p;
        g.dy_stride = g.h_stride = n;
        if (moe_gated_ffn(&a, NULL, 0, p, n, p, n, NULL) == MOE_OK && R != 0) {
          ++failures;
          printf("gated_ffn accepted R=%d d=%d I=%d\n", R, d, n);
        }
        if (R > 0 && moe_gated_ffn_backward(&a, &g, NULL) == MOE_OK) {
          ++failures;
          printf("gated_ffn_backward accepted R=%d d=%d I=%d\n", R, d, n);
        }
        for (int e = 0; e < NUM_SIZES; ++e) {
          const int64_t w = moe_gated_ffn_backward_workspace_bytes(R, d, n, sizes[e]);
          const int fits = R >= 0 && R <= 1 << 24 && d > 0 && d <= 65536 && d % 8 == 0 && n > 0 && n <= 65536 &&
                           n % 8 == 0 && sizes[e] > 0 && sizes[e] <= 1024;
          if (fits ? w < (int64_t)R * n * 4 : w != -1) {
            ++failures;
            printf("workspace %lld for R=%d d=%d I=%d E=%d\n", (long long)w, R, d, n, sizes[e]);
          }
        }
        calls += 3 + NUM_SIZES;
      }
  EXPECT(MOE_ERR_INVALID_ARG, moe_gated_ffn(NULL, p, 8, p, 8, p, 8, NULL));
  EXPECT(MOE_ERR_INVALID_ARG, moe_gated_ffn_backward(NULL, NULL, NULL));
  moe_gated_ffn_args a;
  memset(&a, 0, sizeof(a));
  a.num_rows = 2;
  a.d = a.I = 8;
  a.E = 1;
  a.rows = a.w13 = a.w2 = p;
  a.rows_stride = 8;
  const double bad[] = {-0.1, 1.5, NAN, INFINITY};
  for (int i = 0; i < 4; ++i) {
    a.drop_p = bad[i];
    EXPECT(MOE_ERR_INVALID_ARG, moe_gated_ffn(&a, NULL, 0, p, 8, p, 8, NULL));
    EXPECT(MOE_ERR_INVALID_ARG, moe_dropout(p, 8, NULL, 0, MOE_FP32, 2, 8, bad[i], (const int64_t*)p, 0, p, 8, NULL));
  }
  a.drop_p = 0.0;
  for (int kind = -1; kind <= 3; ++kind) {
    a.activation = kind;
    if (kind < 0 || kind > 1) EXPECT(MOE_ERR_INVALID_ARG, moe_gated_ffn(&a, NULL, 0, p, 8, p, 8, NULL));
  }
  free(p);
  printf("gated checks: %d calls, %d failures\n", calls, failures);
  return failures != 0;
}
