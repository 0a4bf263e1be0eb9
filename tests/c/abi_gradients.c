/* A C99 caller of the gradient operators' C ABI (no C++, no CUDA headers): workspace sizes
 * and documented argument errors.  No device is touched; prints "ok" and returns 0 when
 * every check holds. */
#include <stdio.h>
#include <string.h>

#include "dion.h"

static int failures = 0;

static void expect(int cond, const char* what) {
  if (!cond) {
    printf("FAILED: %s (last error: %s)\n", what, dion_last_error());
    ++failures;
  }
}

int main(void) {
  dion_norm nm;
  memset(&nm, 0, sizeof(nm));
  nm.features = 64; nm.tokens = 1; nm.residual_scale = 1.f;
  expect(dion_norm_forward(&nm, NULL) == DION_ERR_INVALID_ARG, "norm eps check");
  expect(strlen(dion_last_error()) > 0, "error message");
  expect(dion_norm_backward_workspace(16, 64) > 0, "norm workspace");
  expect(dion_norm_backward(NULL, NULL, 0, NULL) == DION_ERR_INVALID_ARG, "norm null args");

  dion_grad_source gs;
  memset(&gs, 0, sizeof(gs));
  gs.kept.features = 64; gs.kept.tokens = 1 << 14; gs.n = 32; gs.ldd = 32; gs.ldg = 32;
  expect(dion_weight_grad_workspace(&gs, 1) > 0, "weight gradient workspace");
  expect(dion_weight_grad(&gs, 1, 0, NULL, 0, NULL, NULL) == DION_ERR_INVALID_ARG, "null rows");
  expect(dion_step_batched_from_saved(NULL, NULL, &gs, 1, 0, 0.1f, NULL, 0, NULL, NULL, NULL) ==
             DION_ERR_NOT_INITIALIZED, "null handle");

  expect(dion_act_save(NULL, 64, DION_FP16, NULL, NULL) == DION_ERR_INVALID_ARG, "null kept rows");
  expect(dion_act_load(NULL, NULL, 64, DION_FP32, NULL) == DION_ERR_INVALID_ARG, "null kept rows");

  dion_embed em;
  memset(&em, 0, sizeof(em));
  expect(dion_embed_lookup(&em, NULL) == DION_ERR_INVALID_ARG, "vocab check");
  expect(dion_embed_backward_workspace(100, 64) > 0, "embedding workspace");
  expect(dion_embed_backward(NULL, NULL, 0, NULL) == DION_ERR_INVALID_ARG, "embedding null args");
  if (failures == 0) printf("ok\n");
  return failures ? 1 : 0;
}
