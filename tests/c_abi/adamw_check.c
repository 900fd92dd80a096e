/* A plain C99 caller of include/adamw.h and include/grad_norm.h: defaults, plans and host-side
 * validation with fake device addresses that are rejected before any HIP call. Prints "abi ok"
 * and exits 0 when every check holds. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "adamw.h"
#include "grad_norm.h"

static int failures = 0;
#define CHECK(cond)                                                      \
  do {                                                                   \
    if (!(cond)) {                                                       \
      fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #cond); \
      ++failures;                                                        \
    }                                                                    \
  } while (0)

int main(void) {
  const uintptr_t base = (uintptr_t)1 << 40; /* never dereferenced */
  muon_adamw_config cfg;
  muon_adamw_config_default(&cfg);
  CHECK(cfg.step == 1 && cfg.stochastic == 1 && cfg.grad_scale == NULL);

  muon_adamw_tensor t;
  memset(&t, 0, sizeof t);
  t.param = (void *)base;
  t.exp_avg = (void *)(base + 4096);
  t.exp_avg_sq = (void *)(base + 8192);
  t.exp_avg_scale = (uint8_t *)(base + 12288);
  t.exp_avg_sq_scale = (uint8_t *)(base + 12288 + 4);
  t.numel = 3 * MUON_ADAMW_BLOCK + 1;
  t.param_dtype = t.grad_dtype = MUON_DT_F32;
  t.wd_mul = 1.0f;
  muon_adamw_plan *plan = NULL;
  CHECK(muon_adamw_plan_create(&plan, &t, 1, MUON_ADAMW_8BIT) == MUON_OK && plan != NULL);
  const void *grad = (const void *)(base + 4096);
  CHECK(muon_adamw_step(plan, &grad, 1, &cfg, NULL) == MUON_ERR_INVALID_ARG);
  CHECK(strstr(muon_last_error(), "overlaps") != NULL);
  grad = NULL;
  CHECK(muon_adamw_step(plan, &grad, 1, &cfg, NULL) == MUON_OK);
  muon_adamw_plan_destroy(plan);
  t.exp_avg_sq_scale = (uint8_t *)(base + 12288 + 3);
  CHECK(muon_adamw_plan_create(&plan, &t, 1, MUON_ADAMW_8BIT) == MUON_ERR_INVALID_ARG);
  CHECK(plan == NULL);

  const int64_t numel[2] = {1000, 0};
  const muon_dtype dt[2] = {MUON_DT_BF16, MUON_DT_F32};
  muon_grad_plan *gp = NULL;
  CHECK(muon_grad_plan_create(&gp, numel, dt, 2) == MUON_OK && gp != NULL);
  CHECK(muon_grad_plan_workspace_size(gp) > 0);
  const void *grads[2] = {(const void *)base, NULL};
  CHECK(muon_grad_norm(gp, grads, 2, 1.0f, (float *)(base + 4096), NULL, NULL, 0, NULL) ==
        MUON_ERR_WORKSPACE);
  CHECK(muon_grad_norm(gp, grads, 2, -1.0f, (float *)(base + 4096), NULL, NULL, 0, NULL) ==
        MUON_ERR_INVALID_ARG);
  void *out[2] = {NULL, NULL};
  CHECK(muon_grad_scale(gp, out, 2, NULL, NULL) == MUON_ERR_INVALID_ARG);
  muon_grad_plan_destroy(gp);
  if (!failures) printf("abi ok\n");
  return failures != 0;
}
