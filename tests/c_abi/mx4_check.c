/* A plain C99 caller of include/mx4.h and include/orthogonalize.h: sizes and host-side validation with
 * fake device addresses that are rejected before any HIP call. Prints "abi ok" and exits 0 when every
 * check holds. */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "mx4.h"
#include "orthogonalize.h"

static int failures = 0;
#define CHECK(cond)                                                      \
  do {                                                                   \
    if (!(cond)) {                                                       \
      fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #cond); \
      ++failures;                                                        \
    }                                                                    \
  } while (0)

int main(void) {
  char *const base = (char *)((uintptr_t)1 << 40); /* never dereferenced */
  CHECK(muon_mx_codes_size(17, 129) == 4 * 1024 && muon_mx_scales_size(17, 129) == 4 * 64);
  CHECK(muon_mx_codes_size(-1, 1) == SIZE_MAX);

  muon_mx_source s;
  memset(&s, 0, sizeof s);
  s.x = base;
  s.rows = 3;
  s.cols = s.row_stride = 100;
  s.dtype = MUON_DT_F32;
  CHECK(muon_mx_quantize(&s, 1, 0, 0, NULL) == MUON_ERR_INVALID_ARG);
  CHECK(strstr(muon_last_error(), "no result") != NULL);
  s.codes = base + 1024;
  s.scales = base + (1 << 20);
  CHECK(muon_mx_quantize(&s, 1, 1, 7, NULL) == MUON_ERR_INVALID_ARG);
  CHECK(strstr(muon_last_error(), "overlaps") != NULL);
  CHECK(muon_mx_quantize(NULL, 0, 0, 0, NULL) == MUON_OK);
  CHECK(muon_mx_dequantize(base, NULL, 3, 100, base + 4096, MUON_DT_BF16, NULL) == MUON_ERR_INVALID_ARG);
  CHECK(muon_mx_dequantize(NULL, NULL, 0, 100, NULL, MUON_DT_BF16, NULL) == MUON_OK);

  CHECK(muon_mx_matmul_workspace_size(128, 128, 1 << 20) > 0);
  CHECK(muon_mx_matmul(base, base + (1 << 28), base + (2 << 28), base + 3 * (1 << 28), 128, 128, 1 << 20,
                       base + ((size_t)1 << 31), MUON_DT_F32, NULL, 0, NULL) == MUON_ERR_WORKSPACE);
  CHECK(strstr(muon_last_error(), "workspace") != NULL);

  muon_config cfg;
  muon_config_default(&cfg);
  muon_stack k;
  memset(&k, 0, sizeof k);
  k.in = base;
  k.out = base + 4;
  k.outer = 1;
  k.inner = 2;
  k.rows = 4;
  k.cols = 8;
  k.in_stride[1] = k.out_stride[1] = 32;
  k.in_stride[2] = k.out_stride[2] = 8;
  k.in_stride[3] = k.out_stride[3] = 1;
  k.dtype = MUON_DT_F32;
  CHECK(muon_orthogonalize_workspace_size(1, 2, 4, 8) == 0);
  CHECK(muon_orthogonalize(&k, &cfg, NULL, 0, NULL) == MUON_ERR_INVALID_ARG);
  CHECK(strstr(muon_last_error(), "overlaps") != NULL);
  k.cols = 0;
  CHECK(muon_orthogonalize(&k, &cfg, NULL, 0, NULL) == MUON_OK);
  if (failures) return 1;
  printf("abi ok\n");
  return 0;
}
