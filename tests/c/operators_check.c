/* Plain-C client of the operators around the loss: the header's structs as C11
 * sees them, and refusals that come before any CUDA call.  Prints "ok <n>"
 * after n passed checks, or "FAIL <what>" and exits 1.                       */
#include <stdio.h>
#include <string.h>

#include "relkl.h"

static int n_ok = 0;
#define CHECK(cond, what)                       \
  do {                                          \
    if (!(cond)) {                              \
      printf("FAIL %s\n", what);                \
      return 1;                                 \
    }                                           \
    ++n_ok;                                     \
  } while (0)

int main(void) {
  char* at = (char*)(size_t)(1 << 24);   /* never dereferenced */
  const size_t step = 1 << 24;

  CHECK(sizeof(relkl_rotary_tensor) == 72 && sizeof(relkl_rotary_plan) == 88, "rotary structs");
  relkl_rotary_tensor t = {at, at + step, {1024, 512, 64}, {1024, 512, 64}, 2, 1};
  relkl_rotary_plan plan;
  memset(&plan, 0, sizeof plan);
  plan.B = 2; plan.N = 8; plan.d = 64; plan.rot = 64;
  plan.mscale = 1.0f; plan.pos_scale = 1.0; plan.inv_freq = (const double*)at;
  plan.rot = 63;
  CHECK(relkl_rotary(1, &t, &plan, NULL) == RELKL_ERR_INVALID, "odd rotated part");
  plan.rot = 64;
  t.y = at + 128;
  CHECK(relkl_rotary(1, &t, &plan, NULL) == RELKL_ERR_INVALID, "output inside the input");
  plan.N = 0;
  CHECK(relkl_rotary(1, &t, &plan, NULL) == RELKL_OK, "no tokens");

  CHECK(sizeof(relkl_adamw_tensor) == 80 && sizeof(relkl_adamw_plan) == 72 &&
            sizeof(relkl_norm_tensor) == 24,
        "adamw structs");
  relkl_adamw_tensor w = {at, at + step, NULL, at + 2 * step, at + 3 * step, NULL, NULL,
                          100, RELKL_FP32, RELKL_FP32, 0.1f, 0};
  relkl_adamw_plan step1 = {32, 0, 1e-3, 0.9, 0.999, 1e-8, 0, NULL, NULL, NULL};
  CHECK(relkl_adamw(1, &w, &step1, NULL) == RELKL_ERR_INVALID, "step 0");
  step1.step = 1;
  w.v = w.m;
  CHECK(relkl_adamw(1, &w, &step1, NULL) == RELKL_ERR_INVALID, "one array for both moments");
  CHECK(relkl_adamw(0, NULL, &step1, NULL) == RELKL_OK, "no tensors");
  relkl_norm_tensor g = {at, 100, RELKL_FP32, 0};
  CHECK(relkl_grad_norm(1, &g, 1.0f, (float*)at, at, 8, NULL) == RELKL_ERR_WORKSPACE,
        "norm with too little scratch");
  CHECK(relkl_grad_norm(1, &g, -1.0f, (float*)at, at, relkl_grad_norm_bytes(1), NULL) ==
            RELKL_ERR_INVALID,
        "norm with a negative bound");

  int8_t* q = (int8_t*)at;
  CHECK(relkl_quantize_rows(4, 100, at, RELKL_BF16, 100, q, 100, (float*)at, NULL) ==
            RELKL_ERR_INVALID,
        "code rows off 16-byte boundaries");
  CHECK(relkl_matmul_i8(4, 8, 131072, q, 131072, (float*)at, q, 131072, (float*)at, NULL, at,
                        RELKL_BF16, 8, at, 256, NULL) == RELKL_ERR_INVALID,
        "sums past int32");
  CHECK(relkl_matmul_i8(0, 8, 64, NULL, 0, NULL, NULL, 0, NULL, NULL, NULL, RELKL_BF16, 8, NULL, 0,
                        NULL) == RELKL_OK,
        "product without rows");
  CHECK(relkl_linear_i8_bytes(4, 4096) == 0 && relkl_linear_i8_bytes(5, 4096) > 0, "scratch sizes");
  CHECK(relkl_linear_i8(9, 8, 4096, at, RELKL_BF16, 4096, q, 4096, (float*)at, NULL, at + step,
                        RELKL_BF16, 8, NULL, 0, at, 256, NULL) == RELKL_ERR_WORKSPACE,
        "linear without scratch");
  printf("ok %d\n", n_ok);
  return 0;
}
