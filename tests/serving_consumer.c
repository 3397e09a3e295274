/* C11 consumer of include/mlra_serving.h: links every entry point and checks
 * the host-side argument validation (no GPU needed). */
#include <stdio.h>

#include "mlra_serving.h"

static void* table[] = {
    (void*)mla_prompt_workspace_bytes, (void*)mla_prompt,   (void*)mlra_absorb, (void*)mlra_attention_weights,
    (void*)latent_evict_workspace_bytes, (void*)latent_evict,
};

int main(void) {
  mlra_dims d = {1, 8, 32, 32, 64, 16, 1, 64, 4, 4, 0.f, 1.f, 0.f, MLRA_F32, 0, MLRA_KERNEL_AUTO};
  mla_prompt_shape s = {8, 10, 10, {256, 32}, {128, 16}, {256, 32}, {256, 32}};
  if (mla_prompt_workspace_bytes(&d, &s) < 256) return 1;
  s.kv_heads = 3;
  if (mla_prompt_workspace_bytes(&d, &s) != 0 || !mlra_last_error()[0]) return 2;
  if (latent_evict_workspace_bytes(&d) < 256) return 3;
  if (latent_evict(&d, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) != MLRA_ERR_INVALID_ARG) return 4;
  if (mlra_absorb(0, 0, 0, 0, 0, 0, 0, 0, 0) != MLRA_ERR_INVALID_ARG) return 5;
  printf("ok %zu entry points\n", sizeof(table) / sizeof(table[0]));
  return 0;
}
