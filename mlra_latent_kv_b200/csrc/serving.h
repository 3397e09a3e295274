// Internal launcher interface of the prompt and eviction operators.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mlra_serving.h"
#include "common.cuh"

namespace mlra {

// A bf16 tensor map, encoded anew for each call (nothing is kept by address):
// `rank` axes, innermost first; strides in bytes of axes 1 .. rank-1; 128-byte
// swizzle; reads outside the tensor give zeros.
bool encode_bf16_map(CUtensorMap* out, int rank, const void* base, const uint64_t* dims, const uint64_t* strides,
                     const uint32_t* box);

struct WeightArgs {
  int B, H, d_c, d_r, n_branch, maxp, num_pages;
};

bool weights_tc_supported(int dtype, int H, int d_c, int d_r, int n_branch);
cudaError_t launch_weights_tc(const void* q_abs, const float* lse, const void* lat, const void* rop,
                              const int* page_table, const int* seq_lens, const float* w_in, float* w_out, int* err,
                              const WeightArgs& a, int sms, cudaStream_t st);
cudaError_t launch_weights_simt(int dtype, const void* q_abs, const float* lse, const void* lat, const void* rop,
                                const int* page_table, const int* seq_lens, const float* w_in, float* w_out, int* err,
                                const WeightArgs& a, int sms, cudaStream_t st);

struct EvictArgs {
  int B, maxp, num_pages, recent;
  int lat_bytes, rope_bytes;  // of one token's row
};
struct EvictWorkspace {
  int* owners;  // [num_pages] how many page-table entries name the page
  int* counts;  // [B] tokens to move
  int* src;     // [B][maxp * 32] slots they leave, ascending
  int* dst;     // [B][maxp * 32] slots they go to, ascending
};
cudaError_t launch_evict(const int* evict_pages, const float* weights, const int* page_table, const int* seq_lens,
                         void* lat, void* rop, float* weights_out, int* page_table_out, int* seq_lens_out, int* err,
                         const EvictWorkspace& ws, const EvictArgs& a, int sms, cudaStream_t st);

struct PromptArgs {
  int B, H, kv_heads, d_h, d_r, d_v, maxp, num_pages, total_q, total_k;
  float scale_log2;
  long long q_nope_s[2], q_rope_s[2], k_nope_s[2], v_s[2];
};

// One packed sequence, checked: a sequence whose offsets are out of range, or
// whose keys the page table cannot hold, is reported and has no rows.
struct PromptSeq {
  int q0, k0, Lq, Lk;
};
__device__ __forceinline__ PromptSeq prompt_seq(const int* cu_q, const int* cu_k, int b, const PromptArgs& a,
                                                int* err) {
  const int q0 = __ldg(cu_q + b), q1 = __ldg(cu_q + b + 1), k0 = __ldg(cu_k + b), k1 = __ldg(cu_k + b + 1);
  const bool ok = 0 <= q0 && q0 <= q1 && q1 <= a.total_q && 0 <= k0 && k0 <= k1 && k1 <= a.total_k &&
                  (long long)(k1 - k0) <= (long long)a.maxp * kPage;
  if (!ok) {
    report_error(err, kErrDeviceCheck, b, k1);
    return PromptSeq{0, 0, 0, 0};
  }
  return PromptSeq{q0, k0, q1 - q0, k1 - k0};
}

bool prompt_tc_supported(int dtype, int d_h, int d_r, int d_v);
// Registers of a thread of the kernel as it was compiled, and the number that it needs (see prompt_path.h).
cudaError_t prompt_tc_registers(int* regs, int* want);
size_t prompt_tc_workspace(const PromptArgs& a);
cudaError_t launch_prompt_tc(const void* q_nope, const void* q_rope, const int* cu_q, const void* k_nope,
                             const void* v, const int* cu_k, const void* rope_cache, const int* page_table, void* out,
                             float* lse, void* workspace, const PromptArgs& a, const RopeTable& tab, int sms,
                             cudaStream_t st);
cudaError_t launch_prompt_simt(int dtype, const void* q_nope, const void* q_rope, const int* cu_q, const void* k_nope,
                               const void* v, const int* cu_k, const void* rope_cache, const int* page_table,
                               void* out, float* lse, int* err, const PromptArgs& a, const RopeTable& tab,
                               cudaStream_t st);

}  // namespace mlra
