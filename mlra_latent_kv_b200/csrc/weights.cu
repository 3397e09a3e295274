// Attention weight of every cached token, summed over heads and branches and
// added to what the token has gathered so far (what an eviction goes by):
//   w[b, t] += sum_{br, h} 2^(q_br[b, h] . c_br[b, t] + q_rot[b, h] . k[b, t] - lse[b, br, h])
// q is the absorbed query, which carries softmax_scale * log2(e) (yololab.net,
// "超越 GQA 的推理革命…", section "矩陣吸收"), so the exponent is a base-2 logit
// minus the log-sum-exp of all of them; branches as in wispaper.ai, "MLRA：突破
// MLA 并行瓶颈…", section "2.1 架构拆解".
//
// Each token belongs to one CTA, its heads are added in a fixed order: no
// atomics, the same bits every time.
#include "host_cache.h"
#include "ptx.cuh"
#include "serving.h"

namespace mlra {
namespace {

using namespace ptx;

// ---------------------------------------------------------------------------
// CUDA cores: every type and shape the dims allow.
//
// A CTA walks its share of the pages (the split plan of the decode kernels);
// its eight warps take a page's tokens in fours, with a token's dims spread
// over the lanes (dim l + 32 k in lane l).  Per head: multiply, add the lanes
// up per branch, exponentiate.  fp32 throughout.  Made for the fp32 cache of
// the tiny configuration and for odd widths: reading each query from shared
// memory once per four tokens is what bounds it.
// ---------------------------------------------------------------------------
constexpr int kWTok = 4;     // tokens a warp takes together
constexpr int kWHeads = 8;   // heads staged in shared memory at a time
constexpr int kWDpl = 16;    // d_c <= 512
constexpr int kWRpl = 2;     // d_r <= 64

template <typename T>
__global__ void __launch_bounds__(256) weights_simt_kernel(const T* __restrict__ q_abs, const float* __restrict__ lse,
                                                           const T* __restrict__ lat, const T* __restrict__ rop,
                                                           const int* __restrict__ page_table,
                                                           const int* __restrict__ seq_lens,
                                                           const float* w_in, float* w_out,
                                                           int* __restrict__ err, WeightArgs a) {
  __shared__ float qs[kWHeads][32 * (kWDpl + kWRpl)];
  __shared__ float ls[kWHeads * 8];
  __shared__ WorkerPlan s_plan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int maxL = a.maxp * kPage, D = a.d_c + a.d_r;
  const int nk = a.d_c / 32, kb = nk / a.n_branch;  // 32-dim steps of the latent, and of one branch
  if (blockIdx.x == 0) check_lengths(seq_lens, a.B, maxL, err);
  if (warp == 0) {
    const WorkerPlan p = plan_worker(seq_lens, a.B, gridDim.x, blockIdx.x, maxL);
    if (lane == 0) s_plan = p;
  }
  __syncthreads();
  SegWalk walk(s_plan, a.B, maxL);
  while (walk.next(seq_lens)) {
    for (int p = walk.pg0; p < walk.pg1; ++p) {
      const int t0 = p * kPage;
      const int pg = page_of(page_table, a.maxp, a.num_pages, walk.b, t0, err);
      for (int r0 = warp * 8; r0 < warp * 8 + 8; r0 += kWTok) {  // this warp's rows of the page
        float c[kWTok][kWDpl], k[kWTok][kWRpl], sum[kWTok];
#pragma unroll
        for (int i = 0; i < kWTok; ++i) {
          const bool in = t0 + r0 + i < walk.L;
          const T* crow = lat + ((size_t)pg * kPage + r0 + i) * a.d_c;
          const T* krow = rop + ((size_t)pg * kPage + r0 + i) * a.d_r;
#pragma unroll
          for (int j = 0; j < kWDpl; ++j) c[i][j] = in && j < nk ? to_f(crow[lane + 32 * j]) : 0.f;
#pragma unroll
          for (int j = 0; j < kWRpl; ++j) k[i][j] = in && lane + 32 * j < a.d_r ? to_f(krow[lane + 32 * j]) : 0.f;
          sum[i] = 0.f;
        }
        for (int h0 = 0; h0 < a.H; h0 += kWHeads) {
          const int nh = min(kWHeads, a.H - h0);
          __syncthreads();
          for (int e = threadIdx.x; e < nh * D; e += blockDim.x)
            qs[e / D][e % D] = to_f(q_abs[((size_t)walk.b * a.H + h0) * D + e]);
          for (int e = threadIdx.x; e < nh * a.n_branch; e += blockDim.x) {
            const float v = __ldg(lse + ((size_t)walk.b * a.n_branch + e / nh) * a.H + h0 + e % nh);
            ls[e] = v == -INFINITY ? INFINITY : v;  // attended nothing: adds nothing
          }
          __syncthreads();
          for (int h = 0; h < nh; ++h) {
            float rs[kWTok];
#pragma unroll
            for (int i = 0; i < kWTok; ++i) {
              rs[i] = 0.f;
#pragma unroll
              for (int j = 0; j < kWRpl; ++j)
                if (lane + 32 * j < a.d_r) rs[i] = fmaf(qs[h][a.d_c + lane + 32 * j], k[i][j], rs[i]);
            }
            for (int br = 0; br < a.n_branch; ++br) {
              float s[kWTok];
#pragma unroll
              for (int i = 0; i < kWTok; ++i) s[i] = rs[i];
#pragma unroll
              for (int j = 0; j < kWDpl; ++j) {
                if (j / kb == br && j < nk) {
                  const float q = qs[h][lane + 32 * j];
#pragma unroll
                  for (int i = 0; i < kWTok; ++i) s[i] = fmaf(q, c[i][j], s[i]);
                }
              }
#pragma unroll
              for (int i = 0; i < kWTok; ++i) sum[i] += exp2f(warp_sum(s[i]) - ls[br * nh + h]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kWTok; ++i) {
          const int t = t0 + r0 + i;
          if (lane == i && t < walk.L) {
            const size_t at = (size_t)walk.b * maxL + t;
            w_out[at] = (w_in ? w_in[at] : 0.f) + sum[i];
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_weights_simt(int dtype, const void* q_abs, const float* lse, const void* lat, const void* rop,
                                const int* page_table, const int* seq_lens, const float* w_in, float* w_out, int* err,
                                const WeightArgs& a, int sms, cudaStream_t st) {
  const dim3 grid(2 * sms);
  if (dtype == MLRA_F32)
    weights_simt_kernel<float><<<grid, 256, 0, st>>>(static_cast<const float*>(q_abs), lse,
                                                      static_cast<const float*>(lat), static_cast<const float*>(rop),
                                                      page_table, seq_lens, w_in, w_out, err, a);
  else
    weights_simt_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(
        static_cast<const __nv_bfloat16*>(q_abs), lse, static_cast<const __nv_bfloat16*>(lat),
        static_cast<const __nv_bfloat16*>(rop), page_table, seq_lens, w_in, w_out, err, a);
  return cudaGetLastError();
}

}  // namespace mlra
