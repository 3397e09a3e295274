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
// The split plan of the decode kernels shares the pages; kSub CTAs share each
// page, and the eight warps of a CTA take kTok tokens each, a token's dims
// spread over the lanes (dim l + 32 k in lane l).  Eight heads at a time: the
// lanes' partial scores are added up and dealt out in one butterfly, after
// which a lane holds the score of one (token, head) pair and exponentiates it
// (16 shuffles for 16 scores, 31 for 32, and no exponential twice).  fp32
// throughout.  Made for the fp32 cache of the tiny configuration and for odd
// widths: reading each query from shared memory once per kTok tokens is what
// bounds it.
// ---------------------------------------------------------------------------
constexpr int kWHeads = 8;   // heads staged in shared memory at a time
constexpr int kWRpl = 2;     // d_r <= 64
constexpr int kWDims = 512;  // d_c at most

// The sums of v[0 .. N-1] over the warp, one per lane: of index lane * N / 32.
template <int N>
__device__ __forceinline__ float warp_deal_sum(float (&v)[N], int lane) {
  int o = 16;
#pragma unroll
  for (int n = N / 2; n >= 1; n >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float keep = up ? v[k + n] : v[k], give = up ? v[k] : v[k + n];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  for (; o >= 1; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

// kDpl: 32-dim steps of the latent at most
template <typename T, int kDpl, int kSub>
__global__ void __launch_bounds__(256) weights_simt_kernel(const T* __restrict__ q_abs, const float* __restrict__ lse,
                                                           const T* __restrict__ lat, const T* __restrict__ rop,
                                                           const int* __restrict__ page_table,
                                                           const int* __restrict__ seq_lens,
                                                           const float* w_in, float* w_out,
                                                           int* __restrict__ err, WeightArgs a) {
  constexpr int kTok = kSub == 1 ? 4 : 2, kRows = kPage / kSub;  // rows of a page that are this CTA's
  constexpr int kN = kTok * kWHeads;
  __shared__ float qs[kWHeads * (kWDims + 32 * kWRpl)];
  __shared__ float ls[kWHeads * 8];
  __shared__ WorkerPlan s_plan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int maxL = a.maxp * kPage, D = a.d_c + a.d_r;
  const int kb = a.d_c / 32 / a.n_branch;  // 32-dim steps of a branch
  const int mine = lane * kN / 32, my_tok = mine / kWHeads, my_head = mine % kWHeads;
  if (blockIdx.x == 0) check_lengths(seq_lens, a.B, maxL, err);
  if (warp == 0) {
    const WorkerPlan p = plan_worker(seq_lens, a.B, gridDim.x / kSub, blockIdx.x / kSub, maxL);
    if (lane == 0) s_plan = p;
  }
  __syncthreads();
  SegWalk walk(s_plan, a.B, maxL);
  while (walk.next(seq_lens)) {
    for (int p = walk.pg0; p < walk.pg1; ++p) {
      const int pg = page_of(page_table, a.maxp, a.num_pages, walk.b, p * kPage, err);
      for (int r0 = blockIdx.x % kSub * kRows; r0 < (blockIdx.x % kSub + 1) * kRows; r0 += 8 * kTok) {
        const int row = r0 + warp * kTok, t0 = p * kPage + row;  // this warp's tokens
        float c[kTok][kDpl], k[kTok][kWRpl], sum = 0.f;
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
          const bool in = t0 + i < walk.L;
          const T* crow = lat + ((size_t)pg * kPage + row + i) * a.d_c;
          const T* krow = rop + ((size_t)pg * kPage + row + i) * a.d_r;
#pragma unroll
          for (int j = 0; j < kDpl; ++j) c[i][j] = in && 32 * j < a.d_c ? to_f(crow[lane + 32 * j]) : 0.f;
#pragma unroll
          for (int j = 0; j < kWRpl; ++j) k[i][j] = in && lane + 32 * j < a.d_r ? to_f(krow[lane + 32 * j]) : 0.f;
        }
        const size_t at = (size_t)walk.b * maxL + t0 + my_tok;
        const bool writes = my_head == 0 && (kN == 32 || lane % 2 == 0) && t0 + my_tok < walk.L;
        const float before = writes && w_in ? w_in[at] : 0.f;
        for (int h0 = 0; h0 < a.H; h0 += kWHeads) {
          const int nh = min(kWHeads, a.H - h0);
          __syncthreads();
          const T* q = q_abs + ((size_t)walk.b * a.H + h0) * D;
          for (int e = threadIdx.x; e < kWHeads * D; e += blockDim.x) qs[e] = e < nh * D ? to_f(q[e]) : 0.f;
          for (int e = threadIdx.x; e < kWHeads * a.n_branch; e += blockDim.x) {
            const int h = e % kWHeads;
            const float v =
                h < nh ? __ldg(lse + ((size_t)walk.b * a.n_branch + e / kWHeads) * a.H + h0 + h) : INFINITY;
            ls[e] = v == -INFINITY ? INFINITY : v;  // attended nothing: adds nothing
          }
          __syncthreads();
          for (int br = 0; br < a.n_branch; ++br) {
            float s[kN];
#pragma unroll
            for (int e = 0; e < kN; ++e) s[e] = 0.f;
#pragma unroll
            for (int j = 0; j < kDpl; ++j)
              if (j >= br * kb && j < (br + 1) * kb) {
#pragma unroll
                for (int h = 0; h < kWHeads; ++h) {
                  const float x = qs[h * D + lane + 32 * j];
#pragma unroll
                  for (int i = 0; i < kTok; ++i) s[i * kWHeads + h] = fmaf(x, c[i][j], s[i * kWHeads + h]);
                }
              }
#pragma unroll
            for (int j = 0; j < kWRpl; ++j)
              if (lane + 32 * j < a.d_r) {
#pragma unroll
                for (int h = 0; h < kWHeads; ++h) {
                  const float x = qs[h * D + a.d_c + lane + 32 * j];
#pragma unroll
                  for (int i = 0; i < kTok; ++i) s[i * kWHeads + h] = fmaf(x, k[i][j], s[i * kWHeads + h]);
                }
              }
            sum += exp2f(warp_deal_sum(s, lane) - ls[br * kWHeads + my_head]);
          }
        }
        // the heads of this lane's token
#pragma unroll
        for (int o = kN == 32 ? 1 : 2; o < (kN == 32 ? 8 : 16); o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (writes) w_out[at] = before + sum;
      }
    }
  }
}

template <typename T>
cudaError_t launch(const void* q_abs, const float* lse, const void* lat, const void* rop, const int* page_table,
                   const int* seq_lens, const float* w_in, float* w_out, int* err, const WeightArgs& a, int sms,
                   cudaStream_t st) {
  auto run = [&](auto kern, long long grid) {
    kern<<<(unsigned)grid, 256, 0, st>>>(static_cast<const T*>(q_abs), lse, static_cast<const T*>(lat),
                                         static_cast<const T*>(rop), page_table, seq_lens, w_in, w_out, err, a);
    return cudaGetLastError();
  };
  // pages enough for every CTA, or several CTAs to a page
  const long long pages = (long long)a.B * a.maxp;
  if (a.d_c <= 128)
    return pages <= 2 * sms ? run(weights_simt_kernel<T, 4, 4>, 4 * pages)
                            : run(weights_simt_kernel<T, 4, 1>, 2 * sms);
  return pages <= 2 * sms ? run(weights_simt_kernel<T, kWDims / 32, 4>, 4 * pages)
                          : run(weights_simt_kernel<T, kWDims / 32, 1>, 2 * sms);
}

}  // namespace

cudaError_t launch_weights_simt(int dtype, const void* q_abs, const float* lse, const void* lat, const void* rop,
                                const int* page_table, const int* seq_lens, const float* w_in, float* w_out, int* err,
                                const WeightArgs& a, int sms, cudaStream_t st) {
  return (dtype == MLRA_F32 ? launch<float> : launch<__nv_bfloat16>)(q_abs, lse, lat, rop, page_table, seq_lens, w_in,
                                                                     w_out, err, a, sms, st);
}

}  // namespace mlra
