// Prompt attention on CUDA cores: every type and width the dims allow, any
// strides.  The path of fp32 and of widths the tcgen05 kernel does not take.
//
//   x[i,j] = scale * (q_nope_i . k_nope_j + RoPE(q_rope_i) . k_j),  j <= Lk - Lq + i
//   out_i  = softmax_j(x) v                      (yololab.net, "超越 GQA 的推理
//   革命…", sections "1. 鍵值聯合低秩壓縮" and "2. 解耦旋轉位置編碼")
//
// A CTA takes 32 queries of one head and passes once over their keys, 32 at a
// time, with the running maximum and sum of the softmax in fp32.  Eight
// threads share a query: each takes four of the 32 keys and an eighth of the
// value dims, which stay in its registers.  Both products read shared memory
// about once per multiplication, which is what bounds it.
#include "host_cache.h"
#include "serving.h"

namespace mlra {
namespace {

constexpr int kPq = 32;       // queries of a CTA
constexpr int kPk = 32;       // keys of a step
constexpr int kPThreads = 8 * kPq;
constexpr int kPDv = 64;      // value dims of a thread: d_v <= 512

template <typename T>
__global__ void __launch_bounds__(kPThreads)
    prompt_simt_kernel(const T* __restrict__ q_nope, const T* __restrict__ q_rope, const int* __restrict__ cu_q,
                       const T* __restrict__ k_nope, const T* __restrict__ v, const int* __restrict__ cu_k,
                       const T* __restrict__ rope_cache, const int* __restrict__ page_table, T* __restrict__ out,
                       float* __restrict__ lse, int* __restrict__ err, PromptArgs a, RopeTable tab) {
  extern __shared__ float sm[];
  const int d = a.d_h + a.d_r, dp = d + 1;  // the pad keeps the eight keys of a query's threads in different banks
  float* sq = sm;                           // [kPq][dp]
  float* sk = sq + kPq * dp;                // [kPk][dp]
  float* sv = sk + kPk * dp;                // [kPk][d_v]
  float* sp = sv + kPk * a.d_v;             // [kPq][kPk + 1]
  __shared__ int s_b, s_tile;
  // tile blockIdx.x of the batch: the tiles of the sequences one after another
  if (threadIdx.x == 0) {
    int t = blockIdx.x, b = 0;
    for (; b < a.B; ++b) {
      const PromptSeq s = prompt_seq(cu_q, cu_k, b, a, blockIdx.y == 0 ? err : nullptr);
      const int n = (s.Lq + kPq - 1) / kPq;
      if (t < n) break;
      t -= n;
    }
    s_b = b;
    s_tile = t;
  }
  __syncthreads();
  const int b = s_b;
  if (b >= a.B) return;
  const PromptSeq s = prompt_seq(cu_q, cu_k, b, a, nullptr);
  const int h = blockIdx.y, g = h / (a.H / a.kv_heads);
  const int i0 = s_tile * kPq, off = s.Lk - s.Lq;
  const int r = threadIdx.x / 8, part = threadIdx.x % 8;
  const int i = i0 + r;  // this thread's query

  for (int e = threadIdx.x; e < kPq * a.d_h; e += kPThreads) {
    const int q = e / a.d_h, c = e % a.d_h;
    sq[q * dp + c] = i0 + q < s.Lq ? to_f(q_nope[(size_t)(s.q0 + i0 + q) * a.q_nope_s[0] + h * a.q_nope_s[1] + c])
                                   : 0.f;
  }
  for (int e = threadIdx.x; e < kPq * (a.d_r / 2); e += kPThreads) {
    const int q = e / (a.d_r / 2), p = e % (a.d_r / 2);
    float x0 = 0.f, x1 = 0.f, sn, cs;
    if (i0 + q < s.Lq) {
      const T* x = q_rope + (size_t)(s.q0 + i0 + q) * a.q_rope_s[0] + h * a.q_rope_s[1] + 2 * p;
      x0 = to_f(x[0]);
      x1 = to_f(x[1]);
    }
    rope_sincos(tab, p, off + i0 + q, &sn, &cs);
    sq[q * dp + a.d_h + 2 * p] = x0 * cs - x1 * sn;
    sq[q * dp + a.d_h + 2 * p + 1] = x0 * sn + x1 * cs;
  }

  float acc[kPDv];
#pragma unroll
  for (int c = 0; c < kPDv; ++c) acc[c] = 0.f;
  float m = -INFINITY, l = 0.f;
  const int keys = min(s.Lk, max(0, off + min(i0 + kPq, s.Lq)));  // up to the last query's own
  for (int j0 = 0; j0 < keys; j0 += kPk) {
    __syncthreads();
    for (int e = threadIdx.x; e < kPk * a.d_h; e += kPThreads) {
      const int j = e / a.d_h, c = e % a.d_h;
      sk[j * dp + c] = j0 + j < keys ? to_f(k_nope[(size_t)(s.k0 + j0 + j) * a.k_nope_s[0] + g * a.k_nope_s[1] + c])
                                     : 0.f;
    }
    for (int e = threadIdx.x; e < kPk * a.d_r; e += kPThreads) {
      const int j = e / a.d_r, c = e % a.d_r;
      float x = 0.f;
      if (j0 + j < keys) {
        const int pg = page_of(page_table, a.maxp, a.num_pages, b, j0 + j, err);
        x = to_f(rope_cache[((size_t)pg * kPage + (j0 + j) % kPage) * a.d_r + c]);
      }
      sk[j * dp + a.d_h + c] = x;
    }
    for (int e = threadIdx.x; e < kPk * a.d_v; e += kPThreads) {
      const int j = e / a.d_v, c = e % a.d_v;
      sv[e] = j0 + j < keys ? to_f(v[(size_t)(s.k0 + j0 + j) * a.v_s[0] + g * a.v_s[1] + c]) : 0.f;
    }
    __syncthreads();
    float x[kPk / 8], top = -INFINITY;
#pragma unroll
    for (int n = 0; n < kPk / 8; ++n) {
      const int j = part + 8 * n;
      float dot = 0.f;
      for (int c = 0; c < d; ++c) dot = fmaf(sq[r * dp + c], sk[j * dp + c], dot);
      x[n] = j0 + j <= off + i && j0 + j < keys ? dot * a.scale_log2 : -INFINITY;
      top = fmaxf(top, x[n]);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float m_new = fmaxf(m, top);
    const float ref = m_new == -INFINITY ? 0.f : m_new;  // a row without keys so far: all terms are 2^-inf = 0
    const float corr = exp2f(m - ref);
    float sum = 0.f;
#pragma unroll
    for (int n = 0; n < kPk / 8; ++n) {
      const float p = exp2f(x[n] - ref);
      sp[r * (kPk + 1) + part + 8 * n] = p;
      sum += p;
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    m = m_new;
    l = l * corr + sum;
    __syncwarp();  // a query's eight threads are in one warp
#pragma unroll
    for (int c = 0; c < kPDv; ++c) acc[c] *= corr;
    for (int j = 0; j < min(kPk, keys - j0); ++j) {
      const float p = sp[r * (kPk + 1) + j];
#pragma unroll
      for (int c = 0; c < kPDv; ++c)
        if (part + 8 * c < a.d_v) acc[c] = fmaf(p, sv[j * a.d_v + part + 8 * c], acc[c]);
    }
  }
  if (i >= s.Lq) return;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  T* o = out + ((size_t)(s.q0 + i) * a.H + h) * a.d_v;
#pragma unroll
  for (int c = 0; c < kPDv; ++c)
    if (part + 8 * c < a.d_v) o[part + 8 * c] = from_f<T>(l == 0.f ? 0.f : acc[c] * inv);
  if (lse && part == 0) lse[(size_t)(s.q0 + i) * a.H + h] = l == 0.f ? -INFINITY : m + log2f(l);
}

template <typename T>
cudaError_t launch(const void* q_nope, const void* q_rope, const int* cu_q, const void* k_nope, const void* v,
                   const int* cu_k, const void* rope_cache, const int* page_table, void* out, float* lse, int* err,
                   const PromptArgs& a, const RopeTable& tab, cudaStream_t st) {
  const int d = a.d_h + a.d_r;
  const int smem = ((kPq + kPk) * (d + 1) + kPk * a.d_v + kPq * (kPk + 1)) * 4;
  auto kern = prompt_simt_kernel<T>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(((long long)a.total_q + kPq - 1) / kPq + a.B), a.H);  // at most that many tiles
  kern<<<grid, kPThreads, smem, st>>>(static_cast<const T*>(q_nope), static_cast<const T*>(q_rope), cu_q,
                                      static_cast<const T*>(k_nope), static_cast<const T*>(v), cu_k,
                                      static_cast<const T*>(rope_cache), page_table, static_cast<T*>(out), lse, err,
                                      a, tab);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_simt(int dtype, const void* q_nope, const void* q_rope, const int* cu_q, const void* k_nope,
                               const void* v, const int* cu_k, const void* rope_cache, const int* page_table,
                               void* out, float* lse, int* err, const PromptArgs& a, const RopeTable& tab,
                               cudaStream_t st) {
  return (dtype == MLRA_F32 ? launch<float> : launch<__nv_bfloat16>)(q_nope, q_rope, cu_q, k_nope, v, cu_k, rope_cache,
                                                                     page_table, out, lse, err, a, tab, st);
}

}  // namespace mlra
