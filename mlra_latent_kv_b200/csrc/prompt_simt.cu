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
// value dims, which stay in its registers, and reads shared memory in 16-byte
// pieces (five for 16 multiplications), which is what bounds it.
#include "host_cache.h"
#include "serving.h"

namespace mlra {
namespace {

constexpr int kPq = 32;       // queries of a CTA
constexpr int kPk = 32;       // keys of a step
constexpr int kPThreads = 8 * kPq;

// Row length in floats of a tile in shared memory: a multiple of four, and an odd number of 16-byte pieces, so that
// the same piece of eight rows lies in different banks.
__host__ __device__ constexpr int padded(int d) { return ((d + 3) / 4 | 1) * 4; }

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// kV: 16-byte pieces of the value dims that a thread keeps (its eighth of at most 32 kV dims)
template <typename T, int kV>
__global__ void __launch_bounds__(kPThreads)
    prompt_simt_kernel(const T* __restrict__ q_nope, const T* __restrict__ q_rope, const int* __restrict__ cu_q,
                       const T* __restrict__ k_nope, const T* __restrict__ v, const int* __restrict__ cu_k,
                       const T* __restrict__ rope_cache, const int* __restrict__ page_table, T* __restrict__ out,
                       float* __restrict__ lse, int* __restrict__ err, PromptArgs a, RopeTable tab) {
  extern __shared__ __align__(16) float sm[];
  const int d = a.d_h + a.d_r, dp = padded(d), vp = padded(a.d_v);
  float* sq = sm;             // [kPq][dp]
  float* sk = sq + kPq * dp;  // [kPk][dp]
  float* sv = sk + kPk * dp;  // [kPk][vp]
  float* sp = sv + kPk * vp;  // [kPq][kPk + 1]
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
    // the grid has a tile more than sequences that do not overlap can have
    if (blockIdx.x == gridDim.x - 1 && b < a.B) {
      report_error(err, kErrDeviceCheck, a.B, a.total_q);
      b = a.B;
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
  const int i = i0 + r;  // this thread's query; its row of every tile, too

  {
    const T* x = q_nope + (size_t)(s.q0 + i) * a.q_nope_s[0] + h * a.q_nope_s[1];
    for (int c = part; c < a.d_h; c += 8) sq[r * dp + c] = i < s.Lq ? to_f(x[c]) : 0.f;
    const T* y = q_rope + (size_t)(s.q0 + i) * a.q_rope_s[0] + h * a.q_rope_s[1];
    for (int p = part; p < a.d_r / 2; p += 8) {
      float x0 = 0.f, x1 = 0.f, sn, cs;
      if (i < s.Lq) {
        x0 = to_f(y[2 * p]);
        x1 = to_f(y[2 * p + 1]);
      }
      rope_sincos(tab, p, off + i, &sn, &cs);
      sq[r * dp + a.d_h + 2 * p] = x0 * cs - x1 * sn;
      sq[r * dp + a.d_h + 2 * p + 1] = x0 * sn + x1 * cs;
    }
    for (int c = d + part; c < dp; c += 8) sq[r * dp + c] = sk[r * dp + c] = 0.f;
    for (int c = a.d_v + part; c < vp; c += 8) sv[r * vp + c] = 0.f;
  }

  float4 acc[kV];
#pragma unroll
  for (int c = 0; c < kV; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  const int keys = min(s.Lk, max(0, off + min(i0 + kPq, s.Lq)));  // up to the last query's own
  for (int j0 = 0; j0 < keys; j0 += kPk) {
    __syncthreads();
    {
      const int j = j0 + r;
      const bool in = j < keys;
      const T* x = k_nope + (size_t)(s.k0 + j) * a.k_nope_s[0] + g * a.k_nope_s[1];
      const T* y = v + (size_t)(s.k0 + j) * a.v_s[0] + g * a.v_s[1];
      const int pg = in ? page_of(page_table, a.maxp, a.num_pages, b, j, err) : 0;
      const T* z = rope_cache + ((size_t)pg * kPage + j % kPage) * a.d_r;
#pragma unroll 4
      for (int c = part; c < a.d_h; c += 8) sk[r * dp + c] = in ? to_f(x[c]) : 0.f;
#pragma unroll 4
      for (int c = part; c < a.d_v; c += 8) sv[r * vp + c] = in ? to_f(y[c]) : 0.f;
#pragma unroll 4
      for (int c = part; c < a.d_r; c += 8) sk[r * dp + a.d_h + c] = in ? to_f(z[c]) : 0.f;
    }
    __syncthreads();
    float x[kPk / 8], top = -INFINITY;
#pragma unroll
    for (int n = 0; n < kPk / 8; ++n) x[n] = 0.f;
    for (int c = 0; c < d; c += 4) {
      const float4 q = ld4(sq + r * dp + c);
#pragma unroll
      for (int n = 0; n < kPk / 8; ++n) {
        const float4 k = ld4(sk + (part + 8 * n) * dp + c);
        x[n] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, x[n]))));
      }
    }
#pragma unroll
    for (int n = 0; n < kPk / 8; ++n) {
      const int j = j0 + part + 8 * n;
      x[n] = j <= off + i && j < keys ? x[n] * a.scale_log2 : -INFINITY;
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
    for (int c = 0; c < kV; ++c) {
      acc[c].x *= corr;
      acc[c].y *= corr;
      acc[c].z *= corr;
      acc[c].w *= corr;
    }
#pragma unroll 4
    for (int j = 0; j < kPk; ++j) {  // keys past the last have p = 0 and values of 0
      const float p = sp[r * (kPk + 1) + j];
#pragma unroll
      for (int c = 0; c < kV; ++c)
        if (4 * (part + 8 * c) < a.d_v) {
          const float4 y = ld4(sv + j * vp + 4 * (part + 8 * c));
          acc[c].x = fmaf(p, y.x, acc[c].x);
          acc[c].y = fmaf(p, y.y, acc[c].y);
          acc[c].z = fmaf(p, y.z, acc[c].z);
          acc[c].w = fmaf(p, y.w, acc[c].w);
        }
    }
  }
  if (i >= s.Lq) return;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  T* o = out + ((size_t)(s.q0 + i) * a.H + h) * a.d_v;
#pragma unroll
  for (int c = 0; c < kV; ++c) {
    const float y[4] = {acc[c].x, acc[c].y, acc[c].z, acc[c].w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int col = 4 * (part + 8 * c) + u;
      if (col < a.d_v) o[col] = from_f<T>(l == 0.f ? 0.f : y[u] * inv);
    }
  }
  if (lse && part == 0) lse[(size_t)(s.q0 + i) * a.H + h] = l == 0.f ? -INFINITY : m + log2f(l);
}

template <typename T, int kV>
cudaError_t launch(const void* q_nope, const void* q_rope, const int* cu_q, const void* k_nope, const void* v,
                   const int* cu_k, const void* rope_cache, const int* page_table, void* out, float* lse, int* err,
                   const PromptArgs& a, const RopeTable& tab, cudaStream_t st) {
  const int smem = ((kPq + kPk) * padded(a.d_h + a.d_r) + kPk * padded(a.d_v) + kPq * (kPk + 1)) * 4;
  auto kern = prompt_simt_kernel<T, kV>;
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
  auto run = [&](auto f) {
    return f(q_nope, q_rope, cu_q, k_nope, v, cu_k, rope_cache, page_table, out, lse, err, a, tab, st);
  };
  const bool f32 = dtype == MLRA_F32;
  if (a.d_v <= 32) return run(f32 ? launch<float, 1> : launch<__nv_bfloat16, 1>);
  if (a.d_v <= 128) return run(f32 ? launch<float, 4> : launch<__nv_bfloat16, 4>);
  return run(f32 ? launch<float, 16> : launch<__nv_bfloat16, 16>);  // d_v <= 512
}

}  // namespace mlra
