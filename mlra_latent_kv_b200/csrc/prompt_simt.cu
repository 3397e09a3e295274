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
// pieces (five for 16 multiplications), which is what bounds it.  Four groups
// of eight warps share a CTA's keys, each with its own running maximum, sum and
// values, joined at the end (where shared memory holds four key tiles): a step
// is a chain of loads, products and barriers, and few rows have nothing else to
// hide it behind (8 heads x 256 tokens: 21 us in a graph, 31 with one group).
// Four groups leave a thread 64 registers, of which 48 bytes are spilled.
// 8 heads x 4096 tokens of the tiny widths, fp32: 1076 us.
#include "host_cache.h"
#include "serving.h"

namespace mlra {
namespace {

constexpr int kPq = 32;       // queries of a CTA
constexpr int kPk = 32;       // keys of a step
constexpr int kPSmem = 226 * 1024;  // dynamic shared memory of a CTA, beside the static
constexpr int kPThreads = 8 * kPq;  // of a group

// Row length in floats of a tile in shared memory: a multiple of four, and an odd number of 16-byte pieces, so that
// the same piece of eight rows lies in different banks.
__host__ __device__ constexpr int padded(int d) { return ((d + 3) / 4 | 1) * 4; }

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// floats of shared memory that a group has for itself
__host__ __device__ constexpr int group_floats(int dp, int vp) { return kPk * (dp + vp) + kPq * (kPk + 4); }

// kV: 16-byte pieces of the value dims that a thread keeps (its eighth of at most 32 kV dims); kG: groups
template <typename T, int kV, int kG>
__global__ void __launch_bounds__(kPThreads * kG)
    prompt_simt_kernel(const T* __restrict__ q_nope, const T* __restrict__ q_rope, const int* __restrict__ cu_q,
                       const T* __restrict__ k_nope, const T* __restrict__ v, const int* __restrict__ cu_k,
                       const T* __restrict__ rope_cache, const int* __restrict__ page_table, T* __restrict__ out,
                       float* __restrict__ lse, int* __restrict__ err, PromptArgs a, RopeTable tab) {
  extern __shared__ __align__(16) float sm[];
  const int d = a.d_h + a.d_r, dp = padded(d), vp = padded(a.d_v);
  float* sq = sm;             // [kPq][dp]
  const int group = threadIdx.x / kPThreads, tid = threadIdx.x % kPThreads;
  float* sk = sq + kPq * dp + group * group_floats(dp, vp);  // [kPk][dp]
  float* sv = sk + kPk * dp;                                 // [kPk][vp], at the end the group's values
  float* sp = sv + kPk * vp;                                 // [kPq][kPk + 1], at the end its maxima and sums
  auto group_sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(kPThreads) : "memory"); };
  __shared__ int s_b, s_tile;
  // Tile blockIdx.x of the batch: the tiles of the sequences one after another.  The grid has room for sequences that
  // do not overlap; overlapping ones have a descending pair of offsets between them, which the last CTA walks past
  // and reports.
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
  const int r = tid / 8, part = tid % 8;
  const int i = i0 + r;  // this thread's query; its row of every tile, too

  if (group == 0) {
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
    for (int c = d + part; c < dp; c += 8) sq[r * dp + c] = 0.f;
  }
  for (int c = d + part; c < dp; c += 8) sk[r * dp + c] = 0.f;
  for (int c = a.d_v + part; c < vp; c += 8) sv[r * vp + c] = 0.f;
  __syncthreads();

  float4 acc[kV];
#pragma unroll
  for (int c = 0; c < kV; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  const int keys = min(s.Lk, max(0, off + min(i0 + kPq, s.Lq)));  // up to the last query's own
  for (int j0 = group * kPk; j0 < keys; j0 += kG * kPk) {
    group_sync();
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
    group_sync();
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
    // up to the query's own key: a later token's value may be a NaN or an infinity, which p = 0 would not hide
    const int own = min(kPk, off + i + 1 - j0);
#pragma unroll 4
    for (int j = 0; j < own; ++j) {  // keys past the last have p = 0 and values of 0
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
  if (kG > 1) {  // the groups' results against the largest of their maxima
    if (group > 0) {
      group_sync();  // its tiles have been read
#pragma unroll
      for (int c = 0; c < kV; ++c)
        if (4 * (part + 8 * c) < a.d_v) *reinterpret_cast<float4*>(sv + r * vp + 4 * (part + 8 * c)) = acc[c];
      if (part == 0) {
        sp[r * (kPk + 1)] = m;
        sp[r * (kPk + 1) + 1] = l;
      }
    }
    __syncthreads();
    if (group > 0) return;
    for (int g2 = 1; g2 < kG; ++g2) {
      const float* v2 = sv + g2 * group_floats(dp, vp);
      const float* p2 = sp + g2 * group_floats(dp, vp) + r * (kPk + 1);
      const float top = fmaxf(m, p2[0]), ref = top == -INFINITY ? 0.f : top;
      const float c1 = exp2f(m - ref), c2 = exp2f(p2[0] - ref);
      m = top;
      l = l * c1 + p2[1] * c2;
#pragma unroll
      for (int c = 0; c < kV; ++c)
        if (4 * (part + 8 * c) < a.d_v) {
          const float4 y = ld4(v2 + r * vp + 4 * (part + 8 * c));
          acc[c] = make_float4(acc[c].x * c1 + y.x * c2, acc[c].y * c1 + y.y * c2, acc[c].z * c1 + y.z * c2,
                               acc[c].w * c1 + y.w * c2);
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

template <typename T, int kV, int kG>
cudaError_t launch_as(const void* q_nope, const void* q_rope, const int* cu_q, const void* k_nope, const void* v,
                      const int* cu_k, const void* rope_cache, const int* page_table, void* out, float* lse, int* err,
                      const PromptArgs& a, const RopeTable& tab, cudaStream_t st) {
  const int dp = padded(a.d_h + a.d_r), smem = (kPq * dp + kG * group_floats(dp, padded(a.d_v))) * 4;
  if (kG > 1 && smem > kPSmem)
    return launch_as<T, kV, 1>(q_nope, q_rope, cu_q, k_nope, v, cu_k, rope_cache, page_table, out, lse, err, a, tab,
                               st);
  auto kern = prompt_simt_kernel<T, kV, kG>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(((long long)a.total_q + kPq - 1) / kPq + a.B), a.H);  // at most that many tiles
  kern<<<grid, kPThreads * kG, smem, st>>>(static_cast<const T*>(q_nope), static_cast<const T*>(q_rope), cu_q,
                                           static_cast<const T*>(k_nope), static_cast<const T*>(v), cu_k,
                                           static_cast<const T*>(rope_cache), page_table, static_cast<T*>(out), lse,
                                           err, a, tab);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const void* q_nope, const void* q_rope, const int* cu_q, const void* k_nope, const void* v,
                   const int* cu_k, const void* rope_cache, const int* page_table, void* out, float* lse, int* err,
                   const PromptArgs& a, const RopeTable& tab, cudaStream_t st) {
  auto run = [&](auto f) {
    return f(q_nope, q_rope, cu_q, k_nope, v, cu_k, rope_cache, page_table, out, lse, err, a, tab, st);
  };
  if (a.d_v <= 32) return run(launch_as<T, 1, 4>);
  if (a.d_v <= 128) return run(launch_as<T, 4, 4>);
  return run(launch_as<T, 16, 1>);  // d_v <= 512
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
