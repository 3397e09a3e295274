// Eviction from the paged latent cache by gathered attention weight: n whole
// pages of a sequence are freed, the 64 n tokens with the least weight leave.
//
// The decode attends a sequence's tokens in any order (each rope key is stored
// rotated at its own position), so nothing is compacted: the first n pages go,
// and only those of their tokens that stay are moved, into the slots that
// tokens leaving the other pages make free.  Sources lie in pages [0, n),
// destinations in pages [n, ..): no slot is both, so all moves run at once and
// in place, and the number of bytes moved is the least that frees those pages.
//
// Two kernels.  evict_select_kernel: a cluster of 8 CTAs per sequence finds
// the 64 n smallest (weight, slot) by a radix select over the weights' bits
// (four 8-bit digits; the CTAs' histograms meet in distributed shared memory)
// and writes both lists, in slot order, beside the shifted weights, table and
// length.  It is bound by latency: a sequence's weights are read from HBM once
// and kept in shared memory.  evict_move_kernel: a warp per token row copies
// the latent and the rope key, 16 bytes a lane, several rows in flight.
#include <cooperative_groups.h>

#include "host_cache.h"
#include "serving.h"

namespace mlra {
namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;        // CTAs per sequence
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kKeyCap = 16384;     // keys a CTA keeps in shared memory (a sequence of 131072 tokens); longer: re-read

// Ascending order of the weights as unsigned integers: -inf and NaN first, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (isnan(w)) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct SelShared {
  int hist[2][256];            // of this CTA, double-buffered over the digits
  int total[256];              // over the cluster
  int ties[kSelWarps];         // equal to the threshold, per warp
  int srcs[kSelWarps];         // tokens to move, per warp
  int holes[kSelWarps];        // slots to move to, per warp
  int digit, below;
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSelThreads)
    evict_select_kernel(const int* __restrict__ evict_pages, const float* __restrict__ weights,
                        const int* __restrict__ page_table, const int* __restrict__ seq_lens,
                        float* __restrict__ weights_out, int* __restrict__ page_table_out,
                        int* __restrict__ seq_lens_out, int* __restrict__ err, EvictWorkspace ws, EvictArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ SelShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int b = blockIdx.x / kCluster, rank = blockIdx.x % kCluster;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slots = a.maxp * kPage;
  const float* w = weights + (size_t)b * slots;

  int L = __ldg(seq_lens + b), n = __ldg(evict_pages + b);
  const bool bad_len = L < 0 || L > slots;
  L = L < 0 ? 0 : min(L, slots);
  const bool bad_n = n < 0 || (n > 0 && (long long)n * kPage > (long long)L - a.recent);
  if (rank == 0 && threadIdx.x == 0 && (bad_len || bad_n)) report_error(err, kErrDeviceCheck, b, bad_len ? L : n);
  if (bad_n) n = 0;
  const int E = n * kPage;                // tokens that leave
  const int C = n > 0 ? L - a.recent : 0;  // tokens that may leave: slots [0, C)

  // this CTA's slots, and within them each warp's
  const int per = (L + kCluster - 1) / kCluster;
  const int lo = min(L, rank * per), hi = min(L, lo + per);
  const bool in_smem = per <= kKeyCap;
  const int wper = ((hi - lo + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int wlo = min(hi, lo + warp * wper), whi = min(hi, wlo + wper);
  auto key_at = [&](int t) { return in_smem ? keys[t - lo] : order_key(__ldg(w + t)); };

  uint32_t T = 0;  // the largest key that leaves
  int spare = 0;   // of the tokens with that key, in slot order, the first `spare` stay
  if (E > 0) {     // uniform over the cluster
    if (in_smem)
      for (int t = lo + threadIdx.x; t < hi; t += kSelThreads) keys[t - lo] = order_key(__ldg(w + t));
    for (int i = threadIdx.x; i < 512; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
    int need = E;  // how many of the keys that share the digits found so far leave
    for (int d = 0; d < 4; ++d) {
      const int shift = 24 - 8 * d;
      const uint32_t mask = d == 0 ? 0u : 0xFFFFFFFFu << (shift + 8);
      int* hist = sh.hist[d & 1];
      for (int t = lo + threadIdx.x; t < min(hi, C); t += kSelThreads) {
        const uint32_t u = key_at(t);
        if ((u & mask) == T) atomicAdd(&hist[(u >> shift) & 255], 1);
      }
      cluster.sync();
      if (threadIdx.x < 256) {
        int s = 0;
#pragma unroll
        for (int r = 0; r < kCluster; ++r) s += cluster.map_shared_rank(hist, r)[threadIdx.x];
        sh.total[threadIdx.x] = s;
        sh.hist[(d + 1) & 1][threadIdx.x] = 0;  // the next digit's (read by the cluster before its last sync)
      }
      __syncthreads();
      if (warp == 0) {  // the digit at which the running count reaches `need`
        int v[8], s = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += (v[i] = sh.total[lane * 8 + i]);
        const int incl = warp_incl_scan(s);
        int before = incl - s;
        if (before < need && need <= incl) {
          int i = 0;
          while (before + v[i] < need) before += v[i++];
          sh.digit = lane * 8 + i;
          sh.below = before;
        }
      }
      __syncthreads();
      T |= (uint32_t)sh.digit << shift;
      need -= sh.below;
      spare = sh.total[sh.digit] - need;
      __syncthreads();  // everyone has them before the next digit's are written
    }

    // ties before each warp, over the cluster: the first `spare` of them stay
    int n_tie = 0;
    for (int t = wlo + lane; t < whi; t += 32) n_tie += t < C && key_at(t) == T;
    n_tie = warp_sum_i(n_tie);
    if (lane == 0) sh.ties[warp] = n_tie;
  }
  cluster.sync();
  // sums of the warps before this one in slot order: all of the CTAs before, and of this CTA the warps before
  auto before = [&](int* mine) {
    int s = 0;
    for (int i = lane; i < kCluster * kSelWarps; i += 32)
      if (i < rank * kSelWarps + warp) s += cluster.map_shared_rank(mine, i / kSelWarps)[i % kSelWarps];
    return warp_sum_i(s);
  };
  const unsigned below = (1u << lane) - 1u;
  int ties0 = 0, n_src = 0, n_hole = 0;
  if (E > 0) {
    ties0 = before(sh.ties);
    int ties = ties0;
    for (int t0 = wlo; t0 < whi; t0 += 32) {
      const int t = t0 + lane;
      const uint32_t u = t < whi ? key_at(t) : 0u;
      const bool tie = t < whi && t < C && u == T;
      const unsigned tm = __ballot_sync(0xffffffffu, tie);
      const bool gone = t < whi && t < C && (u < T || (tie && ties + __popc(tm & below) >= spare));
      ties += __popc(tm);
      n_src += t < whi && t < E && !gone;
      n_hole += t >= E && gone;
    }
    n_src = warp_sum_i(n_src);
    n_hole = warp_sum_i(n_hole);
  }
  if (lane == 0) {
    sh.srcs[warp] = n_src;
    sh.holes[warp] = n_hole;
  }
  cluster.sync();
  int src0 = before(sh.srcs), hole0 = before(sh.holes);
  const int last = kCluster * kSelWarps - 1;
  if (rank * kSelWarps + warp == last && lane == 0) ws.counts[b] = src0 + n_src;
  int* src = ws.src + (size_t)b * a.maxp * (kPage / 2);
  int* dst = ws.dst + (size_t)b * a.maxp * (kPage / 2);
  float* wo = weights_out + (size_t)b * slots;
  {
    int ties = ties0;
    for (int t0 = wlo; t0 < whi; t0 += 32) {
      const int t = t0 + lane;
      bool gone = false;
      if (E > 0) {
        const uint32_t u = t < whi ? key_at(t) : 0u;
        const bool tie = t < whi && t < C && u == T;
        const unsigned tm = __ballot_sync(0xffffffffu, tie);
        gone = t < whi && t < C && (u < T || (tie && ties + __popc(tm & below) >= spare));
        ties += __popc(tm);
      }
      const bool moves = t < whi && t < E && !gone, hole = t >= E && gone;
      const unsigned sm = __ballot_sync(0xffffffffu, moves), hm = __ballot_sync(0xffffffffu, hole);
      if (moves) src[src0 + __popc(sm & below)] = t;
      if (hole) dst[hole0 + __popc(hm & below)] = t;
      src0 += __popc(sm);
      hole0 += __popc(hm);
      if (t < whi && t >= E && !hole) wo[t - E] = __ldg(w + t);  // a hole's weight comes with the token
    }
  }
  // behind the sequence: zeros; the table without its first n entries
  const int all = kCluster * kSelThreads, me = rank * kSelThreads + threadIdx.x;
  for (int t = L - E + me; t < slots; t += all) wo[t] = 0.f;
  const int* row = page_table + (size_t)b * a.maxp;
  for (int p = me; p < a.maxp; p += all) {
    page_table_out[(size_t)b * a.maxp + p] = p + n < a.maxp ? __ldg(row + p + n) : -1;
    if (p * kPage < L) {
      const int pg = __ldg(row + p);
      if (pg >= 0 && pg < a.num_pages) atomicAdd(ws.owners + pg, 1);
    }
  }
  if (me == 0) seq_lens_out[b] = L - E;
  cluster.sync();  // no CTA leaves while another may read its shared memory
}

// ---------------------------------------------------------------------------
// The moves: grid (x, B), a warp per token row, kRows rows in flight.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kRows = 4;

template <typename V>
__device__ __forceinline__ void copy_rows(char* pool, int bytes, const int (&from)[kRows], const int (&to)[kRows]) {
  const int lane = threadIdx.x & 31;
  for (int o = lane * (int)sizeof(V); o < bytes; o += 32 * (int)sizeof(V)) {
    V v[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (to[i] >= 0) v[i] = *reinterpret_cast<const V*>(pool + (size_t)from[i] * bytes + o);
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (to[i] >= 0) *reinterpret_cast<V*>(pool + (size_t)to[i] * bytes + o) = v[i];
  }
}

__global__ void __launch_bounds__(kMoveThreads)
    evict_move_kernel(const float* __restrict__ weights, const int* __restrict__ page_table,
                      const int* __restrict__ evict_pages, char* lat, char* rop, float* __restrict__ weights_out,
                      int* __restrict__ err, EvictWorkspace ws, EvictArgs a) {
  const int b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int count = __ldg(ws.counts + b);
  if (count == 0) return;
  const int E = __ldg(evict_pages + b) * kPage;  // count > 0: the select kernel accepted it
  const int slots = a.maxp * kPage;
  const int* row = page_table + (size_t)b * a.maxp;
  const int* src = ws.src + (size_t)b * a.maxp * (kPage / 2);
  const int* dst = ws.dst + (size_t)b * a.maxp * (kPage / 2);
  const int stride = gridDim.x * (kMoveThreads / 32) * kRows;
  for (int i0 = (blockIdx.x * (kMoveThreads / 32) + warp) * kRows; i0 < count; i0 += stride) {
    // lane i < kRows looks up row i0 + i
    int f = 0, t = -1;
    if (lane < kRows && i0 + lane < count) {
      const int s = __ldg(src + i0 + lane), d = __ldg(dst + i0 + lane);
      const int pf = __ldg(row + s / kPage), pt = __ldg(row + d / kPage);
      weights_out[(size_t)b * slots + d - E] = __ldg(weights + (size_t)b * slots + s);
      if (pf < 0 || pf >= a.num_pages || pt < 0 || pt >= a.num_pages || __ldg(ws.owners + pt) != 1) {
        report_error(err, kErrDeviceCheck, b, d);  // out of the pool, or another sequence's page too
      } else {
        f = pf * kPage + s % kPage;
        t = pt * kPage + d % kPage;
      }
    }
    int from[kRows], to[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      from[i] = __shfl_sync(0xffffffffu, f, i);
      to[i] = __shfl_sync(0xffffffffu, t, i);
    }
    copy_rows<uint4>(lat, a.lat_bytes, from, to);  // d_c is a multiple of 32
    if (a.rope_bytes % 16 == 0)
      copy_rows<uint4>(rop, a.rope_bytes, from, to);
    else
      copy_rows<uint32_t>(rop, a.rope_bytes, from, to);  // d_r is even
  }
}

}  // namespace

cudaError_t launch_evict(const int* evict_pages, const float* weights, const int* page_table, const int* seq_lens,
                         void* lat, void* rop, float* weights_out, int* page_table_out, int* seq_lens_out, int* err,
                         const EvictWorkspace& ws, const EvictArgs& a, int sms, cudaStream_t st) {
  cudaError_t e = cudaMemsetAsync(ws.owners, 0, (size_t)a.num_pages * sizeof(int), st);
  if (e != cudaSuccess) return e;
  const long long per = ((long long)a.maxp * kPage + kCluster - 1) / kCluster;
  const int smem = (int)(per < kKeyCap ? per : kKeyCap) * 4;
  e = ensure_smem(reinterpret_cast<const void*>(evict_select_kernel), smem);
  if (e != cudaSuccess) return e;
  evict_select_kernel<<<a.B * kCluster, kSelThreads, smem, st>>>(evict_pages, weights, page_table, seq_lens,
                                                                 weights_out, page_table_out, seq_lens_out, err, ws,
                                                                 a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // about eight CTAs per SM over all sequences, and no more than the longest list needs
  const int most = a.maxp * (kPage / 2), rows = kMoveThreads / 32 * kRows;
  int x = (8 * sms + a.B - 1) / a.B;
  if (x > (most + rows - 1) / rows) x = (most + rows - 1) / rows;
  evict_move_kernel<<<dim3(x, a.B), kMoveThreads, 0, st>>>(weights, page_table, evict_pages, static_cast<char*>(lat),
                                                            static_cast<char*>(rop), weights_out, err, ws, a);
  return cudaGetLastError();
}

}  // namespace mlra
