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
// Two kernels, after one that clears the pages' owner counts.
// evict_select_kernel: a cluster of CTAs per sequence finds
// the 64 n smallest (weight, slot) by a radix select over the weights' bits
// (four 8-bit digits; the CTAs' histograms meet in distributed shared memory)
// and writes both lists, in slot order, beside the shifted weights, table and
// length.  It is bound by latency: a sequence's weights are read from HBM once
// and kept in shared memory.  evict_move_kernel copies the rows, bound by HBM.
// Measured: 64 sequences of 1024 to 32768 tokens that lose half 83 us, 28 of
// them the selection, then 288 MB at 5.25 TB/s; four of 131072 that lose three
// quarters 74 us, 30 of them the selection.
#include <cooperative_groups.h>

#include "host_cache.h"
#include "ptx.cuh"
#include "serving.h"

namespace mlra {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kKeyCap = 24576;     // keys a CTA keeps in shared memory, two CTAs per SM; beyond: re-read

// Ascending order of the weights as unsigned integers: -inf and NaN first, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (isnan(w)) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kBins = 256;         // of a digit
constexpr int kBatch = 8;          // keys a thread handles at once
constexpr int kAlone = 4096;       // a sequence that one CTA takes alone, without the cluster's barriers
struct SelShared {
  int hist[2][kBins];          // of this CTA, double-buffered over the digits
  int warp_sum[kBins / 32];
  int ties[kSelWarps];         // equal to the threshold, per warp
  int srcs[kSelWarps];         // tokens to move, per warp
  int holes[kSelWarps];        // slots to move to, per warp
  int found[3];                // the digit, the keys below it, the keys that have it
};

__global__ void __launch_bounds__(kSelThreads, 2)
    evict_select_kernel(const int* __restrict__ evict_pages, const float* __restrict__ weights,
                        const int* __restrict__ page_table, const int* __restrict__ seq_lens,
                        float* __restrict__ weights_out, int* __restrict__ page_table_out,
                        int* __restrict__ seq_lens_out, int* __restrict__ err, EvictWorkspace ws, EvictArgs a) {
  ptx::grid_dep_launch();
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) SelShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int cl = cluster.num_blocks();  // CTAs per sequence
  const int b = blockIdx.x / cl, rank = cluster.block_rank();
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
  const bool alone = L <= kAlone || cl == 1;
  const int ctas = alone ? 1 : cl;
  auto meet = [&] {  // all CTAs that share the sequence
    if (alone)
      __syncthreads();
    else
      cluster.sync();
  };
  const int per = (L + ctas - 1) / ctas;
  const int lo = min(L, rank * per), hi = min(L, lo + per);
  const bool in_smem = per <= kKeyCap;
  const int wper = ((hi - lo + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int wlo = min(hi, lo + warp * wper), whi = min(hi, wlo + wper);
  // the keys of slots t, t + stride, .. of this CTA, read at once (0 past its last)
  auto keys_at = [&](int t, int stride, uint32_t (&u)[kBatch]) {
    if (in_smem) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) u[i] = t + i * stride < hi ? keys[t + i * stride - lo] : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) u[i] = t + i * stride < hi ? order_key(__ldg(w + t + i * stride)) : 0u;
    }
  };

  uint32_t T = 0;  // the largest key that leaves
  int spare = 0;   // of the tokens with that key, in slot order, the first `spare` stay
  if (E > 0 && rank < ctas) {  // uniform over the CTAs that meet
    if (in_smem)
      for (int t0 = lo + threadIdx.x; t0 < hi; t0 += 2 * kBatch * kSelThreads) {
        float x[2 * kBatch];
#pragma unroll
        for (int i = 0; i < 2 * kBatch; ++i)
          if (t0 + i * kSelThreads < hi) x[i] = __ldg(w + t0 + i * kSelThreads);
#pragma unroll
        for (int i = 0; i < 2 * kBatch; ++i)
          if (t0 + i * kSelThreads < hi) keys[t0 + i * kSelThreads - lo] = order_key(x[i]);
      }
    for (int i = threadIdx.x; i < 2 * kBins; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
    int need = E;  // how many of the keys that share the digits found so far leave
    for (int d = 0; d < 4; ++d) {
      const int shift = 24 - 8 * d;
      const uint32_t mask = d == 0 ? 0u : 0xFFFFFFFFu << (shift + 8);
      int* hist = sh.hist[d & 1];
      const int end = min(hi, C);
      for (int t0 = lo + threadIdx.x; t0 < end; t0 += kBatch * kSelThreads) {
        uint32_t u[kBatch];
        keys_at(t0, kSelThreads, u);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (t0 + i * kSelThreads < end && (u[i] & mask) == T) atomicAdd(&hist[(u[i] >> shift) & 255u], 1);
      }
      meet();
      int v = 0;
      if (threadIdx.x < kBins) {  // a thread per bin: its count over the cluster, and the running count
        for (int r = 0; r < ctas; ++r) v += alone ? hist[threadIdx.x] : cluster.map_shared_rank(hist, r)[threadIdx.x];
        sh.hist[(d + 1) & 1][threadIdx.x] = 0;  // the next digit's: read before this meeting
      }
      const int incl = warp_incl_scan(v);
      if (lane == 31 && threadIdx.x < kBins) sh.warp_sum[warp] = incl;
      __syncthreads();
      int below_me = incl - v;
      for (int i = 0; i < warp && i < kBins / 32; ++i) below_me += sh.warp_sum[i];
      if (below_me < need && need <= below_me + v) {  // one thread: the count reaches `need` here
        sh.found[0] = threadIdx.x;
        sh.found[1] = below_me;
        sh.found[2] = v;
      }
      __syncthreads();
      T |= (uint32_t)sh.found[0] << shift;
      need -= sh.found[1];
      spare = sh.found[2] - need;
      __syncthreads();  // everyone has them before the next digit's are written
    }

    if (spare > 0) {  // ties before each warp, over the cluster: the first `spare` of them stay
      int n_tie = 0;
      for (int t0 = wlo + lane; t0 < whi; t0 += 32 * kBatch) {
        uint32_t u[kBatch];
        keys_at(t0, 32, u);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) n_tie += t0 + 32 * i < min(whi, C) && u[i] == T;
      }
      n_tie = warp_sum_i(n_tie);
      if (lane == 0) sh.ties[warp] = n_tie;
      meet();
    }
  }
  // sums of the warps before this one in slot order: all of the CTAs before, and of this CTA the warps before
  auto before = [&](int* mine) {
    int s = 0;
    for (int i = lane; i < ctas * kSelWarps; i += 32)
      if (i < rank * kSelWarps + warp)
        s += alone ? mine[i] : cluster.map_shared_rank(mine, i / kSelWarps)[i % kSelWarps];
    return warp_sum_i(s);
  };
  const unsigned below = (1u << lane) - 1u;
  int ties0 = 0, n_src = 0, n_hole = 0;
  // this warp's slots in order, 32 at a time, each with whether its token leaves (false past the warp's last)
  auto walk = [&](auto f) {
    int ties = ties0;
    for (int t0 = wlo + lane; t0 - lane < whi; t0 += 32 * kBatch) {
      uint32_t u[kBatch];
      keys_at(t0, 32, u);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int t = t0 + 32 * i;
        const bool may = t < min(whi, C), tie = may && u[i] == T;
        const unsigned tm = __ballot_sync(0xffffffffu, tie);
        f(t, may && (u[i] < T || (tie && ties + __popc(tm & below) >= spare)));
        ties += __popc(tm);
      }
    }
  };
  if (E > 0) {
    if (spare > 0) ties0 = before(sh.ties);
    walk([&](int t, bool gone) {
      n_src += t < min(whi, E) && !gone;
      n_hole += t >= E && gone;
    });
    n_src = warp_sum_i(n_src);
    n_hole = warp_sum_i(n_hole);
  }
  if (lane == 0) {
    sh.srcs[warp] = n_src;
    sh.holes[warp] = n_hole;
  }
  meet();
  int src0 = before(sh.srcs), hole0 = before(sh.holes);
  const int last = ctas * kSelWarps - 1;
  if (rank * kSelWarps + warp == last && lane == 0) ws.counts[b] = src0 + n_src;
  int* src = ws.src + (size_t)b * a.maxp * (kPage / 2);
  int* dst = ws.dst + (size_t)b * a.maxp * (kPage / 2);
  if (E > 0)
    walk([&](int t, bool gone) {
      const bool moves = t < min(whi, E) && !gone, hole = t >= E && gone;
      const unsigned sm = __ballot_sync(0xffffffffu, moves), hm = __ballot_sync(0xffffffffu, hole);
      if (moves) src[src0 + __popc(sm & below)] = t;
      if (hole) dst[hole0 + __popc(hm & below)] = t;
      src0 += __popc(sm);
      hole0 += __popc(hm);
    });
  // the weights in their new places, zeros behind them (a moved token's weight comes with it, over the one that
  // was there); the table without its first n entries
  const int all = cl * kSelThreads, me = rank * kSelThreads + threadIdx.x;
  float* wo = weights_out + (size_t)b * slots;
#pragma unroll 4
  for (int t = me; t < slots; t += all) wo[t] = t + E < L ? __ldg(w + t + E) : 0.f;
  const int* row = page_table + (size_t)b * a.maxp;
  ptx::grid_dep_wait();  // the owners are cleared
  for (int p = me; p < a.maxp; p += all) {
    page_table_out[(size_t)b * a.maxp + p] = p + n < a.maxp ? __ldg(row + p + n) : -1;
    if (p * kPage < L) {
      const int pg = __ldg(row + p);
      if (pg >= 0 && pg < a.num_pages) atomicAdd(ws.owners + pg, 1);
    }
  }
  if (me == 0) seq_lens_out[b] = L - E;
  if (!alone) cluster.sync();  // no CTA leaves while another may read its shared memory
}

// ---------------------------------------------------------------------------
// The moves.  The lists of all sequences are laid end to end and shared evenly
// by the warps, to the row.  A warp looks up 32 rows at once (a chain of three
// loads: list, page table, owners) and copies them four at a time, every
// 16-byte piece of the four (latent and rope key alike) in flight before the
// first is stored.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kRows = 4;
constexpr int kPieces = 3;  // of a row and lane: 96 x 16 bytes a round

__global__ void __launch_bounds__(kMoveThreads, 2)
    evict_move_kernel(const float* __restrict__ weights, const int* __restrict__ page_table,
                      const int* __restrict__ evict_pages, char* lat, char* rop, float* __restrict__ weights_out,
                      int* __restrict__ err, EvictWorkspace ws, EvictArgs a) {
  const int lane = threadIdx.x & 31;
  const int slots = a.maxp * kPage;
  ptx::grid_dep_wait();  // the lists
  // this warp's rows, and the sequence of the first
  auto rows_of = [&](int b) { return b < a.B ? __ldcg(ws.counts + b) : 0; };
  long long T = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) T += warp_sum_i(rows_of(b0 + lane));
  const int w = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5), W = gridDim.x * (kMoveThreads / 32);
  const long long start = worker_start(w, T, W);
  int left = (int)(worker_start(w + 1, T, W) - start);
  if (left == 0) return;
  int b = 0, i = 0, count = 0;
  {
    long long prefix = 0;
    for (int b0 = 0;; b0 += 32) {
      const int k = rows_of(b0 + lane), incl = warp_incl_scan(k);
      const unsigned m = __ballot_sync(0xffffffffu, prefix + incl > start);
      if (m) {
        const int l = __ffs(m) - 1;
        b = b0 + l;
        count = __shfl_sync(0xffffffffu, k, l);
        i = (int)(start - prefix) - __shfl_sync(0xffffffffu, incl - k, l);
        break;
      }
      prefix += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  const int lat16 = a.lat_bytes / 16;                              // d_c is a multiple of 32
  const int rop16 = a.rope_bytes % 16 == 0 ? a.rope_bytes / 16 : 0;  // else in words: d_r is even
  while (left > 0) {
    while (i == count) {
      count = __ldcg(ws.counts + ++b);
      i = 0;
    }
    const int n = min(32, min(count - i, left));  // rows of this round, a lane each
    int from = 0, to = -1;  // their token slots in the pools, to = -1 for none; the tokens' weights go along
    if (lane < n) {
      const size_t list = (size_t)b * a.maxp * (kPage / 2) + i + lane;
      const int s = __ldcg(ws.src + list), d = __ldcg(ws.dst + list);
      const int* row = page_table + (size_t)b * a.maxp;
      const int pf = __ldg(row + s / kPage), pt = __ldg(row + d / kPage);
      // count > 0: evict_pages[b] was accepted
      weights_out[(size_t)b * slots + d - __ldg(evict_pages + b) * kPage] = __ldg(weights + (size_t)b * slots + s);
      if (pf < 0 || pf >= a.num_pages || pt < 0 || pt >= a.num_pages || __ldcg(ws.owners + pt) != 1) {
        report_error(err, kErrDeviceCheck, b, d);  // out of the pool, or another sequence's page too
      } else {
        from = pf * kPage + s % kPage;
        to = pt * kPage + d % kPage;
      }
    }
    i += n;
    left -= n;
    for (int r = 0; r < n; r += kRows) {
      int f[kRows], t[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        f[k] = __shfl_sync(0xffffffffu, from, r + k);  // past the last row: to = -1
        t[k] = __shfl_sync(0xffffffffu, to, r + k);
      }
      for (int u0 = 0; u0 < lat16 + rop16; u0 += 32 * kPieces) {
        uint4 v[kPieces][kRows];
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
          const int u = u0 + 32 * k + lane;
#pragma unroll
          for (int q = 0; q < kRows; ++q)
            if (t[q] >= 0 && u < lat16 + rop16)
              v[k][q] = *reinterpret_cast<const uint4*>(
                  u < lat16 ? lat + (size_t)f[q] * a.lat_bytes + u * 16
                            : rop + (size_t)f[q] * a.rope_bytes + (u - lat16) * 16);
        }
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
          const int u = u0 + 32 * k + lane;
#pragma unroll
          for (int q = 0; q < kRows; ++q)
            if (t[q] >= 0 && u < lat16 + rop16)
              *reinterpret_cast<uint4*>(u < lat16 ? lat + (size_t)t[q] * a.lat_bytes + u * 16
                                                  : rop + (size_t)t[q] * a.rope_bytes + (u - lat16) * 16) = v[k][q];
        }
      }
      if (rop16 == 0)
        for (int o = lane * 4; o < a.rope_bytes; o += 128)
#pragma unroll
          for (int q = 0; q < kRows; ++q)
            if (t[q] >= 0)
              *reinterpret_cast<uint32_t*>(rop + (size_t)t[q] * a.rope_bytes + o) =
                  *reinterpret_cast<const uint32_t*>(rop + (size_t)f[q] * a.rope_bytes + o);
    }
  }
}

__global__ void __launch_bounds__(1024) evict_clear_kernel(int* owners, int n) {
  ptx::grid_dep_launch();
  for (int i = blockIdx.x * 1024 + threadIdx.x; i < n; i += gridDim.x * 1024) owners[i] = 0;
}

}  // namespace

cudaError_t launch_evict(const int* evict_pages, const float* weights, const int* page_table, const int* seq_lens,
                         void* lat, void* rop, float* weights_out, int* page_table_out, int* seq_lens_out, int* err,
                         const EvictWorkspace& ws, const EvictArgs& a, int sms, cudaStream_t st) {
  // Each kernel is launched while the one before still runs and waits for what it needs of it.
  const int clear = (a.num_pages + 1023) / 1024;
  evict_clear_kernel<<<clear < sms ? clear : sms, 1024, 0, st>>>(ws.owners, a.num_pages);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // A cluster as large as two resident CTAs per SM allow: a few long sequences spread over 16 CTAs each (four of
  // 131072 tokens: 35 us with 8), many over fewer, so that they run in one wave (64 sequences: 35 us with 8).  No
  // cluster where no sequence can be longer than what one CTA takes alone.
  int cl = 16;
  while (cl > 1 && (long long)a.B * cl > 2LL * sms) cl /= 2;
  const int slots = a.maxp * kPage;
  if (slots <= kAlone) cl = 1;
  const int per = (slots + cl - 1) / cl;  // a CTA's keys: its part of a sequence's,
  const int alone = slots < kAlone ? slots : kAlone;              // or all of a short one's
  const int keys = per < kKeyCap ? (per < alone ? alone : per) : kKeyCap;
  e = ensure_smem(reinterpret_cast<const void*>(evict_select_kernel), keys * 4);
  if (e == cudaSuccess && cl > 8)
    e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.B * cl);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = keys * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cl;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, evict_pages, weights, page_table, seq_lens, weights_out,
                         page_table_out, seq_lens_out, err, ws, a);
  if (e != cudaSuccess) return e;
  // what is resident at once, and no more than there can be rows
  const long long most = ((long long)a.B * a.maxp * (kPage / 2) + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
  cfg.gridDim = dim3((unsigned)(most < 2 * sms ? most : 2 * sms));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, weights, page_table, evict_pages, static_cast<char*>(lat),
                            static_cast<char*>(rop), weights_out, err, ws, a);
}

}  // namespace mlra
