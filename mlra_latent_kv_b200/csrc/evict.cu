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
// (three digits; the CTAs' histograms meet in distributed shared memory)
// and writes both lists, in slot order, beside the shifted weights, table and
// length.  It is bound by latency: a sequence's weights are read from HBM once
// and kept in shared memory.  evict_move_kernel copies the rows, bound by HBM.
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

constexpr int kBins = 2048;        // of a digit: 11, 11 and 10 bits
constexpr int kSlice = kBins / kCluster;  // bins that a CTA adds up for the cluster
constexpr int kAlone = 4096;       // a sequence that one CTA takes alone, without the cluster's barriers
static_assert(kSlice % 32 == 0 && kSlice <= kSelThreads, "a thread per bin of a slice");

struct SelShared {
  int hist[2][kBins];          // of this CTA, double-buffered over the digits
  int warp_sum[kSelWarps];
  int ties[kSelWarps];         // equal to the threshold, per warp
  int srcs[kSelWarps];         // tokens to move, per warp
  int holes[kSelWarps];        // slots to move to, per warp
  int slice[kCluster];         // keys in each CTA's slice of the bins
  int found[3];                // the digit, the keys below it, the keys that have it
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSelThreads)
    evict_select_kernel(const int* __restrict__ evict_pages, const float* __restrict__ weights,
                        const int* __restrict__ page_table, const int* __restrict__ seq_lens,
                        float* __restrict__ weights_out, int* __restrict__ page_table_out,
                        int* __restrict__ seq_lens_out, int* __restrict__ err, EvictWorkspace ws, EvictArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) SelShared sh;
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
  const bool alone = L <= kAlone;
  const int ctas = alone ? 1 : kCluster;
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
  auto key_at = [&](int t) { return in_smem ? keys[t - lo] : order_key(__ldg(w + t)); };

  uint32_t T = 0;  // the largest key that leaves
  int spare = 0;   // of the tokens with that key, in slot order, the first `spare` stay
  if (E > 0 && rank < ctas) {  // uniform over the CTAs that meet
    if (in_smem)
      for (int t = lo + threadIdx.x; t < hi; t += kSelThreads) keys[t - lo] = order_key(__ldg(w + t));
    for (int i = threadIdx.x; i < 2 * kBins; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
    int need = E;  // how many of the keys that share the digits found so far leave
    for (int d = 0; d < 3; ++d) {
      const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
      const uint32_t digits = d == 2 ? 1023u : 2047u, mask = d == 0 ? 0u : 0xFFFFFFFFu << (d == 1 ? 21 : 10);
      int* hist = sh.hist[d & 1];
      for (int t = lo + threadIdx.x; t < min(hi, C); t += kSelThreads) {
        const uint32_t u = key_at(t);
        if ((u & mask) == T) atomicAdd(&hist[(u >> shift) & digits], 1);
      }
      meet();
      // Each CTA adds up its slice of the bins over the cluster (all of them, if it is alone) and tells the others
      // the slice's sum; the CTA in whose slice the running count reaches `need` tells them the bin.
      for (int s0 = 0; s0 < kCluster; s0 += ctas) {
        const int sl = s0 + rank, bin = sl * kSlice + threadIdx.x;
        int v = 0;
        if (threadIdx.x < kSlice)
          for (int r = 0; r < ctas; ++r) v += alone ? hist[bin] : cluster.map_shared_rank(hist, r)[bin];
        const int incl = warp_incl_scan(v);
        if (lane == 31 && threadIdx.x < kSlice) sh.warp_sum[warp] = incl;
        __syncthreads();
        int sum = 0;
        for (int i = 0; i < kSlice / 32; ++i) sum += sh.warp_sum[i];
        if ((int)threadIdx.x < ctas) *(alone ? &sh.slice[sl] : cluster.map_shared_rank(&sh.slice[sl], threadIdx.x)) = sum;
        __syncthreads();
      }
      for (int i = threadIdx.x; i < kBins; i += kSelThreads) sh.hist[(d + 1) & 1][i] = 0;  // read before the last meeting
      meet();
      int sl = 0, before = 0;
      while (before + sh.slice[sl] < need) before += sh.slice[sl++];
      if (sl % ctas == rank) {
        const int bin = sl * kSlice + threadIdx.x;
        int v = 0;
        if (threadIdx.x < kSlice)
          for (int r = 0; r < ctas; ++r) v += alone ? hist[bin] : cluster.map_shared_rank(hist, r)[bin];
        const int incl = warp_incl_scan(v);
        if (lane == 31 && threadIdx.x < kSlice) sh.warp_sum[warp] = incl;
        __syncthreads();
        int below_me = before + incl - v;
        for (int i = 0; i < warp && i < kSlice / 32; ++i) below_me += sh.warp_sum[i];
        if (below_me < need && need <= below_me + v) {  // one thread
          for (int r = 0; r < ctas; ++r) {
            int* f = alone ? sh.found : cluster.map_shared_rank(sh.found, r);
            f[0] = bin;
            f[1] = below_me;
            f[2] = v;
          }
        }
      }
      meet();
      T |= (uint32_t)sh.found[0] << shift;
      need -= sh.found[1];
      spare = sh.found[2] - need;
    }

    if (spare > 0) {  // ties before each warp, over the cluster: the first `spare` of them stay
      int n_tie = 0;
      for (int t = wlo + lane; t < whi; t += 32) n_tie += t < C && key_at(t) == T;
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
  if (E > 0) {
    if (spare > 0) ties0 = before(sh.ties);
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
  meet();
  int src0 = before(sh.srcs), hole0 = before(sh.holes);
  const int last = ctas * kSelWarps - 1;
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
  if (!alone) cluster.sync();  // no CTA leaves while another may read its shared memory
}

// ---------------------------------------------------------------------------
// The moves.  The lists of all sequences are laid end to end in chunks of 32
// rows and shared evenly by the CTAs; a warp copies four rows of a chunk at a
// time, every 16-byte piece of them (latent and rope key alike) in flight
// before the first is stored, and looks up the next four meanwhile.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kRows = 4;
constexpr int kChunk = kMoveThreads / 32 * kRows;
constexpr int kPieces = 3;  // of a row and lane: 96 x 16 bytes a round

__global__ void __launch_bounds__(kMoveThreads, 2)
    evict_move_kernel(const float* __restrict__ weights, const int* __restrict__ page_table,
                      const int* __restrict__ evict_pages, char* lat, char* rop, float* __restrict__ weights_out,
                      int* __restrict__ err, EvictWorkspace ws, EvictArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slots = a.maxp * kPage;
  // this CTA's chunks, and the sequence of the first
  auto chunks_of = [&](int b) { return b < a.B ? (__ldg(ws.counts + b) + kChunk - 1) / kChunk : 0; };
  long long T = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) T += warp_sum_i(chunks_of(b0 + lane));
  const long long start = worker_start(blockIdx.x, T, gridDim.x);
  long long left = worker_start(blockIdx.x + 1, T, gridDim.x) - start;
  if (left == 0) return;
  int b = 0, c = 0;
  {
    long long prefix = 0;
    for (int b0 = 0;; b0 += 32) {
      const int k = chunks_of(b0 + lane), incl = warp_incl_scan(k);
      const unsigned m = __ballot_sync(0xffffffffu, prefix + incl > start);
      if (m) {
        const int l = __ffs(m) - 1;
        b = b0 + l;
        c = (int)(start - prefix - __shfl_sync(0xffffffffu, incl - k, l));
        break;
      }
      prefix += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  int count = __ldg(ws.counts + b);
  // lanes 0 .. kRows-1 look up the warp's rows of chunk c of sequence b: the token slots in the pools, to = -1 for
  // none; the tokens' weights go along
  int from = 0, to = -1;
  auto look_up = [&] {
    from = 0;
    to = -1;
    const int i = c * kChunk + warp * kRows + lane;
    if (lane < kRows && i < count) {
      const size_t list = (size_t)b * a.maxp * (kPage / 2) + i;
      const int s = __ldg(ws.src + list), d = __ldg(ws.dst + list);
      const int* row = page_table + (size_t)b * a.maxp;
      const int pf = __ldg(row + s / kPage), pt = __ldg(row + d / kPage);
      // count > 0: evict_pages[b] was accepted
      weights_out[(size_t)b * slots + d - __ldg(evict_pages + b) * kPage] = __ldg(weights + (size_t)b * slots + s);
      if (pf < 0 || pf >= a.num_pages || pt < 0 || pt >= a.num_pages || __ldg(ws.owners + pt) != 1) {
        report_error(err, kErrDeviceCheck, b, d);  // out of the pool, or another sequence's page too
      } else {
        from = pf * kPage + s % kPage;
        to = pt * kPage + d % kPage;
      }
    }
  };
  look_up();
  const int lat16 = a.lat_bytes / 16;                              // d_c is a multiple of 32
  const int rop16 = a.rope_bytes % 16 == 0 ? a.rope_bytes / 16 : 0;  // else in words: d_r is even
  for (; left > 0; --left) {
    int f[kRows], t[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      f[i] = __shfl_sync(0xffffffffu, from, i);
      t[i] = __shfl_sync(0xffffffffu, to, i);
    }
    if (left > 1) {  // the next chunk's rows
      if (++c * kChunk >= count) {
        c = 0;
        do count = __ldg(ws.counts + ++b);
        while (count == 0);
      }
      look_up();
    }
    for (int u0 = 0; u0 < lat16 + rop16; u0 += 32 * kPieces) {
      uint4 v[kPieces][kRows];
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int u = u0 + 32 * k + lane;
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          if (t[i] >= 0 && u < lat16 + rop16)
            v[k][i] = *reinterpret_cast<const uint4*>(u < lat16 ? lat + (size_t)f[i] * a.lat_bytes + u * 16
                                                                : rop + (size_t)f[i] * a.rope_bytes + (u - lat16) * 16);
      }
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int u = u0 + 32 * k + lane;
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          if (t[i] >= 0 && u < lat16 + rop16)
            *reinterpret_cast<uint4*>(u < lat16 ? lat + (size_t)t[i] * a.lat_bytes + u * 16
                                                : rop + (size_t)t[i] * a.rope_bytes + (u - lat16) * 16) = v[k][i];
      }
    }
    if (rop16 == 0)
      for (int o = lane * 4; o < a.rope_bytes; o += 128)
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          if (t[i] >= 0)
            *reinterpret_cast<uint32_t*>(rop + (size_t)t[i] * a.rope_bytes + o) =
                *reinterpret_cast<const uint32_t*>(rop + (size_t)f[i] * a.rope_bytes + o);
  }
}

}  // namespace

cudaError_t launch_evict(const int* evict_pages, const float* weights, const int* page_table, const int* seq_lens,
                         void* lat, void* rop, float* weights_out, int* page_table_out, int* seq_lens_out, int* err,
                         const EvictWorkspace& ws, const EvictArgs& a, int sms, cudaStream_t st) {
  cudaError_t e = cudaMemsetAsync(ws.owners, 0, (size_t)a.num_pages * sizeof(int), st);
  if (e != cudaSuccess) return e;
  const long long per = ((long long)a.maxp * kPage + kCluster - 1) / kCluster;
  const int slots = a.maxp * kPage;  // a CTA's keys: an eighth of a sequence's, or all of a short one's
  const long long keys = per < kKeyCap ? (per < kAlone ? (slots < kAlone ? slots : kAlone) : per) : kKeyCap;
  const int smem = (int)keys * 4;
  e = ensure_smem(reinterpret_cast<const void*>(evict_select_kernel), smem);
  if (e != cudaSuccess) return e;
  evict_select_kernel<<<a.B * kCluster, kSelThreads, smem, st>>>(evict_pages, weights, page_table, seq_lens,
                                                                 weights_out, page_table_out, seq_lens_out, err, ws,
                                                                 a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // what is resident at once, and no more than there can be chunks
  const long long most = (long long)a.B * ((a.maxp * (kPage / 2) + kChunk - 1) / kChunk);
  const int grid = (int)(most < 2 * sms ? most : 2 * sms);
  evict_move_kernel<<<grid, kMoveThreads, 0, st>>>(weights, page_table, evict_pages, static_cast<char*>(lat),
                                                   static_cast<char*>(rop), weights_out, err, ws, a);
  return cudaGetLastError();
}

}  // namespace mlra
