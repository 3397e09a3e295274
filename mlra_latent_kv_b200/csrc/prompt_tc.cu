// tcgen05 prompt attention: causal attention of packed prompts in the
// unabsorbed form, 128 + 64 score dims and 128 value dims (sm_100a).
//
//   x[i,j] = scale * (q_nope_i . k_nope_j + RoPE(q_rope_i) . k_j),  j <= Lk - Lq + i
//   out_i  = softmax_j(x) v                      (yololab.net, "超越 GQA 的推理
//   革命…", sections "1. 鍵值聯合低秩壓縮" and "2. 解耦旋轉位置編碼")
//
// Bound by the tensor cores: 640 flops per (query, key, head); K and V of a
// head come from L2 after the first query tile has fetched them.
//
// Design (B200):
//   * Rows of a tile are (token, head of the kv group) pairs: with grouped
//     heads as many heads as divide the group (a power of two) share a tile,
//     so their keys are read once and a chunk of few tokens still fills the
//     128 rows.  The rotary keys are shared by all heads and come from the
//     paged cache, a page per copy.
//   * A work item is two tiles (256 rows) of one sequence and head group,
//     which share every K and V block; a persistent CTA per SM takes items
//     from a counter, longest first within groups of heads whose K and V fit
//     in L2 together.
//   * TMEM: two score buffers (128 columns each; P, in bf16, overwrites the
//     scores it came from) and two output accumulators, all 512 columns.
//     While one tile's softmax runs, the tensor cores work on the other:
//     PV and the next QK^T of tile A, then of tile B.
//   * Shared memory: the two query tiles (96 KB) and a ring of eight 16 KB
//     blocks; a step's keys (128 tokens) are three of 64 dims, its values two of
//     64 tokens, so that 1.6 steps are loaded or on their way.
//   * Softmax: a thread per row, running maximum and sum in fp32, base 2.  The
//     exponentials are taken against the maximum so far, in the same pass that
//     finds the step's own, with P held back in registers; only when a row's
//     maximum has grown by more than 2^8 the scores are read again and O, which
//     the same thread owns, is rescaled: the scores of step j being there
//     implies that PV of step j - 1 is done.  Masks, the first step's maximum and
//     the rescaling are short loops over TMEM beside the one unrolled body, for
//     instructions that are met once an item come from far away (unrolled, a
//     masked step took 3600 cycles more, now 600).
//   * Value rows past a sequence's end are zeroed in shared memory before the
//     product (a NaN there would get past P = 0); key rows past it are masked.
//     A NaN or an infinity of a later token of the sequence: see rows_again.
//   * The rotation of the queries runs in the kernel before this one, beside
//     the plan (sequences checked, items sorted by length).
//   * Rounded to bf16, because the tensor cores take operands of one type: the
//     rotated queries and P (V is bf16).  The output is within 0.0025 of the
//     exact one (2-norm), its own rounding to bf16 is 0.0017 of that; statistics
//     and sums are fp32.
//   * Measured (calls among others): 128 heads x 4096 tokens 745 to 757 us, 908
//     to 923 TFLOP/s at the 1545 MHz that the power cap leaves, 640 in a burst;
//     16 ragged sequences up to 1900 tokens, 32 heads 146 us; four chunks behind
//     up to 8000 tokens, 32 heads on 8, 264 us.  The tensor pipe is active 55 %.
//   * Registers: 168 a thread with 88 bytes of spill stores and 456 of loads
//     (-Xptxas -v).  Compiled to 116 and 132 the same work takes 3 % longer.
//   * Every wait is bounded; a CTA that gives up records the site, lets its
//     copies and MMAs in flight end and leaves.
#include <cuda.h>

#include <atomic>

#include "host_cache.h"
#include "launch.h"
#include "serving.h"
#include "serving_ptx.cuh"

namespace mlra {
namespace {

using namespace ptx;

constexpr int kPtBlock = 128 * 128;  // 128 rows x 64 bf16, or 64 tokens x 128 bf16 as two halves
constexpr int kPtRing = 8;
constexpr int kPtThreads = 12 * 32;  // 0 loads, 1 and 3 MMAs, 2 value ends, 4-7 softmax of tile A, 8-11 of tile B
constexpr int kPtSmem = 6 * kPtBlock + kPtRing * kPtBlock;
constexpr uint32_t kPtColO = 256;
constexpr float kPtRescale = 8.f;    // log2
constexpr int kPtRegs = 168, kPtRegsAux = 88, kPtRegsSoftmax = 208;  // of a thread: at launch, then by role
static_assert(4 * kPtRegsAux + 8 * kPtRegsSoftmax <= 12 * kPtRegs, "the roles share the registers of the launch");
constexpr int kPlanThreads = 512;
constexpr int kPlanBins = 1024;
constexpr int kPlanAhead = 4;        // pieces of a token's queries that a lane has on their way

struct PromptItem {
  int live;          // 0: no more items
  int head0, kvh;    // first head of the tile's heads, their kv head
  int tok0;          // first token of tile A
  int Lq, Lk, q0, k0, b;
  int n[2];          // key tiles of tile A and B
};

struct PromptBars {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];  // of step t: t % 2
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], o_free[2];
  uint64_t item_full[2], item_empty[2];
  uint64_t v_fixed[2];  // a value tile's end is zeroed; in turn, for the ring may hold two such tiles
  uint64_t turn[2];     // the other tile has issued its step
  uint64_t drain[2];
  PromptItem item[2];
  int odd;              // the last of this CTA's items with rows to be taken again, -1 for none
  uint32_t tmem_base;
  int abort_flag;
};

enum { kPsRing = 60, kPsItem, kPsItemFree, kPsQ, kPsQFree, kPsK, kPsV, kPsP, kPsOFree, kPsS, kPsO, kPsTurn };

// ---------------------------------------------------------------------------
// Plan and query rotation.  Block 0 checks the sequences and lists the pairs
// of tiles, longest first (a counting sort over the number of key tiles);
// the other blocks rotate the queries, a token per warp: lane i forms the
// angle of pair i, each eight lanes take a head; the first heads are on their
// way meanwhile (64 heads x 4096 tokens: 15 us without, 11.6 so).
// ---------------------------------------------------------------------------
__device__ __forceinline__ int key_tiles(const PromptSeq& s, int tok0, int tokens) {
  const int last = min(tok0 + tokens, s.Lq) - 1;  // the tile's last query
  if (last < tok0) return 0;
  return (max(0, s.Lk - s.Lq + last + 1) + 127) / 128;
}

__global__ void __launch_bounds__(kPlanThreads)
    prompt_plan_kernel(const __nv_bfloat16* __restrict__ q_rope, const int* __restrict__ cu_q,
                       const int* __restrict__ cu_k, __nv_bfloat16* __restrict__ q_rot, int2* __restrict__ list,
                       int* __restrict__ counts, int* __restrict__ err, PromptArgs a, int pack, RopeTable tab) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int TT = 128 / pack;  // tokens of a tile
  grid_dep_launch();
  if (blockIdx.x == 0) {
    __shared__ int bins[kPlanBins], s_most, s_warp[32];
    __shared__ unsigned long long s_rows;
    for (int i = threadIdx.x; i < kPlanBins; i += kPlanThreads) bins[i] = 0;
    if (threadIdx.x == 0) {
      s_most = 1;
      s_rows = 0;
    }
    __syncthreads();
    for (int b = threadIdx.x; b < a.B; b += kPlanThreads) {
      const PromptSeq s = prompt_seq(cu_q, cu_k, b, a, err);
      if (s.Lq > 0) {
        atomicMax(&s_most, (s.Lk + 127) / 128);
        atomicAdd(&s_rows, (unsigned long long)s.Lq);
      }
    }
    __syncthreads();
    if (s_rows > (unsigned long long)a.total_q) {  // sequences that overlap: the list has no room for them
      if (threadIdx.x == 0) {
        report_error(err, kErrDeviceCheck, a.B, a.total_q);
        counts[0] = counts[1] = counts[2] = 0;
      }
      return;
    }
    const int most = s_most;
    // bin 0 holds the longest; an order within a bin is as good as another
    auto bin = [&](const PromptSeq& s, int pair) {
      const int n = max(key_tiles(s, 2 * pair * TT, TT), key_tiles(s, (2 * pair + 1) * TT, TT));
      return kPlanBins - 1 - (int)((long long)n * (kPlanBins - 1) / most);
    };
    for (int b = warp; b < a.B; b += kPlanThreads / 32) {
      const PromptSeq s = prompt_seq(cu_q, cu_k, b, a, nullptr);
      for (int p = lane; 2 * p * TT < s.Lq; p += 32) atomicAdd(&bins[bin(s, p)], 1);
    }
    __syncthreads();
    {  // exclusive prefix sums of the bins, two a thread
      const int v0 = bins[2 * threadIdx.x], v1 = bins[2 * threadIdx.x + 1];
      const int incl = warp_incl_scan(v0 + v1);
      if (lane == 31) s_warp[warp] = incl;
      __syncthreads();
      int before = 0;
      for (int i = 0; i < warp; ++i) before += s_warp[i];
      bins[2 * threadIdx.x] = before + incl - v0 - v1;
      bins[2 * threadIdx.x + 1] = before + incl - v1;
      if (threadIdx.x == kPlanThreads - 1) {
        counts[0] = before + incl;  // entries of the list
        counts[1] = 0;              // the next item
        counts[2] = 0;              // items with values that are not finite
      }
    }
    __syncthreads();
    for (int b = warp; b < a.B; b += kPlanThreads / 32) {
      const PromptSeq s = prompt_seq(cu_q, cu_k, b, a, nullptr);
      for (int p = lane; 2 * p * TT < s.Lq; p += 32) list[atomicAdd(&bins[bin(s, p)], 1)] = make_int2(b, p);
    }
    return;
  }
  const int warps = (gridDim.x - 1) * (kPlanThreads / 32);
  for (int t = (blockIdx.x - 1) * (kPlanThreads / 32) + warp; t < a.total_q; t += warps) {
    int lo = 0, hi = a.B - 1;  // the last sequence that starts at t or before
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (__ldg(cu_q + mid) <= t)
        lo = mid;
      else
        hi = mid - 1;
    }
    PromptSeq s = prompt_seq(cu_q, cu_k, lo, a, nullptr);
    auto holds = [&] { return t >= s.q0 && t < s.q0 + s.Lq; };
    if (!holds()) {  // a row of no sequence, or bad offsets led the search astray: all of them, a lane each
      unsigned found = 0;
      for (int b0 = 0; b0 < a.B && !found; b0 += 32) {
        if (b0 + lane < a.B) s = prompt_seq(cu_q, cu_k, b0 + lane, a, nullptr);
        found = __ballot_sync(0xffffffffu, b0 + lane < a.B && holds());
        if (found) s = prompt_seq(cu_q, cu_k, b0 + __ffs(found) - 1, a, nullptr);
      }
      if (!found) continue;
    }
    const int c = lane & 7;  // this lane's 16 bytes of a head: pairs 4 c .. 4 c + 3
    uint4 x[kPlanAhead];
    auto load = [&](int h0) {
#pragma unroll
      for (int k = 0; k < kPlanAhead; ++k) {
        const int h = h0 + 4 * k + (lane >> 3);
        const __nv_bfloat16* head = q_rope + (size_t)t * a.q_rope_s[0] + (size_t)h * a.q_rope_s[1];
        if (h < a.H) x[k] = __ldg(reinterpret_cast<const uint4*>(head) + c);
      }
    };
    load(0);  // on its way while the angles are formed
    float sn, cs;
    rope_sincos(tab, lane, s.Lk - s.Lq + t - s.q0, &sn, &cs);
    float sn4[4], cs4[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sn4[i] = __shfl_sync(0xffffffffu, sn, 4 * c + i);
      cs4[i] = __shfl_sync(0xffffffffu, cs, 4 * c + i);
    }
    for (int h0 = 0; h0 < a.H; h0 += 4 * kPlanAhead) {
#pragma unroll
      for (int k = 0; k < kPlanAhead; ++k) {
        const int h = h0 + 4 * k + (lane >> 3);
        uint32_t* w = &x[k].x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x0 = __uint_as_float(w[i] << 16), x1 = __uint_as_float(w[i] & 0xffff0000u);
          w[i] = pack_bf16x2(x0 * cs4[i] - x1 * sn4[i], x0 * sn4[i] + x1 * cs4[i]);
        }
        if (h < a.H) reinterpret_cast<uint4*>(q_rot + ((size_t)t * a.H + h) * 64)[c] = x[k];
      }
      load(h0 + 4 * kPlanAhead);
    }
  }
}

// ---------------------------------------------------------------------------
// Values that are not finite.  A tile's last steps hold keys past a row's own,
// with P = 0 there, and 0 times a NaN or an infinity is a NaN.  Rows that have
// such a value behind their last key are therefore taken again, over their own
// keys alone.  Warp 2, which has the least to do, looks at those keys' values
// while they lie in shared memory and chains their items; the warps other than
// the softmax's go through the chain behind the CTA's last item, a row each, a
// lane per key for the scores, four columns a lane for the values.
//
// Taken in turns with the kernel that did not look, 128 heads x 4096 tokens
// 736-747 -> 738-742 us, the ragged batch 135-137 -> 138-140, grouped chunks
// 246 -> 250.  (In the epilogue of the softmax warps it cost 3 to 8 %, for the
// compiler then dealt their loop's registers otherwise; in a kernel of its own
// behind this one the second part took 2 to 3 us.)  One token of NaN in all of 128 heads x 4096 tokens
// takes 20 ms: 24 reads of a key and eight values at a time, each from L2.
// ---------------------------------------------------------------------------
struct PromptRows {
  const __nv_bfloat16 *q_nope, *q_rot, *k_nope, *v, *rope_cache;
  __nv_bfloat16* out;
  const int *cu_q, *cu_k, *page_table;
  int4* odd;  // {sequence, first token, first head, the CTA's one before or -1} of items
  int pack;
  PromptArgs a;
};

// The item of an entry of `odd`.
__device__ __forceinline__ PromptItem prompt_item(int4 e, const int* cu_q, const int* cu_k, const PromptArgs& a,
                                                  int pack) {
  const PromptSeq s = prompt_seq(cu_q, cu_k, e.x, a, nullptr);
  PromptItem it;
  it.live = 1;
  it.b = e.x;
  it.head0 = e.z;
  it.kvh = e.z / (a.H / a.kv_heads);
  it.tok0 = e.y;
  it.Lq = s.Lq;
  it.Lk = s.Lk;
  it.q0 = s.q0;
  it.k0 = s.k0;
  it.n[0] = key_tiles(s, it.tok0, 128 / pack);
  it.n[1] = key_tiles(s, it.tok0 + 128 / pack, 128 / pack);
  return it;
}

// The first key of step j, counted from the step's own first, that one of the item's rows in it does not see.
__device__ __forceinline__ int cut_key(const PromptItem& it, int j, int TT) {
  const int own = it.Lk - it.Lq + it.tok0 + (j < it.n[0] ? 0 : TT);  // of the first row that has the step
  return max(0, own + 1 - 128 * j);
}

// z + the values times zero: a NaN once one of them is not finite.
__device__ __forceinline__ void add_zeros(__nv_bfloat162& z, uint4 x) {
  const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
  const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&x.x);
  z = __hadd2(z, __hfma2(p[0], zero, __hfma2(p[1], zero, __hfma2(p[2], zero, __hmul2(p[3], zero)))));
}
__device__ __forceinline__ bool is_odd(__nv_bfloat162 z) { return __hisnan(z.x) || __hisnan(z.y); }

__device__ __forceinline__ bool all_nan(uint2 y) {
  return (y.x & 0x7fffu) > 0x7f80u && (y.x & 0x7fff0000u) > 0x7f800000u && (y.y & 0x7fffu) > 0x7f80u &&
         (y.y & 0x7fff0000u) > 0x7f800000u;
}

// s + the sum of the products of eight pairs.
__device__ __forceinline__ float dot8(uint4 x, uint4 y, float s) {
  const uint32_t *p = &x.x, *q = &y.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(p[i] << 16), __uint_as_float(q[i] << 16), s);
    s = fmaf(__uint_as_float(p[i] & 0xffff0000u), __uint_as_float(q[i] & 0xffff0000u), s);
  }
  return s;
}

// The rows of an item that have to be taken again: rows `first`, first + 4, .. of them.
__device__ __forceinline__ void rows_again(const PromptItem& it, int first, const PromptRows& rows) {
  const PromptArgs& a = rows.a;
  const int pack = rows.pack, lane = threadIdx.x & 31, TT = 128 / pack;
  const __nv_bfloat16* vals = rows.v + (size_t)it.k0 * a.v_s[0] + (size_t)it.kvh * a.v_s[1] + 4 * lane;
  auto value = [&](int j) { return __ldg(reinterpret_cast<const uint2*>(vals + (size_t)j * a.v_s[0])); };
  for (int x = 0; x < 2; ++x) {
    const int tok0 = it.tok0 + x * TT, toks = min(TT, it.Lq - tok0);  // the tile's tokens
    const int own = it.Lk - it.Lq + tok0, end = min(it.Lk, 128 * it.n[x]);
    // of the keys behind the first row's own: the last whose value is not finite, the first whose value is all NaN
    int last = -1, all = end;
    for (int j = max(0, own + 1); j < end && all == end; ++j) {
      const uint2 y = value(j);
      __nv_bfloat162 z = __float2bfloat162_rn(0.f);
      add_zeros(z, make_uint4(y.x, y.y, 0u, 0u));
      if (__any_sync(0xffffffffu, is_odd(z))) last = j;
      if (__all_sync(0xffffffffu, all_nan(y))) all = j;
    }
    // tokens whose own key is before the last (those that see the value that is all NaN are NaN as they are)
    const int stop = min(toks, last - own);
    for (int r = max(0, -own) * pack + first; r < stop * pack; r += 4) {  // those before have no key
      const int tok = it.q0 + tok0 + r / pack, head = it.head0 + r % pack, lim = own + r / pack;
      const uint4* qn = reinterpret_cast<const uint4*>(rows.q_nope + (size_t)tok * a.q_nope_s[0] +
                                                       (size_t)head * a.q_nope_s[1]);
      const uint4* qr = reinterpret_cast<const uint4*>(rows.q_rot + ((size_t)tok * a.H + head) * 64);
      float o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
      for (int j0 = 0; j0 <= lim; j0 += 32) {
        const int j = min(j0 + lane, lim);
        const uint4* kn = reinterpret_cast<const uint4*>(rows.k_nope + (size_t)(it.k0 + j) * a.k_nope_s[0] +
                                                         (size_t)it.kvh * a.k_nope_s[1]);
        int id = __ldg(rows.page_table + (size_t)it.b * a.maxp + j / kPage);
        if (id < 0 || id >= a.num_pages) id = 0;  // reported when its step was loaded
        const uint4* kr = reinterpret_cast<const uint4*>(rows.rope_cache + ((size_t)id * kPage + j % kPage) * 64);
        float s = 0.f;
#pragma unroll 4
        for (int c = 0; c < 16; ++c) s = dot8(__ldg(qn + c), __ldg(kn + c), s);
#pragma unroll 4
        for (int c = 0; c < 8; ++c) s = dot8(qr[c], __ldg(kr + c), s);
        s = j0 + lane <= lim ? s * a.scale_log2 : -INFINITY;
        float top = s;
#pragma unroll
        for (int i = 16; i >= 1; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
        top = fmaxf(top, m);
        const float ref = top == -INFINITY ? 0.f : top, corr = ex2(m - ref), p = ex2(s - ref);
        m = top;
        l = l * corr + warp_sum(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] *= corr;
#pragma unroll 1
        for (int u0 = 0; u0 < 32 && j0 + u0 <= lim; u0 += 8) {
          uint2 y[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) y[u] = j0 + u0 + u <= lim ? value(j0 + u0 + u) : make_uint2(0u, 0u);
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const float pu = __shfl_sync(0xffffffffu, p, u0 + u);
            o[0] = fmaf(pu, __uint_as_float(y[u].x << 16), o[0]);
            o[1] = fmaf(pu, __uint_as_float(y[u].x & 0xffff0000u), o[1]);
            o[2] = fmaf(pu, __uint_as_float(y[u].y << 16), o[2]);
            o[3] = fmaf(pu, __uint_as_float(y[u].y & 0xffff0000u), o[3]);
          }
        }
      }
      const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = l == 0.f ? 0.f : o[i] * inv;
      *reinterpret_cast<uint2*>(rows.out + ((size_t)tok * a.H + head) * 128 + 4 * lane) =
          make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    }
  }
}

// ---------------------------------------------------------------------------
// The attention.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPtThreads, 1)
    prompt_tc_kernel(const __grid_constant__ CUtensorMap tm_qn, const __grid_constant__ CUtensorMap tm_qr,
                     const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_rope, const int* __restrict__ cu_q,
                     const int* __restrict__ cu_k, const int* __restrict__ page_table, const int2* __restrict__ list,
                     int* counts, __nv_bfloat16* __restrict__ out, float* __restrict__ lse, int* __restrict__ err,
                     PromptArgs a, int pack, int unit_group, const __grid_constant__ PromptRows rows) {
  constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, false, false);
  constexpr uint32_t kIdescPV = idesc_bf16_f32(128, 128, false, true);  // V read MN-major
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                 // [tile][64-dim block]
  uint8_t* sR = smem + 6 * kPtBlock;  // the ring
  PromptBars* bars = reinterpret_cast<PromptBars*>(smem + kPtSmem);
  volatile int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int TT = 128 / pack;

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&bars->k_full[x]), 1);
      mbar_init(smem_u32(&bars->k_empty[x]), 2);  // both tiles' MMAs
      mbar_init(smem_u32(&bars->v_full[x]), 1);
      mbar_init(smem_u32(&bars->v_empty[x]), 3);  // and the value ends' warp
      mbar_init(smem_u32(&bars->q_full[x]), 1);
      mbar_init(smem_u32(&bars->q_empty[x]), 1);
      mbar_init(smem_u32(&bars->s_full[x]), 1);
      mbar_init(smem_u32(&bars->p_full[x]), 4);
      mbar_init(smem_u32(&bars->o_full[x]), 1);
      mbar_init(smem_u32(&bars->o_free[x]), 4);
      mbar_init(smem_u32(&bars->v_fixed[x]), 1);
      mbar_init(smem_u32(&bars->turn[x]), 1);
      mbar_init(smem_u32(&bars->drain[x]), 1);
      mbar_init(smem_u32(&bars->item_full[x]), 1);
      mbar_init(smem_u32(&bars->item_empty[x]), 11);  // the MMA threads, warp 2 and eight softmax warps
    }
    bars->abort_flag = 0;
    bars->odd = -1;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  // the item of turn i, for a consumer; false when the CTA has given up
  auto take = [&](uint32_t i, PromptItem* it) {
    const int s = i & 1;
    if (!mbar_wait_warp(smem_u32(&bars->item_full[s]), (i >> 1) & 1, abort_flag, err, kPsItem)) return false;
    *it = bars->item[s];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->item_empty[s]));
    return true;
  };

  // The launch's registers, dealt out anew.  Each half of the roles stands wholly behind its own instruction.
  if (warp >= 4) {
    setmaxnreg_inc<kPtRegsSoftmax>();
    // ------------------------------------------------------------- softmax
    const int x = (warp - 4) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_col = tmem + lane_off + 128u * x, o_col = tmem + lane_off + kPtColO + 128u * x;
    const float sc = a.scale_log2, jump = kPtRescale / sc;
    const bool wide = reinterpret_cast<uintptr_t>(out) % 32 == 0;
    uint32_t steps = 0, tiles = 0;
    bool ok = true;
    PromptItem it;
    for (uint32_t i = 0; ok && take(i, &it) && it.live; ++i) {
      const int tok = it.tok0 + x * TT + row / pack, head = it.head0 + row % pack;
      const bool mine = tok < it.Lq;
      const int n = it.n[x];
      const int lim = min(it.Lk - it.Lq + tok, it.Lk - 1);  // the row's last key
      const size_t at = (size_t)(it.q0 + tok) * a.H + head;
      float m = -INFINITY, l = 0.f;
      auto largest = [&](float t, const uint32_t (&v)[32]) {
        float t0 = t, t1 = __uint_as_float(v[0]);
#pragma unroll
        for (int c = 1; c < 31; c += 3) {
          t0 = fmaxf(fmaxf(t0, __uint_as_float(v[c])), __uint_as_float(v[c + 1]));
          t1 = fmaxf(t1, __uint_as_float(v[c + 2]));
        }
        return fmaxf(fmaxf(t0, t1), __uint_as_float(v[31]));
      };
      for (int j = 0; j < n; ++j, ++steps) {
        ok = mbar_wait_warp(smem_u32(&bars->s_full[x]), steps & 1, abort_flag, err, kPsS);
        if (!ok) break;
        tc_fence_after();
        const int cmax = lim - 128 * j;
        if (__any_sync(0xffffffffu, cmax < 127)) {  // -inf past the row's last key, in place
#pragma unroll 1
          for (int c = 0; c < 128; c += 16) {
            uint32_t v[16];
            tmem_ld16(s_col + c, v);
#pragma unroll
            for (int u = 0; u < 16; ++u)
              if (c + u > cmax) v[u] = 0xff800000u;
            tmem_st16(s_col + c, v);
          }
        }
        if (j == 0) {  // the first step's own maximum
          m = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 128; c += 16) {
            uint32_t v[16];
            tmem_ld16(s_col + c, v);
#pragma unroll
            for (int u = 0; u < 16; u += 2) m = fmaxf(fmaxf(m, __uint_as_float(v[u])), __uint_as_float(v[u + 1]));
          }
        }
        uint32_t p[4][16];  // P of 32 keys each, packed
        float sum;
        while (true) {
          // against the maximum so far; the scores stay where they are until it is known that this will do
          const float ref = m == -INFINITY ? 0.f : -m * sc;  // no key so far: every term is 2^-inf = 0
          const float2 sc2 = make_float2(sc, sc), ref2 = make_float2(ref, ref);
          float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          float top = -INFINITY;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t v[2][32];
            tmem_ld32x2(s_col + 64 * h, s_col + 64 * h + 32, v[0], v[1]);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              top = largest(top, v[g]);
#pragma unroll
              for (int u = 0; u < 16; ++u) {
                float2 e = fma_f32x2(make_float2(__uint_as_float(v[g][2 * u]), __uint_as_float(v[g][2 * u + 1])), sc2,
                                     ref2);
                e.x = ex2(e.x);
                e.y = ex2(e.y);
                s2[u & 1] = add_f32x2(s2[u & 1], e);
                p[2 * h + g][u] = pack_bf16x2(e.x, e.y);
              }
            }
          }
          sum = (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
          if (!__any_sync(0xffffffffu, top > m + jump)) break;
          // a row's maximum has grown by more than 2^8: rescale what there is, and once more
          float corr = 1.f;
          if (top > m + jump) {
            corr = ex2((m - top) * sc);
            m = top;
          }
          l *= corr;
#pragma unroll 1
          for (int c = 0; c < 128; c += 16) {
            uint32_t o[16];
            tmem_ld16(o_col + c, o);
#pragma unroll
            for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * corr);
            tmem_st16(o_col + c, o);
          }
        }
        l += sum;
#pragma unroll
        for (int g = 0; g < 4; ++g) tmem_st16_async(s_col + 16u * g, p[g]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[x]));
      }
      if (!ok) break;
      if (n > 0) {
        ok = mbar_wait_warp(smem_u32(&bars->o_full[x]), tiles & 1, abort_flag, err, kPsO);
        ++tiles;
        if (!ok) break;
        tc_fence_after();
      }
      // O out of TMEM first, so that the next item's PV may go ahead, then the row in 32-byte pieces
      const float inv = l > 0.f ? 1.f / l : 0.f;
      uint32_t pk[64];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (n > 0) tmem_ld32(o_col + 32 * c, o);
#pragma unroll
        for (int u = 0; u < 16; ++u)
          pk[16 * c + u] = l == 0.f ? 0u : pack_bf16x2(__uint_as_float(o[2 * u]) * inv, __uint_as_float(o[2 * u + 1]) * inv);
      }
      if (n > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->o_free[x]));
      }
      if (mine) {
        __nv_bfloat16* dst = out + at * 128;
        if (wide) {
#pragma unroll
          for (int c = 0; c < 64; c += 8) st_global_32(dst + 2 * c, pk + c);
        } else {
#pragma unroll
          for (int c = 0; c < 64; c += 4)
            *reinterpret_cast<uint4*>(dst + 2 * c) = make_uint4(pk[c], pk[c + 1], pk[c + 2], pk[c + 3]);
        }
      }
      if (lse && mine) lse[at] = l == 0.f ? -INFINITY : m * sc + log2f(l);
    }
    asm volatile("bar.arrive 1, %0;" ::"n"(kPtThreads) : "memory");  // the outputs are written
  } else {
    setmaxnreg_dec<kPtRegsAux>();
  if (warp == 0) {
    // --------------------------------------------------------------- loads
    if (lane == 0) {
      tma_prefetch_desc(&tm_qn);
      tma_prefetch_desc(&tm_qr);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_rope);
    }
    grid_dep_wait();  // the plan and the rotated queries
    auto block_at = [&](uint32_t pos) { return smem_u32(sR + (pos % kPtRing) * kPtBlock); };
    const int nlist = *reinterpret_cast<volatile int*>(counts);
    const int units = a.H / pack;
    const long long total = (long long)nlist * units;
    const long long group = (long long)nlist * unit_group;
    uint32_t t = 0, tiles[2] = {0, 0};  // steps (key and value tiles) and query tiles loaded so far
    bool ok = true;
    auto unit_of = [&](long long w, int2* entry) {  // the item's heads, and where its tiles are listed
      const int g = (int)(w / group), r = (int)(w - g * group);
      const int nu = min(unit_group, units - g * unit_group);  // units of this group
      *entry = __ldcg(list + r / nu);
      return g * unit_group + r % nu;
    };
    auto decode = [&](int unit, int2 e) {
      const PromptSeq s = prompt_seq(cu_q, cu_k, e.x, a, nullptr);
      PromptItem it;
      it.live = 1;
      it.b = e.x;
      it.head0 = unit * pack;
      it.kvh = it.head0 / (a.H / a.kv_heads);
      it.tok0 = 2 * e.y * TT;
      it.Lq = s.Lq;
      it.Lk = s.Lk;
      it.q0 = s.q0;
      it.k0 = s.k0;
      it.n[0] = key_tiles(s, it.tok0, TT);
      it.n[1] = key_tiles(s, it.tok0 + TT, TT);
      return it;
    };
    // an item's query tiles and first steps towards L2, a box per lane
    auto fetch = [&](const PromptItem& it) {
      if (lane < 6) {
        const int x = lane / 3, blk = lane % 3, tok = it.q0 + it.tok0 + x * TT;
        if (it.n[x] > 0) tma_prefetch_l2_3d(blk < 2 ? &tm_qn : &tm_qr, 64 * (blk & 1), it.head0, tok);
      } else if (lane >= 8 && lane < 20) {
        const int e = lane - 8, j = e / 6, blk = e % 6;  // step j: two key boxes, four value boxes
        if (j < max(it.n[0], it.n[1])) {
          if (blk < 2)
            tma_prefetch_l2_3d(&tm_k, 64 * blk, it.kvh, it.k0 + 128 * j);
          else
            tma_prefetch_l2_3d(&tm_v, 64 * (blk & 1), it.kvh, it.k0 + 128 * j + 64 * ((blk - 2) >> 1));
        }
      }
      __syncwarp();
    };
    int w = 0;
    if (lane == 0) w = atomicAdd(counts + 1, 1);
    w = __shfl_sync(0xffffffffu, w, 0);
    PromptItem it;
    it.live = 0;
    if (w < total) {
      int2 e;
      const int unit = unit_of(w, &e);
      it = decode(unit, e);
    }
    for (uint32_t i = 0; ok; ++i) {
      int w_next = 0;
      if (lane == 0 && it.live) w_next = atomicAdd(counts + 1, 1);  // looked at from the second step on
      const int sl = i & 1;
      if (i >= 2 && !mbar_wait_warp(smem_u32(&bars->item_empty[sl]), ((i >> 1) - 1) & 1, abort_flag, err, kPsItemFree))
        break;
      if (lane == 0) {
        bars->item[sl] = it;
        mbar_arrive(smem_u32(&bars->item_full[sl]));
      }
      __syncwarp();
      if (!it.live) break;
      const int n = max(it.n[0], it.n[1]), np = npages_of(it.Lk);
      // lane 0, 1: the ids of a key tile's pages, read a tile ahead
      auto page_id = [&](int j) {
        return lane < 2 && 2 * j + lane < np ? __ldg(page_table + (size_t)it.b * a.maxp + 2 * j + lane) : 0;
      };
      // The next item is looked up a bit at a time between this one's loads.
      PromptItem nxt;
      nxt.live = 0;
      int looked = 0, unit = 0;
      int2 entry;
      auto look_ahead = [&] {
        if (looked == 0) {
          w = __shfl_sync(0xffffffffu, w_next, 0);
          if (w < total)
            unit = unit_of(w, &entry);
          else
            looked = 1;
        } else if (w < total) {
          nxt = decode(unit, entry);
          fetch(nxt);
        }
        ++looked;
      };
      int id = page_id(0);
      for (int j = 0; ok && j < n; ++j, ++t) {
        if (j > 0 && looked < 2) look_ahead();
        const int id_next = j + 1 < n ? page_id(j + 1) : 0;
        const int pages = min(2, np - 2 * j);
        // Keys: blocks 5 t .. 5 t + 2 of the ring, where the last of the keys and the values of step t - 2 were.
        if (t >= 2) ok = mbar_wait_warp(smem_u32(&bars->v_empty[t & 1]), ((t >> 1) - 1) & 1, abort_flag, err, kPsRing);
        if (!ok) break;
        {
          const uint32_t fb = smem_u32(&bars->k_full[t & 1]);
          if (lane == 0) mbar_expect_tx(fb, 2 * kPtBlock + pages * (kPtBlock / 2));
          __syncwarp();
          if (lane < pages) {  // the rotary keys, a page a lane
            if (id < 0 || id >= a.num_pages) {  // reported, and read from page 0 instead
              report_error(err, kErrDeviceCheck, it.b, (2 * j + lane) * kPage);
              id = 0;
            }
            tma_load_2d(block_at(5 * t + 2) + lane * (kPtBlock / 2), &tm_rope, fb, 0, id * kPage);
          } else if (lane >= 2 && lane < 4) {
            tma_load_3d(block_at(5 * t + lane - 2), &tm_k, fb, 64 * (lane - 2), it.kvh, it.k0 + 128 * j);
          }
          __syncwarp();
        }
        if (j == 0) {  // the query tiles, once the last QK^T of the item before has read theirs
          for (int x = 0; ok && x < 2; ++x) {
            if (it.n[x] == 0) continue;
            if (tiles[x] > 0)
              ok = mbar_wait_warp(smem_u32(&bars->q_empty[x]), (tiles[x] - 1) & 1, abort_flag, err, kPsQFree);
            if (!ok) break;
            if (lane == 0) {
              const uint32_t fb = smem_u32(&bars->q_full[x]), dst = smem_u32(sQ + 3 * x * kPtBlock);
              const int tok = it.q0 + it.tok0 + x * TT;
              mbar_expect_tx(fb, 3 * kPtBlock);
              tma_load_3d(dst, &tm_qn, fb, 0, it.head0, tok);
              tma_load_3d(dst + kPtBlock, &tm_qn, fb, 64, it.head0, tok);
              tma_load_3d(dst + 2 * kPtBlock, &tm_qr, fb, 0, it.head0, tok);
            }
            __syncwarp();
            ++tiles[x];
          }
          if (!ok) break;
        }
        // Values: blocks 5 t + 3, 5 t + 4, where the first two of the keys of step t - 1 were.
        if (t >= 1)
          ok = mbar_wait_warp(smem_u32(&bars->k_empty[(t - 1) & 1]), ((t - 1) >> 1) & 1, abort_flag, err, kPsRing);
        if (!ok) break;
        {
          const uint32_t fb = smem_u32(&bars->v_full[t & 1]);
          if (lane == 0) mbar_expect_tx(fb, 2 * kPtBlock);
          __syncwarp();
          if (lane < 4)  // 64 tokens x 64 dims a lane
            tma_load_3d(block_at(5 * t + 3 + (lane >> 1)) + (lane & 1) * (kPtBlock / 2), &tm_v, fb, 64 * (lane & 1),
                        it.kvh, it.k0 + 128 * j + 64 * (lane >> 1));
          __syncwarp();
        }
        id = id_next;
      }
      while (looked < 2) look_ahead();
      it = nxt;
    }
    if (*abort_flag) {  // what may still be on its way: the last two steps and the step that was broken off
      for (uint32_t u = t > 1 ? t - 2 : 0; u <= t; ++u) {
        if (u < t || !ok) drain_wait(smem_u32(&bars->k_full[u & 1]), (u >> 1) & 1);
        if (u < t) drain_wait(smem_u32(&bars->v_full[u & 1]), (u >> 1) & 1);
      }
      for (int x = 0; x < 2; ++x)
        if (tiles[x] > 0) drain_wait(smem_u32(&bars->q_full[x]), (tiles[x] - 1) & 1);
    }
  } else if (warp == 1 || warp == 3) {
    // ---------------------------------------------------------------- MMAs
    // One thread per tile waits, issues and commits: QK^T of step j + 1 right behind PV of step j, which
    // reads the P that lies where the new scores go.  A thread's wait drains the tensor pipe of its own
    // MMAs; the other tile's keep it busy.  The tiles take turns, so that one's softmax falls into the
    // other's products.
    if (elect_one()) {
      const int x = warp >> 1;
      uint32_t t0 = 0;                 // steps of the items before
      uint32_t tiles = 0, steps = 0;   // query tiles begun, P buffers taken
      uint32_t ends = 0, turns = 0;    // value tiles with an end, turns taken
      const uint64_t qd0 = sdesc_sw128(smem_u32(sQ + 3 * x * kPtBlock), 16, 1024);
      const uint64_t kd0 = sdesc_sw128(smem_u32(sR), 16, 1024), vd0 = sdesc_sw128(smem_u32(sR), kPtBlock / 2, 1024);
      const uint32_t s_col = tmem + 128u * x, o_col = tmem + kPtColO + 128u * x;
      bool ok = true, owed = false;
      auto wait_keys = [&](uint32_t t) {
        ok = ok && mbar_wait(smem_u32(&bars->k_full[t & 1]), (t >> 1) & 1, abort_flag, err, kPsK);
      };
      auto wait_values = [&](uint32_t t) {
        ok = ok && mbar_wait(smem_u32(&bars->v_full[t & 1]), (t >> 1) & 1, abort_flag, err, kPsV);
      };
      auto block = [&](uint32_t pos) { return (uint64_t)((pos % kPtRing) * (kPtBlock >> 4)); };
      for (uint32_t i = 0; ok; ++i) {
        const int sl = i & 1;
        ok = mbar_wait(smem_u32(&bars->item_full[sl]), (i >> 1) & 1, abort_flag, err, kPsItem);
        if (!ok) break;
        const int live = bars->item[sl].live, n0 = bars->item[sl].n[0], n1 = bars->item[sl].n[1], Lk = bars->item[sl].Lk;
        mbar_arrive(smem_u32(&bars->item_empty[sl]));
        if (!live) break;
        const int mine = x ? n1 : n0, n = max(n0, n1);
        auto qk = [&](int j) {
          const uint32_t t = t0 + j;
          wait_keys(t);
          if (!ok) return;
          tc_fence_after();
#pragma unroll
          for (int blk = 0; blk < 3; ++blk) {
            // the other tile's turn: it is here by the time that the rest has gone into the pipe
            if (blk == 2 && owed) mbar_arrive(smem_u32(&bars->turn[x ^ 1]));
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_ss(s_col, qd0 + (uint64_t)(blk * (kPtBlock >> 4) + 2 * ks), kd0 + block(5 * t + blk) + (uint64_t)(2 * ks),
                     kIdescQK, (blk | ks) ? 1u : 0u);
          }
          mma_commit(smem_u32(&bars->s_full[x]));
          mma_commit(smem_u32(&bars->k_empty[t & 1]));
          if (j + 1 == mine) mma_commit(smem_u32(&bars->q_empty[x]));
        };
        auto pv = [&](int j) {
          const uint32_t t = t0 + j;
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_ts(o_col, s_col + 32u * half + 8u * ks, vd0 + block(5 * t + 3 + half) + (uint64_t)((ks * 2048) >> 4),
                     kIdescPV,
                     (j | half | ks) ? 1u : 0u);
          mma_commit(smem_u32(&bars->v_empty[t & 1]));
          if (j + 1 == mine) mma_commit(smem_u32(&bars->o_full[x]));
        };
        if (mine > 0) {
          ok = mbar_wait(smem_u32(&bars->q_full[x]), tiles & 1, abort_flag, err, kPsQ);
          ++tiles;
          const bool waits = owed;
          owed = false;
          qk(0);
          owed = waits;
          for (int j = 0; ok && j < mine; ++j, ++steps) {
            wait_values(t0 + j);
            if (Lk < 128 * (j + 1))
              ok = ok && mbar_wait(smem_u32(&bars->v_fixed[ends & 1]), (ends >> 1) & 1, abort_flag, err, kPsV);
            if (j == 0 && tiles > 1)  // the item before has read its O
              ok = ok && mbar_wait(smem_u32(&bars->o_free[x]), (tiles - 2) & 1, abort_flag, err, kPsOFree);
            if (x ? j < n0 : owed)  // strictly in turn: no token is passed before the last one was taken
              ok = ok && mbar_wait(smem_u32(&bars->turn[x]), turns++ & 1, abort_flag, err, kPsTurn);
            ok = ok && mbar_poll(smem_u32(&bars->p_full[x]), steps & 1, abort_flag, err, kPsP);
            if (!ok) break;
            tc_fence_after();
            pv(j);
            owed = j < (x ? n0 : n1);  // the other tile has this step too, and waits for its turn
            if (j + 1 < mine)
              qk(j + 1);  // its keys may land while PV runs
            else if (owed)
              mbar_arrive(smem_u32(&bars->turn[x ^ 1]));
          }
        }
        // steps that only the other tile takes: passed on as they come
        for (uint32_t t = t0 + mine; ok && t < t0 + n; ++t) {
          wait_keys(t);
          if (ok) mbar_arrive(smem_u32(&bars->k_empty[t & 1]));
          wait_values(t);
          if (ok) mbar_arrive(smem_u32(&bars->v_empty[t & 1]));
        }
        t0 += n;
        ends += n > 0 && Lk < 128 * n;
      }
      if (*abort_flag) {
        mma_commit(smem_u32(&bars->drain[x]));
        drain_wait(smem_u32(&bars->drain[x]), 0);
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------- value rows past a sequence's end, values that are not finite
    uint32_t t = 0, ends = 0;
    bool ok = true;
    PromptItem it;
    for (uint32_t i = 0; ok && take(i, &it) && it.live; ++i) {
      const int n = max(it.n[0], it.n[1]);
      __nv_bfloat162 z = __float2bfloat162_rn(0.f);
      for (int j = 0; ok && j < n; ++j, ++t) {
        const int left = it.Lk - 128 * j;  // of the value tile, inside the sequence
        ok = mbar_wait_warp(smem_u32(&bars->v_full[t & 1]), (t >> 1) & 1, abort_flag, err, kPsV);
        if (!ok) break;
        if (left < 128) {  // the sequence's last value tile
          for (int half = 0; half < 2; ++half) {
            const int r0 = min(64, max(0, left - 64 * half)), nz = (64 - r0) * 8;  // 16-byte pieces of 64 dims
            uint8_t* to = sR + ((5 * t + 3 + half) % kPtRing) * kPtBlock + r0 * 128;
            for (int e = lane; e < nz; e += 32)
#pragma unroll
              for (int d = 0; d < 2; ++d)
                *reinterpret_cast<uint4*>(to + d * (kPtBlock / 2) + e * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars->v_fixed[ends & 1]));
          ++ends;
        }
        const int key0 = cut_key(it, j, TT);
        for (int half = key0 >> 6; half < 2; ++half) {
          const int r0 = max(0, key0 - 64 * half);
          const uint8_t* from = sR + ((5 * t + 3 + half) % kPtRing) * kPtBlock + r0 * 128;
#pragma unroll 2
          for (int e = lane; e < (64 - r0) * 8; e += 32)
#pragma unroll
            for (int d = 0; d < 2; ++d)
              add_zeros(z, *reinterpret_cast<const uint4*>(from + d * (kPtBlock / 2) + e * 16));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->v_empty[t & 1]));
      }
      if (__any_sync(0xffffffffu, is_odd(z)) && lane == 0) {
        const int at = atomicAdd(counts + 2, 1);
        rows.odd[at] = make_int4(it.b, it.tok0, it.head0, bars->odd);
        bars->odd = at;
      }
    }
  }
  // the outputs are written, all values have been seen
  named_barrier(1, kPtThreads);
  for (int e = *abort_flag ? -1 : *reinterpret_cast<volatile int*>(&bars->odd); e >= 0;) {
    const int4 o = __ldcg(rows.odd + e);
    rows_again(prompt_item(o, rows.cu_q, rows.cu_k, rows.a, rows.pack), warp, rows);
    e = o.w;
  }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// Heads of a kv group that share a tile: the largest power of two that divides the group, at most 128.
int heads_packed(int H, int kv_heads) {
  const int g = H / kv_heads, p = g & -g;
  return p < 128 ? p : 128;
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
long long list_entries(const PromptArgs& a, int pack) { return ((long long)a.total_q * pack + 255) / 256 + a.B; }

// error record | item counts | list of tile pairs | items to be taken again in part | rotated queries
struct PromptLayout {
  size_t list, odd, q_rot, total;
};
PromptLayout prompt_layout(const PromptArgs& a, int pack) {
  const size_t entries = (size_t)list_entries(a, pack);
  PromptLayout l;
  l.list = 512;
  l.odd = round_up(l.list + entries * sizeof(int2), 256);
  l.q_rot = round_up(l.odd + entries * (a.H / pack) * sizeof(int4), 256);
  l.total = round_up(l.q_rot + (size_t)a.total_q * a.H * 64 * 2, 256);
  return l;
}

}  // namespace

bool prompt_tc_supported(int dtype, int d_h, int d_r, int d_v) {
  return dtype == MLRA_BF16 && d_h == 128 && d_r == 64 && d_v == 128;
}

cudaError_t prompt_tc_registers(int* regs, int* want) {
  static std::atomic<int> known{0};  // of the code, the same on every device; a failed query is not kept
  *want = kPtRegs;
  *regs = known.load(std::memory_order_relaxed);
  if (*regs != 0) return cudaSuccess;
  cudaFuncAttributes f;
  const cudaError_t e = cudaFuncGetAttributes(&f, prompt_tc_kernel);
  if (e == cudaSuccess) known.store(*regs = f.numRegs, std::memory_order_relaxed);
  return e;
}

size_t prompt_tc_workspace(const PromptArgs& a) { return prompt_layout(a, heads_packed(a.H, a.kv_heads)).total; }

cudaError_t launch_prompt_tc(const void* q_nope, const void* q_rope, const int* cu_q, const void* k_nope,
                             const void* v, const int* cu_k, const void* rope_cache, const int* page_table, void* out,
                             float* lse, void* workspace, const PromptArgs& a, const RopeTable& tab, int sms,
                             cudaStream_t st) {
  const int pack = heads_packed(a.H, a.kv_heads), units = a.H / pack;
  char* ws = static_cast<char*>(workspace);
  int* err = reinterpret_cast<int*>(ws);
  int* counts = reinterpret_cast<int*>(ws + 256);
  const PromptLayout at = prompt_layout(a, pack);
  int2* list = reinterpret_cast<int2*>(ws + at.list);
  int4* odd = reinterpret_cast<int4*>(ws + at.odd);
  const long long entries = list_entries(a, pack);
  __nv_bfloat16* q_rot = reinterpret_cast<__nv_bfloat16*>(ws + at.q_rot);

  // packed [tokens][heads][width]; an axis of one element takes any valid stride
  auto packed = [&](CUtensorMap* m, const void* p, int width, int heads, int rows, const long long* s, int box_heads,
                    int box_rows) {
    const uint64_t d[3] = {(uint64_t)width, (uint64_t)heads, (uint64_t)(rows > 0 ? rows : 1)};
    const uint64_t by[2] = {(uint64_t)(heads > 1 && rows > 0 ? s[1] : width) * 2,
                            (uint64_t)(rows > 1 ? s[0] : width) * 2};
    const uint32_t box[3] = {64, (uint32_t)box_heads, (uint32_t)box_rows};
    return encode_bf16_map(m, 3, p, d, by, box);
  };
  const long long rot_s[2] = {(long long)a.H * 64, 64};
  CUtensorMap tqn, tqr, tk, tv, tr;
  if (a.total_k == 0) k_nope = v = q_nope;  // no key to load: any address will do
  const uint64_t rd[2] = {64, (uint64_t)a.num_pages * kPage}, rs[1] = {128};
  const uint32_t rbox[2] = {64, 64};
  if (!packed(&tqn, q_nope, 128, a.H, a.total_q, a.q_nope_s, pack, 128 / pack) ||
      !packed(&tqr, q_rot, 64, a.H, a.total_q, rot_s, pack, 128 / pack) ||
      !packed(&tk, k_nope, 128, a.kv_heads, a.total_k, a.k_nope_s, 1, 128) ||
      !packed(&tv, v, 128, a.kv_heads, a.total_k, a.v_s, 1, 64) ||
      !encode_bf16_map(&tr, 2, rope_cache, rd, rs, rbox))
    return cudaErrorInvalidValue;

  const int rot_blocks = (int)(((long long)a.total_q + kPlanThreads / 32 - 1) / (kPlanThreads / 32));
  prompt_plan_kernel<<<1 + (rot_blocks < 8 * sms ? rot_blocks : 8 * sms), kPlanThreads, 0, st>>>(
      static_cast<const __nv_bfloat16*>(q_rope), cu_q, cu_k, q_rot, list, counts, err, a, pack, tab);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  // Units of heads whose K and V (256 values a token and kv head) fit in 112 of L2's 126 MB together, in groups of
  // one size: a last group of few heads is a long wait for its longest items (64 heads x 4096 tokens: 345 us as
  // 48 + 16, 321 as 32 + 32; 32 heads: 188 us as 24 + 8, 165 as one; 128 heads: 694 us as one, 647 as 43 + 43 + 42).
  const long long bytes = (long long)a.total_k * 512 * a.kv_heads / units;
  long long group = bytes > 0 ? (112LL << 20) / bytes : units;
  group = group < 1 ? 1 : (group > units ? units : group);
  const long long groups = (units + group - 1) / group;
  group = (units + groups - 1) / groups;
  const PromptRows rows{static_cast<const __nv_bfloat16*>(q_nope), q_rot, static_cast<const __nv_bfloat16*>(k_nope),
                        static_cast<const __nv_bfloat16*>(v), static_cast<const __nv_bfloat16*>(rope_cache),
                        static_cast<__nv_bfloat16*>(out), cu_q, cu_k, page_table, odd, pack, a};
  const int smem = 1024 + kPtSmem + (int)sizeof(PromptBars);
  e = ensure_smem(reinterpret_cast<const void*>(prompt_tc_kernel), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(entries * units < sms ? entries * units : sms));
  cfg.blockDim = dim3(kPtThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prompt_tc_kernel, tqn, tqr, tk, tv, tr, cu_q, cu_k, page_table,
                            static_cast<const int2*>(list), counts, static_cast<__nv_bfloat16*>(out), lse, err, a, pack,
                            (int)group, rows);
}

}  // namespace mlra
