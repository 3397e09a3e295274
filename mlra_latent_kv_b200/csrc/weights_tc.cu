// tcgen05 kernel of the attention weights (see weights.cu for the formula):
// one pass over the cache, no value product and no softmax state, because the
// log-sum-exp is given.
//
// Bound by HBM: a token is 1152 B (d_c = 512) and 2 * 128 * 576 flops at 128
// heads, 128 flop/B against the card's 250; four branches take 4 * 128
// exponentials a token, 70 % of the exponential unit's rate at full bandwidth.
// Measured (calls among others): 64 sequences of 1024 to 32768 tokens, 32
// heads: 112 us, 6.2 TB/s, 95 % of the copy bandwidth; 32 x 16384 tokens, four
// branches of 128 heads: 149 to 161 us under the power cap, 125 in a burst.
//
// The tensor core's fp32 sums truncate: a logit is a few units in its last
// place low in magnitude.  All weights together are 1e-6 to 2e-6 from the 64-bit
// ones (2-norm), a single one up to 1.2e-5 of itself.  The log-sum-exp of the
// decode kernels comes from sums of the same kind.
//
// Design (B200):
//   * The tokens are the rows of the product: S^T[128 tokens, heads] =
//     [c; k] . q^T, M = 128 tokens (two pages), N = heads (padded to 16), A the
//     cache tile and B the query, both K-major as TMA leaves them.  A thread
//     then holds one token's scores of every head, and the sum over heads is a
//     sum over its own registers: no shuffles, no atomics, and the padding to
//     128 rows is spent on tokens, of which there are plenty, not on heads.
//   * The query of the current sequence stays in shared memory (147 KB at 128
//     heads), the cache passes through two rings of 16 KB blocks (128 tokens x
//     64 dims), latent and rotary, that fill the rest: 64 KB in flight at 128
//     heads, 176 KB at 32 (ring_blocks).
//   * A unit is (tile, branch), its scores one of 512 / heads TMEM buffers.  The
//     tile's rotary block starts each branch's buffer when its turn comes and
//     stays (loaded once) until the last branch's, the branch's latent blocks
//     finish the buffer.  (Started for all branches at once, a tile waits until
//     the exponentials of the whole tile before are done.)
//   * Warps: 0 loads the latent, 3 the rotary keys, 1 issues the MMAs, 2 loads
//     the query of the next sequence as soon as the last MMA of this one is
//     done (the cache keeps streaming meanwhile), 4-11 exponentiate: two warps
//     per TMEM lane quarter, half of the heads each.
//   * CTAs share the tiles evenly, sequences laid end to end, as the decode's
//     split does.
//   * Every mbarrier wait is bounded; a CTA that gives up records the site,
//     lets its copies and MMAs in flight end and leaves.  The exponentiating
//     warps walk all their tiles even then, so that none is missing at their
//     barrier.
#include <cuda.h>

#include <cstddef>

#include "host_cache.h"
#include "serving.h"
#include "serving_ptx.cuh"

namespace mlra {
namespace {

using namespace ptx;

constexpr int kWtTile = 128;        // tokens of a tile: two pages
constexpr int kWtBlock = 128 * 128;  // 128 tokens x 64 bf16
constexpr int kWtStages = 12;        // latent blocks at most
constexpr int kWtRopes = 2;          // rotary blocks at most
constexpr int kWtBufs = 16;          // TMEM buffers at most
constexpr int kWtThreads = 12 * 32;
constexpr int kWtSmx0 = 4;           // first exponentiating warp
constexpr int kWtSmem = 232448;
constexpr int kWtMaxRow = 512;       // n_branch * heads

struct WtBars {
  uint64_t full[kWtStages], empty[kWtStages];
  uint64_t r_full[kWtRopes], r_empty[kWtRopes];
  uint64_t s_full[kWtBufs], s_free[kWtBufs];
  uint64_t q_full, q_empty, drain;
  alignas(16) float lse[2][kWtMaxRow];  // of the sequence, double-buffered; read four at a time
  float half_sum[2][kWtTile];
  uint32_t tmem_base;
  int abort_flag;
};

static_assert(offsetof(WtBars, lse) % 16 == 0 && sizeof(WtBars) % 16 == 0, "16-byte reads");

// 16 KB blocks of both rings beside the query of Hp heads and D dims: a block is missing at 128 heads, where the
// barriers and the log-sum-exps take what is left of it.
constexpr int query_bytes(int Hp, int D) { return D / 64 * Hp * 128; }
constexpr int ring_blocks(int Hp, int D) {
  return (kWtSmem - 1024 - query_bytes(Hp, D) - (int)sizeof(WtBars)) / kWtBlock;
}
static_assert(ring_blocks(128, 576) == 4 && ring_blocks(32, 576) == 11, "64 KB and 176 KB");

// A position in a ring of `n` barriers and the parity of its current round.
struct RingPos {
  int i = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void step(int n) {
    if (++i == n) {
      i = 0;
      round ^= 1u;
    }
  }
};

enum { kWsRing = 40, kWsFull, kWsQEmpty, kWsQFull, kWsFree, kWsScores, kWsRopeRing, kWsRope };

// The tiles of CTA c of G, one after another.
struct TileCursor {
  long long n;   // tiles of this CTA
  int b, t, nt, L;
  bool first;    // the first tile of a sequence here
  const int* lens;
  int B, maxL;
  __device__ __forceinline__ static int tiles_of(int L) { return (L + kWtTile - 1) / kWtTile; }
  __device__ __forceinline__ TileCursor(const int* seq_lens, int B_, int maxL_, int c, int G)
      : n(0), b(0), t(0), nt(0), L(0), first(true), lens(seq_lens), B(B_), maxL(maxL_) {
    const int lane = threadIdx.x & 31;
    long long T = 0;
    for (int b0 = 0; b0 < B; b0 += 32) T += warp_sum_i(b0 + lane < B ? tiles_of(seq_len_at(lens, b0 + lane, maxL)) : 0);
    const long long start = worker_start(c, T, G);
    n = worker_start(c + 1, T, G) - start;
    if (n == 0) return;
    long long prefix = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int k = b0 + lane < B ? tiles_of(seq_len_at(lens, b0 + lane, maxL)) : 0;
      const int incl = warp_incl_scan(k);
      const unsigned m = __ballot_sync(0xffffffffu, prefix + incl > start);
      if (m) {
        const int l = __ffs(m) - 1;
        b = b0 + l;
        t = (int)(start - prefix - __shfl_sync(0xffffffffu, incl - k, l));
        break;
      }
      prefix += __shfl_sync(0xffffffffu, incl, 31);
    }
    L = seq_len_at(lens, b, maxL);
    nt = tiles_of(L);
  }
  __device__ __forceinline__ bool last() const { return t + 1 == nt; }
  __device__ __forceinline__ void step() {
    first = false;
    if (++t < nt) return;
    first = true;
    t = 0;
    do {
      ++b;
      L = b < B ? seq_len_at(lens, b, maxL) : 0;
    } while (b < B && L == 0);
    nt = tiles_of(L);
  }
};

__global__ void __launch_bounds__(kWtThreads, 1)
    weights_tc_kernel(const __grid_constant__ CUtensorMap tm_lat, const __grid_constant__ CUtensorMap tm_rope,
                      const __grid_constant__ CUtensorMap tm_q, const float* __restrict__ lse,
                      const int* __restrict__ page_table, const int* __restrict__ seq_lens, const float* w_in,
                      float* w_out, int* __restrict__ err, WeightArgs a, int Hp, int stages, int ropes, int bufs) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int nlat = a.d_c / 64, nblk = nlat + 1;  // 64-dim blocks of the latent, and with the rotary one
  const int q_block = Hp * 128;
  uint8_t* sQ = smem;                    // [nblk][Hp rows]
  uint8_t* sT = smem + nblk * q_block;   // the rings (Hp is a multiple of 16: 1024-byte aligned)
  uint8_t* sR = sT + stages * kWtBlock;
  WtBars* bars = reinterpret_cast<WtBars*>(sR + ropes * kWtBlock);
  volatile int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int maxL = a.maxp * kPage;
  const int stride = (Hp + 31) / 32 * 32;  // TMEM columns of a buffer

  if (threadIdx.x == 0) {
    for (int k = 0; k < stages; ++k) {
      mbar_init(smem_u32(&bars->full[k]), 1);
      mbar_init(smem_u32(&bars->empty[k]), 1);
    }
    for (int k = 0; k < ropes; ++k) {
      mbar_init(smem_u32(&bars->r_full[k]), 1);
      mbar_init(smem_u32(&bars->r_empty[k]), 1);
    }
    for (int k = 0; k < bufs; ++k) {
      mbar_init(smem_u32(&bars->s_full[k]), 1);
      mbar_init(smem_u32(&bars->s_free[k]), 8);
    }
    mbar_init(smem_u32(&bars->q_full), 1);
    mbar_init(smem_u32(&bars->q_empty), 1);
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  if (blockIdx.x == 0 && warp == 3) {
    for (int b = lane; b < a.B; b += 32) {
      const int Lb = __ldg(seq_lens + b);
      if (Lb < 0 || Lb > maxL) report_error(err, kErrDeviceCheck, b, Lb);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  TileCursor cur(seq_lens, a.B, maxL, blockIdx.x, gridDim.x);
  const long long n = cur.n;

  if (warp == 0 || warp == 3) {
    // ------------------------------------- the cache: latent blocks, rotary blocks
    const bool rope = warp == 3;
    const CUtensorMap* map = rope ? &tm_rope : &tm_lat;
    uint64_t *full = rope ? bars->r_full : bars->full, *empty = rope ? bars->r_empty : bars->empty;
    uint8_t* to = rope ? sR : sT;
    const int size = rope ? ropes : stages, blocks = rope ? 1 : nlat;
    RingPos ring;
    int filled = 0;  // blocks in the ring, up to its size
    bool ok = true;
    // lane j < 2: the id of page j of the tile, read a tile ahead
    auto page_id = [&](const TileCursor& c) {
      return lane < 2 && c.b < a.B && (2 * c.t + lane) * kPage < c.L
                 ? __ldg(page_table + (size_t)c.b * a.maxp + 2 * c.t + lane)
                 : 0;
    };
    int id = n > 0 ? page_id(cur) : 0;
    for (long long i = 0; ok && i < n; ++i) {
      TileCursor next = cur;
      next.step();
      const int id_next = i + 1 < n ? page_id(next) : 0;
      const int np = min(2, npages_of(cur.L) - 2 * cur.t);
      if (lane < np && (id < 0 || id >= a.num_pages)) {  // reported, and read from page 0 instead
        report_error(err, kErrDeviceCheck, cur.b, (2 * cur.t + lane) * kPage);
        id = 0;
      }
      for (int k = 0; k < blocks; ++k) {
        const int s = ring.i;
        if (filled == size) {
          ok = mbar_wait_warp(smem_u32(&empty[s]), ring.round ^ 1u, abort_flag, err, rope ? kWsRopeRing : kWsRing);
          if (!ok) break;
        } else {
          ++filled;
        }
        const uint32_t fb = smem_u32(&full[s]);
        if (lane == 0) mbar_expect_tx(fb, (uint32_t)np * (kWtBlock / 2));
        __syncwarp();
        if (lane < np) tma_load_2d(smem_u32(to + s * kWtBlock + lane * (kWtBlock / 2)), map, fb, 64 * k, id * kPage);
        __syncwarp();
        ring.step(size);
      }
      cur = next;
      id = id_next;
    }
    if (!ok)  // what is still on its way; the block that was waited for had landed before
      for (int k = 0; k < filled; ++k, ring.step(size)) drain_wait(smem_u32(&full[ring.i]), ring.round ^ 1u);
  } else if (warp == 2) {
    // ------------------------------------------------------------ the query
    uint32_t seg = 0;
    for (long long i = 0; i < n; ++i, cur.step()) {
      if (!cur.first) continue;
      if (seg > 0 && !mbar_wait_warp(smem_u32(&bars->q_empty), (seg - 1) & 1, abort_flag, err, kWsQEmpty)) break;
      const uint32_t fb = smem_u32(&bars->q_full);
      if (lane == 0) mbar_expect_tx(fb, (uint32_t)(nblk * q_block));
      __syncwarp();
      if (lane < nblk) tma_load_3d(smem_u32(sQ + lane * q_block), &tm_q, fb, 64 * lane, 0, cur.b);
      __syncwarp();
      ++seg;
    }
    if (*abort_flag && seg > 0) drain_wait(smem_u32(&bars->q_full), (seg - 1) & 1);
  } else if (warp == 1) {
    // ------------------------------------------------------------- the MMAs
    if (elect_one()) {  // one thread: it waits, issues and commits
      const uint32_t idesc = idesc_bf16_f32(128, Hp, false, false);
      const int per = nlat / a.n_branch;  // latent blocks of a branch
      const uint64_t td0 = sdesc_sw128(smem_u32(sT), 16, 1024), qd0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t rd0 = sdesc_sw128(smem_u32(sR), 16, 1024);
      RingPos ring, rope, unit;  // the next latent block, the tile's rotary block, the next score buffer
      bool lap = false;    // every score buffer has been used
      uint32_t seg = 0;
      bool ok = true;
      // block q of the query against the block at td, into the unit's score buffer
      auto product = [&](int q, uint64_t td, bool add) {
        const uint64_t qd = qd0 + (uint64_t)(q * (q_block >> 4));
        const uint32_t d = tmem + (uint32_t)(unit.i * stride);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ss(d, td + (uint64_t)(2 * ks), qd + (uint64_t)(2 * ks), idesc, add || ks ? 1u : 0u);
      };
      auto landed = [&] {
        ok = mbar_wait(smem_u32(&bars->full[ring.i]), ring.round, abort_flag, err, kWsFull);
        tc_fence_after();
        return ok;
      };
      auto release = [&] {
        mma_commit(smem_u32(&bars->empty[ring.i]));
        ring.step(stages);
      };
      for (long long i = 0; ok && i < n; ++i, cur.step()) {
        if (cur.first) {
          ok = mbar_wait(smem_u32(&bars->q_full), seg & 1, abort_flag, err, kWsQFull);
          if (!ok) break;
          ++seg;
        }
        for (int br = 0, k = 0; ok && br < a.n_branch; ++br) {
          if (lap) ok = mbar_wait(smem_u32(&bars->s_free[unit.i]), unit.round ^ 1u, abort_flag, err, kWsFree);
          if (ok && br == 0) ok = mbar_wait(smem_u32(&bars->r_full[rope.i]), rope.round, abort_flag, err, kWsRope);
          if (!ok) break;
          tc_fence_after();
          product(nlat, rd0 + (uint64_t)(rope.i * (kWtBlock >> 4)), false);  // the rotary part starts every branch
          if (br + 1 == a.n_branch) mma_commit(smem_u32(&bars->r_empty[rope.i]));
          for (int e = 0; e < per; ++e, ++k) {
            if (!landed()) break;
            product(k, td0 + (uint64_t)(ring.i * (kWtBlock >> 4)), true);
            if (e + 1 == per) mma_commit(smem_u32(&bars->s_full[unit.i]));
            release();
          }
          unit.step(bufs);
          lap = lap || unit.i == 0;
        }
        rope.step(ropes);
        if (ok && cur.last()) mma_commit(smem_u32(&bars->q_empty));
      }
      if (!ok || *abort_flag) {
        mma_commit(smem_u32(&bars->drain));
        drain_wait(smem_u32(&bars->drain), 0);
      }
    }
    __syncwarp();
  } else if (warp >= kWtSmx0) {
    // ----------------------------------------------------- the exponentials
    const int quarter = warp & 3, half = (warp - kWtSmx0) >> 2;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const int row = quarter * 32 + lane;
    const int mid = (Hp / 16 + 1) / 2 * 16, c0 = half ? mid : 0, c1 = half ? Hp : mid;  // its heads
    RingPos u;
    uint32_t seg = 0;
    // weights gathered before, read a tile ahead
    auto gathered = [&](const TileCursor& c) {
      const int t = c.t * kWtTile + row;
      return half == 0 && w_in && c.b < a.B && t < c.L ? w_in[(size_t)c.b * maxL + t] : 0.f;
    };
    float before = n > 0 ? gathered(cur) : 0.f;
    for (long long i = 0; i < n; ++i) {
      TileCursor next = cur;
      next.step();
      const float before_next = i + 1 < n ? gathered(next) : 0.f;
      if (cur.first) {
        // a padded head, and one that attended nothing, add 2^-inf
        float* l = bars->lse[seg & 1];
        for (int e = threadIdx.x - kWtSmx0 * 32; e < a.n_branch * Hp; e += 256) {
          const int br = e / Hp, h = e % Hp;
          const float v = h < a.H ? __ldg(lse + ((size_t)cur.b * a.n_branch + br) * a.H + h) : INFINITY;
          l[e] = v == -INFINITY ? INFINITY : v;
        }
        named_barrier(1, 256);
        ++seg;
      }
      const int t = cur.t * kWtTile + row;
      const size_t at = (size_t)cur.b * maxL + t;
      const bool mine = half == 0 && t < cur.L;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int br = 0; br < a.n_branch; ++br, u.step(bufs)) {
        const int buf = u.i;
        const bool ok = mbar_wait_warp(smem_u32(&bars->s_full[buf]), u.round, abort_flag, err, kWsScores);
        tc_fence_after();
        if (ok) {
          const float* l = bars->lse[(seg - 1) & 1] + br * Hp;
          const uint32_t col = tmem + lane_off + (uint32_t)(buf * stride);
          // 2^(v - lse) of four heads from column c on
          auto add4 = [&](const uint32_t* v, int c) {
            const float4 r = *reinterpret_cast<const float4*>(l + c);
            sum[0] += ex2(__uint_as_float(v[0]) - r.x);
            sum[1] += ex2(__uint_as_float(v[1]) - r.y);
            sum[2] += ex2(__uint_as_float(v[2]) - r.z);
            sum[3] += ex2(__uint_as_float(v[3]) - r.w);
          };
          int c = c0;
          for (; c + 32 <= c1; c += 32) {
            uint32_t v[32];
            tmem_ld32(col + c, v);
#pragma unroll
            for (int j = 0; j < 32; j += 4) add4(v + j, c + j);
          }
          if (c < c1) {
            uint32_t v[16];
            tmem_ld16(col + c, v);
#pragma unroll
            for (int j = 0; j < 16; j += 4) add4(v + j, c + j);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->s_free[buf]));
      }
      const float s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
      if (half == 1) bars->half_sum[i & 1][row] = s;
      named_barrier(1, 256);
      if (mine) w_out[at] = before + (s + bars->half_sum[i & 1][row]);
      before = before_next;
      cur = next;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

int padded_heads(int H) { return (H + 15) / 16 * 16; }

}  // namespace

bool weights_tc_supported(int dtype, int H, int d_c, int d_r, int n_branch) {
  return dtype == MLRA_BF16 && d_r == 64 && H <= 128 && (d_c / n_branch) % 64 == 0 &&
         n_branch * ((H + 31) / 32 * 32) <= 512;
}

cudaError_t launch_weights_tc(const void* q_abs, const float* lse, const void* lat, const void* rop,
                              const int* page_table, const int* seq_lens, const float* w_in, float* w_out, int* err,
                              const WeightArgs& a, int sms, cudaStream_t st) {
  const int Hp = padded_heads(a.H), D = a.d_c + a.d_r;
  CUtensorMap tl, tr, tq;
  {
    const uint64_t rows = (uint64_t)a.num_pages * kPage;
    const uint64_t ld[2] = {(uint64_t)a.d_c, rows}, rd[2] = {(uint64_t)a.d_r, rows};
    const uint64_t ls[1] = {(uint64_t)a.d_c * 2}, rs[1] = {(uint64_t)a.d_r * 2};
    const uint32_t box[2] = {64, 64};
    const uint64_t qd[3] = {(uint64_t)D, (uint64_t)a.H, (uint64_t)a.B};
    const uint64_t qs[2] = {(uint64_t)D * 2, (uint64_t)D * 2 * a.H};
    const uint32_t qbox[3] = {64, (uint32_t)Hp, 1};  // heads past H read as zeros
    if (!encode_bf16_map(&tl, 2, lat, ld, ls, box) || !encode_bf16_map(&tr, 2, rop, rd, rs, box) ||
        !encode_bf16_map(&tq, 3, q_abs, qd, qs, qbox))
      return cudaErrorInvalidValue;
  }
  const int q_bytes = query_bytes(Hp, D), fit = ring_blocks(Hp, D);
  if (fit < 3) return cudaErrorInvalidValue;
  // a second rotary block where there is room (128 heads: three latent blocks and one)
  const int ropes = fit < 6 ? 1 : kWtRopes, stages = fit - ropes < kWtStages ? fit - ropes : kWtStages;
  const int stride = (Hp + 31) / 32 * 32;
  const int bufs = 512 / stride < kWtBufs ? 512 / stride : kWtBufs;
  const int smem = 1024 + q_bytes + (stages + ropes) * kWtBlock + (int)sizeof(WtBars);
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(weights_tc_kernel), smem);
  if (e != cudaSuccess) return e;
  weights_tc_kernel<<<sms, kWtThreads, smem, st>>>(tl, tr, tq, lse, page_table, seq_lens, w_in, w_out, err, a, Hp,
                                                   stages, ropes, bufs);
  return cudaGetLastError();
}

}  // namespace mlra
