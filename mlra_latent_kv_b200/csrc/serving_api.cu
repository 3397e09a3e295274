// C entry points of the prompt and eviction operators: argument checks,
// workspace layout and launches.  See include/mlra_serving.h.
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "gemm_tc.h"
#include "launch.h"
#include "prompt_path.h"
#include "serving.h"

namespace mlra {

bool encode_bf16_map(CUtensorMap* out, int rank, const void* base, const uint64_t* dims, const uint64_t* strides,
                     const uint32_t* box) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (!encode) return false;
  cuuint64_t d[5], s[4];
  cuuint32_t bx[5], es[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    bx[i] = box[i];
    es[i] = 1;
    if (i + 1 < rank) s[i] = strides[i];
  }
  return encode(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, s, bx, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

mlra_status bad(mlra_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
mlra_status bad(mlra_status st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return internal_fail(st, buf);
}

constexpr size_t kErrBytes = 256;
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Named {
  const void* p;
  const char* name;
  size_t align;
};
mlra_status check_ptrs(const Named* list, int n) {
  for (int i = 0; i < n; ++i) {
    if (!list[i].p) return bad(MLRA_ERR_INVALID_ARG, "%s is NULL", list[i].name);
    if (!aligned(list[i].p, list[i].align))
      return bad(MLRA_ERR_INVALID_ARG, "%s is not %zu-byte aligned", list[i].name, list[i].align);
  }
  return MLRA_OK;
}

mlra_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws) return bad(MLRA_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned(ws, 256)) return bad(MLRA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (have < need) return bad(MLRA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
  return MLRA_OK;
}

mlra_status launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? MLRA_OK : bad(MLRA_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

// SMs of the current device; 0 with the error recorded.
int device_sms() {
  int dev = 0, n = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    bad(MLRA_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
    return 0;
  }
  return n;
}

float scale_log2(const mlra_dims* d) {
  const float scale = d->softmax_scale > 0.f ? d->softmax_scale : 1.0f / std::sqrt((float)(d->d_h + d->d_r));
  return scale * 1.4426950408889634f;
}

// No C++ exception leaves a C entry point.
template <typename F>
mlra_status guarded(F f) {
  try {
    return f();
  } catch (...) {
    return MLRA_ERR_CUDA;
  }
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return x < y + nb && y < x + na;
}

// Outputs (the workspace is one) may share no byte with an input or with one another; an absent buffer has no bytes.
struct Span {
  const void* p;
  size_t n;
};
template <int kIn, int kOut>
mlra_status check_overlap(const Span (&in)[kIn], const Span (&outs)[kOut]) {
  auto meet = [](const Span& a, const Span& b) { return a.p && b.p && a.n && b.n && overlap(a.p, a.n, b.p, b.n); };
  for (int o = 0; o < kOut; ++o) {
    for (const Span& i : in)
      if (meet(i, outs[o])) return bad(MLRA_ERR_INVALID_ARG, "an output overlaps an input");
    for (int q = 0; q < o; ++q)
      if (meet(outs[q], outs[o])) return bad(MLRA_ERR_INVALID_ARG, "two outputs overlap");
  }
  return MLRA_OK;
}

size_t dtype_bytes(const mlra_dims* d) { return d->dtype == MLRA_BF16 ? 2 : 4; }
size_t pool_bytes(const mlra_dims* d, int width) { return (size_t)d->num_pages * kPage * width * dtype_bytes(d); }
size_t table_bytes(const mlra_dims* d) { return (size_t)d->B * d->max_pages_per_seq * 4; }

// ---------------------------------------------------------------------------
// prompt
// ---------------------------------------------------------------------------
mlra_status check_prompt(const mlra_dims* d, const mla_prompt_shape* s) {
  mlra_status st = internal_check_dims(d);
  if (st != MLRA_OK) return st;
  if (!s) return bad(MLRA_ERR_INVALID_ARG, "shape is NULL");
  if (d->n_branch != 1) return bad(MLRA_ERR_INVALID_ARG, "mla_prompt needs n_branch=1");
  if (s->kv_heads < 1 || d->H % s->kv_heads)
    return bad(MLRA_ERR_INVALID_ARG, "H=%d is not a multiple of kv_heads=%d", d->H, s->kv_heads);
  if (s->total_q < 0 || s->total_k < 0) return bad(MLRA_ERR_INVALID_ARG, "total_q and total_k must be >= 0");
  if (d->d_v > 512) return bad(MLRA_ERR_UNSUPPORTED, "d_v=%d: need <= 512", d->d_v);
  if (d->H > 65535) return bad(MLRA_ERR_UNSUPPORTED, "H=%d: need <= 65535", d->H);
  struct {
    const long long* s;
    const char* name;
    int heads, width, rows;
  } axes[] = {{s->q_nope_stride, "q_nope", d->H, d->d_h, s->total_q},
              {s->q_rope_stride, "q_rope", d->H, d->d_r, s->total_q},
              {s->k_nope_stride, "k_nope", s->kv_heads, d->d_h, s->total_k},
              {s->v_stride, "v", s->kv_heads, d->d_v, s->total_k}};
  for (const auto& x : axes) {
    if (x.s[0] < 0 || x.s[1] < 0 || x.s[0] >= (1LL << 37) || x.s[1] >= (1LL << 37))
      return bad(MLRA_ERR_INVALID_ARG, "strides of %s are out of range", x.name);
    if ((x.heads > 1 && x.s[1] < x.width) || (x.rows > 1 && x.s[0] < x.width))
      return bad(MLRA_ERR_INVALID_ARG, "strides of %s are smaller than a row", x.name);
  }
  return MLRA_OK;
}

PromptArgs prompt_args(const mlra_dims* d, const mla_prompt_shape* s) {
  PromptArgs a{d->B,       d->H,       s->kv_heads, d->d_h, d->d_r, d->d_v, d->max_pages_per_seq, d->num_pages,
               s->total_q, s->total_k, scale_log2(d), {}, {}, {}, {}};
  for (int i = 0; i < 2; ++i) {
    a.q_nope_s[i] = s->q_nope_stride[i];
    a.q_rope_s[i] = s->q_rope_stride[i];
    a.k_nope_s[i] = s->k_nope_stride[i];
    a.v_s[i] = s->v_stride[i];
  }
  return a;
}

// The workspace does not depend on the strides: the tcgen05 kernel's where the widths are its own.
size_t prompt_workspace(const mlra_dims* d, const PromptArgs& a) {
  return d->kernel != MLRA_KERNEL_SIMT && prompt_tc_supported(d->dtype, d->d_h, d->d_r, d->d_v) ? prompt_tc_workspace(a)
                                                                                                 : kErrBytes;
}

// Bytes from the first element of a packed array to behind its last.
size_t packed_bytes(const mlra_dims* d, int rows, int heads, int width, const long long* s) {
  return rows == 0 ? 0 : ((size_t)(rows - 1) * s[0] + (size_t)(heads - 1) * s[1] + width) * dtype_bytes(d);
}

// Copies by the tensor memory accelerator: 16-byte addresses and strides.
bool prompt_aligned(const PromptArgs& a, const void* q_nope, const void* q_rope, const void* k_nope, const void* v) {
  const void* p[] = {q_nope, q_rope, k_nope, v};
  const long long* s[] = {a.q_nope_s, a.q_rope_s, a.k_nope_s, a.v_s};
  const int rows[] = {a.total_q, a.total_q, a.total_k, a.total_k}, heads[] = {a.H, a.H, a.kv_heads, a.kv_heads};
  for (int i = 0; i < 4; ++i) {
    if (rows[i] == 0) continue;
    if (!aligned(p[i], 16) || (rows[i] > 1 && s[i][0] % 8) || (heads[i] > 1 && s[i][1] % 8)) return false;
  }
  return true;
}

}  // namespace
}  // namespace mlra

using namespace mlra;

extern "C" {

size_t mla_prompt_workspace_bytes(const mlra_dims* dims, const mla_prompt_shape* shape) {
  size_t n = 0;
  guarded([&] {
    mlra_status st = check_prompt(dims, shape);
    if (st == MLRA_OK) n = prompt_workspace(dims, prompt_args(dims, shape));
    return st;
  });
  return n;
}

mlra_status mla_prompt(const mlra_dims* dims, const mla_prompt_shape* shape, const void* q_nope, const void* q_rope,
                       const int32_t* cu_q, const void* k_nope, const void* v, const int32_t* cu_k,
                       const void* rope_cache, const int32_t* page_table, void* out, float* lse, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream) {
  return guarded([&]() -> mlra_status {
    mlra_status st = check_prompt(dims, shape);
    if (st != MLRA_OK) return st;
    const mlra_dims* d = dims;
    const mla_prompt_shape* s = shape;
    const size_t e = dtype_bytes(d);
    const Named ptrs[] = {{cu_q, "cu_q", 4},     {cu_k, "cu_k", 4}, {rope_cache, "rope_cache", 16},
                          {page_table, "page_table", 4}, {q_nope, "q_nope", e}, {q_rope, "q_rope", e},
                          {out, "out", 16},      {k_nope, "k_nope", e}, {v, "v", e}};
    if (s->total_q == 0) return MLRA_OK;  // nothing to write
    st = check_ptrs(ptrs, s->total_k == 0 ? 7 : 9);
    if (st == MLRA_OK && lse && !aligned(lse, 4)) st = bad(MLRA_ERR_INVALID_ARG, "lse is not 4-byte aligned");
    const PromptArgs a = prompt_args(d, s);
    if (st == MLRA_OK) st = check_workspace(workspace, workspace_bytes, prompt_workspace(d, a));
    if (st != MLRA_OK) return st;
    const bool fits = prompt_tc_supported(d->dtype, d->d_h, d->d_r, d->d_v) &&
                      prompt_aligned(a, q_nope, q_rope, k_nope, v);
    int regs = 0, want = 0;
    if (fits && d->kernel != MLRA_KERNEL_SIMT)
      if (cudaError_t err = prompt_tc_registers(&regs, &want))
        return bad(MLRA_ERR_CUDA, "query of the prompt kernel: %s", cudaGetErrorString(err));
    const PromptPath path = prompt_path(static_cast<mlra_kernel>(d->kernel), fits, regs, want);
    if (path == PromptPath::kNoShape)
      return bad(MLRA_ERR_UNSUPPORTED,
                 "the tcgen05 prompt kernel needs bf16, d_h=128, d_r=64, d_v=128 and 16-byte aligned rows");
    if (path == PromptPath::kNoRegisters)
      return bad(MLRA_ERR_UNSUPPORTED, "the tcgen05 prompt kernel was compiled to %d registers, not %d", regs, want);
    const size_t cu = (size_t)(d->B + 1) * 4, rows = (size_t)s->total_q * d->H;
    const Span in[] = {{q_nope, packed_bytes(d, s->total_q, d->H, d->d_h, s->q_nope_stride)},
                       {q_rope, packed_bytes(d, s->total_q, d->H, d->d_r, s->q_rope_stride)},
                       {k_nope, packed_bytes(d, s->total_k, s->kv_heads, d->d_h, s->k_nope_stride)},
                       {v, packed_bytes(d, s->total_k, s->kv_heads, d->d_v, s->v_stride)},
                       {cu_q, cu},
                       {cu_k, cu},
                       {rope_cache, pool_bytes(d, d->d_r)},
                       {page_table, table_bytes(d)}},
               outs[] = {{out, rows * d->d_v * e}, {lse, rows * 4}, {workspace, prompt_workspace(d, a)}};
    st = check_overlap(in, outs);
    if (st != MLRA_OK) return st;
    const RopeTable tab = internal_rope_table(d);
    if (path == PromptPath::kTc) {
      const int sms = device_sms();
      if (sms == 0) return MLRA_ERR_CUDA;
      return launched(launch_prompt_tc(q_nope, q_rope, cu_q, k_nope, v, cu_k, rope_cache, page_table, out, lse,
                                       workspace, a, tab, sms, stream),
                      "prompt attention");
    }
    int* err = static_cast<int*>(workspace);
    return launched(launch_prompt_simt(d->dtype, q_nope, q_rope, cu_q, k_nope, v, cu_k, rope_cache, page_table, out,
                                       lse, err, a, tab, stream),
                    "prompt attention");
  });
}

mlra_status mlra_absorb(const mlra_dims* dims, const void* q_nope, const void* q_rope, const int32_t* q_pos,
                        const void* W_UK, void* q_abs, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return guarded([&]() -> mlra_status {
    mlra_status st = internal_check_dims(dims);
    if (st != MLRA_OK) return st;
    const mlra_dims* d = dims;
    const Named ptrs[] = {{q_nope, "q_nope", 16}, {q_rope, "q_rope", 16}, {q_pos, "q_pos", 4},
                          {W_UK, "W_UK", 16},     {q_abs, "q_abs", 16}};
    st = check_ptrs(ptrs, 5);
    if (st == MLRA_OK) st = check_workspace(workspace, workspace_bytes, kErrBytes);
    if (st != MLRA_OK) return st;
    // the tcgen05 kernel writes rows of q_abs in 16-byte pieces
    const bool tc_ok = absorb_tc_supported(d->dtype, d->B, d->d_h, d->d_c) && d->d_r % 8 == 0;
    if (d->kernel == MLRA_KERNEL_TC && !tc_ok)
      return bad(MLRA_ERR_UNSUPPORTED, "the tcgen05 absorption does not take this shape");
    const size_t e = dtype_bytes(d), rows = (size_t)d->B * d->H;
    const Span in[] = {{q_nope, rows * d->d_h * e},
                       {q_rope, rows * d->d_r * e},
                       {q_pos, (size_t)d->B * 4},
                       {W_UK, (size_t)d->H * d->d_h * d->d_c * e}},
               outs[] = {{q_abs, rows * (d->d_c + d->d_r) * e}, {workspace, kErrBytes}};
    st = check_overlap(in, outs);
    if (st != MLRA_OK) return st;
    const RopeTable tab = internal_rope_table(d);
    const float q_scale = scale_log2(d);
    if (tc_ok && d->kernel != MLRA_KERNEL_SIMT) {
      const GemmArgs g{d->B, batch_pad(d->B), d->H, d->d_h, d->d_c, d->d_r, d->d_v, 1, d->n_branch,
                       d->max_pages_per_seq, 1.0f, q_scale, 0};
      return launched(launch_absorb_tc(q_nope, q_rope, q_pos, W_UK, q_abs, static_cast<int*>(workspace), g, tab,
                                       stream),
                      "absorption");
    }
    const AbsorbArgs a{d->B, d->H, d->H, d->d_h, d->d_c, d->d_r, q_scale};
    return launched(launch_absorb(d->dtype, d->dtype == MLRA_BF16, q_nope, q_rope, q_pos, W_UK, q_abs, a, tab, stream),
                    "absorption");
  });
}

mlra_status mlra_attention_weights(const mlra_dims* dims, const void* q_abs, const float* lse,
                                   const void* latent_cache, const void* rope_cache, const int32_t* page_table,
                                   const int32_t* seq_lens, const float* weights_in, float* weights, void* workspace,
                                   size_t workspace_bytes, cudaStream_t stream) {
  return guarded([&]() -> mlra_status {
    mlra_status st = internal_check_dims(dims);
    if (st != MLRA_OK) return st;
    const mlra_dims* d = dims;
    const Named ptrs[] = {{q_abs, "q_abs", 16},
                          {lse, "lse", 4},
                          {latent_cache, "latent_cache", 16},
                          {rope_cache, "rope_cache", 16},
                          {page_table, "page_table", 4},
                          {seq_lens, "seq_lens", 4},
                          {weights, "weights", 4}};
    st = check_ptrs(ptrs, 7);
    if (st == MLRA_OK && weights_in && !aligned(weights_in, 4))
      st = bad(MLRA_ERR_INVALID_ARG, "weights_in is not 4-byte aligned");
    const size_t bytes = table_bytes(d) * kPage;
    if (st == MLRA_OK && weights_in && weights_in != weights && overlap(weights_in, bytes, weights, bytes))
      st = bad(MLRA_ERR_INVALID_ARG, "weights_in and weights overlap in part");
    if (st == MLRA_OK) st = check_workspace(workspace, workspace_bytes, kErrBytes);
    if (st != MLRA_OK) return st;
    const bool tc_ok = weights_tc_supported(d->dtype, d->H, d->d_c, d->d_r, d->n_branch);
    if (d->kernel == MLRA_KERNEL_TC && !tc_ok)
      return bad(MLRA_ERR_UNSUPPORTED,
                 "the tcgen05 weights kernel needs bf16, d_r=64, branches of a multiple of 64 dims, H<=128 and "
                 "n_branch * H (in steps of 32) <= 512");
    const Span in[] = {{q_abs, (size_t)d->B * d->H * (d->d_c + d->d_r) * dtype_bytes(d)},
                       {lse, (size_t)d->B * d->n_branch * d->H * 4},
                       {latent_cache, pool_bytes(d, d->d_c)},
                       {rope_cache, pool_bytes(d, d->d_r)},
                       {page_table, table_bytes(d)},
                       {seq_lens, (size_t)d->B * 4}},
               outs[] = {{weights, bytes}, {workspace, kErrBytes}};
    st = check_overlap(in, outs);
    if (st == MLRA_OK && weights_in && overlap(weights_in, bytes, workspace, kErrBytes))
      st = bad(MLRA_ERR_INVALID_ARG, "an output overlaps an input");
    if (st != MLRA_OK) return st;
    const int sms = device_sms();
    if (sms == 0) return MLRA_ERR_CUDA;
    const WeightArgs a{d->B, d->H, d->d_c, d->d_r, d->n_branch, d->max_pages_per_seq, d->num_pages};
    int* err = static_cast<int*>(workspace);
    if (tc_ok && d->kernel != MLRA_KERNEL_SIMT)
      return launched(launch_weights_tc(q_abs, lse, latent_cache, rope_cache, page_table, seq_lens, weights_in,
                                        weights, err, a, sms, stream),
                      "attention weights");
    return launched(launch_weights_simt(d->dtype, q_abs, lse, latent_cache, rope_cache, page_table, seq_lens,
                                        weights_in, weights, err, a, sms, stream),
                    "attention weights");
  });
}

}  // extern "C"

namespace {

// error record | page owners | counts | source slots | destination slots
struct EvictLayout {
  size_t owners, counts, src, dst, total;
};
EvictLayout evict_layout(const mlra_dims* d) {
  EvictLayout l;
  const size_t list = (size_t)d->B * d->max_pages_per_seq * (kPage / 2) * 4;
  l.owners = kErrBytes;
  l.counts = round_up(l.owners + (size_t)d->num_pages * 4, 256);
  l.src = round_up(l.counts + (size_t)d->B * 4, 256);
  l.dst = round_up(l.src + list, 256);
  l.total = round_up(l.dst + list, 256);
  return l;
}

mlra_status check_evict(const mlra_dims* d) {
  mlra_status st = internal_check_dims(d);
  if (st != MLRA_OK) return st;
  if (d->B > 65535) return bad(MLRA_ERR_UNSUPPORTED, "B=%d: need <= 65535", d->B);
  if ((long long)d->num_pages * kPage > 0x7FFFFFFFLL)
    return bad(MLRA_ERR_UNSUPPORTED, "num_pages=%d: the pool's slots need 31 bits", d->num_pages);
  return MLRA_OK;
}

}  // namespace

extern "C" {

size_t latent_evict_workspace_bytes(const mlra_dims* dims) {
  size_t n = 0;
  guarded([&] {
    mlra_status st = check_evict(dims);
    if (st == MLRA_OK) n = evict_layout(dims).total;
    return st;
  });
  return n;
}

mlra_status latent_evict(const mlra_dims* dims, int recent, const int32_t* evict_pages, const float* weights,
                         const int32_t* page_table, const int32_t* seq_lens, void* latent_cache, void* rope_cache,
                         float* weights_out, int32_t* page_table_out, int32_t* seq_lens_out, void* workspace,
                         size_t workspace_bytes, cudaStream_t stream) {
  return guarded([&]() -> mlra_status {
    mlra_status st = check_evict(dims);
    if (st != MLRA_OK) return st;
    const mlra_dims* d = dims;
    if (recent < 0) return bad(MLRA_ERR_INVALID_ARG, "recent must be >= 0");
    const Named ptrs[] = {{evict_pages, "evict_pages", 4},   {weights, "weights", 4},
                          {page_table, "page_table", 4},     {seq_lens, "seq_lens", 4},
                          {latent_cache, "latent_cache", 16}, {rope_cache, "rope_cache", 16},
                          {weights_out, "weights_out", 4},   {page_table_out, "page_table_out", 4},
                          {seq_lens_out, "seq_lens_out", 4}};
    st = check_ptrs(ptrs, 9);
    if (st != MLRA_OK) return st;
    const EvictLayout l = evict_layout(d);
    st = check_workspace(workspace, workspace_bytes, l.total);
    if (st != MLRA_OK) return st;
    const size_t row = table_bytes(d), e = dtype_bytes(d);
    const Span in[] = {{evict_pages, (size_t)d->B * 4}, {weights, row * kPage}, {page_table, row},
                       {seq_lens, (size_t)d->B * 4}},
               outs[] = {{weights_out, row * kPage},
                         {page_table_out, row},
                         {seq_lens_out, (size_t)d->B * 4},
                         {latent_cache, pool_bytes(d, d->d_c)},
                         {rope_cache, pool_bytes(d, d->d_r)},
                         {workspace, l.total}};
    st = check_overlap(in, outs);
    if (st != MLRA_OK) return st;
    const int sms = device_sms();
    if (sms == 0) return MLRA_ERR_CUDA;
    char* ws = static_cast<char*>(workspace);
    const EvictWorkspace w{reinterpret_cast<int*>(ws + l.owners), reinterpret_cast<int*>(ws + l.counts),
                           reinterpret_cast<int*>(ws + l.src), reinterpret_cast<int*>(ws + l.dst)};
    const EvictArgs a{d->B, d->max_pages_per_seq, d->num_pages, recent, (int)(d->d_c * e), (int)(d->d_r * e)};
    return launched(launch_evict(evict_pages, weights, page_table, seq_lens, latent_cache, rope_cache, weights_out,
                                 page_table_out, seq_lens_out, reinterpret_cast<int*>(ws), w, a, sms, stream),
                    "latent_evict");
  });
}

}  // extern "C"
