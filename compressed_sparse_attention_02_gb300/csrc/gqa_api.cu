// C ABI of the grouped-query layer's calls (declared in include/csa.h):
// rotary positions, the paged 8-bit cache's append and single-token attention,
// and packed prompt attention.  Host-side argument checks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/csa.h"
#include "kernels.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool rows_ok(const void* p) { return p && aligned(p, 16); }     // read and written 16 bytes at a time
bool words_ok(const void* p) { return p && aligned(p, 4); }     // int32 / fp32 arrays
bool words_opt(const void* p) { return aligned(p, 4); }

constexpr int kMaxHeads = 1024;
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int32_t kMaxSeqs = 1 << 20;  // (a warp's walk through them then takes some 30 ms)
// Rows of a prompt call: a CTA that walks all keys for one tile of queries then
// takes about a second, inside the limit of its other warps' waits.
constexpr int64_t kMaxPromptRows = int64_t(1) << 27;
constexpr int64_t kMaxStride = int64_t(1) << 38;  // elements (a tensor map's strides stay below 2^40 bytes)

// Element strides of rows and heads of a [rows][heads][dim] tensor.
bool strides_ok(int64_t row, int64_t head, int32_t dim) {
  return row >= dim && head >= dim && row < kMaxStride && head < kMaxStride && row % 8 == 0 && head % 8 == 0;
}

csa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? CSA_OK : CSA_ERR_CUDA; }

csa_status check_rope(const csa_rope_params* r, int32_t head_dim) {
  if (!r) return CSA_ERR_INVALID_ARG;
  if (r->rope_dim < 16 || r->rope_dim > 512 || r->rope_dim % 16 || r->offset < 0 || r->offset % 16)
    return CSA_ERR_UNSUPPORTED;
  if (head_dim > 0 && (r->offset > head_dim || r->rope_dim > head_dim - r->offset)) return CSA_ERR_INVALID_ARG;
  if ((r->layout != CSA_ROPE_INTERLEAVED && r->layout != CSA_ROPE_HALF) || r->scaling < CSA_ROPE_UNSCALED ||
      r->scaling > CSA_ROPE_BY_PARTS)
    return CSA_ERR_INVALID_ARG;
  if (!isfinite(r->theta) || !(r->theta >= 1.f) || !isfinite(r->mscale)) return CSA_ERR_INVALID_ARG;
  if (r->scaling != CSA_ROPE_UNSCALED && (!isfinite(r->factor) || !(r->factor >= 1.f))) return CSA_ERR_INVALID_ARG;
  if (r->scaling == CSA_ROPE_BY_PARTS &&
      (!(r->theta > 1.f) || r->orig_len < 1 || !(r->beta_slow > 0.f) || !(r->beta_fast > r->beta_slow) ||
       !isfinite(r->beta_fast)))
    return CSA_ERR_INVALID_ARG;
  return CSA_OK;
}

csa::RopeArgs rope_args(const csa_rope_params* r, const uint64_t* turns) {
  csa::RopeArgs a = {};
  if (!r) return a;
  a.turns = turns;
  a.rope_dim = r->rope_dim;
  a.offset = r->offset;
  a.half = r->layout == CSA_ROPE_HALF;
  a.mscale = r->mscale;
  return a;
}

// The cache's shape (for the workspace) and, for the calls, its pointers.
csa_status check_cache(const csa_paged_cache* c, bool pointers) {
  if (!c) return CSA_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return CSA_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return CSA_ERR_UNSUPPORTED;
  if (c->n_kv_heads < 1 || c->n_kv_heads > kMaxHeads) return CSA_ERR_INVALID_ARG;
  if (!pointers) return CSA_OK;
  if (c->n_pages < 1 || c->n_pages > 0x7fffffff || c->table_stride < 1 ||
      c->table_stride > kMaxRows / c->page_size)
    return CSA_ERR_INVALID_ARG;
  if (!rows_ok(c->k) || !rows_ok(c->v) || !words_ok(c->k_scale) || !words_ok(c->v_scale) || !words_ok(c->table))
    return CSA_ERR_INVALID_ARG;
  return CSA_OK;
}

csa::PagedCache cache_args(const csa_paged_cache* c) {
  csa::PagedCache a;
  a.n_kv_heads = c->n_kv_heads;
  a.head_dim = c->head_dim;
  a.page = c->page_size;
  a.page_shift = __builtin_ctz(static_cast<unsigned>(c->page_size));
  a.n_pages = c->n_pages;
  a.k = c->k;
  a.v = c->v;
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.table = c->table;
  a.table_stride = c->table_stride;
  return a;
}

bool heads_ok(int32_t n_heads, int32_t n_kv_heads) {
  return n_heads >= 1 && n_heads <= kMaxHeads && n_kv_heads >= 1 && n_heads % n_kv_heads == 0;
}

}  // namespace

namespace csa {

constexpr int kMaxDevices = 64;  // one bit a device

int current_sms() {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev >= 0 && dev < kMaxDevices && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev >= 0 && dev < kMaxDevices) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

cudaError_t kernel_limits(const void* kernel, int smem, int min_regs, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < kMaxDevices ? 1ull << dev : 0ull;
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  if (min_regs > 0) {
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, kernel);
    if (e != cudaSuccess) return e;
    if (at.numRegs < min_regs) return cudaErrorInvalidConfiguration;
  }
  done->fetch_or(bit, std::memory_order_release);
  return cudaSuccess;
}

}  // namespace csa

extern "C" {

void csa_default_rope(csa_rope_params* r) {
  if (!r) return;
  r->rope_dim = 128;
  r->offset = 0;
  r->layout = CSA_ROPE_HALF;
  r->scaling = CSA_ROPE_UNSCALED;
  r->theta = 10000.f;
  r->factor = 1.f;
  r->orig_len = 4096;
  r->beta_fast = 32.f;
  r->beta_slow = 1.f;
  r->mscale = 1.f;
}

csa_status csa_rope_table(const csa_rope_params* r, uint64_t* turns) {
  const csa_status s = check_rope(r, 0);
  if (s != CSA_OK) return s;
  if (!turns) return CSA_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  const double R = r->rope_dim, theta = r->theta, factor = r->factor;
  double low = 0, high = 0;
  if (r->scaling == CSA_ROPE_BY_PARTS) {
    // the pair whose wave turns beta times over the trained length
    auto pair_of = [&](double beta) { return R * log(r->orig_len / (beta * two_pi)) / (2 * log(theta)); };
    low = fmax(floor(pair_of(r->beta_fast)), 0.0);
    high = fmin(ceil(pair_of(r->beta_slow)), R - 1);
  }
  for (int j = 0; j < r->rope_dim / 2; ++j) {
    double f = pow(theta, -2.0 * j / R);
    if (r->scaling == CSA_ROPE_LINEAR) f /= factor;
    if (r->scaling == CSA_ROPE_BY_PARTS) {
      const double g = fmin(fmax((j - low) / fmax(high - low, 1e-3), 0.0), 1.0);
      f = f * (1 - g) + f / factor * g;
    }
    turns[j] = static_cast<uint64_t>(ldexp(f / two_pi, 64));
  }
  return CSA_OK;
}

csa_status csa_rope(const csa_rope_params* r, const uint64_t* turns, int64_t n_rows, int32_t n_heads,
                    int32_t head_dim, const int32_t* pos, const uint16_t* in, int64_t in_stride, int64_t in_stride_h,
                    uint16_t* out, int64_t out_stride, int64_t out_stride_h, int32_t inverse, void* stream) {
  if (head_dim < 16 || head_dim > 512 || head_dim % 16) return CSA_ERR_UNSUPPORTED;
  const csa_status s = check_rope(r, head_dim);
  if (s != CSA_OK) return s;
  if (n_rows < 0 || n_rows > kMaxRows || n_heads < 0 || n_heads > kMaxHeads || (inverse != 0 && inverse != 1))
    return CSA_ERR_INVALID_ARG;
  if (n_rows == 0 || n_heads == 0) return CSA_OK;
  if (!turns || !aligned(turns, 8) || !words_ok(pos) || !rows_ok(in) || !rows_ok(out)) return CSA_ERR_INVALID_ARG;
  if (!strides_ok(in_stride, in_stride_h, head_dim) || !strides_ok(out_stride, out_stride_h, head_dim))
    return CSA_ERR_INVALID_ARG;
  if (in == out && (in_stride != out_stride || in_stride_h != out_stride_h)) return CSA_ERR_INVALID_ARG;
  csa::RopeRowsArgs a = {};
  a.rope = rope_args(r, turns);
  a.n_rows = n_rows;
  a.n_heads = n_heads;
  a.head_dim = head_dim;
  a.pos = pos;
  a.in = in;
  a.in_stride = in_stride;
  a.in_stride_h = in_stride_h;
  a.out = out;
  a.out_stride = out_stride;
  a.out_stride_h = out_stride_h;
  a.inverse = inverse;
  return cuda_status(csa::launch_rope(a, static_cast<cudaStream_t>(stream)));
}

csa_status csa_kv_append(const csa_paged_cache* c, const csa_rope_params* r, const uint64_t* turns, int32_t B,
                         int64_t n_rows, const int32_t* cu_rows, const int32_t* pos0, const uint16_t* k,
                         int64_t k_stride, int64_t k_stride_h, const uint16_t* v, int64_t v_stride,
                         int64_t v_stride_h, void* stream) {
  csa_status s = check_cache(c, true);
  if (s != CSA_OK) return s;
  if (r && (s = check_rope(r, c->head_dim)) != CSA_OK) return s;
  if (B < 0 || B > kMaxSeqs || n_rows < 0 || n_rows > kMaxRows) return CSA_ERR_INVALID_ARG;
  if (!cu_rows && n_rows != B) return CSA_ERR_INVALID_ARG;
  if (B == 0 || n_rows == 0) return CSA_OK;
  if ((r && (!turns || !aligned(turns, 8))) || !words_opt(cu_rows) || !words_ok(pos0) || !rows_ok(k) || !rows_ok(v))
    return CSA_ERR_INVALID_ARG;
  if (!strides_ok(k_stride, k_stride_h, c->head_dim) || !strides_ok(v_stride, v_stride_h, c->head_dim))
    return CSA_ERR_INVALID_ARG;
  csa::KvAppendArgs a = {};
  a.cache = cache_args(c);
  a.rope = rope_args(r, turns);
  a.B = B;
  a.n_rows = n_rows;
  a.cu_rows = cu_rows;
  a.pos0 = pos0;
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.k_stride_h = k_stride_h;
  a.v_stride = v_stride;
  a.v_stride_h = v_stride_h;
  a.status = csa::device_status();
  if (!a.status) return CSA_ERR_CUDA;
  return cuda_status(csa::launch_kv_append(a, static_cast<cudaStream_t>(stream)));
}

size_t csa_paged_attn_workspace_size(const csa_paged_cache* c, int32_t B, int32_t n_heads) {
  if (check_cache(c, false) != CSA_OK || B < 0 || !heads_ok(n_heads, c->n_kv_heads)) return 0;
  const int sms = csa::current_sms();
  return sms > 0 ? csa::paged_attn_bytes(c->head_dim, sms) : 0;
}

csa_status csa_paged_attn(const csa_paged_cache* c, int32_t B, int32_t n_heads, const int32_t* lens,
                          const uint16_t* q, int64_t q_stride, int64_t q_stride_h, float sm_scale, int32_t window,
                          const float* sink, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                          void* stream) {
  const csa_status s = check_cache(c, true);
  if (s != CSA_OK) return s;
  if (B < 0 || B > kMaxSeqs || !heads_ok(n_heads, c->n_kv_heads) || window < 0 || !isfinite(sm_scale) ||
      !(sm_scale > 0.f))
    return CSA_ERR_INVALID_ARG;
  if (B == 0) return CSA_OK;
  if (!words_ok(lens) || !rows_ok(q) || !words_opt(sink) || !rows_ok(out) || !words_opt(lse) ||
      !strides_ok(q_stride, q_stride_h, c->head_dim))
    return CSA_ERR_INVALID_ARG;
  csa::PagedAttnArgs a = {};
  a.status = csa::device_status();
  const int sms = csa::current_sms();
  if (!a.status || sms <= 0) return CSA_ERR_CUDA;
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < csa::paged_attn_bytes(c->head_dim, sms))
    return CSA_ERR_WORKSPACE;
  a.cache = cache_args(c);
  a.B = B;
  a.n_heads = n_heads;
  a.lens = lens;
  a.q = q;
  a.q_stride = q_stride;
  a.q_stride_h = q_stride_h;
  a.sm_scale = sm_scale;
  a.window = window;
  a.sink = sink;
  a.out = out;
  a.lse = lse;
  a.part = static_cast<float*>(workspace);
  return cuda_status(csa::launch_paged_attn(a, sms, static_cast<cudaStream_t>(stream)));
}

csa_status csa_prompt_attn(int32_t B, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int64_t n_q,
                           int64_t n_k, const int32_t* cu_q, const int32_t* cu_k, const uint16_t* q,
                           int64_t q_stride, int64_t q_stride_h, const uint16_t* k, int64_t k_stride,
                           int64_t k_stride_h, const uint16_t* v, int64_t v_stride, int64_t v_stride_h,
                           float sm_scale, int32_t causal, int32_t window, const float* sink, uint16_t* out,
                           float* lse, void* stream) {
  if (head_dim != 64 && head_dim != 128) return CSA_ERR_UNSUPPORTED;
  if (B < 0 || !heads_ok(n_heads, n_kv_heads) || n_q < 0 || n_q > kMaxPromptRows || n_k < 0 ||
      n_k > kMaxPromptRows || B > kMaxSeqs ||
      (causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal) || !isfinite(sm_scale) ||
      !(sm_scale > 0.f))
    return CSA_ERR_INVALID_ARG;
  if (B == 0 || n_q == 0) return CSA_OK;
  if ((n_q / 128 + B) * n_heads >= (int64_t(1) << 30)) return CSA_ERR_UNSUPPORTED;  // tiles of 128 queries, all heads
  if (!words_ok(cu_q) || !words_ok(cu_k) || !rows_ok(q) || !words_opt(sink) || !rows_ok(out) || !words_opt(lse) ||
      (n_k > 0 && (!rows_ok(k) || !rows_ok(v))))
    return CSA_ERR_INVALID_ARG;
  if (!strides_ok(q_stride, q_stride_h, head_dim) || !strides_ok(k_stride, k_stride_h, head_dim) ||
      !strides_ok(v_stride, v_stride_h, head_dim))
    return CSA_ERR_INVALID_ARG;
  csa::PromptAttnArgs a = {};
  a.status = csa::device_status();
  if (!a.status) return CSA_ERR_CUDA;
  a.B = B;
  a.n_heads = n_heads;
  a.n_kv_heads = n_kv_heads;
  a.head_dim = head_dim;
  a.n_q = n_q;
  a.n_k = n_k;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.q_stride_h = q_stride_h;
  a.k_stride = k_stride;
  a.k_stride_h = k_stride_h;
  a.v_stride = v_stride;
  a.v_stride_h = v_stride_h;
  a.sm_scale = sm_scale;
  a.no_key = -1e30f / fmaxf(1.5f * sm_scale, 1.f);  // (the kernel's scale has a factor log2(e) more)
  a.causal = causal;
  a.window = window;
  a.sink = sink;
  a.out = out;
  a.lse = lse;
  return cuda_status(csa::launch_prompt_attn(a, csa::tensor_map_encoder(), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
