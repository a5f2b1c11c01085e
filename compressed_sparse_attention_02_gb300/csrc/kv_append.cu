// Appending key and value rows to a paged E4M3 cache, keys rotated on the way
// ("CSA2 详解" §16 sizes the 8-bit caches; the scale rule is the FP4 indexer
// keys', the least power of two that leaves no code saturated).
//
// For a page and head with the rows that the call adds: s = 2^e, e the
// smallest exponent with max |x| <= 448 * 2^e over the new rows, never below
// the scale of the rows already there; a row's code is the E4M3 value nearest
// to x / s.  A scale that grows re-rounds the page's older codes to the new
// one, which is exact but for codes that become subnormal (powers of two).
//
// One CTA per (page touched, head, K or V): it holds the page's new rows in
// registers, 16 channels an item, rotates them, takes their maximum and
// stores the codes, so the rows are read once and the codes written once.
// Bound by memory for prompts and by latency (sequence search, page table,
// row, scale: dependent loads) for single tokens.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <float.h>

#include "gqa.cuh"
#include "ptx.cuh"

namespace csa {
namespace {

// Two values to E4M3 codes (nearest, ties to even), the first in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float x, float y) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3));
}

// The smallest exponent e >= -126 with amax <= 448 * 2^e: amax = f * 2^E, f
// in [1, 2), and 448 = 1.75 * 2^8.
__device__ __forceinline__ int e4m3_scale_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int E = static_cast<int>(b >> 23) - 127;
  const int e = (b & 0x007FFFFFu) <= 0x00600000u ? E - 8 : E - 7;
  return e < -126 ? -126 : e;
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= FLT_MAX ? a : 0.f;
}

// Pages that n rows from position p touch.
__device__ __forceinline__ int64_t pages_of(int64_t p, int64_t n, int shift) {
  return n > 0 && p >= 0 ? ((p + n - 1) >> shift) - (p >> shift) + 1 : 0;
}

template <int THREADS, int NI>
__global__ void __launch_bounds__(THREADS) kv_append_kernel(const KvAppendArgs a) {
  constexpr int kWarps = THREADS / 32;
  __shared__ int sh[kWarps + 2];
  __shared__ float max_s[kWarps];
  pdl_launch_dependents();
  pdl_wait();
  const PagedCache& c = a.cache;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = blockIdx.y;
  const bool is_v = blockIdx.z != 0;

  // the sequence and the page of this work item
  auto rows_of = [&](int b) -> int64_t {
    if (!a.cu_rows) return 1;
    const int32_t lo = __ldg(a.cu_rows + b), hi = __ldg(a.cu_rows + b + 1);
    if (lo < 0 || hi < lo || hi > a.n_rows) {
      record_error(a.status, kErrIndexRange);
      return 0;
    }
    return hi - lo;
  };
  int b;
  int index = 0;
  if (!a.cu_rows) {
    b = blockIdx.x;
  } else {
    b = find_item<THREADS>(
        a.B, static_cast<int>(blockIdx.x),
        [&](int s) { return static_cast<int>(pages_of(__ldg(a.pos0 + s), rows_of(s), c.page_shift)); }, sh, &index);
    if (b < 0) return;
  }
  const int64_t p0 = __ldg(a.pos0 + b);
  if (p0 < 0) return;
  const int64_t row0 = a.cu_rows ? __ldg(a.cu_rows + b) : b;
  const int64_t n = rows_of(b);
  const int64_t pg = (p0 >> c.page_shift) + index;
  int64_t page = -1;
  if (pg < c.table_stride) page = __ldg(c.table + static_cast<int64_t>(b) * c.table_stride + pg);
  if (page < 0 || page >= c.n_pages) {
    if (tid == 0) record_error(a.status, kErrIndexRange);
    return;
  }
  const int64_t start = pg << c.page_shift;
  const int first = static_cast<int>(p0 > start ? p0 - start : 0);  // rows there before
  const int last = static_cast<int>(min(p0 + n - start, static_cast<int64_t>(c.page)));
  const int64_t slab = page * c.n_kv_heads + head;
  uint8_t* codes = (is_v ? c.v : c.k) + (slab << c.page_shift) * c.head_dim;
  float* scale_at = (is_v ? c.v_scale : c.k_scale) + slab;
  const float was = first > 0 ? *scale_at : 0.f;
  const uint16_t* src = (is_v ? a.v : a.k) + (row0 + (start + first - p0)) * (is_v ? a.v_stride : a.k_stride) +
                        head * (is_v ? a.v_stride_h : a.k_stride_h);
  const int64_t src_stride = is_v ? a.v_stride : a.k_stride;
  RopeArgs rope = a.rope;
  if (is_v) rope.rope_dim = rope.offset = 0;

  // new rows into registers, rotated; their largest magnitude
  const int items = c.head_dim >> 4;  // a power of two
  const int items_shift = __ffs(items) - 1;
  const int n_items = (last - first) << items_shift;
  float lo[NI][8], hi[NI][8];
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int i = tid + k * THREADS;
    if (i >= n_items) continue;
    int cl, ch;
    item_chunks(rope, i & (items - 1), &cl, &ch);
    const uint16_t* row = src + (i >> items_shift) * src_stride;
    unpack_bf16(__ldg(reinterpret_cast<const uint4*>(row + cl)), lo[k]);
    unpack_bf16(__ldg(reinterpret_cast<const uint4*>(row + ch)), hi[k]);
  }
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int i = tid + k * THREADS;
    if (i >= n_items) continue;
    const int it = i & (items - 1);
    if (it < (rope.rope_dim >> 4)) {
      float2 sc[8];
      const int64_t pos = start + first + (i >> items_shift);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        rope_sincos_exact(pos, __ldg(rope.turns + 8 * it + j), &sc[j].x, &sc[j].y);
        sc[j].x *= rope.mscale;
        sc[j].y *= rope.mscale;
      }
      rotate_item(rope.half != 0, sc, lo[k], hi[k]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fmaxf(finite_abs(lo[k][j]), finite_abs(hi[k][j])));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  if (lane == 0) max_s[warp] = amax;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kWarps; ++k) amax = fmaxf(amax, max_s[k]);
  const float s = fmaxf(was, ldexpf(1.f, e4m3_scale_exp(amax)));
  const float inv = __frcp_rn(s);  // exact for a power of two

#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int i = tid + k * THREADS;
    if (i >= n_items) continue;
    int cl, ch;
    item_chunks(rope, i & (items - 1), &cl, &ch);
    uint8_t* row = codes + static_cast<int64_t>(first + (i >> items_shift)) * c.head_dim;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w[j] = e4m3_pair(lo[k][4 * j] * inv, lo[k][4 * j + 1] * inv) |
             e4m3_pair(lo[k][4 * j + 2] * inv, lo[k][4 * j + 3] * inv) << 16;
      w[2 + j] = e4m3_pair(hi[k][4 * j] * inv, hi[k][4 * j + 1] * inv) |
                 e4m3_pair(hi[k][4 * j + 2] * inv, hi[k][4 * j + 3] * inv) << 16;
    }
    *reinterpret_cast<uint2*>(row + cl) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(row + ch) = make_uint2(w[2], w[3]);
  }
  // older rows of the page, re-rounded to a scale that grew
  if (first > 0 && s != was) {
    const float ratio = __fdiv_rn(was, s);
    uint32_t* old = reinterpret_cast<uint32_t*>(codes);
    for (int i = tid; i < (first * c.head_dim) >> 2; i += THREADS) {
      const uint32_t w = old[i];
      const __half2 x(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xFFFFu), __NV_E4M3));
      const __half2 y(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3));
      const float2 fx = __half22float2(x), fy = __half22float2(y);
      old[i] = e4m3_pair(fx.x * ratio, fx.y * ratio) | e4m3_pair(fy.x * ratio, fy.y * ratio) << 16;
    }
  }
  if (tid == 0 && (first == 0 || s != was)) *scale_at = s;
}

template <int THREADS, int NI>
cudaError_t launch_items(const KvAppendArgs& a, unsigned gx, cudaStream_t stream) {
  return launch_pdl(kv_append_kernel<THREADS, NI>, dim3(gx, a.cache.n_kv_heads, 2), dim3(THREADS), 0, stream, a);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream) {
  if (a.B <= 0 || a.n_rows <= 0) return cudaSuccess;
  // Pages touched: n rows touch at most (n - 1) / page + 2 pages and at most
  // n, so all sequences together at most n_rows / page + 2 B and n_rows.
  const int64_t most = (a.n_rows >> a.cache.page_shift) + 2 * static_cast<int64_t>(a.B);
  const int64_t gx = a.cu_rows ? (most < a.n_rows ? most : a.n_rows) : a.B;
  if (gx > 0x7fffffff) return cudaErrorInvalidValue;
  const unsigned x = static_cast<unsigned>(gx);
  // 16-channel items of a page: page * head_dim / 16, 64 .. 1024
  const int items = a.cache.page * a.cache.head_dim / 16;
  if (items <= 64) return launch_items<64, 1>(a, x, stream);
  if (items <= 128) return launch_items<128, 1>(a, x, stream);
  if (items <= 256) return launch_items<128, 2>(a, x, stream);
  if (items <= 512) return launch_items<128, 4>(a, x, stream);
  return launch_items<256, 4>(a, x, stream);
}

}  // namespace csa
