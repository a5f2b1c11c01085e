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
// Bound by memory for prompts (a row's bf16 read once, its codes written once)
// and by latency for single tokens (sequence search, page table, scale: loads
// that depend on each other).  Two forms:
//  - pages: a CTA takes a page's new rows for some heads of K, V or both, one
//    head after the other with the next one's rows on their way: the angles of
//    the page's rows are computed once, and a row's channels stay in registers
//    from their rotation over the maximum to their codes (16000 rows of 8 heads
//    of 128: 26.7 us, 3.7 TB/s, 23.9 where they lie in the L2; 46 % of the issue
//    slots are used: 260 CTAs on 304 places, each a chain from a head's rows over
//    a barrier for their maximum to their codes);
//  - rows: a warp takes the rows of one head of K or V in a page, a CTA eight
//    of them, so a decoded token's heads all run at once.
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

// Rows of sequence b in this call; a bad entry of cu_rows gives none.
__device__ __forceinline__ int64_t rows_of(const KvAppendArgs& a, int b) {
  if (!a.cu_rows) return 1;
  const int32_t lo = __ldg(a.cu_rows + b), hi = __ldg(a.cu_rows + b + 1);
  if (lo < 0 || hi < lo || hi > a.n_rows) {
    record_error(a.status, kErrIndexRange);
    return 0;
  }
  return hi - lo;
}

// A page touched by the call: new rows [first, last) of it, from row src_row
// of k / v on.  (None, last <= first, only where overlapping sequences have more
// pages in all than an int counts.)
struct PageRows {
  int64_t page, pos0, src_row;  // pos0: position of the page's row 0
  int first, last;
};

// The work item's page; false where there is nothing to store.  Every thread
// of the CTA calls it.
template <int THREADS>
__device__ __forceinline__ bool find_page(const KvAppendArgs& a, int* sh, PageRows* p) {
  const PagedCache& c = a.cache;
  int b = blockIdx.x, index = 0;
  if (a.cu_rows) {
    b = find_item<THREADS>(
        a.B, b, b + 1 == static_cast<int>(gridDim.x),
        [&](int s) { return static_cast<int>(pages_of(__ldg(a.pos0 + s), rows_of(a, s), c.page_shift)); }, sh,
        &index);
    if (b < 0) return false;
  }
  const int64_t p0 = __ldg(a.pos0 + b);
  if (p0 < 0) return false;
  const int64_t pg = (p0 >> c.page_shift) + index;
  p->page = pg < c.table_stride ? __ldg(c.table + static_cast<int64_t>(b) * c.table_stride + pg) : -1;
  if (p->page < 0 || p->page >= c.n_pages) {
    if (threadIdx.x == 0) record_error(a.status, kErrIndexRange);
    return false;
  }
  const int64_t n = rows_of(a, b);
  p->pos0 = pg << c.page_shift;
  p->first = static_cast<int>(p0 > p->pos0 ? p0 - p->pos0 : 0);
  p->last = static_cast<int>(min(p0 + n - p->pos0, static_cast<int64_t>(c.page)));
  p->src_row = (a.cu_rows ? __ldg(a.cu_rows + b) : b) + (p->pos0 + p->first - p0);
  return true;
}

// The largest magnitude of an item and amax; NaN does not count, infinities
// do (see finite_max).
__device__ __forceinline__ float item_max(const float (&lo)[8], const float (&hi)[8], float amax) {
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = max3(amax, fabsf(lo[j]), fabsf(hi[j]));
  return amax;
}
__device__ __forceinline__ float finite_max(const float (&lo)[8], const float (&hi)[8], float amax) {
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fmaxf(finite_abs(lo[j]), finite_abs(hi[j])));
  return amax;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

// The scale's reciprocal, by which a power of two divides exactly.  A page that
// another program began can have any scale: its rows are divided here, and 1 is
// returned.
template <int NI>
__device__ __forceinline__ float divide_by(float s, float (&lo)[NI][8], float (&hi)[NI][8]) {
  if ((__float_as_uint(s) & 0x007FFFFFu) == 0u) return __frcp_rn(s);
#pragma unroll
  for (int k = 0; k < NI; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      lo[k][j] = __fdiv_rn(lo[k][j], s);
      hi[k][j] = __fdiv_rn(hi[k][j], s);
    }
  return 1.f;
}

// An item's 16 codes.
__device__ __forceinline__ void store_item(uint8_t* row, int cl, int ch, const float (&lo)[8], const float (&hi)[8],
                                           float inv) {
  const uint64_t inv2 = pair_of(inv, inv);
  auto four = [&](const float* x) {
    float y[4];
    split(mul2(pair_of(x[0], x[1]), inv2), &y[0], &y[1]);
    split(mul2(pair_of(x[2], x[3]), inv2), &y[2], &y[3]);
    return e4m3_pair(y[0], y[1]) | e4m3_pair(y[2], y[3]) << 16;
  };
  const uint32_t w[4] = {four(lo), four(lo + 4), four(hi), four(hi + 4)};
  *reinterpret_cast<uint2*>(row + cl) = make_uint2(w[0], w[1]);
  *reinterpret_cast<uint2*>(row + ch) = make_uint2(w[2], w[3]);
}

// A page's older codes, `bytes` of them, to a scale that grew (threads tid of n).
__device__ __forceinline__ void round_again(uint8_t* codes, int bytes, float ratio, int tid, int n) {
  uint32_t* old = reinterpret_cast<uint32_t*>(codes);
  for (int i = tid; i < bytes >> 2; i += n) {
    const uint32_t w = old[i];
    const __half2 x(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xFFFFu), __NV_E4M3));
    const __half2 y(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3));
    const float2 fx = __half22float2(x), fy = __half22float2(y);
    old[i] = e4m3_pair(fx.x * ratio, fx.y * ratio) | e4m3_pair(fy.x * ratio, fy.y * ratio) << 16;
  }
}

__device__ __forceinline__ float scale_of(float amax, float was) {
  return fmaxf(was, __uint_as_float(static_cast<uint32_t>(e4m3_scale_exp(amax) + 127) << 23));
}

// K or V of the call, of one page and head.
struct Slab {
  uint8_t* codes;
  float* scale;
  const uint16_t* src;  // row `first`
  int64_t src_stride;
};
__device__ __forceinline__ Slab slab_of(const KvAppendArgs& a, const PageRows& p, int head, bool is_v) {
  const PagedCache& c = a.cache;
  const int64_t at = p.page * c.n_kv_heads + head;
  Slab s;
  s.codes = (is_v ? c.v : c.k) + (at << c.page_shift) * c.head_dim;
  s.scale = (is_v ? c.v_scale : c.k_scale) + at;
  s.src_stride = is_v ? a.v_stride : a.k_stride;
  s.src = (is_v ? a.v : a.k) + p.src_row * s.src_stride + head * (is_v ? a.v_stride_h : a.k_stride_h);
  return s;
}

// CTAs an SM (what their registers leave room for).
template <int THREADS, int NI>
constexpr int kPagesCtas = (NI == 1 ? 768 : 512) / THREADS;
template <int THREADS, int NI>
__global__ void __launch_bounds__(THREADS, kPagesCtas<THREADS, NI>)
    kv_append_pages_kernel(const KvAppendArgs a, const int heads) {
  constexpr int kWarps = THREADS / 32;
  extern __shared__ __align__(16) float2 sc_s[];  // K: the rows' (sin, cos), rope_dim / 2 each
  __shared__ int sh[kWarps + 2];
  __shared__ float max_s[2][kWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  PageRows p;
  if (!find_page<THREADS>(a, sh, &p)) return;
  const RopeArgs& rope = a.rope;
  const int pairs = rope.rope_dim >> 1, rotated = rope.rope_dim >> 4;
  const int items = a.cache.head_dim >> 4;  // a power of two
  const int items_shift = __ffs(items) - 1;
  const int n_items = (p.last - p.first) << items_shift;
  // K of the CTA's heads, then V of them, or (two CTAs in z) one of the two.
  // src: where the thread's items of the head to come begin (their second
  // chunks lie gap channels behind); dst: in a head's slab
  const int h0 = blockIdx.y * heads, nh = min(heads, a.cache.n_kv_heads - h0);
  const bool only_v = blockIdx.z != 0;
  const int k_steps = only_v ? 0 : nh, steps = gridDim.z == 1 ? 2 * nh : nh;
  Slab sl = slab_of(a, p, h0, only_v);
  const uint16_t* src[NI];
  int dst[NI], gap[NI];
  int64_t src_next = only_v ? a.v_stride_h : a.k_stride_h;
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int i = tid + k * THREADS;
    int cl, ch;
    item_chunks(rope, i & (items - 1), &cl, &ch);
    src[k] = sl.src + (i >> items_shift) * sl.src_stride + cl;
    dst[k] = (p.first + (i >> items_shift)) * a.cache.head_dim + cl;
    gap[k] = ch - cl;
  }
  uint4 u[NI], v[NI];  // the rows of the head to come
  auto fetch = [&]() {
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      u[k] = v[k] = make_uint4(0u, 0u, 0u, 0u);
      if (tid + k * THREADS >= n_items) continue;
      u[k] = __ldg(reinterpret_cast<const uint4*>(src[k]));
      v[k] = __ldg(reinterpret_cast<const uint4*>(src[k] + gap[k]));
      src[k] += src_next;
    }
  };
  fetch();
  for (int i = tid; k_steps > 0 && i < (p.last - p.first) * pairs; i += THREADS) {
    const int r = i / pairs, j = i - r * pairs;
    float s, c;
    rope_sincos_exact(p.pos0 + p.first + r, __ldg(rope.turns + j), &s, &c);
    sc_s[r * pairs + angle_slot(j, rotated)] = make_float2(s * rope.mscale, c * rope.mscale);
  }
  __syncthreads();
  for (int step = 0; step < steps; ++step) {
    if (step == nh) sl = slab_of(a, p, h0, true);
    const int turned = step < k_steps ? rotated : 0;
    const float was = p.first > 0 ? *sl.scale : 0.f;
    float lo[NI][8], hi[NI][8];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      const int i = tid + k * THREADS, it = i & (items - 1);
      unpack_bf16(u[k], lo[k]);
      unpack_bf16(v[k], hi[k]);
      if (it < turned && i < n_items) {
        float2 sc[8];
        load_angles(sc_s + (i >> items_shift) * pairs, it, rotated, sc);
        rotate_item(rope.half != 0, sc, lo[k], hi[k]);
      }
      amax = item_max(lo[k], hi[k], amax);
    }
    if (step + 1 == nh) {
      const Slab sv = slab_of(a, p, h0, true);
      src_next = a.v_stride_h;
#pragma unroll
      for (int k = 0; k < NI; ++k) {
        const int i = tid + k * THREADS;
        src[k] = sv.src + (i >> items_shift) * sv.src_stride + (dst[k] & (a.cache.head_dim - 1));
      }
    }
    if (step + 1 < steps) fetch();
    // (two arrays of maxima in turn: the next head's do not wait for this one's readers)
    float* top = max_s[step & 1];
    amax = warp_max(amax);
    if (lane == 0) top[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kWarps; ++k) amax = fmaxf(amax, top[k]);
    if (amax > FLT_MAX) {  // an infinity: the largest finite value decides (the whole CTA is here)
      __syncthreads();
      amax = 0.f;
#pragma unroll
      for (int k = 0; k < NI; ++k) amax = finite_max(lo[k], hi[k], amax);
      amax = warp_max(amax);
      if (lane == 0) top[warp] = amax;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kWarps; ++k) amax = fmaxf(amax, top[k]);
    }
    const float s = scale_of(amax, was), inv = divide_by(s, lo, hi);
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      if (tid + k * THREADS < n_items) store_item(sl.codes, dst[k], dst[k] + gap[k], lo[k], hi[k], inv);
    }
    if (p.first > 0 && s != was) round_again(sl.codes, p.first * a.cache.head_dim, __fdiv_rn(was, s), tid, THREADS);
    if (tid == 0 && n_items > 0 && (p.first == 0 || s != was)) *sl.scale = s;
    sl.codes += a.cache.page * a.cache.head_dim;
    ++sl.scale;
  }
}

constexpr int kRowThreads = 256;
__global__ void __launch_bounds__(kRowThreads) kv_append_rows_kernel(const KvAppendArgs a) {
  __shared__ int sh[kRowThreads / 32 + 2];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  PageRows p;
  if (!find_page<kRowThreads>(a, sh, &p)) return;
  const int which = blockIdx.y * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (which >= 2 * a.cache.n_kv_heads) return;
  const bool is_v = (which & 1) != 0;
  const Slab sl = slab_of(a, p, which >> 1, is_v);
  const float was = p.first > 0 ? *sl.scale : 0.f;
  RopeArgs rope = a.rope;
  if (is_v) rope.rope_dim = rope.offset = 0;
  const int items = a.cache.head_dim >> 4;  // 4 or 8: the warp takes 8 or 4 rows at a time
  const int it = lane & (items - 1), at_once = 32 / items;
  int cl, ch;
  item_chunks(rope, it, &cl, &ch);
  const int n = p.last - p.first;
  float lo[1][8], hi[1][8];
  auto load = [&](int r) {
    const uint16_t* row = sl.src + r * sl.src_stride;
    unpack_bf16(__ldg(reinterpret_cast<const uint4*>(row + cl)), lo[0]);
    unpack_bf16(__ldg(reinterpret_cast<const uint4*>(row + ch)), hi[0]);
    if (it < (rope.rope_dim >> 4)) {
      float2 sc[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        rope_sincos_exact(p.pos0 + p.first + r, __ldg(rope.turns + 8 * it + j), &sc[j].x, &sc[j].y);
        sc[j].x *= rope.mscale;
        sc[j].y *= rope.mscale;
      }
      rotate_item(rope.half != 0, sc, lo[0], hi[0]);
    }
  };
  float amax = 0.f;
  for (int r = lane / items; r < n; r += at_once) {
    load(r);
    amax = finite_max(lo[0], hi[0], amax);
  }
  amax = warp_max(amax);
  const float s = scale_of(amax, was);
  for (int r = lane / items; r < n; r += at_once) {
    if (n > at_once) load(r);  // (else still in registers)
    const float inv = divide_by(s, lo, hi);
    store_item(sl.codes + (p.first + r) * a.cache.head_dim, cl, ch, lo[0], hi[0], inv);
  }
  if (p.first > 0 && s != was) round_again(sl.codes, p.first * a.cache.head_dim, __fdiv_rn(was, s), lane, 32);
  if (lane == 0 && n > 0 && (p.first == 0 || s != was)) *sl.scale = s;
}

constexpr int kMaxAngles = 128 * 64 * static_cast<int>(sizeof(float2));  // of 128 rows of width 128
template <int THREADS, int NI>
cudaError_t launch_pages(const KvAppendArgs& a, unsigned items, int sms, cudaStream_t stream) {
  // A CTA a page, K and V of all heads; while the GPU has room for more CTAs, K
  // and V apart, then the heads in groups (each group computes the angles
  // anew).  us, one CTA a page and K and V apart: 5 prompts of 16000 rows in
  // all, 8 heads of 128, pages of 64 25.7 and 27.6; one of 16384, pages of 128
  // 27.1 and 35.0; 32 of up to 500 22.8 and 19.5; 64 times 4 rows 12.8, 6.4 with
  // two groups apart.
  const int H = a.cache.n_kv_heads;
  const int64_t slots = static_cast<int64_t>(sms) * kPagesCtas<THREADS, NI>;
  const int64_t pages = (a.n_rows >> a.cache.page_shift) + a.B;  // about
  const int z = 2 * slots >= 3 * pages ? 2 : 1;
  const int64_t fit = slots / (z * pages);
  const int groups = fit < 1 ? 1 : fit > H ? H : static_cast<int>(fit);
  const int heads = (H + groups - 1) / groups;
  const size_t smem = static_cast<size_t>(a.cache.page) * (a.rope.rope_dim / 2) * sizeof(float2);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = kernel_limits(reinterpret_cast<const void*>(kv_append_pages_kernel<THREADS, NI>), kMaxAngles, 0,
                                      &done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv_append_pages_kernel<THREADS, NI>, dim3(items, (H + heads - 1) / heads, z), dim3(THREADS), smem,
                    stream, a, heads);
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
  // Few rows a sequence: a warp a head (128 tokens of 8 heads of 64 4.2 us, 5.8
  // in the other form; one token 3.3 and 2.9).
  if (a.n_rows <= 2 * static_cast<int64_t>(a.B))
    return launch_pdl(kv_append_rows_kernel, dim3(x, (2 * a.cache.n_kv_heads + 7) / 8), dim3(kRowThreads), 0, stream,
                      a);
  const int sms = current_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // 16-channel items of a page: page * head_dim / 16, 64 .. 1024
  const int items = a.cache.page * a.cache.head_dim / 16;
  if (items <= 64) return launch_pages<64, 1>(a, x, sms, stream);
  if (items <= 128) return launch_pages<64, 2>(a, x, sms, stream);
  if (items <= 256) return launch_pages<128, 2>(a, x, sms, stream);
  if (items <= 512) return launch_pages<256, 2>(a, x, sms, stream);
  return launch_pages<512, 2>(a, x, sms, stream);
}

}  // namespace csa
