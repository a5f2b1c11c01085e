// Single-token attention of grouped query heads over a paged E4M3 cache with
// one scale per page and head.
//
//   l_j = sm_scale * k_scale(page) * q . codes_j,   p_j = e^(l_j - m)
//   out = sum_j p_j v_scale(page) codes^v_j / (sum_j p_j + e^(sink - m))
//
// Bound by memory: each cached row is read once (2 D bytes a token and head)
// for 4 D * group operations, so the products run on tensor cores at the
// group's size, up to 16 query heads as the 16 rows of one m16n8k16 product
// (a 128-row tcgen05 tile would be at least 7/8 empty).  The codes become
// f16 exactly; queries become f16 after scaling each row by a power of two to
// [2^14, 2^15), exact but for values 2^-28 below the row's largest.
//
// The tokens of all (sequence, head) pairs form one line of 32-token units
// that is cut into equal shares, one per resident warp, whatever the lengths
// are; a pair that a cut divides is finished by the merge kernel from fp32
// partial results in a fixed order.  A warp has its own ring of asynchronous
// copies, running maximum and accumulators: it waits for no other, and its
// copies run on into the next pair while it finishes one (with a share a CTA, whose
// warps joined their sums at each pair's end: 256 sequences of up to 600
// tokens 91 us, 47 so; 64 of up to 32768, 393 and 378 us, 6.7 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>

#include <type_traits>

#include "gqa.cuh"
#include "ptx.cuh"

namespace csa {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kUnitShift = 5;             // tokens a unit
constexpr int kUnit = 1 << kUnitShift;
constexpr int kRows = 16;                 // query heads a warp
// A maximum may lag behind by this much (in log2) before the accumulators are
// rescaled: weights are then at most 2^4 times 1, and as f16 they carry 2^11
// more, so weights down to 2^-25 of the largest keep f16's full precision.
constexpr float kLag = 4.f;
constexpr float kWeightExp = 11.f;
// A weight is the product of e^(l - m), which the sum takes, and a factor for
// the value scale and f16's exponents.  Where the factor passes 2^64 (value
// scales or logits far apart: a page of zero values has the scale 2^-126) the
// weight is one exponential instead: the factor could pass fp32, and up to
// here no weight that f16 holds (2^-24 and more) has an e^(l - m) that fp32 flushes.
constexpr float kFar = 64.f - kWeightExp;
constexpr float kNone = -1e31f;           // running maximum before the first token: below every logit times log2 e

// H: halves of the 16 rows that hold query heads (1: groups of up to 8).
template <int D, int H>
struct Cfg {
  // CTAs an SM and tiles in flight a warp.  At width 64 with 8 heads: 64
  // sequences of up to 8192 tokens 66 us with 3 CTAs and no spills, 85 with 4;
  // 96 under a window of 4096 77 and 80; a fourth tile changes nothing.
  static constexpr int kCtas = D == 64 ? 3 : 2;
  static constexpr int kStages = 3;
  static constexpr int kTileBytes = kUnit * D;              // K or V of a unit
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kSmem = kWarps * kWarpBytes;
};

template <int D>
constexpr int kRecord = kRows * (D + 4);  // floats of a partial result: sums, and a float4 a row: m, the weights'
                                          // sum (in units of 2^m), the sums' unit (log2, from m on), nothing

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros without reading.
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_4_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// c += a b; a of the halves that hold heads (the other half's rows are zero,
// and so stay its sums).
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], const uint32_t (&a)[2], uint32_t b0, uint32_t b1) {
  mma_f16_16816(c, {a[0], 0u, a[1], 0u}, b0, b1);
}

// Where 16-byte chunk c of row r of a 32-row tile lies: rows of 128 bytes
// with the chunk number XORed by the row, or two rows of 64 bytes a line with
// it XORed by twice the line, so that both the rows that a K fragment reads
// (8 neighbours) and those of a V fragment (every second one) fall into
// different banks.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  if constexpr (D == 128) return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
  return static_cast<uint32_t>((r >> 1) * 128 + (((((r & 1) << 2) | c) ^ (((r >> 1) & 3) << 1)) << 4));
}

// A sequence's visible tokens [lo, len) and its units.
struct Span {
  int len, lo;
  __device__ __forceinline__ int unit0() const { return lo >> kUnitShift; }
  __device__ __forceinline__ int units() const { return ((len + kUnit - 1) >> kUnitShift) - unit0(); }
};
__device__ __forceinline__ Span span_of(const PagedAttnArgs& a, int b) {
  Span s;
  const int64_t n = __ldg(a.lens + b), cap = a.cache.table_stride << a.cache.page_shift;
  if (n > cap) record_error(a.status, kErrIndexRange);
  s.len = static_cast<int>(n < 0 ? 0 : n > cap ? cap : n);
  s.lo = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
  return s;
}

// A place on the line: unit u of a pair (16-row block of a KV head's queries) of sequence b.
struct Place {
  Span sp;
  int b, pair, u;
  __device__ __forceinline__ int token() const { return (sp.unit0() + u) << kUnitShift; }
  __device__ __forceinline__ void advance(const PagedAttnArgs& a, int pairs) {
    if (++u < sp.units()) return;
    u = 0;
    if (++pair < pairs) return;
    pair = 0;
    do {
      ++b;
      sp.len = sp.lo = 0;
      if (b < a.B) sp = span_of(a, b);
    } while (b < a.B && sp.units() == 0);
  }
};

// What the merge has to know of a pair that begins in one share and ends in a later one.
struct __align__(16) Cut {
  int32_t row;    // first output row ([B][n_heads])
  int32_t rows;   // rows, doubled, + the first share's record of it (later shares: record 0); 0: no such pair
  int32_t first;  // the share in which it begins
  int32_t last;   // and ends
};
// They stand by share, and a share has at most one; by pair where there are few pairs, so that the merge
// needs no search (16 sequences of up to 4000 tokens, 8 heads: 24.9 us, 26.8 with a CTA a share; 32 sequences
// of 100 tokens: 14.5 us, 9.8 with a CTA a share).
__host__ __device__ __forceinline__ bool few_pairs(int64_t pairs, int64_t shares) { return pairs * 8 < shares; }

template <int D, int H>
__global__ void __launch_bounds__(kThreads, Cfg<D, H>::kCtas) paged_attn_kernel(const PagedAttnArgs a) {
  using C = Cfg<D, H>;
  constexpr int kK = D / 16;       // 16-channel steps of q . k
  constexpr int kN = D / 8;        // 8-channel tiles of the output
  constexpr int kChunks = D / 16;  // 16-byte chunks a row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t sh[kWarps], found_at[kWarps];
  __shared__ int found_b[kWarps];
  __shared__ float4 scale_s[kWarps][C::kStages];    // k, k, v, v scales of the unit's two halves
  __shared__ int bad_s[kWarps][C::kStages];         // halves whose page is outside the cache
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, cq = lane & 3;
  const PagedCache& cache = a.cache;
  const int group = a.n_heads / cache.n_kv_heads;
  const int blocks = (group + kRows - 1) / kRows;   // 16-row blocks a KV head
  const int pairs = cache.n_kv_heads * blocks;

  // The warps' shares of the line; neighbouring shares are of different CTAs,
  // so that a short line is spread over the SMs.
  const int64_t shares = static_cast<int64_t>(gridDim.x) * kWarps;
  const bool by_pair = few_pairs(static_cast<int64_t>(a.B) * pairs, shares);
  Cut* cuts = reinterpret_cast<Cut*>(a.part);
  float* records = a.part + shares * (sizeof(Cut) / sizeof(float));
  if (tid < kWarps) found_b[tid] = -1;
  // where the four shares begin, from the sequences' prefix sums; more than a block of sequences takes a pass
  // for the total first
  int64_t per = 1, total = 0;
  for (int pass = a.B > kThreads ? 0 : 1; pass < 2; ++pass) {
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
      const int b = b0 + tid;
      const int64_t n = b < a.B ? static_cast<int64_t>(span_of(a, b).units()) * pairs : 0;
      int64_t x = n;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      if (lane == 31) sh[warp] = x;
      __syncthreads();
      int64_t before = base + x - n;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const int64_t t = sh[k];
        if (k < warp) before += t;
        base += t;
      }
      if (a.B <= kThreads) total = base;
      if (pass == 1) {
        per = max((total + shares - 1) / shares, static_cast<int64_t>(1));
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const int64_t target = (static_cast<int64_t>(k) * gridDim.x + blockIdx.x) * per;
          if (target >= before && target < before + n) {  // one thread at most
            found_b[k] = b;
            found_at[k] = target - before;
          }
        }
      }
      __syncthreads();
    }
    total = base;
  }
  const int64_t share = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
  const int64_t begin = share * per;
  int left = static_cast<int>(max(min(total - begin, per), static_cast<int64_t>(0)));  // units to go
  // empty sequences, in turn over the CTAs
  for (int s = blockIdx.x; s < a.B; s += gridDim.x) {
    if (span_of(a, s).len > 0) continue;
    const int64_t row = static_cast<int64_t>(s) * a.n_heads;
    for (int i = tid; i < a.n_heads * D; i += kThreads) a.out[row * D + i] = 0;
    if (a.lse)
      for (int i = tid; i < a.n_heads; i += kThreads) a.lse[row + i] = a.sink ? __ldg(a.sink + i) : -INFINITY;
    if (by_pair)
      for (int i = tid; i < pairs; i += kThreads) cuts[s * pairs + i].rows = 0;
  }
  Cut cut = {0, 0, 0, 0};
  if (left == 0 || found_b[warp] < 0) {
    if (lane == 0 && !by_pair) cuts[share] = cut;
    return;
  }

  Place p, c;  // of the next copy and of the next unit worked on
  p.b = found_b[warp];
  p.sp = span_of(a, p.b);
  p.pair = static_cast<int>(found_at[warp] / p.sp.units());
  p.u = static_cast<int>(found_at[warp] - static_cast<int64_t>(p.pair) * p.sp.units());
  c = p;
  int to_copy = left, p_stage = 0, c_stage = 0;
  const uint32_t ring = smem_u32(smem) + warp * C::kWarpBytes;
  // page numbers are read a unit ahead (of the 16 tokens of the lane's half)
  auto page_of = [&](const Place& x) -> int32_t {
    const int t = x.token() + (lane & 16);
    return t < x.sp.len && t + 16 > x.sp.lo
               ? __ldg(cache.table + static_cast<int64_t>(x.b) * cache.table_stride + (t >> cache.page_shift))
               : -1;
  };
  int32_t next_page = page_of(p);
  auto issue = [&]() {
    if (to_copy > 0) {
      const int32_t mine = next_page;
      const Span sp = p.sp;
      const int t0 = p.token(), hk = blocks == 1 ? p.pair : p.pair / blocks, st = p_stage;
      if (--to_copy > 0) {
        p.advance(a, pairs);
        next_page = page_of(p);
      }
      p_stage = p_stage + 1 == C::kStages ? 0 : p_stage + 1;
      {
        const uint32_t ks = ring + st * C::kStageBytes, vs = ks + C::kTileBytes;
        const bool ok = mine >= 0 && mine < cache.n_pages;
        const int th = t0 + (lane & 16);
        const bool bad = !ok && th < sp.len && th + 16 > sp.lo;
        if (bad) record_error(a.status, kErrIndexRange);
        const unsigned bads = __ballot_sync(0xffffffffu, bad), oks = __ballot_sync(0xffffffffu, ok);
        const int32_t page_a = __shfl_sync(0xffffffffu, mine, 0), page_b = __shfl_sync(0xffffffffu, mine, 16);
        const bool ok_a = oks & 1u, ok_b = oks >> 31;
        const int in_page = cache.page - 1;
        const int64_t slab_a = ok_a ? static_cast<int64_t>(page_a) * cache.n_kv_heads + hk : 0;
        const int64_t slab_b = ok_b ? static_cast<int64_t>(page_b) * cache.n_kv_heads + hk : 0;
        const int64_t off_a = ((slab_a << cache.page_shift) + (t0 & in_page)) * D;
        const int64_t off_b = ((slab_b << cache.page_shift) + ((t0 + 16) & in_page)) * D - 16 * D;
        constexpr int kRowsAtOnce = 32 / kChunks;
        const int r0 = lane / kChunks, c = lane % kChunks;
        if (t0 >= sp.lo && t0 + kUnit <= sp.len && ok_a && ok_b) {  // (uniform) all rows are there
          const uint8_t *ka = cache.k + off_a + r0 * D + c * 16, *kb = cache.k + off_b + r0 * D + c * 16;
          const uint8_t *va = cache.v + off_a + r0 * D + c * 16, *vb = cache.v + off_b + r0 * D + c * 16;
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            const uint32_t dst = chunk_at<D>(r0 + i * kRowsAtOnce, c);
            const int off = i * kRowsAtOnce * D;
            cp_async_16(ks + dst, (i < kChunks / 2 ? ka : kb) + off);
            cp_async_16(vs + dst, (i < kChunks / 2 ? va : vb) + off);
          }
          if (lane < 4)
            cp_async_4_or_zero(smem_u32(&scale_s[warp][st]) + 4 * lane,
                               ((lane & 2) ? cache.v_scale : cache.k_scale) + ((lane & 1) ? slab_b : slab_a), true);
        } else {
#pragma unroll 1
          for (int i = 0; i < kChunks; ++i) {
            const int r = r0 + i * kRowsAtOnce, t = t0 + r;
            const bool first = i < kChunks / 2;  // rows below 16
            const bool there = (first ? ok_a : ok_b) && t >= sp.lo && t < sp.len;
            const int64_t off = (first ? off_a : off_b) + r * D + c * 16;
            const uint32_t dst = chunk_at<D>(r, c);
            cp_async_16_or_zero(ks + dst, there ? cache.k + off : cache.k, there);
            cp_async_16_or_zero(vs + dst, there ? cache.v + off : cache.v, there);
          }
          if (lane < 4) {
            const bool there = (lane & 1) ? ok_b : ok_a;
            const float* from = ((lane & 2) ? cache.v_scale : cache.k_scale) + ((lane & 1) ? slab_b : slab_a);
            cp_async_4_or_zero(smem_u32(&scale_s[warp][st]) + 4 * lane, from, there);
          }
        }
        if (lane == 0) bad_s[warp][st] = (bads & 1u) | ((bads >> 31) << 1);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) issue();

  bool first = true;
  while (left > 0) {
    const Span sp = c.sp;
    const int nt = sp.units(), take = min(nt - c.u, left);
    const int hk = blocks == 1 ? c.pair : c.pair / blocks, row0 = (c.pair - hk * blocks) * kRows;
    const int rows = min(kRows, group - row0);
    const int head0 = hk * group + row0;

    // the query rows g and g + 8 as fragments: lane cq holds channels
    // cq * D/4 .. of each, in the order in which it reads the keys' bytes
    uint32_t qf[kK][2 * H];
    float fac[H];
#pragma unroll
    for (int half = 0; half < H; ++half) {
      const int r = g + 8 * half;
      float x[D / 4];
      if (r < rows) {
        const uint16_t* row = a.q + c.b * a.q_stride + (head0 + r) * a.q_stride_h;
        const uint4* src = reinterpret_cast<const uint4*>(row + cq * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          float y[8];
          unpack_bf16(__ldg(src + i), y);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[8 * i + j] = y[j];
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 4; ++i) x[i] = 0.f;
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]) <= FLT_MAX ? fabsf(x[i]) : 0.f);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(14 - (static_cast<int>(__float_as_uint(top) >> 23) - 127), 126);
      const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
      fac[half] = a.sm_scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
      for (int s = 0; s < kK; ++s) {
        qf[s][half] = pack_f16(x[4 * s] * up, x[4 * s + 1] * up);
        qf[s][H + half] = pack_f16(x[4 * s + 2] * up, x[4 * s + 3] * up);
      }
    }

    float o[kN][4];
#pragma unroll
    for (int j = 0; j < kN; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    // the sums' reference 2^m; weighted values are in units of 2^(m + d - kWeightExp),
    // d the largest logit + log2(v_scale) seen from m (see finish_row); room: the value
    // scale up to which no weight is far
    float m[H], d[H], room = 0.f;
    uint64_t l2[H];  // sums of weights, as pairs of partial sums
#pragma unroll
    for (int h = 0; h < H; ++h) {
      m[h] = kNone;
      d[h] = 0.f;
      l2[h] = 0ull;
    }

    for (int it = 0; it < take; ++it) {
      cp_async_wait_pending(C::kStages - 2);
      __syncwarp();
      const int t0 = (sp.unit0() + c.u + it) << kUnitShift, st = c_stage;
      c_stage = c_stage + 1 == C::kStages ? 0 : c_stage + 1;
      do {
        const uint32_t ks = ring + st * C::kStageBytes, vs = ks + C::kTileBytes;
        // logits of 32 tokens: 4 tiles of 8
        float x[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
          const int r = 8 * n + g;
          uint32_t w[D / 16];
          if constexpr (D == 128) {
            const uint4 v0 = lds128(ks + chunk_at<D>(r, 2 * cq)), v1 = lds128(ks + chunk_at<D>(r, 2 * cq + 1));
            w[0] = v0.x; w[1] = v0.y; w[2] = v0.z; w[3] = v0.w;
            w[4] = v1.x; w[5] = v1.y; w[6] = v1.z; w[7] = v1.w;
          } else {
            const uint4 v0 = lds128(ks + chunk_at<D>(r, cq));
            w[0] = v0.x; w[1] = v0.y; w[2] = v0.z; w[3] = v0.w;
          }
#pragma unroll
          for (int s = 0; s < kK; ++s) {
            uint32_t b0, b1;
            e4m3x4_to_f16(w[s], b0, b1);
            mma_f16_16816(x[n], qf[s], b0, b1);
          }
        }
        const float4 sc = scale_s[warp][st];
        const int bad = bad_s[warp][st];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const float k = fac[h] * (n < 2 ? sc.x : sc.y);
            split(mul2(pair_of(x[n][2 * h], x[n][2 * h + 1]), pair_of(k, k)), &x[n][2 * h], &x[n][2 * h + 1]);
          }
        if (t0 < sp.lo || t0 + kUnit > sp.len || bad) {
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int t = t0 + 8 * n + 2 * cq + e;
              if (t < sp.lo || t >= sp.len || ((bad >> (n >> 1)) & 1))
#pragma unroll
                for (int h = 0; h < H; ++h) x[n][2 * h + e] = -INFINITY;
            }
        }
        // maxima of the logits, and of logit + log2(v_scale), the weights' exponents
        const float lv[2] = {__log2f(sc.z), __log2f(sc.w)};
        float tops[2][H];
        bool grown = sc.z > room || sc.w > room;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          tops[0][h] = fmaxf(fmaxf(x[0][2 * h], x[0][2 * h + 1]), fmaxf(x[1][2 * h], x[1][2 * h + 1]));
          tops[1][h] = fmaxf(fmaxf(x[2][2 * h], x[2][2 * h + 1]), fmaxf(x[3][2 * h], x[3][2 * h + 1]));
#pragma unroll
          for (int s = 0; s < 2; ++s) grown |= tops[s][h] - m[h] > fminf(kLag, d[h] + kLag - lv[s]);
        }
        uint32_t pf[2][2 * H];
        auto weights = [&](auto apart) {
#pragma unroll
          for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int h = 0; h < H; ++h) {
              const uint64_t mm = pair_of(-m[h], -m[h]);
              float p0, p1, p2, p3;
              split(add2(pair_of(x[2 * s][2 * h], x[2 * s][2 * h + 1]), mm), &p0, &p1);
              split(add2(pair_of(x[2 * s + 1][2 * h], x[2 * s + 1][2 * h + 1]), mm), &p2, &p3);
              const uint64_t p01 = pair_of(ex2(p0), ex2(p1)), p23 = pair_of(ex2(p2), ex2(p3));
              l2[h] = add2(l2[h], add2(p01, p23));
              if constexpr (apart) {
                const float up = lv[s] - d[h] + kWeightExp;
                p0 = ex2(p0 + up);
                p1 = ex2(p1 + up);
                p2 = ex2(p2 + up);
                p3 = ex2(p3 + up);
              } else {
                const float w = ex2(lv[s] - d[h] + kWeightExp);
                const uint64_t ww = pair_of(w, w);
                split(mul2(p01, ww), &p0, &p1);
                split(mul2(p23, ww), &p2, &p3);
              }
              pf[s][h] = pack_f16(p0, p1);
              pf[s][H + h] = pack_f16(p2, p3);
            }
        };
        // out += weights . V: tokens 2cq, 2cq+1, 2cq+8, 2cq+9 of each 16, the
        // bytes of two tokens paired by channel; lane group g holds channels
        // g * D/8 .. + D/8
        auto product = [&]() {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            uint32_t v[4][D / 32];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 16 * s + 2 * cq + (i & 1) + 8 * (i >> 1);
              if constexpr (D == 128) {
                const uint4 q4 = lds128(vs + chunk_at<D>(r, g));
                v[i][0] = q4.x; v[i][1] = q4.y; v[i][2] = q4.z; v[i][3] = q4.w;
              } else {
                const uint2 q2 = lds64(vs + chunk_at<D>(r, g >> 1) + 8 * (g & 1));
                v[i][0] = q2.x; v[i][1] = q2.y;
              }
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
              const uint32_t a01 = __byte_perm(v[0][w], v[1][w], 0x5140), a23 = __byte_perm(v[0][w], v[1][w], 0x7362);
              const uint32_t b01 = __byte_perm(v[2][w], v[3][w], 0x5140), b23 = __byte_perm(v[2][w], v[3][w], 0x7362);
              uint32_t p0, p1, q0, q1;
              e4m3x4_to_f16(a01, p0, p1);
              e4m3x4_to_f16(b01, q0, q1);
              mma_f16_16816(o[4 * w], pf[s], p0, q0);
              mma_f16_16816(o[4 * w + 1], pf[s], p1, q1);
              e4m3x4_to_f16(a23, p0, p1);
              e4m3x4_to_f16(b23, q0, q1);
              mma_f16_16816(o[4 * w + 2], pf[s], p0, q0);
              mma_f16_16816(o[4 * w + 3], pf[s], p1, q1);
            }
          }
        };
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
          for (int h = 0; h < H; ++h) {
            float m1 = fmaxf(m[h], fmaxf(tops[0][h], tops[1][h]));
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, off));
            const float d0 = d[h] + (m[h] - m1);
            float d1 = fmaxf(d0, fmaxf(tops[0][h] - m1 + lv[0], tops[1][h] - m1 + lv[1]));
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) d1 = fmaxf(d1, __shfl_xor_sync(0xffffffffu, d1, off));
            const float fl = ex2(m[h] - m1);
            l2[h] = mul2(l2[h], pair_of(fl, fl));
            const float f = ex2(d0 - d1);
#pragma unroll
            for (int j = 0; j < kN; ++j) {
              o[j][2 * h] *= f;
              o[j][2 * h + 1] *= f;
            }
            m[h] = m1;
            d[h] = d1;
            room = h == 0 ? d1 : fminf(room, d1);
          }
          room = ex2(room + kFar);
          if (__any_sync(0xffffffffu, sc.z > room || sc.w > room)) {
            // (a way of its own, so that the usual one is not cut by a branch: 96
            // sequences of width 64 under a window 78.7 us with the branch)
            weights(std::true_type{});
            product();
            break;
          }
        }
        weights(std::false_type{});
        product();
      } while (false);
      __syncwarp();
      issue();
    }
    // The pair's rows, or this share's part of them in units of 2^(m + d) / 2^kWeightExp
    // (not of 2^m: the two can be further apart than fp32's exponents).
    // Accumulator tile j holds channels 2cq * D/8 + j and (2cq + 1) * D/8 + j.
    const bool whole = take == nt;
    const int slot = first ? 0 : 1;
    float* part = records + (share * 2 + slot) * kRecord<D>;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int r = g + 8 * h;
      float l, other;
      split(l2[h], &l, &other);
      l += other;
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      const float unit = d[h] - kWeightExp;
      if (r >= rows) continue;
      if (whole) {
        const int64_t row = static_cast<int64_t>(c.b) * a.n_heads + head0 + r;
        float lse;
        const float f = finish_row(m[h], unit, l, a.sink, head0 + r, &lse);
        if (a.lse && cq == 0) a.lse[row] = lse;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + (2 * cq + e) * kN);
#pragma unroll
          for (int k = 0; k < kN / 8; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = 8 * k + 2 * i;
              const __nv_bfloat162 y = __floats2bfloat162_rn(o[j][2 * h + e] * f, o[j + 1][2 * h + e] * f);
              w[i] = *reinterpret_cast<const uint32_t*>(&y);
            }
            dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float4* dst = reinterpret_cast<float4*>(part + r * D + (2 * cq + e) * kN);
#pragma unroll
          for (int k = 0; k < kN / 4; ++k)
            dst[k] = make_float4(o[4 * k][2 * h + e], o[4 * k + 1][2 * h + e], o[4 * k + 2][2 * h + e],
                                 o[4 * k + 3][2 * h + e]);
        }
        if (cq == 0) *reinterpret_cast<float4*>(part + kRows * D + 4 * r) = make_float4(m[h], l, unit, 0.f);
      }
    }
    left -= take;
    if (c.u == 0) {  // the pair begins here
      if (!whole) {   // and goes on, so this is the whole of a share of `per` units
        cut.row = c.b * a.n_heads + head0;
        cut.rows = 2 * rows + slot;
        cut.first = static_cast<int>(share);
        cut.last = static_cast<int>((begin + (per - left) - take + nt - 1) / per);
      }
      if (by_pair && lane == 0) cuts[c.b * pairs + c.pair] = cut;
    }
    first = false;
    if (left > 0) {
      c.u += take - 1;
      c.advance(a, pairs);
    }
  }
  cp_async_wait_pending(0);
  if (lane == 0 && !by_pair) cuts[share] = cut;
}

// Finishes the pairs that the shares' borders divide, from their shares' records
// first to last.  With SPLIT 1 a CTA looks at one share's end, and a warp takes
// a row.  Else CTA (x, y) takes row y of pair x, each of its SPLIT warps a
// stretch of the records.
constexpr int merge_warps(int split) { return split == 1 ? 8 : split; }

template <int D, int SPLIT>
__global__ void __launch_bounds__(32 * merge_warps(SPLIT))
    paged_merge_kernel(const PagedAttnArgs a, const int shares) {
  constexpr int kMergeWarps = merge_warps(SPLIT);
  constexpr int kPer = D / 32;  // channels a lane, neighbours
  using Vec = typename std::conditional<kPer == 4, float4, float2>::type;
  __shared__ float m_s[kMergeWarps], u_s[kMergeWarps], l_s[kMergeWarps];
  __shared__ __align__(16) float n_s[kMergeWarps][D];
  pdl_launch_dependents();
  pdl_wait();
  const Cut cut = reinterpret_cast<const Cut*>(a.part)[blockIdx.x];
  const float* records = a.part + shares * (sizeof(Cut) / sizeof(float));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n_rec = cut.last - cut.first + 1, rows = cut.rows >> 1;
  auto record = [&](int k) {
    return records + (static_cast<int64_t>(cut.first + k) * 2 + (k == 0 ? cut.rows & 1 : 0)) * kRecord<D>;
  };
  for (int r = SPLIT == 1 ? warp : blockIdx.y; r < rows; r += SPLIT == 1 ? kMergeWarps : gridDim.y) {
    const int part = SPLIT == 1 ? 0 : warp;
    float m = kNone, unit = 0.f, l = 0.f, n[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) n[j] = 0.f;
    for (int k = part + lane * SPLIT; k < n_rec; k += 32 * SPLIT) {
      const float4 y = *reinterpret_cast<const float4*>(record(k) + kRows * D + 4 * r);
      join_units(m, unit, y.x, y.z);
    }
    join_lanes(m, unit);
#pragma unroll 4
    for (int k = part; k < n_rec; k += SPLIT) {
      const float* p = record(k);
      const float4 w = *reinterpret_cast<const float4*>(p + kRows * D + 4 * r);
      l += w.y * ex2(w.x - m);
      const float f = ex2(in_unit(w.x, w.z, m, unit));
      const Vec v = *reinterpret_cast<const Vec*>(p + r * D + lane * kPer);
      const float* y = reinterpret_cast<const float*>(&v);
#pragma unroll
      for (int j = 0; j < kPer; ++j) n[j] += y[j] * f;
    }
    if (SPLIT > 1) {  // the stretches' sums, first to last
      __syncthreads();
      if (lane == 0) {
        m_s[warp] = m;
        u_s[warp] = unit;
        l_s[warp] = l;
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) n_s[warp][lane * kPer + j] = n[j];
      __syncthreads();
      if (part != 0) continue;
      const float m0 = m, unit0 = unit;
#pragma unroll
      for (int w = 1; w < SPLIT; ++w) m = fmaxf(m, m_s[w]);
      unit += m0 - m;
#pragma unroll
      for (int w = 1; w < SPLIT; ++w) unit = fmaxf(unit, u_s[w] + (m_s[w] - m));
      l *= ex2(m0 - m);
      const float f0 = ex2(in_unit(m0, unit0, m, unit));
#pragma unroll
      for (int j = 0; j < kPer; ++j) n[j] *= f0;
      for (int w = 1; w < SPLIT; ++w) {
        l += l_s[w] * ex2(m_s[w] - m);
        const float f = ex2(in_unit(m_s[w], u_s[w], m, unit));
#pragma unroll
        for (int j = 0; j < kPer; ++j) n[j] += n_s[w][lane * kPer + j] * f;
      }
    }
    const int64_t row = static_cast<int64_t>(cut.row) + r;
    float lse;
    const float f = finish_row(m, unit, l, a.sink, static_cast<int>(row % a.n_heads), &lse);
    uint32_t y[kPer / 2];
#pragma unroll
    for (int j = 0; j < kPer / 2; ++j) {
      const __nv_bfloat162 two = __floats2bfloat162_rn(n[2 * j] * f, n[2 * j + 1] * f);
      y[j] = *reinterpret_cast<const uint32_t*>(&two);
    }
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row * D + lane * kPer);
    if constexpr (kPer == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
    else
      *dst = y[0];
    if (a.lse && lane == 0) a.lse[row] = lse;
  }
}

template <int D, int H>
cudaError_t launch_dim(const PagedAttnArgs& a, int sms, cudaStream_t stream) {
  using C = Cfg<D, H>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = kernel_limits(reinterpret_cast<const void*>(paged_attn_kernel<D, H>), C::kSmem, 0, &done);
  if (e != cudaSuccess) return e;
  const int ctas = sms * C::kCtas;
  e = launch_pdl(paged_attn_kernel<D, H>, dim3(ctas), dim3(kThreads), C::kSmem, stream, a);
  if (e != cudaSuccess) return e;
  const int group = a.n_heads / a.cache.n_kv_heads, rows = group < kRows ? group : kRows;
  const int64_t pairs = static_cast<int64_t>(a.B) * a.cache.n_kv_heads * ((group + kRows - 1) / kRows);
  // Many pairs: few records each, a warp a row.  Few pairs: a CTA a row, of 16
  // warps from 32 records a pair on (4 sequences of 32768 tokens, 4 heads: 22.2
  // us, 28.1 with 8; 16 of up to 4000, 10 records: 24.7 and 22.8).
  const int shares = ctas * kWarps;
  const dim3 grid(static_cast<unsigned>(pairs), rows);
  if (!few_pairs(pairs, shares))
    return launch_pdl(paged_merge_kernel<D, 1>, dim3(shares - 1), dim3(32 * merge_warps(1)), 0, stream, a, shares);
  if (pairs * 32 > shares)
    return launch_pdl(paged_merge_kernel<D, 8>, grid, dim3(32 * merge_warps(8)), 0, stream, a, shares);
  return launch_pdl(paged_merge_kernel<D, 16>, grid, dim3(32 * merge_warps(16)), 0, stream, a, shares);
}

}  // namespace

size_t paged_attn_bytes(int head_dim, int sms) {
  static_assert(Cfg<128, 1>::kCtas == Cfg<128, 2>::kCtas, "one size for both");
  const size_t ctas = static_cast<size_t>(sms) * (head_dim == 64 ? Cfg<64, 2>::kCtas : Cfg<128, 2>::kCtas);
  return ctas * kWarps * (sizeof(Cut) + 2 * kRows * (head_dim + 4) * sizeof(float));
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, int sms, cudaStream_t stream) {
  if (a.B <= 0) return cudaSuccess;
  if (a.cache.head_dim == 64) return launch_dim<64, 2>(a, sms, stream);
  // Groups of up to 8 leave the other half's softmax out (256 sequences of up
  // to 600 tokens, groups of 4: 46.9 us, 50.1 with it; 64 of up to 32768, groups
  // of 8: 378 and 381).  At width 64 that was no faster (96 sequences under a
  // window: 83 and 77 us).
  const bool low = a.n_heads / a.cache.n_kv_heads <= 8;
  return low ? launch_dim<128, 1>(a, sms, stream) : launch_dim<128, 2>(a, sms, stream);
}

}  // namespace csa
