// Shared pieces of the grouped-query layer's kernels: the rotation of an item
// of 16 channels, bf16 unpacking, and the search of a work item among
// sequences of different lengths.
#pragma once

#include <stdint.h>

#include "kernels.h"

namespace csa {

// Sine and cosine of position p at the frequency whose table entry is turns
// (2^-64 turns a position): the angle's fraction of a turn is the low 64 bits
// of p * turns, exact.  The nearest quarter turn is taken off as an integer,
// so the remainder, at most an eighth of a turn, keeps 24 bits of its own: its
// rounding is at most 2.3e-8 rad (an eighth of the whole fraction's), the
// constant's and the product's add 2.2e-8 and 3.0e-8.  The angle is right to
// 8e-8 rad of the table's whatever p is.
// Both functions there are their Taylor polynomials, cut where the next term
// is below 2e-9 and 2e-10 of an angle of pi/4.
__device__ __forceinline__ void rope_sincos_exact(int64_t p, uint64_t turns, float* s, float* c) {
  const uint64_t frac = static_cast<uint64_t>(p) * turns;
  const uint32_t top = static_cast<uint32_t>(frac >> 32);
  const uint32_t quarter = (top + (1u << 29)) >> 30;
  const int32_t rest = static_cast<int32_t>(top - (quarter << 30));  // in 2^-32 turns, at most an eighth of a turn
  const float x = static_cast<float>(rest) * 1.4629180792671596e-09f;  // 2 pi * 2^-32
  const float z = x * x;
  float sr = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  sr = fmaf(z, sr, 1.f / 120.f);
  sr = fmaf(z, sr, -1.f / 6.f);
  sr = fmaf(z * x, sr, x);
  float cr = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
  cr = fmaf(z, cr, -1.f / 720.f);
  cr = fmaf(z, cr, 1.f / 24.f);
  cr = fmaf(z, cr, -0.5f);
  cr = fmaf(z, cr, 1.f);
  const float a = (quarter & 1u) ? cr : sr, b = (quarter & 1u) ? sr : cr;
  *s = (quarter & 2u) ? -a : a;
  *c = ((quarter + 1u) & 2u) ? -b : b;
}

// The two 8-channel chunks of item i of a row: the rotated items first, then
// the channels that stay, in order.
__device__ __forceinline__ void item_chunks(const RopeArgs& r, int i, int* lo, int* hi) {
  const int n = r.rope_dim >> 4;
  if (i < n) {
    *lo = r.offset + (r.half ? 8 * i : 16 * i);
    *hi = r.half ? *lo + (r.rope_dim >> 1) : *lo + 8;
  } else {
    int ch = 16 * (i - n);
    if (ch >= r.offset) ch += r.rope_dim;
    *lo = ch;
    *hi = ch + 8;
  }
}

// A row's (sin, cos) in shared memory, [rope_dim / 2]: the four 16-byte pieces
// of an item's 8 pairs lie apart, each kind of all items together, so that
// neighbouring threads (items) read neighbouring pieces.
__device__ __forceinline__ int angle_slot(int pair, int items) {
  return ((((pair >> 1) & 3) * items + (pair >> 3)) << 1) | (pair & 1);
}
__device__ __forceinline__ void load_angles(const float2* row, int item, int items, float2 (&sc)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 f = *reinterpret_cast<const float4*>(row + ((j * items + item) << 1));
    sc[2 * j] = make_float2(f.x, f.y);
    sc[2 * j + 1] = make_float2(f.z, f.w);
  }
}

__device__ __forceinline__ void unpack_bf16(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(w[j] << 16);
    x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

// Rotates the item's 8 pairs by (sin, cos) sc[0..7]: with half-split pairs
// pair j is (lo[j], hi[j]), with interleaved ones pairs 0..3 are neighbours in
// lo and 4..7 in hi.
__device__ __forceinline__ void rotate_item(bool half, const float2 (&sc)[8], float (&lo)[8], float (&hi)[8]) {
  if (half) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = lo[j], y = hi[j];
      lo[j] = fmaf(x, sc[j].y, -y * sc[j].x);
      hi[j] = fmaf(x, sc[j].x, y * sc[j].y);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = lo[2 * j], y = lo[2 * j + 1], z = hi[2 * j], w = hi[2 * j + 1];
      lo[2 * j] = fmaf(x, sc[j].y, -y * sc[j].x);
      lo[2 * j + 1] = fmaf(x, sc[j].x, y * sc[j].y);
      hi[2 * j] = fmaf(z, sc[4 + j].y, -w * sc[4 + j].x);
      hi[2 * j + 1] = fmaf(z, sc[4 + j].x, w * sc[4 + j].y);
    }
  }
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// Two fp32 values as one register pair: Blackwell's packed multiply-add and
// add take half the issue slots of the scalar ones.
__device__ __forceinline__ uint64_t pair_of(uint32_t x, uint32_t y) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(x), "r"(y));
  return p;
}
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
  return pair_of(__float_as_uint(x), __float_as_uint(y));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ void split(uint64_t p, float* x, float* y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*x), "=f"(*y) : "l"(p));
}
// From a row's sum of weights l in units of 2^m to the factor of its weighted
// values, which are in units of 2^unit, and its lse, the sink's weight in.
__device__ __forceinline__ float finish_row(float m, float unit, float l, const float* sink, int head, float* lse) {
  if (sink) {
    const float s2 = __ldg(sink + head) * kLog2e, m1 = fmaxf(m, s2);
    l = l * ex2(m - m1) + ex2(s2 - m1);
    m = m1;
  }
  *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  return l == 0.f ? 0.f : ex2(unit - m) / l;
}

// Finds the sequence that work item w belongs to, where sequence b has
// count(b) >= 0 items: returns b and the item's index in it, or -1 when w is
// past the last.  Every thread of the CTA calls it (THREADS threads, a multiple
// of 32); sh holds THREADS / 32 + 2 values.  With `every` the sequences behind
// b are counted too (count() reports bad ones).
template <int THREADS, typename Count>
__device__ __forceinline__ int find_item(int B, int w, bool every, Count count, int* sh, int* index) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWarps = THREADS / 32;
  if (threadIdx.x == 0) sh[kWarps] = -1;
  int base = 0;
  for (int b0 = 0; b0 < B; b0 += THREADS) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    const int n = b < B ? count(b) : 0;
    int x = n;
    if (B - b0 > 1) {
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
    }
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    int before = base, all = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const int t = sh[k];
      if (k < warp) before += t;
      all += t;
    }
    before += x - n;
    if (w >= before && w < before + n) {  // one thread at most
      sh[kWarps] = b;
      sh[kWarps + 1] = w - before;
    }
    base += all;
    __syncthreads();
    if (sh[kWarps] >= 0 && !every) break;
  }
  *index = sh[kWarps + 1];
  return sh[kWarps];
}

}  // namespace csa
