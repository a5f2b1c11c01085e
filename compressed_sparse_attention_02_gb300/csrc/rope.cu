// Rotary positions of query and key rows ("CSA2 详解" §12.1 "Partial RoPE" is
// the same rotation on a latent's last channels): pair j of a row at position
// p turns by the angle p * f_j, (x, y) -> m (x cos - y sin, x sin + y cos);
// the inverse turns back (and is the rotation's gradient, its transpose).
//
// Bound by memory: every channel is read and written once.  A CTA computes
// the sines and cosines of its tokens once into shared memory (all heads of a
// token share them), then each thread rotates items of 16 channels, two
// 16-byte loads and stores an item, three items in flight and the first ones
// under way before the sines are computed.
#include <cuda_bf16.h>

#include "gqa.cuh"
#include "ptx.cuh"

namespace csa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTokens = 16;   // tokens a CTA
constexpr int kMaxRopeDim = 512;

struct RopeGrid {
  int tokens;       // tokens a CTA
  int heads;        // heads a CTA
  int items;        // items a row: head_dim / 16, or rope_dim / 16 in place
  uint32_t inv_items, inv_heads;  // ceil(2^32 / items), ceil(2^32 / heads)
};

__device__ __forceinline__ uint32_t div_by(uint32_t x, uint32_t inv, int n) {
  return n == 1 ? x : __umulhi(x, inv);
}

__device__ __forceinline__ uint4 pack_bf16(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16384 tokens of 72 heads of width 128 take 90.4 us (6.7 TB/s, 99% of the copy
// rate) with 3 items a thread in flight and 4 CTAs an SM; 2 items 92.1, 4 items
// with 3 CTAs 93.2.
constexpr int kFlight = 3;
constexpr int kRopeCtas = 4;

__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const RopeRowsArgs a, const RopeGrid g) {
  extern __shared__ __align__(16) float2 sc_s[];  // the tokens' (sin, cos), rope_dim / 2 each
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * g.tokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(g.tokens), a.n_rows - t0));
  const int h0 = static_cast<int>(blockIdx.y) * g.heads;
  const int nh = min(g.heads, a.n_heads - h0);
  const int pairs = a.rope.rope_dim >> 1;
  const int n = nt * g.heads * g.items;  // (a last group of fewer heads leaves its items out)
  const int rotated = a.rope.rope_dim >> 4;
  const uint16_t* in = a.in + t0 * a.in_stride + h0 * a.in_stride_h;
  uint16_t* out = a.out + t0 * a.out_stride + h0 * a.out_stride_h;
  for (int i0 = tid; i0 - tid < n; i0 += kFlight * kRopeThreads) {
    uint4 u[kFlight], v[kFlight];
    int64_t dst[kFlight];
    int at[kFlight];  // token (above bit 5) and rotated item, and above both its second chunk's distance; -1: nothing
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int i = i0 + k * kRopeThreads;
      at[k] = -1;
      if (i >= n) continue;
      const int row = static_cast<int>(div_by(i, g.inv_items, g.items));
      const int it = i - row * g.items;
      const int t = static_cast<int>(div_by(row, g.inv_heads, g.heads));
      const int h = row - t * g.heads;
      if (h >= nh || __ldg(a.pos + t0 + t) < 0) continue;
      int cl, ch;
      item_chunks(a.rope, it, &cl, &ch);
      const uint16_t* src = in + t * a.in_stride + h * a.in_stride_h + cl;
      u[k] = *reinterpret_cast<const uint4*>(src);
      v[k] = *reinterpret_cast<const uint4*>(src + (ch - cl));
      dst[k] = t * a.out_stride + h * a.out_stride_h + cl;
      at[k] = (ch - cl) << 16 | (it < rotated ? t << 5 | it : 0xFFFF);
    }
    if (i0 == tid) {  // the tokens' sines and cosines, while the first loads are on their way
      for (int i = tid; i < nt * pairs; i += kRopeThreads) {
        const int t = i / pairs, j = i - t * pairs;
        float s, c;
        rope_sincos_exact(__ldg(a.pos + t0 + t), __ldg(a.rope.turns + j), &s, &c);
        sc_s[t * pairs + angle_slot(j, rotated)] = make_float2((a.inverse ? -s : s) * a.rope.mscale, c * a.rope.mscale);
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      if (at[k] < 0) continue;
      const int sc_at = at[k] & 0xFFFF;
      if (sc_at != 0xFFFF) {
        float x[8], y[8];
        float2 sc[8];
        unpack_bf16(u[k], x);
        unpack_bf16(v[k], y);
        load_angles(sc_s + (sc_at >> 5) * pairs, sc_at & 31, rotated, sc);
        rotate_item(a.rope.half != 0, sc, x, y);
        u[k] = pack_bf16(x);
        v[k] = pack_bf16(y);
      }
      *reinterpret_cast<uint4*>(out + dst[k]) = u[k];
      *reinterpret_cast<uint4*>(out + dst[k] + (at[k] >> 16)) = v[k];
    }
  }
}

uint32_t inverse_of(int n) { return static_cast<uint32_t>(((1ull << 32) + n - 1) / n); }

}  // namespace

cudaError_t launch_rope(const RopeRowsArgs& a, cudaStream_t stream) {
  if (a.n_rows <= 0 || a.n_heads <= 0) return cudaSuccess;
  RopeGrid g;
  const bool in_place = a.in == a.out;
  g.items = (in_place ? a.rope.rope_dim : a.head_dim) >> 4;
  // A CTA of 256 threads takes about 2400 items (1200: 92.7 us, 4700: 94.8):
  // several tokens of few heads, or one token whose heads are split while the
  // grid would not fill the GPU.
  const int64_t row_items = static_cast<int64_t>(a.n_heads) * g.items;
  int64_t tokens = 2400 / row_items;
  tokens = tokens < 1 ? 1 : tokens > kRopeMaxTokens ? kRopeMaxTokens : tokens;
  while (tokens > 1 && (a.n_rows + tokens - 1) / tokens < 600) tokens >>= 1;
  g.tokens = static_cast<int>(tokens);
  g.heads = a.n_heads;
  // one token a CTA: at most 8192 items (also the range of the reciprocals)
  while (g.tokens == 1 && g.heads > 1 &&
         (static_cast<int64_t>(g.heads) * g.items > 8192 ||
          (g.heads * g.items > kRopeThreads && a.n_rows * ((a.n_heads + g.heads - 1) / g.heads) < 600)))
    g.heads = (g.heads + 1) / 2;
  g.inv_items = inverse_of(g.items);
  g.inv_heads = inverse_of(g.heads);
  const int64_t gx = (a.n_rows + g.tokens - 1) / g.tokens;
  if (gx > 0x7fffffff) return cudaErrorInvalidValue;
  const size_t smem = static_cast<size_t>(g.tokens) * (a.rope.rope_dim / 2) * sizeof(float2);
  static_assert(kRopeMaxTokens * (kMaxRopeDim / 2) * sizeof(float2) <= 48 * 1024, "the default shared-memory limit");
  return launch_pdl(rope_kernel, dim3(static_cast<unsigned>(gx), (a.n_heads + g.heads - 1) / g.heads),
                    dim3(kRopeThreads), smem, stream, a, g);
}

}  // namespace csa
