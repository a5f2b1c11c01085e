// Attention over packed prompts of different lengths, grouped heads, causal
// (aligned at the sequences' ends), optionally windowed, with an optional
// attention sink.  For query row i of a sequence of nq queries and nk keys
//   keys j <= i + nk - nq (causal), j > i + nk - nq - W (window), j < nk
//   out_i = sum_j e^{l_ij} v_j / (sum_j e^{l_ij} + e^{sink}),  l = sm_scale q.k
// in one pass over the keys with a running maximum and sum.
//
// Bound by the tensor cores from a few hundred keys on (4 D operations a
// query, key and head against 4 D bytes a key and head read once a tile of
// 128 queries).  One CTA per QT tiles of 128 queries of one head: one warp
// loads Q and a ring of 128-key K and V tiles by TMA, one thread issues the
// tcgen05 products S = Q K^T and O += P V (S and O in tensor memory, P
// written over S as bf16 and read from there), four warps a tile do the
// softmax with one thread a row, so no value crosses threads.  Keys are
// walked from the diagonal down: the masked tiles come first.
//
// P is rounded to bf16 (the products take one type for both operands, and V
// is bf16); sums and maxima are fp32, over the unrounded weights.
//
// A masked weight is 0, and 0 * NaN is NaN: in tiles that some row of the CTA
// masks, two warps take values that are not finite out of V before the
// product (rows past the sequence's end become zero), and the rows that do see
// such a key get its values added at the end, as the formula has them.
#include <cuda_bf16.h>

#include "gqa.cuh"
#include "ptx.cuh"

namespace csa {
namespace {

constexpr int kTileShift = 7;
constexpr int kTile = 1 << kTileShift;   // queries and keys a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -1e30f;          // running maximum before the first key
// The accumulators are rescaled only when a row's maximum has grown by more
// than 2^8 since (weights up to 256 are exact in range for bf16 and fp32).
constexpr float kLag = 8.f;
// Tiles of keys that some row of a CTA masks: at most 3 that the causal edge
// of 256 rows crosses, 3 that the window's edge crosses, the sequence's last.
constexpr int kMaxMasked = 8;
constexpr int kCleanThreads = 64;

// QT tiles of queries a CTA, CTAS CTAs an SM.
template <int D, int QT, int CTAS>
struct Cfg {
  static constexpr int kThreads = QT * 128 + 128;
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kBlocks = D / 64;              // 128-byte wide blocks of a tile
  static constexpr int kBlockBytes = kTile * 128;
  static constexpr int kStages = CTAS == 2 && D == 128 ? 2 : 4;  // K and V tiles in flight, alternating; a power of two
  static constexpr int kSmem = QT * kTileBytes + kStages * kTileBytes + 1024;
  static constexpr int kSCol(int t) { return t * kTile; }
  static constexpr int kOCol(int t) { return QT * kTile + t * D; }
  static constexpr int kCols = QT == 2 ? 512 : 256;
  // Where 168 (or 128) registers a thread are launched, the softmax warps
  // take some that the other four give up: 256 x 208 + 128 x 88 = 384 x 168,
  // 128 x 208 + 128 x 48 = 256 x 128.
  static constexpr bool kSplit = QT == 2 || CTAS == 2;
  static constexpr int kLaunchRegs = QT == 2 ? 168 : 128;
  static constexpr int kSoftmaxRegs = 208, kOtherRegs = QT == 2 ? 88 : 48;
  static_assert(!kSplit || QT * 128 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "registers of the block");
  // One CTA of one tile an SM: the keys may be shared out over a cluster,
  // whose fp32 sums meet in the rings.
  static constexpr bool kCluster = QT == 1 && CTAS == 1;
  static_assert(!kCluster || kStages * kTileBytes >= kTile * D * 4, "the sums fit the ring");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 values as one register pair: Blackwell's packed multiply-add and
// add take half the issue slots of the scalar ones.
__device__ __forceinline__ uint64_t pair_of(uint32_t x, uint32_t y) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(x), "r"(y));
  return p;
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
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

__device__ __forceinline__ bool not_finite(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }

// Non-zero where a half of the word is a bf16 infinity or NaN (magnitude bits
// of 0x7F80 and more carry into the half's top bit).
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) { return ((w & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u; }
// The word with such halves zeroed.
__device__ __forceinline__ uint32_t finite_halves(uint32_t w) {
  if (not_finite(w)) w &= 0xFFFF0000u;
  if (not_finite(w >> 16)) w &= 0xFFFFu;
  return w;
}

// The tiles of keys [lo, hi) that `rows` queries from row `first` on see.
struct Range {
  int lo, hi;
};

// From a row's reference (in log2) and sum of weights to the factor of its
// weighted values and its lse, the sink's weight in.
__device__ __forceinline__ float finish_row(float m, float l, const float* sink, int head, float* lse) {
  float f = 1.f;
  if (sink) {
    const float s2 = __ldg(sink + head) * kLog2e, m1 = fmaxf(m, s2);
    f = ex2(m - m1);
    l = l * f + ex2(s2 - m1);
    m = m1;
  }
  *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  return l == 0.f ? 0.f : f / l;
}

struct Seq {
  int64_t q0, k0;  // first rows of the sequence
  int nq, nk;
};

template <int D, int QT, int CTAS>
__global__ void __launch_bounds__(Cfg<D, QT, CTAS>::kThreads, CTAS)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PromptAttnArgs a, const int cluster) {
  using C = Cfg<D, QT, CTAS>;
  constexpr int kTmaWarp = 4 * QT, kMmaWarp = 4 * QT + 1, kCleanWarp = 4 * QT + 2;
  constexpr int kRowsCta = QT * kTile;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int sh[C::kThreads / 32 + 2];
  __shared__ uint64_t q_full, full[C::kStages], empty[C::kStages];
  __shared__ uint64_t s_full[QT], p_full[QT], o_full[QT], dirty, cleaned, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s;
  __shared__ uint32_t odd_rows[kMaxMasked][4];  // keys of each masked tile whose values are not all finite
  __shared__ int odd_tile[kMaxMasked], n_odd;
  __shared__ float m_s[C::kCluster ? kTile : 1], l_s[C::kCluster ? kTile : 1];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* q_s = smem;
  uint8_t* ring = smem + QT * C::kTileBytes;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  volatile int* abort_flag = &abort_s;
  if (tid == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&drain, 1);
    mbar_init(&dirty, 1);
    mbar_init(&cleaned, kCleanThreads);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int t = 0; t < QT; ++t) {
      mbar_init(s_full + t, 1);
      mbar_init(p_full + t, kTile);
      mbar_init(o_full + t, 1);
    }
    fence_mbar_init();
    abort_s = 0;
    n_odd = 0;
  }
  if (tid < kMaxMasked * 4) odd_rows[tid >> 2][tid & 3] = 0u;
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  // Tensor memory is taken after the kernel before has ended and before the
  // one after may start: no CTA of either can then hold what this one, or
  // what it waits for, still needs.
  pdl_wait();
  if (warp == kMmaWarp) tmem_alloc(&tmem_slot, C::kCols);
  tc_fence_before();

  // this CTA's sequence and tiles: the later tiles of a sequence (more keys
  // under the causal mask) first
  // (a cluster's CTAs: the same tile, each a part of its keys)
  const int unit = C::kCluster ? static_cast<int>(blockIdx.x) / cluster : static_cast<int>(blockIdx.x);
  const int rank = C::kCluster ? static_cast<int>(blockIdx.x) - unit * cluster : 0;
  const int head = unit % a.n_heads;
  const int kv_head = head / (a.n_heads / a.n_kv_heads);
  auto seq_at = [&](int b) {
    Seq s;
    const int32_t q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + b + 1);
    const int32_t k0 = __ldg(a.cu_k + b), k1 = __ldg(a.cu_k + b + 1);
    const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.n_q && k0 >= 0 && k1 >= k0 && k1 <= a.n_k;
    if (!ok) record_error(a.status, kErrIndexRange);
    s.q0 = q0;
    s.k0 = k0;
    s.nq = ok ? q1 - q0 : 0;
    s.nk = ok ? k1 - k0 : 0;
    return s;
  };
  int index;
  const int b = find_item<C::kThreads>(
      a.B, unit / a.n_heads, [&](int s) { return (seq_at(s).nq + kRowsCta - 1) / kRowsCta; },
      sh, &index);
  // (the search's barriers also order the allocation and the mbarriers' set-up)
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = tmem_slot;
  if (b < 0) {
    if (warp == kMmaWarp) tmem_dealloc(tmem, C::kCols);
    return;
  }
  const Seq sq = seq_at(b);
  const int row0 = ((sq.nq + kRowsCta - 1) / kRowsCta - 1 - index) * kRowsCta;
  const int shift = sq.nk - sq.nq;  // row i sits at position i + shift among the keys

  // tiles of keys that rows [first, first + rows) see
  auto range_of = [&](int first, int rows) {
    const int pos = first + shift;  // (lengths are below 2^30 each: no overflow)
    const int hi = a.causal ? min(sq.nk, pos + rows) : sq.nk;
    const int lo = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
    Range r;
    const bool none = rows <= 0 || hi <= lo;
    r.lo = none ? 0 : lo >> kTileShift;
    r.hi = none ? 0 : (hi + kTile - 1) >> kTileShift;
    return r;
  };
  // some of those rows masks a part of tile j: j >= from or j <= upto
  struct Masked {
    int from, upto;
    __device__ __forceinline__ bool at(int j) const { return j >= from || j <= upto; }
  };
  auto masked_of = [&](int first, int rows) {
    Masked m;
    m.from = sq.nk >> kTileShift;  // the sequence ends inside the tile (or before it)
    const int pos = first + shift;  // the first row's last key
    if (a.causal) m.from = min(m.from, pos < 0 ? 0 : (pos + 1) >> kTileShift);
    const int out = pos + rows - 1;  // the last row's last key: keys up to out - window are outside its window
    m.upto = a.window > 0 && out >= a.window ? (out - a.window) >> kTileShift : -1;
    return m;
  };
  auto rows_of = [&](int t) { return max(0, min(kTile, sq.nq - row0 - t * kTile)); };
  const int rows_cta = min(kRowsCta, sq.nq - row0);
  Range rt[QT];
  int j_lo = 0x7fffffff, j_hi = 0;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    rt[t] = range_of(row0 + t * kTile, rows_of(t));
    if (C::kCluster && cluster > 1) {
      const int per = (rt[t].hi - rt[t].lo + cluster - 1) / cluster, hi = rt[t].hi - rank * per;
      rt[t].lo = max(rt[t].lo, hi - per);
      rt[t].hi = hi;
      if (hi <= rt[t].lo) rt[t].lo = rt[t].hi = 0;
    }
    if (rt[t].lo < rt[t].hi) {
      j_lo = min(j_lo, rt[t].lo);
      j_hi = max(j_hi, rt[t].hi);
    }
  }
  const Masked masked = masked_of(row0, rows_cta);
  const int n_it = j_hi > 0 ? j_hi - j_lo : 0;  // iteration it works on tile j_hi - 1 - it

  if (warp >= 4 * QT) {
    if constexpr (C::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    if (warp == kTmaWarp) {
      // ---------------- loads ----------------
      if (lane == 0 && n_it > 0) {
        mbar_arrive_expect_tx(&q_full, QT * C::kTileBytes);
        for (int t = 0; t < QT; ++t)
          for (int k = 0; k < C::kBlocks; ++k)
            tma_load_3d(q_s + t * C::kTileBytes + k * C::kBlockBytes, &tm_q, k * 64, head,
                        static_cast<int32_t>(sq.q0 + row0 + t * kTile), &q_full);
        int issued = 0;
        for (int s = 0; s < 2 * n_it; ++s) {
          const int slot = s % C::kStages;
          if (s >= C::kStages && !wait_or_abort(empty + slot, ((s / C::kStages) - 1) & 1, abort_flag, a.status)) break;
          mbar_arrive_expect_tx(full + slot, C::kTileBytes);
          const int row = static_cast<int>(sq.k0) + (j_hi - 1 - (s >> 1)) * kTile;
          for (int k = 0; k < C::kBlocks; ++k)
            tma_load_3d(ring + slot * C::kTileBytes + k * C::kBlockBytes, (s & 1) ? &tm_v : &tm_k, k * 64, kv_head, row,
                        full + slot);
          ++issued;
        }
        // every copy lands before the CTA ends (also after an abort)
        mbar_wait(&q_full, 0, a.status);
        for (int s = issued > C::kStages ? issued - C::kStages : 0; s < issued; ++s)
          mbar_wait(full + s % C::kStages, (s / C::kStages) & 1, a.status);
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ---------------- products ----------------
      // The whole warp walks the loop and one elected lane issues: with the
      // loop's values warp-uniform (the shuffles say so to the compiler) an
      // issue costs a few cycles; from a branch on lane 0 each product took
      // about 115, more than it takes to compute.
      constexpr uint32_t idesc_s = instr_desc(kTile, kTile, 1, 1, 0, 0);  // bf16, K-major A and B
      constexpr uint32_t idesc_o = instr_desc(kTile, D, 1, 1, 0, 1);      // A from TMEM, B (= V) MN-major
      auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
      const int u_it = uniform(n_it), u_hi = uniform(j_hi);
      int u_lo[QT], u_end[QT];          // iterations of tile t: [u_lo, u_end)
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        u_lo[t] = uniform(rt[t].lo < rt[t].hi ? j_hi - rt[t].hi : 0);
        u_end[t] = uniform(rt[t].lo < rt[t].hi ? j_hi - rt[t].lo : 0);
      }
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const int m_from = uniform(j_hi - masked.from), m_upto = uniform(j_hi - 1 - masked.upto);
      auto masked_it = [&](int it) { return it < m_from || it >= m_upto; };
      const uint32_t qb = smem_u32(q_s), rb = smem_u32(ring);
      const bool skip_s = test_fault(a.status, kFaultAttn);  // test fault: S is never announced
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, a.status)) != 0;
      };
      auto s_of = [&](int t, uint64_t k_desc) {  // S_t = Q_t K^T (one lane)
        const uint64_t q_desc = smem_desc(qb + t * C::kTileBytes, 16, 1024, kSwizzle128B);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          constexpr int kStep = 32 >> 4;  // 16 channels along a 128-byte line, in the descriptors' units
          const int off = (s >> 2) * (C::kBlockBytes >> 4) + (s & 3) * kStep;
          mma_f16(tm + C::kSCol(t), q_desc + off, k_desc + off, idesc_s, s > 0 ? 1u : 0u);
        }
        if (!skip_s) tc_commit(s_full + t);
      };
      bool ok = u_it == 0 || (wait(&q_full, 0) && wait(full, 0));
      if (ok && u_it > 0) {  // the first tile of keys
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int t = 0; t < QT; ++t)
            if (u_lo[t] == 0 && u_end[t] > 0) s_of(t, smem_desc(rb, 16, 1024, kSwizzle128B));
          tc_commit(empty);
        }
        __syncwarp();
      }
      uint32_t n_cleaned = 0;
      for (int it = 0; it < u_it && ok; ++it) {
        const int v_seq = 2 * it + 1, k_seq = 2 * it + 2;
        const int v_slot = v_seq & (C::kStages - 1), k_slot = k_seq & (C::kStages - 1);
        const uint64_t v_desc = smem_desc(rb + v_slot * C::kTileBytes, C::kBlockBytes, 1024, kSwizzle128B);
        const uint64_t k_desc = smem_desc(rb + k_slot * C::kTileBytes, 16, 1024, kSwizzle128B);
        const bool more = it + 1 < u_it;
        // this tile's values and the next tile's keys are usually there long
        // before the weights are
        ok = wait(full + v_slot, (v_seq / C::kStages) & 1);
        if (ok && masked_it(it)) {  // one masked tile at a time is with the cleaning warps
          if (elect_one()) mbar_arrive(&dirty);
          __syncwarp();
          ok = wait(&cleaned, n_cleaned++ & 1u);
        }
        if (ok && more) ok = wait(full + k_slot, (k_seq / C::kStages) & 1);
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          const bool pv = it >= u_lo[t] && it < u_end[t], next = more && it + 1 >= u_lo[t] && it + 1 < u_end[t];
          if (ok && pv) ok = wait(p_full + t, (it - u_lo[t]) & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            if (pv) {
#pragma unroll
              for (int s = 0; s < kTile / 16; ++s)
                mma_f16_ts(tm + C::kOCol(t), tm + C::kSCol(t) + s * 8, v_desc + (s * 2048 >> 4), idesc_o,
                           (it > u_lo[t] || s > 0) ? 1u : 0u);
              if (it + 1 == u_end[t]) tc_commit(o_full + t);
            }
            if (t == QT - 1) tc_commit(empty + v_slot);
            if (next) s_of(t, k_desc);
            if (t == QT - 1 && more) tc_commit(empty + k_slot);
          }
          __syncwarp();
        }
      }
      // whatever was issued finishes before TMEM and shared memory are released
      if (elect_one()) {
        tc_commit(&drain);
        mbar_wait(&drain, 0, a.status);
      }
      __syncwarp();
    } else {
      // ---------------- values that are not finite, taken out of masked tiles ----------------
      const int ct = tid - kCleanWarp * 32;
      int n_masked = 0;
      for (int it = 0; it < n_it; ++it) {
        const int j = j_hi - 1 - it;
        if (!masked.at(j)) continue;
        const int seq = 2 * it + 1, slot = seq % C::kStages;
        // the MMA thread has seen the tile's copy complete and holds its slot
        // until `cleaned`, so the second wait returns at once (and makes the
        // copied bytes visible here)
        if (!wait_or_abort(&dirty, n_masked & 1, abort_flag, a.status) ||
            !wait_or_abort(full + slot, (seq / C::kStages) & 1, abort_flag, a.status))
          break;
        uint4* tile = reinterpret_cast<uint4*>(ring + slot * C::kTileBytes);
        // rows past the sequence become zero; of the others, eight 16-byte
        // chunks at a time are looked at for an exponent of all ones (the
        // swizzle moves chunks within their row only: chunk i is of row i/8 % 128)
        const int past = min(sq.nk - j * kTile, kTile);
        if (past < kTile)
          for (int i = ct; i < (kTile - past) * 8 * C::kBlocks; i += kCleanThreads) {
            const int block = i / ((kTile - past) * 8);
            tile[block * kTile * 8 + past * 8 + i - block * (kTile - past) * 8] = make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll 1
        for (int i0 = ct; i0 < C::kTileBytes / 16; i0 += 8 * kCleanThreads) {
          uint4 u[8];
          uint32_t any = 0u;
#pragma unroll
          for (int k = 0; k < 8; ++k) u[k] = tile[i0 + k * kCleanThreads];
#pragma unroll
          for (int k = 0; k < 8; ++k) any |= odd_halves(u[k].x) | odd_halves(u[k].y) | odd_halves(u[k].z) | odd_halves(u[k].w);
          if (any == 0u) continue;
#pragma unroll 1
          for (int k = 0; k < 8; ++k) {
            const int i = i0 + k * kCleanThreads, r = (i >> 3) & (kTile - 1);
            uint4 w = tile[i];
            if (r >= past || !(odd_halves(w.x) | odd_halves(w.y) | odd_halves(w.z) | odd_halves(w.w))) continue;
            w.x = finite_halves(w.x);
            w.y = finite_halves(w.y);
            w.z = finite_halves(w.z);
            w.w = finite_halves(w.w);
            tile[i] = w;
            if (n_masked < kMaxMasked) {
              atomicOr(&odd_rows[n_masked][r >> 5], 1u << (r & 31));
              odd_tile[n_masked] = j;
              n_odd = 1;
            }
          }
        }
        ++n_masked;
        fence_proxy_async_smem();
        mbar_arrive(&cleaned);
      }
    }
  } else {
    // ---------------- softmax: one thread a query row ----------------
    if constexpr (C::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int first = row0 + t * kTile, rows = rows_of(t);
    const int i = first + r;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_tmem = tmem + lane_base + C::kSCol(t), o_tmem = tmem + lane_base + C::kOCol(t);
    const float scale2 = a.sm_scale * kLog2e;
    // the row's keys [first_key, last_key]
    const int at_key = i + shift;
    const int last_key = a.causal ? min(at_key, sq.nk - 1) : sq.nk - 1;
    const int first_key = a.window > 0 && at_key >= a.window ? at_key - a.window + 1 : 0;
    float m = kNone, l = 0.f;  // the reference of the weights e^(scale (s - m)), in the products' units
    bool large = false;      // of the warp: some row's logits are large (see below)
    bool ok = true;
    const Masked masked_t = masked_of(first, rows);
    const int n_tiles = rt[t].hi - rt[t].lo;
    for (int n = 0; n < n_tiles; ++n) {
      const int j = rt[t].hi - 1 - n;
      ok = wait_or_abort(s_full + t, n & 1, abort_flag, a.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(s_tmem + 32 * c, s[c]);
      tmem_wait_ld();
      if (masked_t.at(j)) {  // this row's keys among the tile's columns, as a bit each
        const int c_hi = last_key + 1 - j * kTile, c_lo = first_key - j * kTile;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int hi = max(0, min(32, c_hi - 32 * c)), lo = max(0, min(32, c_lo - 32 * c));
          const uint32_t seen = static_cast<uint32_t>((1ull << hi) - (1ull << min(lo, hi)));
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!((seen >> k) & 1u)) s[c][k] = 0xFF800000u;  // -inf
        }
      }
      float top[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        top[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
        for (int k = 2; k < 32; k += 2) top[c] = max3(top[c], __uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1]));
      }
      const float top1 = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
      if (__any_sync(0xffffffffu, (top1 - m) * scale2 > kLag)) {
        const float m1 = fmaxf(m, top1), f = ex2((m - m1) * scale2);
        m = m1;
        l *= f;
        large = __any_sync(0xffffffffu, m > kNone && fabsf(m * scale2) > 65536.f);
        if (n > 0) {  // the products of the tiles before have finished: S was issued after them
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(o_tmem + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st32(o_tmem + 32 * c, o);
          }
        }
      }
      const uint64_t scale_2 = pair_of(__float_as_uint(scale2), __float_as_uint(scale2));
      // scale s - scale m in one rounding; where the logits are so large that
      // the rounding of scale m shows, s - m first
      float offset = -m * scale2;
      if (large) {
        offset = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int k = 0; k < 32; ++k) s[c][k] = __float_as_uint(__uint_as_float(s[c][k]) - m);
      }
      const uint64_t minus_m = pair_of(__float_as_uint(offset), __float_as_uint(offset));
      uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t p[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float x, y;
          split(fma2(pair_of(s[c][2 * k], s[c][2 * k + 1]), scale_2, minus_m), &x, &y);
          x = ex2(x);
          y = ex2(y);
          sum[k & 1] = add2(sum[k & 1], pair_of(__float_as_uint(x), __float_as_uint(y)));
          const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
          p[k] = *reinterpret_cast<const uint32_t*>(&v);
        }
        tmem_st16(s_tmem + 16 * c, p);
      }
      float sx, sy;
      split(add2(sum[0], sum[1]), &sx, &sy);
      l += sx + sy;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(p_full + t);
    }
    if (ok && n_it > 0) {  // (a tile that sees no keys: its queries have landed where its output is staged)
      ok = wait_or_abort(n_tiles > 0 ? o_full + t : &q_full, 0, abort_flag, a.status);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    }
    if (ok && rows > 0) {
      // the masked tiles were cleaned before their products, so n_odd is final
      const int64_t row = (sq.q0 + i) * a.n_heads + head;
      const bool shared = C::kCluster && cluster > 1;
      if (shared) {  // the sums as they are
        m_s[r] = m * scale2;
        l_s[r] = l;
        l = 1.f;
      } else {
        float lse;
        l = finish_row(m * scale2, l, a.sink, head, &lse);
        if (a.lse && r < rows) a.lse[row] = lse;
      }
      const bool odd = *const_cast<volatile int*>(&n_odd) != 0;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (n_tiles > 0) {
          tmem_ld32(o_tmem + 32 * c, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
        // (a row without keys has l = 0 and sums of 0 * value, all finite)
        float x[32];
        const uint64_t l2 = pair_of(__float_as_uint(l), __float_as_uint(l));
#pragma unroll
        for (int k = 0; k < 32; k += 2) split(mul2(pair_of(o[k], o[k + 1]), l2), &x[k], &x[k + 1]);
        if (odd && r < rows) {
          for (int e = 0; e < kMaxMasked * kTile; ++e) {
            const uint32_t word = odd_rows[e >> 7][(e >> 5) & 3];
            if (!((word >> (e & 31)) & 1u)) continue;
            const int64_t key = static_cast<int64_t>(odd_tile[e >> 7]) * kTile + (e & (kTile - 1));
            if (key > last_key || key < first_key) continue;
            const uint16_t* v = a.v + (sq.k0 + key) * a.v_stride + kv_head * a.v_stride_h + 32 * c;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const uint32_t h = v[k];
              if (not_finite(h)) x[k] += __uint_as_float(h << 16);
            }
          }
        }
        if (shared) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<float4*>(ring + r * D * 4 + (((8 * c + k) ^ (r & (D / 4 - 1))) << 4)) =
                make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
          continue;
        }
        uint8_t* line = q_s + t * C::kTileBytes + (c >> 1) * C::kBlockBytes + r * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[8 * k + 2 * e], x[8 * k + 2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&v);
          }
          *reinterpret_cast<uint4*>(line + ((((c & 1) * 4 + k) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      // the warp's 32 rows, staged where its queries were (every product with
      // them has finished), stored with neighbouring lanes on one row
      __syncwarp();
      constexpr int kChunks = D / 8, kRowsAtOnce = 32 / kChunks;
      const int w0 = (warp & 3) * 32;
#pragma unroll 4
      for (int k = 0; k < (shared ? 0 : 32 / kRowsAtOnce); ++k) {
        const int rr = w0 + k * kRowsAtOnce + lane / kChunks, ch = lane % kChunks;
        const uint4 v = *reinterpret_cast<const uint4*>(q_s + t * C::kTileBytes + (ch >> 3) * C::kBlockBytes + rr * 128 +
                                                        (((ch & 7) ^ (rr & 7)) << 4));
        if (rr < rows)
          *reinterpret_cast<uint4*>(a.out + ((sq.q0 + first + rr) * a.n_heads + head) * D + ch * 8) = v;
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
  if constexpr (C::kCluster) {
    if (cluster > 1) {
      // every CTA adds up its share of the rows over the cluster, a row (of
      // 64 channels two) a warp at a time, 4 channels a lane
      cluster_sync();
      constexpr int kLanes = D / 4, kRowsAtOnce = 32 / kLanes;
      const int share = kTile / cluster, rows = min(kTile, sq.nq - row0);
#pragma unroll 2
      for (int k = warp * kRowsAtOnce + lane / kLanes; k < share; k += C::kThreads / 32 * kRowsAtOnce) {
        const int r = rank * share + k, ch = lane % kLanes;
        if (r >= rows) continue;
        float m = kNone, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < cluster; ++p) {  // (few: the maximum is taken along)
          const float mp = dsmem_ld_f32(dsmem_addr(m_s + r, p)), lp = dsmem_ld_f32(dsmem_addr(l_s + r, p));
          const float4 v = dsmem_ld_f32x4(dsmem_addr(ring + r * D * 4 + ((ch ^ (r & (D / 4 - 1))) << 4), p));
          const float m1 = fmaxf(m, mp), f = ex2(m - m1), fp = ex2(mp - m1);
          m = m1;
          l = l * f + lp * fp;
          o.x = o.x * f + v.x * fp;
          o.y = o.y * f + v.y * fp;
          o.z = o.z * f + v.z * fp;
          o.w = o.w * f + v.w * fp;
        }
        const int64_t row = (sq.q0 + row0 + r) * a.n_heads + head;
        float lse;
        const float f = finish_row(m, l, a.sink, head, &lse);
        if (a.lse && ch == 0) a.lse[row] = lse;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * f, o.y * f), hi = __floats2bfloat162_rn(o.z * f, o.w * f);
        *reinterpret_cast<uint2*>(a.out + row * D + 4 * ch) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
      cluster_sync();  // a CTA's shared memory outlives its readers
    }
  }
}

// Rows of `heads` heads as a 3-D tensor, read in boxes of 64 channels of 128
// rows of one head (128-byte swizzle); rows past the end read as zero.
bool encode_rows(CUtensorMap* m, PFN_cuTensorMapEncodeTiled_v12000 encode, const uint16_t* base, int dim, int heads,
                 int64_t rows, int64_t stride, int64_t stride_h) {
  cuuint64_t size[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride_h) * 2, static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[3] = {64, 1, kTile};
  cuuint32_t ones[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(base), size, strides, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int QT, int CTAS>
cudaError_t launch_dim(const PromptAttnArgs& a, PFN_cuTensorMapEncodeTiled_v12000 encode, int cluster,
                       cudaStream_t stream) {
  using C = Cfg<D, QT, CTAS>;
  const auto kernel = prompt_attn_kernel<D, QT, CTAS>;
  CUtensorMap tm_q, tm_k, tm_v;
  const int64_t n_k = a.n_k > 0 ? a.n_k : 1;  // (no keys: the maps are not read)
  if (!encode || !encode_rows(&tm_q, encode, a.q, D, a.n_heads, a.n_q, a.q_stride, a.q_stride_h) ||
      !encode_rows(&tm_k, encode, a.n_k > 0 ? a.k : a.q, D, a.n_kv_heads, n_k, a.k_stride, a.k_stride_h) ||
      !encode_rows(&tm_v, encode, a.n_k > 0 ? a.v : a.q, D, a.n_kv_heads, n_k, a.v_stride, a.v_stride_h))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  if (C::kSplit) {  // the split of registers assumes what the kernel is launched with
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, kernel);
    if (e != cudaSuccess) return e;
    if (at.numRegs < C::kLaunchRegs) return cudaErrorInvalidConfiguration;
  }
  // n rows are at most n / R + 1 tiles of R rows, and at most n
  const int64_t most = a.n_q / (QT * kTile) + a.B;
  const int64_t grid = (most < a.n_q ? most : a.n_q) * a.n_heads * cluster;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(grid)), dim3(C::kThreads), C::kSmem, stream,
                            static_cast<unsigned>(cluster), tm_q, tm_k, tm_v, a, cluster);
}

template <int D>
cudaError_t launch_tiles(const PromptAttnArgs& a, PFN_cuTensorMapEncodeTiled_v12000 encode, cudaStream_t stream) {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t most = a.n_q / kTile + a.B, tiles = (most < a.n_q ? most : a.n_q) * a.n_heads;
  if (tiles <= sms) {
    // Few tiles, an SM each; a cluster shares out the keys of a tile while
    // SMs are left and a CTA has two tiles of keys at least.
    int cluster = 1;
    while (cluster < 8 && tiles * cluster * 2 <= sms && a.n_k >= static_cast<int64_t>(a.B) * 4 * cluster * kTile)
      cluster *= 2;
    return launch_dim<D, 1, 1>(a, encode, cluster, stream);
  }
  // Two tiles a CTA share the keys' copies and overlap one's softmax with the
  // other's products; where sequences are short two CTAs of one tile on an SM
  // overlap their starts and ends instead.  Width 128, 32 heads: 16384 queries
  // 1.42 ms with two tiles, 1.54 ms with one; 32 prompts of 500 189 and 194
  // us; 64 of 128 126 and 79 us.  At width 64 one tile was never slower (16
  // packed prompts, window 1024: 350 us with two, 305 us with one).
  if (D == 64 || a.n_q <= static_cast<int64_t>(256) * a.B) return launch_dim<D, 1, 2>(a, encode, 1, stream);
  return launch_dim<D, D == 64 ? 1 : 2, D == 64 ? 2 : 1>(a, encode, 1, stream);
}

}  // namespace

cudaError_t launch_prompt_attn(const PromptAttnArgs& a, PFN_cuTensorMapEncodeTiled_v12000 encode, cudaStream_t stream) {
  if (a.B <= 0 || a.n_q <= 0) return cudaSuccess;
  return a.head_dim == 128 ? launch_tiles<128>(a, encode, stream) : launch_tiles<64>(a, encode, stream);
}

}  // namespace csa
