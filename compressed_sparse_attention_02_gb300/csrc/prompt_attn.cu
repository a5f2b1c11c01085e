// Attention over packed prompts of different lengths, grouped heads, causal
// (aligned at the sequences' ends), optionally windowed, with an optional
// attention sink.  For query row i of a sequence of nq queries and nk keys
//   keys j <= i + nk - nq (causal), j > i + nk - nq - W (window), j < nk
//   out_i = sum_j e^{l_ij} v_j / (sum_j e^{l_ij} + e^{sink}),  l = sm_scale q.k
// in one pass over the keys with a running maximum and sum.
//
// Bound by the tensor cores from a few hundred keys on (4 D operations a
// query, key and head against 4 D bytes a key and head read once a tile of
// 128 queries); short of that, and at width 64, by the chain from a tile's
// scores over their softmax to the next products.  Resident CTAs walk through
// the items, each QT tiles of 128 queries of one head: one warp finds an item
// and loads Q and a ring of 128-key K and V tiles by TMA, the next item's
// under this one's end, one warp issues the tcgen05 products S = Q K^T and
// O += P V (S and O in tensor memory, P written over S as bf16 and read from
// there), four warps a tile do the softmax with one thread a row, so no value
// crosses threads.  Keys are walked from the diagonal down: the masked tiles
// come first.  With one tile a CTA its keys are worked on in halves, one's
// scores under the other's softmax.  16384 queries of 32 heads of width 128:
// 1.42 ms (1550 TFLOP/s, 82% of the matrix product's rate) in a few passes, 1.48
// ms in calls that follow each other for seconds; 16 prompts of 237 to 2500 under
// a window of 1024 at width 64: 206 us, 550 TFLOP/s.
//
// P is rounded to bf16 (the products take one type for both operands, and V
// is bf16); sums and maxima are fp32, over the unrounded weights.
//
// A masked weight is 0, and 0 * NaN is NaN: in tiles that some row of the CTA
// masks, two warps take values that are not finite out of V as soon as it has
// landed (rows past the sequence's end become zero), and the rows that do see
// such a key get its values added at the end, as the formula has them.
#include <cuda_bf16.h>

#include "gqa.cuh"
#include "ptx.cuh"

namespace csa {
namespace {

constexpr int kTileShift = 7;
constexpr int kTile = 1 << kTileShift;   // queries and keys a tile
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
  // The output is staged 32 channels at a time in a place of its own, so that
  // the next queries are copied and multiplied under it (32 prompts of 500 131
  // us, 143 where the queries were).  Two tiles a CTA stage it whole where their
  // queries were, and the next ones wait for it: in a place of its own, 32
  // channels at a time, 16 of 1000 took 210 us instead of 183.
  static constexpr bool kOwnStage = QT == 1;
  static constexpr int kOutBytes = kOwnStage ? kTile * 64 : 0;
  static constexpr int kSmem = (QT + kStages) * kTileBytes + kOutBytes + 1024;
  // Parts that a tile of keys is worked on in: with one tile of queries the
  // scores of one half are computed while the other's softmax runs.
  static constexpr int kParts = QT == 1 ? 2 : 1;
  static constexpr int kPart = kTile / kParts;
  static constexpr int kSCol(int t) { return t * kTile; }
  static constexpr int kOCol(int t) { return QT * kTile + t * D; }
  static constexpr int kCols = QT == 2 ? 512 : 256;
  // Where 168 (or 128) registers a thread are launched, the softmax warps
  // take some that the other four give up: 256 x 208 + 128 x 88 = 384 x 168,
  // 128 x 168 + 128 x 88 = 256 x 128.
  static constexpr bool kSplit = QT == 2 || CTAS == 2;
  static constexpr int kLaunchRegs = QT == 2 ? 168 : 128;
  static constexpr int kSoftmaxRegs = QT == 2 ? 208 : 168, kOtherRegs = 88;
  static_assert(!kSplit || QT * 128 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "registers of the block");
  // One CTA of one tile an SM: the keys may be shared out over a cluster,
  // whose fp32 sums meet in the rings.
  static constexpr bool kCluster = QT == 1 && CTAS == 1;
  static_assert(!kCluster || kStages * kTileBytes >= kTile * D * 4, "the sums fit the ring");
};

__device__ __forceinline__ bool not_finite(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }

// Non-zero where a half of the word is a bf16 infinity or NaN (magnitude bits
// of 0x7F80 and more carry into the half's top bit).
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) { return ((w & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u; }
// acc + 0 * w, of bf16 pairs: NaN from the first such half on, else still zero.
__device__ __forceinline__ uint32_t probe(uint32_t w, uint32_t acc) {
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w), "r"(0u));
  return acc;
}
// The word with such halves zeroed.
__device__ __forceinline__ uint32_t finite_halves(uint32_t w) {
  if (not_finite(w)) w &= 0xFFFF0000u;
  if (not_finite(w >> 16)) w &= 0xFFFFu;
  return w;
}

// Tiles of keys [lo, hi).
struct Range {
  int lo, hi;
};
// Tiles of keys that some row masks a part of: those from `from` on, and those up to `upto`.
struct Masked {
  int from, upto;
  __device__ __forceinline__ bool at(int j) const { return j >= from || j <= upto; }
};

struct Seq {
  int q0, k0;  // first rows of the sequence
  int nq, nk;
};

// A CTA's tiles of one head: queries row0 .. of a sequence.
struct Work {
  Seq sq;
  int row0, head, shift;  // row i sits at position i + shift among the keys

  __device__ __forceinline__ int rows(int t) const { return max(0, min(kTile, sq.nq - row0 - t * kTile)); }
  // the tiles of keys that rows [first, first + n) see (lengths are below 2^30 each: no overflow)
  __device__ __forceinline__ Range range(const PromptAttnArgs& a, int first, int n) const {
    const int pos = first + shift;
    const int hi = a.causal ? min(sq.nk, pos + n) : sq.nk;
    const int lo = a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
    const bool none = n <= 0 || hi <= lo;
    Range r;
    r.lo = none ? 0 : lo >> kTileShift;
    r.hi = none ? 0 : (hi + kTile - 1) >> kTileShift;
    return r;
  }
  __device__ __forceinline__ Masked masked(const PromptAttnArgs& a, int first, int n) const {
    Masked m;
    m.from = sq.nk >> kTileShift;   // the sequence ends inside the tile (or before it)
    const int pos = first + shift;  // the first row's last key
    if (a.causal) m.from = min(m.from, pos < 0 ? 0 : (pos + 1) >> kTileShift);
    const int last = pos + n - 1;  // the last row's last key: keys up to last - window are outside its window
    m.upto = a.window > 0 && last >= a.window ? (last - a.window) >> kTileShift : -1;
    return m;
  }
};

// The ranges of a CTA's tiles and their union, walked downwards: iteration it
// works on tile j_hi - 1 - it of the keys.  (With a window neighbouring
// tiles' ranges meet, so every iteration has a tile that works.)
template <int QT>
struct Walk {
  Range rt[QT];
  int j_hi, n_it;

  __device__ __forceinline__ void set(const PromptAttnArgs& a, const Work& w, int rank, int cluster) {
    int j_lo = 0x7fffffff;
    j_hi = 0;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      rt[t] = w.range(a, w.row0 + t * kTile, w.rows(t));
      if (cluster > 1) {  // this CTA's part of the keys
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
    n_it = j_hi > 0 ? j_hi - j_lo : 0;
  }
  // iterations [begin, end) of tile t
  __device__ __forceinline__ int begin(int t) const { return rt[t].lo < rt[t].hi ? j_hi - rt[t].hi : 0; }
  __device__ __forceinline__ int end(int t) const { return rt[t].lo < rt[t].hi ? j_hi - rt[t].lo : 0; }
};

// Walks a CTA's share of the work: items (tiles of ROWS queries of a sequence,
// the later ones first: under the causal mask they see more keys) times
// heads.  CTA c of G takes c, 2G - 1 - c, 2G + c, ...: forward and backward in
// turn, so that no CTA gets the longer one of every G.  The places grow, so
// it never looks back.  Offsets that fall can make sequences overlap, whose
// items could pass 32 bits: a CTA takes no more turns than others can need.
template <int ROWS>
struct Walker {
  int b0 = 0, base = 0, round = 0;  // sequences before b0 hold `base` items

  __device__ __forceinline__ bool next(const PromptAttnArgs& a, int cta, int ctas, Work* w) {
    const int place = round * ctas + ((round & 1) ? ctas - 1 - cta : cta);
    ++round;
    return at(a, place, w);
  }
  __device__ __forceinline__ bool at(const PromptAttnArgs& a, int place, Work* w) {
    const int item = place / a.n_heads;
    w->head = place - item * a.n_heads;
    return find(a, item, w);
  }
  __device__ __forceinline__ bool find(const PromptAttnArgs& a, int item, Work* w) {
    const int lane = threadIdx.x & 31;
    for (; b0 < a.B; b0 += 32) {
      Seq s = {0, 0, 0, 0};
      if (b0 + lane < a.B) {
        const int32_t q0 = __ldg(a.cu_q + b0 + lane), q1 = __ldg(a.cu_q + b0 + lane + 1);
        const int32_t k0 = __ldg(a.cu_k + b0 + lane), k1 = __ldg(a.cu_k + b0 + lane + 1);
        if (q0 >= 0 && q1 >= q0 && q1 <= a.n_q && k0 >= 0 && k1 >= k0 && k1 <= a.n_k)
          s = {q0, k0, q1 - q0, k1 - k0};
        else
          record_error(a.status, kErrIndexRange);
      }
      const int n = (s.nq + ROWS - 1) / ROWS;
      int x = n;
      if (a.B - b0 > 1) {
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, off);
          if (lane >= off) x += y;
        }
      }
      const int all = __shfl_sync(0xffffffffu, x, a.B - b0 > 1 ? 31 : 0);
      if (item < base + all) {
        const int from = __ffs(__ballot_sync(0xffffffffu, base + x > item)) - 1;
        w->sq.q0 = __shfl_sync(0xffffffffu, s.q0, from);
        w->sq.k0 = __shfl_sync(0xffffffffu, s.k0, from);
        w->sq.nq = __shfl_sync(0xffffffffu, s.nq, from);
        w->sq.nk = __shfl_sync(0xffffffffu, s.nk, from);
        w->row0 = (base + __shfl_sync(0xffffffffu, x, from) - 1 - item) * ROWS;
        w->shift = w->sq.nk - w->sq.nq;
        return true;
      }
      base += all;
    }
    return false;
  }
};

// A work item as the loading warp finds it and hands it to the others (the
// search costs each item about 1000 cycles, which no other warp waits for).
template <int QT>
struct Order {
  Work w;
  Walk<QT> walk;
  Masked masked;  // over all of the CTA's rows
  int there;      // 0: no more
};

template <int D, int QT, int CTAS>
__global__ void __launch_bounds__(Cfg<D, QT, CTAS>::kThreads, CTAS)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PromptAttnArgs a, const int cluster_size,
                       const int max_turns) {
  using C = Cfg<D, QT, CTAS>;
  constexpr int kTmaWarp = 4 * QT, kMmaWarp = 4 * QT + 1, kCleanWarp = 4 * QT + 2;
  constexpr int kRowsCta = QT * kTile;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t q_full[QT], q_empty[QT], full[C::kStages], empty[C::kStages];
  __shared__ uint64_t s_full[QT][C::kParts], p_full[QT][C::kParts], pv_done[QT][C::kParts];
  __shared__ uint64_t o_full[QT], dirty[C::kStages / 2], cleaned[C::kStages / 2];  // (by the values' ring slots)
  __shared__ uint64_t drain, order_full[2], order_empty[2];
  __shared__ Order<QT> orders[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s;
  // keys of each masked tile whose values are not all finite, as each of the
  // two cleaning warps found them, of three work items (who cleans item n + 2
  // knows that every warp has begun item n): those of item number n are valid
  // if odd_item[n % 3] is n + 1
  __shared__ uint32_t odd_rows[3][2][kMaxMasked][4];
  __shared__ int odd_tile[3][kMaxMasked], odd_item[3][2];
  __shared__ float m_s[C::kCluster ? kTile : 1], l_s[C::kCluster ? kTile : 1];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* q_s = smem;
  uint8_t* ring = smem + QT * C::kTileBytes;
  uint8_t* out_s = ring + C::kStages * C::kTileBytes;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  volatile int* abort_flag = &abort_s;
  if (tid == 0) {
    mbar_init(&drain, 1);
    for (int i = 0; i < C::kStages / 2; ++i) {
      mbar_init(dirty + i, 1);
      mbar_init(cleaned + i, kCleanThreads);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(order_full + i, 1);
      mbar_init(order_empty + i, C::kThreads / 32 - 1);
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int t = 0; t < QT; ++t) {
      mbar_init(q_full + t, 1);
      mbar_init(q_empty + t, kTile + 1);
      for (int h = 0; h < C::kParts; ++h) {
        mbar_init(&s_full[t][h], 1);
        mbar_init(&p_full[t][h], kTile);
        mbar_init(&pv_done[t][h], 1);
      }
      mbar_init(o_full + t, 1);
    }
    fence_mbar_init();
    abort_s = 0;
    for (int i = 0; i < 3; ++i) odd_item[i][0] = odd_item[i][1] = 0;
  }
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
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = tmem_slot;

  // A cluster's CTAs work on one item, each on a part of its keys; other CTAs
  // walk through their share of the items.
  const int cluster = C::kCluster ? cluster_size : 1;
  const int cta = static_cast<int>(blockIdx.x) / cluster, rank = static_cast<int>(blockIdx.x) - cta * cluster;
  // the next item, of every warp but the loading one; false at the end and after an abort
  auto take = [&](int item, Order<QT>* o) {
    const bool ok = wait_or_abort(order_full + (item & 1), (item >> 1) & 1, abort_flag, a.status);
    if (!__all_sync(0xffffffffu, ok)) return false;
    *o = orders[item & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(order_empty + (item & 1));
    return o->there != 0;
  };

  if (warp >= 4 * QT) {
    if constexpr (C::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    if (warp == kTmaWarp) {
      // ---------------- loads ----------------
      int seq = 0, n_q[QT] = {};  // ring slots and query tiles filled so far
      bool ok = true;
      Walker<kRowsCta> walker;
      for (int item = 0, there = 1; ok && there; ++item) {
        Order<QT> o;
        const Work& w = o.w;
        const Walk<QT>& walk = o.walk;
        if (C::kCluster)
          there = item == 0 && walker.at(a, cta, &o.w);
        else
          there = item <= max_turns && walker.next(a, cta, static_cast<int>(gridDim.x), &o.w);
        o.there = there;
        if (there) {
          o.walk.set(a, w, rank, cluster);
          o.masked = w.masked(a, w.row0, min(kRowsCta, w.sq.nq - w.row0));
        }
        if (lane == 0) {
          if (item >= 2) ok = wait_or_abort(order_empty + (item & 1), ((item >> 1) - 1) & 1, abort_flag, a.status);
          if (ok) {
            orders[item & 1] = o;
            mbar_arrive(order_full + (item & 1));
          }
        }
        if (lane == 0 && there && ok) {
          const int kv_head = w.head / (a.n_heads / a.n_kv_heads);
          auto load = [&](int s) {
            const int slot = seq & (C::kStages - 1);
            if (seq >= C::kStages) ok = wait_or_abort(empty + slot, ((seq / C::kStages) - 1) & 1, abort_flag, a.status);
            if (!ok) return;
            mbar_arrive_expect_tx(full + slot, C::kTileBytes);
            const int j = walk.j_hi - 1 - (s >> 1), row = w.sq.k0 + j * kTile;
            for (int k = 0; k < C::kBlocks; ++k)
              tma_load_3d(ring + slot * C::kTileBytes + k * C::kBlockBytes, (s & 1) ? &tm_v : &tm_k, k * 64, kv_head,
                          row, full + slot);
            if ((s & 1) && o.masked.at(j)) mbar_arrive(dirty + (slot >> 1));
            ++seq;
          };
          // the first keys before the queries, which wait for the item before's
          // last scores, and the values, which wait for its last product
          int s = 0;
          for (; ok && s < min(1, walk.n_it); ++s) load(s);
          for (int t = 0; ok && t < QT; ++t) {
            if (item > 0) ok = wait_or_abort(q_empty + t, (item - 1) & 1, abort_flag, a.status);
            if (!ok) break;
            mbar_arrive_expect_tx(q_full + t, C::kTileBytes);
            for (int k = 0; k < C::kBlocks; ++k)
              tma_load_3d(q_s + t * C::kTileBytes + k * C::kBlockBytes, &tm_q, k * 64, w.head,
                          w.sq.q0 + w.row0 + t * kTile, q_full + t);
            ++n_q[t];
          }
          for (; ok && s < 2 * walk.n_it; ++s) load(s);
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      // (the offsets behind the last item are looked at too)
      if (C::kCluster && static_cast<int>(blockIdx.x) + 1 == static_cast<int>(gridDim.x)) {
        Work none;
        walker.find(a, 1 << 30, &none);
      }
      if (lane == 0) {  // every copy lands before the CTA ends (also after an abort)
        for (int t = 0; t < QT; ++t)
          if (n_q[t] > 0) mbar_wait(q_full + t, (n_q[t] - 1) & 1, a.status);
        for (int k = max(0, seq - C::kStages); k < seq; ++k)
          mbar_wait(full + (k & (C::kStages - 1)), (k / C::kStages) & 1, a.status);
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ---------------- products ----------------
      // The whole warp walks the loop and one elected lane issues: with the
      // loop's values warp-uniform (the shuffles say so to the compiler) an
      // issue costs a few cycles; from a branch on lane 0 each product took
      // about 115, more than it takes to compute.
      constexpr uint32_t idesc_s = instr_desc(kTile, C::kPart, 1, 1, 0, 0);  // bf16, K-major A and B
      constexpr uint32_t idesc_o = instr_desc(kTile, D, 1, 1, 0, 1);      // A from TMEM, B (= V) MN-major
      auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t rb = smem_u32(ring);
      const bool skip_s = test_fault(a.status, kFaultAttn);  // test fault: S is never announced
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, a.status)) != 0;
      };
      auto wait_slot = [&](int seq) {
        return wait(full + (seq & (C::kStages - 1)), (seq / C::kStages) & 1);
      };
      bool ok = true;
      int seq0 = 0;               // ring slots of the items before
      uint32_t n_p[QT] = {};      // weights taken so far, by tile
      uint32_t parity_c = 0;      // of `cleaned`, a bit a slot
      Order<QT> order;
      for (int item = 0; ok && take(item, &order); ++item) {
        const Walk<QT>& walk = order.walk;
        const Masked& masked = order.masked;
        const int n_it = uniform(walk.n_it);
        int begin[QT], end[QT];
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          begin[t] = uniform(walk.begin(t));
          end[t] = uniform(walk.end(t));
        }
        const int m_from = uniform(walk.j_hi - masked.from), m_upto = uniform(walk.j_hi - 1 - masked.upto);
        // scores of part h of a tile of keys, S_t = Q_t K^T (one lane)
        auto s_of = [&](int t, int h, uint64_t k_desc) {
          const uint64_t q_desc = smem_desc(smem_u32(q_s) + t * C::kTileBytes, 16, 1024, kSwizzle128B);
          k_desc += h * (C::kPart * 128 >> 4);
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            constexpr int kStep = 32 >> 4;  // 16 channels along a 128-byte line, in the descriptors' units
            const int off = (s >> 2) * (C::kBlockBytes >> 4) + (s & 3) * kStep;
            mma_f16(tm + C::kSCol(t) + h * C::kPart, q_desc + off, k_desc + off, idesc_s, s > 0 ? 1u : 0u);
          }
          if (!skip_s) tc_commit(&s_full[t][h]);
        };
        // the first tile of keys (the queries are waited for even without one:
        // a phase that is not waited for could be taken for a later one)
        if (n_it > 0) ok = wait_slot(seq0);
        const uint64_t k_first = smem_desc(rb + (seq0 & (C::kStages - 1)) * C::kTileBytes, 16, 1024, kSwizzle128B);
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          if (ok) ok = wait(q_full + t, item & 1);
          if (ok) {
            tc_fence_after();
            if (elect_one()) {
              mbar_arrive(q_empty + t);  // (a tile without keys would be freed without this warp)
              if (begin[t] == 0 && end[t] > 0) {
#pragma unroll
                for (int h = 0; h < C::kParts; ++h) s_of(t, h, k_first);
              }
            }
            __syncwarp();
          }
        }
        if (ok && n_it > 0 && elect_one()) tc_commit(empty + (seq0 & (C::kStages - 1)));
        __syncwarp();
        for (int it = 0; it < n_it && ok; ++it) {
          const int v_seq = seq0 + 2 * it + 1, v_slot = v_seq & (C::kStages - 1), k_slot = (v_seq + 1) & (C::kStages - 1);
          const uint64_t v_desc = smem_desc(rb + v_slot * C::kTileBytes, C::kBlockBytes, 1024, kSwizzle128B);
          const uint64_t k_desc = smem_desc(rb + k_slot * C::kTileBytes, 16, 1024, kSwizzle128B);
          const bool again = it + 1 < n_it;
          // this tile's values and the next tile's keys are usually there long
          // before the weights are
          ok = wait_slot(v_seq);
          if (ok && (it < m_from || it >= m_upto)) {
            ok = wait(cleaned + (v_slot >> 1), (parity_c >> (v_slot >> 1)) & 1u);
            parity_c ^= 1u << (v_slot >> 1);
          }
          if (ok && again) ok = wait_slot(v_seq + 1);
#pragma unroll
          for (int t = 0; t < QT; ++t) {
            const bool pv = it >= begin[t] && it < end[t], next = again && it + 1 >= begin[t] && it + 1 < end[t];
            // (unrolled, the long products of width 128 spill where two CTAs share
            // an SM's registers: 32 prompts of 500 130 us, 119 so)
#pragma unroll(C::kStages == 2 ? 1 : C::kParts)
            for (int h = 0; h < C::kParts; ++h) {
              const bool last = t == QT - 1 && h == C::kParts - 1;
              if (ok && pv) ok = wait(&p_full[t][h], n_p[t] & 1u);
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) {
                if (pv) {
#pragma unroll
                  for (int s = 0; s < C::kPart / 16; ++s)
                    mma_f16_ts(tm + C::kOCol(t), tm + C::kSCol(t) + h * C::kPart + s * 8,
                               v_desc + ((h * C::kPart + 16 * s) * 128 >> 4), idesc_o,
                               (it > begin[t] || h > 0 || s > 0) ? 1u : 0u);
                  if (C::kParts > 1) tc_commit(&pv_done[t][h]);
                  if (it + 1 == end[t] && h == C::kParts - 1) tc_commit(o_full + t);
                }
                if (last) tc_commit(empty + v_slot);
                if (next) s_of(t, h, k_desc);
                if (last && again) tc_commit(empty + k_slot);
              }
              __syncwarp();
            }
            if (pv) ++n_p[t];
          }
        }
        seq0 += 2 * n_it;
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
      int seq0 = 0;
      uint32_t parity_d = 0;  // of `dirty`, a bit a slot
      bool ok = true;
      Order<QT> order;
      for (int item = 0; ok && take(item, &order); ++item) {
        const Work& w = order.w;
        const Walk<QT>& walk = order.walk;
        const Masked& masked = order.masked;
        const int o = item % 3, half = warp - kCleanWarp;
        static_assert(kMaxMasked * 4 == 32, "a word a lane");
        int n_masked = 0;
        for (int it = 0; it < walk.n_it; ++it) {
          const int j = walk.j_hi - 1 - it;
          if (!masked.at(j)) continue;
          const int seq = seq0 + 2 * it + 1, slot = seq & (C::kStages - 1);
          // the tile's copy has been issued, so its slot's phase before is over
          // (without that the second wait could take it for this one), and
          // the product warp holds the slot until `cleaned`
          ok = wait_or_abort(dirty + (slot >> 1), (parity_d >> (slot >> 1)) & 1u, abort_flag, a.status) &&
               wait_or_abort(full + slot, (seq / C::kStages) & 1, abort_flag, a.status);
          parity_d ^= 1u << (slot >> 1);
          ok = __all_sync(0xffffffffu, ok) != 0;
          if (!ok) break;
          if (n_masked == 0) {  // (the item three before, whose places these were, is done with)
            odd_rows[o][half][lane >> 2][lane & 3] = 0u;
            __syncwarp();
          }
          uint4* tile = reinterpret_cast<uint4*>(ring + slot * C::kTileBytes);
          // rows past the sequence become zero; of the others, eight 16-byte
          // chunks at a time are looked at for an exponent of all ones (the
          // swizzle moves chunks within their row only: chunk i is of row i/8 % 128)
          const int past = min(w.sq.nk - j * kTile, kTile);
          if (past < kTile)
            for (int i = ct; i < (kTile - past) * 8 * C::kBlocks; i += kCleanThreads) {
              const int block = i / ((kTile - past) * 8);
              tile[block * kTile * 8 + past * 8 + i - block * (kTile - past) * 8] = make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll 1
          for (int i0 = ct; i0 < C::kTileBytes / 16; i0 += 8 * kCleanThreads) {
            uint4 u[8];
            uint32_t any[4] = {};
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] = tile[i0 + k * kCleanThreads];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              any[0] = probe(u[k].x, any[0]);
              any[1] = probe(u[k].y, any[1]);
              any[2] = probe(u[k].z, any[2]);
              any[3] = probe(u[k].w, any[3]);
            }
            if (odd_halves(any[0] | any[1] | any[2] | any[3]) == 0u) continue;
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
              const int i = i0 + k * kCleanThreads, r = (i >> 3) & (kTile - 1);
              uint4 v = tile[i];
              if (r >= past || !(odd_halves(v.x) | odd_halves(v.y) | odd_halves(v.z) | odd_halves(v.w))) continue;
              v.x = finite_halves(v.x);
              v.y = finite_halves(v.y);
              v.z = finite_halves(v.z);
              v.w = finite_halves(v.w);
              tile[i] = v;
              if (n_masked < kMaxMasked) {
                atomicOr(&odd_rows[o][half][n_masked][r >> 5], 1u << (r & 31));
                odd_tile[o][n_masked] = j;
                odd_item[o][half] = item + 1;
              }
            }
          }
          ++n_masked;
          fence_proxy_async_smem();
          mbar_arrive(cleaned + (slot >> 1));
        }
        seq0 += 2 * walk.n_it;
      }
    }
  } else {
    // ---------------- softmax: one thread a query row ----------------
    if constexpr (C::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_tmem = tmem + lane_base + C::kSCol(t), o_tmem = tmem + lane_base + C::kOCol(t);
    const float scale2 = a.sm_scale * kLog2e;
    uint32_t n_s = 0, n_o = 0;  // tiles of scores and sums taken so far
    bool ok = true;
    for (int item = 0; ok; ++item) {
      Work w;
      int n_tiles, j_top, last_key, first_key;
      bool loaded;
      Masked masked_t;
      {
        Order<QT> order;
        if (!take(item, &order)) break;
        w = order.w;
        const Range mine = QT == 1 || t == 0 ? order.walk.rt[0] : order.walk.rt[QT - 1];
        n_tiles = mine.hi - mine.lo;
        j_top = mine.hi - 1;
        masked_t = w.masked(a, w.row0 + t * kTile, w.rows(t));
        // the row's keys [first_key, last_key]
        const int at_key = w.row0 + t * kTile + r + w.shift;
        last_key = a.causal ? min(at_key, w.sq.nk - 1) : w.sq.nk - 1;
        first_key = a.window > 0 && at_key >= a.window ? at_key - a.window + 1 : 0;
        loaded = n_tiles > 0;
      }
      float m = a.no_key, l = 0.f;  // the reference of the weights e^(scale (s - m)), in the products' units
      bool large = false;        // of the warp: some row's logits are large (see below)
      auto is_large = [&]() { return m > a.no_key && fabsf(m * scale2) > 65536.f; };
      for (int part = 0; part < n_tiles * C::kParts; ++part) {
        const int n = part / C::kParts, h = part % C::kParts, j = j_top - n;
        ok = wait_or_abort(&s_full[t][h], (n_s + n) & 1, abort_flag, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (C::kOwnStage && part + 1 == n_tiles * C::kParts) mbar_arrive(q_empty + t);  // the queries' last scores
        constexpr int kC = C::kPart / 32;
        uint32_t s[kC][32];
#pragma unroll
        for (int c = 0; c < kC; ++c) tmem_ld32(s_tmem + h * C::kPart + 32 * c, s[c]);
        tmem_wait_ld();
        if (masked_t.at(j)) {  // this row's keys among the tile's columns, as a bit each
          const int c0 = j * kTile + h * C::kPart, c_hi = last_key + 1 - c0, c_lo = first_key - c0;
#pragma unroll
          for (int c = 0; c < kC; ++c) {
            const int hi = max(0, min(32, c_hi - 32 * c)), lo = max(0, min(32, c_lo - 32 * c));
            const uint32_t seen = static_cast<uint32_t>((1ull << hi) - (1ull << min(lo, hi)));
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!((seen >> k) & 1u)) s[c][k] = 0xFF800000u;  // -inf
          }
        }
        float top[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          top[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
          for (int k = 2; k < 32; k += 2) top[c] = max3(top[c], __uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1]));
        }
        float top1 = top[0];
#pragma unroll
        for (int c = 1; c < kC; ++c) top1 = fmaxf(top1, top[c]);
        // (a row whose own maximum has not grown keeps its reference, so that no bit
        // of it depends on what only the warp's other rows see)
        const bool grown = (top1 - m) * scale2 > kLag;
        if (__any_sync(0xffffffffu, grown)) {
          const float f = grown ? ex2((m - top1) * scale2) : 1.f;
          if (grown) m = top1;
          l *= f;
          large = __any_sync(0xffffffffu, is_large());
          if (part > 0) {
            // the products of the parts before have finished: these scores were
            // issued after them, but for the last one's where parts alternate
            if (C::kParts > 1) {
              ok = wait_or_abort(&pv_done[t][h ^ 1], (n_s + n - (h ^ 1)) & 1, abort_flag, a.status);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              tc_fence_after();
            }
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
        const uint64_t scale_2 = pair_of(scale2, scale2);
        // scale s - scale m in one rounding; where the logits are so large that
        // the rounding of scale m shows, s - m first
        float offset = -m * scale2;
        if (large) {
          const float less = is_large() ? m : 0.f;
          if (is_large()) offset = 0.f;
#pragma unroll
          for (int c = 0; c < kC; ++c)
#pragma unroll
            for (int k = 0; k < 32; ++k) s[c][k] = __float_as_uint(__uint_as_float(s[c][k]) - less);
        }
        const uint64_t minus_m = pair_of(offset, offset);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float x, y;
            split(fma2(pair_of(s[c][2 * k], s[c][2 * k + 1]), scale_2, minus_m), &x, &y);
            x = ex2(x);
            y = ex2(y);
            sum[k & 1] = add2(sum[k & 1], pair_of(x, y));
            const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
            p[k] = *reinterpret_cast<const uint32_t*>(&v);
          }
          tmem_st16(s_tmem + h * C::kPart + 16 * c, p);
        }
        float sx, sy;
        split(add2(sum[0], sum[1]), &sx, &sy);
        l += sx + sy;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[t][h]);
      }
      n_s += n_tiles;
      if (ok) {  // (a tile that sees no keys: not before its queries have landed, so that no phase is passed by)
        ok = loaded ? wait_or_abort(o_full + t, n_o++ & 1, abort_flag, a.status)
                    : wait_or_abort(q_full + t, item & 1, abort_flag, a.status);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        if (C::kOwnStage && !loaded) mbar_arrive(q_empty + t);
      }
      if (!ok) break;
      const int rows = w.rows(t);
      if (rows > 0) {
        // (masked tiles were cleaned before their products, so odd_item is final)
        const int64_t row = static_cast<int64_t>(w.sq.q0 + w.row0 + t * kTile + r) * a.n_heads + w.head;
        const bool shared = C::kCluster && cluster > 1;
        if (shared) {  // the sums as they are
          m_s[r] = m * scale2;
          l_s[r] = l;
          l = 1.f;
        } else {
          float lse;
          l = finish_row(m * scale2, 0.f, l, a.sink, w.head, &lse);
          if (a.lse && r < rows) a.lse[row] = lse;
        }
        const int o2 = item % 3;
        const bool odd0 = *const_cast<volatile int*>(&odd_item[o2][0]) == item + 1;
        const bool odd1 = *const_cast<volatile int*>(&odd_item[o2][1]) == item + 1;
        // the warp's 32 rows are staged, then stored with neighbouring lanes on
        // one row
        uint16_t* out = a.out + (static_cast<int64_t>(w.sq.q0 + w.row0 + t * kTile) * a.n_heads + w.head) * D;
        const int w0 = (warp & 3) * 32;
        uint8_t* stage = C::kOwnStage ? out_s + w0 * 64 : q_s + t * C::kTileBytes + w0 * 128;
#pragma unroll 1  // (code that runs once waits for its instructions)
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
          const uint64_t l2 = pair_of(l, l);
#pragma unroll
          for (int k = 0; k < 32; k += 2) split(mul2(pair_of(o[k], o[k + 1]), l2), &x[k], &x[k + 1]);
          if ((odd0 || odd1) && r < rows) {
            const uint16_t* values =
                a.v + w.sq.k0 * a.v_stride + w.head / (a.n_heads / a.n_kv_heads) * a.v_stride_h + 32 * c;
            for (int e = 0; e < kMaxMasked * kTile; ++e) {
              const uint32_t word = (odd0 ? odd_rows[o2][0][e >> 7][(e >> 5) & 3] : 0u) |
                                    (odd1 ? odd_rows[o2][1][e >> 7][(e >> 5) & 3] : 0u);
              if (!((word >> (e & 31)) & 1u)) continue;
              const int key = odd_tile[o2][e >> 7] * kTile + (e & (kTile - 1));
              if (key > last_key || key < first_key) continue;
              const uint16_t* v = values + key * a.v_stride;
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
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 y = __floats2bfloat162_rn(x[8 * k + 2 * e], x[8 * k + 2 * e + 1]);
              v[e] = *reinterpret_cast<const uint32_t*>(&y);
            }
            uint8_t* to = C::kOwnStage ? stage + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)
                                       : stage + (c >> 1) * C::kBlockBytes + lane * 128 +
                                             ((((c & 1) * 4 + k) ^ (lane & 7)) << 4);
            *reinterpret_cast<uint4*>(to) = make_uint4(v[0], v[1], v[2], v[3]);
          }
          if (C::kOwnStage) {
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int rr = 8 * k + lane / 4, ch = lane % 4;
              const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 64 + ((ch ^ ((rr >> 1) & 3)) << 4));
              if (w0 + rr < rows)
                *reinterpret_cast<uint4*>(out + static_cast<int64_t>(w0 + rr) * a.n_heads * D + 32 * c + 8 * ch) = v;
            }
            __syncwarp();
          }
        }
        if (!C::kOwnStage) {
          __syncwarp();
          constexpr int kChunks = D / 8, kRowsAtOnce = 32 / kChunks;
#pragma unroll 4
          for (int k = 0; k < 32 / kRowsAtOnce; ++k) {
            const int rr = k * kRowsAtOnce + lane / kChunks, ch = lane % kChunks;
            const uint4 v = *reinterpret_cast<const uint4*>(stage + (ch >> 3) * C::kBlockBytes + rr * 128 +
                                                            (((ch & 7) ^ (rr & 7)) << 4));
            if (w0 + rr < rows)
              *reinterpret_cast<uint4*>(out + static_cast<int64_t>(w0 + rr) * a.n_heads * D + 8 * ch) = v;
          }
        }
      }
      if (!C::kOwnStage) {
        fence_proxy_async_smem();  // the next queries are copied over what was staged
        mbar_arrive(q_empty + t);
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
  if constexpr (C::kCluster) {
    if (cluster > 1) {
      // Every CTA adds up its share of the rows over the cluster, 16 / cluster
      // rows a warp: the references and sums of all its rows and CTAs at once,
      // one a lane, then a row (of 64 channels two) at a time, 4 channels a lane.
      const bool there = *abort_flag == 0 && orders[0].there != 0;
      Work w = {};  // (one item, the whole cluster's)
      if (there) w = orders[0].w;
      cluster_sync();
      constexpr int kLanes = D / 4, kRowsAtOnce = 32 / kLanes;
      const int per_warp = 16 / cluster, rows = there ? w.rows(0) : 0;
      const int first = rank * (kTile / cluster) + warp * per_warp;
      static_assert(C::kThreads == 256, "eight warps");
      float g;
      {
        const int p = lane % cluster, r = first + (lane & 15) / cluster;
        const float m = dsmem_ld_f32(dsmem_addr(m_s + r, p)), l = dsmem_ld_f32(dsmem_addr(l_s + r, p));
        float top = m;
        for (int off = 1; off < cluster; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float f = ex2(m - top);
        float sum = l * f;
        for (int off = 1; off < cluster; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        float lse;
        g = f * finish_row(top, 0.f, sum, a.sink, w.head, &lse);
        if (a.lse && lane < 16 && p == 0 && r < rows)
          a.lse[static_cast<int64_t>(w.sq.q0 + w.row0 + r) * a.n_heads + w.head] = lse;
      }
#pragma unroll 2
      for (int i0 = 0; i0 < per_warp; i0 += kRowsAtOnce) {
        const int i = i0 + lane / kLanes, ch = lane % kLanes, r = first + i;
        float4 v[8];
#pragma unroll
        for (int p = 0; p < 8; ++p)
          if (p < cluster) v[p] = dsmem_ld_f32x4(dsmem_addr(ring + r * D * 4 + ((ch ^ (r & (D / 4 - 1))) << 4), p));
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int p = 0; p < 8; ++p)
          if (p < cluster) {
            const float f = __shfl_sync(0xffffffffu, g, i * cluster + p);
            o.x = fmaf(v[p].x, f, o.x);
            o.y = fmaf(v[p].y, f, o.y);
            o.z = fmaf(v[p].z, f, o.z);
            o.w = fmaf(v[p].w, f, o.w);
          }
        if (r < rows) {
          const int64_t row = static_cast<int64_t>(w.sq.q0 + w.row0 + r) * a.n_heads + w.head;
          const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
          *reinterpret_cast<uint2*>(a.out + row * D + 4 * ch) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        }
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

// Tiles of `rows` queries that the sequences have at most: n rows are at most
// n / R + 1 tiles of R rows, and at most n.
int64_t max_items(const PromptAttnArgs& a, int rows) {
  const int64_t most = a.n_q / rows + a.B;
  return most < a.n_q ? most : a.n_q;
}

template <int D, int QT, int CTAS>
cudaError_t launch_dim(const PromptAttnArgs& a, PFN_cuTensorMapEncodeTiled_v12000 encode, int sms,
                       int cluster, cudaStream_t stream) {
  using C = Cfg<D, QT, CTAS>;
  const auto kernel = prompt_attn_kernel<D, QT, CTAS>;
  CUtensorMap tm_q, tm_k, tm_v;
  const int64_t n_k = a.n_k > 0 ? a.n_k : 1;  // (no keys: the maps are not read)
  if (!encode || !encode_rows(&tm_q, encode, a.q, D, a.n_heads, a.n_q, a.q_stride, a.q_stride_h) ||
      !encode_rows(&tm_k, encode, a.n_k > 0 ? a.k : a.q, D, a.n_kv_heads, n_k, a.k_stride, a.k_stride_h) ||
      !encode_rows(&tm_v, encode, a.n_k > 0 ? a.v : a.q, D, a.n_kv_heads, n_k, a.v_stride, a.v_stride_h))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done{0};
  // (the split of registers assumes what the kernel is launched with)
  const cudaError_t e = kernel_limits(reinterpret_cast<const void*>(kernel), C::kSmem, C::kSplit ? C::kLaunchRegs : 0,
                                      &done);
  if (e != cudaSuccess) return e;
  int64_t grid = max_items(a, QT * kTile) * a.n_heads, turns = 1;
  if (grid > 0x3fffffff) return cudaErrorInvalidValue;
  if (C::kCluster)
    grid *= cluster;  // an item a cluster
  else if (grid > static_cast<int64_t>(sms) * CTAS) {
    turns = grid;
    grid = static_cast<int64_t>(sms) * CTAS;  // resident CTAs, that walk through the items
    turns = (turns + grid - 1) / grid;
  }
  return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(grid)), dim3(C::kThreads), C::kSmem, stream,
                            static_cast<unsigned>(cluster), tm_q, tm_k, tm_v, a, cluster, static_cast<int>(turns));
}

template <int D>
cudaError_t launch_tiles(const PromptAttnArgs& a, PFN_cuTensorMapEncodeTiled_v12000 encode, cudaStream_t stream) {
  const int sms = current_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int64_t tiles = max_items(a, kTile) * a.n_heads;
  if (tiles <= sms) {
    // Few tiles, an SM each; a cluster shares out the keys of a tile while
    // SMs are left and a CTA has two tiles of keys at least.
    int cluster = 1;
    while (cluster < 8 && tiles * cluster * 2 <= sms && a.n_k >= static_cast<int64_t>(a.B) * 4 * cluster * kTile)
      cluster *= 2;
    return launch_dim<D, 1, 1>(a, encode, sms, cluster, stream);
  }
  // Two tiles a CTA share the keys' copies and overlap one's softmax with the
  // other's products; where a tile sees few keys, or a sequence has one tile,
  // two CTAs of one tile on an SM overlap their starts and ends instead.
  // Width 128, 32 heads, us with one and with two tiles a CTA: 64 prompts of
  // 300 152 and 227, 24 of 640 125 and 163, 16 of 1000 177 and 184, of 1200 245
  // and 247, 8 of 2000 292 and 280, one of 16384 1.72 and 1.42 ms; 16 of 4000
  // under a window of 512 684 and 775, of 1024 1003 and 999; 64 times 200
  // queries over 1200 keys 326 and 297, 64 times 120 over 1120 167 and 239.  At
  // width 64 one tile was never slower (16 packed prompts, window 1024: 206 and
  // 281; 8 of 2048 185 and 232).  The rule knows the totals only: among many
  // short sequences, or ones without rows, a few long ones get one tile a CTA
  // (one of 8000 and 60 of 200 533 us, 473 with two; 16 of 2000 and 48 empty ones
  // 542 and 520; two of 4000 and 32 of 300 339 and 344).
  constexpr int64_t kFewKeys = 1024;
  const int64_t in_windows = static_cast<int64_t>(a.window) * a.B;
  const int64_t keys = a.window > 0 && in_windows < a.n_k ? in_windows : a.n_k;
  if (D == 64 || a.n_q <= static_cast<int64_t>(kTile) * a.B || keys <= kFewKeys * a.B)
    return launch_dim<D, 1, 2>(a, encode, sms, 1, stream);
  return launch_dim<D, D == 64 ? 1 : 2, D == 64 ? 2 : 1>(a, encode, sms, 1, stream);
}

}  // namespace

cudaError_t launch_prompt_attn(const PromptAttnArgs& a, PFN_cuTensorMapEncodeTiled_v12000 encode, cudaStream_t stream) {
  if (a.B <= 0 || a.n_q <= 0) return cudaSuccess;
  return a.head_dim == 128 ? launch_tiles<128>(a, encode, stream) : launch_tiles<64>(a, encode, stream);
}

}  // namespace csa
