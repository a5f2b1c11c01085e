// Attention of a chunk of new tokens a sequence over its pages of E4M3 codes,
// grouped heads, causal (the chunk's tokens are the sequence's last), optionally
// windowed, with an optional attention sink:
//   l_ij = sm_scale k_scale(page of j) q_i . codes_j,   p_ij = e^(l_ij - m_i)
//   out_i = sum_j p_ij v_scale(page) codes^v_j / (sum_j p_ij + e^(sink - m_i))
// over j <= len - n + i and, with a window W, j > len - n + i - W.
//
// The heads that share a key head are rows of one problem: row r of a key head
// is head r % group of query r / group, so that the keys are read once for all
// of them and few queries fill a tile.  A tile is 256 rows, two halves of 128
// that work in turn on each block of 128 keys, one's softmax under the other's
// products; one of at most 128 rows has its blocks shared out to the two halves,
// whose sums are joined at its end.
//
// The blocks of all tiles form one line that is cut into equal shares, one a
// CTA, whatever the lengths are; a tile that a cut divides is finished by the
// merge kernel from fp32 partial results in a fixed order.
//
// S = Q K^T takes the codes as they are: a query row, scaled by a power of two,
// is the sum of two E4M3 rows (a bf16 value has 8 significant bits, each part
// holds 4), two products at twice the 16-bit rate.  The scales of keys are
// factors of the logits.  The codes of values become f16, exactly, written by
// four warps for the product O += P V; their scales go into the weights, whose
// exponents they shift.  S and O are in tensor memory, P is written over S as
// f16 and read from there.  The softmax has one thread a row, so no value
// crosses threads.
//
// Roles of a CTA's 16 warps: 0..7 the softmax of the two halves, 8..11 queries
// into their two parts and values into f16, 12 the walk along the CTA's share, 13
// the products, 14 keys and scales, 15 values.  The softmax has 200 registers a
// thread (a row's 128 scores and what goes with them, no spills), the converting
// warps 48, the others 64.
//
// What bounds it: at width 128 the products of a block for 256 rows take 2050 cycles
// alone; a block takes some 3500, a half's scores, softmax and product one after the
// other while the other half is half a turn away (tensor pipe 58 % active, 62 % of
// the issue slots used, memory 1 %).  A half's softmax is some 1600 of them, with one
// warp a scheduler at a time.  Code that is not run again at once is fetched at some
// 3 cycles an instruction, so the softmax is rolled where it can be, and so is all
// that runs once a tile.  (2048 tokens at 62000, 32 heads on 4 of width 128: 1638 us,
// 1.32 PFLOP/s counting each product once, 70 % of what a 16-bit library product
// reaches; 12 prompts of up to 1000 tokens behind up to 6000: 554 us; 48 mixed
// sequences of width 64 under a window of 4096: 307 us; 5 tokens after 900: 17 us,
// of which two launches and the chain of loads before the first product are 12.)
// A block of few rows costs what one of 128 does, some 2000 to 2900 cycles: 64
// sequences of 4096 with 64 heads on 8 take 147 us at width 64 and 163 at 128 with
// four new tokens each, 141 and 154 with one (csa_paged_attn 58 and 92).
//
// A masked weight is 0, and 0 * NaN is NaN: in blocks that some row of the tile
// masks, NaN codes of values are taken out as they become f16, and the rows that
// do see such a key get its NaN at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>

#include <type_traits>

#include "gqa.cuh"
#include "ptx.cuh"

namespace csa {
namespace {

constexpr int kTileShift = 7;
constexpr int kTile = 1 << kTileShift;      // rows of a half, keys of a block
constexpr int kTileRows = 2 * kTile;
constexpr int kGroups = kTile / 16;         // groups of 16 keys, whose page is one
constexpr int kThreads = 512;
constexpr int kConvWarp = 8, kWalkWarp = 12, kMmaWarp = 13, kKeyWarp = 14, kValueWarp = 15;
constexpr int kConvThreads = 128;
constexpr int kOrders = 4;                  // tiles that the walking warp may be ahead
// The walking warp waits for whole tiles (2^30 tokens: some 15 s), all others for a
// block at most: what stops is theirs to report, and ends its wait too.
constexpr int kTileWaits = 16;
// A maximum may lag behind by this much (in log2) before the sums are rescaled:
// weights are then at most 2^8 times 1, and as f16 they carry 2^7 more, so that
// weights down to 2^-21 of the largest keep f16's full precision.
constexpr float kLag = 8.f;
constexpr float kWeightExp = 7.f;
// The weights' sum is taken from the weights, value scale in, a group of keys
// at a time.  Where that scale takes weights further down than this, they may
// pass fp32 while e^(l - m) counts: the sum then has exponentials of its own.
constexpr float kFar = -64.f;
constexpr float kLarge = 65536.f;           // a maximum whose half step, 2^-8, may show in a weight
constexpr float kNone = -1e31f;             // running maximum before the first key: below every logit times log2 e
// Blocks that some row of a tile masks: the causal edge of 256 rows crosses at
// most 3, the window's edge 3.
constexpr int kMaxMasked = 8;
// Tiles of up to this many rows have their partial results by rows, which the
// merge adds up with a CTA a row; others by channels, so that the threads of a
// warp, a row each, store neighbouring words.
constexpr int kFewRows = 64;
// What a tile costs, in the units of the shares: a block for two halves, for
// one, and the tile itself: its queries, its outputs and the pipeline that runs
// empty between it and the next.  The tile's 16 were found by timing, not from its
// some 7500 cycles, which are 6 or 7 units: with 4, 8, 12, 16 and 24, 12 prompts of
// width 128 take 636, 581, 552, 555 and 561 us, of width 64 479, 475, 477, 482 and
// 491; 48 mixed sequences of width 64 299, 301, 303, 306 and 312, of width 128 361,
// 351, 350, 353 and 357; 30 prompts of up to 300 111, 105, 104, 103 and 105.
constexpr int kCostTwo = 3, kCostOne = 2, kCostTile = 16;

// Registers a thread: 512 threads are launched with 128 each.
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 200, kConvRegs = 48, kOtherRegs = 64;
static_assert(2 * kSoftmaxRegs + kConvRegs + kOtherRegs <= 4 * kLaunchRegs, "registers of the block");

template <int D>
struct Cfg {
  static constexpr int kQBytes = kTile * D * 2;     // of a half: two E4M3 parts
  static constexpr int kCodeBytes = kTile * D;      // of a block's keys or values
  static constexpr int kVBytes = kTile * D * 2;     // of a block's values as f16
  static constexpr int kKStages = D == 128 ? 3 : 6;
  static constexpr int kRawStages = D == 128 ? 2 : 4;
  static constexpr int kVStages = 2;
  static constexpr int kMeta = 2 * kKStages;
  static constexpr int kSearch = kThreads * 12;     // of the sequences' costs, at the start
  static constexpr int kSmem =
      2 * kQBytes + kKStages * kCodeBytes + kRawStages * kCodeBytes + kVStages * kVBytes + kSearch + 1024;
  static constexpr int kSCol(int t) { return t * kTile; }
  static constexpr int kOCol(int t) { return 2 * kTile + t * D; }
  static constexpr int kCols = 512;
  static constexpr int64_t kRecord = static_cast<int64_t>(kTileRows) * (D + 4);  // floats of a partial result
};

// A tile that a share's end divides, for the merge.
struct __align__(16) Cut {
  int32_t q0, row0, head0, rows;  // rows 0: no such tile
  int32_t first, last, pad0, pad1;
};

struct Seq {
  int q0, n, len;  // rows of q from q0 on, cached tokens
};
// A sequence as its arrays have it: n is 0 where its offsets are wrong.
__device__ __forceinline__ Seq read_seq(const ChunkAttnArgs& a, int b) {
  const int32_t q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + b + 1);
  const int64_t len = __ldg(a.lens + b), cap = a.cache.table_stride << a.cache.page_shift;
  Seq s;
  s.q0 = q0;
  s.n = q1 - q0;
  if (q0 < 0 || q1 < q0 || q1 > a.n_q) {
    record_error(a.status, kErrIndexRange);
    s.q0 = s.n = 0;
  }
  if (len > cap) record_error(a.status, kErrIndexRange);
  s.len = static_cast<int>(len < 0 ? 0 : len > cap ? cap : len);
  return s;
}

// A tile of a sequence: its rows (of one key head) and the keys they see.
struct Tile {
  int rows, lo, hi;  // keys [lo, hi)
  int j_hi, blocks;  // blocks j_hi - 1 downwards; one at least
  __device__ __forceinline__ int unit() const { return rows > kTile ? kCostTwo : kCostOne; }
  __device__ __forceinline__ int cost() const { return kCostTile + unit() * blocks; }  // (blocks: below 2^23)
};
__device__ __noinline__ Tile tile_of(const Seq& s, int group, int window, int t) {
  Tile x;
  const uint32_t row0 = static_cast<uint32_t>(t) * kTileRows, all = static_cast<uint32_t>(s.n) * group;
  x.rows = static_cast<int>(min(all - row0, static_cast<uint32_t>(kTileRows)));
  const int shift = s.len - s.n;  // (lengths and rows are below 2^30 and 2^27: no overflow)
  const int first = shift + static_cast<int>(row0 / group);
  const int last = shift + static_cast<int>((row0 + x.rows - 1) / group);
  x.hi = last + 1;
  x.lo = window > 0 && first >= window ? first - window + 1 : 0;
  if (x.hi <= 0) x.hi = x.lo = 0;
  x.j_hi = x.hi > 0 ? (x.hi + kTile - 1) >> kTileShift : 1;
  x.blocks = x.j_hi - (x.lo >> kTileShift);
  return x;
}
__device__ __forceinline__ int tiles_of(const Seq& s, int group) {
  return static_cast<int>((static_cast<uint32_t>(s.n) * group + kTileRows - 1) / kTileRows);
}

// What a warp of a CTA has to know of a tile that it works on.
struct Order {
  int there;                    // 0: no more
  int b, q0, row0, rows, head0, kv_head;
  int shift;                    // query i stands at key i + shift
  int lo, hi, from, upto;       // the tile's keys; its masked blocks: from `from` on, and up to `upto`
  int j_top, blocks;            // this share's blocks: j_top downwards
  int split;                    // the halves share out the blocks
  int record;                   // -1: the tile is whole, else which of the share's records takes it
  __device__ __forceinline__ bool masked(int j) const { return j >= from || j <= upto; }
};

// Asks for a tile of a tensor map in L2.
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(c0), "r"(c1),
               "r"(c2)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The nearest E4M3 codes of four f16 values, the first in the low byte.
__device__ __forceinline__ uint32_t f16x4_to_e4m3(uint32_t xy, uint32_t zw) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f16x2 l, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "r"(xy), "r"(zw));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t x, uint32_t y) {
  const __half2 z = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&z);
}
// Non-zero where a byte is a NaN code (magnitude 0x7F, which carries into the
// byte's top bit).
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Keeps what is computed from r behind the wait for its load.
__device__ __forceinline__ void landed(uint32_t (&r)[32]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               :);
}

__device__ __forceinline__ void landed(uint32_t (&r)[16]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               :);
}

// x, as something that the compiler cannot move out of a loop: it would copy the
// loop for each value (the loading warps' loop had 25 KB of code, the product
// warp's as much), and the kernel's hot code has to fit the instruction caches.
__device__ __forceinline__ bool here(bool x) {
  uint32_t y = x ? 1u : 0u;
  asm volatile("" : "+r"(y));
  return y != 0u;
}

// wait_or_abort in few instructions, its limit (ns) in shared memory: with all
// waits in full and all loops unrolled the kernel's code was 160 KB, and the
// softmax waited for its instructions.
struct Watch {
  volatile int abort;
  uint32_t limit;
  unsigned* status;
};
__device__ __forceinline__ uint32_t timer_low() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool await(uint64_t* bar, uint32_t parity, Watch* w) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = timer_low();
  while (w->abort == 0) {
    if (mbar_try_wait(bar, parity)) return true;
    if (timer_low() - t0 > w->limit) {
      record_error(w->status, kErrTimeout);
      w->abort = 1;
    }
  }
  return false;
}
// The same for up to kTileWaits limits.
__device__ __noinline__ bool await_tile(uint64_t* bar, uint32_t parity, Watch* w) {
  uint32_t t0 = timer_low();
  int limits = kTileWaits;
  while (w->abort == 0) {
    if (mbar_try_wait(bar, parity)) return true;
    if (timer_low() - t0 <= w->limit) continue;
    t0 = timer_low();
    if (--limits > 0) continue;
    record_error(w->status, kErrTimeout);
    w->abort = 1;
  }
  return false;
}

// What every CTA finds out first: its share of the line, and where it begins.
struct Start {
  int64_t per, total, offset;  // offset: units of sequence b before the share's first
  int64_t per_head;            // units of a key head of it
  Seq s;
  int b;
};

// The cost of a sequence's tiles of one key head, by a whole warp.
__device__ __noinline__ int64_t head_cost(const Seq& s, int group, int window) {
  const int tiles = tiles_of(s, group);
  int64_t sum = 0;
#pragma unroll 1
  for (int t = threadIdx.x & 31; t < tiles; t += 32) sum += tile_of(s, group, window, t).cost();
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  return sum;
}

// (64-bit divisions are long: one copy for all)
__device__ __noinline__ int64_t quotient(int64_t x, int64_t y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// What share each CTA has of `total` units.  (A share holds a block at least, so
// that no CTA between a tile's first and last has none.)
__device__ __forceinline__ int64_t share_of(int64_t total) {
  return max(quotient(total + gridDim.x - 1, gridDim.x), static_cast<int64_t>(kCostTwo));
}

// The largest of the lanes' values up to this one, and their sum.
__device__ __forceinline__ int max_upto(int x) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if ((threadIdx.x & 31) >= off) x = max(x, y);
  }
  return x;
}
__device__ __forceinline__ int64_t sum_upto(int64_t x) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
    if ((threadIdx.x & 31) >= off) x += y;
  }
  return x;
}

// The start of a CTA's share among at most 32 sequences, by one warp.
constexpr int kFewSeqs = 32;
__device__ __forceinline__ Start find_start(const ChunkAttnArgs& a, int group) {
  const int lane = threadIdx.x & 31;
  Seq s = {0, 0, 0};
  if (lane < a.B) s = read_seq(a, lane);
  const int top = __shfl_up_sync(0xffffffffu, max_upto(s.q0 + s.n), 1);
  if (lane > 0 && s.q0 < top) s.n = 0;  // offsets that fall: rows that an earlier sequence has
  const int tiles = tiles_of(s, group);
  int64_t per_head = 0;
#pragma unroll 1
  for (int t = 0; t < min(tiles, 2); ++t) per_head += tile_of(s, group, a.window, t).cost();
#pragma unroll 1
  for (unsigned more = __ballot_sync(0xffffffffu, tiles > 2); more; more &= more - 1) {
    const int from = __ffs(more) - 1;
    Seq x;
    x.q0 = 0;
    x.n = __shfl_sync(0xffffffffu, s.n, from);
    x.len = __shfl_sync(0xffffffffu, s.len, from);
    const int64_t c = head_cost(x, group, a.window);
    if (lane == from) per_head = c;
  }
  const int64_t n = per_head * a.cache.n_kv_heads, upto = sum_upto(n);
  Start st;
  st.total = __shfl_sync(0xffffffffu, upto, 31);
  st.per = share_of(st.total);
  const int64_t target = blockIdx.x * st.per;
  const unsigned in = __ballot_sync(0xffffffffu, target < upto);
  st.b = in ? __ffs(in) - 1 : -1;
  const int from = max(st.b, 0);
  st.offset = target - __shfl_sync(0xffffffffu, upto - n, from);
  st.per_head = __shfl_sync(0xffffffffu, per_head, from);
  st.s.q0 = __shfl_sync(0xffffffffu, s.q0, from);
  st.s.n = __shfl_sync(0xffffffffu, s.n, from);
  st.s.len = __shfl_sync(0xffffffffu, s.len, from);
  return st;
}

// Walks the tiles of a share; one warp.
struct Walker {
  Seq s;
  int b, top, head, t, tiles;
  int x0;                 // units of the tile before the share
  int64_t left, tile_at;  // units to go, the tile's place on the line
  Tile tile;

  // The sequence from b on that has rows; false: none.
  __device__ __noinline__ bool seek(const ChunkAttnArgs& a) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (; b < a.B; b += 32) {
      Seq mine = {0, 0, 0};
      if (b + lane < a.B) mine = read_seq(a, b + lane);
      int before = mine.q0 + mine.n;  // the largest end so far, this sequence's not counted
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, off);
        if (lane >= off) before = max(before, y);
      }
      const int through = __shfl_sync(0xffffffffu, before, 31);
      before = __shfl_up_sync(0xffffffffu, before, 1);
      before = lane == 0 ? top : max(before, top);
      const unsigned ok = __ballot_sync(0xffffffffu, mine.n > 0 && mine.q0 >= before);
      if (ok) {
        const int from = __ffs(ok) - 1;
        s.q0 = __shfl_sync(0xffffffffu, mine.q0, from);
        s.n = __shfl_sync(0xffffffffu, mine.n, from);
        s.len = __shfl_sync(0xffffffffu, mine.len, from);
        top = s.q0 + s.n;
        b += from;
        return true;
      }
      top = max(top, through);
    }
    return false;
  }

  // To the share's first tile.
  __device__ __forceinline__ bool begin(const ChunkAttnArgs& a, const Start& st, int group) {
    left = min(st.per, st.total - blockIdx.x * st.per);
    if (left <= 0) return false;
    b = st.b;
    s = st.s;
    top = s.q0 + s.n;
    tiles = tiles_of(s, group);
    const int lane = threadIdx.x & 31;
    head = static_cast<int>(quotient(st.offset, st.per_head));
    int64_t at = st.offset - head * st.per_head;  // units of the head's tiles before the share
#pragma unroll 1
    for (t = 0; t < tiles; t += 32) {  // the tile that it begins in
      const int64_t c = t + lane < tiles ? tile_of(s, group, a.window, t + lane).cost() : 0;
      int64_t x = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      const unsigned in = __ballot_sync(0xffffffffu, x > at);
      if (in) {
        const int from = __ffs(in) - 1;
        at -= __shfl_sync(0xffffffffu, x - c, from);
        t += from;
        break;
      }
      at -= __shfl_sync(0xffffffffu, x, 31);
    }
    tile = tile_of(s, group, a.window, t);
    x0 = static_cast<int>(at);
    tile_at = blockIdx.x * st.per - x0;
    return true;
  }

  // To the next tile, whose units before the share are none.
  __device__ __forceinline__ bool next(const ChunkAttnArgs& a, int group) {
    tile_at += tile.cost();
    x0 = 0;
    if (++t == tiles) {
      t = 0;
      if (++head == a.cache.n_kv_heads) {
        head = 0;
        ++b;
        if (!seek(a)) return false;
        tiles = tiles_of(s, group);
      }
    }
    tile = tile_of(s, group, a.window, t);
    return true;
  }
};

// The block, counted from the tile's first, at or behind place x of a tile.
__device__ __forceinline__ int block_at(const Tile& t, int x) {
  const int y = max(x - kCostTile, 0);
  return t.rows > kTile ? (y + kCostTwo - 1) / kCostTwo : (y + kCostOne - 1) / kCostOne;
}
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const ChunkAttnArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t order_full[kOrders], order_empty[kOrders], q_full[2], q_empty;
  __shared__ uint64_t k_full[C::kKStages], k_empty[C::kKStages], raw_full[C::kRawStages], raw_empty[C::kRawStages];
  __shared__ uint64_t v_full[C::kVStages], v_empty[C::kVStages], meta_full[C::kMeta];
  __shared__ uint64_t s_full[2], p_full[2], o_full[2], joined, left_off, drain;
  __shared__ Order orders[kOrders];
  __shared__ __align__(16) float k_scale_s[C::kMeta][kGroups], v_log_s[C::kMeta][kGroups];
  __shared__ float v_min_s[C::kMeta];          // the least of the block's value scales, in log2
  __shared__ uint32_t bad_s[C::kMeta];         // groups whose page is outside the pool
  __shared__ float q_scale_s[2][kTile];
  __shared__ float m_s[2][kTile], d_s[2][kTile], l_s[2][kTile];
  // keys of masked blocks whose values had NaN codes, as each converting warp
  // found them, of three tiles (who converts for tile n + 2 knows that every warp
  // has begun tile n): those of tile number n are valid if odd_item[n % 3] is n + 1
  __shared__ uint32_t odd_rows[3][4][kMaxMasked][4];
  __shared__ int odd_block[3][4][kMaxMasked], odd_item[3][4];
  __shared__ uint32_t tmem_slot;
  __shared__ Watch watch;
  __shared__ int64_t sum_sh[kThreads / 32];
  __shared__ int max_sh[kThreads / 32];
  __shared__ Start start_s;
  __shared__ int n_long;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* q_s = smem;
  uint8_t* k_ring = q_s + 2 * C::kQBytes;
  uint8_t* v_ring = k_ring + C::kKStages * C::kCodeBytes;
  uint8_t* raw_ring = v_ring + C::kVStages * C::kVBytes;
  int64_t* cost_s = reinterpret_cast<int64_t*>(raw_ring + C::kRawStages * C::kCodeBytes);
  int* long_s = reinterpret_cast<int*>(cost_s + kThreads);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = a.n_heads / a.cache.n_kv_heads;
  // the barriers, a thread a kind
  auto init = [&](int who, uint64_t* bars, int n, uint32_t count) {
    if (tid == 32 * who)
#pragma unroll 1
      for (int i = 0; i < n; ++i) mbar_init(bars + i, count);
  };
  init(0, order_full, kOrders, 1);
  init(1, order_empty, kOrders, kThreads / 32 - 1);
  init(2, q_full, 2, kConvThreads);
  init(2, &q_empty, 1, kTileRows + 1);
  init(3, k_full, C::kKStages, 1);
  init(4, k_empty, C::kKStages, 1);
  init(5, raw_full, C::kRawStages, 1);
  init(6, raw_empty, C::kRawStages, kConvThreads);
  init(7, v_full, C::kVStages, kConvThreads);
  init(7, v_empty, C::kVStages, 1);
  init(8, meta_full, C::kMeta, 1);
  init(9, s_full, 2, 1);
  init(9, p_full, 2, kTile);
  init(10, o_full, 2, 1);
  init(10, &joined, 1, kTileRows);
  init(10, &left_off, 1, kTileRows);
  init(10, &drain, 1, 1);
  if (lane == 0 && warp <= 10) fence_mbar_init();
  if (tid == 32 * 11) {
    watch.abort = 0;
    watch.limit = static_cast<uint32_t>(min(wait_limit_ns(a.status), static_cast<uint64_t>(4000000000u)));
    watch.status = a.status;
    start_s.b = -1;
    n_long = 0;
  }
  if (tid < 12) odd_item[tid >> 2][tid & 3] = 0;
  if (warp == kKeyWarp && lane == 0) prefetch_tensormap(&tm_k);
  if (warp == kValueWarp && lane == 0) prefetch_tensormap(&tm_v);
  // Tensor memory is taken after the kernel before has ended and before the
  // one after may start: no CTA of either can then hold what this one, or
  // what it waits for, still needs.
  pdl_wait();
  if (warp == kMmaWarp) tmem_alloc(&tmem_slot, C::kCols);

  // ---------------- the CTA's share ----------------
  // Prefix sums of the sequences' costs; more than a block of sequences takes a
  // pass for the total first.  Up to kFewSeqs the walking warp finds it by itself
  // (one sequence, 5 tokens after 900: 19.3 us, 18.1 so).
  if (a.B > kFewSeqs) {
    int64_t per = 1, total = 0;
#pragma unroll 1
    for (int pass = a.B > kThreads ? 0 : 1; pass < 2; ++pass) {
      int64_t base = 0;
      int top = 0;  // rows of q that sequences so far reach
#pragma unroll 1
      for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        Seq s = {0, 0, 0};
        if (b < a.B) s = read_seq(a, b);
        const int end = max_upto(s.q0 + s.n);
        if (lane == 31) max_sh[warp] = end;
        __syncthreads();
        int before_top = __shfl_up_sync(0xffffffffu, end, 1), through = top;
        before_top = lane == 0 ? top : max(before_top, top);
#pragma unroll 4
        for (int k = 0; k < kThreads / 32; ++k) {
          const int y = max_sh[k];
          if (k < warp) before_top = max(before_top, y);
          through = max(through, y);
        }
        top = through;
        if (s.q0 < before_top) s.n = 0;  // offsets that fall: rows that an earlier sequence has
        // Sequences of one tile or two are a thread's own, the others a warp's each.
        const int tiles = tiles_of(s, group);
        int64_t n = 0;
        if (tiles > 2) {
          long_s[atomicAdd(&n_long, 1)] = tid;
        } else {
#pragma unroll 1
          for (int t = 0; t < tiles; ++t) n += tile_of(s, group, a.window, t).cost();
        }
        __syncthreads();
#pragma unroll 1
        for (int i = warp; i < n_long; i += kThreads / 32) {
          const int64_t c = head_cost(read_seq(a, b0 + long_s[i]), group, a.window);
          if (lane == 0) cost_s[long_s[i]] = c;
        }
        __syncthreads();
        if (tiles > 2) n = cost_s[tid];
        if (tid == 0) n_long = 0;
        const int64_t per_head = n;
        n *= a.cache.n_kv_heads;
        const int64_t x = sum_upto(n);
        if (lane == 31) sum_sh[warp] = x;
        __syncthreads();
        int64_t before = base + x - n;
#pragma unroll 4
        for (int k = 0; k < kThreads / 32; ++k) {
          const int64_t y = sum_sh[k];
          if (k < warp) before += y;
          base += y;
        }
        if (a.B <= kThreads) total = base;
        if (pass == 1) {
          per = share_of(total);
          const int64_t target = blockIdx.x * per;
          if (target >= before && target < before + n) {  // one thread at most
            start_s.b = b;
            start_s.offset = target - before;
            start_s.per_head = per_head;
            start_s.s = s;
          }
        }
        __syncthreads();
      }
      total = base;
    }
    if (tid == 0) {
      start_s.per = per;
      start_s.total = total;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = tmem_slot;

  // the next tile, of every warp but the walking one (read where it lies, until
  // `done` with it); false at the end and after an abort
  auto take = [&](int item) {
    const bool ok = await(order_full + item % kOrders, (item / kOrders) & 1, &watch);
    return __all_sync(0xffffffffu, ok) && orders[item % kOrders].there != 0;
  };
  auto done = [&](int item) {
    __syncwarp();
    if (lane == 0) mbar_arrive(order_empty + item % kOrders);
  };

  if (warp >= kWalkWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kWalkWarp) {
      // ---------------- the tiles of the share ----------------
      Walker w;
      const Start st = a.B > kFewSeqs ? start_s : find_start(a, group);
      bool there = st.b >= 0 && w.begin(a, st, group), ok = true;
      Cut cut = {};
#pragma unroll 1
      for (int item = 0; ok; ++item) {
        Order o = {};
        while (there) {
          const int x1 = static_cast<int>(min(static_cast<int64_t>(w.tile.cost()), w.x0 + w.left));
          const int k0 = block_at(w.tile, w.x0), k1 = block_at(w.tile, x1);
          const bool last_one = x1 - w.x0 == w.left;
          if (k1 > k0) {
            const Tile& t = w.tile;
            o.there = 1;
            o.b = w.b;
            o.q0 = w.s.q0;
            o.row0 = w.t * kTileRows;
            o.rows = t.rows;
            o.kv_head = w.head;
            o.head0 = w.head * group;
            o.shift = w.s.len - w.s.n;
            o.lo = t.lo;
            o.hi = t.hi;
            const int first = o.shift + static_cast<int>(static_cast<uint32_t>(o.row0) / group);
            const int last = o.shift + static_cast<int>(static_cast<uint32_t>(o.row0 + o.rows - 1) / group);
            o.from = first < 0 ? 0 : (first + 1) >> kTileShift;
            o.upto = a.window > 0 && last >= a.window ? (last - a.window) >> kTileShift : -1;
            o.j_top = t.j_hi - 1 - k0;
            o.blocks = k1 - k0;
            o.split = t.rows <= kTile;
            o.record = k0 == 0 && k1 == t.blocks ? -1 : k0 == 0 ? 1 : 0;
            if (o.record == 1) {
              cut.q0 = o.q0;
              cut.row0 = o.row0;
              cut.head0 = o.head0;
              cut.rows = o.rows;
              cut.first = blockIdx.x;
              cut.last = static_cast<int>(quotient(w.tile_at + kCostTile + t.unit() * (t.blocks - 1), st.per));
            }
          }
          w.left -= x1 - w.x0;
          there = !last_one && w.next(a, group);
          if (o.there) break;
        }
        if (lane == 0) {
          if (item >= kOrders)
            ok = await_tile(order_empty + item % kOrders, (item / kOrders - 1) & 1, &watch);
          if (ok) {
            orders[item % kOrders] = o;
            mbar_arrive(order_full + item % kOrders);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!o.there) break;
      }
      if (lane == 0) reinterpret_cast<Cut*>(a.part)[blockIdx.x] = cut;
    } else if (warp != kMmaWarp) {
      // ---------------- loads: a warp for keys and scales, one for values ----------------
      const bool keys = warp == kKeyWarp;
      const CUtensorMap* tm = keys ? &tm_k : &tm_v;
      uint64_t* full = keys ? k_full : raw_full;
      uint64_t* empty = keys ? k_empty : raw_empty;
      uint8_t* ring = keys ? k_ring : raw_ring;
      const int stages = keys ? C::kKStages : C::kRawStages;
      const int ps = a.cache.page_shift, g = lane & 7;
      int n = 0, slot = 0, meta = 0;  // blocks so far, their places
      uint32_t parity = 1;            // of the phase before the slot's
      bool ok = true;
#pragma unroll 1
      for (int item = 0; ok && take(item); ++item) {
        const Order& o = orders[item % kOrders];
        const int blocks = o.blocks, j_top = o.j_top, lo = o.lo, hi = o.hi, kv_head = o.kv_head;
        // a lane looks after a group of 16 keys of one of four blocks; their pages
        // are read eight blocks ahead, and their contents asked for four ahead
        const int32_t* row = a.cache.table + static_cast<int64_t>(o.b) * a.cache.table_stride;
        constexpr int32_t kNotNeeded = INT32_MIN;
        auto entry = [&](int q0) -> int32_t {
          const int q = q0 + (lane >> 3), t = (j_top - q) * kTile + 16 * g, p0 = (t >> ps) << ps;
          if (q >= blocks || p0 >= hi || p0 + a.cache.page <= lo) return kNotNeeded;
          return max(__ldg(row + (t >> ps)), -1);
        };
        auto in_pool = [&](int32_t page) { return page >= 0 && page < a.cache.n_pages; };
        auto scale = [&](int32_t page, const float* of, float none) {
          return here(keys) && in_pool(page) ? __ldg(of + static_cast<int64_t>(page) * a.cache.n_kv_heads + kv_head) : none;
        };
        const bool first_of_page = ((16 * g) & (a.cache.page - 1)) == 0;
        int32_t page = entry(0), next = entry(4);
        float ks = scale(page, a.cache.k_scale, 1.f), vs = scale(page, a.cache.v_scale, 0.f);
#pragma unroll 1
        for (int q0 = 0; q0 < blocks && ok; q0 += 4) {
          const int32_t after = entry(q0 + 8);
          if (in_pool(next) && first_of_page) tma_prefetch_3d(tm, 0, kv_head << ps, next);
          const float ks_next = scale(next, a.cache.k_scale, 1.f), vs_next = scale(next, a.cache.v_scale, 0.f);
          const bool in = in_pool(page);
          const unsigned bads = __ballot_sync(0xffffffffu, page != kNotNeeded && !in);
          if (bads && here(keys)) record_error(a.status, kErrIndexRange);
          const float lv = in ? __log2f(vs) : 1e30f;
          float least = lv;
#pragma unroll
          for (int off = 1; off < 8; off <<= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, off));
          const unsigned copies = __ballot_sync(0xffffffffu, in && first_of_page);
          const int n_q = min(4, blocks - q0);
#pragma unroll 1
          for (int i = 0; i < n_q; ++i) {
            const bool mine = (lane >> 3) == i;
            if (n >= stages) ok = __all_sync(0xffffffffu, await(empty + slot, parity, &watch));
            if (!ok) break;
            if (here(keys)) {
              if (mine) {
                k_scale_s[meta][g] = ks;
                v_log_s[meta][g] = lv;
                if (g == 0) {
                  v_min_s[meta] = least;
                  bad_s[meta] = (bads >> (8 * i)) & 0xFFu;
                }
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(meta_full + meta);
              meta = meta + 1 == C::kMeta ? 0 : meta + 1;
            }
            if (lane == 0)
              mbar_arrive_expect_tx(full + slot, __popc(copies & (0xFFu << (8 * i))) * a.cache.page * D);
            __syncwarp();
            if (mine && in && first_of_page)
              tma_load_3d(ring + slot * C::kCodeBytes + 16 * g * D, tm, 0, kv_head << ps, page, full + slot);
            ++n;
            if (++slot == stages) {
              slot = 0;
              parity ^= 1u;
            }
          }
          page = next;
          next = after;
          ks = ks_next;
          vs = vs_next;
        }
        if (!ok) break;
        done(item);
      }
      if (lane == 0)  // every copy lands before the CTA ends (also after an abort)
#pragma unroll 1
        for (int k = max(0, n - stages); k < n; ++k) mbar_wait(full + k % stages, (k / stages) & 1, a.status);
      __syncwarp();
    } else {
      // ---------------- products ----------------
      // (the whole warp walks the loop and one elected lane issues, so that the
      // loop's values are uniform)
      constexpr uint32_t idesc_s = instr_desc(kTile, kTile, 0, 0, 0, 0);  // E4M3, K-major A and B
      constexpr uint32_t idesc_o = instr_desc(kTile, D, 0, 0, 0, 1);     // f16, A from TMEM, B (= V) MN-major
      // A descriptor's upper half is the same for all operands of a kind; its lower
      // half is the address, for values the distance of their channel blocks too.
      constexpr uint32_t kLineHi = static_cast<uint32_t>(1024 >> 4) | 1u << 14 | kSwizzle128B << 29;
      constexpr uint32_t kKeyHi = D == 128 ? kLineHi : static_cast<uint32_t>(512 >> 4) | 1u << 14 | kSwizzle64B << 29;
      constexpr uint32_t kValueLo = static_cast<uint32_t>(kTile * 128 >> 4) << 16;
      auto uniform = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
      auto desc = [](uint32_t hi, uint32_t lo) { return static_cast<uint64_t>(hi) << 32 | lo; };
      const uint32_t tm = uniform(tmem), q_lo = uniform(smem_u32(q_s) >> 4);
      const uint32_t k_lo = uniform(smem_u32(k_ring) >> 4), v_lo = uniform(smem_u32(v_ring) >> 4 | kValueLo);
      const bool skip_s = test_fault(a.status, kFaultAttn);  // test fault: S is never announced
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
               __all_sync(0xffffffffu, await(bar, parity, &watch));
      };
      // S of half t with the queries of half qs and the keys at slot (one lane)
      auto s_of = [&](int t, int qs, uint32_t slot) {
        const uint32_t kl = k_lo + slot * (C::kCodeBytes >> 4), ql = q_lo + qs * (C::kQBytes >> 4);
        // the high parts' products, then the low ones': at width 64 both parts
        // are in one 128-byte line
        constexpr int kLow = D == 128 ? kTile * 128 >> 4 : 64 >> 4;
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int s = 0; s < D / 32; ++s)
            mma_f8(tm + C::kSCol(t), desc(kLineHi, ql + part * kLow + 2 * s), desc(kKeyHi, kl + 2 * s), idesc_s,
                   part + s > 0 ? 1u : 0u);
        if (!skip_s) tc_commit(s_full + t);
      };
      auto pv_of = [&](int t, uint32_t slot, bool add) {
        const uint32_t vl = v_lo + slot * (C::kVBytes >> 4);
#pragma unroll
        for (int s = 0; s < kTile / 16; ++s)
          mma_f16_ts(tm + C::kOCol(t), tm + C::kSCol(t) + s * 8, desc(kLineHi, vl + (16 * s * 128 >> 4)), idesc_o,
                     s > 0 ? 1u : add ? 1u : 0u);
      };
      bool ok = true;
      uint32_t k_slot = 0, k_parity = 0, v_slot = 0, v_parity = 0, p_parity = 0;  // (p_parity: a bit a half)
      auto next_k = [&]() {
        if (++k_slot == C::kKStages) {
          k_slot = 0;
          k_parity ^= 1u;
        }
      };
      auto next_v = [&]() {
        if (++v_slot == C::kVStages) {
          v_slot = 0;
          v_parity ^= 1u;
        }
      };
#pragma unroll 1
      for (int item = 0; ok && take(item); ++item) {
        // The halves take turns, a step each: all blocks each, or, where they share
        // them out, a block a step with the queries of the first half.
        const bool split = uniform(orders[item % kOrders].split) != 0;
        const int steps = static_cast<int>(uniform(orders[item % kOrders].blocks)) << (split ? 0 : 1);
        done(item);
#pragma unroll 1
        for (int t = 0; t < 2 && ok; ++t) {
          ok = wait(q_full + t, item & 1);
          if (t >= steps) {  // (only now: the next queries would pass the phase)
            if (elect_one()) tc_commit(&q_empty);
            break;
          }
          if (ok && (here(split) || t == 0)) ok = wait(k_full + k_slot, k_parity);
          tc_fence_after();
          if (ok && elect_one()) {
            s_of(t, here(split) ? 0 : t, k_slot);
            if (here(split) || t == 1) tc_commit(k_empty + k_slot);
            if (t == 1 && steps == 2) tc_commit(&q_empty);
          }
          __syncwarp();
          if (here(split) || t == 1) next_k();
        }
#pragma unroll 1
        for (int i = 0; i < steps && ok; ++i) {
          const int t = i & 1;
          const bool again = i + 2 < steps, last_of_block = here(split) || t == 1;
          if (here(split) || t == 0) {
            ok = wait(v_full + v_slot, v_parity);
            if (ok && again) ok = wait(k_full + k_slot, k_parity);
          }
          if (ok) ok = wait(p_full + t, p_parity >> t & 1u);
          if (!ok) break;
          p_parity ^= 1u << t;
          tc_fence_after();
          if (elect_one()) {
            pv_of(t, v_slot, i >= 2);
            if (!again) tc_commit(o_full + t);
            if (last_of_block) tc_commit(v_empty + v_slot);
            if (again) {
              s_of(t, here(split) ? 0 : t, k_slot);
              if (last_of_block) tc_commit(k_empty + k_slot);
              if (i + 3 == steps) tc_commit(&q_empty);
            }
          }
          __syncwarp();
          if (last_of_block) {
            next_v();
            if (again) next_k();
          }
        }
      }
      // whatever was issued finishes before TMEM and shared memory are released
      if (elect_one()) {
        tc_commit(&drain);
        mbar_wait(&drain, 0, a.status);
      }
      __syncwarp();
    }
  } else if (warp >= kConvWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    // ---------------- queries into two parts, values into f16 ----------------
    constexpr int kChunks = D / 16;               // 16-channel chunks a row
    constexpr int kRowsAtOnce = kConvThreads / kChunks;
    // (at width 64 two chunks at a time: 48 mixed sequences 316 us, 306 so; at width
    // 128 12 prompts 570 us, 595 so)
    constexpr int kFlight = D == 128 ? 4 : 2;
    const int ct = tid - kConvWarp * 32, cw = warp - kConvWarp;
    const int r0 = ct / kChunks, c = ct % kChunks;
    const float scale2 = a.sm_scale * kLog2e;
    int n0 = 0;
    bool ok = true;
#pragma unroll 1
    for (int item = 0; ok && take(item); ++item) {
      const Order& o = orders[item % kOrders];
      if (item > 0) ok = __all_sync(0xffffffffu, await(&q_empty, (item - 1) & 1, &watch));
      if (!ok) break;
      // a thread's 16 channels of its rows are copied to where their two parts
      // will be, and turned into these in place
      auto q_at = [&](int h, int r, int part) {
        uint8_t* line = q_s + h * C::kQBytes + r * 128;
        return D == 128 ? line + part * (kTile * 128) + ((c ^ (r & 7)) << 4) : line + (((c + 4 * part) ^ (r & 7)) << 4);
      };
      const int halves = o.split ? 1 : 2, step_q = kRowsAtOnce / group, step_h = kRowsAtOnce - step_q * group;
      {
        const uint32_t at = static_cast<uint32_t>(o.row0 + r0);
        const int qi = static_cast<int>(at / group);
        int hd = static_cast<int>(at - static_cast<uint32_t>(qi) * group), left = o.rows - r0;
        const uint16_t* src = a.q + static_cast<int64_t>(o.q0 + qi) * a.q_stride + (o.head0 + hd) * a.q_stride_h + c * 16;
        const int64_t step = step_q * a.q_stride + step_h * a.q_stride_h, wrap = a.q_stride - group * a.q_stride_h;
        uint8_t* to = q_at(0, r0, 0);
        const int apart = static_cast<int>(q_at(0, r0, 1) - to);
#pragma unroll 1
        for (int h = 0; h < halves; ++h) {
#pragma unroll 2
          for (int k = 0; k < kChunks; ++k) {
            if (left > 0) {
              cp_async_16(to, src);
              cp_async_16(to + apart, src + 8);
            }
            to += kRowsAtOnce * 128;  // (rows 8 apart and more have their chunks in the same places)
            left -= kRowsAtOnce;
            hd += step_h;
            src += step;
            if (hd >= group) {
              hd -= group;
              src += wrap;
            }
          }
          to += C::kQBytes - kTile * 128;
          cp_async_commit();
        }
      }
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        if (h < halves) {
          cp_async_wait_pending(halves - 1 - h);
          // (rows past the tile's keep what was there: nothing of theirs is used)
          const int n_rows = min(o.rows - h * kTile, kTile);
#pragma unroll 1
          for (int k = 0; k * kRowsAtOnce < n_rows; ++k) {
            const int r = r0 + k * kRowsAtOnce;
            uint4* part[2] = {reinterpret_cast<uint4*>(q_at(h, r, 0)), reinterpret_cast<uint4*>(q_at(h, r, 1))};
            const uint4 u = *part[0], v = *part[1];
            const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
            // the largest magnitude, two at a time as whole numbers (past 0x7F7F: not finite)
            uint32_t both = 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j) both = __vmaxu2(both, w[j] & 0x7FFF7FFFu);
#pragma unroll
            for (int off = 1; off < kChunks; off <<= 1) both = __vmaxu2(both, __shfl_xor_sync(0xffffffffu, both, off));
            const uint32_t top = max(both & 0xFFFFu, both >> 16);
            const bool finite = top < 0x7F80u;
            const int e = min(7 - (static_cast<int>(top >> 7) - 127), 126);
            const float up = finite ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : 0.f;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // (exact in f16 but for what is below both parts)
              const uint32_t y01 = pack_f16(__uint_as_float(w[2 * j] << 16) * up, __uint_as_float(w[2 * j] & 0xFFFF0000u) * up);
              const uint32_t y23 =
                  pack_f16(__uint_as_float(w[2 * j + 1] << 16) * up, __uint_as_float(w[2 * j + 1] & 0xFFFF0000u) * up);
              hi[j] = f16x4_to_e4m3(y01, y23);
              uint32_t h01, h23;
              e4m3x4_to_f16(hi[j], h01, h23);
              lo[j] = f16x4_to_e4m3(sub_f16x2(y01, h01), sub_f16x2(y23, h23));
              if (!finite) {
                hi[j] = 0x7F7F7F7Fu;
                lo[j] = 0u;
              }
            }
            *part[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *part[1] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            if (c == 0) q_scale_s[h][r] = finite ? scale2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 1.f;
          }
          fence_proxy_async_smem();
        }
        mbar_arrive(q_full + h);
      }
      const int odd = item % 3;
      int n_masked = 0;
      odd_rows[odd][cw][lane >> 2][lane & 3] = 0u;  // (the tile three before, whose places these were, is done with)
      static_assert(kMaxMasked * 4 == 32, "a word a lane");
      __syncwarp();
#pragma unroll 1
      for (int q = 0; q < o.blocks && ok; ++q) {
        const int n = n0 + q, j = o.j_top - q;
        const int raw_slot = n % C::kRawStages, v_slot = n % C::kVStages, meta = n % C::kMeta;
        ok = await(meta_full + meta, (n / C::kMeta) & 1, &watch) &&
             await(raw_full + raw_slot, (n / C::kRawStages) & 1, &watch);
        if (ok && n >= C::kVStages)
          ok = await(v_empty + v_slot, (n / C::kVStages - 1) & 1, &watch);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint8_t* raw = raw_ring + raw_slot * C::kCodeBytes;
        uint8_t* to = v_ring + v_slot * C::kVBytes + (D == 128 ? (c >> 2) * (kTile * 128) : 0);
        const uint32_t bad = bad_s[meta];
        const bool masked = o.masked(j);
        const int first = o.lo - j * kTile, past = o.hi - j * kTile;  // the block's keys that the tile sees
#pragma unroll 1
        for (int k0 = 0; k0 < kChunks; k0 += kFlight) {
          uint4 u[kFlight];
#pragma unroll
          for (int i = 0; i < kFlight; ++i) {
            const int r = r0 + (k0 + i) * kRowsAtOnce;
            u[i] = *reinterpret_cast<const uint4*>(raw + r * D + c * 16);
          }
          if (here(masked || bad)) {
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
              const int r = r0 + (k0 + i) * kRowsAtOnce;
              if (r < first || r >= past || ((bad >> (r >> 4)) & 1u)) {
                u[i] = make_uint4(0u, 0u, 0u, 0u);
              } else if (masked) {
                const uint32_t x = nan_codes(u[i].x), y = nan_codes(u[i].y), z = nan_codes(u[i].z), w = nan_codes(u[i].w);
                if (x | y | z | w) {  // (0x80 of a NaN byte becomes all ones)
                  u[i].x &= ~((x >> 7) * 255u);
                  u[i].y &= ~((y >> 7) * 255u);
                  u[i].z &= ~((z >> 7) * 255u);
                  u[i].w &= ~((w >> 7) * 255u);
                  if (n_masked < kMaxMasked) {
                    atomicOr(&odd_rows[odd][cw][n_masked][r >> 5], 1u << (r & 31));
                    odd_block[odd][cw][n_masked] = j;
                    odd_item[odd][cw] = item + 1;
                  }
                }
              }
            }
          }
#pragma unroll
          for (int i = 0; i < kFlight; ++i) {
            const int r = r0 + (k0 + i) * kRowsAtOnce;
            uint4 x, y;
            e4m3x4_to_f16(u[i].x, x.x, x.y);
            e4m3x4_to_f16(u[i].y, x.z, x.w);
            e4m3x4_to_f16(u[i].z, y.x, y.y);
            e4m3x4_to_f16(u[i].w, y.z, y.w);
            // (chunks of the upper 64 channels store their second half first: the
            // eight lanes of a row then write to eight different places of a line)
            const int q0 = 2 * (c & 3), q1 = D == 128 ? c >> 2 : 0;
            uint8_t* line = to + r * 128;
            *reinterpret_cast<uint4*>(line + (((q0 + q1) ^ (r & 7)) << 4)) = q1 ? y : x;
            *reinterpret_cast<uint4*>(line + (((q0 + 1 - q1) ^ (r & 7)) << 4)) = q1 ? x : y;
          }
        }
        if (masked) ++n_masked;
        fence_proxy_async_smem();
        mbar_arrive(v_full + v_slot);
        mbar_arrive(raw_empty + raw_slot);
      }
      n0 += o.blocks;
      done(item);
    }
  } else {
    // ---------------- softmax: one thread a row ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int t = warp >> 2;                   // the half
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_tmem = tmem + lane_base + C::kSCol(t), o_tmem = tmem + lane_base + C::kOCol(t);
    uint32_t n_s = 0, n_o[2] = {}, n_split = 0;  // scores and sums taken so far, tiles whose halves were joined
    int n0 = 0;
    bool ok = true;
#pragma unroll 1
    for (int item = 0; ok && take(item); ++item) {
      const Order& o = orders[item % kOrders];
      const bool split = o.split != 0;
      const int half = split ? 0 : t;                    // of the queries
      ok = __all_sync(0xffffffffu, await(q_full + half, item & 1, &watch));
      if (!ok) break;
      const int row = half * kTile + r;                  // in the tile
      const float fac = row < o.rows ? q_scale_s[half][r] : 0.f;
      mbar_arrive(&q_empty);
      const uint32_t at = static_cast<uint32_t>(o.row0 + row);
      const int qi = static_cast<int>(at / group), hd = static_cast<int>(at - static_cast<uint32_t>(qi) * group);
      // the row's keys [first_key, last_key]
      const int last_key = row < o.rows ? qi + o.shift : -1;
      const int first_key = a.window > 0 && last_key >= a.window ? last_key - a.window + 1 : 0;
      // The sum l is in units of 2^m, m the largest logit so far; the weighted values
      // are in units of 2^(m + d - kWeightExp), d the largest logit + log2(v_scale),
      // seen from m.  (As a number of its own that would be a multiple of 32 where
      // logits are of 2^28, and weights would leave f16.)
      float m = kNone, d = 0.f, l = 0.f;
      const int step = split ? 2 : 1;
      bool began = false;
      auto factor = [&](float ks) { return fmaxf(fac * ks, FLT_MIN); };  // (not 0: a masked score is -inf, and stays so under it)
#pragma unroll 1
      for (int q = split ? t : 0; q < o.blocks; q += step) {
        const int n = n0 + q, j = o.j_top - q, meta = n % C::kMeta;
        ok = await(meta_full + meta, (n / C::kMeta) & 1, &watch);
        const float v_min = v_min_s[meta];
        const uint32_t bad = bad_s[meta];
        ok = ok && await(s_full + t, n_s & 1u, &watch);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++n_s;
        tc_fence_after();
        // This row's keys alone, where a block has others: the scores of the rest
        // become -inf where they lie, 32 at a time (for its 128 keys at once, in
        // registers, the code is four times as long and in every block's way).
        if (o.masked(j) || bad) {
          const int c_hi = last_key + 1 - j * kTile, c_lo = first_key - j * kTile;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t x[32];
            tmem_ld32(s_tmem + 32 * c, x);
            const int hi = max(0, min(32, c_hi - 32 * c)), lo = max(0, min(32, c_lo - 32 * c));
            uint32_t seen = static_cast<uint32_t>((1ull << hi) - (1ull << min(lo, hi)));
            if (bad & (1u << (2 * c))) seen &= 0xFFFF0000u;
            if (bad & (2u << (2 * c))) seen &= 0x0000FFFFu;
            tmem_wait_ld();
            landed(x);
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!((seen >> k) & 1u)) x[k] = 0xFF800000u;
            tmem_st32(s_tmem + 32 * c, x);
          }
          tmem_wait_st();
        }
        uint32_t x[4][32];
        float ks[kGroups], vs[kGroups];
        float top = -INFINITY, w[kGroups];
        {
          tmem_ld32(s_tmem, x[0]);
          tmem_ld32(s_tmem + 32, x[1]);
          tmem_ld32(s_tmem + 64, x[2]);
          tmem_ld32(s_tmem + 96, x[3]);
          const float4 k0 = *reinterpret_cast<const float4*>(&k_scale_s[meta][0]);
          const float4 k1 = *reinterpret_cast<const float4*>(&k_scale_s[meta][4]);
          const float4 v0 = *reinterpret_cast<const float4*>(&v_log_s[meta][0]);
          const float4 v1 = *reinterpret_cast<const float4*>(&v_log_s[meta][4]);
          const float ku[kGroups] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
          const float vu[kGroups] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            ks[g] = factor(ku[g]);
            vs[g] = vu[g];
          }
          tmem_wait_ld();
          landed(x[0]);
          landed(x[1]);
          landed(x[2]);
          landed(x[3]);
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            const uint32_t* u = x[g >> 1] + (g & 1) * 16;
            w[g] = fmaxf(__uint_as_float(u[0]), __uint_as_float(u[1]));
#pragma unroll
            for (int k = 2; k < 16; k += 2) w[g] = max3(w[g], __uint_as_float(u[k]), __uint_as_float(u[k + 1]));
            w[g] *= ks[g];
            top = fmaxf(top, w[g]);
          }
        }
        // d so far and of this block, both seen from the larger maximum
        const float both = fmaxf(m, top), d_old = d + (m - both);
        float d_new = -INFINITY;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) d_new = fmaxf(d_new, w[g] - both + vs[g]);
        // (a row whose own maximum has not grown keeps its reference, so that no bit
        // of it depends on what only the warp's other rows see)
        const bool grown = top - m > kLag || d_new - d_old > kLag;
        if (__any_sync(0xffffffffu, grown)) {
          float f = 1.f;
          if (grown) {
            const float d1 = fmaxf(d_old, d_new);
            l *= ex2(m - both);
            f = ex2(d_old - d1);
            m = both;
            d = d1;
          }
          if (began) {  // (the half's products before have finished: these scores were issued after them)
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t x[16];
              tmem_ld16(o_tmem + 16 * c, x);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * f);
              tmem_st16(o_tmem + 16 * c, x);
            }
          }
        }
        began = true;
        const float down = d - kWeightExp;
        const bool large = fabsf(m) > kLarge && m > kNone, far = v_min - down < kFar;
        if (!__any_sync(0xffffffffu, large || far)) {
          // 32 keys a turn, the scores behind them moved up in the registers: code for all
          // 128 is faster where one long sequence keeps the loop in the instruction
          // caches (2048 tokens at 62000 1535 us, 1604 so) and slower where tiles end
          // often (12 prompts 584 us, 546 so; 48 mixed sequences 312, 304).  Reading the
          // scores again from tensor memory instead takes 1690 and 564 us.  (All with m
          // and d as one sum; d apart takes 2 % on the first, 1 % on the others, and as
          // much with the exact form of d_new for rows of large logits alone: 1616, 564
          // and 312 us against 1636, 554 and 307.)
          const float up = -down - m;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t p[16];
            uint64_t y[16];
#pragma unroll
            for (int k = 0; k < 16; ++k)
              y[k] = fma2(pair_of(x[0][2 * k], x[0][2 * k + 1]), pair_of(ks[k >> 3], ks[k >> 3]),
                          pair_of(vs[k >> 3] + up, vs[k >> 3] + up));
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              uint64_t sum = 0ull;
              float u, v;
#pragma unroll
              for (int k = 8 * g; k < 8 * g + 8; ++k) {
                csa::split(y[k], &u, &v);
                u = ex2(u);
                v = ex2(v);
                sum = add2(sum, pair_of(u, v));
                p[k] = pack_f16(u, v);
              }
              csa::split(sum, &u, &v);
              l = fmaf(u + v, ex2(down - vs[g]), l);
            }
            tmem_st16(s_tmem + 16 * c, p);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              x[0][k] = x[1][k];
              x[1][k] = x[2][k];
              x[2][k] = x[3][k];
            }
#pragma unroll
            for (int g = 0; g < 6; ++g) {
              ks[g] = ks[g + 2];
              vs[g] = vs[g + 2];
            }
          }
        } else {
          // Rare: exponents are one rounding, factor s - m, but where logits are so large
          // that the rounding of m shows the products come first; where the weights' sum
          // cannot be taken from the weights it has exponentials of its own.
          const float less = large ? m : 0.f, up = large ? -down : -down - m;
          const float minus_m = large ? 0.f : -m;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t y[32], p[16];
            tmem_ld32(s_tmem + 32 * c, y);
            tmem_wait_ld();
            landed(y);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float f = factor(k_scale_s[meta][2 * c + h]);
              const float vs = v_log_s[meta][2 * c + h];
              const float f_first = large ? f : 1.f;
              if (large) f = 1.f;
              float sum_u = 0.f, sum_v = 0.f, sum_far = 0.f;  // (in the order of the other way)
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float y0 = __fsub_rn(__fmul_rn(__uint_as_float(y[16 * h + 2 * k]), f_first), less);
                const float y1 = __fsub_rn(__fmul_rn(__uint_as_float(y[16 * h + 2 * k + 1]), f_first), less);
                const float u = ex2(fmaf(y0, f, vs + up)), v = ex2(fmaf(y1, f, vs + up));
                sum_u += u;
                sum_v += v;
                sum_far += ex2(fmaf(y0, f, minus_m)) + ex2(fmaf(y1, f, minus_m));
                p[8 * h + k] = pack_f16(u, v);
              }
              l = far ? l + sum_far : fmaf(sum_u + sum_v, ex2(down - vs), l);
            }
            tmem_st16(s_tmem + 16 * c, p);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full + t);
      }
      if (!ok) break;
      n0 += o.blocks;
      // ---------------- the tile's rows, or this share's part of them ----------------
      const bool have[2] = {true, !split || o.blocks > 1};
      if (split) {
        m_s[t][r] = m;
        d_s[t][r] = d;
        l_s[t][r] = l;
        mbar_arrive(&joined);
        ok = await(&joined, n_split & 1u, &watch) &&
             await(o_full + 0, n_o[0] & 1u, &watch);
        if (ok && have[1]) ok = await(o_full + 1, n_o[1] & 1u, &watch);
      } else {
        ok = await(o_full + t, n_o[t] & 1u, &watch);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ++n_o[0];
      if (have[1]) ++n_o[1];
      tc_fence_after();
      float f0 = 1.f, f1 = 0.f;  // of the halves' sums
      if (split) {
        const float ma = m_s[0][r], mb = m_s[1][r], da = d_s[0][r], db = d_s[1][r];
        m = ma;
        d = da;
        join_units(m, d, mb, db);
        l = l_s[0][r] * ex2(ma - m) + l_s[1][r] * ex2(mb - m);
        f0 = ex2(in_unit(ma, da, m, d));
        f1 = ex2(in_unit(mb, db, m, d));
      }
      const float unit = d - kWeightExp;
      const int64_t out_row = static_cast<int64_t>(o.q0 + qi) * a.n_heads + o.head0 + hd;
      float* part = a.part + gridDim.x * (sizeof(Cut) / sizeof(float)) + (blockIdx.x * 2 + max(o.record, 0)) * C::kRecord;
      float f = 1.f;
      const bool writes = row < o.rows, few = o.rows <= kFewRows;
      if (o.record < 0) {
        float lse;
        f = finish_row(m, unit, l, a.sink, o.head0 + hd, &lse);
        if (a.lse && writes && (!split || t == 0)) a.lse[out_row] = lse;
      } else if (!split || t == 0) {
        *reinterpret_cast<float4*>(part + kTileRows * D + 4 * row) = make_float4(m, l, unit, 0.f);
      }
      f0 *= f;
      f1 *= f;
      const int odd = item % 3;
      bool any_odd = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) any_odd |= *const_cast<volatile int*>(&odd_item[odd][k]) == item + 1;
      // the halves of a split tile take half of the channels each
      const int c_lo = split ? t * (D / 32) : 0, c_hi = split ? (t + 1) * (D / 32) : D / 16;
      const uint32_t oa = split ? tmem + lane_base + C::kOCol(0) : o_tmem, ob = tmem + lane_base + C::kOCol(1);
      const uint64_t f00 = pair_of(f0, f0), f11 = pair_of(f1, f1);
      uint16_t* out = a.out + out_row * D;
      const bool two = split && have[1];
      uint32_t x[16], y[16];
      tmem_ld16(oa + 16 * c_lo, x);
      if (two)
        tmem_ld16(ob + 16 * c_lo, y);
      else
#pragma unroll
        for (int k = 0; k < 16; ++k) y[k] = 0u;
#pragma unroll 1
      for (int c = c_lo; c < c_hi; ++c) {
        tmem_wait_ld();
        landed(x);
        landed(y);
        float z[16];
        uint64_t zz[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) zz[k] = mul2(pair_of(x[2 * k], x[2 * k + 1]), f00);
        if (two) {
#pragma unroll
          for (int k = 0; k < 8; ++k) zz[k] = fma2(pair_of(y[2 * k], y[2 * k + 1]), f11, zz[k]);
        }
        if (c + 1 < c_hi) {  // (the next ones, under what follows)
          tmem_ld16(oa + 16 * (c + 1), x);
          if (two) tmem_ld16(ob + 16 * (c + 1), y);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) csa::split(zz[k], &z[2 * k], &z[2 * k + 1]);
        if (any_odd && writes) {
#pragma unroll 1
          for (int e = 0; e < 4 * kMaxMasked * kTile; ++e) {
            const int cw = e / (kMaxMasked * kTile), i = (e / kTile) % kMaxMasked, k = e % kTile;
            if (*const_cast<volatile int*>(&odd_item[odd][cw]) != item + 1) {
              e += kMaxMasked * kTile - 1;
              continue;
            }
            const uint32_t word = odd_rows[odd][cw][i][k >> 5];
            if (word == 0u) {
              e |= 31;
              continue;
            }
            const int key = odd_block[odd][cw][i] * kTile + k;
            if (!((word >> (k & 31)) & 1u) || key > last_key || key < first_key) continue;
            const int64_t page = a.cache.table[o.b * a.cache.table_stride + (key >> a.cache.page_shift)];
            const uint8_t* v = a.cache.v + (((page * a.cache.n_kv_heads + o.kv_head) << a.cache.page_shift) +
                                            (key & (a.cache.page - 1))) * D + 16 * c;
#pragma unroll
            for (int d = 0; d < 16; ++d)
              if ((v[d] & 0x7Fu) == 0x7Fu) z[d] = NAN;
          }
        }
        if (o.record >= 0) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<float4*>(part + (few ? row * D + 16 * c + 4 * k : ((4 * c + k) * kTileRows + row) * 4)) =
                make_float4(z[4 * k], z[4 * k + 1], z[4 * k + 2], z[4 * k + 3]);
          continue;
        }
        if (!writes) continue;
        uint4* to = reinterpret_cast<uint4*>(out + 16 * c);
        to[0] = make_uint4(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]), pack_bf16(z[4], z[5]), pack_bf16(z[6], z[7]));
        to[1] = make_uint4(pack_bf16(z[8], z[9]), pack_bf16(z[10], z[11]), pack_bf16(z[12], z[13]), pack_bf16(z[14], z[15]));
      }
      done(item);
      tc_fence_before();
      if (split) {  // the other half has read these sums, and its own, before either is written again
        mbar_arrive(&left_off);
        ok = __all_sync(0xffffffffu, await(&left_off, n_split & 1u, &watch));
        ++n_split;
      }
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
}

// Finishes the tiles that the shares' borders divide, from their records: the
// first share's second one, the later shares' first.  CTAs (x, 0..) take the rows
// of the tile that begins in share x and goes on: with few rows one at a time,
// each warp a part of the records; else 16 at a time, a thread four channels.
// (8 tokens at 60000 53.7 us with the second way alone, 48.5 so; 64 tokens at 1000
// 22.7 us, 27.6 with a warp a row.)
constexpr int kMergeWarps = 8, kMergeThreads = 32 * kMergeWarps, kMergeRows = 16;
constexpr int kMergeCtas = kTileRows / kMergeRows;  // a tile

__device__ __forceinline__ void store_row(const ChunkAttnArgs& a, const Cut& cut, int r, float m, float unit, float l,
                                          bool first, float* factor, int64_t* row) {
  const uint32_t group = a.n_heads / a.cache.n_kv_heads;
  const uint32_t at = static_cast<uint32_t>(cut.row0 + r), qi = at / group;
  const int head = cut.head0 + static_cast<int>(at - qi * group);
  *row = (cut.q0 + static_cast<int64_t>(qi)) * a.n_heads + head;
  float lse;
  *factor = finish_row(m, unit, l, a.sink, head, &lse);
  if (a.lse && first) a.lse[*row] = lse;
}

template <int D>
__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(const ChunkAttnArgs a, const int shares) {
  using C = Cfg<D>;
  __shared__ float l_s[kMergeWarps];
  __shared__ __align__(16) float n_s[kMergeWarps][D];
  pdl_launch_dependents();
  pdl_wait();
  const Cut cut = reinterpret_cast<const Cut*>(a.part)[blockIdx.x];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = cut.last - cut.first + 1;
  const float* records = a.part + shares * (sizeof(Cut) / sizeof(float));
  auto record = [&](int k) { return records + (static_cast<int64_t>(cut.first + k) * 2 + (k == 0)) * C::kRecord; };
  auto stats = [&](int k, int r) { return *reinterpret_cast<const float4*>(record(k) + kTileRows * D + 4 * r); };
  if (cut.rows > kFewRows) {
    const int r = blockIdx.y * kMergeRows + tid % kMergeRows;
    if (r >= cut.rows) return;
    float m = kNone, unit = 0.f;
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const float4 y = stats(k, r);
      join_units(m, unit, y.x, y.z);
    }
    for (int c = tid / kMergeRows; c < D / 4; c += kMergeThreads / kMergeRows) {
      float l = 0.f;
      float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int k = 0; k < n; ++k) {
        const float4 y = stats(k, r), x = *reinterpret_cast<const float4*>(record(k) + (c * kTileRows + r) * 4);
        l += y.y * ex2(y.x - m);
        const float f = ex2(in_unit(y.x, y.z, m, unit));
        z.x = fmaf(x.x, f, z.x);
        z.y = fmaf(x.y, f, z.y);
        z.z = fmaf(x.z, f, z.z);
        z.w = fmaf(x.w, f, z.w);
      }
      float f;
      int64_t row;
      store_row(a, cut, r, m, unit, l, c == 0, &f, &row);
      *reinterpret_cast<uint2*>(a.out + row * D + 4 * c) =
          make_uint2(pack_bf16(z.x * f, z.y * f), pack_bf16(z.z * f, z.w * f));
    }
    return;
  }
  constexpr int kPer = D / 32;  // channels a lane, neighbours
  using Vec = typename std::conditional<kPer == 4, float4, float2>::type;
  for (int r = blockIdx.y; r < cut.rows; r += kMergeCtas) {
    float m = kNone, unit = 0.f, l = 0.f, z[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) z[j] = 0.f;
    for (int k = lane; k < n; k += 32) {
      const float4 y = stats(k, r);
      join_units(m, unit, y.x, y.z);
    }
    join_lanes(m, unit);
#pragma unroll 4
    for (int k = warp; k < n; k += kMergeWarps) {
      const float4 y = stats(k, r);
      const Vec v = *reinterpret_cast<const Vec*>(record(k) + r * D + lane * kPer);
      l += y.y * ex2(y.x - m);
      const float f = ex2(in_unit(y.x, y.z, m, unit));
      const float* x = reinterpret_cast<const float*>(&v);
#pragma unroll
      for (int j = 0; j < kPer; ++j) z[j] = fmaf(x[j], f, z[j]);
    }
    __syncthreads();  // the warps' sums, first to last
    if (lane == 0) l_s[warp] = l;
#pragma unroll
    for (int j = 0; j < kPer; ++j) n_s[warp][lane * kPer + j] = z[j];
    __syncthreads();
    if (warp != 0) continue;
    for (int w = 1; w < kMergeWarps; ++w) {
      l += l_s[w];
#pragma unroll
      for (int j = 0; j < kPer; ++j) z[j] += n_s[w][lane * kPer + j];
    }
    float f;
    int64_t row;
    store_row(a, cut, r, m, unit, l, lane == 0, &f, &row);
    uint32_t y[kPer / 2];
#pragma unroll
    for (int j = 0; j < kPer / 2; ++j) y[j] = pack_bf16(z[2 * j] * f, z[2 * j + 1] * f);
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row * D + lane * kPer);
    if constexpr (kPer == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
    else
      *dst = y[0];
  }
}

// The codes of a pool, [pages][kv heads * page size][channels], read a page of
// one head at a time.
bool encode_codes(CUtensorMap* m, PFN_cuTensorMapEncodeTiled_v12000 encode, const PagedCache& c, uint8_t* base,
                  CUtensorMapSwizzle swizzle) {
  cuuint64_t size[3] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.n_kv_heads) * c.page,
                        static_cast<cuuint64_t>(c.n_pages)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.head_dim), size[1] * c.head_dim};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(c.head_dim), static_cast<cuuint32_t>(c.page), 1};
  cuuint32_t ones[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, size, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_dim(const ChunkAttnArgs& a, int sms, PFN_cuTensorMapEncodeTiled_v12000 encode, cudaStream_t stream) {
  using C = Cfg<D>;
  CUtensorMap tm_k, tm_v;
  if (!encode ||
      !encode_codes(&tm_k, encode, a.cache, a.cache.k, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) ||
      !encode_codes(&tm_v, encode, a.cache, a.cache.v, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done{0};
  // (the split of registers assumes what the kernel is launched with)
  cudaError_t e = kernel_limits(reinterpret_cast<const void*>(chunk_attn_kernel<D>), C::kSmem, kLaunchRegs, &done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(chunk_attn_kernel<D>, dim3(sms), dim3(kThreads), C::kSmem, stream, tm_k, tm_v, a);
  if (e != cudaSuccess || sms < 2) return e;
  return launch_pdl(chunk_merge_kernel<D>, dim3(sms - 1, kMergeCtas), dim3(kMergeThreads), 0, stream, a, sms);
}

}  // namespace

size_t chunk_attn_bytes(int head_dim, int sms) {
  const int64_t record = head_dim == 64 ? Cfg<64>::kRecord : Cfg<128>::kRecord;
  return static_cast<size_t>(sms) * (sizeof(Cut) + 2 * record * sizeof(float));
}

cudaError_t launch_chunk_attn(const ChunkAttnArgs& a, int sms, PFN_cuTensorMapEncodeTiled_v12000 encode,
                              cudaStream_t stream) {
  if (a.B <= 0 || a.n_q <= 0) return cudaSuccess;
  return a.cache.head_dim == 128 ? launch_dim<128>(a, sms, encode, stream) : launch_dim<64>(a, sms, encode, stream);
}

}  // namespace csa
