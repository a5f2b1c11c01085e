// Bookkeeping of a paged cache's pages, and the copy of their contents.
//
// A page is free where its count is 0 (or less); pages are handed out lowest
// number first, in the order of the sequences and of their tables, so that the
// result is the same whatever runs when.  A call is two launches: the first
// reads the counts once (4 bytes a page, all that grows with the pool), keeps a
// bit a page and the free pages of each stretch, and sums up what the sequences
// need; in the second a CTA a sequence finds its pages by their rank: the
// stretch from the stretches' sums, the page from its bits.  Bound by the two
// launches and the handful of dependent loads in each, some 3 us a launch: 64
// sequences given 8 tokens and taken back 11.7 us replayed from a graph (two calls;
// 15 to 16 as eager ones, which the host's side bounds), 1024 that grow by up to 500
// tokens in a pool of 2^20 pages and back 25.5 us.  One launch of a cluster of 8 CTAs
// with the cluster's barrier between the steps took 14 (eager) and 149 us: eight SMs
// read the counts no faster.
#include "gqa.cuh"
#include "ptx.cuh"

namespace csa {
namespace {

constexpr int kScanThreads = 256;
constexpr int kSumThreads = 1024;    // of the CTA that sums up what the sequences need
constexpr int kSeqThreads = 128;     // of a sequence's CTA
constexpr int kMaxStretches = 1024;
constexpr int kMinStretch = 4096;    // pages

// Stretches of 2^shift pages, at most kMaxStretches.
__host__ __device__ __forceinline__ int stretch_shift(int64_t n_pages) {
  int s = 12;
  while ((n_pages + (int64_t(1) << s) - 1) >> s > kMaxStretches) ++s;
  return s;
}
static_assert(kMinStretch == 1 << 12, "the first shift");

// The workspace's parts.
struct Work {
  int32_t* free_of;    // [stretches] free pages of each
  int64_t* before;     // [n_seqs + 1] pages that the sequences before need
  int32_t* lens;       // [n_seqs] lengths before the call (fork: the parent's; -1: no child)
  uint32_t* bits;      // [n_pages / 32] free pages
  int32_t* rank;       // [n_pages] place of a page in the lists of a compaction
};
__host__ __device__ __forceinline__ size_t round16(size_t n) { return (n + 15) & ~size_t(15); }
__host__ __device__ __forceinline__ size_t work_bytes(int n_seqs, int64_t n_pages, void* base, Work* w) {
  uint8_t* p = static_cast<uint8_t*>(base);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* x = p + at;
    at += round16(bytes);
    return x;
  };
  Work parts;
  parts.free_of = reinterpret_cast<int32_t*>(take(kMaxStretches * 4));
  parts.before = reinterpret_cast<int64_t*>(take((static_cast<size_t>(n_seqs) + 1) * 8));
  parts.lens = reinterpret_cast<int32_t*>(take(static_cast<size_t>(n_seqs) * 4));
  parts.bits = reinterpret_cast<uint32_t*>(take(static_cast<size_t>((n_pages + 31) / 32) * 4));
  parts.rank = reinterpret_cast<int32_t*>(take(static_cast<size_t>(n_pages) * 4));
  if (w) *w = parts;
  return at;
}

enum Op { kResize = 0, kFork = 1, kCompact = 2 };

__device__ __forceinline__ int64_t capacity(const PageBook& k) { return k.table_stride << k.page_shift; }
__device__ __forceinline__ int pages_of(const PageBook& k, int tokens) {
  return static_cast<int>((static_cast<int64_t>(tokens) + k.page - 1) >> k.page_shift);
}
// A sequence's length, within its table.
__device__ __forceinline__ int length_of(const PageBook& k, int b, unsigned* status) {
  const int64_t n = k.lens[b], cap = capacity(k);
  if (n > cap) record_error(status, kErrIndexRange);
  return static_cast<int>(n < 0 ? 0 : n > cap ? cap : n);
}
__device__ __forceinline__ bool in_pool(const PageBook& k, int32_t page) { return page >= 0 && page < k.n_pages; }

// Pages that a sequence of L tokens takes from the free ones to grow to t (0:
// it does not grow, or cannot): those of the new tokens, and one in the place
// of a last page that is partly filled and that others hold too.
__device__ __forceinline__ int growth(const PageBook& k, int b, int L, int t, unsigned* status) {
  if (t <= L || t > capacity(k)) return 0;
  int n = pages_of(k, t) - pages_of(k, L);
  if (L & (k.page - 1)) {
    const int32_t last = k.table[b * k.table_stride + (L >> k.page_shift)];
    if (!in_pool(k, last))
      record_error(status, kErrIndexRange);
    else if (k.refs[last] > 1)
      ++n;
  }
  return n;
}

// Sums over the CTA's threads before this one (of n), and the sum of all.
template <int THREADS, typename T>
__device__ __forceinline__ T sum_before(T n, T* sh, T* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = n;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  T before = x - n, sum = 0;
#pragma unroll
  for (int k = 0; k < THREADS / 32; ++k) {
    const T y = sh[k];
    if (k < warp) before += y;
    sum += y;
  }
  *all = sum;
  return before;
}

// Looks at a stretch of the counts: a bit a page and the free pages' number.  Every
// thread of the CTA calls it; sh holds kSumThreads / 32 values.
__device__ __forceinline__ void scan_stretch(const PageBook& k, const Work& w, int shift, int s, int64_t* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = static_cast<int64_t>(s) << shift, end = min(first + (int64_t(1) << shift), k.n_pages);
  int n = 0;
  constexpr int kFlight = 4;  // words a warp
  for (int64_t p0 = first + warp * 32; p0 < end; p0 += kFlight * kSumThreads) {
    int32_t r[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int64_t p = p0 + i * kSumThreads + lane;
      r[i] = p < end ? k.refs[p] : 1;
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const uint32_t word = __ballot_sync(0xffffffffu, r[i] <= 0);
      const int64_t p = p0 + i * kSumThreads;
      if (lane == 0 && p < end) w.bits[p >> 5] = word;
      n += __popc(word);
    }
  }
  int64_t all;
  sum_before<kSumThreads, int64_t>(lane == 0 ? n : 0, sh, &all);
  if (threadIdx.x == 0) w.free_of[s] = static_cast<int32_t>(all);
}

// Sums up what the sequences need, by one CTA.
template <int OP>
__device__ __forceinline__ void sum_needs(const PageBook& k, const Work& w, const int32_t* want, unsigned* status,
                                          int64_t* sh) {
  int64_t base = 0;
  for (int b0 = 0; b0 < k.n_seqs; b0 += kSumThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    int64_t n = 0;
    if (b < k.n_seqs) {
      const int t = want[b];
      int L = 0;
      if (OP == kResize) {
        L = length_of(k, b, status);
        if (t > capacity(k)) record_error(status, kErrIndexRange);
        n = growth(k, b, L, t, status);
      } else if (t < 0) {
        L = -1;
      } else if (t >= k.n_seqs || k.lens[b] > 0) {  // no such parent, or a sequence that has tokens
        record_error(status, kErrIndexRange);
        L = -1;
      } else {
        L = length_of(k, t, status);
        n = (L & (k.page - 1)) != 0;
      }
      w.lens[b] = L;
    }
    int64_t all;
    const int64_t before = base + sum_before<kSumThreads, int64_t>(n, sh, &all);
    if (b < k.n_seqs) w.before[b] = before;
    base += all;
  }
  if (threadIdx.x == 0) w.before[k.n_seqs] = base;
}

// Free pages before each stretch, in shared memory (kMaxStretches + 1), and in
// all; every thread of the CTA calls it.
template <int THREADS>
__device__ __forceinline__ int64_t free_before(const Work& w, int stretches, int32_t* before, int64_t* sh) {
  int64_t base = 0;
  for (int s0 = 0; s0 < stretches; s0 += THREADS) {
    const int s = s0 + static_cast<int>(threadIdx.x);
    int64_t all;
    const int64_t x = base + sum_before<THREADS, int64_t>(s < stretches ? w.free_of[s] : 0, sh, &all);
    if (s < stretches) before[s] = static_cast<int32_t>(x);
    base += all;
  }
  if (threadIdx.x == 0) before[stretches] = static_cast<int32_t>(base);
  __syncthreads();
  return base;
}

// The free pages of ranks r0 .. r0 + n - 1, in order, by one warp: give(i, page).
template <typename Give>
__device__ __forceinline__ void free_pages(const PageBook& k, const Work& w, int shift, int stretches,
                                           const int32_t* before, int32_t r0, int n, Give give) {
  if (n <= 0) return;
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = stretches - 1;  // the last stretch with at most r0 free pages before it
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (before[mid] <= r0) lo = mid; else hi = mid - 1;
  }
  const int32_t r1 = r0 + n;
  const int64_t words = (k.n_pages + 31) >> 5, per = int64_t(1) << (shift - 5);
  for (int s = lo; s < stretches && before[s] < r1; ++s) {
    int32_t rank = before[s];
    const int64_t end = min((s + 1) * per, words);
    for (int64_t i0 = s * per; i0 < end && rank < r1; i0 += 128) {
      uint32_t word[4];
      int c = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // a lane holds four neighbours
        const int64_t i = i0 + 4 * lane + j;
        word[j] = i < end ? w.bits[i] : 0u;
        c += __popc(word[j]);
      }
      int x = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      const int32_t mine = rank + x - c;
      rank += __shfl_sync(0xffffffffu, x, 31);
      // a word at a time, a lane a page
      for (unsigned hit = __ballot_sync(0xffffffffu, mine < r1 && mine + c > r0); hit; hit &= hit - 1) {
        const int l = __ffs(hit) - 1;
        int32_t r = __shfl_sync(0xffffffffu, mine, l);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t u = __shfl_sync(0xffffffffu, word[j], l);
          const int32_t q = r + __popc(u & ((1u << lane) - 1u));
          if (((u >> lane) & 1u) && q >= r0 && q < r1)
            give(q - r0, static_cast<int32_t>((i0 + 4 * l + j) * 32 + lane));
          r += __popc(u);
        }
      }
    }
  }
}

// Takes one holder off each of entries [from, to) of a row, which become -1; a CTA.
// (A count that is 0 already stays so.)
__device__ __forceinline__ void give_back(const PageBook& k, int32_t* row, int from, int to, unsigned* status) {
  constexpr int kFlight = 4;
  for (int j0 = from + static_cast<int>(threadIdx.x); j0 < to; j0 += kFlight * kSeqThreads) {
    int32_t page[kFlight], held[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) page[i] = j0 + i * kSeqThreads < to ? row[j0 + i * kSeqThreads] : -1;
#pragma unroll
    for (int i = 0; i < kFlight; ++i) held[i] = in_pool(k, page[i]) ? atomicSub(k.refs + page[i], 1) : 0;
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      if (j0 + i * kSeqThreads >= to) continue;
      row[j0 + i * kSeqThreads] = -1;
      if (held[i] > 0) continue;
      if (in_pool(k, page[i])) atomicAdd(k.refs + page[i], 1);
      record_error(status, kErrIndexRange);
    }
  }
}

// What a call is given and gives beside the book.
struct Lists {
  const int32_t* want;         // targets, or parents
  int32_t *pos0, *src, *dst;
};

__global__ void __launch_bounds__(kSeqThreads)
    pages_resize_kernel(const PageBook k, const Work w, const int shift, const int stretches, const Lists x,
                        unsigned* status) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ int32_t before[kMaxStretches + 1];
  __shared__ int64_t sh[kSeqThreads / 32];
  const int b = blockIdx.x, tid = threadIdx.x;
  const int L = w.lens[b], t = x.want[b];
  const int64_t r0 = w.before[b], need = w.before[b + 1] - r0;
  int32_t* row = k.table + b * k.table_stride;
  const int n0 = pages_of(k, L);
  int now = L, first = -1, old = -1;
  if (t > L && t <= capacity(k)) {
    const int64_t all = need > 0 ? free_before<kSeqThreads>(w, stretches, before, sh) : 0;
    const int n1 = pages_of(k, t), from = n1 - static_cast<int>(need);
    const bool apart = from < n0;  // the last page is left to its other holders
    if ((need > 0 && r0 + need > all) || (apart && !x.src)) {
      if (tid == 0) record_error(status, kErrIndexRange);
    } else {
      if (apart) old = row[from];
      __syncthreads();
      if (tid < 32)
        free_pages(k, w, shift, stretches, before, static_cast<int32_t>(r0), static_cast<int>(need),
                   [&](int i, int32_t page) {
                     row[from + i] = page;
                     k.refs[page] = 1;
                     if (apart && i == 0) x.dst[b] = page;
                   });
      if (apart && tid == 0) atomicSub(k.refs + old, 1);  // (it has other holders)
      now = t;
      first = L;
    }
  } else if (t >= 0 && t < L) {
    give_back(k, row, pages_of(k, t), n0, status);
    now = t;
  }
  if (tid == 0) {
    k.lens[b] = now;
    if (x.pos0) x.pos0[b] = first;
    if (x.src) {
      x.src[b] = old;
      if (old < 0) x.dst[b] = -1;
    }
  }
}

__global__ void __launch_bounds__(kSeqThreads)
    pages_fork_kernel(const PageBook k, const Work w, const int shift, const int stretches, const Lists x,
                      unsigned* status) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ int32_t before[kMaxStretches + 1];
  __shared__ int64_t sh[kSeqThreads / 32];
  const int b = blockIdx.x, tid = threadIdx.x;
  const int L = w.lens[b];
  int32_t from = -1;
  if (L > 0) {
    const int64_t r0 = w.before[b];
    const int whole = L >> k.page_shift, need = (L & (k.page - 1)) != 0;
    const int32_t* theirs = k.table + static_cast<int64_t>(x.want[b]) * k.table_stride;
    int32_t* row = k.table + b * k.table_stride;
    const int64_t all = need ? free_before<kSeqThreads>(w, stretches, before, sh) : 0;
    if (need && r0 + need > all) {
      if (tid == 0) record_error(status, kErrIndexRange);
    } else {
      constexpr int kFlight = 4;
      for (int j0 = tid; j0 < whole; j0 += kFlight * kSeqThreads) {
        int32_t page[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) page[i] = j0 + kSeqThreads * i < whole ? theirs[j0 + kSeqThreads * i] : 0;
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          if (j0 + kSeqThreads * i >= whole) continue;
          row[j0 + kSeqThreads * i] = page[i];
          if (in_pool(k, page[i]))
            atomicAdd(k.refs + page[i], 1);
          else
            record_error(status, kErrIndexRange);
        }
      }
      if (need) {
        from = theirs[whole];
        if (!in_pool(k, from)) {  // (the child has its page, and nothing to copy there)
          if (tid == 0) record_error(status, kErrIndexRange);
          from = -1;
        }
        if (tid < 32)
          free_pages(k, w, shift, stretches, before, static_cast<int32_t>(r0), 1, [&](int, int32_t page) {
            row[whole] = page;
            k.refs[page] = 1;
            if (from >= 0) x.dst[b] = page;
          });
      }
      if (tid == 0) k.lens[b] = L;
    }
  }
  if (tid == 0) {
    x.src[b] = from;
    if (from < 0) x.dst[b] = -1;
  }
}

// CTAs 0 .. stretches - 1 look at a stretch of the counts each, the last one at
// the sequences.
template <int OP>
__global__ void __launch_bounds__(kSumThreads)
    pages_scan_kernel(const PageBook k, const Work w, const int shift, const int stretches, const int32_t* want,
                      unsigned* status) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ int64_t sh[kSumThreads / 32];
  if (static_cast<int>(blockIdx.x) < stretches)
    scan_stretch(k, w, shift, blockIdx.x, sh);
  else if (OP != kCompact)
    sum_needs<OP>(k, w, want, status, sh);
}

// Lists of a compaction: with U used pages, the used ones from U on (src) and
// the free ones below U (dst), as many, both in order; rank: each one's place.
// A CTA a stretch.
__global__ void __launch_bounds__(kScanThreads)
    pages_list_kernel(const PageBook k, const Work w, const int shift, const int stretches, int32_t* src, int32_t* dst,
                      int32_t* used) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ int32_t before[kMaxStretches + 1];
  __shared__ int64_t sh[kScanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, stretch = blockIdx.x;
  const int64_t U = k.n_pages - free_before<kScanThreads>(w, stretches, before, sh);
  if (stretch == 0 && tid == 0) *used = static_cast<int32_t>(U);
  const int64_t words = (k.n_pages + 31) >> 5, per = int64_t(1) << (shift - 5);
  // free pages below U
  int64_t holes = 0;
  if (U < k.n_pages) {
    const int s = static_cast<int>(U >> shift);
    int32_t n = 0;
    for (int64_t i = s * per + tid; i <= U >> 5; i += kScanThreads) {
      uint32_t u = w.bits[i];
      if (i == U >> 5) u &= (1u << (U & 31)) - 1u;
      n += __popc(u);
    }
    int64_t all;
    sum_before<kScanThreads, int64_t>(n, sh, &all);
    holes = before[s] + all;
  }
  int64_t rank = before[stretch];
  const int64_t end = min((stretch + 1) * per, words);
  for (int64_t i0 = stretch * per; i0 < end; i0 += kScanThreads) {
    const int64_t i = i0 + tid;
    const uint32_t word = i < end ? w.bits[i] : 0u;
    int64_t all;
    const int32_t mine = static_cast<int32_t>(rank + sum_before<kScanThreads, int64_t>(__popc(word), sh, &all));
    rank += all;
    // a warp takes its lanes' words in turn, a lane a page
    const int here = static_cast<int>(min(end - (i - lane), static_cast<int64_t>(32)));
#pragma unroll 4
    for (int l = 0; l < here; ++l) {
      const uint32_t u = __shfl_sync(0xffffffffu, word, l);
      const int32_t free_here = __shfl_sync(0xffffffffu, mine, l);
      const int64_t p = (i - lane + l) * 32 + lane;
      if (p >= k.n_pages) continue;
      const int32_t f = free_here + __popc(u & ((1u << lane) - 1u));  // free pages before p
      const bool is_free = (u >> lane) & 1u;
      if (is_free && p < U) {
        dst[f] = static_cast<int32_t>(p);
        w.rank[p] = f;
      } else if (!is_free && p >= U) {
        const int32_t r = static_cast<int32_t>(p - f - (U - holes));  // used pages before p, less those below U
        src[r] = static_cast<int32_t>(p);
        w.rank[p] = r;
      }
    }
  }
  for (int64_t r = holes + static_cast<int64_t>(stretch) * kScanThreads + tid; r < k.n_pages / 2;
       r += static_cast<int64_t>(stretches) * kScanThreads) {
    src[r] = -1;
    dst[r] = -1;
  }
}

__device__ __forceinline__ bool is_free(const Work& w, int64_t p) { return (w.bits[p >> 5] >> (p & 31)) & 1u; }

// The counts under the pages' new numbers, by `threads` threads of which this is number i.
__device__ __forceinline__ void renumber_counts(const PageBook& k, const Work& w, int64_t U, int64_t i,
                                                int64_t threads, const int32_t* src, int32_t* refs) {
  constexpr int kFlight = 4;
  for (int64_t p0 = i; p0 < k.n_pages; p0 += kFlight * threads) {
    int32_t n[kFlight];
    int64_t from[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const int64_t p = p0 + j * threads;
      from[j] = -1;
      if (p >= k.n_pages) continue;
      from[j] = !is_free(w, p) ? (p < U ? p : -1) : p < U ? src[w.rank[p]] : -2;
    }
#pragma unroll
    for (int j = 0; j < kFlight; ++j) n[j] = from[j] >= 0 ? k.refs[from[j]] : 0;
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const int64_t p = p0 + j * threads;
      if (from[j] == -1) continue;  // (a page that moves: its count is written by the thread of its new place)
      refs[p] = n[j];
      if (from[j] >= 0 && from[j] != p) refs[from[j]] = 0;
    }
  }
}

// A sequence's table under the new numbers, by `threads` threads.
__device__ __forceinline__ void renumber_table(const PageBook& k, const Work& w, int64_t U, int b, int i, int threads,
                                               const int32_t* dst, int32_t* table, unsigned* status) {
  const int n = pages_of(k, length_of(k, b, status));
  constexpr int kFlight = 4;
  for (int64_t j0 = i; j0 < k.table_stride; j0 += kFlight * threads) {
    int32_t page[kFlight];
#pragma unroll
    for (int q = 0; q < kFlight; ++q) {
      const int64_t j = j0 + q * threads;
      page[q] = j < k.table_stride ? k.table[b * k.table_stride + j] : 0;
    }
#pragma unroll
    for (int q = 0; q < kFlight; ++q) {
      const int64_t j = j0 + q * threads;
      if (j >= k.table_stride) continue;
      if (j < n) {
        if (!in_pool(k, page[q]))
          record_error(status, kErrIndexRange);
        else if (page[q] >= U && !is_free(w, page[q]))
          page[q] = dst[w.rank[page[q]]];
      }
      table[b * k.table_stride + j] = page[q];
    }
  }
}

__global__ void __launch_bounds__(kScanThreads)
    pages_renumber_kernel(const PageBook k, const Work w, const int page_ctas, const int32_t* src, const int32_t* dst,
                          const int32_t* used, int32_t* table, int32_t* refs, unsigned* status) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t U = *used;
  if (static_cast<int>(blockIdx.x) < page_ctas) {
    renumber_counts(k, w, U, static_cast<int64_t>(blockIdx.x) * kScanThreads + threadIdx.x,
                    static_cast<int64_t>(page_ctas) * kScanThreads, src, refs);
    return;
  }
  for (int b = blockIdx.x - page_ctas; b < k.n_seqs; b += gridDim.x - page_ctas)
    renumber_table(k, w, U, b, threadIdx.x, kScanThreads, dst, table, status);
}

// Copies of pages' contents, bound by memory: 5000 pages of 131 KB 207 us, 6.3 TB/s
// read and written.  A unit is a slice of a pair; a CTA looks at 256 of its units at
// a time, so that a long list of which most is empty costs little, and copies the
// slices that are there.
constexpr int kCopyThreads = 256;
constexpr int kCopyFlight = 4;  // 16-byte loads a thread on their way
constexpr int kSliceBytes = kCopyThreads * kCopyFlight * 16 * 2;  // of k and of v together

__global__ void __launch_bounds__(kCopyThreads)
    pages_copy_kernel(const PagedCache c, const int64_t n, const int32_t* src, const int32_t* dst, const int slices,
                      unsigned* status) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ int64_t unit_s[kCopyThreads];
  __shared__ int2 pair_s[kCopyThreads];
  __shared__ int count_s;
  const int tid = threadIdx.x;
  const int64_t units = n * slices;
  const int64_t page_bytes = static_cast<int64_t>(c.n_kv_heads) * c.page * c.head_dim;
  for (int64_t u0 = blockIdx.x; u0 < units; u0 += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
    __syncthreads();
    if (tid == 0) count_s = 0;
    __syncthreads();
    const int64_t u = u0 + static_cast<int64_t>(tid) * gridDim.x;
    if (u < units) {
      const int64_t i = u / slices;
      const int32_t from = src[i], to = dst[i];
      if (from >= c.n_pages || to >= c.n_pages)
        record_error(status, kErrIndexRange);
      else if (from >= 0 && to >= 0 && from != to) {
        const int at = atomicAdd(&count_s, 1);
        unit_s[at] = u - i * slices;
        pair_s[at] = make_int2(from, to);
      }
    }
    __syncthreads();
    const int count = count_s;
    for (int q = 0; q < count; ++q) {
      const int2 pair = pair_s[q];
      const int64_t slice = unit_s[q];
      const int64_t from = pair.x * page_bytes, to = pair.y * page_bytes;
      const int64_t begin = slice * (kSliceBytes / 2) + tid * 16;
      uint4 x[2][kCopyFlight];
#pragma unroll
      for (int i = 0; i < kCopyFlight; ++i) {
        const int64_t at = begin + i * (kCopyThreads * 16);
        if (at < page_bytes) {
          x[0][i] = __ldcs(reinterpret_cast<const uint4*>(c.k + from + at));
          x[1][i] = __ldcs(reinterpret_cast<const uint4*>(c.v + from + at));
        }
      }
      if (slice == 0)
        for (int h = tid; h < c.n_kv_heads; h += kCopyThreads) {
          const int64_t a = static_cast<int64_t>(pair.x) * c.n_kv_heads + h;
          const int64_t z = static_cast<int64_t>(pair.y) * c.n_kv_heads + h;
          c.k_scale[z] = c.k_scale[a];
          c.v_scale[z] = c.v_scale[a];
        }
#pragma unroll
      for (int i = 0; i < kCopyFlight; ++i) {
        const int64_t at = begin + i * (kCopyThreads * 16);
        if (at < page_bytes) {
          __stcs(reinterpret_cast<uint4*>(c.k + to + at), x[0][i]);
          __stcs(reinterpret_cast<uint4*>(c.v + to + at), x[1][i]);
        }
      }
    }
  }
}

}  // namespace

size_t pages_bytes(int n_seqs, int64_t n_pages) { return work_bytes(n_seqs, n_pages, nullptr, nullptr); }

namespace {

int stretches_of(int64_t n_pages, int shift) { return static_cast<int>((n_pages + (int64_t(1) << shift) - 1) >> shift); }

template <int OP>
cudaError_t launch_change(const PageBook& k, const Lists& x, void* workspace, unsigned* status, cudaStream_t stream) {
  Work w;
  work_bytes(k.n_seqs, k.n_pages, workspace, &w);
  const int shift = stretch_shift(k.n_pages), stretches = stretches_of(k.n_pages, shift);
  const cudaError_t e = launch_pdl(pages_scan_kernel<OP>, dim3(stretches + 1), dim3(kSumThreads), 0, stream, k, w,
                                   shift, stretches, x.want, status);
  if (e != cudaSuccess) return e;
  return launch_pdl(OP == kResize ? pages_resize_kernel : pages_fork_kernel, dim3(k.n_seqs), dim3(kSeqThreads), 0,
                    stream, k, w, shift, stretches, x, status);
}

}  // namespace

cudaError_t launch_pages_resize(const PageBook& k, const int32_t* target, int32_t* pos0, int32_t* src, int32_t* dst,
                                void* workspace, unsigned* status, cudaStream_t stream) {
  return launch_change<kResize>(k, {target, pos0, src, dst}, workspace, status, stream);
}

cudaError_t launch_pages_fork(const PageBook& k, const int32_t* parent, int32_t* src, int32_t* dst, void* workspace,
                              unsigned* status, cudaStream_t stream) {
  return launch_change<kFork>(k, {parent, nullptr, src, dst}, workspace, status, stream);
}

cudaError_t launch_pages_compact(const PageBook& k, int32_t* src, int32_t* dst, int32_t* used, int32_t* table,
                                 int32_t* refs, void* workspace, unsigned* status, int sms, cudaStream_t stream) {
  Work w;
  work_bytes(k.n_seqs, k.n_pages, workspace, &w);
  const int shift = stretch_shift(k.n_pages), stretches = stretches_of(k.n_pages, shift);
  cudaError_t e = launch_pdl(pages_scan_kernel<kCompact>, dim3(stretches), dim3(kSumThreads), 0, stream, k, w, shift,
                             stretches, static_cast<const int32_t*>(nullptr), status);
  if (e != cudaSuccess) return e;
  e = launch_pdl(pages_list_kernel, dim3(stretches), dim3(kScanThreads), 0, stream, k, w, shift, stretches, src, dst,
                 used);
  if (e != cudaSuccess) return e;
  const int64_t most = static_cast<int64_t>(sms) * 8;
  const int64_t page_ctas = (k.n_pages + 4 * kScanThreads - 1) / (4 * kScanThreads), seq_ctas = k.n_seqs;
  const int pc = static_cast<int>(page_ctas < most ? page_ctas : most);
  const int sc = static_cast<int>(seq_ctas < most ? seq_ctas : most);
  return launch_pdl(pages_renumber_kernel, dim3(pc + sc), dim3(kScanThreads), 0, stream, k, w, pc,
                    static_cast<const int32_t*>(src), static_cast<const int32_t*>(dst),
                    static_cast<const int32_t*>(used), table, refs, status);
}

cudaError_t launch_pages_copy(const PagedCache& c, int64_t n, const int32_t* src, const int32_t* dst, unsigned* status,
                              int sms, cudaStream_t stream) {
  if (n <= 0) return cudaSuccess;
  const int64_t page_bytes = static_cast<int64_t>(c.n_kv_heads) * c.page * c.head_dim;
  const int slices = static_cast<int>((page_bytes + kSliceBytes / 2 - 1) / (kSliceBytes / 2));
  const int64_t units = n * slices, most = static_cast<int64_t>(sms) * 8;
  return launch_pdl(pages_copy_kernel, dim3(static_cast<unsigned>(units < most ? units : most)), dim3(kCopyThreads), 0,
                    stream, c, n, src, dst, slices, status);
}

}  // namespace csa
