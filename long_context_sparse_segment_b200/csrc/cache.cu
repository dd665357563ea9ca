// A paged K/V cache whose page table lives on the device (pbs_cache_*).
//
// Bookkeeping (reserve, fork, trim, the compaction's plan) reads a page's
// reference count and a table entry once each: 4 bytes a page and an entry.
// The arrays are small (65536 pages: 256 KB, in L2), so these kernels are
// bound by latency; what one CTA can scan in a few microseconds is not
// spread over several, and every answer is the same on every run: free
// pages are ranked by index, sequences by row. Moving data (append, copy,
// accept, the compaction's moves) reads and writes each byte once.
#include "common.cuh"
#include "decode.h"

namespace pbs {
namespace {

constexpr int kPlanThreads = 1024;  // one CTA for the plans that rank pages
constexpr int kWarps = kPlanThreads / 32;

__device__ __forceinline__ int warp_scan(int x, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Exclusive sums of one value per warp (thread 0 of each brings it); returns
// the warp's own sum and the total. Two barriers.
__device__ __forceinline__ int warps_exclusive(int x, int *sh, int *total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int v = sh[lane], s = warp_scan(v, lane);
    sh[lane] = s - v;
    if (lane == 31) sh[32] = s;
  }
  __syncthreads();
  *total = sh[32];
  return sh[warp];
}

// The run of `n` items that warp w of the plan's CTA ranks: [lo, hi).
__device__ __forceinline__ void warp_run(int n, int *lo, int *hi) {
  const int per = ((n + kWarps - 1) / kWarps + 31) & ~31;
  const int warp = threadIdx.x >> 5;
  *lo = min(n, warp * per);
  *hi = min(n, *lo + per);
}

// ------------------------------------------------------------------ reserve
// While the plan runs, an entry that has to be replaced is kept as -2 - page.
__device__ __forceinline__ int held(int e) { return e <= -2 ? -2 - e : e; }

struct Span {  // table columns that the sequence will write
  int first, last;
};

__device__ __forceinline__ Span write_span(int len, int want, const pbs_cache &c) {
  if (len < 0 || want <= len || (int64_t)want > (int64_t)c.width * c.page) return {0, 0};
  return {len / c.page, (want - 1) / c.page + 1};
}

// ws: the free pages in order [pages], new pages wanted before each sequence
// [seqs]
__global__ void __launch_bounds__(kPlanThreads)
    reserve_kernel(int32_t *table, int32_t *refs, const int32_t *__restrict__ lens,
                   const int32_t *__restrict__ want, int32_t *copy_src, int32_t *copy_dst,
                   pbs_cache c, int32_t *free_list, int32_t *before, int *err) {
  __shared__ int sh[33];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // 1: entries to fill (missing, or shared with somebody who keeps the page)
  for (int s = warp; s < c.seqs; s += kWarps) {
    const int len = lens[s], w = want[s];
    const Span sp = write_span(len, w, c);
    if (lane == 0 && (len < 0 || (w > len && sp.last == 0))) report(err, PBS_ERR_DEVICE_ASSERT);
    int32_t *row = table + (size_t)s * c.width;
    int need = 0;
    for (int j0 = sp.first; j0 < sp.last; j0 += 32) {
      const int j = j0 + lane;
      int e = j < sp.last ? row[j] : 0;
      bool shared = false;
      if (e < -1 || e >= c.pages) report(err, PBS_ERR_DEVICE_ASSERT);
      if (e < -1) *(volatile int32_t *)(row + j) = e = -1;
      const int holders = j < sp.last && e >= 0 && e < c.pages ? refs[e] : 0;
      // a page with several holders: those of earlier rows that write it too
      // will have left it
      unsigned todo = __ballot_sync(0xffffffffu, holders > 1);
      while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const int page = __shfl_sync(0xffffffffu, e, src), col = j0 + src;
        int n = 0;
        for (int r = lane; r < s; r += 32) {
          const Span o = write_span(lens[r], want[r], c);
          if (col >= o.first && col < o.last &&
              held(*(volatile int32_t *)(table + (size_t)r * c.width + col)) == page)
            ++n;
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == src) shared = holders - n > 1;
      }
      const bool fresh = j < sp.last && (e < 0 || shared);
      if (shared) *(volatile int32_t *)(row + j) = -2 - e;
      need += __popc(__ballot_sync(0xffffffffu, fresh));
    }
    if (lane == 0) before[s] = need;
  }
  __syncthreads();
  // 2: new pages wanted before each sequence, and in all
  int lo, hi, wanted;
  {
    warp_run(c.seqs, &lo, &hi);
    int sum = 0;
    for (int i = lo + lane; i < hi; i += 32) sum += before[i];
    sum = __reduce_add_sync(0xffffffffu, sum);
    int at = warps_exclusive(sum, sh, &wanted);
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane, x = i < hi ? before[i] : 0, inc = warp_scan(x, lane);
      if (i < hi) before[i] = at + inc - x;
      at += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  __syncthreads();
  if (wanted == 0) {
    for (int s = tid; s < c.seqs; s += kPlanThreads) copy_src[s] = copy_dst[s] = -1;
    return;
  }
  // 3: the free pages in order
  int total;
  {
    warp_run(c.pages, &lo, &hi);
    int n = 0;
#pragma unroll 4
    for (int i = lo + lane; i < hi; i += 32) n += refs[i] <= 0;
    n = __reduce_add_sync(0xffffffffu, n);
    int at = warps_exclusive(n, sh, &total);
#pragma unroll 4
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      const unsigned m = __ballot_sync(0xffffffffu, i < hi && refs[i] <= 0);
      const int r = at + __popc(m & ((1u << lane) - 1));
      if ((m >> lane & 1) && r < wanted) free_list[r] = i;
      at += __popc(m);
    }
  }
  __syncthreads();
  const bool enough = total >= wanted;
  if (!enough && tid == 0) report(err, PBS_ERR_PAGES);
  // 4: fill the entries, or put them back
  for (int s = warp; s < c.seqs; s += kWarps) {
    const int len = lens[s];
    const Span sp = write_span(len, want[s], c);
    int32_t *row = table + (size_t)s * c.width;
    int at = before[s], from = -1, to = -1;
    for (int j0 = sp.first; j0 < sp.last; j0 += 32) {
      const int j = j0 + lane;
      const int e = j < sp.last ? row[j] : 0;
      const unsigned m = __ballot_sync(0xffffffffu, e < 0);
      if (e < 0 && enough) {
        const int page = free_list[at + __popc(m & ((1u << lane) - 1))];
        row[j] = page;
        refs[page] = 1;
        if (e <= -2) {
          atomicSub(refs + held(e), 1);
          if (j == sp.first && len % c.page) from = held(e), to = page;
        }
      } else if (e <= -2) {
        row[j] = held(e);
      }
      at += __popc(m);
    }
    if (lane == 0) copy_src[s] = from, copy_dst[s] = to;  // column `first` is lane 0's
  }
}

// --------------------------------------------------------------- fork, trim
__global__ void __launch_bounds__(128)
    fork_kernel(int32_t *table, int32_t *refs, int32_t *lens, const int32_t *__restrict__ src,
                const int32_t *__restrict__ dst, int n, pbs_cache c, int *err) {
  const int i = blockIdx.x, tid = threadIdx.x;
  const int s = src[i], t = dst[i];
  if (s < 0 && t < 0) return;
  bool bad = s < 0 || t < 0 || s >= c.seqs || t >= c.seqs;
  for (int j = tid; j < n; j += 128) {
    const int o = dst[j];
    bad |= o >= 0 && ((o == t && j < i) || o == s);
  }
  // a destination named twice is only read by its first pair's block
  if (__syncthreads_or(bad)) {
    if (tid == 0) report(err, PBS_ERR_DEVICE_ASSERT);
    return;
  }
  int32_t *from = table + (size_t)s * c.width, *to = table + (size_t)t * c.width;
  const int len = lens[s];
  const int64_t have = ((int64_t)len + c.page - 1) / c.page;
  bad = len < 0 || have > c.width || lens[t] != 0;
  for (int j = tid; j < c.width; j += 128) bad |= to[j] >= 0;
  for (int j = tid; j < have && j < c.width; j += 128) bad |= from[j] < 0 || from[j] >= c.pages;
  if (__syncthreads_or(bad)) {
    if (tid == 0) report(err, PBS_ERR_DEVICE_ASSERT);
    return;
  }
  for (int j = tid; j < have; j += 128) {
    const int page = from[j];
    to[j] = page;
    atomicAdd(refs + page, 1);
  }
  if (tid == 0) lens[t] = len;
}

__global__ void __launch_bounds__(128)
    trim_kernel(int32_t *table, int32_t *refs, int32_t *lens, const int32_t *__restrict__ keep,
                pbs_cache c, int *err) {
  const int s = blockIdx.x, tid = threadIdx.x, k = keep[s];
  if (k < 0) return;
  const int len = min(max(lens[s], 0), k);
  int32_t *row = table + (size_t)s * c.width;
  for (int j = (int)(((int64_t)len + c.page - 1) / c.page) + tid; j < c.width; j += 128) {
    const int page = row[j];
    if (page < 0) continue;
    row[j] = -1;
    if (page >= c.pages || atomicSub(refs + page, 1) <= 0) {
      if (page < c.pages) atomicAdd(refs + page, 1);  // nobody held it
      report(err, PBS_ERR_DEVICE_ASSERT);
    }
  }
  __syncthreads();
  if (tid == 0) lens[s] = len;
}

// ------------------------------------------------------------------ compact
// ws: each page's new place [pages], the number of moves [1]
__global__ void __launch_bounds__(kPlanThreads)
    compact_kernel(int32_t *refs, int32_t *src, int32_t *dst, pbs_cache c, int32_t *to,
                   int32_t *moves) {
  __shared__ int sh[33];
  const int tid = threadIdx.x, lane = tid & 31;
  int lo, hi, live, n, skip;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  warp_run(c.pages, &lo, &hi);
  n = 0;
#pragma unroll 4
  for (int i = lo + lane; i < hi; i += 32) {
    n += refs[i] > 0;
    to[i] = i, src[i] = -1, dst[i] = -1;
  }
  n = __reduce_add_sync(0xffffffffu, n);
  warps_exclusive(n, sh, &live);
  __syncthreads();
  // movers: held pages from `live` on; holes: free pages below it; equally many
  int mv = 0, ho = 0;
#pragma unroll 4
  for (int i = lo + lane; i < hi; i += 32) {
    const bool held_page = refs[i] > 0;
    mv += held_page && i >= live;
    ho += !held_page && i < live;
  }
  mv = __reduce_add_sync(0xffffffffu, mv);
  ho = __reduce_add_sync(0xffffffffu, ho);
  int at_mv = warps_exclusive(mv, sh, &n);
  __syncthreads();
  int at_ho = warps_exclusive(ho, sh, &skip);
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const bool held_page = i < hi && refs[i] > 0;
    const unsigned a = __ballot_sync(0xffffffffu, held_page && i >= live);
    const unsigned b = __ballot_sync(0xffffffffu, i < hi && !held_page && i < live);
    const unsigned below = (1u << lane) - 1;
    if (a >> lane & 1) src[at_mv + __popc(a & below)] = i;
    if (b >> lane & 1) dst[at_ho + __popc(b & below)] = i;
    at_mv += __popc(a), at_ho += __popc(b);
  }
  __syncthreads();
  for (int i = tid; i < n; i += kPlanThreads) {
    const int a = src[i], b = dst[i];
    to[a] = b;
    refs[b] = refs[a];
    refs[a] = 0;
  }
  if (tid == 0) *moves = n;
}

// --------------------------------------------------------------- page copies
// Pairs up to this many are checked against each other by every CTA (4 KB of
// reads from L2); more go through an owner table, a memset and a launch more:
// 512 pairs of 4 KB take 5.5 us scanned and 5.0 by the table, but the host 5 us
// longer; 8000 pairs 92 us scanned and 58 by the table. The copies themselves
// run at the copy rate: 96 pages of 32 layers (1.6 GB read and written) 249 us.
constexpr int kScanPairs = 512;
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;  // 16-byte loads in flight per thread
constexpr int kPiece = kCopyThreads * kCopyUnroll;  // 16-byte words a CTA copies at a time

__global__ void __launch_bounds__(256)
    owner_kernel(const int32_t *__restrict__ dst, int n, int pages, int32_t *owner) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n && dst[i] >= 0 && dst[i] < pages) atomicMin((unsigned *)owner + dst[i], (unsigned)i);
}

// The CTAs walk the pieces of every (pair, pool, layer). COMPACT: the pairs are
// a compaction's, sound by construction, `count` of them, and the CTAs first
// put the pages' new places `to` into the table; the kernel is launched while
// the plan still runs and waits for it here.
template <bool COMPACT>
__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(uint4 *k, uint4 *v, const int32_t *src, const int32_t *dst, int n,
                const int32_t *count, const int32_t *to_page, int32_t *table,
                const int32_t *owner, pbs_cache c, int64_t page_words, int pieces, int *err) {
  const int tid = threadIdx.x;
  const int64_t per_pair = 2LL * c.layers * pieces;
  if (COMPACT) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t entries = (int64_t)c.seqs * c.width;
    for (int64_t i = (int64_t)blockIdx.x * kCopyThreads + tid; i < entries;
         i += (int64_t)gridDim.x * kCopyThreads) {
      const int e = table[i];
      if (e < 0 || e >= c.pages) continue;
      const int t = to_page[e];
      if (t != e) table[i] = t;
    }
  }
  const int pairs = COMPACT ? *count : n;
  for (int64_t w = blockIdx.x; w < per_pair * pairs; w += gridDim.x) {
    const int i = (int)(w / per_pair), part = (int)(w - i * per_pair);
    const int a = src[i], b = dst[i];
    if (a < 0 && b < 0) continue;
    if (!COMPACT) {
      bool bad = a < 0 || b < 0 || a >= c.pages || b >= c.pages;
      if (!bad && owner) {
        bad = owner[b] != i || owner[a] != -1;
      } else if (!bad) {
        for (int j = tid; j < n; j += kCopyThreads) {
          const int o = dst[j];
          bad |= o >= 0 && ((o == b && j < i) || o == a);
        }
      }
      if (__syncthreads_or(bad)) {
        if (tid == 0) report(err, PBS_ERR_DEVICE_ASSERT);
        continue;
      }
    }
    const int piece = part % pieces, lp = part / pieces;
    uint4 *pool = (lp & 1) ? v : k;
    const int64_t layer = (int64_t)(lp >> 1) * c.pages;
    const uint4 *from = pool + (layer + a) * page_words;
    uint4 *to = pool + (layer + b) * page_words;
    const int64_t w0 = (int64_t)piece * kPiece + tid;
    uint4 r[kCopyUnroll];
#pragma unroll
    for (int x = 0; x < kCopyUnroll; ++x)
      if (w0 + x * kCopyThreads < page_words) r[x] = from[w0 + x * kCopyThreads];
#pragma unroll
    for (int x = 0; x < kCopyUnroll; ++x)
      if (w0 + x * kCopyThreads < page_words) to[w0 + x * kCopyThreads] = r[x];
  }
}

// ------------------------------------------------------------ append, accept
// The word offset of token t of sequence s in one layer's pool (head 0, first
// word), or -1 for a token that no page holds; `write`: or, with c.refs, one
// whose page several sequences hold.
__device__ __forceinline__ int64_t token_word(const int32_t *row, int64_t t, const pbs_cache &c,
                                              int words, bool write) {
  if (t < 0 || t > 0x7fffffff) return -1;
  const unsigned j = (unsigned)t / (unsigned)c.page;
  if (j >= (unsigned)c.width) return -1;
  const int page = row[j];
  if (page < 0 || page >= c.pages) return -1;
  if (write && c.refs && c.refs[page] > 1) return -1;
  return ((int64_t)page * c.hkv * c.page + ((unsigned)t - j * c.page)) * words;
}

// A thread moves one 16-byte word of a K row and of the V row beside it.
__global__ void __launch_bounds__(256)
    append_kernel(pbs_rows k, pbs_rows v, int n, uint4 *kp, uint4 *vp,
                  const int32_t *__restrict__ table, const int32_t *__restrict__ start,
                  const int32_t *__restrict__ count, pbs_cache c, int64_t total, int *err) {
  const int words = c.d / 8;
  for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < total;
       at += (int64_t)gridDim.x * 256) {
    const int w = (int)(at % words);
    int64_t x = at / words;
    const int i = (int)(x % n);
    x /= n;
    const int h = (int)(x % c.hkv);
    x /= c.hkv;
    const int s = (int)(x % c.seqs), l = (int)(x / c.seqs);
    if (count && i >= count[s]) continue;
    const int64_t o =
        token_word(table + (size_t)s * c.width, (int64_t)start[s] + i, c, words, true);
    if (o < 0) {
      report(err, PBS_ERR_DEVICE_ASSERT);
      continue;
    }
    const int64_t to = o + ((int64_t)l * c.pages * c.hkv + h) * c.page * words + w;
    const uint16_t *ks = (const uint16_t *)k.p + l * k.layer + s * k.batch + h * k.head + i * k.row;
    const uint16_t *vs = (const uint16_t *)v.p + l * v.layer + s * v.batch + h * v.head + i * v.row;
    const uint4 a = reinterpret_cast<const uint4 *>(ks)[w];
    const uint4 b = reinterpret_cast<const uint4 *>(vs)[w];
    kp[to] = a;
    vp[to] = b;
  }
}

// Rows move down inside a sequence: token start + path[i] to start + i, path
// ascending, so a row that is written is read by no later one. A thread owns
// one 16-byte column of one pool and layer and takes the rows in order,
// kRows at a time: all loads of a group before its stores, and no other
// thread touches the column. The rows' places are looked up once per CTA (in
// every thread, between its loads: 12.5 us instead of 6 for 32 sequences and
// 32 layers); then it is bound by the latency of four dependent reads.
constexpr int kRows = 8;
constexpr int kAcceptThreads = 128;  // rows whose places are held at a time, too

// Row i of an accepted path `p`, which moves from token st + p[i] to st + i: the
// words of both. False for a row that may not move.
__device__ __forceinline__ bool accept_row(const int32_t *row, const int32_t *__restrict__ p, int i,
                                           int st, const pbs_cache &c, int words, int64_t *from,
                                           int64_t *to) {
  const int x = __ldg(p + i), before = i > 0 ? __ldg(p + i - 1) : -1;
  if (x < 0 || before >= x) return false;
  *from = token_word(row, (int64_t)st + x, c, words, false);
  *to = token_word(row, (int64_t)st + i, c, words, true);
  const bool good = *from >= 0 && *to >= 0;
  if (x == i) *to = -1;  // stays
  return good;
}

__global__ void __launch_bounds__(kAcceptThreads)
    accept_kernel(uint4 *k, uint4 *v, const int32_t *__restrict__ table,
                  const int32_t *__restrict__ start, const int32_t *__restrict__ path,
                  const int32_t *__restrict__ count, int32_t *lens, int tree, pbs_cache c,
                  int col_blocks, int *err) {
  __shared__ int64_t from[kAcceptThreads], to[kAcceptThreads];  // to -1: stays
  const int s = blockIdx.y, lp = blockIdx.x / col_blocks, tid = threadIdx.x;
  const int n = count ? min(__ldg(count + s), tree) : tree;
  const int st = __ldg(start + s);
  const int32_t *row = table + (size_t)s * c.width, *p = path + (size_t)s * tree;
  const int words = c.d / 8;
  // the places of rows i0 .. i0 + 127; false for a row that may not move
  auto look_up = [&](int i0) {
    return i0 + tid >= n || accept_row(row, p, i0 + tid, st, c, words, &from[tid], &to[tid]);
  };
  bool bad = st < 0;
  for (int i0 = (n - 1) / kAcceptThreads * kAcceptThreads; i0 >= 0; i0 -= kAcceptThreads)
    bad |= !look_up(i0);  // the first rows last: their places stay
  if (__syncthreads_or(bad)) {
    if (tid == 0) report(err, PBS_ERR_DEVICE_ASSERT);
    return;
  }
  if (lens && blockIdx.x == 0 && tid == 0) lens[s] = st + max(n, 0);
  const int col = (blockIdx.x % col_blocks) * kAcceptThreads + tid;
  const int h = col / words, w = col - h * words;
  uint4 *pool = ((lp & 1) ? v : k) +
                ((int64_t)(lp >> 1) * c.pages * c.hkv + h) * c.page * words + w;
  for (int i0 = 0; i0 < n; i0 += kAcceptThreads) {
    if (i0 > 0) {
      __syncthreads();
      look_up(i0);
      __syncthreads();
    }
    if (col >= c.hkv * words) continue;
    for (int j0 = 0; j0 < min(n - i0, kAcceptThreads); j0 += kRows) {
      uint4 r[kRows];
#pragma unroll
      for (int x = 0; x < kRows; ++x)
        if (i0 + j0 + x < n && to[j0 + x] >= 0) r[x] = pool[from[j0 + x]];
#pragma unroll
      for (int x = 0; x < kRows; ++x)
        if (i0 + j0 + x < n && to[j0 + x] >= 0) pool[to[j0 + x]] = r[x];
    }
  }
}

// The lengths behind an acceptance whose `start` or `count` is `lens` itself: the
// rows' kernel reads those in every block of a sequence until its end, so the
// lengths are written behind it, where the path is good (one block a sequence, 2 us);
// and behind one of no rows at all.
__global__ void __launch_bounds__(kAcceptThreads)
    accept_lens_kernel(const int32_t *__restrict__ table, const int32_t *start,
                       const int32_t *__restrict__ path, const int32_t *count, int32_t *lens,
                       int tree, pbs_cache c, int *err) {
  const int s = blockIdx.x;
  const int n = count ? min(count[s], tree) : tree, st = start[s];
  bool bad = st < 0;
  if (bad && threadIdx.x == 0) report(err, PBS_ERR_DEVICE_ASSERT);
  for (int i = threadIdx.x; i < n; i += kAcceptThreads) {
    int64_t from, to;
    bad |= !accept_row(table + (size_t)s * c.width, path + (size_t)s * tree, i, st, c, c.d / 8,
                       &from, &to);
  }
  if (!__syncthreads_or(bad) && threadIdx.x == 0) lens[s] = st + max(n, 0);
}

bool cache_ok(const pbs_cache &c) {
  return c.layers >= 1 && c.pages >= 1 && c.hkv >= 1 && c.page >= 1 && c.d >= 8 && c.d % 8 == 0 &&
         c.seqs >= 0 && c.width >= 1 && c.pages < (1 << 30) && c.hkv <= 65536 &&
         c.page <= 65536 && c.d <= 65536 && c.layers <= 16384 &&
         (int64_t)c.seqs * c.width < (1ll << 31);
}

bool ints_ok(const void *p) { return p && ((uintptr_t)p & 3u) == 0; }
bool pool_ok(const void *p) { return p && ((uintptr_t)p & 15u) == 0; }
pbs_status done() { return cudaGetLastError() == cudaSuccess ? PBS_OK : PBS_ERR_CUDA; }

int64_t pool_bytes(const pbs_cache &c) {
  return 2ll * c.layers * c.pages * c.hkv * c.page * c.d;
}
int64_t page_words(const pbs_cache &c) { return (int64_t)c.hkv * c.page * c.d / 8; }
int pieces(const pbs_cache &c) { return (int)ceil_div(page_words(c), kPiece); }

unsigned copy_grid(const pbs_cache &c, int64_t pairs) {
  // eight CTAs of 256 threads fit an SM
  const int64_t w = 2LL * c.layers * pieces(c) * pairs, most = 8LL * 4 * sm_count_cached();
  return (unsigned)(w < most ? w : most);
}

}  // namespace
}  // namespace pbs

using namespace pbs;

extern "C" {

size_t pbs_cache_workspace_bytes(pbs_cache c, int op, int n) {
  if (!cache_ok(c)) return 0;
  switch (op) {
    case PBS_CACHE_RESERVE:
      return 4 * ((size_t)c.pages + c.seqs);
    case PBS_CACHE_COPY:
      return n > kScanPairs ? 4 * (size_t)c.pages : 0;
    case PBS_CACHE_COMPACT:
      return 4 * ((size_t)c.pages + 1);
    default:
      return 0;
  }
}

pbs_status pbs_cache_reserve(int32_t *table, int32_t *refs, const int32_t *lens,
                             const int32_t *want, int32_t *copy_src, int32_t *copy_dst,
                             pbs_cache c, void *ws, size_t ws_bytes, pbs_stream_t st) {
  if (!cache_ok(c)) return PBS_ERR_INVALID_ARG;
  if (c.seqs == 0) return PBS_OK;
  if (!ints_ok(table) || !ints_ok(refs) || !ints_ok(lens) || !ints_ok(want) ||
      !ints_ok(copy_src) || !ints_ok(copy_dst) || !ints_ok(ws))
    return PBS_ERR_INVALID_ARG;
  if (ws_bytes < pbs_cache_workspace_bytes(c, PBS_CACHE_RESERVE, 0)) return PBS_ERR_WORKSPACE;
  reserve_kernel<<<1, kPlanThreads, 0, (cudaStream_t)st>>>(table, refs, lens, want, copy_src,
                                                          copy_dst, c, (int32_t *)ws,
                                                          (int32_t *)ws + c.pages, error_word());
  return done();
}

pbs_status pbs_cache_append(pbs_rows k, pbs_rows v, int n, void *k_pages, void *v_pages,
                            const int32_t *table, const int32_t *start, const int32_t *count,
                            pbs_cache c, pbs_stream_t st) {
  if (!cache_ok(c) || n < 0) return PBS_ERR_INVALID_ARG;
  if (c.seqs == 0 || n == 0) return PBS_OK;
  if (!rows_ok(k, 2) || !rows_ok(v, 2) || !pool_ok(k_pages) || !pool_ok(v_pages) ||
      k_pages == v_pages || !ints_ok(table) || !ints_ok(start) || (count && !ints_ok(count)) ||
      (c.refs && !ints_ok(c.refs)))
    return PBS_ERR_INVALID_ARG;
  // the pools, apart from one another, hold neither the rows nor what says where
  // they go
  const int64_t pool = pool_bytes(c), each = 4ll * c.seqs;
  bool meet = bytes_meet(k_pages, pool, v_pages, pool);
  for (const void *to : {(const void *)k_pages, (const void *)v_pages}) {
    for (const pbs_rows &x : {k, v}) {
      const RowSet rows{x, c.seqs, c.hkv, n, c.d, 2};
      const int64_t up = 2 * x.layer * (c.layers - 1);  // bytes from the first layer to the last
      meet |= bytes_meet(rows.low() + (up < 0 ? up : 0), rows.bytes() + (up < 0 ? -up : up), to,
                         pool);
    }
    meet |= bytes_meet(to, pool, table, each * c.width) || bytes_meet(to, pool, start, each) ||
            bytes_meet(to, pool, count, each) || bytes_meet(to, pool, c.refs, 4ll * c.pages);
  }
  if (meet) return PBS_ERR_INVALID_ARG;
  const int64_t total = (int64_t)c.layers * c.seqs * c.hkv * n * (c.d / 8);
  const int64_t blocks = ceil_div(total, 256), most = 32 * sm_count_cached();
  append_kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, (cudaStream_t)st>>>(
      k, v, n, (uint4 *)k_pages, (uint4 *)v_pages, table, start, count, c, total, error_word());
  return done();
}

pbs_status pbs_cache_copy(void *k_pages, void *v_pages, const int32_t *src, const int32_t *dst,
                          int n, pbs_cache c, void *ws, size_t ws_bytes, pbs_stream_t st) {
  if (!cache_ok(c) || n < 0) return PBS_ERR_INVALID_ARG;
  if (n == 0) return PBS_OK;
  if (!pool_ok(k_pages) || !pool_ok(v_pages) || !ints_ok(src) || !ints_ok(dst))
    return PBS_ERR_INVALID_ARG;
  const size_t need = pbs_cache_workspace_bytes(c, PBS_CACHE_COPY, n);
  if (need && !ints_ok(ws)) return PBS_ERR_INVALID_ARG;
  if (ws_bytes < need) return PBS_ERR_WORKSPACE;
  cudaStream_t cs = (cudaStream_t)st;
  int32_t *owner = nullptr;
  if (need) {
    owner = (int32_t *)ws;
    if (cudaMemsetAsync(owner, 0xff, need, cs) != cudaSuccess) return PBS_ERR_CUDA;
    owner_kernel<<<n / 256 + 1, 256, 0, cs>>>(dst, n, c.pages, owner);
  }
  copy_kernel<false><<<copy_grid(c, n), kCopyThreads, 0, cs>>>(
      (uint4 *)k_pages, (uint4 *)v_pages, src, dst, n, nullptr, nullptr, nullptr, owner, c,
      page_words(c), pieces(c), error_word());
  return done();
}

pbs_status pbs_cache_fork(int32_t *table, int32_t *refs, int32_t *lens, const int32_t *src,
                          const int32_t *dst, int n, pbs_cache c, pbs_stream_t st) {
  if (!cache_ok(c) || n < 0) return PBS_ERR_INVALID_ARG;
  if (n == 0 || c.seqs == 0) return PBS_OK;
  if (!ints_ok(table) || !ints_ok(refs) || !ints_ok(lens) || !ints_ok(src) || !ints_ok(dst))
    return PBS_ERR_INVALID_ARG;
  fork_kernel<<<n, 128, 0, (cudaStream_t)st>>>(table, refs, lens, src, dst, n, c, error_word());
  return done();
}

pbs_status pbs_cache_trim(int32_t *table, int32_t *refs, int32_t *lens, const int32_t *keep,
                          pbs_cache c, pbs_stream_t st) {
  if (!cache_ok(c)) return PBS_ERR_INVALID_ARG;
  if (c.seqs == 0) return PBS_OK;
  if (!ints_ok(table) || !ints_ok(refs) || !ints_ok(lens) || !ints_ok(keep))
    return PBS_ERR_INVALID_ARG;
  trim_kernel<<<c.seqs, 128, 0, (cudaStream_t)st>>>(table, refs, lens, keep, c, error_word());
  return done();
}

pbs_status pbs_cache_compact(void *k_pages, void *v_pages, int32_t *table, int32_t *refs,
                             int32_t *move_src, int32_t *move_dst, pbs_cache c, void *ws,
                             size_t ws_bytes, pbs_stream_t st) {
  if (!cache_ok(c)) return PBS_ERR_INVALID_ARG;
  if (!pool_ok(k_pages) || !pool_ok(v_pages) || (c.seqs > 0 && !ints_ok(table)) ||
      !ints_ok(refs) || !ints_ok(move_src) || !ints_ok(move_dst) || !ints_ok(ws))
    return PBS_ERR_INVALID_ARG;
  if (ws_bytes < pbs_cache_workspace_bytes(c, PBS_CACHE_COMPACT, 0)) return PBS_ERR_WORKSPACE;
  cudaStream_t cs = (cudaStream_t)st;
  int32_t *to = (int32_t *)ws, *moves = to + c.pages;
  compact_kernel<<<1, kPlanThreads, 0, cs>>>(refs, move_src, move_dst, c, to, moves);
  if (cudaGetLastError() != cudaSuccess) return PBS_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(copy_grid(c, c.pages / 2 + 1));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = cs;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(
      &cfg, copy_kernel<true>, (uint4 *)k_pages, (uint4 *)v_pages, (const int32_t *)move_src,
      (const int32_t *)move_dst, c.pages, (const int32_t *)moves, (const int32_t *)to, table,
      (const int32_t *)nullptr, c, page_words(c), pieces(c), error_word());
  return e == cudaSuccess ? PBS_OK : PBS_ERR_CUDA;
}

pbs_status pbs_cache_accept(void *k_pages, void *v_pages, const int32_t *table,
                            const int32_t *start, const int32_t *path, const int32_t *count,
                            int32_t *lens, int tree, pbs_cache c, pbs_stream_t st) {
  if (!cache_ok(c) || tree < 0) return PBS_ERR_INVALID_ARG;
  if (c.seqs > 65535) return PBS_ERR_UNSUPPORTED;
  if (c.seqs == 0) return PBS_OK;
  if (tree == 0) {  // nothing moves, the lengths are the starts
    if (!lens || lens == start) return PBS_OK;
    const int64_t each = 4ll * c.seqs;
    if (!ints_ok(start) || !ints_ok(lens) || bytes_meet(lens, each, start, each))
      return PBS_ERR_INVALID_ARG;
    accept_lens_kernel<<<c.seqs, kAcceptThreads, 0, (cudaStream_t)st>>>(
        nullptr, start, nullptr, nullptr, lens, 0, c, error_word());
    return done();
  }
  // one pool for both would be moved twice at once
  if (!pool_ok(k_pages) || !pool_ok(v_pages) || k_pages == v_pages || !ints_ok(table) ||
      !ints_ok(start) || !ints_ok(path) || (count && !ints_ok(count)) || (lens && !ints_ok(lens)) ||
      (c.refs && !ints_ok(c.refs)))
    return PBS_ERR_INVALID_ARG;
  // lens may be start or count, but otherwise nothing that other sequences read
  const int64_t each = 4ll * c.seqs, pool = pool_bytes(c);
  if (bytes_meet(k_pages, pool, v_pages, pool) ||
      (lens != start && bytes_meet(lens, each, start, each)) ||
      (lens != count && bytes_meet(lens, each, count, each)) ||
      bytes_meet(lens, each, path, each * tree) || bytes_meet(lens, each, table, each * c.width) ||
      bytes_meet(lens, each, c.refs, 4ll * c.pages))
    return PBS_ERR_INVALID_ARG;
  const int col_blocks = (int)ceil_div((int64_t)c.hkv * (c.d / 8), kAcceptThreads);
  const int64_t gx = 2LL * c.layers * col_blocks;
  if (gx > 0x7fffffff) return PBS_ERR_UNSUPPORTED;
  const bool behind = lens && (lens == start || lens == count);
  accept_kernel<<<dim3((unsigned)gx, c.seqs), kAcceptThreads, 0, (cudaStream_t)st>>>(
      (uint4 *)k_pages, (uint4 *)v_pages, table, start, path, count, behind ? nullptr : lens, tree,
      c, col_blocks, error_word());
  if (behind)
    accept_lens_kernel<<<c.seqs, kAcceptThreads, 0, (cudaStream_t)st>>>(table, start, path, count,
                                                                       lens, tree, c,
                                                                       error_word());
  return done();
}

}  // extern "C"
