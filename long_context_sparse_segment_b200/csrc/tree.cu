// Attention of a tree of drafted tokens over a paged K/V cache
// (pbs_tree_mask, pbs_tree_attn).
//
// Draft i of sequence s sees the start[s] cached tokens and the drafts whose
// bit its mask row has: o_i = sum_j softmax_j(sigma q_i . k_j) v_j. The G =
// hq / hkv query heads of a KV head share its K and V, so the rows of one
// work item are (draft i, head g), row r = i G + g: every cached row is read
// once per item and serves them all. With few rows this is bound by reading
// the cache.
//
// This kernel: up to 16 rows an item, warp MMA. Eight warps take tiles of 64
// keys, four warps a tile (16 keys each), each with its own maximum, sum and
// output, joined when the item ends; one warp more brings the tiles by TMA,
// page by page, into a ring. The eight are one CTA, whose halves take the tiles
// of an item in turn, or two CTAs an SM with half the ring each, so that one
// item's beginning and end go beside the other CTA's tiles (mma_warps has the
// rule, with both sides). A unit keeps a warp
// busy for 1,450 cycles, two warps a scheduler, while its 32 KB (d = 128) take
// 1,450 to arrive at the copy rate: the tensor core of tcgen05 would have 4 to
// 16 of its 128 rows to do. Measured: a new token of each of 48 sequences of
// 100 to 32768 tokens (3.29 GB of K and V) 490-502 us, 6.6-6.7 TB/s (the copy
// rate is 6.56); one sequence of 8192 tokens 16 us, of which the bytes are 5
// and the rest launches, the run's start and the combining kernel.
#include <stdlib.h>
#include <string.h>

#include "internal.h"
#include "tree_tc.h"

namespace pbs {
namespace {

using namespace tree;

// ------------------------------------------------------------- warp-MMA kernel
constexpr int kKeys = 64;       // keys of a unit

template <int D, int W>  // W: consumer warps
struct MmaCfg {
  static constexpr int ROWS = 16;
  static constexpr uint32_t KV = kKeys * D * 2;   // bytes of a K or V tile
  // 192 KB in flight an SM (128 KB: 6 % slower on a ragged batch, 64 KB: 30 %);
  // even with two halves: a stage stays with one of them
  static constexpr int ST = (D == 128 ? 6 : 12) * W / 8;
  static constexpr int CTAS = 8 / W;              // an SM
  static constexpr int THREADS = 32 * (W + 1);
  static constexpr int RJ = 4;                    // rows joined at a time
  static constexpr int PAD = 4;                   // floats behind a joined row
  static constexpr size_t JOIN = (size_t)W * RJ * (D + PAD) * 4;
  struct Bars {
    uint64_t full[ST], empty[ST], q_full[2], q_empty[2];
    int abort;
    int bad[W];
    Segment g[2];
    float2 ml[W][ROWS];
    int sum[W + 1];
  };
  static constexpr size_t SMEM = 2 * KV * ST + 2 * ROWS * D * 2 + JOIN + sizeof(Bars);
  // 228 KB an SM, of which every CTA takes 1 KB more than it asks for
  static_assert((SMEM + 1024) * CTAS <= 233472, "shared memory");
};

template <typename T, int D, int W>
__global__ void __launch_bounds__(MmaCfg<D, W>::THREADS, MmaCfg<D, W>::CTAS)
    tree_mma_kernel(const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TreeArgs a) {
  using C = MmaCfg<D, W>;
  constexpr int ST = C::ST, ROWS = C::ROWS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];  // the swizzle's alignment
  uint8_t *ring = smem_raw;                          // [ST][K tile, V tile]
  T *sQ = reinterpret_cast<T *>(ring + 2 * C::KV * ST);  // [2][ROWS][D]
  float *join = reinterpret_cast<float *>(sQ + 2 * ROWS * D);
  auto *bar = reinterpret_cast<typename C::Bars *>(reinterpret_cast<uint8_t *>(join) + C::JOIN);
  volatile int *abort = &bar->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(ring) & 1023u) {  // never: the declaration's alignment
    if (tid == 0) report(a.err, PBS_ERR_DEVICE_ASSERT);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) mbar_init(&bar->full[i], 1), mbar_init(&bar->empty[i], 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->q_full[i], 33);  // each lane's copies, and the segment
      mbar_init(&bar->q_empty[i], W);
    }
    bar->abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  wait_previous();
  allow_next();  // not before the wait: the next kernel looks at the lengths at once
  Place place;
  if (!find_place<ROWS, kKeys, C::THREADS>(a, bar->sum, &place)) return;
  // r / G of a row r < 16 is r by_g >> 16
  const unsigned by_g = 65536u / a.G + 1;
  // a tile in shared memory: [piece of a page][64-column half][row][128 bytes]
  const int box = min(a.page, kKeys);

  if (warp == W) {
    // ------------------------------------------------------------- producer
    // Finds the segments, brings each one's Q rows (a segment ahead of the
    // consumers, as the ring allows) and its units: up to 4 pieces of pages,
    // K and V, one lane each. Rows of a page behind the last token come along;
    // pages behind it do not. The table is read 32 entries at a time, 32 early:
    // one entry a unit early held a unit to the latency of L2 (700 cycles, more
    // than the 64 keys of d = 64 take to arrive).
    Segment g;
    Walk<ROWS, kKeys> walk(a, place, &g);
    const int kv = lane & 1, piece = lane >> 1, shift = 31 - __clz(a.page);
    const bool mine = piece < kKeys / box;
    int it = 0, seg = 0;
    if (lane == 0) prefetch_map(&tmK), prefetch_map(&tmV);
    for (bool more = true, ok = true; more && ok; ++seg) {
      more = walk.next(a, &g);
      const int slot = seg & 1;
      if (seg >= 2 && !mbar_wait_warp(&bar->q_empty[slot], (seg / 2 - 1) & 1, abort, a.err, 12))
        break;
      if (lane == 0) {
        if (!more) g.count = 0;  // the end
        bar->g[slot] = g;
        mbar_arrive(&bar->q_full[slot]);
      }
      if (more) {
        const int n = g.count * a.G * (D / 8);
        for (int x = lane; x < n; x += 32) {  // rows behind: anything
          const int r = x / (D / 8), ch = x % (D / 8);
          const int i = r * by_g >> 16, hd = g.h * a.G + r - i * a.G;
          cp_async16(sQ + slot * ROWS * D + swz<D>(r, ch * 8),
                     (const T *)a.q.p + (int64_t)g.s * a.q.batch + hd * a.q.head + i * a.q.row +
                         ch * 8);
        }
      }
      cp_async_mbar_arrive(&bar->q_full[slot]);
      if (!more) break;
      const int len = g.start + g.count;
      const int32_t *row = a.table + (size_t)g.s * a.width;
      int t = g.k0 * kKeys + piece * box;
      const int last = (min(len, g.k1 * kKeys) - 1) >> shift;  // column
      int col = g.k0 * kKeys >> shift;                         // of lane 0's entry
      auto entry = [&](int c) { return c + lane <= last ? row[c + lane] : 0; };
      int held = entry(col), ahead = entry(col + 32);
      for (int k = g.k0; k < g.k1; ++k, ++it, t += kKeys) {
        const int st = it % ST;
        const bool load = mine && t < len;
        // a unit's columns never straddle the 32: both begin at multiples of
        // the columns of a unit
        if ((k * kKeys >> shift) - col >= 32) col += 32, held = ahead, ahead = entry(col + 32);
        int page = __shfl_sync(0xffffffffu, held, ((t >> shift) - col) & 31);
        if (load && (page < 0 || page >= a.pages)) {
          report(a.err, PBS_ERR_DEVICE_ASSERT);
          page = 0;
        }
        const int y = (page * a.hkv + g.h) * a.page + (t & (a.page - 1));
        const int boxes = __popc(__ballot_sync(0xffffffffu, load));
        if (it >= ST && !mbar_wait_warp(&bar->empty[st], (it / ST - 1) & 1, abort, a.err, 11)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_expect_tx(&bar->full[st], boxes * box * D * 2);
        __syncwarp();
        if (load && !(a.fault && it == 0 && kv == 0))
          tma_load_3d(ring + (size_t)(2 * st + kv) * C::KV + piece * box * D * 2,
                      kv ? &tmV : &tmK, &bar->full[st], 0, y, 0);
        __syncwarp();
      }
    }
    // every copy started here lands before the CTA exits
    cp_async_wait_all();
    int never = 0;
    for (int i = it > ST ? it - ST : 0; i < it; ++i)
      if (!(a.fault && i == 0)) mbar_wait(&bar->full[i % ST], (i / ST) & 1, &never, nullptr);
    return;
  }

  // --------------------------------------------------------------- consumers
  const int half_id = warp >> 2, key16 = (warp & 3) * 16;
  const int gr = lane >> 2, qc = (lane & 3) * 2;
  // The consumers meet in named barriers (a bounded mbarrier wait instead costs
  // 0.2 us each, up to eight an item). So a warp whose wait ran out goes on to
  // every barrier of the segment, and all leave together at the next one.
  auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 * W) : "memory"); };
  bool failed = false;
  auto agree = [&]() {
    int any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, %2, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"((int)failed), "n"(32 * W)
        : "memory");
    failed = any != 0;
  };
  const uint32_t half_bytes = box * 128;  // from one column half to the other
  const uint32_t key_bytes = key16 / box * (box * D * 2) + key16 % box * 128;
  int it = 0;
  for (int seg = 0;; ++seg) {
    if (!mbar_wait_warp(&bar->q_full[seg & 1], seg >> 1 & 1, abort, a.err, 42)) failed = true;
    agree();  // also: the join buffer's last readers are through
    if (failed) return;
    const Segment g = bar->g[seg & 1];
    if (g.count == 0) return;
    const int rows = g.count * a.G;  // one row tile an item
    const int len = g.start + g.count;
    int draft[2];  // of this thread's rows
#pragma unroll
    for (int x = 0; x < 2; ++x) draft[x] = min((int)((gr + 8 * x) * by_g >> 16), g.count - 1);
    uint32_t q[D / 16][4];
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      ldsm_x4(q[kk], sQ + (seg & 1) * ROWS * D + swz<D>(lane & 15, kk * 16 + ((lane >> 4) << 3)));
    warp_arrive(&bar->q_empty[seg & 1], lane);
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    bool bad = false;
    for (int k = g.k0; k < g.k1; ++k, ++it) {
      if (W == 8 && (it & 1) != half_id) continue;
      const int st = it % ST;
      if (!failed && !mbar_wait_warp(&bar->full[st], (it / ST) & 1, abort, a.err, 41))
        failed = true;
      const uint8_t *tK = ring + (size_t)(2 * st) * C::KV + key_bytes, *tV = tK + C::KV;
      const int key0 = k * kKeys + key16;  // this warp's 16 keys
      if (key0 < len && !failed) {
        // S = Q K^T
        float s[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
        {
          const int row = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const int ch = kk * 2 + ((lane >> 3) & 1);
            uint32_t b[4];
            ldsm_x4(b, tK + (ch >> 3) * half_bytes + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
            Two<T>::mma(s[0], q[kk], b[0], b[1]);
            Two<T>::mma(s[1], q[kk], b[2], b[3]);
          }
        }
        // masks: drafts, and keys behind the last token
        const bool edge = key0 + 16 > g.start;
        if (edge) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t seen = seen_word(a, g, draft[x], key0) >> qc;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (!(seen >> (n * 8 + e) & 1)) s[n][2 * x + e] = -INFINITY;
          }
        }
        // running reference (the maximum, or below it); P rounded to 16 bits (see
        // tree.cuh)
        uint32_t p[4];
        float alpha[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float t = fmaxf(fmaxf(s[0][2 * x], s[0][2 * x + 1]), fmaxf(s[1][2 * x], s[1][2 * x + 1]));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
          const float top = fmaxf(m[x], reference<T>(t, a.sl2, 0.f));
          alpha[x] = part_scale(m[x], top);
          m[x] = top;
          const float mu = top == -INFINITY ? 0.f : top;
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float p0 = ex2_approx(fmaf(s[n][2 * x], a.sl2, -mu));
            const float p1 = ex2_approx(fmaf(s[n][2 * x + 1], a.sl2, -mu));
            sum += p0 + p1;
            p[2 * n + x] = Two<T>::pack(p0, p1);
          }
          l[x] = l[x] * alpha[x] + sum;
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] *= alpha[e >> 1];
        }
        // O += P V; V rows behind the last token are left out, and NaN or
        // infinity in a drafted row (see add_wild)
        unsigned keep[2] = {3, 3}, drafted[2] = {0, 0};
        if (edge) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int t = key0 + qc + 8 * x;
            keep[x] = (t < len) | (t + 1 < len) << 1;
            drafted[x] = (t >= g.start) | (t + 1 >= g.start) << 1;
          }
        }
        const int row = lane & 15;
#pragma unroll
        for (int n = 0; n < D / 16; n += 2) {
          uint32_t b[2][4];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int ch = (n + y) * 2 + (lane >> 4);
            ldsm_x4_t(b[y],
                      tV + (ch >> 3) * half_bytes + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
            if (edge) {
#pragma unroll
              for (int x = 0; x < 4; ++x)
                b[y][x] = clean2<T>(b[y][x], keep[x & 1], drafted[x & 1], &bad);
            }
          }
#pragma unroll
          for (int y = 0; y < 4; ++y)
            Two<T>::mma(o[2 * n + y], p, b[y >> 1][2 * (y & 1)], b[y >> 1][2 * (y & 1) + 1]);
        }
      }
      // not after a wait ran out: the producer would fill a stage whose barrier
      // still expects its last bytes
      if (!failed) warp_arrive(&bar->empty[st], lane);
    }
    // ------------------------------------------------ join the warps
    bad = __any_sync(0xffffffffu, bad);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    }
    const int slot = 2 * blockIdx.x + (seg > 0);
    if (tid == 0) tell_item(a, g, place.run, slot);
    constexpr int RJ = C::RJ, N = D * RJ / (32 * W);  // columns a thread joins
    auto any_bad = [&]() {
      int x = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) x |= bar->bad[w];
      return x;
    };
    for (int r0 = 0; r0 < rows; r0 += RJ) {
      if (r0 > 0) sync();  // the buffer's last readers are through
      if (r0 == 0) {
        if (lane == 0) bar->bad[warp] = bad;
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if ((lane & 3) == 0) bar->ml[warp][gr + 8 * x] = make_float2(m[x], l[x]);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if ((unsigned)(gr + 8 * x - r0) < RJ) {
          float *dst = join + (warp * RJ + gr + 8 * x - r0) * (D + C::PAD) + qc;
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<float2 *>(dst + n * 8) = make_float2(o[n][2 * x], o[n][2 * x + 1]);
        }
      sync();
      const int r = r0 + tid % RJ, col = tid / RJ * N;
      if (r < rows) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) top = fmaxf(top, bar->ml[w][r].x);
        float sum = 0.f, acc[N];
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float2 ml = bar->ml[w][r];
          const float f = part_scale(ml.x, top);
          const float *src = join + (w * RJ + r - r0) * (D + C::PAD) + col;
          sum += ml.y * f;
#pragma unroll
          for (int e = 0; e < N; ++e) acc[e] += src[e] * f;
        }
        if (g.whole) {
          const int i = r * by_g >> 16, hd = g.h * a.G + r - i * a.G;
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
          for (int e = 0; e < N; ++e) acc[e] *= inv;
          if (any_bad())
            add_wild<T, N>(a, g.s, g.h, Seq{g.start, g.count}, i, D, col, acc);
          write_row<T, N>(a, g.s, hd, i, D, col, acc);
          if (col == 0) write_lse(a, g.s, hd, i, top, sum);
        } else {
          float *dst = reinterpret_cast<float *>(
              a.part_o + ((size_t)slot * (D / 4) + col / 4) * ROWS + r) + col % 4;
#pragma unroll
          for (int e = 0; e < N; ++e) dst[e] = acc[e];
          if (col == 0) a.part_ml[(size_t)slot * ROWS + r] = make_float2(top, sum);
          if (tid == 0 && r0 == 0) a.part_bad[slot] = any_bad();
        }
      }
    }
  }
}

// ----------------------------------------------------------------- tree masks
// A warp per draft walks its ancestors; lane w holds mask word w.
__global__ void __launch_bounds__(256)
    tree_mask_kernel(const int32_t *__restrict__ parents, uint32_t *mask, int32_t *depth, int tree,
                     int words, int *err) {
  __shared__ int par[kMaxTree];
  allow_next();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  for (int x = threadIdx.x; x < tree; x += 256) {
    int p = parents[(size_t)b * tree + x];
    if (p < -1 || p >= x) {
      if (blockIdx.x == 0) report(err, PBS_ERR_DEVICE_ASSERT);
      p = -1;
    }
    par[x] = p;
  }
  __syncthreads();
  if (i >= tree) return;
  uint32_t word = 0;
  int n = -1;
  for (int p = i; p >= 0; p = par[p], ++n)
    if (p >> 5 == lane) word |= 1u << (p & 31);
  if (lane < words) mask[((size_t)b * tree + i) * words + lane] = word;
  if (depth && lane == 0) depth[(size_t)b * tree + i] = n;
}

// ------------------------------------------------------------------ host side
}  // namespace

int sm_count_cached() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return sm_count();
  int n = known[dev].load(std::memory_order_relaxed);
  if (!n) known[dev].store(n = sm_count(), std::memory_order_relaxed);
  return n;
}

namespace {

bool tree_shape_ok(int hq, int tree, const pbs_cache &c) {
  return hq >= 1 && c.hkv >= 1 && hq % c.hkv == 0 && tree >= 0 && c.seqs >= 0 && c.pages >= 1 &&
         c.page >= 1 && c.width >= 1;
}

// What the kernels take, beyond what makes sense.
bool tree_supported(int hq, int tree, const pbs_cache &c) {
  if ((c.d != 64 && c.d != 128) || c.page < 16 || c.page > 256 || (c.page & (c.page - 1)) ||
      tree > kMaxTree || c.seqs > 65535 || hq > 65536 || c.hkv > 65535 ||
      (int64_t)c.pages * c.hkv * c.page >= (1ll << 31) ||
      (int64_t)c.width * c.page >= (1ll << 31) - 2 * kMaxTree)
    return false;
  const int64_t rows = (int64_t)(hq / c.hkv) * tree;
  // units of a call, at most (the smallest tiles)
  return rows < (1 << 22) &&
         (double)c.seqs * c.hkv * ceil_div(rows, 16) *
                 (ceil_div((int64_t)c.width * c.page, kKeys) + kExtra<256>) < 2e9;
}

// The rows of an item: 16 by warp MMA, 128 or 256 (in pairs) by tcgen05, by the
// most rows that a KV head can have. Both sides, us a call (32 / 8 heads, d =
// 128, 64-token pages):
//   rows, sequences x tokens    16 by MMA   128 alone   256 in pairs
//   4    8 x 16K                     91.9        89.4          -
//   16   8 x 16K                     96.2        90.2          -
//   4    64 x 1000                   54.4        75.4          -
//   16   64 x 1000                   58.6        75.6          -
//   4    1 x 8K                      17.2        20.0          -
//   32   8 x 16K                        -        94.1      107.5
//   128  8 x 16K                        -       105.6      114.8
//   192  8 x 16K                        -       183.1      152.5
//   256  8 x 16K                        -       191.4      162.5
// (the lengths, which would settle 4 to 16 rows, are on the device).
int row_tile(int hq, int tree, const pbs_cache &c) {
  const int64_t rows = (int64_t)(hq / c.hkv) * tree;
  return rows <= 16 ? 16 : rows <= 128 ? 128 : 256;
}

// Consumer warps of a CTA of the warp-MMA kernel: 8, or 4 in each of two CTAs an
// SM. Two CTAs hide the 2 to 4 us that an item's beginning and end cost, and
// have two warps to issue the copies, where 16-token pages of d = 64 keep one
// busy; their twice as many runs leave more parts to join, and a long item reads
// a little slower. Us a call (4 rows, 8 KV heads, captured, taken with one block a
// head in the joining kernel; its later form takes 40 off 2000 x 50 and 9 off 512 x
// 200, the later scan for a run's place 10 more off the former):
//   d, page   sequences x tokens       8 warps   2 x 4
//   128, 64    2000 x 50                  395.8   227.3
//   128, 64    512 x 200                  148.2   108.0
//   128, 64    32 x 300                    20.6    17.7
//   128, 64    32 x 500, 16 rows           31.2    25.9
//   128, 64    64 x 1000                   53.7    54.8
//   128, 64    64 x 1000, 16 rows          63.0    58.6
//   128, 64    32 x 8000                  170.6   172.1
//   128, 64    64 x 4000                  172.4   173.0
//   128, 16    64 x 4000                  167.8   172.0
//   128, 64    1 x 32000                   34.2    35.8
//   128, 64    1 x 131072, 1 KV head       30.7    43.0
//   64, 64     256 x 1000                 119.3   100.5
//   64, 64     32 x 8000                   97.1    94.8
//   64, 16     32 x 8000                  143.0    90.6
//   64, 16     1 x 32000                   26.1    21.9
//   64, 64     1 x 32000                   22.4    22.5
// The lengths are on the device; the host knows the items (a KV head of a
// sequence) and the most tokens that a table row can name.
int mma_warps(const pbs_cache &c) {
  const int64_t items = (int64_t)c.seqs * c.hkv, most = (int64_t)c.width * c.page;
  if (c.d == 64) return items >= 8 ? 4 : 8;
  return items >= 512 || (items >= 128 && most <= 1024) ? 4 : 8;
}

// CTAs of the attention kernel.
int ctas(int rows, const pbs_cache &c) {
  return sm_count_cached() * (rows == 16 ? 8 / mma_warps(c) : 1);
}

struct Parts {
  size_t o, ml, items, bad, bytes;
  int tiles;
};
Parts parts(int rows, int hq, int tree, const pbs_cache &c) {
  const size_t slots = 2 * (size_t)ctas(rows, c);
  Parts p;
  p.tiles = (int)ceil_div((int64_t)(hq / c.hkv) * tree, rows);
  p.o = 0;
  p.ml = slots * rows * c.d * 4;
  p.items = p.ml + slots * rows * 8;
  p.bad = p.items + (size_t)c.seqs * c.hkv * p.tiles * 8;
  p.bytes = p.bad + slots * 4;
  return p;
}

template <typename T, int D, int W>
cudaError_t run_mma(const CUtensorMap &mk, const CUtensorMap &mv, const TreeArgs &a, int grid,
                    cudaStream_t st) {
  using C = MmaCfg<D, W>;
  constexpr auto kern = tree_mma_kernel<T, D, W>;
  cudaError_t e = allow_smem<kern>((int)C::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_behind(kern, dim3(grid), C::THREADS, C::SMEM, st, mk, mv, a);
  if (e != cudaSuccess) return e;
  return launch_combine<T, D, C::ROWS>(a, grid, st);
}

template <typename T>
cudaError_t run_mma(const CUtensorMap &mk, const CUtensorMap &mv, const TreeArgs &a, int d,
                    int warps, int grid, cudaStream_t st) {
  if (d == 64)
    return warps == 4 ? run_mma<T, 64, 4>(mk, mv, a, grid, st)
                      : run_mma<T, 64, 8>(mk, mv, a, grid, st);
  return warps == 4 ? run_mma<T, 128, 4>(mk, mv, a, grid, st)
                    : run_mma<T, 128, 8>(mk, mv, a, grid, st);
}

}  // namespace
}  // namespace pbs

using namespace pbs;

extern "C" {

pbs_status pbs_tree_mask(const int32_t *parents, uint32_t *mask, int32_t *depth, int batch,
                         int tree, pbs_stream_t st) {
  if (batch < 0 || tree < 0) return PBS_ERR_INVALID_ARG;
  if (tree > kMaxTree || batch > 65535) return PBS_ERR_UNSUPPORTED;
  if (batch == 0 || tree == 0) return PBS_OK;
  if (!parents || !mask || ((uintptr_t)parents & 3u) || ((uintptr_t)mask & 3u) ||
      ((uintptr_t)depth & 3u))
    return PBS_ERR_INVALID_ARG;
  tree_mask_kernel<<<dim3((tree + 7) / 8, batch), 256, 0, (cudaStream_t)st>>>(
      parents, mask, depth, tree, (tree + 31) / 32, error_word());
  return cudaGetLastError() == cudaSuccess ? PBS_OK : PBS_ERR_CUDA;
}

size_t pbs_tree_workspace_bytes(int hq, int tree, pbs_cache c) {
  if (!tree_shape_ok(hq, tree, c) || !tree_supported(hq, tree, c) || c.seqs == 0 || tree == 0)
    return 0;
  return parts(row_tile(hq, tree, c), hq, tree, c).bytes;
}

pbs_status pbs_tree_attn(pbs_rows q, const void *k_pages, const void *v_pages,
                         const int32_t *table, const int32_t *start, const int32_t *count,
                         const uint32_t *mask, void *out, float *lse, int hq, int tree,
                         pbs_cache c, float scale, int zero_rest, int dtype, void *ws,
                         size_t ws_bytes, pbs_stream_t st) {
  if (!tree_shape_ok(hq, tree, c) || (dtype != PBS_BF16 && dtype != PBS_FP16))
    return PBS_ERR_INVALID_ARG;
  if (!tree_supported(hq, tree, c)) return PBS_ERR_UNSUPPORTED;
  if (c.seqs == 0 || tree == 0) return PBS_OK;
  auto ints = [](const void *p) { return p && ((uintptr_t)p & 3u) == 0; };
  if (!rows_ok(q, 2) || !aligned16(k_pages) || !aligned16(v_pages) || !k_pages || !v_pages ||
      !ints(table) || !ints(start) || (count && !ints(count)) || (mask && !ints(mask)) || !out ||
      !aligned16(out) || ((uintptr_t)lse & 3u) || !ws || !aligned16(ws))
    return PBS_ERR_INVALID_ARG;
  const int rows = row_tile(hq, tree, c);
  const Parts p = parts(rows, hq, tree, c);
  if (ws_bytes < p.bytes) return PBS_ERR_WORKSPACE;
  // what is written meets nothing else
  {
    const int64_t some = (int64_t)c.seqs * hq * tree, pool = 2ll * c.pages * c.hkv * c.page * c.d;
    const pbs_rows dense{out, 0, (int64_t)hq * tree * c.d, (int64_t)tree * c.d, c.d};
    const RowSet qs{q, c.seqs, hq, tree, c.d, 2}, os{dense, c.seqs, hq, tree, c.d, 2};
    const void *ptr[] = {out, lse, ws, k_pages, v_pages, table, start, count, mask};
    const int64_t len[] = {some * c.d * 2, some * 4, (int64_t)p.bytes, pool, pool,
                           4ll * c.seqs * c.width, 4ll * c.seqs, 4ll * c.seqs,
                           4ll * c.seqs * tree * ((tree + 31) / 32)};
    bool meet = rows_meet(qs, os) || rows_meet(qs, lse, len[1]) || rows_meet(qs, ws, len[2]);
    for (int o = 0; o < 3; ++o)
      for (int i = o + 1; i < 9; ++i) meet |= bytes_meet(ptr[o], len[o], ptr[i], len[i]);
    if (meet) return PBS_ERR_INVALID_ARG;
  }
  TreeArgs a{};
  a.q = q, a.table = table, a.start = start, a.count = count, a.mask = mask, a.v_pages = v_pages;
  a.out = out, a.lse = lse;
  a.part_o = (float4 *)((uint8_t *)ws + p.o);
  a.part_ml = (float2 *)((uint8_t *)ws + p.ml);
  a.part_bad = (int *)((uint8_t *)ws + p.bad);
  a.items = (int2 *)((uint8_t *)ws + p.items);
  a.tiles = p.tiles;
  a.err = error_word();
  a.hq = hq, a.hkv = c.hkv, a.G = hq / c.hkv, a.tree = tree, a.words = (tree + 31) / 32;
  a.seqs = c.seqs, a.width = c.width, a.page = c.page, a.pages = c.pages;
  const float sigma = scale > 0.f ? scale : (float)(1.0 / sqrt((double)c.d));
  a.sl2 = sigma * kLog2e;
  a.zero_rest = zero_rest != 0;
  // PBS_FAULT_INJECT=tree makes every CTA leave its first K tile out, so that
  // bounded waits run out (used by the failure-detection tests)
  const char *fi = getenv("PBS_FAULT_INJECT");
  a.fault = fi && strcmp(fi, "tree") == 0;
  CUtensorMap mk, mv;
  const uint64_t all = (uint64_t)c.pages * c.hkv * c.page;
  const int keys = rows == 16 ? kKeys : 128, box = c.page < keys ? c.page : keys;
  auto make = rows == 16 ? make_tile_map_halves : make_tile_map;
  if (!make(&mk, k_pages, all, c.d, box) || !make(&mv, v_pages, all, c.d, box))
    return PBS_ERR_CUDA;
  cudaStream_t cs = (cudaStream_t)st;
  const int grid = ctas(rows, c);
  const bool bf16 = dtype == PBS_BF16;
  cudaError_t e;
  if (rows > 16)
    e = launch_tree_tc(mk, mv, a, c.d, rows, bf16, grid, cs);
  else
    e = bf16 ? run_mma<__nv_bfloat16>(mk, mv, a, c.d, mma_warps(c), grid, cs)
             : run_mma<__half>(mk, mv, a, c.d, mma_warps(c), grid, cs);
  return e == cudaSuccess ? PBS_OK : PBS_ERR_CUDA;
}

}  // extern "C"
