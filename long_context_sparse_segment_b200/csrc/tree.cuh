// Shared by the kernels of pbs_tree_attn: what a call asks for, how its work
// is cut into runs, the types, and the kernel that joins the parts.
//
// Work. The key tiles of all items (sequence, KV head, tile of rows) form
// one line of units, cut into equal runs, one per CTA (one CTA per SM, or two
// of half the size): a ragged batch and a single long sequence load every SM
// alike, and the lengths are read on the device. A run that holds all of an item's units
// writes its rows; an item cut by a run's end leaves its running maximum,
// sum and output (fp32) in the workspace, at most two per CTA, and the
// combining kernel joins them in unit order, so results do not depend on
// timing.
//
// The weights P are rounded to 16 bits for the product with V; their sum takes
// the unrounded ones. They are taken relative to a reference: in bf16 the running
// maximum; in fp16 a power of two below it (`reference`), since fp16 loses weights
// below 2^-25 altogether: 131071 keys 2^25.1 below one of the same item would come
// out 0.36 % short. So fp16 keeps weights down to 2^-40 of the maximum, or 2^-32
// under the tcgen05 kernel's, which lags. A weight is off by half a step at most,
// independently from key to key, so the output gains about as much error as its
// own rounding has (1.4 times it together). A second 16-bit part would take that
// away: under the power limit it cost 5 % of a decoding step and 10 % of 7 drafts
// over 128K.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "decode.h"
#include "tc.cuh"

namespace pbs {
namespace tree {

using namespace tc;

// Programmatic dependent launch. The kernels of a call are launched while the
// kernel in front of them may still run, set themselves up, and wait for its end
// before they read or write anything that another kernel knows: 1 to 2 us a call.
// Every block waits, so that a kernel never ends before the one in front. Nothing is
// read through the read-only path (__ldg, ld.global.nc), which is for memory that
// nobody writes while the kernel is in flight and need not stay behind the wait:
// the kernel in front may still write the lengths, tables and masks.

// Allows the kernel launched behind this one to start.
__device__ __forceinline__ void allow_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// Waits until the kernel launched before this one has ended, its writes visible.
__device__ __forceinline__ void wait_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_behind(void (*kern)(P...), dim3 grid, int threads, size_t smem,
                          cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

constexpr int kMaxTree = 1024;  // 32 mask words a row

struct TreeArgs {
  pbs_rows q;
  const int32_t *table, *start, *count;
  const uint32_t *mask;
  const void *v_pages;  // for the non-finite rows of drafts
  void *out;
  float *lse;
  float4 *part_o;   // [2 grid][d / 4][rows]: neighbouring rows side by side
  float2 *part_ml;  // [2 grid][rows]: the weights' reference (log2) and sum
  int *part_bad;    // [2 grid]: drafted V rows with NaN or infinity met
  int2 *items;      // [seqs][hkv][tiles]: an item's first part, and its last CTA
  int *err;
  int hq, hkv, G, tree, words, seqs, width, page, pages;
  int tiles;  // row tiles of `tree` drafts
  int fault;      // the first K tile of every CTA stays out (failure tests)
  int zero_rest;  // rows behind a sequence's count become 0 instead of staying
  float sl2;
};

// What a sequence asks for: its cached tokens and drafts (0 where the call
// has to leave it alone, which the joining kernel reports).
struct Seq {
  int start, count;
};

// Its lengths as they stand in memory; 0 behind the last sequence.
__device__ __forceinline__ Seq read_seq(const TreeArgs &a, int s) {
  if (s >= a.seqs) return {0, 0};
  return {a.start[s], a.count ? a.count[s] : a.tree};
}
// They will be read soon (held in registers from here on instead, they cost the
// tcgen05 kernel more in spills: 7 drafts over 128K tokens 93.6 us, so 92.7).
__device__ __forceinline__ void touch_seq(const TreeArgs &a, int s) {
  if (s >= a.seqs) return;
  asm volatile("prefetch.global.L1 [%0];" ::"l"(a.start + s));
  if (a.count) asm volatile("prefetch.global.L1 [%0];" ::"l"(a.count + s));
}
__device__ __forceinline__ Seq check_seq(const TreeArgs &a, Seq q) {
  q.count = min(q.count, a.tree);
  if (q.count <= 0 || q.start < 0 || (int64_t)q.start + q.count > (int64_t)a.width * a.page)
    return {0, 0};
  return q;
}
__device__ __forceinline__ Seq seq_of(const TreeArgs &a, int s) {
  return check_seq(a, read_seq(a, s));
}

__device__ __forceinline__ int cdiv(int x, int y) { return (x + y - 1) / y; }

// What an item's beginning and end cost a CTA, in key tiles: so many units are
// counted in front of an item's own, and a run that begins an item gets fewer
// tiles. Measured with clocks in the kernels: 7 us of 1.9 us tiles (256 rows),
// 5 of 1.6 (128 rows), 1.5 of 0.7 (16 rows, 64 keys). Without it 7 drafts over
// 128K tokens take 94.4 instead of 92.4 us, one sequence of 8K 17.1 instead of 15.9,
// 64 drafts of 64 sequences of 1000 tokens 160-170 instead of 155-161; twice as
// much: 92.4, 15.4 and 151.
template <int ROWS>
constexpr int kExtra = ROWS == 16 ? 2 : 3;

// Units of a sequence: its items (KV head, row tile) times its key tiles.
template <int ROWS, int KEYS>
__device__ __forceinline__ int units_of(const TreeArgs &a, const Seq &q) {
  return q.count ? a.hkv * cdiv(q.count * a.G, ROWS) *
                       (cdiv(q.start + q.count, KEYS) + kExtra<ROWS>)
                 : 0;
}

// The units of CTA c: [start(c), start(c + 1)); none is empty with
// runs = min(total, CTAs) of them, the first `extra` one unit longer. The run
// that unit u belongs to.
struct Runs {
  int base, extra;
  Runs() = default;
  __device__ __forceinline__ Runs(int total, int runs)
      : base(total / runs), extra(total - total / runs * runs) {}
  __device__ __forceinline__ int start(int c) const { return c * base + min(c, extra); }
  __device__ __forceinline__ int owner(int u) const {
    const int cut = extra * (base + 1);
    return u < cut ? u / (base + 1) : extra + (u - cut) / base;
  }
};

// The place of a CTA's run: its first and end unit, and the sequence that the
// first lies in with what it asks for and the units before it.
struct Place {
  int u0, u1, s, before;
  Seq q;
  Runs run;
};

// Every thread of the block (NT of them, a multiple of 32) calls it; false
// for a CTA without units. `sum`: NT / 32 words of shared memory.
template <int ROWS, int KEYS, int NT>
__device__ __forceinline__ bool find_place(const TreeArgs &a, int *sum, Place *p) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // up to 32 sequences a warp holds them all and nobody waits for another; more
  // are summed by the block first (a barrier and a second look at the lengths)
  Seq ahead = read_seq(a, lane);  // of the next 32 sequences
  int total = 0;
  if (a.seqs > 32) {
    for (int s = tid; s < a.seqs; s += NT) total += units_of<ROWS, KEYS>(a, seq_of(a, s));
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0) sum[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) total += sum[w];
  } else {
    total = __reduce_add_sync(0xffffffffu, units_of<ROWS, KEYS>(a, check_seq(a, ahead)));
  }
  const int runs = min(total, (int)gridDim.x);
  if ((int)blockIdx.x >= runs) return false;
  const Runs run(total, runs);
  p->u0 = run.start(blockIdx.x), p->u1 = run.start(blockIdx.x + 1), p->run = run;
  int base = 0;
#pragma unroll 1
  for (int s0 = 0; s0 < a.seqs; s0 += 32) {
    const Seq q = check_seq(a, ahead);
    ahead = read_seq(a, s0 + 32 + lane);
    const int x = units_of<ROWS, KEYS>(a, q);
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    inc += base;
    const unsigned m = __ballot_sync(0xffffffffu, inc > p->u0);
    if (m) {
      const int l = __ffs(m) - 1;
      p->s = s0 + l, p->before = __shfl_sync(0xffffffffu, inc - x, l);
      p->q = Seq{__shfl_sync(0xffffffffu, q.start, l), __shfl_sync(0xffffffffu, q.count, l)};
      return true;
    }
    base = __shfl_sync(0xffffffffu, inc, 31);
  }
  return false;  // only when somebody changes the lengths under this call
}

// A piece of a CTA's run inside one item.
struct Segment {
  int s, h, rt;      // sequence, KV head, row tile
  int start, count;  // tokens, drafts
  int k0, k1;        // key tiles
  int whole;         // all of the item's key tiles
  int last;          // the item's last unit
};

// Where an item's parts are, told by the CTA that has its first tile: the slot
// of that part, and the CTA that has its last tile (the same one: no parts).
__device__ __forceinline__ void tell_item(const TreeArgs &a, const Segment &g, const Runs &run,
                                          int slot) {
  if (g.k0 == 0)
    a.items[((size_t)g.s * a.hkv + g.h) * a.tiles + g.rt] =
        make_int2(slot, g.whole ? (int)blockIdx.x : run.owner(g.last));
}

// The segments of a run, one after the other. A sequence's lengths are read when
// the walk comes to it; the segment holds them from one call to the next.
template <int ROWS, int KEYS>
struct Walk {
  int u, u1, s, before;
  __device__ __forceinline__ Walk(const TreeArgs &a, const Place &p, Segment *g)
      : u(p.u0), u1(p.u1), s(p.s), before(p.before) {
    g->start = p.q.start, g->count = p.q.count;
    touch_seq(a, s + 1);
  }
  __device__ __forceinline__ bool next(const TreeArgs &a, Segment *g) {
    while (u < u1) {
      Seq q{g->start, g->count};
      for (int n; u >= before + (n = units_of<ROWS, KEYS>(a, q));) {
        before += n;
        if (++s >= a.seqs) return false;  // the lengths changed under this call
        q = seq_of(a, s);
        touch_seq(a, s + 1);
      }
      g->start = q.start, g->count = q.count;
      constexpr int X = kExtra<ROWS>;
      const int kt = cdiv(q.start + q.count, KEYS), rts = cdiv(q.count * a.G, ROWS);
      const int x = u - before, item = x / (kt + X), at = x - item * (kt + X) - X;
      g->s = s, g->h = item / rts, g->rt = item - g->h * rts;
      g->k0 = max(at, 0);
      g->k1 = min(kt, at + u1 - u);
      g->whole = g->k1 - g->k0 == kt;
      g->last = u - at + kt - 1;
      u += min(kt - at, u1 - u);
      if (g->k1 > g->k0) return true;  // else the run ends before the item's first tile
    }
    return false;
  }
};

// Whether draft i sees draft j (j < count).
__device__ __forceinline__ bool sees(const TreeArgs &a, int s, int i, int j) {
  if (!a.mask) return j <= i;
  return a.mask[((size_t)s * a.tree + i) * a.words + (j >> 5)] >> (j & 31) & 1;
}

// Bit x of the result: whether draft i of sequence s sees key `key` + x, given
// that some of the 32 keys are drafts or lie behind the last token.
__device__ __forceinline__ uint32_t seen_word(const TreeArgs &a, const Segment &g, int i, int key) {
  const int j = key - g.start, left = g.count - j;  // drafts from the first key on
  if (left <= 0) return 0;
  auto word = [&](int w) -> uint32_t {
    if (w < 0) return 0xffffffffu;  // the prefix
    if (w >= a.words) return 0;
    if (a.mask) return a.mask[((size_t)g.s * a.tree + i) * a.words + w];
    return w < i >> 5 ? 0xffffffffu : w > i >> 5 ? 0u : (2u << (i & 31)) - 1;
  };
  const int w = j >> 5;
  uint32_t x = word(w);
  if (j & 31) x = __funnelshift_r(x, word(w + 1), j & 31);
  return left < 32 ? x & ((1u << left) - 1) : x;
}

// ---------------------------------------------------------------- 16-bit types
template <typename T>
struct Two;
template <>
struct Two<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t pack(float x, float y) { return pack_bf16(x, y); }
  static constexpr uint32_t kExp = 0x7f80u;
  static constexpr float kTop = 0.f;
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    mma_16816(c, a, b0, b1);
  }
};
template <>
struct Two<__half> {
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
  static constexpr uint32_t kExp = 0x7c00u;
  static constexpr float kTop = 15.f;  // 2^15, the largest power of two below 65504
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
        "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// The reference of the weights under a maximum logit `s` (times sl2: log2) that
// may rise by up to `lag` before it is moved: so far below that the largest
// weight is 2^kTop. Rounded up, so that it is never more (fp16 has no room above).
template <typename T>
__device__ __forceinline__ float reference(float s, float sl2, float lag) {
  return Two<T>::kTop == 0.f ? s * sl2 : __fmaf_ru(s, sl2, lag - Two<T>::kTop);
}
// How high the reference of a new maximum may lie before it replaces m; rounded
// down for the same reason.
template <typename T>
__device__ __forceinline__ float may_rise(float m, float lag) {
  return Two<T>::kTop == 0.f ? m + lag : __fadd_rd(m, lag);
}

// NaN or infinity in a 16-bit value.
template <typename T>
__device__ __forceinline__ bool wild16(uint32_t x) {
  return (x & Two<T>::kExp) == Two<T>::kExp;
}

// Nonzero when a half of u is NaN or infinite: the exponent's all-ones carries
// into the sign's place.
template <typename T>
__device__ __forceinline__ uint32_t wild2(uint32_t u) {
  constexpr uint32_t e = Two<T>::kExp * 0x10001u;
  constexpr uint32_t one = (0x8000u - Two<T>::kExp) * 0x10001u;
  return ((u & e) + one) & 0x80008000u;
}

// The two halves of u that `keep` (bits 0, 1) has; with `drafted` (bits 0, 1)
// a NaN or infinity in such a half becomes 0 and *bad is set.
template <typename T>
__device__ __forceinline__ uint32_t clean2(uint32_t u, unsigned keep, unsigned drafted, bool *bad) {
  uint32_t lo = keep & 1 ? u & 0xffffu : 0, hi = keep & 2 ? u & 0xffff0000u : 0;
  if ((drafted & 1) && wild16<T>(lo)) lo = 0, *bad = true;
  if ((drafted & 2) && wild16<T>(hi >> 16)) hi = 0, *bad = true;
  return lo | hi;
}

// The product P V leaves NaN and infinite values of drafted V rows out, since
// 0 times them would reach the rows that do not see them. This adds them to a
// row that does: columns [col, col + N) of draft i's output.
template <typename T, int N>
__device__ __noinline__ void add_wild(const TreeArgs &a, int s, int h, const Seq &q, int i,
                                      int d, int col, float (&o)[N]) {
  for (int j = 0; j < q.count; ++j) {
    if (!sees(a, s, i, j)) continue;
    const int t = q.start + j;
    const int page = a.table[(size_t)s * a.width + t / a.page];
    if (page < 0 || page >= a.pages) continue;
    const T *v = (const T *)a.v_pages +
                 (((size_t)page * a.hkv + h) * a.page + t % a.page) * d + col;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float x = (float)v[e];
      if (!isfinite(x)) o[e] += x;
    }
  }
}

// N output columns of a query head's draft i, from fp32.
template <typename T, int N>
__device__ __forceinline__ void write_row(const TreeArgs &a, int s, int head, int i, int d, int col,
                                          const float (&o)[N]) {
  T *dst = (T *)a.out + (((size_t)s * a.hq + head) * a.tree + i) * d + col;
  if constexpr (N == 1) {
    *reinterpret_cast<uint16_t *>(dst) = (uint16_t)Two<T>::pack(o[0], 0.f);
  } else {
    uint32_t p[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e) p[e] = Two<T>::pack(o[2 * e], o[2 * e + 1]);
    if constexpr (N == 8)
      *reinterpret_cast<uint4 *>(dst) = make_uint4(p[0], p[1], p[2], p[3]);
    else if constexpr (N == 4)
      *reinterpret_cast<uint2 *>(dst) = make_uint2(p[0], p[1]);
    else
      *reinterpret_cast<uint32_t *>(dst) = p[0];
  }
}

__device__ __forceinline__ void write_lse(const TreeArgs &a, int s, int head, int i, float m, float l) {
  if (a.lse)
    a.lse[((size_t)s * a.hq + head) * a.tree + i] =
        l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// 2^(m - top) for a part whose reference is m, top the highest of all parts'.
__device__ __forceinline__ float part_scale(float m, float top) {
  return m == top ? 1.f : ex2_approx(m - top);
}

// -------------------------------------------------------------------- combine
// Joins the parts of the rows that several CTAs worked on. A block takes groups
// of RB rows of one (sequence, KV head), or with MANY of `heads` of them, one
// after the other: a thread holds 4 columns of a row and every PG-th part of it,
// in order; the PG partial results are joined in shared memory. Bound by latency:
// a part is read once, a thread's reads in flight together; most blocks find that
// nobody shared their items and end.
constexpr int kCombineThreads = 512;

struct Part {
  float m, l;
  float4 o;
};

__device__ __forceinline__ void join(Part &p, const Part &q) {
  const float top = fmaxf(p.m, q.m), f = part_scale(p.m, top), g = part_scale(q.m, top);
  p.m = top, p.l = p.l * f + q.l * g;
  p.o.x = p.o.x * f + q.o.x * g, p.o.y = p.o.y * f + q.o.y * g;
  p.o.z = p.o.z * f + q.o.z * g, p.o.w = p.o.w * f + q.o.w * g;
}

template <typename T, int D, int ROWS, int RB, bool MANY>
__global__ void __launch_bounds__(kCombineThreads)
    tree_combine_kernel(const __grid_constant__ TreeArgs a, int grid, int heads) {
  constexpr int C4 = D / 4, E = RB * C4;  // results of a group, 4 columns each
  constexpr int PG = kCombineThreads / E;
  static_assert(PG * E == kCombineThreads && ROWS % RB == 0, "threads");
  __shared__ float4 so[kCombineThreads];
  __shared__ float2 sml[PG][RB];
  const int tid = threadIdx.x, lane = tid & 31;
  const int r = tid % RB, c4 = tid / RB % C4, pg = tid / E;
  // results: neighbouring threads along a row
  const int er = tid / C4, ec = tid % C4 * 4;
  allow_next();
  // MANY: every warp finds those of the block's heads that have something to do
  const int first = blockIdx.x * heads;
  const int pair = MANY ? min(first + lane, a.seqs * a.hkv - 1) : 0;
  // the attention kernel has not changed the lengths
  const Seq asked = read_seq(a, MANY ? pair / a.hkv : blockIdx.z), own = check_seq(a, asked);
  if (asked.count > 0 && own.count == 0) report(a.err, PBS_ERR_DEVICE_ASSERT);
  wait_previous();
  unsigned todo = 1;
  if constexpr (MANY) {
    bool need = a.zero_rest && own.count < a.tree;
    for (int t = 0; t < cdiv(own.count * a.G, ROWS) && !need; ++t) {
      const int2 item = a.items[(size_t)pair * a.tiles + t];
      need = item.x >> 1 != item.y;
    }
    todo = __ballot_sync(0xffffffffu, need && lane < heads && pair == first + lane);
  }
  for (; todo; todo &= todo - 1) {
    const int at = MANY ? __ffs(todo) - 1 : 0;
    const int s = MANY ? (first + at) / a.hkv : blockIdx.z;
    const int h = MANY ? (first + at) % a.hkv : blockIdx.y;
    const Seq q = MANY ? Seq{__shfl_sync(0xffffffffu, own.start, at),
                             __shfl_sync(0xffffffffu, own.count, at)}
                       : own;
    const int rows = q.count * a.G, all = a.tree * a.G;  // of the (sequence, KV head)
    const int group = MANY ? blockIdx.y : blockIdx.x, groups = MANY ? gridDim.y : gridDim.x;
    for (int r0 = group * RB; r0 < all; r0 += groups * RB) {
      if (a.zero_rest && tid < E && r0 + er >= rows && r0 + er < all) {
        const float o[4] = {};
        const int i = (r0 + er) / a.G, head = h * a.G + (r0 + er) % a.G;
        write_row<T, 4>(a, s, head, i, D, ec, o);
        if (ec == 0 && a.lse) a.lse[((size_t)s * a.hq + head) * a.tree + i] = 0.f;
      }
      if (r0 >= rows) continue;
      const int2 item = a.items[((size_t)s * a.hkv + h) * a.tiles + r0 / ROWS];
      const int slot0 = item.x, c0 = slot0 >> 1, c1 = item.y;
      if (c0 == c1) continue;
      if (c0 < 0 || c1 < c0 || c1 >= grid) {  // the attention kernel gave up before
        if (tid == 0) report(a.err, PBS_ERR_DEVICE_ASSERT);
        continue;
      }
      Part p{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      int bad = 0;
      if (r0 + r < rows) {
        const int rr = r0 % ROWS + r;
#pragma unroll 4
        for (int c = c0 + pg; c <= c1; c += PG) {
          const size_t slot = c == c0 ? slot0 : 2 * c;
          const float2 ml = a.part_ml[slot * ROWS + rr];
          join(p, Part{ml.x, ml.y, a.part_o[(slot * C4 + c4) * ROWS + rr]});
          bad |= a.part_bad[slot];
        }
      }
      if (PG > 1) {
        so[tid] = p.o;
        if (c4 == 0) sml[pg][r] = make_float2(p.m, p.l);
      }
      bad = __syncthreads_or(bad);
      if (PG > 1) {
        if (pg == 0) {
#pragma unroll
          for (int g = 1; g < PG; ++g)
            join(p, Part{sml[g][r].x, sml[g][r].y, so[tid + g * E]});
        }
        __syncthreads();
      }
      if (pg == 0) {
        so[r * C4 + c4] = p.o;
        if (c4 == 0) sml[0][r] = make_float2(p.m, p.l);
      }
      __syncthreads();
      if (tid < E && r0 + er < rows) {
        const float2 ml = sml[0][er];
        const float4 v = so[tid];
        const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;
        float o[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
        const int i = (r0 + er) / a.G, head = h * a.G + (r0 + er) % a.G;
        if (bad) add_wild<T, 4>(a, s, h, q, i, D, ec, o);
        write_row<T, 4>(a, s, head, i, D, ec, o);
        if (ec == 0) write_lse(a, s, head, i, ml.x, ml.y);
      }
      __syncthreads();
    }
  }
}

template <typename T, int D, int ROWS>
cudaError_t launch_combine(const TreeArgs &a, int grid, cudaStream_t st) {
  // 4 rows a group, and 16 where that makes more groups than fit the GPU at once
  // (four blocks an SM): 4 rows, with 4 threads a part, are 3 us quicker on one
  // sequence over 8192 tokens, 16 rows 14 us on 64 drafts of 8 sequences. Blocks
  // for four such rounds, then they walk the groups.
  const int64_t rows = (int64_t)a.G * a.tree, heads = (int64_t)a.hkv * a.seqs;
  const int64_t fit = 4 * sm_count_cached();
  const int rb = ceil_div(rows, 4) * heads <= fit ? 4 : 16;
  int64_t groups = ceil_div(rows, rb);
  // Where that is more than one round and the heads are twice the CTAs, a block
  // looks after several heads, of which no more than one is cut on average (a
  // block a head is 37 us slower behind 16000 heads, 65 behind 4096 of 256 rows;
  // the same code for one head costs 16 registers, a block an SM).
  if (groups * heads > fit && heads >= 2 * grid) {
    const int64_t per = heads / grid > 32 ? 32 : heads / grid, gx = ceil_div(heads, per);
    if (groups * gx > 4 * fit) groups = ceil_div(4 * fit, gx);
    return launch_behind(tree_combine_kernel<T, D, ROWS, 16, true>,
                         dim3((unsigned)gx, (unsigned)groups), kCombineThreads, 0, st, a, grid,
                         (int)per);
  }
  if (groups * heads > 4 * fit) groups = ceil_div(4 * fit, heads);
  const dim3 blocks((unsigned)groups, a.hkv, a.seqs);
  return rb == 4 ? launch_behind(tree_combine_kernel<T, D, ROWS, 4, false>, blocks,
                                 kCombineThreads, 0, st, a, grid, 1)
                 : launch_behind(tree_combine_kernel<T, D, ROWS, 16, false>, blocks,
                                 kCombineThreads, 0, st, a, grid, 1);
}

}  // namespace tree
}  // namespace pbs
