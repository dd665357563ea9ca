// pbs_tree_attn on the sm_100a tensor cores: items of up to 128 rows, or 256.
//
// Two streams of 128-row products run against each other, so that the tensor
// core works on one while the softmax of the other runs:
//   PAIR       the item has up to 256 rows: two tiles of 128, each with its
//              own S, P and O, on the same K and V tiles;
//   otherwise  up to 128 rows, and the streams take the key tiles in turn,
//              each with its own maximum, sum and O, joined at the end.
// Per key tile of 128: S = Q K^T (tcgen05.mma, A and B in shared memory), a
// row per thread of softmax, P as 16-bit pairs over S in TMEM, O += P V.
// 384 threads:
//   warp 0      K and V tiles by TMA, page by page, into two rings;
//   warp 1      the products;
//   warps 2, 3  tiles that reach past the prefix: V rows behind the last
//               token become zero, and NaN and infinities in drafted rows
//               (add_wild puts those where they are seen);
//   warps 4-11  the softmax of the two streams, Q into shared memory, the
//               item's end.
// TMEM: S_0, S_1 (128 columns each), O_0, O_1 (D each).
//
// What bounds it. 256 rows: a tile takes 3,490 cycles, in which the tensor core
// has 2,048 of products (59 %) and the exponentials 2,048: a stream's softmax and
// products follow one another, and the two streams overlap as far as the one
// in-order tensor core lets them. (Over a whole call of 8 sequences of 16K tokens,
// with its start, items' ends and parts, the profiler has the tensor core 46 % and
// the XU 53 % busy.) Up to 128 rows: reading the cache. Measured on the device: 64
// drafts of 8 sequences of 8K to 32K tokens 139 us (157 under the power limit), 800
// TFLOP/s of drafts, of which 128 us are this kernel; 7 drafts over 131072 tokens
// 92.7 us, of which 88 are this kernel (6.1 TB/s).
#include "internal.h"
#include "tree_tc.h"

namespace pbs {
namespace {

using namespace tree;

constexpr int kTile = 128;  // rows of a stream, keys of a unit
constexpr int kThreads = 384;
// setmaxnreg moves registers inside the block's launch allocation: 168 a
// thread x 384 threads = 64512 = 128 x 56 + 256 x 224.
constexpr int kLaunchRegs = 168, kCtrlRegs = 56, kSoftmaxRegs = 224;
static_assert(128 * kCtrlRegs + 256 * kSoftmaxRegs <= kThreads * kLaunchRegs, "register split");
constexpr float kRescaleLog2 = 8.f;  // the weights' reference moves by more than 2^8 or not at all
constexpr int kBadSlots = 8;         // segments in flight: at most VS + 2

template <int D, bool PAIR>
struct Cfg {
  static constexpr int H = D / 64;
  static constexpr int ROWS = PAIR ? 256 : 128;
  static constexpr uint32_t TILE = kTile * D * 2, HALF = kTile * 128;
  static constexpr int KS = D == 64 ? 5 : 2, VS = D == 64 ? 5 : 3;
  static_assert(VS + 2 < kBadSlots, "bad flags");
  struct Shared {
    uint64_t q_full, seg, k_full[KS], k_empty[KS], v_full[VS], v_empty[VS], v_clean[VS], s_full[2],
        p_full[2][2], o_final[2], mma_done;
    uint32_t tmem;
    int abort;
    int bad[kBadSlots][2];  // by warp
    int sum[kThreads / 32];
    Place place;
  };
  static constexpr size_t SMEM =
      1024 + (size_t)(ROWS / kTile + KS + VS) * TILE + sizeof(Shared);
};
static_assert(Cfg<128, true>::SMEM <= 232448 && Cfg<128, false>::SMEM <= 232448 &&
                  Cfg<64, true>::SMEM <= 232448,
              "shared memory");

// Instruction descriptor, kind::f16, fp32 accumulator; A and B of type T.
template <typename T>
__host__ __device__ constexpr uint32_t idesc16(int m, int n, bool b_mn_major);
template <>
__host__ __device__ constexpr uint32_t idesc16<__nv_bfloat16>(int m, int n, bool b) {
  return idesc_bf16(m, n, b);
}
template <>
__host__ __device__ constexpr uint32_t idesc16<__half>(int m, int n, bool b) {
  return idesc_bf16(m, n, b) & ~((1u << 7) | (1u << 10));
}

// A 16-byte word of V without its NaN and infinities. Out of line: it hardly
// ever runs, and code that runs once an item is paid for in instruction fetches.
template <typename T>
__device__ __noinline__ void clean_word(uint4 *p) {
  bool bad = false;
  const uint4 v = *p;
  *p = make_uint4(clean2<T>(v.x, 3, 3, &bad), clean2<T>(v.y, 3, 3, &bad),
                  clean2<T>(v.z, 3, 3, &bad), clean2<T>(v.w, 3, 3, &bad));
}

template <typename T, int D, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TreeArgs a) {
  using C = Cfg<D, PAIR>;
  constexpr int ROWS = C::ROWS, KS = C::KS, VS = C::VS, H = C::H;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t *sQ = base;
  uint8_t *sK = sQ + (ROWS / kTile) * C::TILE;
  uint8_t *sV = sK + KS * C::TILE;
  auto *sh = reinterpret_cast<typename C::Shared *>(sV + VS * C::TILE);
  volatile int *abort = &sh->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 1) {
    tmem_alloc(&sh->tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(&sh->q_full, 8);
    mbar_init(&sh->seg, 8);
    for (int i = 0; i < KS; ++i) mbar_init(&sh->k_full[i], 1), mbar_init(&sh->k_empty[i], 1);
    for (int i = 0; i < VS; ++i) {
      mbar_init(&sh->v_full[i], 1);
      mbar_init(&sh->v_empty[i], 3);  // the products, and warps 2 and 3
      mbar_init(&sh->v_clean[i], 2);  // warps 2 and 3
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sh->s_full[x], 1);
      mbar_init(&sh->p_full[x][0], 4), mbar_init(&sh->p_full[x][1], 4);
      mbar_init(&sh->o_final[x], 1);
    }
    mbar_init(&sh->mma_done, 1);
    sh->abort = 0;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  wait_previous();
  allow_next();  // not before the wait: the next kernel looks at the lengths at once
  const uint32_t tbase = sh->tmem;
  {
    Place place;
    if (!find_place<ROWS, kTile, kThreads>(a, sh->sum, &place)) {
      if (warp == 1) tmem_dealloc(tbase, 512);
      return;
    }
    if (tid == 0) sh->place = place;
  }
  __syncthreads();
  Segment g{};
  Walk<ROWS, kTile> walk(a, sh->place, &g);
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtrlRegs));
    if (warp == 0) {
      // ------------------------------------------------------------ loads
      // In the order in which the products take them: PAIR K0, V0 K1, V1 K2
      // ...; otherwise K0 K1, V0 K2, V1 K3, ... A tile is up to 8 boxes of
      // page rows x H halves of 64 columns, one lane each.
      // A tile's page numbers are read one tile early and serve K, then V.
      const int box = min(a.page, kTile), shift = 31 - __clz(a.page);
      const int half = lane % H, piece = lane / H;
      const bool mine = piece < kTile / box;
      constexpr int AHEAD = PAIR ? 1 : 2;  // K tiles in front of their V
      int kseq = 0, vseq = 0;
      bool ok = true;
      auto load = [&](bool is_v, int k, int y) {  // y: the row, or -1: none
        int &seq = is_v ? vseq : kseq;
        const int S = is_v ? VS : KS, st = seq % S, use = seq / S;
        const int boxes = __popc(__ballot_sync(0xffffffffu, y >= 0));
        uint64_t *full = is_v ? &sh->v_full[st] : &sh->k_full[st];
        if (use > 0 && !mbar_wait_warp(is_v ? &sh->v_empty[st] : &sh->k_empty[st], (use - 1) & 1,
                                       abort, a.err, is_v ? 21 : 11))
          return false;
        if (lane == 0) mbar_expect_tx(full, boxes * box * 128);
        __syncwarp();
        if (y >= 0 && !(a.fault && !is_v && seq == 0))
          tma_load_2d((is_v ? sV : sK) + (size_t)st * C::TILE + half * C::HALF + piece * box * 128,
                      is_v ? &tmV : &tmK, full, half * 64, y);
        __syncwarp();
        ++seq;
        return true;
      };
      if (lane == 0) prefetch_map(&tmK), prefetch_map(&tmV);
      while (ok && walk.next(a, &g)) {
        const int len = g.start + g.count;
        const int32_t *row = a.table + (size_t)g.s * a.width;
        auto page_of = [&](int k) {
          const int t = k * kTile + piece * box;
          return mine && k < g.k1 && t < len ? row[t >> shift] : -1;
        };
        auto row_of = [&](int k, int page) {
          const int t = k * kTile + piece * box;
          if (!mine || k >= g.k1 || t >= len) return -1;
          if (page < 0 || page >= a.pages) {
            report(a.err, PBS_ERR_DEVICE_ASSERT);
            page = 0;
          }
          return (page * a.hkv + g.h) * a.page + (t & (a.page - 1));
        };
        int y[AHEAD + 1];  // rows of tiles k .. k + AHEAD
        int page = page_of(g.k0);
        for (int k = g.k0; k < g.k0 + AHEAD && ok; ++k) {
          const int ahead = page_of(k + 1);
          y[k - g.k0] = row_of(k, page);
          if (k < g.k1) ok = load(false, k, y[k - g.k0]);
          page = ahead;
        }
        for (int k = g.k0; k < g.k1 && ok; ++k) {
          const int ahead = page_of(k + AHEAD + 1);
          y[AHEAD] = row_of(k + AHEAD, page);
          ok = load(true, k, y[0]);
          if (ok && k + AHEAD < g.k1) ok = load(false, k + AHEAD, y[AHEAD]);
#pragma unroll
          for (int e = 0; e < AHEAD; ++e) y[e] = y[e + 1];
          page = ahead;
        }
      }
      // every copy started here lands before the CTA exits
      int never = 0;
      for (int i = kseq > KS ? kseq - KS : 0; i < kseq; ++i)
        if (!(a.fault && i == 0)) mbar_wait(&sh->k_full[i % KS], (i / KS) & 1, &never, nullptr);
      for (int i = vseq > VS ? vseq - VS : 0; i < vseq; ++i)
        mbar_wait(&sh->v_full[i % VS], (i / VS) & 1, &never, nullptr);
    } else if (warp == 1) {
      // --------------------------------------------------------- products
      const bool leader = elect_one();
      constexpr uint32_t kIdQK = idesc16<T>(kTile, kTile, false);
      constexpr uint32_t kIdPV = idesc16<T>(kTile, D, true);
      const uint32_t hi = sw128_desc_hi(1024);
      const uint32_t lo_q = sw128_desc_lo(smem_u32(sQ), 16);
      const uint32_t lo_k = sw128_desc_lo(smem_u32(sK), 16);
      const uint32_t lo_v = sw128_desc_lo(smem_u32(sV), C::HALF);
      int kseq = 0, vseq = 0;
      uint32_t q_phase = 0, p_phase = 0;  // p_phase: bit x
      bool ok = true;
      // S_x = Q K^T with the K tile at kseq; `first`: nobody waited for it yet;
      // `last`: nobody needs it after
      auto qk = [&](int x, bool first, bool last) {
        const int st = kseq % KS;
        if (first) {
          if (!mbar_wait_warp(&sh->k_full[st], (kseq / KS) & 1, abort, a.err, 32)) return false;
          tc_fence_after();
        }
        const uint32_t lq = lo_q + (PAIR ? x : 0) * (C::TILE >> 4), lk = lo_k + st * (C::TILE >> 4);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t step = ((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4;
            mma_ss(tbase + x * 128, desc_words(lq + step, hi), desc_words(lk + step, hi), kIdQK,
                   kk > 0);
          }
          if (last) mma_commit(&sh->k_empty[st]);
          mma_commit(&sh->s_full[x]);
        }
        __syncwarp();
        if (last) ++kseq;
        return true;
      };
      // O_x (+)= P_x V, the halves of P as they are written
      auto pv = [&](int x, bool first, bool last, bool add) {
        const int st = vseq % VS;
        if (!mbar_wait_warp(&sh->p_full[x][0], p_phase >> x & 1, abort, a.err, 33)) return false;
        if (first) {
          if (!mbar_wait_warp(&sh->v_full[st], (vseq / VS) & 1, abort, a.err, 34)) return false;
          if (!mbar_wait_warp(&sh->v_clean[st], (vseq / VS) & 1, abort, a.err, 36)) return false;
        }
        tc_fence_after();
        const uint32_t lv = lo_v + st * (C::TILE >> 4);
        for (int h = 0; h < 2; ++h) {
          if (h == 1) {
            if (!mbar_wait_warp(&sh->p_full[x][1], p_phase >> x & 1, abort, a.err, 35))
              return false;
            tc_fence_after();
          }
          if (leader) {
#pragma unroll
            for (int k2 = 0; k2 < 4; ++k2) {
              const int kk = h * 4 + k2;
              mma_ts(tbase + 256 + x * 128, tbase + x * 128 + kk * 8,
                     desc_words(lv + kk * (2048 >> 4), hi), kIdPV, add || kk > 0);
            }
          }
          __syncwarp();
        }
        p_phase ^= 1u << x;
        if (leader && last) mma_commit(&sh->v_empty[st]);
        __syncwarp();
        if (last) ++vseq;
        return true;
      };
      auto finish = [&](int x) {
        if (leader) mma_commit(&sh->o_final[x]);
        __syncwarp();
      };
      while (ok && walk.next(a, &g)) {
        const int n = g.k1 - g.k0;
        ok = mbar_wait_warp(&sh->q_full, q_phase, abort, a.err, 31);
        q_phase ^= 1;
        if (!ok) break;
        tc_fence_after();
        if (PAIR) {
          const int X = g.count * a.G - g.rt * ROWS > kTile ? 2 : 1;
          for (int x = 0; x < X && ok; ++x) ok = qk(x, x == 0, x == X - 1);
          for (int j = 0; j < n && ok; ++j)
            for (int x = 0; x < X && ok; ++x) {
              ok = pv(x, x == 0, x == X - 1, j > 0);
              if (ok && j + 1 < n) ok = qk(x, x == 0, x == X - 1);
              if (ok && j + 1 == n) finish(x);
            }
        } else {
          ok = qk(0, true, true);
          if (ok && n > 1) ok = qk(1, true, true);
          for (int j = 0; j < n && ok; ++j) {
            ok = pv(j & 1, true, true, j > 1);
            if (ok && j + 2 < n) ok = qk(j & 1, true, true);
            if (ok && j + 2 >= n) finish(j & 1);
          }
        }
      }
      // every product issued here completes before TMEM is released
      if (leader) mma_commit(&sh->mma_done);
      __syncwarp();
      int never = 0;
      mbar_wait(&sh->mma_done, 0, &never, nullptr);
    } else {
      // ------------------------------------------- V rows of the last tiles
      // Both warps follow every V tile and pass it on, so that no barrier's
      // phase runs past a role that waits for it.
      int vseq = 0, seg = 0;
      const int t64 = tid - 64;
      bool ok = true;
      for (; ok && walk.next(a, &g); ++seg) {
        volatile int *flag = &sh->bad[seg % kBadSlots][warp - 2];
        if (lane == 0) *flag = 0;
        __syncwarp();
        for (int k = g.k0; k < g.k1 && ok; ++k, ++vseq) {
          const int st = vseq % VS;
          ok = mbar_wait_warp(&sh->v_full[st], (vseq / VS) & 1, abort, a.err, 22);
          if (!ok) break;
          if ((k + 1) * kTile > g.start) {
            uint8_t *tile = sV + (size_t)st * C::TILE;
            const int first = max(0, g.start - k * kTile), len = g.start + g.count - k * kTile;
#pragma unroll 1
            for (int x = t64; x < (kTile - first) * (D / 8); x += 64) {
              const int row = first + x / (D / 8), ch = x % (D / 8);
              uint4 *p = reinterpret_cast<uint4 *>(tile + (ch >> 3) * C::HALF + row * 128 +
                                                   (((ch & 7) ^ (row & 7)) << 4));
              if (row >= len) {
                *p = make_uint4(0, 0, 0, 0);
              } else {
                const uint4 v = *p;
                if (wild2<T>(v.x) | wild2<T>(v.y) | wild2<T>(v.z) | wild2<T>(v.w)) {
                  clean_word<T>(p);
                  *flag = 1;
                }
              }
            }
            fence_proxy_async_smem();
          }
          warp_arrive(&sh->v_clean[st], lane);
          warp_arrive(&sh->v_empty[st], lane);
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
      __syncwarp();
      tc_fence_after();
      tmem_dealloc(tbase, 512);
    }
    return;
  }
  // ------------------------------------------------------------------ softmax
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
  const int x = (warp - 4) >> 2, quarter = warp & 3;
  const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
  const uint32_t tS = tbase + x * 128 + lane_off;
  const uint32_t tO = tbase + 256 + x * 128 + lane_off;
  const int lrow = quarter * 32 + lane;              // row of the stream's tile
  const int row = (PAIR ? x * kTile : 0) + lrow;     // row of the row tile
  uint32_t seg_phase = 0, s_phase = 0, o_phase = 0;  // o_phase: bit per stream
  auto seg_sync = [&]() {  // the eight warps
    tc_fence_before();
    warp_arrive(&sh->seg, lane);
    const bool ok = mbar_wait_warp(&sh->seg, seg_phase, abort, a.err, 51);
    tc_fence_after();
    seg_phase ^= 1;
    return ok;
  };
  // A thread's 16-byte words of Q: LOADS rows, STEP apart, HELD of them in flight
  // (one after the other: 12 us for 256 rows). The first are read before the wait
  // for Q's place; before the end of the segment in front their registers cost
  // more than they save (5 % on short contexts).
  constexpr int CPR = D / 8, STEP = 256 / CPR, LOADS = ROWS / STEP, HELD = LOADS < 8 ? LOADS : 8;
  const int ch = (tid - 128) % CPR, rq = (tid - 128) / CPR;
  uint4 qv[HELD];
  auto read_q = [&](const Segment &g, int first) {
    const int rows = min(ROWS, g.count * a.G - g.rt * ROWS);
#pragma unroll
    for (int e = 0; e < HELD; ++e) {
      const int r = rq + (first + e) * STEP;
      qv[e] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const int rr = g.rt * ROWS + r, i = rr / a.G, hd = g.h * a.G + rr - i * a.G;
        qv[e] = *reinterpret_cast<const uint4 *>((const T *)a.q.p + (int64_t)g.s * a.q.batch +
                                                 hd * a.q.head + i * a.q.row + ch * 8);
      }
    }
  };
  bool ok = true;
  for (int seg = 0; ok && walk.next(a, &g); ++seg) {
    read_q(g, 0);
    const int rows = min(ROWS, g.count * a.G - g.rt * ROWS);
    const int n = g.k1 - g.k0;
    // Q's place is free once everybody is through with the segment before
    ok = seg_sync();
    if (!ok) break;
#pragma unroll 1
    for (int first = 0; first < LOADS; first += HELD) {
      if (first > 0) read_q(g, first);
#pragma unroll
      for (int e = 0; e < HELD; ++e) {
        const int r = rq + (first + e) * STEP;
        *reinterpret_cast<uint4 *>(sQ + (r / kTile) * C::TILE + (ch >> 3) * C::HALF +
                                   (r % kTile) * 128 + (((ch & 7) ^ (r & 7)) << 4)) = qv[e];
      }
    }
    fence_proxy_async_smem();
    warp_arrive(&sh->q_full, lane);
    const int steps = PAIR ? (rows > x * kTile ? n : 0) : (n + 1 - x) / 2;
    const bool live = (PAIR ? x * kTile : 0) + quarter * 32 < rows;  // warp-uniform
    const int draft = min((g.rt * ROWS + row) / a.G, g.count - 1);
    float m_used = -INFINITY, l = 0.f;
    for (int j = 0; j < steps; ++j) {
      const int key = (g.k0 + (PAIR ? j : 2 * j + x)) * kTile;
      // the masks' words are on their way while S is computed
      const bool edge = key + kTile > g.start;
      uint32_t seen[4];
      if (edge && live) {
#pragma unroll
        for (int c = 0; c < 4; ++c) seen[c] = seen_word(a, g, draft, key + 32 * c);
      }
      if (!mbar_wait_warp(&sh->s_full[x], s_phase, abort, a.err, 41)) {
        ok = false;
        break;
      }
      s_phase ^= 1;
      tc_fence_after();
      if (!live) {  // no row of this warp's exists: its P may be anything
        tc_fence_before();
        warp_arrive(&sh->p_full[x][0], lane);
        warp_arrive(&sh->p_full[x][1], lane);
        continue;
      }
      uint32_t v[kTile];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[c * 32]));
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < kTile; ++c) asm volatile("" : "+r"(v[c]));
      if (edge) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(seen[c] >> e & 1)) v[c * 32 + e] = 0xff800000u;  // -inf
      }
      float m8[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) m8[e] = __uint_as_float(v[e]);
#pragma unroll
      for (int c = 8; c < kTile; c += 8)
#pragma unroll
        for (int e = 0; e < 8; ++e) m8[e] = fmaxf(m8[e], __uint_as_float(v[c + e]));
      const float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                             fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
      const float mxs = reference<T>(mx, a.sl2, kRescaleLog2);
      float alpha = 1.f;
      if (mxs > may_rise<T>(m_used, kRescaleLog2)) {
        alpha = ex2_approx(m_used - mxs);
        m_used = mxs;
      }
      const float mu = m_used == -INFINITY ? 0.f : m_used;
      __syncwarp();
      // O holds every tile before this one: S was signalled after their products
      if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[32];
          tmem_ld32(tO + c * 32, r);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
          tmem_st32(tO + c * 32, r);
        }
        tmem_wait_st();
      }
      const float2 sl = make_float2(a.sl2, a.sl2), neg = make_float2(-mu, -mu);
      float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                       make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 y = __ffma2_rn(make_float2(__uint_as_float(v[c * 32 + 2 * e]),
                                                  __uint_as_float(v[c * 32 + 2 * e + 1])),
                                      sl, neg);
          const float2 p = make_float2(ex2_approx(y.x), ex2_approx(y.y));
          acc[e & 3] = __fadd2_rn(acc[e & 3], p);
          pk[e] = Two<T>::pack(p.x, p.y);
        }
        tmem_st16(tS + c * 16, pk);
        if (c & 1) {
          tmem_wait_st();
          tc_fence_before();
          warp_arrive(&sh->p_full[x][c >> 1], lane);
        }
      }
      const float2 t = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
      l = l * alpha + (t.x + t.y);
    }
    if (!ok) break;
    // ------------------------------------------------------- the item's end
    const int slot = 2 * blockIdx.x + (seg > 0);
    if (tid == 128) tell_item(a, g, sh->place.run, slot);
    const int rr = g.rt * ROWS + row, i = rr / a.G, head = g.h * a.G + rr - i * a.G;
    float top = m_used, sum = l, f[2] = {1.f, 1.f};
    if (!PAIR) {
      // both streams' outputs, half of the columns by each group of warps;
      // the products are through with Q, whose place takes the sums
      for (int y = 0; y < 2 && ok; ++y)
        if (y == 0 || n > 1) {
          ok = mbar_wait_warp(&sh->o_final[y], o_phase >> y & 1, abort, a.err, 44);
          o_phase ^= 1u << y;
        }
      if (!ok) break;
      float2 *ml = reinterpret_cast<float2 *>(sQ);  // [2][kTile]
      ml[x * kTile + lrow] = make_float2(m_used, l);
      ok = seg_sync();
      const float2 p0 = ml[lrow], p1 = ml[kTile + lrow];
      top = fmaxf(p0.x, p1.x);
      f[0] = part_scale(p0.x, top), f[1] = n > 1 ? part_scale(p1.x, top) : 0.f;
      sum = p0.y * f[0] + (n > 1 ? p1.y * f[1] : 0.f);
    } else if (steps) {
      ok = mbar_wait_warp(&sh->o_final[x], o_phase & 1, abort, a.err, 44);
      o_phase ^= 1;
    }
    if (!ok) break;
    tc_fence_after();
    if (live && (!PAIR || steps)) {
      const bool edge = g.k1 * kTile > g.start;
      const volatile int *flags = sh->bad[seg % kBadSlots];
      const int bad = edge ? flags[0] | flags[1] : 0;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      constexpr int CH = PAIR ? D / 32 : D / 64;  // chunks of 32 columns here
#pragma unroll 1
      for (int c = 0; c < CH; ++c) {
        const int col = ((PAIR ? 0 : x * CH) + c) * 32;
        float o[32];
        {
          uint32_t r[32];
          tmem_ld32(tbase + 256 + (PAIR ? x * 128 : 0) + lane_off + col, r);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(r[e]) * f[0];
          if (!PAIR && n > 1) {
            tmem_ld32(tbase + 256 + 128 + lane_off + col, r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] += __uint_as_float(r[e]) * f[1];
          }
        }
        if (row < rows) {
          if (g.whole) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= inv;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              float *w = o + e;
              float y[8] = {w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]};
              if (bad)
                add_wild<T, 8>(a, g.s, g.h, Seq{g.start, g.count}, i, D, col + e, y);
              write_row<T, 8>(a, g.s, head, i, D, col + e, y);
            }
          } else {
            float4 *dst = a.part_o + ((size_t)slot * (D / 4) + col / 4) * ROWS + row;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e * ROWS] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        __syncwarp();
      }
      if (row < rows && (PAIR || x == 0)) {
        if (g.whole)
          write_lse(a, g.s, head, i, top, sum);
        else
          a.part_ml[(size_t)slot * ROWS + row] = make_float2(top, sum);
      }
      if (!g.whole && row == 0 && x == 0) a.part_bad[slot] = bad;
    }
  }
  tc_fence_before();
  __syncthreads();
}

template <typename T, int D, bool PAIR>
cudaError_t run(const CUtensorMap &mk, const CUtensorMap &mv, const TreeArgs &a, int grid,
                cudaStream_t st) {
  using C = Cfg<D, PAIR>;
  constexpr auto kern = tree_tc_kernel<T, D, PAIR>;
  cudaError_t e = allow_smem<kern>((int)C::SMEM);
  if (e != cudaSuccess) return e;
  // the register split is only sound at the launch allocation it is made for
  static std::atomic<int> regs{0};
  if (!regs.load(std::memory_order_relaxed)) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != kLaunchRegs) return cudaErrorInvalidConfiguration;
  e = launch_behind(kern, dim3(grid), kThreads, C::SMEM, st, mk, mv, a);
  if (e != cudaSuccess) return e;
  return launch_combine<T, D, C::ROWS>(a, grid, st);
}

template <typename T>
cudaError_t run_rows(const CUtensorMap &mk, const CUtensorMap &mv, const TreeArgs &a, int d,
                     int rows, int grid, cudaStream_t st) {
  if (d == 64)
    return rows == 256 ? run<T, 64, true>(mk, mv, a, grid, st)
                       : run<T, 64, false>(mk, mv, a, grid, st);
  return rows == 256 ? run<T, 128, true>(mk, mv, a, grid, st)
                     : run<T, 128, false>(mk, mv, a, grid, st);
}

}  // namespace

cudaError_t launch_tree_tc(const CUtensorMap &mk, const CUtensorMap &mv, const TreeArgs &a, int d,
                           int rows, bool bf16, int grid, cudaStream_t st) {
  return bf16 ? run_rows<__nv_bfloat16>(mk, mv, a, d, rows, grid, st)
              : run_rows<__half>(mk, mv, a, d, rows, grid, st);
}

}  // namespace pbs
