// Rotary positions of Q and K in one launch (pbs_rope).
//
// A pair (x0, x1) of a row at position t turns by a = t f:
//   y0 = g (x0 cos a - x1 sin a),  y1 = g (x1 cos a + x0 sin a).
// The work is one read and one write of every element, so the kernel is
// bound by memory (small batches: by latency). A token's angles are the
// same in every head: a thread computes the cosines and sines of its pairs
// once and walks the heads with them, four heads' reads in flight (one at a
// time 123 us, two 112, four 109, eight 133 for 32768 tokens of 32 + 8 heads, d =
// 128, where 671 MB at the copy rate take 102): 6.1 TB/s. 256 threads a block
// write 8 KB in a row of each head (128 threads: 3 % slower, 512: 18 %). A step
// of 16 tokens takes 2.5 us on the device.
//
// Angles. t f in fp32 is off by up to t f 2^-24 radians (0.008 at 131072),
// more than a bf16 result's rounding, and fp64 sine and cosine are slow. So
// f is turned into a 64-bit fixed-point fraction of a turn; t times it in
// integers, modulo 2^64, is the angle modulo one turn without rounding. The
// nearest quarter turn comes off in integers too; what remains is at most an
// eighth of a turn, is cut to 2^-34 turns, rounds to fp32 within 2^-24 of itself and
// goes through sincospif. So an angle is off by pi (2^-27 + 2^-33) radians at most
// (rounded at once, with a half turn's bits: four times as much), besides f's own
// rounding (2^-53 relative, times t).
#include <cuda_fp16.h>

#include "common.cuh"
#include "decode.h"

namespace pbs {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;  // heads whose reads are in flight together

struct RopeArgs {
  pbs_rows q, qo, k, ko;
  const int32_t *pos;
  const double *inv_freq;
  int64_t pos_batch, tokens;
  float gain;
  int hq, heads, n, d, rot, heads_per, transpose;
};

template <typename T>
struct Vec {  // 16 bytes of T as fp32
  static constexpr int V = 16 / sizeof(T);
};

__device__ __forceinline__ void unpack(const uint4 &u, float (&x)[8], __nv_bfloat16) {
  const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(p[i]);
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack(const uint4 &u, float (&x)[8], __half) {
  const __half2 *p = reinterpret_cast<const __half2 *>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(p[i]);
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack(const uint4 &u, float (&x)[4], float) {
  x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y);
  x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint4 pack(const float (&x)[8], __nv_bfloat16) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ uint4 pack(const float (&x)[8], __half) {
  uint4 u;
  __half2 *p = reinterpret_cast<__half2 *>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
  return u;
}
__device__ __forceinline__ uint4 pack(const float (&x)[4], float) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                    __float_as_uint(x[3]));
}

// The V pairs of two vectors turned by their angles. HALF: pair e is element e
// of each; else elements 2e and 2e + 1 of the two together.
template <typename T, bool HALF, int V>
__device__ __forceinline__ void turn(uint4 &v0, uint4 &v1, const float (&c)[V],
                                     const float (&s)[V]) {
  float x0[V], x1[V], y0[V], y1[V];
  unpack(v0, x0, T());
  unpack(v1, x1, T());
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if (HALF) {
      y0[e] = x0[e] * c[e] - x1[e] * s[e];
      y1[e] = x1[e] * c[e] + x0[e] * s[e];
    } else {
      const float p = 2 * e < V ? x0[2 * e % V] : x1[2 * e % V];
      const float r = 2 * e < V ? x0[2 * e % V + 1] : x1[2 * e % V + 1];
      (2 * e < V ? y0 : y1)[2 * e % V] = p * c[e] - r * s[e];
      (2 * e < V ? y0 : y1)[2 * e % V + 1] = r * c[e] + p * s[e];
    }
  }
  v0 = pack(y0, T());
  v1 = pack(y1, T());
}

// A unit is two 16-byte vectors of a head's row. HALF: a rotated unit u
// holds elements [uV, uV + V) and the same from rot/2 on; else the 2V
// elements from 2uV on, V pairs side by side. Units behind rot are copied.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int V = Vec<T>::V;
  const int units = a.d / (2 * V);
  const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t token = at / units;
  if (token >= a.tokens) return;
  const int u = (int)(at - token * units);
  const int64_t b = token / a.n, i = token - b * a.n;
  const bool turns = 2 * u * V < a.rot;
  const int lo = HALF && turns ? u * V : 2 * u * V;
  const int hi = HALF && turns ? a.rot / 2 + u * V : lo + V;
  float c[V], s[V];
  if (turns) {
    const uint64_t t = (uint64_t)(int64_t)__ldg(a.pos + b * a.pos_batch + i);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      double f = __ldg(a.inv_freq + u * V + e) * 0.15915494309189535;  // turns per position
      f -= floor(f);
      const uint64_t angle = t * (uint64_t)(f * 18446744073709551616.0);
      // an eighth of a turn further: whole quarters in the upper two bits, and the
      // rest, less that eighth, in [-1/8, 1/8) turns, its upper 32 bits in 2^-34
      const uint32_t high = (uint32_t)(angle >> 32) + (1u << 29);
      const uint32_t quarter = high >> 30;
      const uint32_t rest = (high << 2 | (uint32_t)angle >> 30) - (1u << 31);
      float sn, cs;
      sincospif((float)(int32_t)rest * 0x1p-33f, &sn, &cs);  // half turns
      const uint32_t x = __float_as_uint(quarter & 1 ? sn : cs);
      const uint32_t y = __float_as_uint(quarter & 1 ? cs : sn);
      c[e] = __uint_as_float(x ^ ((quarter + 1) & 2) << 30) * a.gain;
      s[e] = __uint_as_float(y ^ (quarter & 2) << 30) * (a.transpose ? -a.gain : a.gain);
    }
  }
  const int h0 = blockIdx.y * a.heads_per, h1 = min(h0 + a.heads_per, a.heads);
  // the q heads of this block's share, then the k heads
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const pbs_rows &x = part ? a.k : a.q, &y = part ? a.ko : a.qo;
    const int off = part ? a.hq : 0;
    const int first = max(h0, off) - off, end = (part ? h1 : min(h1, a.hq)) - off;
    const T *src = (const T *)x.p + b * x.batch + i * x.row;
    T *dst = (T *)y.p + b * y.batch + i * y.row;
#pragma unroll 1
    for (int h = first; h < end; h += kHeads) {
      uint4 v0[kHeads], v1[kHeads];
#pragma unroll
      for (int e = 0; e < kHeads; ++e)
        if (h + e < end) {
          const T *p = src + (h + e) * x.head;
          v0[e] = *reinterpret_cast<const uint4 *>(p + lo);
          v1[e] = *reinterpret_cast<const uint4 *>(p + hi);
        }
#pragma unroll
      for (int e = 0; e < kHeads; ++e)
        if (h + e < end) {
          if (turns) turn<T, HALF>(v0[e], v1[e], c, s);
          T *p = dst + (h + e) * y.head;
          *reinterpret_cast<uint4 *>(p + lo) = v0[e];
          *reinterpret_cast<uint4 *>(p + hi) = v1[e];
        }
    }
  }
}

template <typename T>
void launch(const RopeArgs &a, dim3 grid, bool half, cudaStream_t st) {
  if (half)
    rope_kernel<T, true><<<grid, kThreads, 0, st>>>(a);
  else
    rope_kernel<T, false><<<grid, kThreads, 0, st>>>(a);
}

// Whether some i < n, j < m of every dimension have sum (i - j) s = off, up to
// less than d elements; `dims` by falling stride.
struct MeetDim {
  int64_t s, n, m;
};
bool dims_meet(const MeetDim *dims, int k, int64_t off, int d) {
  if (k == 0) return off < d && -off < d;
  int64_t rest = d - 1;
  for (int i = 1; i < k; ++i)
    rest += dims[i].s * ((dims[i].n > dims[i].m ? dims[i].n : dims[i].m) - 1);
  // |off - t s| <= rest, -m < t < n
  auto down = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
  int64_t lo = -down(rest - off, dims->s), hi = down(off + rest, dims->s);
  if (lo < 1 - dims->m) lo = 1 - dims->m;
  if (hi > dims->n - 1) hi = dims->n - 1;
  if (hi - lo > 3) return true;  // strides that reach into one another: taken to meet
  for (int64_t t = lo; t <= hi; ++t)
    if (dims_meet(dims + 1, k - 1, off - t * dims->s, d)) return true;
  return false;
}

}  // namespace

bool rows_meet(const RowSet &x, const void *p, int64_t bytes) {
  if (x.empty()) return false;
  return bytes_meet(x.low(), x.bytes(), p, bytes);
}

bool rows_meet(const RowSet &x, const RowSet &y) {
  if (x.empty() || y.empty()) return false;
  if (!bytes_meet(x.low(), x.bytes(), y.low(), y.bytes())) return false;
  const int64_t bytes = (intptr_t)y.r.p - (intptr_t)x.r.p;
  if (!x.plain() || !y.plain() || x.elem != y.elem || x.d != y.d || bytes % x.elem) return true;
  const int64_t s[2][3] = {{x.r.batch, x.r.head, x.r.row}, {y.r.batch, y.r.head, y.r.row}};
  const int64_t n[2][3] = {{x.batch, x.heads, x.n}, {y.batch, y.heads, y.n}};
  MeetDim dims[3];
  int k = 0;
  for (int i = 0; i < 3; ++i) {
    if (n[0][i] == 1 && n[1][i] == 1) continue;
    const int64_t st = n[0][i] == 1 ? s[1][i] : s[0][i];
    if (n[0][i] > 1 && n[1][i] > 1 && s[0][i] != s[1][i]) return true;
    if (st == 0) continue;
    int at = k++;
    for (; at > 0 && dims[at - 1].s < st; --at) dims[at] = dims[at - 1];
    dims[at] = {st, n[0][i], n[1][i]};
  }
  return dims_meet(dims, k, bytes / x.elem, x.d);
}

}  // namespace pbs

using namespace pbs;

extern "C" pbs_status pbs_rope(pbs_rows q, pbs_rows q_out, int hq, pbs_rows k, pbs_rows k_out,
                               int hkv, const int32_t *pos, int64_t pos_batch,
                               const double *inv_freq, float gain, int batch, int n, int d,
                               int rot, int layout, int transpose, int dtype, pbs_stream_t st) {
  if (batch < 0 || n < 0 || hq < 0 || hkv < 0 || hq > (1 << 20) || hkv > (1 << 20) || d < 16 ||
      d > 1024 || d % 16 || rot < 0 || rot > d || rot % 16 || layout < 0 || layout > 1 ||
      dtype < PBS_BF16 || dtype > PBS_FP32)
    return PBS_ERR_INVALID_ARG;
  if (batch == 0 || n == 0 || hq + hkv == 0) return PBS_OK;
  const int elem = dtype == PBS_FP32 ? 4 : 2;
  if ((hq > 0 && (!rows_ok(q, elem) || !rows_ok(q_out, elem))) ||
      (hkv > 0 && (!rows_ok(k, elem) || !rows_ok(k_out, elem))) || !pos ||
      ((uintptr_t)pos & 3u) || (rot > 0 && (!inv_freq || ((uintptr_t)inv_freq & 7u))))
    return PBS_ERR_INVALID_ARG;
  // an output may be its own input, rows and all, and otherwise meets nothing
  const RowSet sets[4] = {{q, batch, hq, n, d, elem},
                          {k, batch, hkv, n, d, elem},
                          {q_out, batch, hq, n, d, elem},
                          {k_out, batch, hkv, n, d, elem}};
  const int64_t pos_reach = pos_batch * (batch - 1);
  const int32_t *pos_low = pos + (pos_reach < 0 ? pos_reach : 0);
  const int64_t pos_bytes = 4 * ((pos_reach < 0 ? -pos_reach : pos_reach) + n);
  for (int o = 2; o < 4; ++o) {
    for (int i = 0; i < o; ++i) {
      const pbs_rows &x = sets[i].r, &y = sets[o].r;
      const bool own = i == o - 2 && x.p == y.p && (batch == 1 || x.batch == y.batch) &&
                       (sets[i].heads == 1 || x.head == y.head) && (n == 1 || x.row == y.row);
      if (!own && rows_meet(sets[i], sets[o])) return PBS_ERR_INVALID_ARG;
    }
    if (rows_meet(sets[o], pos_low, pos_bytes) || rows_meet(sets[o], inv_freq, 4ll * rot))
      return PBS_ERR_INVALID_ARG;
  }
  RopeArgs a{q, q_out, k, k_out, pos, inv_freq, pos_batch, (int64_t)batch * n, gain};
  a.hq = hq, a.heads = hq + hkv, a.n = n, a.d = d, a.rot = rot, a.transpose = transpose != 0;
  const int64_t bx = ceil_div(a.tokens * (d * elem / 32), kThreads);
  if (bx > 0x7fffffff) return PBS_ERR_UNSUPPORTED;
  // few tokens: the heads are split over blocks until there are sixteen blocks
  // an SM, and the angles computed again in each (12252 tokens of 15 fp32 heads:
  // 33.7 us, with eight blocks an SM 35.8)
  int64_t split = ceil_div(16 * sm_count_cached(), bx);
  if (split > a.heads) split = a.heads;
  a.heads_per = (int)ceil_div(a.heads, split);
  if (ceil_div(a.heads, a.heads_per) > 65535) return PBS_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)bx, (unsigned)ceil_div(a.heads, a.heads_per));
  cudaStream_t cs = (cudaStream_t)st;
  if (dtype == PBS_BF16)
    launch<__nv_bfloat16>(a, grid, layout == 0, cs);
  else if (dtype == PBS_FP16)
    launch<__half>(a, grid, layout == 0, cs);
  else
    launch<float>(a, grid, layout == 0, cs);
  return cudaGetLastError() == cudaSuccess ? PBS_OK : PBS_ERR_CUDA;
}
