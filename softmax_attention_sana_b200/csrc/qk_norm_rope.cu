// Rotary positions of queries and keys, with or without the per-head RMS norm
// in the same pass, and the gradient of that pass.
//
//   y = m R(p) (w * x * r),   r = 1 / sqrt(mean_d x_d^2 + eps)   (norm)
//   y = m R(p) x                                                 (rotation only)
//
// for every (token, head) row x of head_dim elements; R(p) turns pair j by the
// table's angle at the token's position p, m is a factor of the queries.  Both
// layouts fold into one form: with the pair partner x' of each element,
//   y = r (c x + s x'),  c = m w cos,  s = -+ m w' sin,
// so a warp forms c and s once per token and spends two multiply-adds per
// element and head.  Gradient, with g = m R(p)^T dy:
//   dw = sum_rows g x r,   dx = r (w g - x r^2 mean_d(w g x)).
//
// Bound by HBM: each element is read once and written once (the gradient reads
// x and dy and writes dx); the table adds 8 bytes per pair and token.  What holds
// it from there is the instruction count, so arithmetic runs in packed pairs and
// a warp walks all heads of one token, queries and then keys, with one lookup of
// the angles.  A lane holds 8 consecutive elements of a row (16-byte accesses) and
// a row sits in head_dim / 8 neighbouring lanes (the partner in the half layout
// is a shuffle away), several row groups in flight.  480p grid (32760 tokens, 16 + 16
// heads of 128, bf16): 85 us for 537 MB, 96% of the measured HBM rate; 2 x 8192 tokens,
// 32 + 8 heads (335 MB) from flushed caches: 62 us interleaved, 68 half (which spills,
// kResident), the rotation alone 61 and 62; their gradient (503 MB) 100 and 106 us (two
// tensors to load: 77 and 72%).  Bulk copies into a ring in shared memory instead of
// loads to registers, on the 480p grid: 126 us.
#include "f32x2.cuh"
#include "pdl_read.cuh"
#include "rope_dev.cuh"
#include "sana_common.cuh"
#include "sana_internal.h"

namespace sana {
namespace {

constexpr int kWarps = 4;      // warps per CTA: a warp does one token, short CTAs drain evenly
constexpr int kWarpsBwd = 8;   // warps per CTA of the gradient, which is persistent
constexpr int kUnroll = 4;     // row groups a warp has in flight (forward)
// The same for the gradient, which loads two tensors (fp32 rows are twice as wide).
template <class T>
constexpr int kUnrollBwd = sizeof(T) == 2 ? 4 : 2;
// CTAs on an SM that the forward's registers are held to (bf16: 480p grid, 16 heads
// of 128, interleaved: 87 us against 91 us unheld; fp32 rows need the registers).  Held
// so, every bf16 form of the half layout spills (156 to 252 bytes of stores a thread);
// a bound of its own has not been measured.
template <class T>
constexpr int kResident = sizeof(T) == 2 ? 7 : 4;

__device__ __forceinline__ void report_bad_position(int* status) {
  atomicCAS(status, 0, kDevBadPosition << 16);
}

// Eight consecutive elements of a row as loaded.
template <class T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint32_t r[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
    r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
  }
  __device__ __forceinline__ void zero() { r[0] = r[1] = r[2] = r[3] = 0; }
  __device__ __forceinline__ Vec8 from_lane(int src) const {
    Vec8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.r[i] = __shfl_sync(0xffffffffu, r[i], src);
    return o;
  }
  __device__ __forceinline__ void get(uint64_t (&f)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = bf2_to_f2(r[i]);
      f[i] = pk2(v.x, v.y);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const uint64_t (&f)[4]) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      up2(f[i], a, b);
      o[i] = f2_to_bf2(a, b);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(o[0], o[1], o[2], o[3]));
  }
};
template <>
struct Vec8<float> {
  float r[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
    r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = 0.f;
  }
  __device__ __forceinline__ Vec8 from_lane(int src) const {
    Vec8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.r[i] = __shfl_sync(0xffffffffu, r[i], src);
    return o;
  }
  __device__ __forceinline__ void get(uint64_t (&f)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pk2(r[2 * i], r[2 * i + 1]);
  }
  static __device__ __forceinline__ void store(float* p, const uint64_t (&f)[4]) {
    float o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) up2(f[i], o[2 * i], o[2 * i + 1]);
    __stcs(reinterpret_cast<float4*>(p), make_float4(o[0], o[1], o[2], o[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(o[4], o[5], o[6], o[7]));
  }
};

// cos and sin of this lane's elements at one token: four pairs where neighbours
// pair up, eight where element i pairs with element i + pairs (the lane's own
// pairs then start at its column, taken modulo the half).
template <int LPR, bool HALF>
struct Turn {
  static constexpr int kP = HALF ? 8 : 4;
  float c[kP], s[kP];
  bool on;       // this lane's eight elements are rotated (rotary_dim is a multiple of 16)
  bool second;   // half layout: the lane holds the pairs' second elements
  int partner;   // half layout: the warp lane that holds the partners

  __device__ __forceinline__ void init(const RotaryDev& rt, int lane) {
    const int sub = lane % LPR;
    on = sub * 8 < 2 * rt.pairs;
    second = HALF && sub * 8 >= rt.pairs;
    const int hop = rt.pairs / 8;
    partner = HALF && on ? (second ? lane - hop : lane + hop) : lane;
  }
  // The table entries at token (b, n); a position outside the table is taken as
  // its nearest row and reported.
  __device__ __forceinline__ void fetch(const RotaryDev& rt, int b, int n, int lane, int* status) {
    if (!on) {
#pragma unroll
      for (int i = 0; i < kP; ++i) c[i] = 1.f, s[i] = 0.f;
      return;
    }
    const int sub = lane % LPR;
    const int j0 = HALF ? (second ? sub * 8 - rt.pairs : sub * 8) : sub * 4;
    if (rt.table) {
      int p = rt.offset + n;
      if (rt.positions) {
        const long long at = (long long)rt.offset + rt.positions[(size_t)b * rt.N + n];
        p = (int)(at < 0 ? 0 : at >= rt.max_positions ? rt.max_positions - 1 : at);
        if (p != at) report_bad_position(status);
      }
      const float4* row = reinterpret_cast<const float4*>(rt.table + ((size_t)p * rt.pairs + j0) * 2);
#pragma unroll
      for (int i = 0; i < kP / 2; ++i) {
        const float4 v = __ldg(row + i);
        c[2 * i] = v.x; s[2 * i] = v.y; c[2 * i + 1] = v.z; s[2 * i + 1] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        const float2 cs = rope_cs_global(rt.rope, rt.grid, b, n, j0 + i);
        c[i] = cs.x;
        s[i] = cs.y;
      }
    }
    if (rt.inverse) {
#pragma unroll
      for (int i = 0; i < kP; ++i) s[i] = -s[i];
    }
  }
  // Element i of the turned row is own(i) * x_i + other(i) * x'_i; `back` gives
  // the transposed rotation.
  __device__ __forceinline__ float own(int i) const { return HALF ? c[i % kP] : c[(i >> 1) % kP]; }
  __device__ __forceinline__ float other(int i, bool back) const {
    if (HALF) return second != back ? s[i % kP] : -s[i % kP];
    return ((i & 1) != 0) != back ? s[(i >> 1) % kP] : -s[(i >> 1) % kP];
  }
  // a * x + b * x' for the row of v, x its elements in pairs (partners count as
  // zero where the lane is not rotated, so that an infinity there meets no 0 * inf).
  template <class T>
  __device__ __forceinline__ void apply(const Vec8<T>& v, const uint64_t (&x)[4], const uint64_t (&a)[4],
                                        const uint64_t (&b)[4], uint64_t (&y)[4]) const {
    uint64_t xp[4];
    if (HALF) {
      v.from_lane(partner).get(xp);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        up2(x[i], lo, hi);
        xp[i] = pk2(hi, lo);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = fma2(b[i], on ? xp[i] : 0ull, mul2(a[i], x[i]));
  }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = LPR / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Sums of u and v over a row's LPR lanes: neighbours share the work after the
// first step (one shuffle for both), and swap the results at the end.
template <int LPR>
__device__ __forceinline__ void row_sum2(float& u, float& v, int lane) {
  const bool odd = lane & 1;
  float mine = odd ? v : u;
  mine += __shfl_xor_sync(0xffffffffu, odd ? u : v, 1);
#pragma unroll
  for (int m = 2; m < LPR; m <<= 1) mine += __shfl_xor_sync(0xffffffffu, mine, m);
  const float other = __shfl_xor_sync(0xffffffffu, mine, 1);
  u = odd ? other : mine;
  v = odd ? mine : other;
}
__device__ __forceinline__ float sum_squares(const uint64_t (&f)[4]) {
  uint64_t s = mul2(f[0], f[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fma2(f[i], f[i], s);
  float a, b;
  up2(s, a, b);
  return a + b;
}
__device__ __forceinline__ void load_w(const float* w, int col, uint64_t (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = w ? pk2(__ldg(w + col + 2 * i), __ldg(w + col + 2 * i + 1)) : pk2(1.f, 1.f);
}

// One warp: one token and `per_warp` row groups of it (a group: 32 / LPR heads),
// numbered through its queries and then its keys.
template <class T, int LPR, bool HALF, bool NORM>
__global__ void __launch_bounds__(32 * kWarps, kResident<T>)
    qk_norm_rope_kernel(const QkTensors a, const RotaryDev rt, int chunks, int per_warp, float eps,
                        float q_mul, int* status) {
  constexpr int D = LPR * 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31;
  const long long task = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long token = chunks == 1 ? task : task / chunks;
  if (token >= (long long)a.B * a.N) return;
  const int chunk = chunks == 1 ? 0 : (int)(task - token * chunks);
  const int b = (int)((unsigned)token / (unsigned)a.N), n = (int)token - b * a.N;
  const int groups_q = (a.heads + RPW - 1) / RPW, groups_k = (a.kv_heads + RPW - 1) / RPW;
  const int g0 = chunk * per_warp, g1 = min(groups_q + groups_k, g0 + per_warp);
  const int col = (lane % LPR) * 8, sub_row = lane / LPR;

  Turn<LPR, HALF> turn;
  turn.init(rt, lane);
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const bool is_q = side == 0;
    const int heads = is_q ? a.heads : a.kv_heads;
    const int lo = is_q ? g0 : max(g0 - groups_q, 0), hi = is_q ? min(g1, groups_q) : g1 - groups_q;
    if (lo < hi) {
      const int h1 = min(heads, hi * RPW);
      const T* x = static_cast<const T*>(is_q ? a.q : a.k) + (size_t)token * (is_q ? a.q_stride : a.k_stride) + col;
      T* y = static_cast<T*>(is_q ? a.q_out : a.k_out) + (size_t)token * heads * D + col;
      Vec8<T> raw[kUnroll];
      auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int hr = h + u * RPW + sub_row;
          if (hr < h1) raw[u].load(x + (size_t)hr * D);
          else raw[u].zero();
        }
      };
      load(lo * RPW);  // the rows' loads start before the table is looked up
      if (is_q || g0 >= groups_q) turn.fetch(rt, b, n, lane, status);
      uint64_t ca[4], cb[4];
      {
        const float m = is_q ? q_mul : 1.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ca[i] = pk2(m * turn.own(2 * i), m * turn.own(2 * i + 1));
          cb[i] = pk2(m * turn.other(2 * i, false), m * turn.other(2 * i + 1, false));
        }
        const float* w = is_q ? a.wq : a.wk;
        if (NORM && w) {
          uint64_t wo[4], wp[4];
          load_w(w, col, wo);
          if (HALF) load_w(w, (turn.partner % LPR) * 8, wp);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (!HALF) {
              float p0, p1;
              up2(wo[i], p0, p1);
              wp[i] = pk2(p1, p0);
            }
            ca[i] = mul2(ca[i], wo[i]);
            cb[i] = mul2(cb[i], wp[i]);
          }
        }
      }
      for (int h = lo * RPW; h < h1; h += kUnroll * RPW) {
        if (h > lo * RPW) load(h);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (h + u * RPW >= h1) break;  // warp-uniform
          const int hr = h + u * RPW + sub_row;
          uint64_t f[4], o[4];
          raw[u].get(f);
          turn.apply(raw[u], f, ca, cb, o);
          if (NORM) {
            const float r = rsqrtf(row_sum<LPR>(sum_squares(f)) * (1.f / D) + eps);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = mul2(o[i], pk2(r, r));
          }
          if (hr < h1) Vec8<T>::store(y + (size_t)hr * D, o);
        }
      }
    }
  }
}

// Gradient.  The work is a row of steps, per token those of its query heads
// (kUnrollBwd row groups each) and then those of its key heads; every warp takes
// an equal run of them (whole tokens to a warp left the last round a third empty:
// 2 x 4001 tokens 56 against 51 us) and adds the weights' gradient in registers
// over its run; the CTA's warps are then added in warp order and the CTA's sums
// written out, to be added in CTA order by the next kernel: the summation order
// depends on the shape alone.
template <class T, int LPR, bool HALF>
__global__ void __launch_bounds__(32 * kWarpsBwd, 2)
    qk_norm_rope_bwd_kernel(const QkTensors a, const RotaryDev rt, float eps, float q_mul,
                            float* __restrict__ dw_part, int* status) {
  griddep_launch_next();
  constexpr int D = LPR * 8, RPW = 32 / LPR, kU = kUnrollBwd<T>;
  __shared__ float red[kWarpsBwd][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = (lane % LPR) * 8, sub_row = lane / LPR;
  Turn<LPR, HALF> turn;
  turn.init(rt, lane);
  uint64_t dw[2][4] = {};
  const int steps_q = (a.heads + kU * RPW - 1) / (kU * RPW), steps_k = (a.kv_heads + kU * RPW - 1) / (kU * RPW);
  const int per_token = steps_q + steps_k;
  const long long all = (long long)a.B * a.N * per_token, warps = (long long)gridDim.x * kWarpsBwd;
  const long long me = (long long)blockIdx.x * kWarpsBwd + warp;
  long long left = all * (me + 1) / warps - all * me / warps;
  long long token = all * me / warps / per_token;
  int step = (int)(all * me / warps - token * per_token);
  bool fresh = true;  // the token's angles have to be looked up
  for (; left > 0; --left) {
    const bool is_q = step < steps_q;
    const int heads = is_q ? a.heads : a.kv_heads;
    const int h = (is_q ? step : step - steps_q) * kU * RPW;
    const T* x = static_cast<const T*>(is_q ? a.q : a.k) + (size_t)token * (is_q ? a.q_stride : a.k_stride) + col;
    const T* dy = static_cast<const T*>(is_q ? a.dq_out : a.dk_out) + (size_t)token * heads * D + col;
    T* dx = static_cast<T*>(is_q ? a.q_out : a.k_out) + (size_t)token * heads * D + col;
    Vec8<T> rx[kU], rg[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int hr = h + u * RPW + sub_row;
      if (hr < heads) {
        rx[u].load(x + (size_t)hr * D);
        rg[u].load(dy + (size_t)hr * D);
      } else {
        rx[u].zero();
        rg[u].zero();
      }
    }
    if (fresh) {
      const int b = (int)((unsigned)token / (unsigned)a.N);
      turn.fetch(rt, b, (int)token - b * a.N, lane, status);
    }
    const float m = is_q ? q_mul : 1.f;
    uint64_t ca[4], cb[4], w[4], sum[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ca[i] = pk2(m * turn.own(2 * i), m * turn.own(2 * i + 1));
      cb[i] = pk2(m * turn.other(2 * i, true), m * turn.other(2 * i + 1, true));
    }
    load_w(is_q ? a.wq : a.wk, col, w);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (h + u * RPW >= heads) break;  // warp-uniform
      const int hr = h + u * RPW + sub_row;
      uint64_t f[4], d[4], g[4];
      rx[u].get(f);
      rg[u].get(d);
      turn.apply(rg[u], d, ca, cb, g);
      float ss = sum_squares(f), dot, t1;
      uint64_t gf = 0, gw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        gw[i] = mul2(g[i], w[i]);
        gf = fma2(gw[i], f[i], gf);
      }
      up2(gf, dot, t1);
      dot += t1;
      row_sum2<LPR>(ss, dot, lane);
      // (rows past the last head: 1 / sqrt(0) of their zeros would reach dw for eps = 0)
      const float r = hr < heads ? rsqrtf(ss * (1.f / D) + eps) : 0.f;
      // dot is of the size of 1 / r: taken in turn with it, r^3 leaves fp32 on neither side
      const float k3 = -(dot * (1.f / D) * r) * (r * r);
      const uint64_t r2 = pk2(r, r), k32 = pk2(k3, k3);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum[i] = fma2(g[i], mul2(f[i], r2), sum[i]);
        g[i] = fma2(k32, f[i], mul2(r2, gw[i]));
      }
      if (hr < heads) Vec8<T>::store(dx + (size_t)hr * D, g);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (is_q) dw[0][i] = add2(dw[0][i], sum[i]);
      else dw[1][i] = add2(dw[1][i], sum[i]);
    }
    fresh = ++step == per_token;
    if (fresh) {
      step = 0;
      ++token;
    }
  }
  // rows of the warp, then warps of the CTA, in a fixed order
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v, v1;
      up2(dw[side][i >> 1], v, v1);
      if (i & 1) v = v1;
#pragma unroll
      for (int mk = LPR; mk < 32; mk <<= 1) v += __shfl_xor_sync(0xffffffffu, v, mk);
      if (sub_row == 0) red[warp][side][col + i] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += 32 * kWarpsBwd) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWarpsBwd; ++k) v += red[k][i / D][i % D];
    dw_part[(size_t)blockIdx.x * 2 * D + i] = v;
  }
}

// dw[i] = sum over CTAs of part[cta][i]: 32 columns per CTA, each thread row
// adds every 32nd partial, then the 32 rows are added in order.
__global__ void __launch_bounds__(1024)
    qk_dw_reduce_kernel(const float* part, int parts, int D, float* dwq, float* dwk) {
  part = griddep_wait_for(part);
  __shared__ float red[32][33];
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + c;
  float v = 0.f;
  if (i < 2 * D)
    for (int p = r; p < parts; p += 32) v += part[(size_t)p * 2 * D + i];
  red[r][c] = v;
  __syncthreads();
  if (r != 0 || i >= 2 * D) return;
  v = 0.f;
  for (int k = 0; k < 32; ++k) v += red[k][c];
  if (i < D) {
    if (dwq) dwq[i] = v;
  } else if (dwk) {
    dwk[i - D] = v;
  }
}

struct Inv128 {
  double f[128];
};
// cos and sin of every (position, pair), angles and functions in 64 bits.
__global__ void rotary_table_kernel(float2* table, int max_positions, int pairs, const Inv128 inv,
                                    double mul) {
  const long long total = (long long)max_positions * pairs;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const long long p = i / pairs;
    double s, c;
    sincos((double)p * inv.f[(int)(i - p * pairs)], &s, &c);
    table[i] = make_float2((float)(c * mul), (float)(s * mul));
  }
}

// Grid of the gradient kernel: two CTAs per SM, fewer for few tokens.
int bwd_ctas(long long tokens) {
  const long long c = (tokens + kWarpsBwd - 1) / kWarpsBwd;
  return (int)(c < 2 * kNumSMs ? c : 2 * kNumSMs);
}

template <class T, int LPR, bool HALF>
void launch_fwd(const QkTensors& a, const RotaryDev& rt, bool norm, float eps, float q_mul,
                cudaStream_t st) {
  constexpr int RPW = 32 / LPR;
  // A warp takes as many heads of its token as leave 16 warps for every SM:
  // all of them for long inputs (the table lookup is then shared by all
  // heads), one row group each for a decoding step (latency).
  const long long tokens = (long long)a.B * a.N;
  const int groups = (a.heads + RPW - 1) / RPW + (a.kv_heads + RPW - 1) / RPW;
  const long long want = (16 * kNumSMs + tokens - 1) / tokens;  // warps per token
  int per = (int)((groups + want - 1) / want);
  if (per < 1) per = 1;
  const int chunks = (groups + per - 1) / per;
  const dim3 grid((unsigned)((tokens * chunks + kWarps - 1) / kWarps));
  int* sw = status_word();
  if (norm)
    qk_norm_rope_kernel<T, LPR, HALF, true><<<grid, 32 * kWarps, 0, st>>>(a, rt, chunks, per, eps, q_mul, sw);
  else
    qk_norm_rope_kernel<T, LPR, HALF, false><<<grid, 32 * kWarps, 0, st>>>(a, rt, chunks, per, eps, q_mul, sw);
}

template <class T, int LPR, bool HALF>
void launch_bwd(const QkTensors& a, const RotaryDev& rt, float eps, float q_mul, float* dwq,
                float* dwk, float* ws, cudaStream_t st) {
  const int ctas = bwd_ctas((long long)a.B * a.N);
  if (ctas)  // no tokens: the sums over nothing below are zeros
    qk_norm_rope_bwd_kernel<T, LPR, HALF><<<ctas, 32 * kWarpsBwd, 0, st>>>(a, rt, eps, q_mul, ws, status_word());
  launch_dependent(qk_dw_reduce_kernel, dim3((2 * LPR * 8 + 31) / 32), dim3(1024), 0, st, ws, ctas, LPR * 8, dwq, dwk);
}

// Calls f with the compile-time (type, lanes per row, layout) of the call.
template <class F>
bool dispatch(sana_dtype dt, int head_dim, bool half, F&& f) {
  auto by_dim = [&](auto t, auto hf) {
    switch (head_dim) {
      case 16: f(t, std::integral_constant<int, 2>{}, hf); return true;
      case 32: f(t, std::integral_constant<int, 4>{}, hf); return true;
      case 64: f(t, std::integral_constant<int, 8>{}, hf); return true;
      case 128: f(t, std::integral_constant<int, 16>{}, hf); return true;
      case 256: f(t, std::integral_constant<int, 32>{}, hf); return true;
      default: return false;
    }
  };
  auto by_layout = [&](auto t) {
    return half ? by_dim(t, std::true_type{}) : by_dim(t, std::false_type{});
  };
  return dt == SANA_BF16 ? by_layout(__nv_bfloat16{}) : by_layout(float{});
}

}  // namespace

sana_status rotary_table_run(float* table, int max_positions, int pairs, const double* inv,
                             double mul, cudaStream_t st) {
  Inv128 v{};
  for (int i = 0; i < pairs; ++i) v.f[i] = inv[i];
  const long long total = (long long)max_positions * pairs;
  const long long blocks = (total + 255) / 256;
  rotary_table_kernel<<<(unsigned)(blocks < 16 * kNumSMs ? blocks : 16 * kNumSMs), 256, 0, st>>>(
      reinterpret_cast<float2*>(table), max_positions, pairs, v, mul);
  return check_launch("rotary_table_kernel");
}

sana_status qk_norm_rope_run(const QkTensors& a, sana_dtype dt, const RotaryDev& rt, bool norm,
                             float eps, float q_mul, cudaStream_t st) {
  dispatch(dt, a.head_dim, rt.half, [&](auto t, auto lpr, auto hf) {
    launch_fwd<decltype(t), decltype(lpr)::value, decltype(hf)::value>(a, rt, norm, eps, q_mul, st);
  });
  return check_launch("qk_norm_rope_kernel");
}

size_t qk_norm_rope_bwd_ws_bytes(long long tokens, int head_dim) {
  return align_up((size_t)bwd_ctas(tokens) * 2 * head_dim * sizeof(float), 256);
}

sana_status qk_norm_rope_bwd_run(const QkTensors& a, sana_dtype dt, const RotaryDev& rt, float eps,
                                 float q_mul, float* dwq, float* dwk, void* ws, cudaStream_t st) {
  dispatch(dt, a.head_dim, rt.half, [&](auto t, auto lpr, auto hf) {
    launch_bwd<decltype(t), decltype(lpr)::value, decltype(hf)::value>(
        a, rt, eps, q_mul, dwq, dwk, static_cast<float*>(ws), st);
  });
  return check_launch("qk_norm_rope_bwd_kernel");
}

}  // namespace sana
