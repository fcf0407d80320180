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
// x and dy and writes dx); the table adds 8 bytes per pair and token.  A lane
// holds 8 consecutive elements of a row (16-byte accesses), a row sits in
// head_dim / 8 neighbouring lanes (the partner in the half layout is a shuffle
// away), and a warp walks the heads of one token, four row groups in flight.
#include "pdl.cuh"
#include "rope_dev.cuh"
#include "sana_common.cuh"
#include "sana_internal.h"

namespace sana {
namespace {

constexpr int kWarps = 8;      // warps per CTA
constexpr int kUnroll = 4;     // row groups a warp has in flight (forward)
constexpr int kUnrollBwd = 2;  // the same for the gradient, which loads two tensors

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
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = bf2_to_f2(r[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8]) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(f2_to_bf2(f[0], f[1]), f2_to_bf2(f[2], f[3]),
                                                  f2_to_bf2(f[4], f[5]), f2_to_bf2(f[6], f[7])));
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
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = r[i];
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
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
  // The pair partners of v (zeros where the lane is not rotated, so that an
  // infinity there meets no 0 * inf).
  template <class T>
  __device__ __forceinline__ void partners(const Vec8<T>& v, const float (&x)[8], float (&xp)[8]) const {
    if (HALF) {
      v.from_lane(partner).get(xp);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) xp[i] = x[i ^ 1];
    }
    if (!on) {
#pragma unroll
      for (int i = 0; i < 8; ++i) xp[i] = 0.f;
    }
  }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = LPR / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

__device__ __forceinline__ void load_w(const float* w, int col, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = w ? __ldg(w + col + i) : 1.f;
}

// One warp: one token and `per_warp` of its query heads, or of its key heads.
template <class T, int LPR, bool HALF, bool NORM>
__global__ void __launch_bounds__(32 * kWarps)
    qk_norm_rope_kernel(const QkTensors a, const RotaryDev rt, int chunks_q, int chunks_k,
                        int per_warp, float eps, float q_mul, int* status) {
  constexpr int D = LPR * 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31;
  const long long task = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int chunks = chunks_q + chunks_k;
  const long long token = task / chunks;
  if (token >= (long long)a.B * a.N) return;
  const int chunk = (int)(task - token * chunks);
  const bool is_q = chunk < chunks_q;
  const int b = (int)(token / a.N), n = (int)(token - (long long)b * a.N);
  const int heads = is_q ? a.heads : a.kv_heads;
  const int h0 = (is_q ? chunk : chunk - chunks_q) * per_warp;
  const int h1 = min(heads, h0 + per_warp);
  const T* x = static_cast<const T*>(is_q ? a.q : a.k) + (size_t)token * (is_q ? a.q_stride : a.k_stride);
  T* y = static_cast<T*>(is_q ? a.q_out : a.k_out) + (size_t)token * heads * D;
  const int col = (lane % LPR) * 8, sub_row = lane / LPR;

  // the rows' loads start before the table is looked up
  Vec8<T> raw[kUnroll];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int hr = h + u * RPW + sub_row;
      if (hr < h1) raw[u].load(x + (size_t)hr * D + col);
      else raw[u].zero();
    }
  };
  load(h0);

  Turn<LPR, HALF> turn;
  turn.init(rt, lane);
  turn.fetch(rt, b, n, lane, status);
  float ca[8], cb[8];
  {
    const float m = is_q ? q_mul : 1.f;
    const float* w = is_q ? a.wq : a.wk;
    float wo[8], wp[8];
    if (NORM) {
      load_w(w, col, wo);
      load_w(w, HALF ? (turn.partner % LPR) * 8 : col, wp);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ca[i] = m * turn.own(i) * (NORM ? wo[i] : 1.f);
      cb[i] = m * turn.other(i, false) * (NORM ? (HALF ? wp[i] : wp[i ^ 1]) : 1.f);
    }
  }
  for (int h = h0; h < h1; h += kUnroll * RPW) {
    if (h > h0) load(h);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h + u * RPW >= h1) break;  // warp-uniform
      const int hr = h + u * RPW + sub_row;
      float f[8], fp[8];
      raw[u].get(f);
      turn.partners(raw[u], f, fp);
      float r = 1.f;
      if (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
        r = 1.f / sqrtf(row_sum<LPR>(ss) * (1.f / D) + eps);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] = fmaf(cb[i], fp[i], ca[i] * f[i]);
        if (NORM) f[i] *= r;
      }
      if (hr < h1) Vec8<T>::store(y + (size_t)hr * D + col, f);
    }
  }
}

// Gradient.  A warp takes whole tokens (token index = warp, warp + all warps,
// ...), its query heads and then its key heads, and adds the weights' gradient
// in registers over all of them; the CTA's warps are then added in warp order
// and the CTA's sums written out, to be added in CTA order by the next kernel:
// the summation order depends on the shape alone.
template <class T, int LPR, bool HALF>
__global__ void __launch_bounds__(32 * kWarps, 2)
    qk_norm_rope_bwd_kernel(const QkTensors a, const RotaryDev rt, float eps, float q_mul,
                            float* __restrict__ dw_part, int* status) {
  constexpr int D = LPR * 8, RPW = 32 / LPR;
  __shared__ float red[kWarps][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = (lane % LPR) * 8, sub_row = lane / LPR;
  Turn<LPR, HALF> turn;
  turn.init(rt, lane);
  float dw[2][8] = {};
  const long long tokens = (long long)a.B * a.N;
  for (long long token = (long long)blockIdx.x * kWarps + warp; token < tokens;
       token += (long long)gridDim.x * kWarps) {
    const int b = (int)(token / a.N), n = (int)(token - (long long)b * a.N);
    turn.fetch(rt, b, n, lane, status);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const bool is_q = side == 0;
      const int heads = is_q ? a.heads : a.kv_heads;
      const T* x = static_cast<const T*>(is_q ? a.q : a.k) + (size_t)token * (is_q ? a.q_stride : a.k_stride);
      const T* dy = static_cast<const T*>(is_q ? a.dq_out : a.dk_out) + (size_t)token * heads * D;
      T* dx = static_cast<T*>(is_q ? a.q_out : a.k_out) + (size_t)token * heads * D;
      const float m = is_q ? q_mul : 1.f;
      float w[8];
      load_w(is_q ? a.wq : a.wk, col, w);
      for (int h = 0; h < heads; h += kUnrollBwd * RPW) {
        Vec8<T> rx[kUnrollBwd], rg[kUnrollBwd];
#pragma unroll
        for (int u = 0; u < kUnrollBwd; ++u) {
          const int hr = h + u * RPW + sub_row;
          if (hr < heads) {
            rx[u].load(x + (size_t)hr * D + col);
            rg[u].load(dy + (size_t)hr * D + col);
          } else {
            rx[u].zero();
            rg[u].zero();
          }
        }
#pragma unroll
        for (int u = 0; u < kUnrollBwd; ++u) {
          if (h + u * RPW >= heads) break;  // warp-uniform
          const int hr = h + u * RPW + sub_row;
          float f[8], g[8], gp[8];
          rx[u].get(f);
          rg[u].get(g);
          turn.partners(rg[u], g, gp);
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            g[i] = m * fmaf(turn.other(i, true), gp[i], turn.own(i) * g[i]);
            ss = fmaf(f[i], f[i], ss);
            dot = fmaf(g[i] * w[i], f[i], dot);
          }
          const float r = 1.f / sqrtf(row_sum<LPR>(ss) * (1.f / D) + eps);
          const float k3 = r * r * (row_sum<LPR>(dot) * (1.f / D));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dw[side][i] = fmaf(g[i], f[i] * r, dw[side][i]);
            g[i] = r * fmaf(-k3, f[i], g[i] * w[i]);
          }
          if (hr < heads) Vec8<T>::store(dx + (size_t)hr * D + col, g);
        }
      }
    }
  }
  // rows of the warp, then warps of the CTA, in a fixed order
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = dw[side][i];
#pragma unroll
      for (int mk = LPR; mk < 32; mk <<= 1) v += __shfl_xor_sync(0xffffffffu, v, mk);
      if (sub_row == 0) red[warp][side][col + i] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += 32 * kWarps) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v += red[k][i / D][i % D];
    dw_part[(size_t)blockIdx.x * 2 * D + i] = v;
  }
}

// dw[i] = sum over CTAs of part[cta][i]: 32 columns per CTA, each thread row
// adds every 32nd partial, then the 32 rows are added in order.
__global__ void __launch_bounds__(1024)
    qk_dw_reduce_kernel(const float* __restrict__ part, int parts, int D, float* dwq, float* dwk) {
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
  const long long c = (tokens + kWarps - 1) / kWarps;
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
  const int groups_q = (a.heads + RPW - 1) / RPW, groups_k = (a.kv_heads + RPW - 1) / RPW;
  long long want = (16 * kNumSMs + tokens - 1) / tokens;  // warps per token
  int per = (int)((groups_q + groups_k + want - 1) / want);
  if (per < 1) per = 1;
  const int cq = (groups_q + per - 1) / per, ck = (groups_k + per - 1) / per;
  const long long tasks = tokens * (cq + ck);
  const dim3 grid((unsigned)((tasks + kWarps - 1) / kWarps));
  int* sw = status_word();
  if (norm)
    qk_norm_rope_kernel<T, LPR, HALF, true><<<grid, 32 * kWarps, 0, st>>>(a, rt, cq, ck, per * RPW, eps, q_mul, sw);
  else
    qk_norm_rope_kernel<T, LPR, HALF, false><<<grid, 32 * kWarps, 0, st>>>(a, rt, cq, ck, per * RPW, eps, q_mul, sw);
}

template <class T, int LPR, bool HALF>
void launch_bwd(const QkTensors& a, const RotaryDev& rt, float eps, float q_mul, float* dwq,
                float* dwk, float* ws, cudaStream_t st) {
  const int ctas = bwd_ctas((long long)a.B * a.N);
  if (ctas)  // no tokens: the sums over nothing below are zeros
    qk_norm_rope_bwd_kernel<T, LPR, HALF><<<ctas, 32 * kWarps, 0, st>>>(a, rt, eps, q_mul, ws, status_word());
  qk_dw_reduce_kernel<<<(2 * LPR * 8 + 31) / 32, 1024, 0, st>>>(ws, ctas, LPR * 8, dwq, dwk);
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
