// Windowed softmax anchor over a ring cache: the newest N tokens (usually one)
// of every sequence against its sinks and its window.
//
// Bound by HBM: every visible key and value row is read once (512 bytes for
// 4 * 128 flops per query row), so the work is split over the keys until all
// SMs load, and the arithmetic only has to keep up.  That is what the warp-wide
// m16n8k16 products do here, straight from registers: a tcgen05 tile would put
// 128 keys against 8 query rows through shared memory and TMEM, a longer way
// for the same bytes.
//
// The query rows of one key head (N tokens x heads / kv_heads) form tiles of 8
// (NT of them, 1 or 2, per CTA).  A warp takes 16 keys at a time:
//   S^T (16 keys x 8 rows) = K Q^T   A = K: lane (a = lane / 4, c = lane % 4)
//       holds 16-byte pieces c, c + 4, c + 8, c + 12 of keys a and a + 8; the
//       order of d inside a product is free as long as Q uses the same one, so
//       the pieces feed the products as loaded
//   P^T = 2^(sl S^T - m) in bf16, turned to (row, key) order by movmatrix
//   O^T (128 d x 8 rows) += V^T P^T   A = V^T: the lane holds 16-byte pieces a
//       and a + 8 of keys 2c, 2c + 1, 2c + 8, 2c + 9; a byte permutation pairs
//       two keys per d, and product e of 8 covers d = 8a + e and 64 + 8a + e
// K of the next 16 keys is requested as soon as the scores are made, V as soon
// as it is used: 8 KB stay in flight per warp with no shared memory.  Running
// maximum and sum in fp32; the warps of a CTA and then the CTAs of a (sequence,
// key head) are joined in a fixed order.
#include <cuda_bf16.h>

#include "f32x2.cuh"
#include "pdl.cuh"
#include "sana_internal.h"

namespace sana {
namespace {

constexpr int kD = 128;
constexpr int kWarps = 4;
constexpr int kKeys = 16;  // keys a warp takes at a time
constexpr float kLog2e = 1.4426950408889634f;

struct DecodeDev {
  const __nv_bfloat16 *q, *k_new, *v_new, *gate;
  __nv_bfloat16 *k_cache, *v_cache, *out;
  const int* lengths;
  int B, N, heads, kv_heads, capacity, window, sinks;
  float sl;
  int row_tiles;  // tiles of 8 * NT query rows per key head
  float* part;    // [item][split][8 NT rows][128] sums, then [..][2] max and sum
};

// The keys of one sequence in this call: m in [0, S) sinks at position m, then
// positions lo, lo + 1, ... up to the new tokens at [len, len + N).
struct KeyList {
  int S, count;
  long long lo, len;  // positions may pass 2^31 by the N new tokens
  long long slot_lo;  // slot of position lo
  __device__ __forceinline__ long long pos(int m) const { return m < S ? m : lo + (m - S); }
};
__device__ __forceinline__ KeyList key_list(const DecodeDev& d, int len) {
  KeyList k;
  const long long ring = d.capacity - d.sinks, total = (long long)len + d.N;
  k.len = len;
  k.lo = 0;
  if (d.window && len + 1LL - d.window > k.lo) k.lo = len + 1LL - d.window;
  if (total - ring > k.lo && total > d.capacity) k.lo = total - ring;
  k.S = (int)(k.lo < d.sinks ? k.lo : d.sinks);
  k.count = (int)(k.S + total - k.lo);
  k.slot_lo = k.lo < d.capacity ? k.lo : d.sinks + (k.lo - d.sinks) % ring;
  return k;
}
// Row of key m: in the new tokens, or in its slot (at most one turn of the ring
// after lo's).
__device__ __forceinline__ const __nv_bfloat16* key_row(const DecodeDev& d, const KeyList& k,
                                                        const __nv_bfloat16* cache,
                                                        const __nv_bfloat16* fresh, int m) {
  const long long p = k.pos(m);
  const size_t pitch = (size_t)d.kv_heads * kD;
  if (p >= k.len) return fresh + (size_t)(p - k.len) * pitch;
  long long s = m < k.S ? m : k.slot_lo + (m - k.S);
  if (s >= d.capacity) s -= d.capacity - d.sinks;
  return cache + (size_t)s * pitch;
}

__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
      " {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 transpose of 16-bit values across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Output of one (row, column): o / l, gated.
__device__ __forceinline__ void write_out(const DecodeDev& d, int b, int hk, int row, int col,
                                          float o, float l) {
  const int group = d.heads / d.kv_heads;
  const int h = hk * group + row % group;
  const size_t at = (((size_t)b * d.N + row / group) * d.heads + h) * kD + col;
  float y = l > 0.f ? o / l : 0.f;
  if (d.gate) y *= sigmoid_fast(__bfloat162float(d.gate[at]));
  d.out[at] = __float2bfloat16(y);
}

template <int NT>
__global__ void __launch_bounds__(32 * kWarps, NT == 1 ? 3 : 2) window_decode_kernel(const DecodeDev d) {
  constexpr int kRowsT = 8 * NT;
  __shared__ float sm_o[kWarps][kRowsT][kD + 4];
  __shared__ float sm_m[kWarps][kRowsT], sm_l[kWarps][kRowsT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, a = lane >> 2, c = lane & 3;
  const int splits = gridDim.x, split = blockIdx.x, b = blockIdx.z;
  const int hk = blockIdx.y / d.row_tiles, rt = blockIdx.y - hk * d.row_tiles;
  const int group = d.heads / d.kv_heads, rows = group * d.N, row0 = rt * kRowsT;
  const int len = __ldg(d.lengths + b);
  griddep_launch_next();

  if (len < 0) {  // an empty batch entry
    if (split == 0)
      for (int i = threadIdx.x; i < min(kRowsT, rows - row0) * kD; i += 32 * kWarps)
        write_out(d, b, hk, row0 + i / kD, i % kD, 0.f, 0.f);
    return;
  }
  const KeyList keys = key_list(d, len);
  const size_t pitch = (size_t)d.kv_heads * kD;
  const __nv_bfloat16* kn = d.k_new + ((size_t)b * d.N * d.kv_heads + hk) * kD;
  const __nv_bfloat16* vn = d.v_new + ((size_t)b * d.N * d.kv_heads + hk) * kD;
  __nv_bfloat16* kc = d.k_cache + ((size_t)b * d.capacity * d.kv_heads + hk) * kD;
  __nv_bfloat16* vc = d.v_cache + ((size_t)b * d.capacity * d.kv_heads + hk) * kD;

  // The new tokens go to their slots.  What a slot held before is a position
  // that no query of this call sees, so nobody reads it meanwhile.
  if (split == 0 && rt == 0) {
    for (int i = threadIdx.x; i < d.N * 32; i += 32 * kWarps) {
      const int t = i >> 5, piece = (i & 15) * 8;
      const long long p = keys.len + t;
      const size_t s = p < d.capacity ? (size_t)p : (size_t)(d.sinks + (p - d.sinks) % (d.capacity - d.sinks));
      const bool is_v = (i & 16) != 0;
      *reinterpret_cast<uint4*>((is_v ? vc : kc) + s * pitch + piece) =
          *reinterpret_cast<const uint4*>((is_v ? vn : kn) + (size_t)t * pitch + piece);
    }
  }

  // this CTA's groups of 16 keys, and this warp's: g, g + 4, ...
  const int groups = (keys.count + kKeys - 1) / kKeys;
  const int per = (groups + splits - 1) / splits;
  const int g1 = min(groups, (split + 1) * per);
  int g = split * per + warp;

  uint4 kr[2][4], vr[4][2];
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto load_k = [&](int gg) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = gg * kKeys + a + 8 * i;
      const bool in = gg < g1 && m < keys.count;
      const __nv_bfloat16* p = in ? key_row(d, keys, kc, kn, m) : nullptr;
#pragma unroll
      for (int j = 0; j < 4; ++j) kr[i][j] = in ? load16(p + (c + 4 * j) * 8) : zero;
    }
  };
  auto load_v = [&](int gg) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = gg * kKeys + 2 * c + (i & 1) + 8 * (i >> 1);
      const bool in = gg < g1 && m < keys.count;
      const __nv_bfloat16* p = in ? key_row(d, keys, vc, vn, m) : nullptr;
#pragma unroll
      for (int j = 0; j < 2; ++j) vr[i][j] = in ? load16(p + a * 8 + 64 * j) : zero;
    }
  };
  load_k(g);
  load_v(g);

  // Q: row a of each tile, the same pieces of d as K's
  uint4 qr[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = row0 + t * 8 + a;
    const __nv_bfloat16* p = d.q + (((size_t)b * d.N + row / group) * d.heads + hk * group + row % group) * kD;
#pragma unroll
    for (int j = 0; j < 4; ++j) qr[t][j] = row < rows ? *reinterpret_cast<const uint4*>(p + (c + 4 * j) * 8) : zero;
  }
  // position of query rows 2c, 2c + 1 of each tile
  long long qpos[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) qpos[t][e] = keys.len + min(row0 + t * 8 + 2 * c + e, rows - 1) / group;
  const bool one = d.N == 1;  // then every listed key is visible

  float o[NT][8][4] = {};
  float mx[NT][2], sum[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) mx[t][e] = -INFINITY, sum[t][e] = 0.f;

  for (; g < g1; g += kWarps) {
    float s[NT][4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma16816(s[t], kr[0][j].x, kr[1][j].x, kr[0][j].y, kr[1][j].y, qr[t][j].x, qr[t][j].y);
        mma16816(s[t], kr[0][j].z, kr[1][j].z, kr[0][j].w, kr[1][j].w, qr[t][j].z, qr[t][j].w);
      }
    load_k(g + kWarps);
    // s[t][e + 2 i]: key a + 8 i, query row 2c + e
    uint32_t p0[NT], p1[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int m = g * kKeys + a + 8 * i;
        const bool in = m < keys.count;
        const long long p = keys.pos(m);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool sees = in && (one || (p <= qpos[t][e] &&
                                           (d.window == 0 || p > qpos[t][e] - d.window || p < d.sinks)));
          s[t][e + 2 * i] = sees ? s[t][e + 2 * i] * d.sl : -INFINITY;
        }
      }
      float f[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = fmaxf(s[t][e], s[t][e + 2]);
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        const float now = fmaxf(mx[t][e], top);
        const float ref = now == -INFINITY ? 0.f : now;
        const float corr = ex2(mx[t][e] - ref);  // 1 where the maximum stayed, 0 before the first key
        if (__any_sync(0xffffffffu, now != mx[t][e])) {
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            o[t][n][e] *= corr;
            o[t][n][e + 2] *= corr;
          }
        }
        mx[t][e] = now;
        f[e][0] = ex2(s[t][e] - ref);
        f[e][1] = ex2(s[t][e + 2] - ref);
        sum[t][e] = sum[t][e] * corr + (f[e][0] + f[e][1]);
      }
      p0[t] = transpose8(f2_to_bf2(f[0][0], f[1][0]));
      p1[t] = transpose8(f2_to_bf2(f[0][1], f[1][1]));
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      auto word = [&](const uint4& v) { return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w; };
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        const uint32_t sel = hi ? 0x7632 : 0x5410;
        const uint32_t a0 = __byte_perm(word(vr[0][0]), word(vr[1][0]), sel);
        const uint32_t a1 = __byte_perm(word(vr[0][1]), word(vr[1][1]), sel);
        const uint32_t a2 = __byte_perm(word(vr[2][0]), word(vr[3][0]), sel);
        const uint32_t a3 = __byte_perm(word(vr[2][1]), word(vr[3][1]), sel);
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816(o[t][2 * w + hi], a0, a1, a2, a3, p0[t], p1[t]);
      }
    }
    load_v(g + kWarps);
  }

  // join the warps: rows 2c + e, d = 8a + n and 64 + 8a + n
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = t * 8 + 2 * c + e;
      float l = sum[t][e];
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float* dst = &sm_o[warp][r][64 * hh + 8 * a];
        *reinterpret_cast<float4*>(dst) = make_float4(o[t][0][e + 2 * hh], o[t][1][e + 2 * hh], o[t][2][e + 2 * hh], o[t][3][e + 2 * hh]);
        *reinterpret_cast<float4*>(dst + 4) = make_float4(o[t][4][e + 2 * hh], o[t][5][e + 2 * hh], o[t][6][e + 2 * hh], o[t][7][e + 2 * hh]);
      }
      if (a == 0) {
        sm_m[warp][r] = mx[t][e];
        sm_l[warp][r] = l;
      }
    }
  __syncthreads();
  const size_t item = ((size_t)b * gridDim.y + blockIdx.y) * splits + split;
  float* part = d.part + item * kRowsT * kD;
  float* part_ml = d.part + (size_t)d.B * gridDim.y * splits * kRowsT * kD + item * kRowsT * 2;
  for (int r = 0; r < kRowsT; ++r) {
    if (row0 + r >= rows) break;
    float top = sm_m[0][r];
#pragma unroll
    for (int k = 1; k < kWarps; ++k) top = fmaxf(top, sm_m[k][r]);
    const float ref = top == -INFINITY ? 0.f : top;
    float l = 0.f, v = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float f = ex2(sm_m[k][r] - ref);
      l = fmaf(f, sm_l[k][r], l);
      v = fmaf(f, sm_o[k][r][threadIdx.x], v);
    }
    if (splits == 1) {
      write_out(d, b, hk, row0 + r, threadIdx.x, v, l);
    } else {
      part[r * kD + threadIdx.x] = v;
      if (threadIdx.x == 0) {
        part_ml[2 * r] = top;
        part_ml[2 * r + 1] = l;
      }
    }
  }
}

// Joins the splits of one query row in order; thread = column.
__global__ void __launch_bounds__(kD) window_decode_join_kernel(const DecodeDev d, int splits, int rows_t) {
  const int b = blockIdx.z, hk = blockIdx.y, row = blockIdx.x;
  griddep_wait();
  if (__ldg(d.lengths + b) < 0) return;  // zeros are written already
  const int rt = row / rows_t, r = row - rt * rows_t;
  const size_t items = (size_t)d.B * d.kv_heads * d.row_tiles * splits;
  const size_t item = (((size_t)b * d.kv_heads + hk) * d.row_tiles + rt) * splits;
  const float* part = d.part + (item * rows_t + r) * kD + threadIdx.x;
  const float* ml = d.part + items * rows_t * kD + (item * rows_t + r) * 2;
  float top = -INFINITY, l = 0.f, v = 0.f;
  for (int s = 0; s < splits; ++s) top = fmaxf(top, ml[(size_t)s * rows_t * 2]);
  const float ref = top == -INFINITY ? 0.f : top;
  for (int s = 0; s < splits; ++s) {
    const float f = ex2(ml[(size_t)s * rows_t * 2] - ref);
    l = fmaf(f, ml[(size_t)s * rows_t * 2 + 1], l);
    v = fmaf(f, part[(size_t)s * rows_t * kD], v);
  }
  write_out(d, b, hk, row, threadIdx.x, v, l);
}

struct DecodePlan {
  int nt, row_tiles, splits;
};
// Rows: one tile of 8 where they fit, else tiles of 16 (a second pass over the
// keys costs more than the registers of 16 rows).  Splits: three CTAs for every
// SM, each with 64 keys (16 a warp) at least.
DecodePlan decode_plan(const DecodeCall& c) {
  DecodePlan p{};
  const int rows = c.heads / c.kv_heads * c.N;
  p.nt = rows <= 8 ? 1 : 2;
  p.row_tiles = (rows + 8 * p.nt - 1) / (8 * p.nt);
  const long long items = (long long)c.B * c.kv_heads * p.row_tiles;
  long long keys = c.capacity;
  if (c.window && (long long)c.window + c.sinks + c.N < keys) keys = (long long)c.window + c.sinks + c.N;
  long long s = 3LL * kNumSMs / items;
  const long long most = (keys + kWarps * kKeys - 1) / (kWarps * kKeys);
  if (s > most) s = most;
  p.splits = (int)(s < 1 ? 1 : s);
  return p;
}

}  // namespace

size_t window_decode_ws_bytes(const DecodeCall& c) {
  const DecodePlan p = decode_plan(c);
  if (p.splits == 1) return 0;
  return align_up((size_t)c.B * c.kv_heads * p.row_tiles * p.splits * 8 * p.nt * (kD + 2) * sizeof(float), 256);
}

sana_status window_decode_run(const DecodeCall& c, const void* q, const void* k_new,
                              const void* v_new, const void* gate, void* k_cache, void* v_cache,
                              const int* lengths, void* out, void* ws, cudaStream_t st) {
  using bf = __nv_bfloat16;
  const DecodePlan p = decode_plan(c);
  const DecodeDev d{(const bf*)q, (const bf*)k_new, (const bf*)v_new, (const bf*)gate, (bf*)k_cache, (bf*)v_cache,
                    (bf*)out, lengths, c.B, c.N, c.heads, c.kv_heads, c.capacity, c.window, c.sinks,
                    c.scale * kLog2e, p.row_tiles, (float*)ws};
  const dim3 grid(p.splits, c.kv_heads * p.row_tiles, c.B);
  if (p.nt == 1) window_decode_kernel<1><<<grid, 32 * kWarps, 0, st>>>(d);
  else window_decode_kernel<2><<<grid, 32 * kWarps, 0, st>>>(d);
  if (sana_status e = check_launch("window_decode_kernel")) return e;
  if (p.splits > 1) {
    launch_dependent(window_decode_join_kernel, dim3(c.heads / c.kv_heads * c.N, c.kv_heads, c.B), dim3(kD), 0, st,
                     d, p.splits, 8 * p.nt);
    return check_launch("window_decode_join_kernel");
  }
  return SANA_OK;
}

}  // namespace sana
