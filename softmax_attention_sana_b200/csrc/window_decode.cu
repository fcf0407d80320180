// Windowed softmax anchor over a ring cache: the newest N tokens (usually one)
// of every sequence against its sinks and its window.
//
// Bound by HBM: every visible key and value row is read once (512 bytes for
// 4 * 128 flops per query row), so the work is split over the keys until all
// SMs load, and the arithmetic only has to keep up.  That is what the warp-wide
// m16n8k16 products do here: a tcgen05 tile would put 128 keys against 8 query
// rows through TMEM, a longer way for the same bytes.
//
// The visible keys of a sequence are a few runs of slots (sinks, the window up
// to the ring's end and from its start, the new tokens), cut into tiles of 64.  A
// CTA takes a share of the tiles of one key head: a producer warp brings them in
// by TMA (whole tiles, or those boxes of 16 rows that hold visible keys) through a
// ring of three stages, four warps take 16 keys of each.  The query rows of the key head
// (N tokens x heads / kv_heads) form tiles of 8 (NT of them, 1 or 2, per CTA):
//   S^T (16 keys x 8 rows) = K Q^T      A = K by ldmatrix
//   P^T = 2^(sl S^T - m) in bf16, turned to (row, key) order by movmatrix
//   O^T (128 d x 8 rows) += V^T P^T     A = V^T by ldmatrix.trans
// Running maximum and sum in fp32; the warps of a CTA and then the CTAs of a
// (sequence, key head) are joined in a fixed order: where they fit a cluster of up
// to eight, in one another's shared memory, else through the workspace and a second
// kernel.  64 sequences of 8320 visible keys, 16 query heads on 2 key heads: 84 us
// for 545 MB, 98% of the measured HBM rate, in a run of calls (two splits in a cluster;
// 88 us alone); of ragged lengths, 407 MB, 65 us (an earlier form that brought every tile
// in by boxes of 16 rows, one thread issuing 16 copies for each, took 74 us).
#include <cuda.h>
#include <cuda_bf16.h>

#include "f32x2.cuh"
#include "pair.cuh"
#include "pdl.cuh"
#include "sana_internal.h"

namespace sana {
namespace {

constexpr int kD = 128;
constexpr int kWarps = 4;               // consumer warps; one more warp loads
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kTile = 64;               // keys of a tile: 16 for each warp
constexpr int kBox = 16;                // rows of a TMA box of a tile that is not full
constexpr int kStages = 3;
constexpr int kHalf = kTile * 128;      // 64 columns of a tile's K or V, 8 KB
constexpr int kStageB = 4 * kHalf;      // K and V of a tile, 32 KB
constexpr int kCluster = 8;             // splits that are joined within a cluster
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

// The visible keys of one sequence: runs of slots (runs 0..2; run 3: rows of the
// new tokens) that hold consecutive positions.
struct KeyRuns {
  long long pos[4];  // positions may pass 2^31 by the N new tokens
  int slot[4], rows[4], tiles;
};
// A walk over the tiles (every index is a constant, so that the runs stay in
// registers).
struct KeyTile {
  long long pos;         // of its first key
  int run, slot, left;   // keys of the run from here on
  __device__ __forceinline__ void enter(const KeyRuns& k, int i) {
    run = i;
    pos = k.pos[i];
    slot = k.slot[i];
    left = k.rows[i];
  }
  __device__ __forceinline__ void seek(const KeyRuns& k, int t) {
    enter(k, 0);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int n = (k.rows[i] + kTile - 1) / kTile;
      if (run == i && t >= n) {
        t -= n;
        enter(k, i + 1);
      }
    }
    step(t * kTile);
  }
  __device__ __forceinline__ void next(const KeyRuns& k) {
    step(kTile);
    if (left <= 0) {
#pragma unroll
      for (int i = 1; i < 4; ++i)
        if (run < i && left <= 0) enter(k, i);
    }
  }
  __device__ __forceinline__ void step(int n) {
    pos += n;
    slot += n;
    left -= n;
  }
};
__device__ __forceinline__ KeyRuns key_runs(const DecodeDev& d, int len) {
  KeyRuns k;
  const long long ring = d.capacity - d.sinks, total = (long long)len + d.N;
  // first position of the window of the first new token that the ring still
  // holds once all N are in
  long long lo = 0;
  if (d.window && len + 1LL - d.window > lo) lo = len + 1LL - d.window;
  if (total > d.capacity && total - ring > lo) lo = total - ring;
  const int old = (int)(len - lo);  // keys of the window in the cache
  const int s = (int)(lo < d.sinks ? lo : d.sinks);
  const int at = (int)(lo < d.capacity ? lo : d.sinks + (lo - d.sinks) % ring);
  const int upto = min(old, d.capacity - at);
  k.pos[0] = 0;
  k.slot[0] = 0;
  k.rows[0] = s;
  k.pos[1] = lo;
  k.slot[1] = at;
  k.rows[1] = upto;
  // the window follows the sinks' slots: one run, if the positions follow too or do
  // not matter (a single query sees every listed key)
  if (at == s && (lo == s || d.N == 1)) {
    k.rows[0] += upto;
    k.rows[1] = 0;
  }
  k.pos[2] = lo + upto;
  k.slot[2] = d.sinks;
  k.rows[2] = old - upto;
  k.pos[3] = len;
  k.slot[3] = 0;
  k.rows[3] = d.N;
  k.tiles = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) k.tiles += (k.rows[i] + kTile - 1) / kTile;
  return k;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
      " {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 transpose of 16-bit values across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Output of one (row, column): o / l, gated.
__device__ __forceinline__ size_t out_at(const DecodeDev& d, int b, int hk, int row, int col) {
  const int group = d.heads / d.kv_heads;
  const int h = hk * group + row % group;
  return (((size_t)b * d.N + row / group) * d.heads + h) * kD + col;
}
__device__ __forceinline__ void write_out(const DecodeDev& d, int b, int hk, int row, int col,
                                          float o, float l) {
  const size_t at = out_at(d, b, hk, row, col);
  float y = o / l;  // (every row sees itself: l = 0 only where all its scores are -inf)
  if (d.gate) y *= sigmoid_fast(__bfloat162float(d.gate[at]));
  d.out[at] = __float2bfloat16(y);
}

struct DecodeCtl {
  uint64_t full[kStages], empty[kStages];
  int abort_flag;
};
// Dynamic shared memory: the ring; when its last tile is used, the warps' sums.
constexpr size_t kDecodeSmem = kStages * (size_t)kStageB + 1024;

__device__ __forceinline__ float load_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// kJoined: the splits of an item are one cluster.
template <int NT, bool kJoined>
__global__ void __launch_bounds__(kThreads, 2)
    window_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ CUtensorMap tm_kt, const __grid_constant__ CUtensorMap tm_vt,
                         const __grid_constant__ CUtensorMap tm_kn, const __grid_constant__ CUtensorMap tm_vn,
                         const DecodeDev d, int* status) {
  constexpr int kRowsT = 8 * NT;
  extern __shared__ uint8_t smem_raw[];
  __shared__ DecodeCtl ctl;
  __shared__ float sm_m[kWarps][kRowsT], sm_l[kWarps][kRowsT], sm_ml[kRowsT][2];
  uint8_t* ring = align1024(smem_raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, a = lane >> 2, c = lane & 3;
  const int splits = gridDim.x, split = blockIdx.x, b = blockIdx.z;
  const int hk = blockIdx.y / d.row_tiles, rt = blockIdx.y - hk * d.row_tiles;
  const int group = d.heads / d.kv_heads, rows = group * d.N, row0 = rt * kRowsT;
  const int len = __ldg(d.lengths + b);
  if (!kJoined) griddep_launch_next();

  if (len < 0) {  // an empty batch entry
    if (split == 0)
      for (int i = threadIdx.x; i < min(kRowsT, rows - row0) * kD; i += kThreads)
        d.out[out_at(d, b, hk, row0 + i / kD, i % kD)] = __float2bfloat16(0.f);
    return;
  }
  const KeyRuns keys = key_runs(d, len);
  const int per = (keys.tiles + splits - 1) / splits;
  const int t0 = min(split * per, keys.tiles), count = min(per, keys.tiles - t0);
  const WaitCtx wc{&ctl.abort_flag, status};
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], kWarps);
    }
    ctl.abort_flag = 0;
    mbar_fence_init();
  }
  __syncthreads();

  if (warp == kWarps) {
    // ------------------------------------------------ producer
    if (lane == 0) {
      int n = 0;
      KeyTile at;
      at.seek(keys, t0);
      for (int t = 0; t < count; ++t, at.next(keys)) {
        const int st = t % kStages;
        if (t >= kStages && !mbar_wait(&ctl.empty[st], ((t / kStages) - 1) & 1, wc, 0xc1)) break;
        uint8_t* dst = ring + st * kStageB;
        if (at.left >= kTile && at.run < 3) {
          mbar_arrive_expect_tx(&ctl.full[st], kStageB);
          for (int hh = 0; hh < 2; ++hh) {
            tma_load_3d(dst + hh * kHalf, &tm_kt, &ctl.full[st], hk * kD + hh * 64, at.slot, b);
            tma_load_3d(dst + (2 + hh) * kHalf, &tm_vt, &ctl.full[st], hk * kD + hh * 64, at.slot, b);
          }
        } else {
          const int boxes = (min(kTile, at.left) + kBox - 1) / kBox;
          const CUtensorMap* mk = at.run == 3 ? &tm_kn : &tm_k;
          const CUtensorMap* mv = at.run == 3 ? &tm_vn : &tm_v;
          mbar_arrive_expect_tx(&ctl.full[st], boxes * 4 * kBox * 128);
          for (int x = 0; x < boxes; ++x)  // (rows past the cache's end read as zeros)
            for (int hh = 0; hh < 2; ++hh) {
              tma_load_3d(dst + hh * kHalf + x * kBox * 128, mk, &ctl.full[st], hk * kD + hh * 64, at.slot + x * kBox, b);
              tma_load_3d(dst + (2 + hh) * kHalf + x * kBox * 128, mv, &ctl.full[st], hk * kD + hh * 64, at.slot + x * kBox, b);
            }
        }
        ++n;
      }
      if (*wc.abort_flag)  // loads still in flight land before the CTA exits
        for (int t = n > kStages ? n - kStages : 0; t < n; ++t) mbar_drain(&ctl.full[t % kStages], (t / kStages) & 1);
    }
    // The new tokens go to their slots.  What a slot held before is a position
    // that no query of this call sees; a box may touch it, its rows are masked.
    if (split == 0 && rt == 0) {
      const size_t pitch = (size_t)d.kv_heads * kD, new0 = ((size_t)b * d.N * d.kv_heads + hk) * kD;
      const size_t cache0 = ((size_t)b * d.capacity * d.kv_heads + hk) * kD;
      for (int t = 0; t < d.N; ++t) {
        const long long p = (long long)len + t;
        const size_t s = p < d.capacity ? (size_t)p : (size_t)(d.sinks + (p - d.sinks) % (d.capacity - d.sinks));
        const size_t piece = (lane & 15) * 8;
        const __nv_bfloat16* src = (lane & 16 ? d.v_new : d.k_new) + new0 + t * pitch + piece;
        *reinterpret_cast<uint4*>((lane & 16 ? d.v_cache : d.k_cache) + cache0 + s * pitch + piece) =
            *reinterpret_cast<const uint4*>(src);
      }
    }
    __syncthreads();  // the ring has become the warps' sums
    __syncthreads();
    if (kJoined) {
      cluster_sync();
      cluster_sync();
    }
    return;
  }

  // ------------------------------------------------ consumers
  // Q as B operand: row a of each tile, d = 16 j + 2 c (+ 8)
  uint32_t qr[NT][8][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = row0 + t * 8 + a;
    const __nv_bfloat16* p = d.q + (((size_t)b * d.N + row / group) * d.heads + hk * group + row % group) * kD + 2 * c;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        qr[t][j][e] = row < rows ? *reinterpret_cast<const uint32_t*>(p + 16 * j + 8 * e) : 0u;
  }
  long long qpos[NT][2];  // position of query rows 2c, 2c + 1 of each tile
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) qpos[t][e] = (long long)len + min(row0 + t * 8 + 2 * c + e, rows - 1) / group;
  const bool one = d.N == 1;  // then every listed key is visible

  float o[NT][8][4] = {};  // [d / 16][2 (d / 8 % 2) + row % 2]: d = 16 j + a (+ 8), rows 2c, 2c + 1
  float mx[NT][2], sum[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) mx[t][e] = -INFINITY, sum[t][e] = 0.f;
  // ldmatrix rows of this lane: K: key lane % 16, piece lane / 16; V: key lane % 8 +
  // 8 (lane / 16), piece lane / 8 % 2
  const int k_row = warp * 16 + (lane & 15), k_piece = lane >> 4;
  const int v_row = warp * 16 + (lane & 7) + ((lane >> 4) << 3), v_piece = (lane >> 3) & 1;
  bool ok = true;
  KeyTile at;
  at.seek(keys, t0);
  for (int u = 0; u < count; ++u, at.next(keys)) {
    const int st = u % kStages;
    ok = __all_sync(0xffffffffu, mbar_wait(&ctl.full[st], (u / kStages) & 1, wc, 0xc2));
    if (!ok) break;
    const int left = at.left - warp * 16;  // keys of this warp
    if (left > 0) {
      const uint32_t kb = smem_u32(ring + st * kStageB), vb = kb + 2 * kHalf;
      float s[NT][4] = {}, s1[NT][4] = {};  // two chains of products, added below
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t ka[4];
        ldsm4(ka, kb + (j >> 2) * kHalf + sw128_off(k_row, (j & 3) * 2 + k_piece));
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816(j & 1 ? s1[t] : s[t], ka, qr[t][j][0], qr[t][j][1]);
      }
      // s[t][e + 2 i]: key a + 8 i, query row 2c + e
      uint32_t p0[NT], p1[NT];
      const long long first = at.pos + warp * 16;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][i] += s1[t][i];
        if (!one || left < 16) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const long long p = first + a + 8 * i;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const bool sees = one || (p <= qpos[t][e] &&
                                        (d.window == 0 || p > qpos[t][e] - d.window || p < d.sinks));
              if (a + 8 * i >= left || !sees) s[t][e + 2 * i] = -INFINITY;
            }
          }
        }
        float f[2][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(s[t][e], s[t][e + 2]);
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
          const float now = fmaxf(mx[t][e], top * d.sl);
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
          // (scaled and referred in one rounding: of large scores only the differences count)
          f[e][0] = ex2(fmaf(s[t][e], d.sl, -ref));
          f[e][1] = ex2(fmaf(s[t][e + 2], d.sl, -ref));
          sum[t][e] = sum[t][e] * corr + (f[e][0] + f[e][1]);
        }
        p0[t] = transpose8(f2_to_bf2(f[0][0], f[1][0]));
        p1[t] = transpose8(f2_to_bf2(f[0][1], f[1][1]));
      }
      // rows of V past the run hold anything (P is 0 there): keys 2c, 2c + 1 and + 8
      uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
      if (left < 16) {
        keep0 = (2 * c < left ? 0xffffu : 0u) | (2 * c + 1 < left ? 0xffff0000u : 0u);
        keep1 = (2 * c + 8 < left ? 0xffffu : 0u) | (2 * c + 9 < left ? 0xffff0000u : 0u);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t va[4];
        ldsm4_trans(va, vb + (j >> 2) * kHalf + sw128_off(v_row, (j & 3) * 2 + v_piece));
        va[0] &= keep0;
        va[1] &= keep0;
        va[2] &= keep1;
        va[3] &= keep1;
#pragma unroll
        for (int t = 0; t < NT; ++t) mma16816(o[t][j], va, p0[t], p1[t]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl.empty[st]);
  }

  // join the warps: rows 2c + e, d = 16 j + a (+ 8)
  __syncthreads();
  float(*sm_o)[kRowsT][kD + 4] = reinterpret_cast<float(*)[kRowsT][kD + 4]>(ring);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = t * 8 + 2 * c + e;
      float l = sum[t][e];
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sm_o[warp][r][16 * j + a] = o[t][j][e];
        sm_o[warp][r][16 * j + a + 8] = o[t][j][e + 2];
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
    } else if (kJoined) {
      sm_o[0][r][threadIdx.x] = v;
      if (threadIdx.x == 0) {
        sm_ml[r][0] = top;
        sm_ml[r][1] = l;
      }
    } else {
      part[r * kD + threadIdx.x] = v;
      if (threadIdx.x == 0) {
        part_ml[2 * r] = top;
        part_ml[2 * r + 1] = l;
      }
    }
  }
  if (kJoined) {
    cluster_sync();
    // this CTA joins every splits-th row over the cluster
    for (int r = split; r < kRowsT && row0 + r < rows; r += splits) {
      float mk[kCluster], lk[kCluster], vk[kCluster];  // all on their way at once
#pragma unroll
      for (int k = 0; k < kCluster; ++k) {
        mk[k] = -INFINITY;
        lk[k] = vk[k] = 0.f;
        if (k < splits) {
          mk[k] = load_cluster(cluster_addr(&sm_ml[r][0], k));
          lk[k] = load_cluster(cluster_addr(&sm_ml[r][1], k));
          vk[k] = load_cluster(cluster_addr(&sm_o[0][r][threadIdx.x], k));
        }
      }
      float top = mk[0], l = 0.f, v = 0.f;
#pragma unroll
      for (int k = 1; k < kCluster; ++k) top = fmaxf(top, mk[k]);
      const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int k = 0; k < kCluster; ++k) {
        const float f = ex2(mk[k] - ref);
        l = fmaf(f, lk[k], l);
        v = fmaf(f, vk[k], v);
      }
      write_out(d, b, hk, row0 + r, threadIdx.x, v, l);
    }
    cluster_sync();  // nobody leaves while its sums are read
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
  bool joined;  // the splits of an item are a cluster
};
// Rows: one tile of 8 where they fit, else tiles of 16 (a second pass over the
// keys costs more than the registers of 16 rows).  Splits: of those that the key
// tiles allow, the one whose waves of CTAs (two fit on an SM) are soonest done, with
// a CTA's start and end counted as two tiles, the second kernel as one and each split
// that it sums as a fifth.  Splits of one wave are clusters where they fit one; in
// several waves clusters wait for room.  Measured in captured runs over caches beyond
// L2, splits (j: in clusters):
//   64 sequences of 8320 keys, 2 key heads: 1 90, 2 88, 2j 84, 4 88, 9 94 us
//   4 of 1028, 8 key heads: 4j 8.5, 6j 8.7, 8j 8.7, 9 11.1
//   2 of 8196, 2 key heads: 8j 15.4, 16 12.8, 32 13.0, 64 15.9
//   1 of 4100, 8 key heads: 8j 10.0, 16 10.6, 32 12.3 (17, taken here: 11.0)
//   16 of 2052, 24 key heads: 1 71, 2 69, 3 69, 3j 74
DecodePlan decode_plan(const DecodeCall& c) {
  DecodePlan p{};
  const int rows = c.heads / c.kv_heads * c.N;
  p.nt = rows <= 8 ? 1 : 2;
  p.row_tiles = (rows + 8 * p.nt - 1) / (8 * p.nt);
  const long long items = (long long)c.B * c.kv_heads * p.row_tiles, slots = 2 * kNumSMs;
  long long keys = c.capacity;
  if (c.window && (long long)c.window + c.sinks + c.N < keys) keys = (long long)c.window + c.sinks + c.N;
  const long long tiles = (keys + kTile - 1) / kTile + 2;  // (runs of keys end inside tiles)
  long long most = 4 * slots / items;  // four waves at most
  most = most < 1 ? 1 : most > tiles ? tiles : most;
  long long best = 0;
  for (long long s = 1; s <= most; ++s) {
    const bool joined = s <= kCluster && items * s <= slots;
    const long long waves = (items * s + slots - 1) / slots;
    const long long cost = 5 * waves * ((tiles + s - 1) / s + 2) + (s == 1 || joined ? 0 : 5 + s);
    if (best == 0 || cost < best) {
      best = cost;
      p.splits = (int)s;
      p.joined = joined && s > 1;
    }
  }
  return p;
}

}  // namespace

size_t window_decode_ws_bytes(const DecodeCall& c) {
  const DecodePlan p = decode_plan(c);
  if (p.splits == 1 || p.joined) return 0;
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
  const uint64_t C = (uint64_t)c.kv_heads * kD, cap = c.capacity, N = c.N;
  CUtensorMap tk, tv, tkt, tvt, tkn, tvn;
  if (!make_tmap_bf16_3d(&tk, k_cache, C, cap, c.B, C, cap * C, kBox) ||
      !make_tmap_bf16_3d(&tv, v_cache, C, cap, c.B, C, cap * C, kBox) ||
      !make_tmap_bf16_3d(&tkt, k_cache, C, cap, c.B, C, cap * C, kTile) ||
      !make_tmap_bf16_3d(&tvt, v_cache, C, cap, c.B, C, cap * C, kTile) ||
      !make_tmap_bf16_3d(&tkn, k_new, C, N, c.B, C, N * C, kBox) ||
      !make_tmap_bf16_3d(&tvn, v_new, C, N, c.B, C, N * C, kBox))
    return fail(SANA_ERR_CUDA, "windowed anchor step: cuTensorMapEncodeTiled failed");
  once_per_context(kAttrWindowDecode, [] {
    cudaFuncSetAttribute(window_decode_kernel<1, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDecodeSmem);
    cudaFuncSetAttribute(window_decode_kernel<2, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDecodeSmem);
    cudaFuncSetAttribute(window_decode_kernel<1, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDecodeSmem);
    cudaFuncSetAttribute(window_decode_kernel<2, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDecodeSmem);
  });
  int* sw = status_word();
  const dim3 grid(p.splits, c.kv_heads * p.row_tiles, c.B);
  if (p.joined) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kDecodeSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.nt == 1) cudaLaunchKernelEx(&cfg, window_decode_kernel<1, true>, tk, tv, tkt, tvt, tkn, tvn, d, sw);
    else cudaLaunchKernelEx(&cfg, window_decode_kernel<2, true>, tk, tv, tkt, tvt, tkn, tvn, d, sw);
    return check_launch("window_decode_kernel");
  }
  if (p.nt == 1) window_decode_kernel<1, false><<<grid, kThreads, kDecodeSmem, st>>>(tk, tv, tkt, tvt, tkn, tvn, d, sw);
  else window_decode_kernel<2, false><<<grid, kThreads, kDecodeSmem, st>>>(tk, tv, tkt, tvt, tkn, tvn, d, sw);
  if (sana_status e = check_launch("window_decode_kernel")) return e;
  if (p.splits > 1) {
    launch_dependent(window_decode_join_kernel, dim3(c.heads / c.kv_heads * c.N, c.kv_heads, c.B), dim3(kD), 0, st,
                     d, p.splits, 8 * p.nt);
    return check_launch("window_decode_join_kernel");
  }
  return SANA_OK;
}

}  // namespace sana
