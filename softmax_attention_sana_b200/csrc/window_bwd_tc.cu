// Windowed softmax anchor, backward, bf16 on tcgen05 (the mask: window.cuh).
//
// With s_ij = scale q_i . k_j, p_ij = exp(s_ij - lse_i), o_i = sum_j p_ij v_j and
// y_i = sigmoid(g_i) o_i, for dy:
//   do = sigmoid(g) dy,  dg = dy y (1 - sigmoid(g)),  delta_i = dy_i . y_i (= do_i . o_i)
//   ds_ij = p_ij (do_i . v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i,
// dk and dv summed over the query heads that share the key head.
//
// Three kernels, each started while the one before it ends; every sum runs in an
// order that the shape alone fixes:
//   prep   row statistics (-lse log2 e, -delta), and with a gate do and dg (HBM)
//   grad   dkv blocks, one CTA per (key tile, key head, batch, share of its query
//          tiles): scores transposed (thread = key), S^T = K Q^T and dP^T = V dO^T,
//          then dV += P^T dO and dK += dS^T Q with P^T and dS^T from TMEM;
//          dq blocks, one CTA per (query tile, query head, batch): S and dP once
//          more, then dQ += dS K
//   join   sums the shares of key tiles that were split (few key tiles, or the
//          sinks, which every later query sees).
// Making S and dP twice costs 7 products instead of 5, and keeps dQ out of
// memory until it is whole: the other way round it would be added up in fp32
// over the key tiles, 64 KB through L2 for every tile pair, in an order to be
// enforced.
//
// dkv and dq share one plan: whole 128 x 128 products (a product of 64 columns
// reads its 128-row A operand from shared memory for half the work, and took
// three times as long), one tile pair at a time, and 16 softmax warps (thread =
// row and 32 columns) whose two phases -- exponentials, then dS -- run while the
// tensor core does the products that do not need their result:
//   dkv    tensor: dV(t) | S(t+1) | dK(t) | dP(t+1)     warps: dS(t) | P(t+1)
//          (P over the S columns, dS over the dP columns)
//   dq     tensor: dP(t+1) | dQ(t) | S(t+2)             warps: dS(t) | P(t+1)
//          (two S buffers; dS over the S columns of its tile)
// A product that overwrites what another reads waits for it by its barrier.
// 16384 rows, 16 heads on 4 key heads, window 2048, 16 sinks: 815 us in all, 861 us
// with dkv and dq as launches of their own (480 and 350 us: the dq blocks fill the
// SMs that the last dkv wave leaves); 2 x 1023 rows, 8 heads, window 256, gate: 40
// against 49 us, and 34 with the key tiles left whole (dkv_plan).  Tensor pipe about
// 70% busy; in a long run the power cap holds it.  One warp issues all products: with
// a second one for the dP chain dkv took 542 us (the products then come in a worse
// order).
#include <cuda.h>

#include "f32x2.cuh"
#include "pdl_read.cuh"
#include "sana_internal.h"
#include "tc_warp.cuh"
#include "window.cuh"

namespace sana {
namespace {

constexpr int kD = 128;
constexpr int kRows = kWinTile;
constexpr int kHalf = kRows * 64 * 2;  // 16 KB: 64 columns of a tile
constexpr int kTileB = 2 * kHalf;      // 32 KB
constexpr int kDeep = 3, kShort = 2;    // stages of the ring whose tiles live long / short
constexpr int kThreads = 576;          // 16 softmax warps + producer + MMA
constexpr int kSoft = 512;             // softmax threads
constexpr int kWarpProd = 16, kWarpMma = 17;
// of every 8 pairs of exponentials, on the FMA pipe (the MUFU unit alone would
// take as long as two of the four products that hide it)
constexpr int kEmuPairs = 2;
constexpr float kLog2e = 1.4426950408889634f;

// Untiled bulk copy global -> shared (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// ---------------------------------------------------------------- prep
// Bound by HBM: 16384 rows of 16 heads, 134 MB, 21 us (97% of the measured rate).
// A CTA takes 32 consecutive rows of one head (so that their statistics, which
// lie together, are written together; CTAs of neighbouring heads run side by side
// and share DRAM pages), a half-warp two of them.  Rows [N, n_pad) only get their
// statistics.
constexpr int kPrepRows = 32;
template <bool kGate>
__global__ void __launch_bounds__(256)
    window_prep_kernel(const __nv_bfloat16* __restrict__ y, const __nv_bfloat16* __restrict__ dy,
                       const __nv_bfloat16* __restrict__ gate, long long gate_stride,
                       const float* __restrict__ lse, const WindowDev w, int n_pad,
                       float* __restrict__ nlse, float* __restrict__ ndelta,
                       __nv_bfloat16* __restrict__ d_o, __nv_bfloat16* __restrict__ dg) {
  griddep_launch_next();
  const int sub = threadIdx.x & 15, hw = threadIdx.x >> 4;
  const int h = blockIdx.x % w.heads, b = blockIdx.z;
  const int len = window_length(w, b);
  const int n0 = blockIdx.x / w.heads * kPrepRows + hw;  // and n0 + 16
  uint4 yv[2], dv[2], gv[2];
  bool live[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int n = n0 + 16 * i;
    live[i] = n < w.N && w.off + n < len;
    const size_t tok = (size_t)b * w.N + n, at = (tok * w.heads + h) * kD + sub * 8;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    yv[i] = live[i] ? __ldcs(reinterpret_cast<const uint4*>(y + at)) : zero;
    dv[i] = live[i] ? __ldcs(reinterpret_cast<const uint4*>(dy + at)) : zero;
    gv[i] = zero;
    if (kGate && live[i])
      gv[i] = __ldcs(reinterpret_cast<const uint4*>(gate + tok * gate_stride + (size_t)h * kD + sub * 8));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int n = n0 + 16 * i;
    const uint32_t ya[4] = {yv[i].x, yv[i].y, yv[i].z, yv[i].w}, da[4] = {dv[i].x, dv[i].y, dv[i].z, dv[i].w};
    const uint32_t ga[4] = {gv[i].x, gv[i].y, gv[i].z, gv[i].w};
    uint32_t dow[4] = {0, 0, 0, 0}, dgw[4] = {0, 0, 0, 0};
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 a = bf2_to_f2(ya[k]), d = bf2_to_f2(da[k]);
      const float t0 = a.x * d.x, t1 = a.y * d.y;
      sum += t0 + t1;
      if (kGate) {
        const float2 g = bf2_to_f2(ga[k]);
        dow[k] = f2_to_bf2(d.x * sigmoid_fast(g.x), d.y * sigmoid_fast(g.y));
        dgw[k] = f2_to_bf2(t0 * sigmoid_fast(-g.x), t1 * sigmoid_fast(-g.y));
      }
    }
#pragma unroll
    for (int k = 8; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    if (kGate && n < w.N) {  // (zeros for padding)
      const size_t at = (((size_t)b * w.N + n) * w.heads + h) * kD + sub * 8;
      *reinterpret_cast<uint4*>(d_o + at) = make_uint4(dow[0], dow[1], dow[2], dow[3]);
      __stcs(reinterpret_cast<uint4*>(dg + at), make_uint4(dgw[0], dgw[1], dgw[2], dgw[3]));
    }
    if (n < n_pad && sub == 0) {
      const size_t row = (size_t)b * w.heads + h;
      // a row that sees nothing has lse = -inf; its terms are 2^-inf here
      const float l = live[i] ? lse[row * w.N + n] : -INFINITY;
      nlse[row * n_pad + n] = l == -INFINITY ? -INFINITY : -l * kLog2e;
      ndelta[row * n_pad + n] = live[i] ? -sum : 0.f;
    }
  }
}

// ---------------------------------------------------------------- dkv
// Positions of the queries that see key j: [first, last).
__device__ __forceinline__ int key_first(const WindowDev& w, int j) {
  return w.block == 1 ? j : j / w.block * w.block;
}
__device__ __forceinline__ int key_last(const WindowDev& w, int j) {
  if (w.window == 0 || j < w.sinks) return 0x7fffffff;
  return w.block == 1 ? j + w.window : (j + w.window) / w.block * w.block;
}

// Query tiles (of rows) that see some key of tile kt: [first, first + count).
struct QSpan {
  int first, count;
};
__device__ __forceinline__ QSpan query_span(const WindowDev& w, int kt, int len) {
  const int j0 = kt * kWinTile, j1 = min(j0 + kWinTile, len) - 1;
  QSpan s{0, 0};
  if (j1 < j0) return s;
  const int a = max(key_first(w, j0), w.off);
  int z = min(w.off + w.N, len);
  z = min(z, j0 < w.sinks ? 0x7fffffff : key_last(w, j1));
  if (a >= z) return s;
  s.first = (a - w.off) / kRows;
  s.count = (z - 1 - w.off) / kRows - s.first + 1;
  return s;
}

// How the host cut the work: key tiles [0, sink_tiles) into sink_parts shares of
// sink_chunk (query head, query tile) steps each, the others into win_parts of
// win_chunk.
struct DkvPlan {
  int tiles, sink_tiles, sink_parts, sink_chunk, win_parts, win_chunk;
};

struct DkvCtl {
  uint64_t kv_full;
  uint64_t q_full[kDeep], q_empty[kDeep];      // Q tiles
  uint64_t do_full[kShort], do_empty[kShort];  // do tiles and row statistics
  uint64_t s_full, dp_full, p_full, ds_full, dv_done, dk_done;
  uint32_t tmem;
  int abort_flag;
};
// Dynamic shared memory: K, V, Q ring, do ring (each tile a multiple of 1024
// bytes from the 1024-aligned start), row statistics of each do stage.
constexpr size_t kDkvSmem = (2 + kDeep + kShort) * (size_t)kTileB + kShort * 2 * kRows * sizeof(float);

// Share x of the key head hk and batch entry b, which have `slots` places in part.
__device__ __forceinline__ void dkv_block(uint8_t* smem, int x, int slots, int hk, int b,
                                          const CUtensorMap& tm_q, const CUtensorMap& tm_do,
                                          const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                          const WindowDev& w, const DkvPlan& plan, float sl,
                                          float scale, int n_pad, const float* __restrict__ nlse,
                                          const float* __restrict__ ndelta, float* __restrict__ part,
                                          __nv_bfloat16* __restrict__ dk,
                                          __nv_bfloat16* __restrict__ dv, int* status) {
  uint8_t* k_s = smem;
  uint8_t* v_s = k_s + kTileB;
  uint8_t* q_s = v_s + kTileB;
  uint8_t* do_s = q_s + kDeep * kTileB;
  float* stat = reinterpret_cast<float*>(do_s + kShort * kTileB);  // [stage][-lse, -delta][row]
  DkvCtl& ctl = *reinterpret_cast<DkvCtl*>(stat + kShort * 2 * kRows);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = w.heads / w.kv_heads;
  int kt, share, parts;
  {
    const int in_sinks = plan.sink_tiles * plan.sink_parts;
    if (x < in_sinks) {
      parts = plan.sink_parts;
      kt = x / parts;
      share = x - kt * parts;
    } else {
      parts = plan.win_parts;
      kt = (x - in_sinks) / parts;
      share = x - in_sinks - kt * parts;
      kt += plan.sink_tiles;
    }
  }
  const int len = window_length(w, b);
  const QSpan qs = query_span(w, kt, len);
  const int chunk = kt < plan.sink_tiles ? plan.sink_chunk : plan.win_chunk;
  const int step0 = share * chunk;
  const int steps = max(0, min(group * qs.count - step0, chunk));
  const WaitCtx wc{&ctl.abort_flag, status};
  auto head_of = [&](int t) { return hk * group + (step0 + t) / qs.count; };
  auto qrow_of = [&](int t) { return (qs.first + (step0 + t) % qs.count) * kRows; };

  auto load_tile = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int head, int row) {
    tma_load_3d(dst, map, bar, head * kD, row, b);
    tma_load_3d(dst + kHalf, map, bar, head * kD + 64, row, b);
  };
  auto load_q = [&](int t) {
    const int st = t % kDeep;
    mbar_arrive_expect_tx(&ctl.q_full[st], kTileB);
    load_tile(q_s + st * kTileB, &tm_q, &ctl.q_full[st], head_of(t), qrow_of(t));
  };
  auto load_do = [&](int t) {
    const int st = t % kShort, h = head_of(t), row = qrow_of(t);
    const size_t at = ((size_t)b * w.heads + h) * n_pad + row;
    mbar_arrive_expect_tx(&ctl.do_full[st], kTileB + 2 * kRows * 4);
    load_tile(do_s + st * kTileB, &tm_do, &ctl.do_full[st], h, row);
    bulk_load(stat + st * 2 * kRows, nlse + at, kRows * 4, &ctl.do_full[st]);
    bulk_load(stat + st * 2 * kRows + kRows, ndelta + at, kRows * 4, &ctl.do_full[st]);
  };
  if (warp == kWarpProd && lane == 0) {
    mbar_init(&ctl.kv_full, 1);
    for (int i = 0; i < kDeep; ++i) {
      mbar_init(&ctl.q_full[i], 1);
      mbar_init(&ctl.q_empty[i], 1);
    }
    for (int i = 0; i < kShort; ++i) {
      mbar_init(&ctl.do_full[i], 1);
      mbar_init(&ctl.do_empty[i], 1);
    }
    mbar_init(&ctl.s_full, 1);
    mbar_init(&ctl.dp_full, 1);
    mbar_init(&ctl.p_full, kSoft);
    mbar_init(&ctl.ds_full, kSoft);
    mbar_init(&ctl.dv_done, 1);
    mbar_init(&ctl.dk_done, 1);
    ctl.abort_flag = 0;
    mbar_fence_init();
    if (steps > 0) {  // the first loads run while the rest of the CTA sets up
      mbar_arrive_expect_tx(&ctl.kv_full, 2 * kTileB);
      load_tile(k_s, &tm_k, &ctl.kv_full, hk, kt * kRows);
      load_q(0);
      load_tile(v_s, &tm_v, &ctl.kv_full, hk, kt * kRows);
    }
    griddep_wait();  // do and the statistics come from prep
    if (steps > 0) load_do(0);
  }
  if (warp == kWarpMma) {
    tmem_alloc(&ctl.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  const uint32_t t_s = tmem, t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 384;

  if (warp == kWarpProd) {
    if (lane == 0 && steps > 0) {
      int nq = 1, nd = 1;
      for (int t = 1; t < steps; ++t) {
        if (t >= kDeep && !mbar_wait(&ctl.q_empty[t % kDeep], ((t / kDeep) - 1) & 1, wc, 0xa1)) break;
        load_q(t);
        ++nq;
        // a do slot is free once dV has read it, its statistics' slot once dS is
        // made, which dK's end (q_empty) implies
        if (t >= kShort && (!mbar_wait(&ctl.do_empty[t % kShort], ((t / kShort) - 1) & 1, wc, 0xab) ||
                            !mbar_wait(&ctl.q_empty[(t - kShort) % kDeep], ((t - kShort) / kDeep) & 1, wc, 0xb0)))
          break;
        load_do(t);
        ++nd;
      }
      if (*wc.abort_flag) {  // loads still in flight land before the CTA exits
        mbar_drain(&ctl.kv_full, 0);
        for (int t = nq > kDeep ? nq - kDeep : 0; t < nq; ++t) mbar_drain(&ctl.q_full[t % kDeep], (t / kDeep) & 1);
        for (int t = nd > kShort ? nd - kShort : 0; t < nd; ++t) mbar_drain(&ctl.do_full[t % kShort], (t / kShort) & 1);
      }
    }
  } else if (warp == kWarpMma) {
    if (steps > 0) {  // the whole warp, its elected lane issues
      const uint32_t lead = elect_lead();
      const uint32_t idesc_s = idesc_bf16_f32(128, 128, 0, 0);  // K Q^T, V do^T
      const uint32_t idesc_g = idesc_bf16_f32(128, 128, 0, 1);  // P^T do, dS^T Q (rows of B along K)
      const uint64_t dk0 = smem_desc_sw128(smem_u32(k_s), 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(smem_u32(v_s), 16, 1024);
      const uint64_t dq0 = smem_desc_sw128(smem_u32(q_s), 16, 1024);
      const uint64_t dd0 = smem_desc_sw128(smem_u32(do_s), 16, 1024);
      const uint64_t mq0 = smem_desc_sw128(smem_u32(q_s), kHalf, 1024);
      const uint64_t md0 = smem_desc_sw128(smem_u32(do_s), kHalf, 1024);
      auto issue_ab = [&](uint32_t d, uint64_t a, uint64_t bt) {  // D = A B^T
        a = desc_local(a);
        bt = desc_local(bt);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint32_t o = (kk >> 2) * kHalf + (kk & 3) * 32;
          umma_ss_lead(lead, d, desc_advance(a, o), desc_advance(bt, o), idesc_s, kk != 0);
        }
      };
      // D += A B, A in TMEM: the 32 columns of each warp quarter over the first
      // half of its 32 score columns
      auto issue_acc = [&](uint32_t d, uint32_t a, uint64_t bm, bool acc) {
        bm = desc_local(bm);
#pragma unroll
        for (int kk = 0; kk < kRows / 16; ++kk)
          umma_ts_lead(lead, d, a + (kk >> 1) * 32 + (kk & 1) * 8, desc_advance(bm, kk * 2048), idesc_g, acc || kk != 0);
      };
      bool ok = mbar_wait(&ctl.kv_full, 0, wc, 0xa2) && mbar_wait(&ctl.q_full[0], 0, wc, 0xa3);
      if (ok) {
        tc_fence_after();
        issue_ab(t_s, dk0, dq0);
        umma_commit_lead(lead, &ctl.s_full);
        ok = mbar_wait(&ctl.do_full[0], 0, wc, 0xac);
      }
      if (ok) {
        tc_fence_after();
        issue_ab(t_dp, dv0, dd0);
        umma_commit_lead(lead, &ctl.dp_full);
      }
      for (int t = 0; ok && t < steps; ++t) {
        const bool more = t + 1 < steps;
        const uint32_t qc = (t % kDeep) * kTileB, qn = ((t + 1) % kDeep) * kTileB;
        const uint32_t dc = (t % kShort) * kTileB, dn = ((t + 1) % kShort) * kTileB;
        if (!mbar_wait(&ctl.p_full, t & 1, wc, 0xa4)) break;
        tc_fence_after();
        issue_acc(t_dv, t_s, desc_advance(md0, dc), t > 0);
        umma_commit_lead(lead, &ctl.dv_done);
        umma_commit_lead(lead, &ctl.do_empty[t % kShort]);
        if (more) {
          if (!mbar_wait(&ctl.q_full[(t + 1) % kDeep], ((t + 1) / kDeep) & 1, wc, 0xa3) ||
              !mbar_wait(&ctl.dv_done, t & 1, wc, 0xa6))
            break;
          tc_fence_after();
          issue_ab(t_s, dk0, desc_advance(dq0, qn));
          umma_commit_lead(lead, &ctl.s_full);
        }
        if (!mbar_wait(&ctl.ds_full, t & 1, wc, 0xa5)) break;
        tc_fence_after();
        issue_acc(t_dk, t_dp, desc_advance(mq0, qc), t > 0);
        umma_commit_lead(lead, &ctl.dk_done);
        umma_commit_lead(lead, &ctl.q_empty[t % kDeep]);
        if (more) {
          if (!mbar_wait(&ctl.do_full[(t + 1) % kShort], ((t + 1) / kShort) & 1, wc, 0xac) ||
              !mbar_wait(&ctl.dk_done, t & 1, wc, 0xad))
            break;
          tc_fence_after();
          issue_ab(t_dp, dv0, desc_advance(dd0, dn));
          umma_commit_lead(lead, &ctl.dp_full);
        }
      }
    }
  } else {
    // ------------------------------------------------ softmax warps: thread = key row, 32 queries
    const int cg = warp >> 2;              // which quarter of the query tile
    const int r = (warp & 3) * 32 + lane;  // key row
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t my_s = t_s + cg * 32 + lane_base, my_dp = t_dp + cg * 32 + lane_base;
    const int j0 = kt * kRows, j = j0 + r;
    const int q_end = min(w.off + w.N, len);
    const int first = key_first(w, j), last = j < len ? min(key_last(w, j), q_end) : 0;
    // every key of the tile is seen from all_first on, up to all_last
    const int all_first = key_first(w, j0 + kRows - 1);
    const int all_last = j0 + kRows <= len ? min(j0 + kRows <= w.sinks ? 0x7fffffff : key_last(w, max(j0, w.sinks)), q_end) : 0;
    const uint64_t sl2 = pk2(sl, sl);
    bool ok = true;
    for (int t = 0; t < steps; ++t) {
      const int sq = t % kDeep, sd = t % kShort;
      const int p0 = w.off + qrow_of(t) + cg * 32;
      const float* st = stat + sd * 2 * kRows + cg * 32;
      ok = mbar_wait(&ctl.do_full[sd], (t / kShort) & 1, wc, 0xa7) && mbar_wait(&ctl.s_full, t & 1, wc, 0xa8);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool masked = p0 < all_first || p0 + 32 > all_last;
      const uint32_t vis = masked ? bits_below(last - p0) & ~bits_below(first - p0) : ~0u;
      uint32_t buf[32], pk[16];
      tmem_ld32(my_s, buf);
      tmem_ld_wait();
      tmem_tie(buf);
      float p[32];
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(st + i);
        const uint64_t n2[2] = {pk2(v.x, v.y), pk2(v.z, v.w)};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int k = i + 2 * e;
          const uint64_t x = fma2(pk2(__uint_as_float(buf[k]), __uint_as_float(buf[k + 1])), sl2, n2[e]);
          if (((k >> 1) & 7) >= 8 - kEmuPairs) {
            exp2_pair(x, p[k], p[k + 1]);
          } else {
            up2(x, p[k], p[k + 1]);
            p[k] = ex2(p[k]);
            p[k + 1] = ex2(p[k + 1]);
          }
        }
      }
      if (masked) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (!(vis & (1u << i))) p[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) pk[i] = f2_to_bf2(p[2 * i], p[2 * i + 1]);
      tmem_st16(my_s, pk);  // over columns already read
      const bool pad = p0 + 32 > len && len < w.off + w.N;
      if (pad) {
        // padding rows of do meet P = 0: zero them, whatever they hold (do is
        // read only by the products that wait for p_full from here on)
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.dp_full, t & 1, wc, 0xae));
        if (!ok) break;
        if (r < 32 && p0 + r >= len) {
#pragma unroll
          for (int c = 0; c < 16; ++c)
            *reinterpret_cast<uint4*>(do_s + sd * kTileB + (c >> 3) * kHalf + sw128_off(cg * 32 + r, c & 7)) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&ctl.p_full);
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl.dp_full, t & 1, wc, 0xaf));
      if (!ok) break;
      tc_fence_after();
      tmem_ld32(my_dp, buf);
      tmem_ld_wait();
      tmem_tie(buf);
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(st + kRows + i);
        const uint64_t n2[2] = {pk2(v.x, v.y), pk2(v.z, v.w)};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int k = i + 2 * e;
          const uint64_t d = add2(pk2(__uint_as_float(buf[k]), __uint_as_float(buf[k + 1])), n2[e]);
          up2(mul2(d, pk2(p[k], p[k + 1])), p[k], p[k + 1]);
        }
      }
      if (masked) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (!(vis & (1u << i))) p[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) pk[i] = f2_to_bf2(p[2 * i], p[2 * i + 1]);
      tmem_st16(my_dp, pk);
      if (pad) {  // and padding rows of Q meet dS = 0 (S of this tile is done)
        if (r < 32 && p0 + r >= len) {
#pragma unroll
          for (int c = 0; c < 16; ++c)
            *reinterpret_cast<uint4*>(q_s + sq * kTileB + (c >> 3) * kHalf + sw128_off(cg * 32 + r, c & 7)) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&ctl.ds_full);
    }
    // ---------------- epilogue: quarters 0, 1 write dV, 2, 3 dK, 64 columns each
    if (steps > 0 && ok) {
      ok = mbar_wait(&ctl.dk_done, (steps - 1) & 1, wc, 0xa9) && mbar_wait(&ctl.dv_done, (steps - 1) & 1, wc, 0xaa);
      ok = __all_sync(0xffffffffu, ok);
    }
    if (ok && (parts == 1 || steps > 0)) {
      tc_fence_after();
      const int which = cg >> 1, col = (cg & 1) * 64;
      const float mul = which ? scale : 1.f;
      __nv_bfloat16* dst = (which ? dk : dv) + (((size_t)b * w.N_keys + j) * w.kv_heads + hk) * kD + col;
      float* pdst = part + (((((size_t)b * w.kv_heads + hk) * slots + x) * 2 + which) * kRows + r) * kD + col;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t o[32];
        if (steps > 0) {
          tmem_ld32((which ? t_dk : t_dv) + lane_base + col + c * 32, o);
          tmem_ld_wait();
          tmem_tie(o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0;
        }
        if (parts > 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(pdst + c * 32 + 4 * i) =
                make_float4(mul * __uint_as_float(o[4 * i]), mul * __uint_as_float(o[4 * i + 1]),
                            mul * __uint_as_float(o[4 * i + 2]), mul * __uint_as_float(o[4 * i + 3]));
        } else if (j < w.N_keys) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = f2_to_bf2(mul * __uint_as_float(o[8 * i + 2 * e]), mul * __uint_as_float(o[8 * i + 2 * e + 1]));
            *reinterpret_cast<uint4*>(dst + c * 32 + 8 * i) = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    if (*wc.abort_flag && steps > 0) {  // MMAs in flight finish before TMEM is freed
      mbar_drain(&ctl.dv_done, (steps - 1) & 1);
      mbar_drain(&ctl.dk_done, (steps - 1) & 1);
    }
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Sums the shares of the split key tiles in order.  One CTA per (slice of 16 rows
// of a split key tile's dV or dK; key head; batch); thread = 4 columns of a row.
constexpr int kJoinRows = 16;
__global__ void __launch_bounds__(kJoinRows * kD / 4)
    window_join_kernel(const float* part, const WindowDev w, const DkvPlan plan,
                       int slots, __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv) {
  constexpr int kSlices = kRows / kJoinRows;
  part = griddep_wait_for(part);
  const int hk = blockIdx.y, b = blockIdx.z, slice = blockIdx.x % kSlices;
  const int which = blockIdx.x / kSlices & 1, s = blockIdx.x / (2 * kSlices);
  const int split_sinks = plan.sink_parts > 1 ? plan.sink_tiles : 0;
  const int kt = s < split_sinks ? s : plan.sink_tiles + (s - split_sinks);
  const bool sink = kt < plan.sink_tiles;
  const int item = sink ? kt * plan.sink_parts
                        : plan.sink_tiles * plan.sink_parts + (kt - plan.sink_tiles) * plan.win_parts;
  const QSpan qs = query_span(w, kt, window_length(w, b));
  const int chunk = sink ? plan.sink_chunk : plan.win_chunk;
  const int n = (w.heads / w.kv_heads * qs.count + chunk - 1) / chunk;  // shares written
  const int i = slice * kJoinRows * (kD / 4) + threadIdx.x, j = kt * kRows + i / (kD / 4);
  if (j >= w.N_keys) return;
  const float4* p = reinterpret_cast<const float4*>(
                        part + ((((size_t)b * w.kv_heads + hk) * slots + item) * 2 + which) * kRows * kD) + i;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int k = 0; k < n; ++k) {
    const float4 v = __ldcs(p + (size_t)k * 2 * kRows * kD / 4);
    a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
  }
  *reinterpret_cast<uint2*>((which ? dk : dv) + (((size_t)b * w.N_keys + j) * w.kv_heads + hk) * kD + (i % (kD / 4)) * 4) =
      make_uint2(f2_to_bf2(a.x, a.y), f2_to_bf2(a.z, a.w));
}

// ---------------------------------------------------------------- dq
struct DqCtl {
  uint64_t q_full;
  uint64_t k_full[kDeep], k_empty[kDeep];
  uint64_t v_full[kShort], v_empty[kShort];
  uint64_t s_full[2], dp_full, ds_full, dq_done;
  uint64_t dq_last;  // the last product, and with it all before: completes once
  uint32_t tmem;
  int abort_flag;
};
// Dynamic shared memory: Q, do, K ring, V ring.
constexpr size_t kDqSmem = (2 + kDeep + kShort) * (size_t)kTileB;

__device__ __forceinline__ void dq_block(uint8_t* smem, int qt, int h, int b, const CUtensorMap& tm_q,
                                         const CUtensorMap& tm_do, const CUtensorMap& tm_k,
                                         const CUtensorMap& tm_v, const WindowDev& w, float sl,
                                         float scale, int n_pad, const float* __restrict__ nlse,
                                         const float* __restrict__ ndelta,
                                         __nv_bfloat16* __restrict__ dq, int* status) {
  uint8_t* q_s = smem;
  uint8_t* do_s = q_s + kTileB;
  uint8_t* k_s = do_s + kTileB;
  uint8_t* v_s = k_s + kDeep * kTileB;
  DqCtl& ctl = *reinterpret_cast<DqCtl*>(v_s + kShort * kTileB);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = h / (w.heads / w.kv_heads);
  const int row0 = qt * kRows;
  const int len = window_length(w, b);
  const TileSpan span = window_span(w, w.off + row0, w.off + min(row0 + kRows, w.N) - 1, len);
  const int steps = span.count();
  auto tile_of = [&](int t) { return t < span.ns ? t : span.w0 + t - span.ns; };
  auto width_of = [&](int t) { return span.width(tile_of(t), w.sinks); };
  const WaitCtx wc{&ctl.abort_flag, status};

  auto load_tile = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int head, int row) {
    tma_load_3d(dst, map, bar, head * kD, row, b);
    tma_load_3d(dst + kHalf, map, bar, head * kD + 64, row, b);
  };
  auto load_k = [&](int t) {
    const int st = t % kDeep;
    mbar_arrive_expect_tx(&ctl.k_full[st], kTileB);
    load_tile(k_s + st * kTileB, &tm_k, &ctl.k_full[st], hk, tile_of(t) * kRows);
  };
  auto load_v = [&](int t) {
    const int st = t % kShort;
    mbar_arrive_expect_tx(&ctl.v_full[st], kTileB);
    load_tile(v_s + st * kTileB, &tm_v, &ctl.v_full[st], hk, tile_of(t) * kRows);
  };
  if (warp == kWarpProd && lane == 0) {
    mbar_init(&ctl.q_full, 1);
    for (int i = 0; i < kDeep; ++i) {
      mbar_init(&ctl.k_full[i], 1);
      mbar_init(&ctl.k_empty[i], 1);
    }
    for (int i = 0; i < kShort; ++i) {
      mbar_init(&ctl.v_full[i], 1);
      mbar_init(&ctl.v_empty[i], 1);
    }
    mbar_init(&ctl.s_full[0], 1);
    mbar_init(&ctl.s_full[1], 1);
    mbar_init(&ctl.dp_full, 1);
    mbar_init(&ctl.ds_full, kSoft);
    mbar_init(&ctl.dq_done, 1);
    mbar_init(&ctl.dq_last, 1);
    ctl.abort_flag = 0;
    mbar_fence_init();
    if (steps > 0) {  // the first loads run while the rest of the CTA sets up
      mbar_arrive_expect_tx(&ctl.q_full, 2 * kTileB);
      load_tile(q_s, &tm_q, &ctl.q_full, h, row0);
      load_k(0);
      load_v(0);
      griddep_wait();  // do and the statistics come from prep
      load_tile(do_s, &tm_do, &ctl.q_full, h, row0);
    }
  }
  if (warp == kWarpMma) {
    tmem_alloc(&ctl.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  const uint32_t t_dp = tmem + 256, t_dq = tmem + 384;  // S buffers at 0 and 128

  if (warp == kWarpProd) {
    if (lane == 0 && steps > 0) {
      int nk = 1, nv = 1;
      for (int t = 1; t < steps; ++t) {
        if (t >= kDeep && !mbar_wait(&ctl.k_empty[t % kDeep], ((t / kDeep) - 1) & 1, wc, 0xb1)) break;
        load_k(t);
        ++nk;
        if (t >= kShort && !mbar_wait(&ctl.v_empty[t % kShort], ((t / kShort) - 1) & 1, wc, 0xbb)) break;
        load_v(t);
        ++nv;
      }
      if (*wc.abort_flag) {
        mbar_drain(&ctl.q_full, 0);
        for (int t = nk > kDeep ? nk - kDeep : 0; t < nk; ++t) mbar_drain(&ctl.k_full[t % kDeep], (t / kDeep) & 1);
        for (int t = nv > kShort ? nv - kShort : 0; t < nv; ++t) mbar_drain(&ctl.v_full[t % kShort], (t / kShort) & 1);
      }
    }
  } else if (warp == kWarpMma) {
    if (steps > 0) {  // the whole warp, its elected lane issues
      const uint32_t lead = elect_lead();
      const uint32_t idesc_s = idesc_bf16_f32(128, 0, 0, 0);  // Q K^T, do V^T; N by the tile's width
      const uint32_t idesc_g = idesc_bf16_f32(128, 128, 0, 1);  // dS K
      const uint64_t dq0 = smem_desc_sw128(smem_u32(q_s), 16, 1024);
      const uint64_t dd0 = smem_desc_sw128(smem_u32(do_s), 16, 1024);
      const uint64_t dk0 = smem_desc_sw128(smem_u32(k_s), 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(smem_u32(v_s), 16, 1024);
      const uint64_t mk0 = smem_desc_sw128(smem_u32(k_s), kHalf, 1024);
      auto issue_ab = [&](uint32_t d, uint64_t a, uint64_t bt, int width) {  // D = A B^T over `width` keys
        const uint32_t idesc = idesc_s | (uint32_t)(width >> 3) << 17;
        a = desc_local(a);
        bt = desc_local(bt);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint32_t o = (kk >> 2) * kHalf + (kk & 3) * 32;
          umma_ss_lead(lead, d, desc_advance(a, o), desc_advance(bt, o), idesc, kk != 0);
        }
      };
      auto issue_s = [&](int t) {
        issue_ab(tmem + (t & 1) * 128, dq0, desc_advance(dk0, (t % kDeep) * kTileB), width_of(t));
        umma_commit_lead(lead, &ctl.s_full[t & 1]);
      };
      auto issue_dp = [&](int t) {
        issue_ab(t_dp, dd0, desc_advance(dv0, (t % kShort) * kTileB), width_of(t));
        umma_commit_lead(lead, &ctl.dp_full);
        umma_commit_lead(lead, &ctl.v_empty[t % kShort]);
      };
      bool ok = mbar_wait(&ctl.q_full, 0, wc, 0xb2) && mbar_wait(&ctl.k_full[0], 0, wc, 0xb3);
      if (ok) {
        tc_fence_after();
        issue_s(0);
        ok = mbar_wait(&ctl.v_full[0], 0, wc, 0xbc);
      }
      if (ok) {
        tc_fence_after();
        issue_dp(0);
      }
      if (ok && steps > 1) {
        ok = mbar_wait(&ctl.k_full[1], 0, wc, 0xb3);
        if (ok) {
          tc_fence_after();
          issue_s(1);
        }
      }
      for (int t = 0; ok && t < steps; ++t) {
        if (!mbar_wait(&ctl.ds_full, t & 1, wc, 0xb5)) break;  // dS is written, dP read
        tc_fence_after();
        if (t + 1 < steps) {
          if (!mbar_wait(&ctl.v_full[(t + 1) % kShort], ((t + 1) / kShort) & 1, wc, 0xbc)) break;
          tc_fence_after();
          issue_dp(t + 1);
        }
        const uint64_t bm = desc_local(desc_advance(mk0, (t % kDeep) * kTileB));
        const int ksteps = width_of(t) / 16;
#pragma unroll
        for (int kk = 0; kk < kRows / 16; ++kk)
          if (kk < ksteps) umma_ts_lead(lead, t_dq, tmem + (t & 1) * 128 + (kk >> 1) * 32 + (kk & 1) * 8, desc_advance(bm, kk * 2048),
                       idesc_g, (t | kk) != 0);
        umma_commit_lead(lead, t + 1 < steps ? &ctl.dq_done : &ctl.dq_last);
        umma_commit_lead(lead, &ctl.k_empty[t % kDeep]);
        if (t + 2 < steps) {
          if (!mbar_wait(&ctl.k_full[(t + 2) % kDeep], ((t + 2) / kDeep) & 1, wc, 0xb3) ||
              !mbar_wait(&ctl.dq_done, t & 1, wc, 0xb6))  // dS of this buffer has been read
            break;
          tc_fence_after();
          issue_s(t + 2);
        }
      }
    }
  } else {
    // ------------------------------------------------ softmax warps: thread = query row, 32 keys
    const int cg = warp >> 2;              // which quarter of the key tile
    const int r = (warp & 3) * 32 + lane;  // query row
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const int row = row0 + r, pos = w.off + row;
    const int end = min(window_end(w, pos), len), low = window_low(w, window_end(w, pos));
    const int pos1 = min(min(w.off + row0 + kRows, w.off + w.N), len) - 1;
    const int all_end = pos1 - w.off - row0 < kRows - 1 ? 0 : min(window_end(w, w.off + row0), len);
    const int all_low = window_low(w, window_end(w, max(pos1, 0)));
    const size_t at = ((size_t)b * w.heads + h) * n_pad + row;  // row < n_pad
    const float nl = griddep_wait_for(nlse)[at], nd = griddep_wait_for(ndelta)[at];
    const bool live = nl != -INFINITY;
    const uint64_t sl2 = pk2(sl, sl), nl2 = pk2(nl, nl), nd2 = pk2(nd, nd);
    bool ok = true;
    for (int t = 0; t < steps; ++t) {
      const int key0 = tile_of(t) * kRows + cg * 32;
      const uint32_t my_s = tmem + (t & 1) * 128 + cg * 32 + lane_base, my_dp = t_dp + cg * 32 + lane_base;
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl.s_full[t & 1], (t >> 1) & 1, wc, 0xb8));
      if (!ok) break;
      tc_fence_after();
      // (a tile with dead rows is always masked)
      const bool masked = key0 + 32 > all_end || (key0 < all_low && key0 + 32 > w.sinks);
      if (cg * 32 >= width_of(t)) {  // columns that no row of the tile sees were not made
        ok = __all_sync(0xffffffffu, mbar_wait(&ctl.dp_full, t & 1, wc, 0xbd));
        if (!ok) break;
        mbar_arrive(&ctl.ds_full);
        continue;
      }
      uint32_t buf[32], pk[16];
      tmem_ld32(my_s, buf);
      tmem_ld_wait();
      tmem_tie(buf);
      float p[32];
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const uint64_t x = fma2(pk2(__uint_as_float(buf[i]), __uint_as_float(buf[i + 1])), sl2, nl2);
        if (((i >> 1) & 7) >= 8 - kEmuPairs) {
          exp2_pair(x, p[i], p[i + 1]);
        } else {
          up2(x, p[i], p[i + 1]);
          p[i] = ex2(p[i]);
          p[i + 1] = ex2(p[i + 1]);
        }
      }
      ok = __all_sync(0xffffffffu, mbar_wait(&ctl.dp_full, t & 1, wc, 0xb9));
      if (!ok) break;
      tc_fence_after();
      tmem_ld32(my_dp, buf);
      tmem_ld_wait();
      tmem_tie(buf);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const uint64_t d = add2(pk2(__uint_as_float(buf[i]), __uint_as_float(buf[i + 1])), nd2);
        up2(mul2(d, pk2(p[i], p[i + 1])), p[i], p[i + 1]);
      }
      if (masked) {
        const uint32_t vis = live ? visible_bits(key0, low, end, w.sinks) : 0u;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (!(vis & (1u << i))) p[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) pk[i] = f2_to_bf2(p[2 * i], p[2 * i + 1]);
      tmem_st16(my_s, pk);
      if (key0 + 32 > len && len < w.N_keys) {
        // padding rows of K meet dS = 0: zero them, whatever they hold
        if (r < 32 && key0 + r >= len) {
#pragma unroll
          for (int c = 0; c < 16; ++c)
            *reinterpret_cast<uint4*>(k_s + (t % kDeep) * kTileB + (c >> 3) * kHalf + sw128_off(cg * 32 + r, c & 7)) =
                make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&ctl.ds_full);
    }
    // ---------------- epilogue: each quarter writes its 32 columns
    // The last product has a barrier of its own: nothing here follows dq_done phase
    // by phase, and both of its parities come round while these warps finish dS.
    if (steps > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait(&ctl.dq_last, 0, wc, 0xba));
    if (ok) {
      tc_fence_after();
      __nv_bfloat16* dst = dq + (((size_t)b * w.N + row) * w.heads + h) * kD + cg * 32;
      uint32_t o[32];
      if (steps > 0) {
        tmem_ld32(t_dq + lane_base + cg * 32, o);
        tmem_ld_wait();
        tmem_tie(o);
      }
      if (row < w.N) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = live && steps > 0 ? f2_to_bf2(scale * __uint_as_float(o[8 * i + 2 * e]),
                                                 scale * __uint_as_float(o[8 * i + 2 * e + 1]))
                                     : 0u;
          *reinterpret_cast<uint4*>(dst + 8 * i) = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    if (*wc.abort_flag && steps > 0) mbar_drain(&ctl.dq_last, 0);  // MMAs in flight finish before TMEM is freed
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- both
constexpr size_t kDkvAll = kDkvSmem + sizeof(DkvCtl), kDqAll = kDqSmem + sizeof(DqCtl);
constexpr size_t kGradSmem = kDkvAll > kDqAll ? kDkvAll : kDqAll;
static_assert(kGradSmem <= 227 * 1024, "shared memory");

// The dkv blocks, then the dq blocks, which fill the SMs of the last dkv wave.
__global__ void __launch_bounds__(kThreads, 1)
    window_grad_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                       const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const WindowDev w, const DkvPlan plan, int items, int slots, int dkv_blocks, int q_tiles, float sl,
                       float scale, int n_pad, const float* __restrict__ nlse,
                       const float* __restrict__ ndelta, float* __restrict__ part,
                       __nv_bfloat16* __restrict__ dq, __nv_bfloat16* __restrict__ dk,
                       __nv_bfloat16* __restrict__ dv, int* status) {
  extern __shared__ __align__(1024) uint8_t smem[];
  griddep_launch_next();
  int i = blockIdx.x;
  if (i < dkv_blocks) {
    const int x = i % items;
    i /= items;
    dkv_block(smem, x, slots, i % w.kv_heads, i / w.kv_heads, tm_q, tm_do, tm_k, tm_v, w, plan, sl, scale,
              n_pad, nlse, ndelta, part, dk, dv, status);
  } else {
    i -= dkv_blocks;
    const int qt = q_tiles - 1 - i % q_tiles;  // the longest first
    i /= q_tiles;
    dq_block(smem, qt, i % w.heads, i / w.heads, tm_q, tm_do, tm_k, tm_v, w, sl, scale, n_pad, nlse, ndelta,
             dq, status);
  }
}

// A dkv block takes at most as many steps as would keep every SM busy equally long
// (`even`: a dq block's step takes 7/10 of a dkv block's), so that the dq blocks can
// fill what the dkv blocks leave, and a share at least kLeast.  The sinks' tiles,
// which all later queries see, are cut to half of that.  Against cutting into two
// blocks for every SM, down to 4 steps: 16000 rows, 1 head, window 1000, 54 against
// 83 us; 2 x 4000 rows, 16 heads on 4, window 512, 216 against 265; 1023 rows, 8
// heads on 1, no window, 40 against 34.  kLeast 4 or 6 against 8: 2000 rows, 4 heads,
// no window, 52 against 42 us.
constexpr long long kLeast = 8;
DkvPlan dkv_plan(const WindowCall& c) {
  DkvPlan p{};
  const long long group = c.heads / c.kv_heads, columns = (long long)c.kv_heads * c.B;
  const long long q_tiles = (c.N + kRows - 1) / kRows;
  p.tiles = (c.N_keys + kRows - 1) / kRows;
  // query tiles that a key tile's window can reach
  long long reach = q_tiles;
  if (c.window) {
    const long long span = ((long long)c.window + c.block + 2 * kRows - 3) / kRows + 1;
    reach = span < q_tiles ? span : q_tiles;
    p.sink_tiles = (c.sinks + kRows - 1) / kRows;
    if (p.sink_tiles > p.tiles) p.sink_tiles = p.tiles;
  }
  const long long base = group * reach, sink_steps = group * q_tiles;
  // The last key tiles are seen from fewer query tiles.  (Tiles before the first
  // window, which nobody sees, count too: their shares would take workspace.)
  const long long pairs = columns * (group * (p.tiles * reach - reach * (reach - 1) / 2) + p.sink_tiles * sink_steps);
  const long long even = (pairs * 17 / 10 + kNumSMs - 1) / kNumSMs;
  long long chunk = even < kLeast ? kLeast : even;
  if (chunk > base) chunk = base;
  p.win_chunk = (int)chunk;
  p.win_parts = (int)((base + chunk - 1) / chunk);
  chunk = even / 2 < kLeast ? kLeast : even / 2;
  if (chunk > sink_steps) chunk = sink_steps;
  p.sink_chunk = (int)chunk;
  p.sink_parts = (int)((sink_steps + chunk - 1) / chunk);
  return p;
}
int dkv_items(const DkvPlan& p) {
  return p.sink_tiles * p.sink_parts + (p.tiles - p.sink_tiles) * p.win_parts;
}
// Shares that are written out (the sinks' come first).
int dkv_slots(const DkvPlan& p) {
  if (p.win_parts > 1) return dkv_items(p);
  return p.sink_parts > 1 ? p.sink_tiles * p.sink_parts : 0;
}

struct BwdWs {
  __nv_bfloat16* d_o;
  float *nlse, *ndelta, *part;
  size_t bytes;
};
int pad_rows(int n) { return (n + kRows - 1) / kRows * kRows; }
BwdWs carve(const WindowCall& c, void* ws) {
  Carver cv(ws, ~size_t(0));
  BwdWs w{};
  const size_t rows = (size_t)c.B * c.heads * pad_rows(c.N);
  w.nlse = cv.take<float>(rows);
  w.ndelta = cv.take<float>(rows);
  if (c.gate) w.d_o = cv.take<__nv_bfloat16>((size_t)c.B * c.N * c.heads * kD);
  const DkvPlan p = dkv_plan(c);
  if (const int slots = dkv_slots(p)) w.part = cv.take<float>((size_t)c.B * c.kv_heads * slots * 2 * kRows * kD);
  w.bytes = align_up(cv.used, 256);
  return w;
}

}  // namespace

size_t window_bwd_ws_bytes(const WindowCall& c) { return carve(c, nullptr).bytes; }

sana_status window_bwd_run(const WindowCall& c, const void* y, const float* lse, const void* dy,
                           void* dq, void* dk, void* dv, void* dg, void* ws, cudaStream_t st) {
  const BwdWs m = carve(c, ws);
  const int n_pad = pad_rows(c.N);
  const DkvPlan p = dkv_plan(c);
  const int items = dkv_items(p), slots = dkv_slots(p), q_tiles = n_pad / kRows;
  const long long dkv_blocks = (long long)items * c.kv_heads * c.B, dq_blocks = (long long)q_tiles * c.heads * c.B;
  if (dkv_blocks + dq_blocks > 0x7fffffffLL)
    return fail(SANA_ERR_UNSUPPORTED, "windowed anchor backward: too many tiles (%lld)", dkv_blocks + dq_blocks);
  const WindowDev w{c.N, c.N_keys, c.N_keys - c.N, c.window, c.sinks, c.block, c.heads, c.kv_heads, c.lengths};
  const uint64_t N = c.N, Nk = c.N_keys, C = (uint64_t)c.heads * kD, Ck = (uint64_t)c.kv_heads * kD;
  const void* d_o = c.gate ? static_cast<const void*>(m.d_o) : dy;
  CUtensorMap tq, td, tk, tv;
  if (!make_tmap_bf16_3d(&tq, c.q, C, N, c.B, c.q_stride, N * c.q_stride, kRows) ||
      !make_tmap_bf16_3d(&td, d_o, C, N, c.B, C, N * C, kRows) ||
      !make_tmap_bf16_3d(&tk, c.k, Ck, Nk, c.B, c.k_stride, Nk * c.k_stride, kRows) ||
      !make_tmap_bf16_3d(&tv, c.v, Ck, Nk, c.B, c.v_stride, Nk * c.v_stride, kRows))
    return fail(SANA_ERR_CUDA, "windowed anchor backward: cuTensorMapEncodeTiled failed");
  once_per_context(kAttrWindowBwd, [] {
    cudaFuncSetAttribute(window_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGradSmem);
  });
  using bf = __nv_bfloat16;
  const dim3 prep((unsigned)c.heads * (unsigned)(n_pad / kPrepRows), 1, c.B);
  if (c.gate)
    window_prep_kernel<true><<<prep, 256, 0, st>>>((const bf*)y, (const bf*)dy, (const bf*)c.gate, c.gate_stride, lse,
                                                   w, n_pad, m.nlse, m.ndelta, m.d_o, (bf*)dg);
  else
    window_prep_kernel<false><<<prep, 256, 0, st>>>((const bf*)y, (const bf*)dy, nullptr, 0, lse, w, n_pad, m.nlse,
                                                    m.ndelta, nullptr, nullptr);
  if (sana_status e = check_launch("window_prep_kernel")) return e;
  const float sl = c.scale * kLog2e;
  int* sw = status_word();
  launch_dependent(window_grad_kernel, dim3((unsigned)(dkv_blocks + dq_blocks)), dim3(kThreads), kGradSmem, st, tq, td,
                   tk, tv, w, p, items, slots, (int)dkv_blocks, q_tiles, sl, c.scale, n_pad, m.nlse, m.ndelta, m.part, (bf*)dq,
                   (bf*)dk, (bf*)dv, sw);
  if (sana_status e = check_launch("window_grad_kernel")) return e;
  const int split = (p.sink_parts > 1 ? p.sink_tiles : 0) + (p.win_parts > 1 ? p.tiles - p.sink_tiles : 0);
  if (!split) return SANA_OK;
  launch_dependent(window_join_kernel, dim3(2 * split * (kRows / kJoinRows), c.kv_heads, c.B), dim3(kJoinRows * kD / 4),
                   0, st, m.part, w, p, slots, (bf*)dk, (bf*)dv);
  return check_launch("window_join_kernel");
}

}  // namespace sana
