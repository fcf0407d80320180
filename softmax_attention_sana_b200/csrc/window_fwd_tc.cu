// Windowed softmax anchor, forward, bf16 on tcgen05 (the mask: window.cuh).
//
//   Y_i = sigmoid(G_i) * sum_j p_ij V_j,  p_ij = exp(s_ij - lse_i) over the
//   visible j,  s_ij = scale q_i . k_j,  lse_i = log sum_j exp(s_ij).
//
// One pass over the visible key tiles with a running maximum and sum in fp32
// (base 2; the sum is taken over the fp32 exponentials, which are then rounded
// to bf16 as the A operand of P V: each rounding is 2^-9 of its term and they
// average out).
//
// One CTA per (batch, kQ 128-query tiles: of one query head, or of two that share a
// key head).  With two query tiles they share the K and V tiles in shared memory
// and their softmax warpgroups alternate with the tensor core; with one, two CTAs
// share an SM, alternate the same way, and one's start and end run under the
// other's loop, at twice the K and V traffic: the form for short windows.
//   producer warp : TMA Q_i once; K_u, V_u in rings of kQ stages over the key
//                   tiles that any query tile sees (sinks, then the window); the
//                   gate at the end, into the K ring
//   two MMA warps : for each of them, where query tile i sees it, one S_i = Q_i K^T,
//                   the other O_i += P_i V (waits and issues of one warp alone took
//                   longer than the products)
//   kQ x 4 softmax warps (thread = query row): the score row in registers, masked
//                   where some row of the query tile sees the key tile in part;
//                   row max, lazy rescaling of O in TMEM (where a max passes the
//                   reference by more than 2^16), exponentials, P to TMEM in two
//                   halves, each handed on at once; at the end 1/l, gate, lse and
//                   the TMA store.
// Registers: a softmax thread holds 128 scores, more than the 168 registers of
// an even share, so the other warps give some of theirs up.
// TMEM, two query tiles: one S buffer for both in turn (a warpgroup takes its
// scores to registers at once, so the next product need not wait for its
// exponentials), P_0, P_1 of 64 columns, O_0, O_1: 512 in all.  (With P over S a
// step of both tiles took 3010 cycles, its four products take 2048; 16384 x 16
// rows, window 4096: 477 against 452 us, 32768 x 32 under the power cap 2240
// against 2095 us.)  One query tile: S with P over its first half, and O, 256
// columns.
//
// The products (4 * 128 flops per pair and head) fill a little over half of the
// time: 8192 rows, 32 heads on 8, window 4096: 351 k of a launch's 670 k cycles, tensor
// pipe 58% active.  The softmax warps are longer at a step of two tiles than its
// products (about 3350 cycles against 2048, in a trace of an earlier form), and some
// seven CTAs follow one another on an SM, each with its start and end in the open.
// In a long run the power cap takes the clock down as well.  32768 rows, 32 heads on 8,
// window 4096: 1794 us for single calls (1.15 PFLOP/s), 2090 us in a run of 2 s (at 1 kW,
// 986 TFLOP/s).
#include <cuda.h>

#include "f32x2.cuh"
#include "sana_internal.h"
#include "tc_warp.cuh"
#include "window.cuh"

namespace sana {
namespace {

constexpr int kD = 128;
constexpr int kRows = kWinTile;
constexpr int kHalf = kRows * 64 * 2;  // 16 KB: 64 columns of a tile
constexpr int kTileB = 2 * kHalf;      // 32 KB
// Shape of a CTA with kQ query tiles: 4 kQ softmax warps, producer, two MMA warps, an
// idle one; kQ stages of K and V.  Registers a thread: the softmax warps take more
// than an even share from the others (3 - kQ CTAs on an SM).
template <int kQ>
struct Form {
  static constexpr int kThreads = 128 * kQ + 128;
  static constexpr int kWarpProd = 4 * kQ, kWarpS = 4 * kQ + 1, kWarpPv = 4 * kQ + 2;
  static constexpr int kStages = kQ;
  static constexpr int kLaunchRegs = kQ == 2 ? 168 : 128;
  static constexpr int kRegsSoftmax = kQ == 2 ? 216 : 208, kRegsOther = kQ == 2 ? 72 : 48;
  static_assert(128 * kQ * kRegsSoftmax + 128 * kRegsOther <= kThreads * kLaunchRegs, "more registers than at launch");
  static constexpr int kTmemCols = 256 * kQ;
  static constexpr size_t kSmem = 1024 + 3 * kQ * (size_t)kTileB;
};
constexpr float kRescaleLog2 = 16.f;
// Query tiles that see at most this many key tiles run one to a CTA, and so does a
// call whose tiles have an SM each.  One against two to a CTA, 16384 rows, 4 sinks:
//   16 heads on 16: window 256 (5 tiles) 104 against 120 us, 512 (7) 142 against 154,
//     1024 (11) 205 against 208, 2048 (19) 310 against 301
//   16 heads on 4 (pairs of heads): 102 against 106, 131 against 131, 190 against
//     182, 301 against 282
//   32 heads on 8, gate: 242 against 233, 310 against 283, 418 against 383
// no window, 4 heads on 1: 4096 rows (128 tiles) 66 against 70 us, 6000 (188) 98
// against 96.
constexpr int kSingleReach = 10, kSingleReachByHead = 6;
// Of every 8 pairs of exponentials, on the FMA pipe.  Under the power cap, 32768 rows,
// 32 heads on 8, window 4096: none 2110 us, one 2090, two 2097 us; 18720 rows, 16 heads,
// blocks of 4680, gate: 1437, 1433, 1462 us.
constexpr int kEmuPairs = 1;
constexpr float kLn2 = 0.6931471805599453f;

template <int kQ>
struct WinCtl {
  uint64_t q_full, g_full;
  uint64_t k_full[kQ], k_empty[kQ];
  uint64_t v_full[kQ], v_empty[kQ];
  uint64_t s_full[kQ], p_full[kQ][2], pv_done[kQ];  // p_full[tile][half of the keys]
  uint64_t s_taken;  // two tiles: the scores last made are in registers
  uint64_t ysync[kQ];
  uint32_t tmem;
  int abort_flag;
};

// The key tiles of a CTA: those that any of its query tiles sees, sinks first.
template <int kQ>
struct CtaSpan {
  TileSpan s[kQ];
  int ns, w0, n;
  __device__ __forceinline__ int tile(int u) const { return u < ns ? u : w0 + (u - ns); }
  __device__ __forceinline__ bool active(int i, int u) const { return u < n && s[i].has(tile(u)); }
};
template <int kQ>
__device__ __forceinline__ CtaSpan<kQ> cta_span(const WindowDev& w, int row0, int row_step, int len) {
  CtaSpan<kQ> p;
  int last = -1;
  p.w0 = 0x7fffffff;
  p.ns = 0;
#pragma unroll
  for (int i = 0; i < kQ; ++i) {
    const int a = row0 + i * row_step, b = min(a + kRows, w.N) - 1;
    p.s[i] = window_span(w, w.off + a, w.off + b, len);
    if (p.s[i].w1 >= p.s[i].w0) {
      p.w0 = min(p.w0, p.s[i].w0);
      last = max(last, p.s[i].w1);
      p.ns = max(p.ns, p.s[i].ns);
    }
  }
  p.ns = min(p.ns, p.w0);
  p.n = last < 0 ? 0 : p.ns + last - p.w0 + 1;
  return p;
}

template <int kQ, bool kGate>
__global__ void __launch_bounds__(Form<kQ>::kThreads, 3 - kQ)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_g,
                      const __grid_constant__ CUtensorMap tm_y, const WindowDev w, int by_head, float sl,
                      float* __restrict__ lse, int* status) {
  using F = Form<kQ>;
  constexpr int kStages = F::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ WinCtl<kQ> ctl;
  uint8_t* smem = align1024(smem_raw);
  uint8_t* q_s = smem;                    // Q_i (later: Y staging)
  uint8_t* k_s = q_s + kQ * kTileB;       // K ring (later: gate tiles)
  uint8_t* v_s = k_s + kStages * kTileB;  // V ring

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the last query tiles see the most keys where the window is open: they start first
  const int qp = gridDim.x - 1 - blockIdx.x, b = blockIdx.z;
  // query tile i: head h0 + i * head_step, rows from row0 + i * row_step on
  const int head_step = kQ == 2 && by_head, row_step = head_step ? 0 : kRows;
  const int h0 = blockIdx.y * (1 + head_step);
  const int hk = h0 / (w.heads / w.kv_heads);
  const int row0 = qp * (head_step ? kRows : kQ * kRows);
  const int len = window_length(w, b);
  const CtaSpan<kQ> span = cta_span<kQ>(w, row0, row_step, len);
  const WaitCtx wc{&ctl.abort_flag, status};

  auto load_tile = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int head, int row) {
    tma_load_3d(dst, map, bar, head * kD, row, b);
    tma_load_3d(dst + kHalf, map, bar, head * kD + 64, row, b);
  };
  auto load_k = [&](int u) {
    const int st = u % kStages;
    mbar_arrive_expect_tx(&ctl.k_full[st], kTileB);
    load_tile(k_s + st * kTileB, &tm_k, &ctl.k_full[st], hk, span.tile(u) * kRows);
  };
  auto load_v = [&](int u) {
    const int st = u % kStages;
    mbar_arrive_expect_tx(&ctl.v_full[st], kTileB);
    load_tile(v_s + st * kTileB, &tm_v, &ctl.v_full[st], hk, span.tile(u) * kRows);
  };
  if (warp == F::kWarpProd && lane == 0) {
    mbar_init(&ctl.q_full, 1);
    mbar_init(&ctl.g_full, 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&ctl.k_full[i], 1);
      mbar_init(&ctl.k_empty[i], 1);
      mbar_init(&ctl.v_full[i], 1);
      mbar_init(&ctl.v_empty[i], 1);
    }
    for (int i = 0; i < kQ; ++i) {
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.p_full[i][0], 128);
      mbar_init(&ctl.p_full[i][1], 128);
      mbar_init(&ctl.pv_done[i], 1);
      mbar_init(&ctl.ysync[i], 128);
    }
    mbar_init(&ctl.s_taken, 128);
    ctl.abort_flag = 0;
    mbar_fence_init();
    if (span.n > 0) {  // the first loads run while the rest of the CTA sets up
      mbar_arrive_expect_tx(&ctl.q_full, kQ * kTileB);
      for (int i = 0; i < kQ; ++i)  // a tile past N reads as zeros
        load_tile(q_s + i * kTileB, &tm_q, &ctl.q_full, h0 + i * head_step, row0 + i * row_step);
      for (int u = 0; u < min(span.n, kStages); ++u) {
        load_k(u);
        load_v(u);
      }
    }
  }
  if (warp == F::kWarpS) {
    tmem_alloc(&ctl.tmem, F::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  const uint32_t t_s = tmem, t_p = kQ == 2 ? tmem + 128 : tmem, t_o = tmem + kQ * 128;  // P_i 64, O_i 128 columns on

  if (warp >= F::kWarpProd) {
    warpgroup_regs_dec<F::kRegsOther>();
    if (warp == F::kWarpProd) {
      // ------------------------------------------------ TMA producer
      if (lane == 0 && span.n > 0) {
        int nk = min(span.n, kStages), nv = nk;  // loads so far
        bool ok = true;
        for (int u = kStages; u < span.n; ++u) {
          if (!mbar_wait(&ctl.k_empty[u % kStages], ((u / kStages) - 1) & 1, wc, 0x91)) {
            ok = false;
            break;
          }
          load_k(u);
          ++nk;
          if (!mbar_wait(&ctl.v_empty[u % kStages], ((u / kStages) - 1) & 1, wc, 0x92)) {
            ok = false;
            break;
          }
          load_v(u);
          ++nv;
        }
        // the gate goes into the K ring once the last S products have read it
        if (ok && kGate) {
          for (int u = max(span.n - kStages, 0); u < span.n && ok; ++u)
            ok = mbar_wait(&ctl.k_empty[u % kStages], (u / kStages) & 1, wc, 0x9c);
          if (ok) {
            mbar_arrive_expect_tx(&ctl.g_full, kQ * kTileB);
            for (int i = 0; i < kQ; ++i) load_tile(k_s + i * kTileB, &tm_g, &ctl.g_full, h0 + i * head_step, row0 + i * row_step);
          }
        }
        if (*wc.abort_flag) {  // loads still in flight land before the CTA exits
          mbar_drain(&ctl.q_full, 0);
          for (int u = max(nk - kStages, 0); u < nk; ++u) mbar_drain(&ctl.k_full[u % kStages], (u / kStages) & 1);
          for (int u = max(nv - kStages, 0); u < nv; ++u) mbar_drain(&ctl.v_full[u % kStages], (u / kStages) & 1);
          if (ok && kGate) mbar_drain(&ctl.g_full, 0);
        }
      }
    } else if (warp == F::kWarpS) {
      // ------------------------------------------------ S products
      if (span.n > 0) {  // the whole warp, its elected lane issues
        const uint32_t lead = elect_lead();
        const uint32_t idesc_s = idesc_bf16_f32(128, 0, 0, 0);  // Q K^T, both K-major; N by the tile's width
        const uint64_t dq0 = smem_desc_sw128(smem_u32(q_s), 16, 1024);
        const uint64_t dk0 = smem_desc_sw128(smem_u32(k_s), 16, 1024);
        int made = 0, mine[kQ] = {};  // S products issued, in all and for each query tile
        bool ok = mbar_wait(&ctl.q_full, 0, wc, 0x93);
        for (int u = 0; ok && u < span.n; ++u) {
          if (!mbar_wait(&ctl.k_full[u % kStages], (u / kStages) & 1, wc, 0x96)) break;
#pragma unroll
          for (int i = 0; i < kQ; ++i) {
            if (!ok || !span.active(i, u)) continue;
            // S may be overwritten: it is in registers (two tiles), or the product
            // that reads P from it has finished
            if (kQ == 2) ok = made == 0 || mbar_wait(&ctl.s_taken, (made - 1) & 1, wc, 0x97);
            else ok = mine[i] == 0 || mbar_wait(&ctl.pv_done[i], (mine[i] - 1) & 1, wc, 0x97);
            if (!ok) continue;
            tc_fence_after();
            const uint32_t idesc = idesc_s | (uint32_t)(span.s[i].width(span.tile(u), w.sinks) >> 3) << 17;
            const uint64_t a = desc_local(desc_advance(dq0, i * kTileB));
            const uint64_t bk = desc_local(desc_advance(dk0, (u % kStages) * kTileB));
#pragma unroll
            for (int kk = 0; kk < kD / 16; ++kk) {
              const uint32_t o = (kk >> 2) * kHalf + (kk & 3) * 32;
              umma_ss_lead(lead, t_s, desc_advance(a, o), desc_advance(bk, o), idesc, kk != 0);
            }
            umma_commit_lead(lead, &ctl.s_full[i]);
            ++made;
            ++mine[i];
          }
          if (ok) umma_commit_lead(lead, &ctl.k_empty[u % kStages]);
        }
      }
    } else if (warp == F::kWarpPv) {
      // ------------------------------------------------ O += P V products
      if (span.n > 0) {
        const uint32_t lead = elect_lead();
        const uint32_t idesc_o = idesc_bf16_f32(128, 128, 0, 1);  // P (TMEM) V, V MN-major
        const uint64_t dv0 = smem_desc_sw128(smem_u32(v_s), kHalf, 1024);
        int done[kQ] = {};
        bool ok = true;
        for (int u = 0; ok && u < span.n; ++u) {
          if (!mbar_wait(&ctl.v_full[u % kStages], (u / kStages) & 1, wc, 0x95)) break;
          const int key0 = span.tile(u) * kRows;
          if (len < w.N_keys && key0 + kRows > len) {
            // Padding rows of V meet P = 0: they are zeroed, whatever they hold, by this
            // warp, the one that follows v_full phase by phase (the softmax warps skip
            // tiles that their query tile does not see).
            uint8_t* vt = v_s + (u % kStages) * kTileB;
            for (int r = len - key0 + (lane >> 4); r < kRows; r += 2)
              *reinterpret_cast<uint4*>(vt + (lane >> 3 & 1) * kHalf + sw128_off(r, lane & 7)) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < kQ; ++i) {
            if (!ok || !span.active(i, u)) continue;
            const int steps = span.s[i].width(span.tile(u), w.sinks) / 16;
            // half by half as P_i comes (O_i has been rescaled if needed)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              ok = ok && mbar_wait(&ctl.p_full[i][half], done[i] & 1, wc, 0x94);
              if (!ok) continue;
              tc_fence_after();
              const uint64_t bv = desc_local(desc_advance(dv0, (u % kStages) * kTileB + half * 8192));
              const uint32_t ap = t_p + i * 64 + half * 32;
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                if (half * 4 + kk < steps)
                  umma_ts_lead(lead, t_o + i * 128, ap + kk * 8, desc_advance(bv, kk * 2048), idesc_o,
                               (done[i] | half | kk) != 0);
            }
            if (!ok) continue;
            umma_commit_lead(lead, &ctl.pv_done[i]);
            ++done[i];
          }
          if (ok) umma_commit_lead(lead, &ctl.v_empty[u % kStages]);
        }
      }
    }
  } else {
    // ------------------------------------------------ softmax warps: thread = query row
    warpgroup_regs_inc<F::kRegsSoftmax>();
    const int qi = kQ == 1 ? 0 : warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tmem_s = t_s + lane_base, tmem_p = t_p + qi * 64 + lane_base, tmem_o = t_o + qi * 128 + lane_base;
    const int h = h0 + qi * head_step, tile0 = row0 + qi * row_step, row = tile0 + r;
    const int pos = w.off + row;
    const bool row_live = row < w.N && pos < len;
    // this row's limits, and those of the tile's first and last live rows
    const int end = min(window_end(w, pos), len), low = window_low(w, window_end(w, pos));
    const int pos0 = w.off + tile0;
    const int pos1 = min(min(pos0 + kRows, w.off + w.N), len) - 1;
    const int all_end = min(window_end(w, pos0), len);       // every live row sees below it
    const int all_low = window_low(w, window_end(w, max(pos1, 0)));  // every live row sees from it on
    const uint64_t sl2 = pk2(sl, sl);
    float m = -INFINITY, l = 0.f;  // row max reference and sum, base 2
    bool ok = true;
    int done = 0;
    for (int u = 0; ok && u < span.n; ++u) {
      if (!span.active(qi, u)) continue;
      const int key0 = span.tile(u) * kRows;
      const int chunks = span.s[qi].width(span.tile(u), w.sinks) / 32;  // of 32 columns
      if (!__all_sync(0xffffffffu, mbar_wait(&ctl.s_full[qi], done & 1, wc, 0x98))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool masked = key0 + kRows > all_end || (key0 < all_low && key0 + kRows > w.sinks);
      uint32_t sc[4][32];  // the whole row
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < chunks) tmem_ld32(tmem_s + c * 32, sc[c]);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_tie(sc[c]);
      if (kQ == 2) {
        tc_fence_before();
        mbar_arrive(&ctl.s_taken);
      }
      auto chunk_max = [&](const uint32_t (&x)[32]) {  // two chains of 3-input max
        float t = max3_nan(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
        float t2 = max3_nan(__uint_as_float(x[3]), __uint_as_float(x[4]), __uint_as_float(x[5]));
#pragma unroll
        for (int i = 6; i < 30; i += 4) {
          t = max3_nan(t, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
          t2 = max3_nan(t2, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
        }
        return max_nan(max3_nan(t, __uint_as_float(x[30]), __uint_as_float(x[31])), t2);
      };
      if (masked) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t vis = visible_bits(key0 + 32 * c, low, end, w.sinks);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(vis & (1u << i))) sc[c][i] = __float_as_uint(-INFINITY);
        }
      }
      float top = -INFINITY;
      if (chunks == 4) {
        top = max3_nan(max_nan(chunk_max(sc[0]), chunk_max(sc[1])), chunk_max(sc[2]), chunk_max(sc[3]));
      } else {
#pragma unroll
        for (int c = 0; c < 3; ++c)
          if (c < chunks) top = max_nan(top, chunk_max(sc[c]));
      }
      top *= sl;
      // The reference moves where the row's max passes it, on its first key or
      // by more than 2^16.  It is rounded up to an integer: rescaling is then exact.
      // A row that has seen no key yet keeps -inf and works against 0: its terms are
      // 2^-inf (or 2^-126, dropped by the factor 0 when its first key comes).
      const bool grow = top > m + kRescaleLog2;
      if (__any_sync(0xffffffffu, grow)) {
        const float m_next = grow ? ceilf(top) : m;
        const float corr = grow ? ex2(m - m_next) : 1.f;
        m = m_next;
        l *= corr;
        if (done >= 1) {
          // O_i holds the sum over the tiles before this one (warp-uniform:
          // TMEM access is warp-collective)
          if (!__all_sync(0xffffffffu, mbar_wait(&ctl.pv_done[qi], (done - 1) & 1, wc, 0x99))) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            tmem_ld16(tmem_o + c * 16, o);
            tmem_ld_wait();
            tmem_tie(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
            tmem_st16(tmem_o + c * 16, o);
          }
        }
      }
      const float m_use = m == -INFINITY ? 0.f : m;
      const uint64_t neg_m = pk2(-m_use, -m_use);
      uint64_t rs2 = pk2(0.f, 0.f);
      if (kQ == 2 && done >= 1) {  // P of the tile before has been read
        if (!__all_sync(0xffffffffu, mbar_wait(&ctl.pv_done[qi], (done - 1) & 1, wc, 0x90))) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c < chunks) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float s0 = __uint_as_float(sc[c][i]), s1 = __uint_as_float(sc[c][i + 1]);
            const uint64_t x = fma2(pk2(s0, s1), sl2, neg_m);
            float p0, p1;
            if (((i >> 1) & 7) >= 8 - kEmuPairs) {
              exp2_pair(x, p0, p1);
            } else {
              up2(x, p0, p1);
              p0 = ex2(p0);
              p1 = ex2(p1);
            }
            rs2 = add2(rs2, pk2(p0, p1));
            pk[i / 2] = f2_to_bf2(p0, p1);
          }
          // (one tile: over S columns that are in registers); after each half of the keys the
          // product with V may start on it
          tmem_st16(tmem_p + c * 16, pk);
        }
        if (c & 1) {
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&ctl.p_full[qi][c >> 1]);
        }
      }
      float rs0, rs1;
      up2(rs2, rs0, rs1);
      // a NaN or +inf score makes its row NaN (the exponentials on the FMA pipe would
      // not show it)
      l = top < INFINITY ? l + (rs0 + rs1) : NAN;
      ++done;
    }
    // ---------------- epilogue
    const bool any = span.s[qi].count() > 0;
    ok = __all_sync(0xffffffffu, ok && (!any || (done > 0 && mbar_wait(&ctl.pv_done[qi], (done - 1) & 1, wc, 0x9a))));
    // Q_i becomes the output's staging: its load has landed before the first S,
    // and where this tile had none, it is waited for here
    if (!any && span.n > 0) ok = ok && __all_sync(0xffffffffu, mbar_wait(&ctl.q_full, 0, wc, 0x9f));
    if (kGate && span.n > 0) ok = ok && __all_sync(0xffffffffu, mbar_wait(&ctl.g_full, 0, wc, 0x9e));
    uint8_t* ybuf = q_s + qi * kTileB;  // Q_i is no longer read
    const uint8_t* gbuf = k_s + qi * kTileB;
    if (ok) {
      tc_fence_after();
      // A live row sees itself at least; where all its scores are -inf there is no
      // softmax.  Dead rows get zeros.
      const bool some = row_live;
      if (m == -INFINITY) l = NAN;
      const float inv = some ? 1.f / l : 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (any) {  // else nothing was accumulated for this tile
          tmem_ld32(tmem_o + c * 32, o);
          tmem_ld_wait();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int ch = (c & 1) * 4 + q;
          const uint32_t off = (c >> 1) * kHalf + sw128_off(r, ch);
          uint32_t gw[4] = {0, 0, 0, 0};
          if (kGate && some) {
            const uint4 gr = *reinterpret_cast<const uint4*>(gbuf + off);
            gw[0] = gr.x; gw[1] = gr.y; gw[2] = gr.z; gw[3] = gr.w;
          }
          uint32_t out[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float y0 = __uint_as_float(o[q * 8 + 2 * i]) * inv;
            float y1 = __uint_as_float(o[q * 8 + 2 * i + 1]) * inv;
            if (kGate) {
              const float2 gg = bf2_to_f2(gw[i]);
              y0 *= sigmoid_fast(gg.x);
              y1 *= sigmoid_fast(gg.y);
            }
            out[i] = some ? f2_to_bf2(y0, y1) : 0u;
          }
          *reinterpret_cast<uint4*>(ybuf + off) = make_uint4(out[0], out[1], out[2], out[3]);
        }
      }
      if (lse && row < w.N)
        lse[((size_t)b * w.heads + h) * w.N + row] = some ? (m + log2f(l)) * kLn2 : -INFINITY;
      fence_proxy_async_smem();
    }
    mbar_arrive(&ctl.ysync[qi]);
    ok = mbar_wait(&ctl.ysync[qi], 0, wc, 0x9b) && ok;
    if (ok && r == 0 && tile0 < w.N) {  // a tile past N has nothing to store
      tma_store_3d(&tm_y, ybuf, h * kD, tile0, b);
      tma_store_3d(&tm_y, ybuf + kHalf, h * kD + 64, tile0, b);
      bulk_commit();
      bulk_wait_read0();  // the staging may go; the grid's end makes the rows visible
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == F::kWarpS) {
    if (*wc.abort_flag) {  // MMAs in flight finish before TMEM is freed
      for (int i = 0; i < kQ; ++i) {
        const int n = span.s[i].count();
        if (n) mbar_drain(&ctl.pv_done[i], (n - 1) & 1);
      }
    }
    tc_fence_after();
    tmem_dealloc(tmem, F::kTmemCols);
  }
}

// Two query heads of one key head make the better pair: both tiles see the same
// keys (two tiles of rows leave each other idle at one end of the window: 16384
// rows, 32 heads on 8, window 2048, 617 against 575 us).
bool pairs_by_head(const WindowDev& w) { return w.heads / w.kv_heads % 2 == 0; }

template <int kQ, bool kGate>
void launch(const CUtensorMap* t, const WindowDev& w, int B, float sl, float* lse, cudaStream_t st) {
  const int by_head = kQ == 2 && pairs_by_head(w);
  const int rows = by_head ? kRows : kQ * kRows;
  const dim3 grid((w.N + rows - 1) / rows, by_head ? w.heads / 2 : w.heads, B);
  window_fwd_kernel<kQ, kGate><<<grid, Form<kQ>::kThreads, Form<kQ>::kSmem, st>>>(t[0], t[1], t[2], t[3], t[4], w,
                                                                                by_head, sl, lse, status_word());
}
template <int kQ, bool kGate>
void allow_smem() {
  cudaFuncSetAttribute(window_fwd_kernel<kQ, kGate>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Form<kQ>::kSmem);
}

}  // namespace

sana_status window_fwd_run(const WindowCall& c, float* lse, void* out, cudaStream_t st) {
  const uint64_t N = c.N, Nk = c.N_keys, C = (uint64_t)c.heads * kD, Ck = (uint64_t)c.kv_heads * kD;
  CUtensorMap t[5];  // q, k, v, gate, out
  bool okm = make_tmap_bf16_3d(&t[0], c.q, C, N, c.B, c.q_stride, N * c.q_stride, kRows) &&
             make_tmap_bf16_3d(&t[1], c.k, Ck, Nk, c.B, c.k_stride, Nk * c.k_stride, kRows) &&
             make_tmap_bf16_3d(&t[2], c.v, Ck, Nk, c.B, c.v_stride, Nk * c.v_stride, kRows) &&
             make_tmap_bf16_3d(&t[4], out, C, N, c.B, C, N * C, kRows);
  if (c.gate) okm = okm && make_tmap_bf16_3d(&t[3], c.gate, C, N, c.B, c.gate_stride, N * c.gate_stride, kRows);
  else t[3] = t[0];
  if (!okm) return fail(SANA_ERR_CUDA, "windowed anchor: cuTensorMapEncodeTiled failed");
  once_per_context(kAttrWindowFwd, [] {
    allow_smem<1, false>();
    allow_smem<1, true>();
    allow_smem<2, false>();
    allow_smem<2, true>();
  });
  const WindowDev w{c.N, c.N_keys, c.N_keys - c.N, c.window, c.sinks, c.block, c.heads, c.kv_heads, c.lengths};
  const float sl = c.scale * 1.4426950408889634f;
  // key tiles that a query tile sees at most
  const long long all = (c.N_keys + kRows - 1) / kRows;
  const long long reach = c.window ? ((long long)c.window + c.block + 2 * kRows - 3) / kRows + 1 +
                                         (c.sinks + kRows - 1) / kRows
                                   : all;
  const bool single = (reach < all ? reach : all) <= (pairs_by_head(w) ? kSingleReachByHead : kSingleReach) ||
                      ((long long)c.N + kRows - 1) / kRows * c.heads * c.B <= kNumSMs;
  if (single && c.gate) launch<1, true>(t, w, c.B, sl, lse, st);
  else if (single) launch<1, false>(t, w, c.B, sl, lse, st);
  else if (c.gate) launch<2, true>(t, w, c.B, sl, lse, st);
  else launch<2, false>(t, w, c.B, sl, lse, st);
  return check_launch("window_fwd_kernel");
}

}  // namespace sana
