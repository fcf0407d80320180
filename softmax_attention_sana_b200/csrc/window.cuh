// What a query of the windowed anchor sees, shared by its kernels.
//
// Query row i stands at position p = off + i of its sequence.  Blocks of
// `block` positions see each other whole (block = 1: causal); e = (p / block +
// 1) * block is the end of p's own block.  Key j is visible iff
//   j < min(e, len)  and  (j >= e - window  or  j < sinks)
// with len the sequence's length (padding behind it sees nothing and is seen
// by nothing) and window = 0 for no limit.
#pragma once

#include "sana_common.cuh"

namespace sana {

constexpr int kWinTile = 128;  // rows of a query tile and of a key tile

struct WindowDev {
  int N, N_keys, off;       // off = N_keys - N
  int window, sinks, block;
  int heads, kv_heads;
  const int* lengths;       // [B] or null
};

__device__ __forceinline__ int window_length(const WindowDev& w, int b) {
  if (!w.lengths) return w.N_keys;
  const int len = __ldg(w.lengths + b);
  return len < 0 ? 0 : len < w.N_keys ? len : w.N_keys;
}
// End of p's block, and the first position of its window (0 when unlimited).
// Positions stay below 2^30 and block <= 2^30 (checked on the host), so e does
// not overflow.
__device__ __forceinline__ int window_end(const WindowDev& w, int p) {
  return w.block == 1 ? p + 1 : (p / w.block + 1) * w.block;
}
__device__ __forceinline__ int window_low(const WindowDev& w, int e) {
  return w.window == 0 || e < w.window ? 0 : e - w.window;
}

// Key tiles that query positions [p0, p1] of a sequence of `len` tokens see:
// [0, ns) (sinks outside the window) and [w0, w1].  No tile: w1 < w0, ns = 0.
struct TileSpan {
  int ns, w0, w1;
  __device__ __forceinline__ bool has(int t) const { return t < ns || (t >= w0 && t <= w1); }
  __device__ __forceinline__ int count() const { return ns + (w1 >= w0 ? w1 - w0 + 1 : 0); }
  // Columns of tile t that some row sees, a multiple of 32: of a tile outside the
  // window only the sinks (a few tokens: the tile then costs a fraction).
  __device__ __forceinline__ int width(int t, int sinks) const {
    return t >= w0 ? kWinTile : min(kWinTile, (sinks - t * kWinTile + 31) & ~31);
  }
};
__device__ __forceinline__ TileSpan window_span(const WindowDev& w, int p0, int p1, int len) {
  TileSpan s{0, 0, -1};
  if (p1 >= len) p1 = len - 1;
  if (p0 > p1) return s;
  const int top = min(window_end(w, p1), len);  // >= 1
  s.w0 = window_low(w, window_end(w, p0)) / kWinTile;
  s.w1 = (top - 1) / kWinTile;
  s.ns = min((min(w.sinks, top) + kWinTile - 1) / kWinTile, s.w0);
  return s;
}

// Bits 0..31: positions below x (x counted from bit 0).
__device__ __forceinline__ uint32_t bits_below(int x) {
  return x <= 0 ? 0u : x >= 32 ? 0xffffffffu : (1u << x) - 1u;
}
// Of 32 consecutive keys from `key` on, those visible to a row with these limits.
__device__ __forceinline__ uint32_t visible_bits(int key, int low, int end, int sinks) {
  return bits_below(end - key) & (~bits_below(low - key) | bits_below(sinks - key));
}

}  // namespace sana
