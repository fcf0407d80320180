// C entry points of the windowed anchor: argument checks and dispatch.
#include <cmath>

#include "sana_internal.h"

namespace sana {
namespace {

constexpr int kHeadDim = 128;
constexpr int kMost = 1 << 30;  // positions, window, sinks, block: sums of two stay in 32 bits

struct Range {
  const void* p;
  size_t bytes;
  unsigned align = 16;
};
bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}
sana_status check_buffers(const char* who, const Range* in, int n_in, const Range* out, int n_out) {
  for (int i = 0; i < n_in + n_out; ++i) {
    const Range& r = i < n_in ? in[i] : out[i - n_in];
    if (reinterpret_cast<uintptr_t>(r.p) % r.align)
      return fail(SANA_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned (lse: 4)", who);
  }
  for (int o = 0; o < n_out; ++o) {
    for (int i = 0; i < n_in; ++i)
      if (overlap(out[o], in[i])) return fail(SANA_ERR_INVALID_ARG, "%s: an output aliases an input", who);
    for (int i = 0; i < o; ++i)
      if (overlap(out[o], out[i])) return fail(SANA_ERR_INVALID_ARG, "%s: outputs alias each other", who);
  }
  return SANA_OK;
}
sana_status check_ws(const char* who, const void* ws, size_t have, size_t need) {
  if (need && (!ws || have < need))
    return fail(SANA_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", who, ws ? have : 0, need);
  if (reinterpret_cast<uintptr_t>(ws) & 255u)
    return fail(SANA_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  return SANA_OK;
}
sana_status check_heads(const char* who, int B, int heads, int kv_heads, int head_dim) {
  if (B < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads != 0)
    return fail(SANA_ERR_INVALID_ARG, "%s: bad shape B=%d heads=%d kv_heads=%d", who, B, heads, kv_heads);
  if (head_dim != kHeadDim) return fail(SANA_ERR_UNSUPPORTED, "%s: head_dim must be 128 (got %d)", who, head_dim);
  if (B > 65535 || heads > 65535)  // grid dimensions
    return fail(SANA_ERR_UNSUPPORTED, "%s: B=%d heads=%d are too many", who, B, heads);
  return SANA_OK;
}

sana_status check_shape(const char* who, const sana_window_shape* s, WindowCall* c) {
  if (!s) return fail(SANA_ERR_INVALID_ARG, "%s: shape is NULL", who);
  if (sana_status e = check_heads(who, s->B, s->heads, s->kv_heads, s->head_dim)) return e;
  if (s->N < 0 || s->N_keys < s->N)
    return fail(SANA_ERR_INVALID_ARG, "%s: the N=%d queries must be the last of N_keys=%d positions", who, s->N, s->N_keys);
  if (s->sinks < 0 || s->block < 1 || s->window < 0 || (s->window && s->window < s->block))
    return fail(SANA_ERR_INVALID_ARG, "%s: bad window=%d sinks=%d block=%d (window 0 or at least block)", who,
                s->window, s->sinks, s->block);
  if (s->N_keys > kMost || s->window > kMost || s->sinks > kMost || s->block > kMost)
    return fail(SANA_ERR_UNSUPPORTED, "%s: N_keys, window, sinks and block go up to 2^30", who);
  if (!std::isfinite(s->scale)) return fail(SANA_ERR_INVALID_ARG, "%s: scale must be finite", who);
  *c = WindowCall{};
  c->B = s->B;
  c->N = s->N;
  c->N_keys = s->N_keys;
  c->heads = s->heads;
  c->kv_heads = s->kv_heads;
  c->window = s->window;
  c->sinks = s->sinks;
  c->block = s->block;
  c->lengths = s->lengths;
  c->scale = s->scale > 0.f ? s->scale : 1.f / sqrtf((float)kHeadDim);
  const long long cq = (long long)s->heads * kHeadDim, ck = (long long)s->kv_heads * kHeadDim;
  const long long given[4] = {s->q_stride, s->k_stride, s->v_stride, s->gate_stride};
  long long* out[4] = {&c->q_stride, &c->k_stride, &c->v_stride, &c->gate_stride};
  for (int i = 0; i < 4; ++i) {
    const long long width = i == 1 || i == 2 ? ck : cq;
    *out[i] = given[i] ? given[i] : width;
    if (*out[i] < width || *out[i] % 8 != 0)
      return fail(SANA_ERR_INVALID_ARG, "%s: token strides must be multiples of 8 and cover a token's heads", who);
    // the tensor maps hold strides below 2^40 bytes
    if (*out[i] > (1LL << 32) || (unsigned long long)*out[i] * 2 * (unsigned long long)s->N_keys >= 1ULL << 40)
      return fail(SANA_ERR_UNSUPPORTED, "%s: a sequence may span 2^40 bytes at most", who);
  }
  if (reinterpret_cast<uintptr_t>(s->lengths) & 3u)
    return fail(SANA_ERR_INVALID_ARG, "%s: lengths must be 4-byte aligned", who);
  return SANA_OK;
}

sana_status check_decode(const char* who, const sana_window_decode_shape* s, DecodeCall* c) {
  if (!s) return fail(SANA_ERR_INVALID_ARG, "%s: shape is NULL", who);
  if (sana_status e = check_heads(who, s->B, s->heads, s->kv_heads, s->head_dim)) return e;
  if (s->N < 0 || s->sinks < 0 || s->window < 0 || s->capacity < 1 || s->capacity - (long long)s->sinks < s->N ||
      s->capacity <= s->sinks)
    return fail(SANA_ERR_INVALID_ARG,
                "%s: bad N=%d sinks=%d window=%d capacity=%d (capacity above sinks, at least sinks + N)", who, s->N,
                s->sinks, s->window, s->capacity);
  if (s->capacity > kMost || s->window > kMost || (long long)s->heads / s->kv_heads * s->N > 65535)
    return fail(SANA_ERR_UNSUPPORTED, "%s: capacity and window go up to 2^30, query rows of a key head to 65535", who);
  const long long tiles = ((long long)s->heads / s->kv_heads * s->N + 15) / 16;
  if (s->kv_heads * tiles > 65535) return fail(SANA_ERR_UNSUPPORTED, "%s: too many query rows", who);
  // the tensor maps hold strides below 2^40 bytes
  if ((unsigned long long)s->capacity * s->kv_heads * kHeadDim * 2 >= 1ULL << 40)
    return fail(SANA_ERR_UNSUPPORTED, "%s: a cache may span 2^40 bytes at most", who);
  if (!std::isfinite(s->scale)) return fail(SANA_ERR_INVALID_ARG, "%s: scale must be finite", who);
  *c = DecodeCall{s->B, s->N, s->heads, s->kv_heads, s->capacity, s->window, s->sinks,
                  s->scale > 0.f ? s->scale : 1.f / sqrtf((float)kHeadDim)};
  return SANA_OK;
}

size_t span(long long tokens, long long stride, int heads) {
  return tokens > 0 ? ((size_t)(tokens - 1) * stride + (size_t)heads * kHeadDim) * 2 : 0;
}

}  // namespace
}  // namespace sana

using namespace sana;

extern "C" {

sana_status sana_window_anchor_fwd(const sana_window_shape* s, const void* q, const void* k,
                                   const void* v, const void* g, void* out, float* lse,
                                   sana_stream_t stream) {
  const char* who = "sana_window_anchor_fwd";
  WindowCall c;
  if (sana_status e = check_shape(who, s, &c)) return e;
  if (c.B == 0 || c.N == 0) return SANA_OK;
  if (!q || !k || !v || !out) return fail(SANA_ERR_INVALID_ARG, "%s: NULL tensor pointer", who);
  const long long tq = (long long)c.B * c.N, tk = (long long)c.B * c.N_keys;
  const Range in[] = {{q, span(tq, c.q_stride, c.heads)}, {k, span(tk, c.k_stride, c.kv_heads)},
                      {v, span(tk, c.v_stride, c.kv_heads)}, {g, span(tq, c.gate_stride, c.heads)}};
  const Range outs[] = {{out, (size_t)tq * c.heads * kHeadDim * 2}, {lse, (size_t)tq * c.heads * 4, 4}};
  if (sana_status e = check_buffers(who, in, 4, outs, 2)) return e;
  if (overlap({c.lengths, (size_t)c.B * 4}, outs[0]) || overlap({c.lengths, (size_t)c.B * 4}, outs[1]))
    return fail(SANA_ERR_INVALID_ARG, "%s: an output aliases the lengths", who);
  c.q = q;
  c.k = k;
  c.v = v;
  c.gate = g;
  return window_fwd_run(c, lse, out, stream);
}

size_t sana_window_anchor_bwd_workspace_size(const sana_window_shape* s, int gated) {
  WindowCall c;
  if (check_shape("sana_window_anchor_bwd_workspace_size", s, &c) != SANA_OK || c.B == 0 || c.N == 0) return 0;
  c.gate = gated ? s : nullptr;  // only whether there is one counts here
  return window_bwd_ws_bytes(c);
}

sana_status sana_window_anchor_bwd(const sana_window_shape* s, const void* q, const void* k,
                                   const void* v, const void* g, const void* out, const float* lse,
                                   const void* dy, void* dq, void* dk, void* dv, void* dg, void* ws,
                                   size_t ws_bytes, sana_stream_t stream) {
  const char* who = "sana_window_anchor_bwd";
  WindowCall c;
  if (sana_status e = check_shape(who, s, &c)) return e;
  if (!g != !dg) return fail(SANA_ERR_INVALID_ARG, "%s: gate_logits and d_gate go together", who);
  if (c.B == 0 || c.N_keys == 0) return SANA_OK;
  if (c.N == 0)
    return fail(SANA_ERR_UNSUPPORTED, "%s: keys without queries have no backward (their gradient is zero)", who);
  if (!q || !k || !v || !out || !lse || !dy || !dq || !dk || !dv)
    return fail(SANA_ERR_INVALID_ARG, "%s: NULL tensor pointer", who);
  const long long tq = (long long)c.B * c.N, tk = (long long)c.B * c.N_keys;
  const size_t nq = (size_t)tq * c.heads * kHeadDim * 2, nk = (size_t)tk * c.kv_heads * kHeadDim * 2;
  c.q = q;
  c.k = k;
  c.v = v;
  c.gate = g;
  const size_t need = window_bwd_ws_bytes(c);
  const Range in[] = {{q, span(tq, c.q_stride, c.heads)}, {k, span(tk, c.k_stride, c.kv_heads)},
                      {v, span(tk, c.v_stride, c.kv_heads)}, {g, span(tq, c.gate_stride, c.heads)},
                      {out, nq}, {lse, (size_t)tq * c.heads * 4, 4}, {dy, nq}};
  const Range outs[] = {{dq, nq}, {dk, nk}, {dv, nk}, {dg, nq}, {ws, need}};
  if (sana_status e = check_buffers(who, in, 7, outs, 5)) return e;
  for (const Range& o : outs)
    if (overlap({c.lengths, (size_t)c.B * 4}, o))
      return fail(SANA_ERR_INVALID_ARG, "%s: an output aliases the lengths", who);
  if (sana_status e = check_ws(who, ws, ws_bytes, need)) return e;
  return window_bwd_run(c, out, lse, dy, dq, dk, dv, dg, ws, stream);
}

size_t sana_window_anchor_decode_workspace_size(const sana_window_decode_shape* s) {
  DecodeCall c;
  if (check_decode("sana_window_anchor_decode_workspace_size", s, &c) != SANA_OK || c.B == 0 || c.N == 0) return 0;
  return window_decode_ws_bytes(c);
}

sana_status sana_window_anchor_decode(const sana_window_decode_shape* s, const void* q,
                                      const void* k_new, const void* v_new, const void* g,
                                      void* k_cache, void* v_cache, const int* lengths, void* out,
                                      void* ws, size_t ws_bytes, sana_stream_t stream) {
  const char* who = "sana_window_anchor_decode";
  DecodeCall c;
  if (sana_status e = check_decode(who, s, &c)) return e;
  if (c.B == 0 || c.N == 0) return SANA_OK;
  if (!q || !k_new || !v_new || !k_cache || !v_cache || !lengths || !out)
    return fail(SANA_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (reinterpret_cast<uintptr_t>(lengths) & 3u)
    return fail(SANA_ERR_INVALID_ARG, "%s: lengths must be 4-byte aligned", who);
  const size_t row = (size_t)kHeadDim * 2, nq = (size_t)c.B * c.N * c.heads * row;
  const size_t nk = (size_t)c.B * c.N * c.kv_heads * row, nc = (size_t)c.B * c.capacity * c.kv_heads * row;
  const size_t need = window_decode_ws_bytes(c);
  const Range in[] = {{q, nq}, {k_new, nk}, {v_new, nk}, {g, nq}};
  const Range outs[] = {{out, nq}, {k_cache, nc}, {v_cache, nc}, {ws, need}};
  if (sana_status e = check_buffers(who, in, 4, outs, 4)) return e;
  for (const Range& o : outs)
    if (overlap({lengths, (size_t)c.B * 4}, o))
      return fail(SANA_ERR_INVALID_ARG, "%s: an output aliases the lengths", who);
  if (sana_status e = check_ws(who, ws, ws_bytes, need)) return e;
  return window_decode_run(c, q, k_new, v_new, g, k_cache, v_cache, lengths, out, ws, stream);
}

}  // extern "C"
