// C entry points of the rotary and query/key norm operators: argument checks,
// the rotary frequencies, dispatch.
#include <cmath>

#include "sana_internal.h"

namespace sana {
namespace {

constexpr double kPi = 3.14159265358979323846;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Byte ranges of the tensors of one call, for the aliasing check.
struct Range {
  const void* p;
  size_t bytes;
};
bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

// Checks shape and positions, and fills in what the kernels need of them.
sana_status check_call(const char* who, const sana_qk_shape* s, sana_dtype dt,
                       const sana_qk_positions* at, QkTensors* a, RotaryDev* rt) {
  if (!s || !at) return fail(SANA_ERR_INVALID_ARG, "%s: shape or positions is NULL", who);
  if (dt != SANA_F32 && dt != SANA_BF16)
    return fail(SANA_ERR_INVALID_ARG, "%s: bad dtype %d", who, (int)dt);
  if (s->B < 0 || s->N < 0 || s->heads < 1 || s->kv_heads < 0 || s->heads > 65536 ||
      s->kv_heads > 65536)
    return fail(SANA_ERR_INVALID_ARG, "%s: bad shape B=%d N=%d heads=%d kv_heads=%d", who, s->B,
                s->N, s->heads, s->kv_heads);
  const int D = s->head_dim;
  if (D != 16 && D != 32 && D != 64 && D != 128 && D != 256)
    return fail(SANA_ERR_UNSUPPORTED, "%s: head_dim must be 16/32/64/128/256 (got %d)", who, D);
  const long long tokens = (long long)s->B * s->N;
  if (tokens >= 1LL << 31)
    return fail(SANA_ERR_UNSUPPORTED, "%s: %lld tokens are too many", who, tokens);
  *a = QkTensors{};
  a->B = s->B;
  a->N = s->N;
  a->heads = s->heads;
  a->kv_heads = s->kv_heads;
  a->head_dim = D;
  a->q_stride = s->q_stride ? s->q_stride : (long long)s->heads * D;
  a->k_stride = s->k_stride ? s->k_stride : (long long)s->kv_heads * D;
  if (a->q_stride < (long long)s->heads * D || a->k_stride < (long long)s->kv_heads * D ||
      a->q_stride % 8 != 0 || a->k_stride % 8 != 0)
    return fail(SANA_ERR_INVALID_ARG,
                "%s: token strides must be multiples of 8 and cover a token's heads (q %lld, k %lld)",
                who, s->q_stride, s->k_stride);
  if (!at->rotary == !at->rope)
    return fail(SANA_ERR_INVALID_ARG, "%s: exactly one of rotary and rope must be given", who);
  *rt = RotaryDev{};
  rt->positions = at->positions;
  rt->offset = at->offset;
  rt->N = s->N;
  if (const sana_rotary* r = at->rotary) {
    if (!r->table || !aligned16(r->table) || r->max_positions < 1 ||
        (r->layout != SANA_ROTARY_INTERLEAVED && r->layout != SANA_ROTARY_HALF))
      return fail(SANA_ERR_INVALID_ARG, "%s: bad rotary table", who);
    if (r->rotary_dim < 16 || r->rotary_dim % 16 != 0 || r->rotary_dim > D)
      return fail(SANA_ERR_UNSUPPORTED,
                  "%s: rotary_dim must be a multiple of 16 up to head_dim (got %d of %d)", who,
                  r->rotary_dim, D);
    if (at->positions && (reinterpret_cast<uintptr_t>(at->positions) & 3u))
      return fail(SANA_ERR_INVALID_ARG, "%s: positions must be 4-byte aligned", who);
    if (!at->positions && (at->offset < 0 || (long long)at->offset + s->N > r->max_positions))
      return fail(SANA_ERR_INVALID_ARG, "%s: positions [%d, %lld) are outside the table of %d", who,
                  at->offset, (long long)at->offset + s->N, r->max_positions);
    rt->table = r->table;
    rt->pairs = r->rotary_dim / 2;
    rt->max_positions = r->max_positions;
    rt->half = r->layout == SANA_ROTARY_HALF;
  } else {
    const sana_rope* g = at->rope;
    if (at->positions)
      return fail(SANA_ERR_INVALID_ARG, "%s: a grid's tokens have no positions of their own", who);
    if (at->T < 0 || at->H < 1 || at->W < 1 || (long long)at->T * at->H * at->W != s->N)
      return fail(SANA_ERR_INVALID_ARG, "%s: grid %dx%dx%d does not hold N=%d tokens", who, at->T,
                  at->H, at->W, s->N);
    if (g->n_t < 0 || g->n_h < 0 || g->n_w < 0 || g->n_t + g->n_h + g->n_w != D / 2)
      return fail(SANA_ERR_INVALID_ARG, "%s: rope split %d/%d/%d does not cover head_dim/2=%d", who,
                  g->n_t, g->n_h, g->n_w, D / 2);
    if (g->H != at->H || g->W != at->W || at->offset < 0 ||
        g->T_total < (long long)at->offset + at->T)
      return fail(SANA_ERR_INVALID_ARG, "%s: rope tables (T_total=%d, H=%d, W=%d) do not cover the grid",
                  who, g->T_total, g->H, g->W);
    if ((g->n_t && (!g->cos_t || !g->sin_t)) || (g->n_h && (!g->cos_h || !g->sin_h)) ||
        (g->n_w && (!g->cos_w || !g->sin_w)))
      return fail(SANA_ERR_INVALID_ARG, "%s: rope table pointer is NULL", who);
    rt->pairs = D / 2;
    rt->rope = RopeDev{g->cos_t, g->sin_t, g->cos_h, g->sin_h, g->cos_w, g->sin_w, g->n_t, g->n_h, g->n_w};
    rt->grid = GridDev{at->T, at->H, at->W, at->offset, s->N, s->heads};
  }
  return SANA_OK;
}

size_t esize(sana_dtype dt) { return dt == SANA_BF16 ? 2 : 4; }

// Bytes from the first to the last element of a strided (or contiguous) tensor.
size_t span(const QkTensors& a, sana_dtype dt, long long stride, int heads) {
  const size_t tokens = (size_t)a.B * a.N;
  return tokens && heads ? ((tokens - 1) * stride + (size_t)heads * a.head_dim) * esize(dt) : 0;
}

sana_status check_buffers(const char* who, const Range* in, int n_in, const Range* out, int n_out) {
  for (int i = 0; i < n_in + n_out; ++i)
    if (!aligned16(i < n_in ? in[i].p : out[i - n_in].p))
      return fail(SANA_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  for (int o = 0; o < n_out; ++o) {
    for (int i = 0; i < n_in; ++i)
      if (overlap(out[o], in[i])) return fail(SANA_ERR_INVALID_ARG, "%s: an output aliases an input", who);
    for (int i = 0; i < o; ++i)
      if (overlap(out[o], out[i])) return fail(SANA_ERR_INVALID_ARG, "%s: outputs alias each other", who);
  }
  return SANA_OK;
}

sana_status forward(const char* who, const sana_qk_shape* s, sana_dtype dt,
                    const sana_qk_positions* at, bool norm, int inverse, const void* q,
                    const void* k, const float* wq, const float* wk, float eps, float q_mul,
                    void* q_out, void* k_out, cudaStream_t st) {
  QkTensors a;
  RotaryDev rt;
  if (sana_status e = check_call(who, s, dt, at, &a, &rt)) return e;
  if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(q_mul))
    return fail(SANA_ERR_INVALID_ARG, "%s: eps must be finite and >= 0, q_mul finite", who);
  if ((size_t)a.B * a.N == 0) return SANA_OK;
  if (!q || !q_out || (a.kv_heads && (!k || !k_out)))
    return fail(SANA_ERR_INVALID_ARG, "%s: NULL tensor pointer", who);
  if (!a.kv_heads && (k || k_out))
    return fail(SANA_ERR_INVALID_ARG, "%s: keys given with kv_heads == 0", who);
  const Range in[] = {{q, span(a, dt, a.q_stride, a.heads)},
                      {k, span(a, dt, a.k_stride, a.kv_heads)},
                      {wq, (size_t)a.head_dim * 4},
                      {wk, (size_t)a.head_dim * 4},
                      {rt.table, (size_t)rt.max_positions * rt.pairs * 8}};
  const Range out[] = {{q_out, span(a, dt, (long long)a.heads * a.head_dim, a.heads)},
                       {k_out, span(a, dt, (long long)a.kv_heads * a.head_dim, a.kv_heads)}};
  if (sana_status e = check_buffers(who, in, 5, out, 2)) return e;
  if (overlap({rt.positions, (size_t)a.B * a.N * 4}, out[0]) ||
      overlap({rt.positions, (size_t)a.B * a.N * 4}, out[1]))
    return fail(SANA_ERR_INVALID_ARG, "%s: an output aliases the positions", who);
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.wq = wq;
  a.wk = wk;
  rt.inverse = inverse != 0;
  return qk_norm_rope_run(a, dt, rt, norm, eps, q_mul, st);
}

}  // namespace
}  // namespace sana

using namespace sana;

extern "C" {

sana_status sana_rotary_table(int max_positions, int rotary_dim, double theta,
                              const sana_rotary_scaling* sc, float* table, sana_stream_t stream) {
  const char* who = "sana_rotary_table";
  if (max_positions < 1) return fail(SANA_ERR_INVALID_ARG, "%s: max_positions=%d", who, max_positions);
  if (rotary_dim < 16 || rotary_dim % 16 != 0 || rotary_dim > 256)
    return fail(SANA_ERR_UNSUPPORTED, "%s: rotary_dim must be a multiple of 16 up to 256 (got %d)",
                who, rotary_dim);
  if (!std::isfinite(theta) || theta <= 1.0)
    return fail(SANA_ERR_INVALID_ARG, "%s: theta must be finite and above 1", who);
  if (!table || !aligned16(table))
    return fail(SANA_ERR_INVALID_ARG, "%s: table must be a 16-byte aligned device pointer", who);
  const int kind = sc ? sc->kind : SANA_ROTARY_PLAIN;
  if (kind < SANA_ROTARY_PLAIN || kind > SANA_ROTARY_YARN)
    return fail(SANA_ERR_INVALID_ARG, "%s: bad scaling kind %d", who, kind);
  if (kind != SANA_ROTARY_PLAIN && (!std::isfinite(sc->factor) || sc->factor < 1.0))
    return fail(SANA_ERR_INVALID_ARG, "%s: scaling factor must be finite and >= 1", who);
  const int n = rotary_dim / 2;
  double base = theta, mul = 1.0, lo = 0.0, hi = 0.0;
  if (kind == SANA_ROTARY_NTK) base = theta * std::pow(sc->factor, (double)n / (n - 1));
  if (kind == SANA_ROTARY_YARN) {
    if (sc->original < 1 || !(sc->beta_slow > 0.0) || !(sc->beta_fast >= sc->beta_slow) ||
        !std::isfinite(sc->beta_fast) || !std::isfinite(sc->attention_factor) ||
        sc->attention_factor < 0.0)
      return fail(SANA_ERR_INVALID_ARG,
                  "%s: YaRN needs original >= 1, beta_fast >= beta_slow > 0, attention_factor >= 0", who);
    auto dim = [&](double turns) { return n * std::log(sc->original / (2.0 * kPi * turns)) / std::log(theta); };
    // The ramp may end past the last pair (which then turns more than beta_slow times
    // over the original positions, and is blended in part): both ends are bounded by the
    // elements of the head, as the published form has it, not by the pairs.
    const double top = rotary_dim - 1.0;
    lo = std::fmin(std::fmax(std::floor(dim(sc->beta_fast)), 0.0), top);
    hi = std::fmin(std::fmax(std::ceil(dim(sc->beta_slow)), 0.0), top);
    mul = sc->attention_factor > 0.0 ? sc->attention_factor : 0.1 * std::log(sc->factor) + 1.0;
  }
  double inv[128];
  for (int j = 0; j < n; ++j) {
    inv[j] = std::pow(base, -(double)j / n);
    if (kind == SANA_ROTARY_LINEAR) inv[j] /= sc->factor;
    if (kind == SANA_ROTARY_YARN) {
      // an empty ramp (lo == hi) is a step after lo
      double g = (j - lo) / std::fmax(hi - lo, 1e-3);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      inv[j] = inv[j] * (1.0 - g) + inv[j] / sc->factor * g;
    }
  }
  return rotary_table_run(table, max_positions, n, inv, mul, stream);
}

sana_status sana_rotary_apply(const sana_qk_shape* s, sana_dtype dt, const sana_qk_positions* at,
                              int inverse, const void* q, const void* k, float q_mul, void* q_out,
                              void* k_out, sana_stream_t stream) {
  return forward("sana_rotary_apply", s, dt, at, false, inverse, q, k, nullptr, nullptr, 0.f, q_mul,
                 q_out, k_out, stream);
}

sana_status sana_qk_norm_rope(const sana_qk_shape* s, sana_dtype dt, const sana_qk_positions* at,
                              const void* q, const void* k, const float* q_weight,
                              const float* k_weight, float eps, float q_mul, void* q_out,
                              void* k_out, sana_stream_t stream) {
  return forward("sana_qk_norm_rope", s, dt, at, true, 0, q, k, q_weight, k_weight, eps, q_mul,
                 q_out, k_out, stream);
}

size_t sana_qk_norm_rope_bwd_workspace_size(const sana_qk_shape* s) {
  if (!s || s->B < 0 || s->N < 0 || s->head_dim < 1 || s->head_dim > 256) return 0;
  return qk_norm_rope_bwd_ws_bytes((long long)s->B * s->N, s->head_dim);
}

sana_status sana_qk_norm_rope_bwd(const sana_qk_shape* s, sana_dtype dt,
                                  const sana_qk_positions* at, const void* q, const void* k,
                                  const float* q_weight, const float* k_weight, float eps,
                                  float q_mul, const void* dq_out, const void* dk_out, void* dq,
                                  void* dk, float* d_q_weight, float* d_k_weight, void* ws,
                                  size_t ws_bytes, sana_stream_t stream) {
  const char* who = "sana_qk_norm_rope_bwd";
  QkTensors a;
  RotaryDev rt;
  if (sana_status e = check_call(who, s, dt, at, &a, &rt)) return e;
  if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(q_mul))
    return fail(SANA_ERR_INVALID_ARG, "%s: eps must be finite and >= 0, q_mul finite", who);
  const size_t tokens = (size_t)a.B * a.N;
  if (tokens && (!q || !dq_out || !dq || (a.kv_heads && (!k || !dk_out || !dk))))
    return fail(SANA_ERR_INVALID_ARG, "%s: NULL tensor pointer", who);
  if (!a.kv_heads && (k || dk_out || dk))
    return fail(SANA_ERR_INVALID_ARG, "%s: keys given with kv_heads == 0", who);
  const long long cq = (long long)a.heads * a.head_dim, ck = (long long)a.kv_heads * a.head_dim;
  const size_t wb = (size_t)a.head_dim * 4;
  const Range in[] = {{q, span(a, dt, a.q_stride, a.heads)}, {k, span(a, dt, a.k_stride, a.kv_heads)},
                      {dq_out, span(a, dt, cq, a.heads)},    {dk_out, span(a, dt, ck, a.kv_heads)},
                      {q_weight, wb},                        {k_weight, wb},
                      {rt.table, (size_t)rt.max_positions * rt.pairs * 8}};
  const size_t need = qk_norm_rope_bwd_ws_bytes((long long)tokens, a.head_dim);
  const Range out[] = {{dq, span(a, dt, cq, a.heads)}, {dk, span(a, dt, ck, a.kv_heads)},
                       {d_q_weight, wb}, {d_k_weight, wb}, {ws, need}};
  if (sana_status e = check_buffers(who, in, 7, out, 5)) return e;
  for (const Range& o : out)
    if (overlap({rt.positions, tokens * 4}, o))
      return fail(SANA_ERR_INVALID_ARG, "%s: an output aliases the positions", who);
  if (need && (!ws || ws_bytes < need))
    return fail(SANA_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", who, ws ? ws_bytes : 0, need);
  if (reinterpret_cast<uintptr_t>(ws) & 255u)
    return fail(SANA_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  a.q = q;
  a.k = k;
  a.dq_out = dq_out;
  a.dk_out = dk_out;
  a.q_out = dq;
  a.k_out = dk;
  a.wq = q_weight;
  a.wk = k_weight;
  return qk_norm_rope_bwd_run(a, dt, rt, eps, q_mul, d_q_weight, d_k_weight, ws, stream);
}

}  // extern "C"
