"""The windowed anchor -- forward, backward, ring-cache step -- against dense masked formulas in 64 bits.

Tolerances, elementwise, from the roundings of the operands (u = 2^-8, half a bf16 step at most;
sums of absolute values in 64 bits):
  y   P is rounded (u), a quarter of the exponentials are a cubic (8e-5), the result is rounded (u):
      (u + 2e-4) sigma sum_j p_j |v_j| + u |y|
  lse the cubic (8e-5) and 128 fp32 additions of the scores, 128 * 2^-24 sum_d |q_d k_d| scale:
      below 2e-4 for the N(0, 1) inputs here
  dv  P (u), do = sigma dy (u with a gate) and lse: (2 u + 6e-4) sum_i p |do| + u |dv|
  ds  its own rounding (u) and lse; dp from the rounded do (u with a gate); delta from the rounded y:
      tol_ds = (u + 6e-4) |ds| + p (u sum_d |do v| + sum_d |dy| tol_y)
  dq, dk   scale * sum tol_ds |k| (|q|) + u |dq|
  dg  |dy| (1 - sigma) tol_y + (u + 1e-4) |dg|"""

import math

import pytest
import torch

from tests._sana import sana

pytestmark = pytest.mark.gpu

U = torch.finfo(torch.bfloat16).eps / 2  # 2^-8
D = 128


def visible(N, Nk, window, sinks, block, length):
    p = torch.arange(Nk - N, Nk, device="cuda")[:, None]
    j = torch.arange(Nk, device="cuda")[None]
    e = (p // block + 1) * block
    near = (j >= e - window) if window else torch.ones_like(j, dtype=torch.bool)
    return (j < e) & (j < length) & (p < length) & (near | (j < sinks))


def reference(q, k, v, gate, dy, heads, kv, window, sinks, block, lengths, scale):
    """Dense 64-bit forward and backward, with the tolerances above."""
    B, N, Nk, g = q.shape[0], q.shape[1], k.shape[1], heads // kv
    split = lambda x, n: torch.nan_to_num(x.double(), 0.0, 0.0, 0.0).view(B, x.shape[1], n, D).transpose(1, 2)  # noqa: E731
    lens = [Nk] * B if lengths is None else lengths
    sees = torch.stack([visible(N, Nk, window, sinks, block, n) for n in lens])[:, None]
    alive = sees.any(-1)[..., None]                      # (B, 1, N, 1)
    Q, G, DY = split(q, heads), None if gate is None else split(gate, heads), split(dy, heads)
    K, V = (split(x, kv).repeat_interleave(g, 1) for x in (k, v))
    s = (Q @ K.transpose(-1, -2) * scale).masked_fill(~sees, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(sees, torch.exp(s - torch.where(alive, lse[..., None], 0.0)), 0.0)
    sg = torch.ones_like(Q) if G is None else torch.sigmoid(G)
    sg = sg * alive
    o = p @ V
    y = sg * o
    ty = (U + 2e-4) * sg * (p @ V.abs()) + U * y.abs()
    do = sg * DY
    dyv = DY * alive
    ds = p * (do @ V.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
    tds = (U + 6e-4) * ds.abs() + p * ((U if gate is not None else 1e-5) * (do.abs() @ V.abs().transpose(-1, -2)) +
                                       (dyv.abs() * ty).sum(-1, keepdim=True))
    fold = lambda x: x.view(B, kv, g, Nk, D).sum(2)  # noqa: E731
    dq, tq = scale * ds @ K, scale * tds @ K.abs()
    dk, tk = fold(scale * ds.transpose(-1, -2) @ Q), fold(scale * tds.transpose(-1, -2) @ Q.abs())
    dv, tv = fold(p.transpose(-1, -2) @ do), fold((2 * U + 6e-4) * p.transpose(-1, -2) @ do.abs())
    dg = dyv * o * sg * (1 - sg)
    tg = dyv.abs() * (1 - sg) * ty + (U + 1e-4) * dg.abs()
    flat = lambda x: x.transpose(1, 2).flatten(2)  # noqa: E731
    out = dict(y=(flat(y), flat(ty)), lse=(lse, torch.full_like(lse, 2e-4)))
    for n, x, t in (("dq", dq, tq), ("dk", dk, tk), ("dv", dv, tv)):
        out[n] = flat(x), flat(t + U * x.abs())
    if gate is not None:
        out["dg"] = flat(dg), flat(tg)
    return out


def check(name, got, ref):
    want, tol = ref[name]
    got = got.double()
    if name == "lse":
        assert torch.equal(torch.isinf(got), torch.isinf(want)) and not torch.isnan(got).any()
        got, want = torch.nan_to_num(got, neginf=0), torch.nan_to_num(want, neginf=0)
    bad = ~((got - want).abs() <= tol + 1e-30)
    assert not bad.any(), (name, int(bad.sum()), torch.nonzero(bad)[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())


def inputs(seed, B, N, Nk, heads, kv, gated, packed, lengths):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    if packed and N == Nk:
        x = rnd(B, N, (2 * heads + 2 * kv) * D)
        q, k, v, gate = x.split([heads * D, kv * D, kv * D, heads * D], dim=2)
    else:
        q, k, v, gate = rnd(B, N, heads * D), rnd(B, Nk, kv * D), rnd(B, Nk, kv * D), rnd(B, N, heads * D)
    dy = rnd(B, N, heads * D)
    if lengths is not None:  # padding holds anything
        for b, n in enumerate(lengths):
            k[b, n:], v[b, n:] = math.nan, math.inf
            i = max(0, n - (Nk - N))
            q[b, i:], gate[b, i:], dy[b, i:] = math.nan, math.nan, -math.inf
    return q, k, v, gate if gated else None, dy


CASES = [  # B, N, Nk, heads, kv, window, sinks, block, lengths, gated, packed
    (1, 1, 1, 1, 1, 0, 0, 1, None, False, False),
    (1, 1, 1, 2, 1, 1, 0, 1, None, True, False),
    (2, 5, 5, 2, 2, 3, 1, 1, None, True, True),
    (1, 128, 128, 1, 1, 0, 0, 1, None, False, False),
    (1, 129, 129, 2, 1, 64, 0, 1, None, True, True),
    (2, 257, 257, 4, 2, 100, 4, 1, None, False, True),
    (1, 700, 700, 3, 3, 1, 0, 1, None, True, False),       # a row sees itself alone
    (1, 700, 700, 2, 1, 1, 300, 1, None, True, False),     # and many sinks
    (1, 640, 640, 8, 1, 128, 128, 1, None, False, True),   # limits on tile borders
    (1, 900, 900, 2, 2, 0, 7, 1, None, True, False),       # no limit: sinks change nothing
    (1, 777, 777, 2, 1, 5000, 5000, 1, None, False, False),
    (1, 600, 600, 2, 2, 150, 3, 50, None, True, True),     # blocks of 50
    (1, 600, 600, 2, 2, 600, 0, 600, None, False, False),  # one block: bidirectional
    (2, 515, 515, 2, 1, 130, 131, 130, None, True, False),
    (1, 600, 600, 2, 2, 0, 0, 170, None, True, False),
    (1, 3, 1000, 4, 2, 300, 5, 1, None, True, False),      # the last rows of a longer sequence
    (2, 300, 813, 4, 4, 200, 20, 1, None, False, False),
    (1, 130, 640, 5, 1, 256, 1, 64, None, True, False),
    (4, 200, 200, 2, 1, 60, 2, 1, [200, 0, 1, 129], True, True),
    (3, 260, 260, 2, 2, 0, 0, 1, [128, 259, 64], False, False),
    (3, 300, 500, 4, 1, 120, 9, 1, [500, 200, 201], True, False),  # nothing, then one row, is alive
    (2, 300, 300, 2, 2, 80, 0, 40, [290, 33], True, True),
    (2, 1100, 1100, 6, 2, 256, 4, 1, [1100, 900], True, True),
    (1, 2300, 2300, 1, 1, 512, 16, 1, None, False, False),
    (1, 2000, 2000, 8, 1, 64, 300, 1, None, False, True),          # three tiles of sinks, cut into shares
    (1, 2500, 2500, 2, 1, 100, 1, 1, None, True, False),           # the sinks' tile cut, the others whole
    (2, 5000, 5000, 1, 1, 4000, 2, 1, [5000, 3100], False, False),  # long key tiles beside short ones
    # more than ten key tiles to a query tile
    (1, 1700, 1700, 2, 1, 0, 0, 1, None, True, False),
    (2, 1500, 1900, 4, 2, 1400, 9, 1, [1900, 1333], True, False),
    (1, 1537, 1537, 2, 2, 1536, 100, 512, None, True, True),
    (3, 1665, 1665, 2, 1, 1500, 40, 1, [1665, 130, 0], False, False),
    (2, 1600, 1600, 3, 1, 0, 0, 1, [1600, 700], True, True),
    # the same with more tiles than SMs
    (1, 1700, 1700, 12, 6, 0, 0, 1, None, True, False),
    (2, 1500, 1900, 8, 4, 1400, 9, 1, [1900, 1333], True, False),
    (1, 1537, 1537, 12, 12, 1536, 100, 512, None, True, True),      # pairs of rows
    (3, 1665, 1665, 4, 2, 1500, 40, 1, [1665, 130, 0], False, False),
    (2, 1600, 1600, 6, 2, 0, 0, 1, [1600, 700], True, True),
    (1, 1300, 1300, 16, 4, 700, 4, 1, None, False, True),
    (2, 1111, 1500, 10, 5, 0, 0, 77, [1499, 0], False, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_backward_match_the_dense_formulas(case):
    B, N, Nk, heads, kv, window, sinks, block, lengths, gated, packed = case
    q, k, v, gate, dy = inputs(1, B, N, Nk, heads, kv, gated, packed, lengths)
    scale = 0.0 if N % 2 else 0.06
    ref = reference(q, k, v, gate, dy, heads, kv, window, sinks, block, lengths, scale or 1 / math.sqrt(D))
    lt = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    kw = dict(window=window, sinks=sinks, block=block, lengths=lt, scale=scale)
    y, lse = sana.window_anchor_fwd(q, k, v, gate, heads, kv, want_lse=True, **kw)
    sana.sync_status()
    check("y", y, ref)
    check("lse", lse, ref)
    assert torch.equal(y, sana.window_anchor_fwd(q, k, v, gate, heads, kv, **kw))
    got = sana.window_anchor_bwd(q, k, v, gate, y, lse, dy, heads, kv, **kw)
    sana.sync_status()
    for n, x in zip(("dq", "dk", "dv", "dg"), got):
        if x is not None:
            check(n, x, ref)
    again = sana.window_anchor_bwd(q, k, v, gate, y, lse, dy, heads, kv, **kw)
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))
    sana.sync_status()


@pytest.mark.parametrize("N,heads,kv,window,block,lengths", [(1232, 16, 4, 561, 242, None), (700, 8, 8, 300, 1, [700, 433]),
                                                           (2500, 4, 1, 0, 1, None), (900, 16, 2, 128, 1, None)])
def test_many_runs_give_the_same_bits(N, heads, kv, window, block, lengths):
    """Every sum has its order: 40 forward and backward runs, with work on the GPU before and after
    each, agree bit by bit (a product read before it is whole shows here)."""
    B = 1 if lengths is None else len(lengths)
    q, k, v, gate, dy = inputs(9, B, N, N, heads, kv, True, False, lengths)
    lt = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    kw = dict(window=window, sinks=3, block=block, lengths=lt)
    first = None
    for _ in range(40):
        y, lse = sana.window_anchor_fwd(q, k, v, gate, heads, kv, want_lse=True, **kw)
        run = (y, lse) + sana.window_anchor_bwd(q, k, v, gate, y, lse, dy, heads, kv, **kw)
        if first is None:
            first = run
        assert all(torch.equal(a, b) for a, b in zip(run, first))
    sana.sync_status()


def test_gradients_agree_with_differences():
    """Along random directions, the 64-bit forward's central differences match the gradients to the
    gradients' own error (2 % of the directional derivative's scale: 2^-8 roundings of some hundred
    terms of random sign)."""
    B, N, heads, kv = 1, 150, 2, 1
    q, k, v, gate, dy = inputs(3, B, N, N, heads, kv, True, False, None)
    kw = dict(window=40, sinks=2)
    y, lse = sana.window_anchor_fwd(q, k, v, gate, heads, kv, want_lse=True, **kw)
    grads = sana.window_anchor_bwd(q, k, v, gate, y, lse, dy, heads, kv, **kw)
    sana.sync_status()
    gen = torch.Generator(device="cuda").manual_seed(4)

    def loss(*xs):
        return (reference64(*xs, heads, kv, 40, 2) * dy.double()).sum()

    for i, g in enumerate(grads):
        xs = [x.double() for x in (q, k, v, gate)]
        u = torch.randn(xs[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        hi, lo = list(xs), list(xs)
        hi[i], lo[i] = xs[i] + 1e-5 * u, xs[i] - 1e-5 * u
        want = (loss(*hi) - loss(*lo)) / 2e-5
        size = g.double().norm()   # the standard deviation of <g, u>
        assert (want - (g.double() * u).sum()).abs() <= 0.02 * size


def reference64(q, k, v, gate, heads, kv, window, sinks):
    N = q.shape[1]
    split = lambda x, n: x.view(1, N, n, D).transpose(1, 2)  # noqa: E731
    K, V = (split(x, kv).repeat_interleave(heads // kv, 1) for x in (k, v))
    s = split(q, heads) @ K.transpose(-1, -2) / math.sqrt(D)
    p = torch.softmax(s.masked_fill(~visible(N, N, window, sinks, 1, N), -math.inf), -1)
    return (p @ V).transpose(1, 2).flatten(2) * torch.sigmoid(gate)


# ------------------------------------------------------------------ the ring cache

def decode_reference(seqs, pos0, q, gate, b, n, heads, kv, window, sinks, capacity, scale):
    """64-bit step of one sequence from its whole history seqs = (keys, values), (tokens, kv * D)."""
    keys, values = (x.double().view(-1, kv, D).transpose(0, 1).repeat_interleave(heads // kv, 0) for x in seqs)
    total = pos0 + n
    j = torch.arange(total, device="cuda")[None]
    p = torch.arange(pos0, total, device="cuda")[:, None]
    sees = (j <= p) & ((j < sinks) | ((j > p - window) if window else (j >= 0)))
    sees &= (j < sinks) | (j >= total - (capacity - sinks))      # what the ring still holds
    Q = q[b].double().view(n, heads, D).transpose(0, 1)
    s = (Q @ keys.transpose(-1, -2) * scale).masked_fill(~sees, -math.inf)
    pr = torch.softmax(s, -1)
    o, tol = pr @ values, (U + 1e-5) * (pr @ values.abs())
    if gate is not None:
        sg = torch.sigmoid(gate[b].double().view(n, heads, D).transpose(0, 1))
        o, tol = o * sg, (tol + 2e-5 * o.abs()) * sg
    flat = lambda x: x.transpose(0, 1).flatten(1)  # noqa: E731
    return flat(o), flat(tol + U * o.abs())


DECODE = [  # B, N, heads, kv, capacity, window, sinks, gated, tokens already seen
    (1, 1, 1, 1, 1, 1, 0, False, [0]),
    (1, 1, 4, 1, 1, 0, 0, True, [57]),                    # a ring of one slot
    (3, 1, 8, 2, 132, 128, 4, True, [0, 131, 1000]),
    (4, 1, 24, 24, 300, 200, 0, False, [299, 300, 301, 7]),
    (2, 2, 6, 2, 70, 64, 4, True, [69, 400]),
    (2, 4, 10, 2, 104, 100, 0, False, [101, 3]),          # 20 rows: two tiles of 16
    (1, 16, 4, 1, 600, 500, 20, True, [1234]),
    (2, 3, 16, 1, 4000, 0, 0, False, [3500, 100]),        # an ordinary cache, everything visible
    (1, 1, 8, 8, 9000, 9000, 100, True, [20000]),
    (1, 5, 3, 3, 64, 8, 50, False, [1000]),
    (2, 7, 2, 1, 17, 300, 10, False, [40, 2]),            # the window is longer than the ring
    (5, 1, 40, 8, 257, 250, 6, True, [-1, 0, 1, 256, -7]),
    (12, 3, 4, 2, 17, 9, 5, False, list(range(24, 36))),  # windows from every slot of the ring
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(map(str, c)))
def test_decode_steps_match_the_whole_history(case):
    """Two steps in a row from a cache that a plain loop filled: the outputs, the written slots and
    nothing else; lengths are left as they are."""
    B, N, heads, kv, cap, window, sinks, gated, seen = case
    gen = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    slot = lambda p: p if p < cap else sinks + (p - sinks) % (cap - sinks)  # noqa: E731
    hist = [[rnd(max(n, 0), kv * D) for _ in range(2)] for n in seen]
    caches = [torch.full((B, cap, kv * D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for b, n in enumerate(seen):
        for p in range(max(0, n - cap), max(n, 0)):
            for c, h in zip(caches, hist[b]):
                c[b, slot(p)] = h[p]
        for p in range(min(sinks, max(n, 0))):
            for c, h in zip(caches, hist[b]):
                c[b, slot(p)] = h[p]
    scale = 0.0 if B % 2 else 0.11
    for step in range(2):
        q, k, v = rnd(B, N, heads * D), rnd(B, N, kv * D), rnd(B, N, kv * D)
        gate = rnd(B, N, heads * D) if gated else None
        now = [n + step * N if n >= 0 else n for n in seen]
        lengths = torch.tensor(now, dtype=torch.int32, device="cuda")
        want = [c.clone() for c in caches]
        for b, n in enumerate(now):
            if n < 0:
                continue
            hist[b] = [torch.cat([h, x[b]]) for h, x in zip(hist[b], (k, v))]
            for i in range(N):
                for c, x in zip(want, (k, v)):
                    c[b, slot(n + i)] = x[b, i]
        y = sana.window_anchor_decode(q, k, v, gate, *caches, lengths, heads, kv, window=window, sinks=sinks,
                                      scale=scale)
        sana.sync_status()
        assert lengths.tolist() == now
        for c, w in zip(caches, want):
            assert torch.equal(c.view(torch.int16), w.view(torch.int16))
        for b, n in enumerate(now):
            if n < 0:
                assert (y[b] == 0).all()
                continue
            o, tol = decode_reference(hist[b], n, q, gate, b, N, heads, kv, window, sinks, cap, scale or D ** -0.5)
            bad = ~((y[b].double() - o).abs() <= tol + 1e-30)
            assert not bad.any(), (step, b, int(bad.sum()), (y[b].double() - o).abs().max().item())
