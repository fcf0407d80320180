"""The rotary, norm and windowed-anchor operators together, as a layer uses them, and the ways a
program calls them: captured and replayed, on streams of its own, over long caches.

Bars: a chain of operators is held to the 2e-2 max relative error of the library's bf16 results
(each operator alone is held to its own roundings elsewhere); what has to be the same computation is
compared exactly."""

import math

import pytest
import torch

import sana_inputs as si
from oracle import sana_oracle as orc
from tests._sana import sana
from tests.test_gpu_rotary import frequencies, norm_turn
from tests.test_gpu_window import D, check, decode_reference, inputs, reference, visible

pytestmark = pytest.mark.gpu

BF16_TOL = 2e-2


def max_rel(got, want):
    return ((got.double().cpu() - want.cpu()).abs().max() / want.abs().max().cpu()).item()


def test_projection_norm_rotation_window_and_all_gradients():
    """A causal layer from its packed projection: forward and the gradients of the projection's
    output and of the norm weights, against autograd through the 64-bit formulas."""
    B, N, C, heads, kv, W, sinks = 2, 300, 256, 4, 2, 96, 3
    gen = torch.Generator().manual_seed(11)
    x = torch.randn(B, N, C, generator=gen).bfloat16().cuda()
    wqkvg = (torch.randn((2 * heads + 2 * kv) * D, C, generator=gen) / math.sqrt(C)).bfloat16().cuda()
    wq, wk = (1 + 0.2 * torch.randn(D, generator=gen) for _ in range(2))
    dy = torch.randn(B, N, heads * D, generator=gen).bfloat16()
    rt = sana.Rotary(N, D, layout="half", scaling=("ntk", 2.0))
    lens = torch.tensor([N, 221], dtype=torch.int32, device="cuda")

    packed = sana.gemm_bf16(x.view(B * N, C), wqkvg).view(B, N, -1)
    q, k, v, g = packed.split([heads * D, kv * D, kv * D, heads * D], dim=2)
    qn, kn = sana.qk_norm_rope(q, k, wq.cuda(), wk.cuda(), rt, heads, kv)
    kw = dict(window=W, sinks=sinks, lengths=lens)
    y, lse = sana.window_anchor_fwd(qn, kn, v, g, heads, kv, want_lse=True, **kw)
    dqn, dkn, dv, dg = sana.window_anchor_bwd(qn, kn, v, g, y, lse, dy.cuda(), heads, kv, **kw)
    dq, dk, dwq, dwk = sana.qk_norm_rope_bwd(dqn, dkn, q, k, wq.cuda(), wk.cuda(), rt, heads, kv)
    sana.sync_status()

    p64 = packed.double().requires_grad_()
    w64 = [w.double().cuda().requires_grad_() for w in (wq, wk)]
    q6, k6, v6, g6 = p64.split([heads * D, kv * D, kv * D, heads * D], dim=2)
    inv, mul = frequencies(D, 10000.0, ("ntk", 2.0))
    ang = (torch.arange(N, dtype=torch.float64)[:, None] * inv)[None].cuda()
    q6 = norm_turn(q6.unflatten(2, (-1, D)), w64[0], ang, mul, True).transpose(1, 2)
    k6 = norm_turn(k6.unflatten(2, (-1, D)), w64[1], ang, mul, True).transpose(1, 2).repeat_interleave(2, 1)
    v6 = v6.unflatten(2, (-1, D)).transpose(1, 2).repeat_interleave(2, 1)
    sees = torch.stack([visible(N, N, W, sinks, 1, n) for n in (N, 221)])[:, None]
    s = (q6 @ k6.transpose(-1, -2) / math.sqrt(D)).masked_fill(~sees, -1e30)
    o = torch.where(sees.any(-1, keepdim=True), torch.softmax(s, -1) @ v6, 0.0)
    y6 = o.transpose(1, 2).flatten(2) * torch.sigmoid(g6)
    (y6 * dy.double().cuda()).sum().backward()
    dp = torch.cat([dq, dk, dv, dg], dim=2)
    assert max_rel(y, y6.detach()) <= BF16_TOL
    for a, b in zip(dp.split([heads * D, kv * D, kv * D, heads * D], dim=2),
                    p64.grad.split([heads * D, kv * D, kv * D, heads * D], dim=2)):
        assert max_rel(a, b) <= BF16_TOL
    assert max_rel(dwq, w64[0].grad) <= BF16_TOL and max_rel(dwk, w64[1].grad) <= BF16_TOL


def test_prompt_then_steps_continue_the_sequence():
    """A prompt through the forward, then one step after the other over ring caches that the prompt
    filled: the rows are those of the forward over the whole sequence."""
    B, heads, kv, W, sinks, n0, n = 2, 6, 2, 48, 5, 130, 40
    q, k, v, gate, _ = inputs(21, B, n0 + n, n0 + n, heads, kv, True, False, None)
    rt = sana.Rotary(n0 + n, D, layout="half")
    qn, kn = sana.rotary_apply(q, k, rt, heads, kv)
    ref = reference(qn, kn, v, gate, torch.zeros_like(q), heads, kv, W, sinks, 1, None, 1 / math.sqrt(D))
    whole = sana.window_anchor_fwd(qn, kn, v, gate, heads, kv, W, sinks)
    first = sana.window_anchor_fwd(qn[:, :n0].contiguous(), kn[:, :n0].contiguous(), v[:, :n0].contiguous(),
                                   gate[:, :n0].contiguous(), heads, kv, W, sinks)
    cap = sinks + W
    kc, vc = (torch.zeros(B, cap, kv * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for p in list(range(sinks)) + list(range(n0 - W, n0)):
        s = p if p < cap else sinks + (p - sinks) % W
        kc[:, s], vc[:, s] = kn[:, p], v[:, p]
    lengths = torch.full((B,), n0, dtype=torch.int32, device="cuda")
    rows = [first]
    for i in range(n0, n0 + n):
        at = lengths[:, None].contiguous()
        qi, ki = sana.rotary_apply(q[:, i:i + 1], k[:, i:i + 1], rt, heads, kv, positions=at)
        assert torch.equal(qi[:, 0], qn[:, i]) and torch.equal(ki[:, 0], kn[:, i])
        rows.append(sana.window_anchor_decode(qi, ki, v[:, i:i + 1].contiguous(), gate[:, i:i + 1].contiguous(),
                                              kc, vc, lengths, heads, kv, W, sinks))
        lengths += 1
    sana.sync_status()
    check("y", whole, ref)
    check("y", torch.cat(rows, dim=1), ref)


def test_one_block_is_the_dense_anchor():
    """Over a whole clip (one block, no window) the operators give the anchor: through its own
    rotated entry point after the norm, and against the oracle without one."""
    T, H, W, heads = 3, 7, 19, 2
    N = T * H * W
    q, k, v, g = (si.normal(9700 + i, (1, N, heads * D)).cuda() for i in range(4))
    rope = sana.Rope(T, H, W, (22, 21, 21))
    w = torch.linspace(0.5, 1.5, D).cuda()
    grid = (T, H, W)
    qs, ks = sana.qk_norm_rope(q, k, w, w, rope, heads, heads, grid=grid, q_mul=math.log2(math.e) / math.sqrt(D))
    ya = sana.softmax_anchor_rotated_fwd(qs, ks, v, g, grid, heads)
    qn, kn = sana.qk_norm_rope(q, k, w, w, rope, heads, heads, grid=grid)
    yw = sana.window_anchor_fwd(qn, kn, v, g, heads, heads, 0, block=N)
    sana.sync_status()
    assert max_rel(yw, ya.double()) <= BF16_TOL
    qr, kr = sana.rotary_apply(q, k, rope, heads, heads, grid=grid)
    yw = sana.window_anchor_fwd(qr, kr, v, g, heads, heads, 0, block=N)
    sana.sync_status()
    f64 = si.as_f64
    yo = orc.softmax_anchor(f64(q.cpu()), f64(k.cpu()), f64(v.cpu()), grid, (22, 21, 21), heads, gate=f64(g.cpu()))
    assert orc.max_rel_err(f64(yw.cpu()), yo) <= BF16_TOL


def test_step_is_captured_once_and_replayed_as_the_sequence_grows():
    """The rotation and the step in one graph; between replays only lengths (on the device) and the
    inputs' contents change.  Replays equal the eager calls."""
    B, heads, kv, W, sinks, cap = 3, 8, 2, 64, 4, 70
    gen = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    rt = sana.Rotary(200, D, layout="half")
    start = torch.tensor([0, 60, 69], dtype=torch.int32, device="cuda")
    seed_caches = [rnd(B, cap, kv * D) for _ in range(2)]
    xs = [[rnd(B, 1, n * D) for n in (heads, kv, kv)] for _ in range(9)]
    ws = torch.empty(sana.window_anchor_decode_workspace_size(B, 1, heads, kv, cap, W, sinks) + 256,
                     dtype=torch.uint8, device="cuda")

    def step(q, k, v, lengths, caches):
        qr, kr = sana.rotary_apply(q, k, rt, heads, kv, positions=lengths.view(B, 1))
        return sana.window_anchor_decode(qr, kr, v, None, *caches, lengths, heads, kv, W, sinks, ws=ws)

    lengths, caches, want = start.clone(), [c.clone() for c in seed_caches], []
    for x in xs:
        want.append(step(*x, lengths, caches).clone())
        lengths += 1
    end = [c.clone() for c in caches]

    lengths, caches = start.clone(), [c.clone() for c in seed_caches]
    static = [t.clone() for t in xs[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        spare = [c.clone() for c in seed_caches]
        step(*static, lengths, spare)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            y = step(*static, lengths, caches)
    for x, w in zip(xs, want):
        for s, t in zip(static, x):
            s.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, w)
        lengths += 1
    assert all(torch.equal(a, b) for a, b in zip(caches, end))
    sana.sync_status()


def test_training_step_captured_beside_an_eager_one_and_on_two_streams():
    """A captured forward and backward with a workspace, replayed while another stream runs other
    calls with a workspace of its own: all results are those of calls on their own."""
    B, N, heads, kv = 1, 700, 4, 2
    kw = dict(window=200, sinks=3)
    sets = [inputs(30 + i, B, N, N, heads, kv, True, False, None) for i in range(2)]
    size = sana.window_anchor_bwd_workspace_size(B, N, N, heads, kv, 200, 3, gated=True)
    wss = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def step(i, ws):
        q, k, v, g, dy = sets[i]
        y, lse = sana.window_anchor_fwd(q, k, v, g, heads, kv, want_lse=True, **kw)
        return (y, lse) + sana.window_anchor_bwd(q, k, v, g, y, lse, dy, heads, kv, ws=ws, **kw)

    want = [step(i, wss[i]) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(streams[0]):
        with torch.cuda.graph(graph, stream=streams[0]):
            captured = step(0, wss[0])
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            got.append(step(1, wss[1]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, want[0]))
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want[1]))
    sana.sync_status()


def test_given_outputs_are_written_whole_and_nothing_beside_them():
    B, N, heads, kv = 2, 261, 2, 1
    q, k, v, gate, _ = inputs(41, B, N, N, heads, kv, True, True, [261, 100])
    lens = torch.tensor([261, 100], dtype=torch.int32, device="cuda")
    store = torch.full((B + 2, N, heads * D), math.nan, dtype=torch.bfloat16, device="cuda")
    lse_store = torch.full((B + 2, heads, N), math.nan, device="cuda")
    y, lse = sana.window_anchor_fwd(q, k, v, gate, heads, kv, 50, 2, lengths=lens, out=store[1:-1], lse=lse_store[1:-1])
    sana.sync_status()
    assert y.data_ptr() == store[1:-1].data_ptr() and torch.isfinite(y).all() and not torch.isnan(lse).any()
    assert torch.isnan(store[0]).all() and torch.isnan(store[-1]).all()
    assert torch.isnan(lse_store[0]).all() and torch.isnan(lse_store[-1]).all()
    assert (y[1, 100:] == 0).all() and (lse[1, :, 100:] == -math.inf).all()


def test_lengths_outside_the_sequence_count_as_its_ends():
    q, k, v, gate, dy = inputs(43, 2, 200, 200, 2, 2, False, False, None)
    kw = dict(window=30, sinks=1)
    runs = []
    for lens in ([1000, -5], [200, 0]):
        t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        y, lse = sana.window_anchor_fwd(q, k, v, gate, 2, 2, want_lse=True, lengths=t, **kw)
        runs.append((y, lse) + sana.window_anchor_bwd(q, k, v, gate, y, lse, dy, 2, 2, lengths=t, **kw)[:3])
    sana.sync_status()
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    assert all((x[1] == 0).all() for x in (runs[0][0],) + runs[0][2:])


def test_a_cache_past_32_bit_offsets():
    """3 x 2^20 slots x 1024 elements: the last sequence starts past 2^31 elements."""
    B, cap, heads, kv, W, sinks = 3, 1 << 20, 8, 8, 300, 4
    kc, vc = (torch.zeros(B, cap, kv * D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    n = cap + 1000  # wrapped: the window lies in the middle, past the ring's start
    hist = [rnd(n, kv * D) for _ in range(2)]
    for p in list(range(sinks)) + list(range(n - W, n)):
        s = p if p < cap else sinks + (p - sinks) % (cap - sinks)
        kc[2, s], vc[2, s] = hist[0][p], hist[1][p]
    q, k, v = rnd(B, 1, heads * D), rnd(B, 1, kv * D), rnd(B, 1, kv * D)
    lengths = torch.tensor([-1, 0, n], dtype=torch.int32, device="cuda")
    y = sana.window_anchor_decode(q, k, v, None, kc, vc, lengths, heads, kv, W, sinks)
    sana.sync_status()
    keep = list(range(sinks)) + list(range(n - W, n))
    # the reference sees only what the call may see, at its true positions
    hist = [torch.cat([h[keep], x[2]]) for h, x in zip(hist, (k, v))]
    o, tol = decode_reference(hist, len(keep), q, None, 2, 1, heads, kv, W, sinks, 1 << 30, D ** -0.5)
    assert ((y[2].double() - o).abs() <= tol).all()
    assert torch.equal(y[1], v[1]) and (y[0] == 0).all()
    assert torch.equal(kc[2, sinks + (n - sinks) % (cap - sinks)], k[2, 0])


def test_tensors_past_32_bit_offsets():
    """600,000 tokens of 32 heads: the last rows lie past 2^31 elements."""
    N, heads, kv, W = 600_000, 32, 1, 60
    gen = torch.Generator(device="cuda").manual_seed(8)
    q = torch.empty(1, N, heads * D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    k, v = (torch.empty(1, N, kv * D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in range(2))
    y, lse = sana.window_anchor_fwd(q, k, v, None, heads, kv, W, want_lse=True)
    dq, dk, dv, _ = sana.window_anchor_bwd(q, k, v, None, y, lse, q, heads, kv, W)
    sana.sync_status()
    tail = 300
    sl = slice(N - tail, N)
    ref = reference(q[:, sl], k[:, sl], v[:, sl], None, q[:, sl], heads, kv, W, 0, 1, None, 1 / math.sqrt(D))
    for name, x in (("y", y), ("dq", dq), ("dk", dk), ("dv", dv)):
        want, tol = ref[name]
        got = x[:, sl].double()
        bad = ~((got - want).abs() <= tol)[:, W:]  # rows whose window lies in the tail
        assert not bad.any(), (name, int(bad.sum()))
    rt = sana.Rotary(N, D, layout="half")
    qr, _ = sana.rotary_apply(q, None, rt, heads, 0)
    back, _ = sana.rotary_apply(qr, None, rt, heads, 0, inverse=True)
    sana.sync_status()
    # there and back: two roundings of a pair's larger element
    assert ((back[:, sl] - q[:, sl]).abs().float().max() <= 2 * 2.0 ** -8 * 2 * q[:, sl].abs().float().max())


def test_binding_refusals():
    q = torch.zeros(2, 8, 2 * D, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(2, 8, D, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    f = sana.window_anchor_fwd
    for bad in (dict(q=q.transpose(0, 1)), dict(k=k[:1]), dict(v=k[:, :4]), dict(gate=k), dict(q=q.cpu()),
                dict(lengths=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(lengths=i32(1, 2, 3)),
                dict(lengths=torch.zeros(2, dtype=torch.int32)), dict(out=torch.zeros_like(k)),
                dict(lse=torch.zeros(2, 8, 2, device="cuda"))):
        with pytest.raises(ValueError):
            f(**{**dict(q=q, k=k, v=k, gate=None, heads=2, kv_heads=1, window=4), **bad})
    with pytest.raises(TypeError):
        f(q.float(), k, k, None, 2, 1, 4)
    with pytest.raises(sana.SanaError):
        f(q, k, k, None, 2, 1, 4, block=8)
    with pytest.raises(sana.SanaError):
        f(q, k[:, :4].contiguous(), k[:, :4].contiguous(), None, 2, 1, 4)   # fewer keys than queries
    with pytest.raises(sana.SanaError):
        f(q, k, k, None, 2, 1, 4, out=q)
    y, lse = f(q, k, k, None, 2, 1, 4, want_lse=True)
    with pytest.raises(ValueError):
        sana.window_anchor_bwd(q, k, k, None, y, lse, k, 2, 1, 4)
    with pytest.raises(sana.SanaError):
        sana.window_anchor_bwd(q, k, k, None, y, lse, y, 2, 1, 4, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    g = sana.window_anchor_decode
    cache = torch.zeros(2, 16, D, dtype=torch.bfloat16, device="cuda")
    ok = dict(q=q[:, :1].contiguous(), k=k[:, :1].contiguous(), v=k[:, :1].contiguous(), gate=None, k_cache=cache,
              v_cache=cache.clone(), lengths=i32(0, 3), heads=2, kv_heads=1, window=4)
    g(**ok)
    for bad in (dict(k=k), dict(k_cache=cache[:, ::2]), dict(v_cache=cache[:1]), dict(lengths=i32(0)), dict(gate=k)):
        with pytest.raises(ValueError):
            g(**{**ok, **bad})
    with pytest.raises(sana.SanaError):
        g(**{**ok, "v_cache": cache})
    with pytest.raises(sana.SanaError):
        g(**{**ok, "sinks": 16})
    e = q[:, :0]
    assert f(e, k, k, None, 2, 1, 4).shape == e.shape
    grads = sana.window_anchor_bwd(e, k, k, None, e, torch.zeros(2, 2, 0, device="cuda"), e, 2, 1, 4)
    assert (grads[1] == 0).all() and (grads[2] == 0).all()
    sana.sync_status()
