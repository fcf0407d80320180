"""Rotary positions and query/key norm with rotation against plain 64-bit formulas.

Tolerances: bf16 outputs are rounded once from fp32 values, half a step is at most 2^-8 of the
value; the fp32 arithmetic before it (a sum over up to 256
squares, one square root and division, two products and an addition) adds less than 40 roundings of
2^-24 on the larger of the two products.  fp32: those 40 roundings, 40 * 2^-24 < 3e-6, of the row's
largest element (the two products of an element may cancel).  Weight gradients sum `rows` terms in
fp32 in chains of at most rows / 2368 + 300 additions: 1e-5 of the sum of absolute values covers
every shape here."""

import math

import pytest
import torch

from tests._sana import _lib, sana

pytestmark = pytest.mark.gpu

BF16_HALF_STEP = torch.finfo(torch.bfloat16).eps / 2  # 2^-8
F32_TOL = 3e-6


def frequencies(rot, theta, scaling):
    n = rot // 2
    j = torch.arange(n, dtype=torch.float64)
    inv, mul = theta ** (-j / n), 1.0
    if scaling is None:
        return inv, mul
    kind, factor = scaling[:2]
    if kind == "linear":
        inv = inv / factor
    elif kind == "ntk":
        inv = (theta * factor ** (rot / (rot - 2))) ** (-j / n)
    else:
        orig, fast, slow, att = (list(scaling[2:]) + [None] * 4)[:4]
        fast, slow = fast or 32.0, slow or 1.0
        d = lambda b: n * math.log(orig / (2 * math.pi * b)) / math.log(theta)  # noqa: E731
        lo, hi = min(max(math.floor(d(fast)), 0), n - 1), min(max(math.ceil(d(slow)), 0), n - 1)
        g = ((j - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        inv, mul = inv * (1 - g) + inv / factor * g, att or 0.1 * math.log(factor) + 1
    return inv, mul


def turn(x, ang, mul, half):
    """x (B, N, h, D) float64, ang (B or 1, N, pairs)."""
    R = 2 * ang.shape[-1]
    c, s = torch.cos(ang)[:, :, None] * mul, torch.sin(ang)[:, :, None] * mul
    y = x.clone()
    a, b = (slice(0, R // 2), slice(R // 2, R)) if half else (slice(0, R, 2), slice(1, R, 2))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def norm_turn(x, w, ang, mul, half, eps=1e-6):
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return turn(y if w is None else y * w, ang, mul, half)


def close(got, want, dtype, extra=0.0):
    """Elementwise: one rounding to the type, plus the fp32 arithmetic on the scale of the row."""
    got, want = got.double().cpu(), want.cpu()
    row = want.abs().amax(-1, keepdim=True)
    tol = F32_TOL * row + extra
    if dtype == torch.bfloat16:
        tol = tol + BF16_HALF_STEP * want.abs()
    bad = ((got - want).abs() > tol + 1e-30)
    assert not bad.any(), (bad.sum().item(), (got - want).abs().max().item())


def make(seed, B, N, heads, kv, D, dtype, packed):
    g = torch.Generator().manual_seed(seed)
    full = torch.randn(B, N, (heads + 2 * kv) * D, generator=g).to(dtype).cuda()
    q, k, _ = full.split([heads * D, kv * D, kv * D], dim=2)
    return (q, k) if packed else (q.contiguous(), k.contiguous())


CASES = [  # B, N, heads, kv, D, rot, layout, scaling, dtype, packed
    (1, 1, 1, 1, 128, 128, "half", None, torch.bfloat16, False),
    (3, 1, 32, 8, 128, 128, "half", ("linear", 4.0), torch.bfloat16, True),
    (2, 37, 5, 3, 128, 64, "half", ("ntk", 4.0), torch.bfloat16, True),
    (2, 37, 5, 1, 64, 16, "interleaved", ("yarn", 8.0, 1024), torch.bfloat16, True),
    (1, 301, 24, 24, 128, 128, "interleaved", None, torch.bfloat16, False),
    (2, 19, 7, 2, 256, 256, "half", ("yarn", 4.0, 64, 16.0, 2.0, 1.25), torch.float32, True),
    (1, 50, 3, 3, 128, 96, "half", None, torch.float32, True),
    (2, 33, 9, 2, 32, 32, "interleaved", ("yarn", 2.0, 1 << 20), torch.float32, False),
    (1, 23, 17, 4, 16, 16, "half", None, torch.float32, True),
    (1, 23, 17, 4, 16, 16, "interleaved", None, torch.bfloat16, True),
    (1, 700, 40, 8, 64, 48, "half", ("ntk", 2.0), torch.bfloat16, True),
    (1, 65, 6, 2, 256, 128, "interleaved", None, torch.bfloat16, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("scattered", [False, True])
def test_rotation_norm_and_gradient_match_the_formulas(case, scattered):
    B, N, heads, kv, D, rot, layout, scaling, dtype, packed = case
    half, top, theta = layout == "half", 5000, 10000.0
    q, k = make(1, B, N, heads, kv, D, dtype, packed)
    rt = sana.Rotary(top, rot, theta=theta, layout=layout, scaling=scaling)
    inv, mul = frequencies(rot, theta, scaling)
    if scattered:
        positions = torch.randint(0, top - 7, (B, N), dtype=torch.int32)
        positions.view(-1)[0] = top - 8
        at = dict(positions=positions.cuda(), offset=7)
        pos = positions.double() + 7
    else:
        at = dict(offset=top - N)
        pos = torch.arange(N, dtype=torch.float64)[None] + top - N
    ang = pos[..., None] * inv
    split = lambda x: x.cpu().double().unflatten(2, (-1, D))  # noqa: E731
    q_mul = 0.375

    for inverse in (False, True):
        yq, yk = sana.rotary_apply(q, k, rt, heads, kv, inverse=inverse, q_mul=q_mul, **at)
        sana.sync_status()
        sg = -ang if inverse else ang
        close(yq.unflatten(2, (-1, D)), q_mul * turn(split(q), sg, mul, half), dtype)
        close(yk.unflatten(2, (-1, D)), turn(split(k), sg, mul, half), dtype)

    g = torch.Generator().manual_seed(2)
    wq = (1 + 0.3 * torch.randn(D, generator=g))
    for w in (wq, None):
        xq, xk = split(q).requires_grad_(), split(k).requires_grad_()
        wqd = (torch.ones(D) if w is None else w).double().requires_grad_()
        wkd = torch.ones(D, dtype=torch.float64).requires_grad_()
        wg = None if w is None else w.cuda()
        yq, yk = sana.qk_norm_rope(q, k, wg, None, rt, heads, kv, q_mul=q_mul, **at)
        tq, tk = q_mul * norm_turn(xq, wqd, ang, mul, half), norm_turn(xk, wkd, ang, mul, half)
        close(yq.unflatten(2, (-1, D)), tq.detach(), dtype)
        close(yk.unflatten(2, (-1, D)), tk.detach(), dtype)
        dyq = torch.randn(B, N, heads * D, generator=g).to(dtype)
        dyk = torch.randn(B, N, kv * D, generator=g).to(dtype)
        got = sana.qk_norm_rope_bwd(dyq.cuda(), dyk.cuda(), q, k, wg, None, rt, heads, kv, q_mul=q_mul, **at)
        again = sana.qk_norm_rope_bwd(dyq.cuda(), dyk.cuda(), q, k, wg, None, rt, heads, kv, q_mul=q_mul, **at)
        sana.sync_status()
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        (tq * split(dyq)).sum().backward()
        (tk * split(dyk)).sum().backward()
        # the two terms of dx are each of the size of |w g| r: take the fp32 slack on the largest gradient of all
        slack = 2 * F32_TOL * max(xq.grad.abs().max().item(), xk.grad.abs().max().item())
        close(got[0].unflatten(2, (-1, D)), xq.grad, dtype, slack)
        close(got[1].unflatten(2, (-1, D)), xk.grad, dtype, slack)
        for dw, want, x, dy in ((got[2], wqd.grad, xq, split(dyq) * q_mul), (got[3], wkd.grad, xk, split(dyk))):
            xh = (x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)).detach()
            # |g| <= mul * (|dy| + |dy'|) elementwise, summed over the rows
            big = (mul * dy.abs().amax(-1, keepdim=True) * 2 * xh.abs()).sum((0, 1, 2))
            assert ((dw.cpu().double() - want).abs() <= 1e-5 * big).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_video_grid_is_the_anchors_rotation(dtype):
    """With a Rope the rotation is rope_apply's; the norm form follows the formula on its angles."""
    T, H, W, heads, D, off = 3, 5, 7, 4, 128, 2
    N = T * H * W
    q, k = make(5, 2, N, heads, 2, D, dtype, True)
    rope = sana.Rope(T + off, H, W, (22, 21, 21))
    yq, yk = sana.rotary_apply(q, k, rope, heads, 2, grid=(T, H, W), offset=off, q_mul=0.125)
    n = torch.arange(N)
    ang = torch.cat([p.double()[:, None] * 10000.0 ** (-torch.arange(m, dtype=torch.float64) / m)
                     for p, m in ((n // (H * W) + off, 22), (n // W % H, 21), (n % W, 21))], dim=1)[None]
    split = lambda x: x.cpu().double().unflatten(2, (-1, D))  # noqa: E731
    close(split(yq), 0.125 * turn(split(q), ang, 1.0, False), dtype)
    close(split(yk), turn(split(k), ang, 1.0, False), dtype)
    if off == 0:
        assert torch.equal(yk, sana.rope_apply(k.contiguous(), rope, (T, H, W), 2))
    w = torch.linspace(0.5, 1.5, D)
    yq, _ = sana.qk_norm_rope(q, None, w.cuda(), None, rope, heads, 0, grid=(T, H, W), offset=off)
    sana.sync_status()
    close(split(yq), norm_turn(split(q), w.double(), ang, 1.0, False), dtype)


def test_far_positions_keep_their_angles():
    """At position 2^20 an angle in fp32 would be off by up to 2^-4; the table's is rounded once."""
    top, rot = (1 << 20) + 3, 64
    rt = sana.Rotary(top, rot, theta=500000.0, layout="half")
    inv, _ = frequencies(rot, 500000.0, None)
    ang = torch.arange(top - 5, top, dtype=torch.float64)[:, None] * inv
    t = rt.table[top - 5:].cpu().double()
    assert (t[..., 0] - torch.cos(ang)).abs().max() <= 2 ** -24
    assert (t[..., 1] - torch.sin(ang)).abs().max() <= 2 ** -24


def test_zero_rows_infinities_and_positions_outside_the_table():
    D = 128
    q = torch.zeros(1, 3, 2 * D, dtype=torch.bfloat16, device="cuda")
    q[0, 1, 0] = 1.0
    q[0, 2, 100] = math.inf   # in the part that is not rotated
    rt = sana.Rotary(64, 64, layout="half")
    y, _ = sana.rotary_apply(q, None, rt, 2, 0)
    assert (y[0, 0] == 0).all() and y[0, 2, 100] == math.inf and (y[0, 2, :100] == 0).all()
    y, _ = sana.qk_norm_rope(q[:, :2], None, None, None, rt, 2, 0)
    assert (y[0, 0] == 0).all() and torch.isfinite(y).all()
    dq, _, dw, _ = sana.qk_norm_rope_bwd(torch.ones_like(y), None, q[:, :2], None, None, None, rt, 2, 0)
    assert torch.isfinite(dq).all() and torch.isfinite(dw).all()
    sana.sync_status()
    for bad in (-1, 64, 2 ** 31 - 1, -2 ** 31):
        p = torch.tensor([[0, bad, 63]], dtype=torch.int32, device="cuda")
        y, _ = sana.rotary_apply(torch.ones_like(q), None, rt, 2, 0, positions=p)
        with pytest.raises(sana.SanaError, match="outside the rotary table"):
            sana.sync_status()
        sana.sync_status()  # reported once
        near = torch.tensor([[0, 0 if bad < 0 else 63, 63]], dtype=torch.int32, device="cuda")
        assert torch.equal(y, sana.rotary_apply(torch.ones_like(q), None, rt, 2, 0, positions=near)[0])
        sana.sync_status()


def test_own_stream_captured_graph_and_given_outputs():
    B, N, h, kv, D = 2, 65, 8, 2, 128
    q, k = make(9, B, N, h, kv, D, torch.bfloat16, True)
    rt = sana.Rotary(N, D, layout="half")
    w = torch.rand(D, device="cuda")
    want = sana.qk_norm_rope(q, k, w, w, rt, h, kv)
    wb = sana.qk_norm_rope_bwd(*want, q, k, w, w, rt, h, kv)
    qo, ko = torch.empty_like(want[0]), torch.empty_like(want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        sana.qk_norm_rope(q, k, w, w, rt, h, kv, q_out=qo, k_out=ko)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            sana.qk_norm_rope(q, k, w, w, rt, h, kv, q_out=qo, k_out=ko)
            grads = sana.qk_norm_rope_bwd(qo, ko, q, k, w, w, rt, h, kv)
    for _ in range(2):
        qo.zero_(), ko.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
        assert all(torch.equal(a, b) for a, b in zip(grads, wb))
    sana.sync_status()


def test_binding_refusals():
    q = torch.zeros(2, 3, 256, dtype=torch.bfloat16, device="cuda")
    rt = sana.Rotary(8, 64)
    with pytest.raises(ValueError):
        sana.rotary_apply(q.transpose(0, 1), None, rt, 2, 0)       # sequences interleaved
    with pytest.raises(ValueError):
        sana.rotary_apply(q, q, rt, 2, 0)
    with pytest.raises(ValueError):
        sana.rotary_apply(q, q[:, :2], rt, 2, 2)
    with pytest.raises(ValueError):
        sana.rotary_apply(q, None, rt, 2, 0, positions=torch.zeros(2, 3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        sana.rotary_apply(q, None, rt, 2, 0, grid=(1, 1, 3))
    with pytest.raises(ValueError):
        sana.rotary_apply(q, None, rt, 2, 0, q_out=torch.empty(2, 3, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        sana.qk_norm_rope(q, None, torch.ones(64, device="cuda"), None, rt, 2, 0)
    with pytest.raises(ValueError):
        sana.rotary_apply(q.cpu(), None, rt, 2, 0)
    with pytest.raises(TypeError):
        sana.rotary_apply(q.half(), None, rt, 2, 0)
    with pytest.raises(ValueError):
        sana.Rotary(8, 64, layout="other")
    with pytest.raises(ValueError):
        sana.Rotary(8, 64, scaling=("yarn", 2.0))
    with pytest.raises(sana.SanaError):
        sana.rotary_apply(q, None, rt, 2, 0, offset=6)
    e = torch.zeros(2, 0, 256, dtype=torch.bfloat16, device="cuda")
    assert sana.rotary_apply(e, None, rt, 2, 0)[0].shape == e.shape
    dq, _, dw, _ = sana.qk_norm_rope_bwd(e, None, e, None, None, None, rt, 2, 0)
    assert (dw == 0).all()
    sana.sync_status()
