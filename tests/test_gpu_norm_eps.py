"""The norm's gradient at small eps, against the formulas in 64 bits.  Tolerances: those of
test_gpu_rotary.py -- one rounding to the type, 3e-6 of a row's largest element for the fp32 arithmetic
(of dx, whose two terms may cancel, twice that of the largest of all), and of a weight gradient 1e-5 of
the sum of its terms' absolute values."""

import pytest
import torch

from tests._sana import sana
from tests.test_gpu_rotary import F32_TOL, close, frequencies, make, norm_turn

pytestmark = pytest.mark.gpu


def compare(q, k, dq, dk, wq, heads, kv, D, eps, layout="half"):
    dtype, N = q.dtype, q.shape[1]
    rt = sana.Rotary(N, D, layout=layout)
    outs = sana.qk_norm_rope(q, k, wq, None, rt, heads, kv, eps=eps)
    grads = sana.qk_norm_rope_bwd(dq, dk, q, k, wq, None, rt, heads, kv, eps=eps)
    sana.sync_status()
    ang = (torch.arange(N, dtype=torch.float64)[:, None] * frequencies(D, 10000.0, None)[0])[None]
    for i, (x, dy, w) in enumerate(((q, dq, wq), (k, dk, None))):
        x, dy = (t.cpu().double().unflatten(2, (-1, D)) for t in (x, dy))
        x.requires_grad_()
        w = (torch.ones(D) if w is None else w.cpu()).double().requires_grad_()
        y = norm_turn(x, w, ang, 1.0, layout == "half", eps)
        y.backward(dy)
        got_y, got_x, got_w = outs[i], grads[i], grads[2 + i]
        assert all(torch.isfinite(t).all() for t in (got_y, got_x, got_w))
        close(got_y.unflatten(2, (-1, D)), y.detach(), dtype)
        close(got_x.unflatten(2, (-1, D)), x.grad, dtype, 2 * F32_TOL * x.grad.abs().max().item())
        xh = (x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)).detach()
        terms = (2 * dy.abs().amax(-1, keepdim=True) * xh.abs()).sum((0, 1, 2))
        assert ((got_w.cpu().double() - w.grad).abs() <= 1e-5 * terms).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("heads,kv,D", [(1, 1, 128), (3, 1, 128), (5, 3, 64), (7, 2, 16), (9, 5, 256), (2, 3, 32)])
def test_no_eps(heads, kv, D, dtype, layout):
    """eps = 0, and heads that do not fill a warp's row groups: everything is finite and right."""
    B, N = 2, 9
    q, k = make(1, B, N, heads, kv, D, dtype, True)
    dq, dk = make(2, B, N, heads, kv, D, dtype, False)
    wq = torch.linspace(0.5, 1.5, D).cuda()
    compare(q, k, dq, dk, wq, heads, kv, D, 0.0, layout)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [2.0 ** -46, 2.0 ** -30, 2.0 ** 30, 2.0 ** 46])
def test_rows_far_from_one(size, dtype):
    """Rows of 1e-14 to 1e14 with eps = 0: 1 / rms is a plain fp32 number, its cube is not."""
    heads, kv, D = 4, 2, 128
    q, k = (t * size for t in make(3, 2, 9, heads, kv, D, dtype, False))
    dq, dk = make(4, 2, 9, heads, kv, D, dtype, False)
    compare(q, k, dq, dk, torch.linspace(0.5, 1.5, D).cuda(), heads, kv, D, 0.0)
