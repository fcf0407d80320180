"""Scores of any size: a large common part in every score of a row cancels in its softmax.

The products are made so that fp32 holds every sum exactly: element 0 of q and k gives +-2^c to every
score, the others multiples of 2^(c - 22), so the scores' differences are those of the 64-bit formulas
and the tolerance of y is the usual one (test_gpu_window.py).  lse is of the size of the common part:
its relative error is that of scale * log2 e in fp32, of the running reference and sum put together and of
ln 2, half a step of 2^-23 each, with the result's own at most 4 * 2^-24 in all."""

import math

import pytest
import torch

from tests._sana import sana
from tests.test_gpu_window import D, check, reference

pytestmark = pytest.mark.gpu


def rows(seed, N, heads, kv, c, sign):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.zeros(1, N, heads, D, device="cuda")
    k = torch.zeros(1, N, kv, D, device="cuda")
    q[..., 0], k[..., 0] = 2.0 ** (c // 2), sign * 2.0 ** (c - c // 2)
    q[..., 1:40] = 2.0 ** (c - 22)
    k[..., 1:40] = torch.randint(-1, 2, (1, N, kv, 39), generator=gen, device="cuda").float()
    v, g, dy = (torch.randn(1, N, n * D, generator=gen, device="cuda").bfloat16() for n in (kv, heads, heads))
    return q.bfloat16().flatten(2), k.bfloat16().flatten(2), v, g, dy


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("c,scale", [(10, 1.0), (22, 0.5), (23, 0.5), (24, 0.1), (26, 0.0), (30, 2.0 ** -9), (40, 2.0 ** -19)])
@pytest.mark.parametrize("N,heads,kv,window,block", [(260, 2, 1, 0, 1), (300, 2, 2, 64, 32), (1700, 12, 6, 0, 1)], ids=str)
def test_a_large_common_score_cancels(N, heads, kv, window, block, c, scale, sign):
    q, k, v, g, dy = rows(c, N, heads, kv, c, sign)
    ref = reference(q, k, v, g, dy, heads, kv, window, 0, block, None, scale or 1 / math.sqrt(D))
    y, lse = sana.window_anchor_fwd(q, k, v, g, heads, kv, window, block=block, scale=scale, want_lse=True)
    sana.sync_status()
    check("y", y, ref)
    want = ref["lse"][0]
    assert ((lse.double() - want).abs() <= 4 * 2.0 ** -24 * want.abs() + 2e-4).all()


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("c,scale", [(22, 0.5), (26, 0.0), (30, 2.0 ** -9)])
def test_the_step_too(c, scale, sign):
    N, heads, kv = 70, 4, 2
    q, k, v, g, dy = rows(c, N, heads, kv, c, sign)
    ref = reference(q, k, v, g, dy, heads, kv, 0, 0, 1, None, scale or 1 / math.sqrt(D))
    caches = [torch.zeros(1, 80, kv * D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    out = [sana.window_anchor_decode(*(t[:, i:i + 1].contiguous() for t in (q, k, v, g)), *caches,
                                     torch.full((1,), i, dtype=torch.int32, device="cuda"), heads, kv, 0, scale=scale)
           for i in range(N)]
    sana.sync_status()
    check("y", torch.cat(out, dim=1), ref)
