"""Expanded tensors at the entry points that take strided ones: refused before anything is launched,
or, as a copy, what the copy gives."""

import pytest
import torch

from tests._sana import sana

pytestmark = pytest.mark.gpu

D = 128


@pytest.mark.parametrize("B,N", [(4, 1), (1, 6), (3, 6)])
def test_expanded_inputs_are_refused(B, N):
    gen = torch.Generator(device="cuda").manual_seed(3)
    one = lambda h: torch.randn(1, 1, h * D, generator=gen, device="cuda").bfloat16().expand(B, N, h * D)  # noqa: E731
    whole = lambda h: torch.randn(B, N, h * D, generator=gen, device="cuda").bfloat16()  # noqa: E731
    q, k, v, g, dy = whole(4), whole(2), whole(2), whole(4), whole(4)
    rt = sana.Rotary(8, D, layout="half")
    for x in (dict(q=one(4)), dict(k=one(2))):
        a = {**dict(q=q, k=k), **x}
        with pytest.raises(ValueError, match="rows of their own"):
            sana.rotary_apply(a["q"], a["k"], rt, 4, 2)
        with pytest.raises(ValueError, match="rows of their own"):
            sana.qk_norm_rope(a["q"], a["k"], None, None, rt, 4, 2)
        with pytest.raises(ValueError, match="rows of their own"):
            sana.qk_norm_rope_bwd(q, k, a["q"], a["k"], None, None, rt, 4, 2)
    y, lse = sana.window_anchor_fwd(q, k, v, g, 4, 2, 4, want_lse=True)
    for x in (dict(q=one(4)), dict(k=one(2)), dict(v=one(2)), dict(gate=one(4))):
        a = {**dict(q=q, k=k, v=v, gate=g), **x}
        with pytest.raises(ValueError, match="rows of their own"):
            sana.window_anchor_fwd(**a, heads=4, kv_heads=2, window=4)
        with pytest.raises(ValueError, match="rows of their own"):
            sana.window_anchor_bwd(**a, out=y, lse=lse, dy=dy, heads=4, kv_heads=2, window=4)
    e = one(4)
    yc, _ = sana.rotary_apply(e.contiguous(), None, rt, 4, 0)
    assert torch.equal(yc, sana.rotary_apply(e[:1, :1].repeat(B, N, 1), None, rt, 4, 0)[0])
    sana.sync_status()
