"""NaN and overflow in what a row sees come out as NaN, as from the formulas -- never as the zeros of a
row that sees nothing; rows that do not see them keep their bits."""

import math

import pytest
import torch

from tests._sana import sana
from tests.test_gpu_window import D, inputs, visible

pytestmark = pytest.mark.gpu

LAYOUTS = [  # N, heads, kv, window, sinks, block: one query tile to a CTA, two (rows, heads), blocks
    (300, 2, 1, 100, 3, 1), (1600, 7, 7, 1500, 0, 1), (1700, 16, 4, 0, 0, 1), (500, 2, 2, 170, 0, 50),
    (200, 4, 2, 1, 0, 1),
]


def rows_that_see(N, window, sinks, block, j, length=None):
    return visible(N, N, window, sinks, block, N if length is None else length)[:, j]


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("N,heads,kv,window,sinks,block", LAYOUTS, ids=str)
def test_a_bad_key_shows_in_every_row_that_sees_it(N, heads, kv, window, sinks, block, value):
    """One element of one key, at columns of every kind (of 16: the last two are where one forward
    exponential in eight is computed another way).  An infinite element gives scores of both signs:
    +inf makes a row NaN, -inf takes the key's weight to 0, so those rows stay finite."""
    q, k, v, gate, _ = inputs(5, 1, N, N, heads, kv, True, False, None)
    kw = dict(window=window, sinks=sinks, block=block, want_lse=True)
    clean, clean_lse = sana.window_anchor_fwd(q, k, v, gate, heads, kv, **kw)
    for j in (0, 1, 14, 15, 16 * 7 + 13, 16 * 9 + 15, N - 1):
        bad = k.clone()
        bad[0, j, 5] = value
        y, lse = sana.window_anchor_fwd(q, bad, v, gate, heads, kv, **kw)
        sana.sync_status()
        sees = rows_that_see(N, window, sinks, block, j)
        nan = sees[None].expand(heads, N)               # (heads, N)
        first = (torch.arange(heads, device="cuda") < heads // kv)[:, None]   # those of key head 0
        nan = nan & first
        if math.isinf(value):
            nan = nan & ((q[0].view(N, heads, D)[..., 5].T.float() * value) > 0)
        y4, c4 = y[0].view(N, heads, D).transpose(0, 1), clean[0].view(N, heads, D).transpose(0, 1)
        assert torch.isnan(y4[nan]).all() and torch.isnan(lse[0][nan]).all(), j
        free = ~(sees[None] & first)
        assert torch.equal(y4[free], c4[free]) and torch.equal(lse[0][free], clean_lse[0][free]), j
        if value == -math.inf or value == math.inf:
            rest = sees[None] & first & ~nan
            alone = torch.isinf(lse[0]) | torch.isnan(lse[0])  # nothing left: all of its scores are -inf
            assert (torch.isfinite(y4[rest]).all(-1) | alone[rest]).all()
            assert torch.isnan(y4[rest & alone]).all() and torch.isnan(lse[0][rest & alone]).all()


def test_the_backward_of_a_bad_row_is_nan():
    """A NaN query: its own dq, and dk, dv of every key that it sees, whichever column of a tile the
    query and the key fall on."""
    N, heads, kv, window = 400, 2, 1, 60
    q, k, v, gate, dy = inputs(6, 1, N, N, heads, kv, True, False, None)
    kw = dict(window=window)
    for i in (0, 12, 15, 111, 127, 128 + 14, 128 + 31, 399):
        bad = q.clone()
        bad[0, i, 3] = math.nan                          # of head 0
        y, lse = sana.window_anchor_fwd(bad, k, v, gate, heads, kv, want_lse=True, **kw)
        dq, dk, dv, dg = sana.window_anchor_bwd(bad, k, v, gate, y, lse, dy, heads, kv, **kw)
        sana.sync_status()
        assert torch.isnan(y[0, i, :D]).all() and torch.isfinite(y[0, i, D:]).all()
        assert torch.isnan(dq[0, i, :D]).all() and torch.isnan(dg[0, i, :D]).all()
        seen = visible(N, N, window, 0, 1, N)[i]
        assert torch.isnan(dk[0, seen]).all() and torch.isnan(dv[0, seen]).all(), i


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_the_step_shows_a_bad_key(value):
    """In the cache (every slot of a tile's kind), or the new one; at one CTA, a cluster and a split
    with a second kernel."""
    for B, heads, kv, cap in ((2, 4, 2, 40), (2, 8, 8, 1030), (1, 8, 8, 8200), (2, 6, 1, 8200)):
        gen = torch.Generator(device="cuda").manual_seed(9)
        rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
        kc, vc = rnd(B, cap, kv * D), rnd(B, cap, kv * D)
        lengths = torch.full((B,), cap - 1, dtype=torch.int32, device="cuda")
        for j in (0, 15, 38, cap // 2, cap - 1):
            for N in (1, 3):
                q, k, v = rnd(B, N, heads * D).abs(), rnd(B, N, kv * D), rnd(B, N, kv * D)
                a, b = kc.clone(), vc.clone()
                at = lengths - N + 1
                (k[0, 0] if j == cap - 1 else a[0, j])[5] = value
                y = sana.window_anchor_decode(q, k, v, None, a, b, at, heads, kv, 0)
                sana.sync_status()
                g = heads // kv
                seen = j == cap - 1 or j < cap - N      # (the last slots before the new ones)
                assert torch.isnan(y[0].view(N, heads, D)[:, :g]).all() or not seen, (cap, j, N)
                assert torch.isfinite(y[0].view(N, heads, D)[:, g:]).all() and torch.isfinite(y[1:]).all()


def test_scores_that_are_all_minus_infinity():
    """A row whose only key gives -inf: 0 / 0, in the forward and in the step."""
    q = torch.full((1, 4, D), 1e30, dtype=torch.bfloat16, device="cuda")
    k, v = -q, torch.ones_like(q)
    y, lse = sana.window_anchor_fwd(q, k, v, None, 1, 1, 1, want_lse=True)
    assert torch.isnan(y).all() and torch.isnan(lse).all()
    cache = torch.zeros(1, 8, D, dtype=torch.bfloat16, device="cuda")
    one = lambda t: t[:, :1].contiguous()  # noqa: E731
    y = sana.window_anchor_decode(one(q), one(k), one(v), None, cache, cache.clone(),
                                  torch.zeros(1, dtype=torch.int32, device="cuda"), 1, 1, 0)
    sana.sync_status()
    assert torch.isnan(y).all()


def test_empty_entries_and_padding_stay_zero_whatever_they_hold():
    nan = lambda *s: torch.full(s, math.nan, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    for cap in (16, 1030, 8200):
        y = sana.window_anchor_decode(nan(2, 1, 4 * D), nan(2, 1, D), nan(2, 1, D), nan(2, 1, 4 * D), nan(2, cap, D),
                                      nan(2, cap, D), torch.tensor([-1, -5], dtype=torch.int32, device="cuda"), 4, 1, 0)
        assert (y == 0).all()
    q, k, v, gate, _ = inputs(7, 2, 300, 300, 2, 1, True, False, [300, 150])
    y, lse = sana.window_anchor_fwd(q, k, v, gate, 2, 1, 50, 2, want_lse=True,
                                    lengths=torch.tensor([300, 150], dtype=torch.int32, device="cuda"))
    sana.sync_status()
    assert torch.isfinite(y).all() and (y[1, 150:] == 0).all() and (lse[1, :, 150:] == -math.inf).all()
