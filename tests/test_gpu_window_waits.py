"""Waits of the windowed anchor's kernels that nothing but a barrier may order: the last products of
dQ, and key tiles with padding that one of a CTA's two query tiles does not see.  The forms that reach
them, many times over with other work in between; every run has to give the first one's bits, and those
the 64-bit formulas' values.  (A wait that is missed ends in a status, which sync_status raises.)"""

import math

import pytest
import torch

from tests._sana import sana
from tests.test_gpu_window import D, check, inputs, reference

pytestmark = pytest.mark.gpu


def runs(B, N, Nk, heads, kv, window, sinks, block, lengths, gated, times, names):
    q, k, v, gate, dy = inputs(17, B, N, Nk, heads, kv, gated, False, lengths)
    ref = reference(q, k, v, gate, dy, heads, kv, window, sinks, block, lengths, 1 / math.sqrt(D))
    lt = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    kw = dict(window=window, sinks=sinks, block=block, lengths=lt)
    noise = torch.randn(2048, 2048, device="cuda")
    first = None
    for i in range(times):
        y, lse = sana.window_anchor_fwd(q, k, v, gate, heads, kv, want_lse=True, **kw)
        got = dict(zip(("dq", "dk", "dv", "dg"),
                       sana.window_anchor_bwd(q, k, v, gate, y, lse, dy, heads, kv, **kw)), y=y, lse=lse)
        if i % 3 == 0:
            noise = noise @ noise * 1e-4
        first = first or got
        for n in names:
            assert torch.equal(got[n], first[n]), (n, i)
    sana.sync_status()
    for n in names:
        check(n, first[n], ref)


@pytest.mark.parametrize("N,Nk,window,sinks", [
    (128, 128, 0, 0),       # one key tile to a query tile
    (256, 256, 0, 0),       # one and two
    (900, 900, 0, 0),       # one to eight
    (700, 700, 100, 5),     # the last tile a whole one, the first the sinks' narrow one
    (40, 1000, 0, 0),
    (3, 1000, 200, 130),    # two tiles of sinks, the second narrow
])
def test_dq_is_read_after_its_last_product(N, Nk, window, sinks):
    runs(2, N, Nk, 6, 2, window, sinks, 1, None, False, 60, ("dq", "dk", "dv"))


@pytest.mark.parametrize("B,N,Nk,heads,kv,window,sinks,block,lengths", [
    # pairs of query tiles in different blocks: a run of key tiles that the first does not see
    (2, 2600, 2600, 8, 8, 0, 0, 1280, [2500, 2600]),
    (3, 2304, 2304, 8, 8, 1408, 3, 1152, [2304, 1300, 1153]),
    # the first tile's window begins before the second's, sinks between
    (2, 2000, 2300, 12, 12, 1500, 140, 1, [2299, 2050]),
    # padding inside a tile that only the second tile sees; a sequence that ends in its first row
    (4, 1600, 1600, 7, 7, 1500, 0, 1, [1409, 1408, 1537, 1]),
    # two heads to a CTA
    (2, 1700, 1700, 16, 4, 1500, 0, 1, [1601, 1700]),
    # one query tile to a CTA
    (3, 300, 300, 2, 1, 90, 2, 1, [300, 131, 128]),
])
def test_padded_values_are_cleared_by_whoever_reads_them(B, N, Nk, heads, kv, window, sinks, block, lengths):
    """Values behind a sequence's end are infinite here (inputs() fills them in); the forward's result
    alone is compared between runs, all of it with the formulas."""
    runs(B, N, Nk, heads, kv, window, sinks, block, lengths, True, 25, ("y", "lse"))
