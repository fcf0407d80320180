"""Refusals of the windowed anchor's entry points: every bad call is turned back on the host (no
GPU; the pointers below are never read)."""

import pytest

from tests._sana import _lib

L = _lib.lib
INVALID, UNSUPPORTED, WORKSPACE = _lib.SANA_ERR_INVALID_ARG, _lib.SANA_ERR_UNSUPPORTED, _lib.SANA_ERR_WORKSPACE
MB = 1 << 20


def call(fn="fwd", B=1, N=8, Nk=16, heads=4, kv_heads=2, D=128, qs=0, ks=0, vs=0, gs=0, window=4, sinks=1, block=1,
         lengths=None, scale=0.0, q=1 * MB, k=2 * MB, v=3 * MB, g=4 * MB, out=5 * MB, lse=6 * MB, dy=7 * MB,
         dq=8 * MB, dk=9 * MB, dv=10 * MB, dg=11 * MB, ws=64 * MB, ws_bytes=256 * MB):
    s = _lib.WindowShape(B, N, Nk, heads, kv_heads, D, qs, ks, vs, gs, window, sinks, block, lengths, scale)
    if fn == "fwd":
        return L.sana_window_anchor_fwd(s, q, k, v, g, out, lse, None)
    return L.sana_window_anchor_bwd(s, q, k, v, g, out, lse, dy, dq, dk, dv, dg, ws, ws_bytes, None)


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), INVALID), (dict(heads=3), INVALID), (dict(kv_heads=0), INVALID), (dict(heads=0), INVALID),
    (dict(D=64), UNSUPPORTED), (dict(N=17), INVALID), (dict(N=-1), INVALID), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(block=0), INVALID), (dict(window=4, block=5), INVALID),
    (dict(Nk=(1 << 30) + 1), UNSUPPORTED), (dict(window=(1 << 30) + 1), UNSUPPORTED),
    (dict(B=65536), UNSUPPORTED), (dict(heads=131072), UNSUPPORTED), (dict(ks=1 << 31, Nk=1 << 20), UNSUPPORTED),
    (dict(qs=504), INVALID), (dict(qs=516), INVALID), (dict(ks=248), INVALID), (dict(vs=257), INVALID),
    (dict(gs=8), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(lengths=2), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(q=MB + 2), INVALID), (dict(g=4 * MB + 8), INVALID), (dict(out=None), INVALID),
])
def test_bad_calls_are_refused(fn, bad, status):
    assert call(fn, **bad) == status, _lib.last_error()


@pytest.mark.parametrize("bad", [dict(out=MB), dict(out=2 * MB + 256), dict(lse=5 * MB), dict(out=4 * MB),
                                 dict(lengths=5 * MB)])
def test_forward_outputs_must_not_overlap_anything(bad):
    assert call("fwd", **bad) == INVALID and "alias" in _lib.last_error()


@pytest.mark.parametrize("bad,status", [
    (dict(dq=MB), INVALID), (dict(dk=9 * MB, dv=9 * MB), INVALID), (dict(dv=7 * MB), INVALID),
    (dict(ws=5 * MB), INVALID), (dict(lengths=9 * MB), INVALID), (dict(ws=64 * MB + 128), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=64), WORKSPACE), (dict(g=None), INVALID), (dict(dg=None), INVALID),
    (dict(lse=None), INVALID), (dict(dy=None), INVALID), (dict(N=0), UNSUPPORTED),
])
def test_backward_buffers(bad, status):
    assert call("bwd", **bad) == status


def test_empty_calls_do_nothing():
    assert call("fwd", N=0) == _lib.SANA_OK and call("fwd", B=0) == _lib.SANA_OK
    assert call("bwd", B=0) == _lib.SANA_OK and call("bwd", N=0, Nk=0) == _lib.SANA_OK


def test_workspace_sizes():
    size = _lib.window_anchor_bwd_workspace_size
    plain = size(1, 1000, 1000, 64, 64, 128)     # 512 key tiles: none is split
    stats = 2 * 64 * 1024 * 4
    assert plain == stats
    assert size(1, 1000, 1000, 64, 64, 128, gated=True) == stats + 1000 * 64 * 256
    assert size(1, 1000, 1000, 64, 64, 128, sinks=4) == plain  # nor the sinks': 8 query tiles see it
    share = 2 * 128 * 128 * 4                    # 32 query tiles: four shares of it, the others whole
    assert size(1, 4000, 4000, 2, 2, 128, sinks=4) == 2 * 2 * 4096 * 4 + 2 * 4 * share
    assert size(1, 128, 100000, 32, 2, 0) == 2 * 32 * 128 * 4  # many more keys than queries: none is split
    assert size(1, 1000, 1000, 2, 2, 0) > size(1, 1000, 1000, 2, 2, 0, head_dim=64) == 0
    dec = _lib.window_anchor_decode_workspace_size
    assert dec(1, 1, 8, 8, 8192, 0) == 8 * 26 * 8 * 130 * 4
    assert dec(1, 1, 8, 8, 1024, 0) == 0         # joined within a cluster
    assert dec(512, 1, 8, 8, 4096, 0) == 0


def decode(B=1, N=1, heads=4, kv_heads=2, D=128, capacity=16, window=8, sinks=2, scale=0.0, q=1 * MB, k=2 * MB,
           v=3 * MB, g=4 * MB, kc=5 * MB, vc=6 * MB, lengths=7 * MB, out=8 * MB, ws=64 * MB, ws_bytes=64 * MB):
    s = _lib.WindowDecodeShape(B, N, heads, kv_heads, D, capacity, window, sinks, scale)
    return L.sana_window_anchor_decode(s, q, k, v, g, kc, vc, lengths, out, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), INVALID), (dict(heads=5), INVALID), (dict(D=64), UNSUPPORTED), (dict(N=-1), INVALID),
    (dict(N=15), INVALID), (dict(sinks=16), INVALID), (dict(sinks=-1), INVALID), (dict(window=-1), INVALID),
    (dict(capacity=0), INVALID), (dict(capacity=(1 << 30) + 1), UNSUPPORTED), (dict(heads=4096, kv_heads=1, N=16, capacity=64), UNSUPPORTED),
    (dict(scale=float("nan")), INVALID), (dict(q=None), INVALID), (dict(lengths=None), INVALID),
    (dict(kc=None), INVALID), (dict(q=MB + 8), INVALID), (dict(lengths=7 * MB + 2), INVALID), (dict(out=MB), INVALID),
    (dict(kc=2 * MB), INVALID), (dict(vc=5 * MB), INVALID), (dict(out=7 * MB), INVALID),
])
def test_bad_decode_calls_are_refused(bad, status):
    assert decode(**bad) == status, _lib.last_error()


def test_decode_workspace_and_empty():
    big = dict(capacity=4096, window=0, kc=128 * MB, vc=192 * MB)
    assert decode(**big, ws_bytes=16) == WORKSPACE
    assert decode(**big, ws=None) == WORKSPACE
    assert decode(**big, ws=64 * MB + 16) == INVALID
    assert decode(**big, ws=128 * MB) == INVALID and "alias" in _lib.last_error()
    assert decode(B=0) == _lib.SANA_OK and decode(N=0) == _lib.SANA_OK
