"""Refusals of the rotary and query/key norm entry points: every bad call is turned back on the
host, before anything is enqueued (no GPU; the pointers below are never read)."""

import ctypes

import pytest

from tests._sana import _lib

L = _lib.lib
INVALID, UNSUPPORTED, WORKSPACE = _lib.SANA_ERR_INVALID_ARG, _lib.SANA_ERR_UNSUPPORTED, _lib.SANA_ERR_WORKSPACE
MB = 1 << 20


def call(fn="apply", dtype=_lib.SANA_BF16, B=1, N=4, heads=2, kv_heads=1, D=64, qs=0, ks=0, table=64 * MB,
         top=16, rot=64, layout=1, positions=None, offset=0, q=1 * MB, k=2 * MB, qo=3 * MB, ko=4 * MB, wq=5 * MB,
         wk=6 * MB, eps=1e-6, mul=1.0, ws=40 * MB, ws_bytes=MB, dq=7 * MB, dk=8 * MB, rope=None, grid=(0, 0, 0)):
    s = _lib.QkShape(B, N, heads, kv_heads, D, qs, ks)
    at = _lib.QkPositions(positions=positions, offset=offset)
    rt = _lib.RotaryStruct(table, top, rot, layout)
    if rope is None:
        at.rotary = ctypes.pointer(rt)
    else:
        at.rope = ctypes.pointer(rope)
        at.T, at.H, at.W = grid
    if fn == "apply":
        return L.sana_rotary_apply(s, dtype, at, 0, q, k, mul, qo, ko, None)
    if fn == "norm":
        return L.sana_qk_norm_rope(s, dtype, at, q, k, wq, wk, eps, mul, qo, ko, None)
    return L.sana_qk_norm_rope_bwd(s, dtype, at, q, k, wq, wk, eps, mul, qo, ko, dq, dk, 9 * MB, 10 * MB, ws,
                                   ws_bytes, None)


@pytest.mark.parametrize("fn", ["apply", "norm", "bwd"])
@pytest.mark.parametrize("bad,status", [
    (dict(dtype=7), INVALID), (dict(heads=0), INVALID), (dict(kv_heads=-1), INVALID), (dict(B=-1), INVALID),
    (dict(D=48), UNSUPPORTED), (dict(rot=24), UNSUPPORTED), (dict(rot=128), UNSUPPORTED), (dict(rot=0), UNSUPPORTED),
    (dict(B=1 << 16, N=1 << 15, top=1 << 20), UNSUPPORTED),
    (dict(qs=120), INVALID), (dict(qs=132), INVALID), (dict(ks=32), INVALID),
    (dict(table=None), INVALID), (dict(table=64 * MB + 4), INVALID), (dict(layout=2), INVALID),
    (dict(offset=13), INVALID), (dict(offset=-1), INVALID), (dict(N=17), INVALID), (dict(positions=2), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(q=MB + 8), INVALID), (dict(ko=None), INVALID),
    (dict(kv_heads=0), INVALID), (dict(mul=float("nan")), INVALID),
])
def test_bad_calls_are_refused(fn, bad, status):
    assert call(fn, **bad) == status, _lib.last_error()


@pytest.mark.parametrize("bad", [dict(qo=MB), dict(ko=2 * MB + 16), dict(qo=64 * MB), dict(qo=3 * MB, ko=3 * MB + 16),
                                 dict(positions=3 * MB)])
def test_outputs_must_not_overlap_anything(bad):
    assert call("apply", **bad) == INVALID and "alias" in _lib.last_error()


def test_norm_checks():
    assert call("norm", eps=-1.0) == INVALID
    assert call("norm", eps=float("inf")) == INVALID
    assert call("norm", qo=5 * MB) == INVALID and "alias" in _lib.last_error()
    assert call("bwd", ws_bytes=16) == WORKSPACE
    assert call("bwd", ws=None) == WORKSPACE
    assert call("bwd", ws=40 * MB + 16) == INVALID
    assert call("bwd", ws=7 * MB) == INVALID and "alias" in _lib.last_error()
    assert call("bwd", dq=3 * MB) == INVALID and "alias" in _lib.last_error()


def test_grid_positions():
    rope = _lib.RopeStruct(16, 16, 16, 16, 16, 16, 12, 10, 10, 2, 3, 4)
    ok = dict(rope=rope, N=24, grid=(2, 3, 4))
    for bad in (dict(ok, N=23), dict(ok, grid=(2, 4, 3)), dict(ok, offset=1), dict(ok, positions=4096),
                dict(ok, D=128), dict(ok, grid=(2, 0, 4)),
                dict(ok, rope=_lib.RopeStruct(None, 16, 16, 16, 16, 16, 12, 10, 10, 2, 3, 4))):
        assert call("apply", **bad) == INVALID, bad
    both = _lib.QkPositions(ctypes.pointer(_lib.RotaryStruct(16, 16, 64, 0)), ctypes.pointer(rope), 2, 3, 4, None, 0)
    s = _lib.QkShape(1, 24, 2, 1, 64, 0, 0)
    assert L.sana_rotary_apply(s, 1, both, 0, MB, 2 * MB, 1.0, 3 * MB, 4 * MB, None) == INVALID
    assert L.sana_rotary_apply(s, 1, _lib.QkPositions(), 0, MB, 2 * MB, 1.0, 3 * MB, 4 * MB, None) == INVALID
    assert L.sana_rotary_apply(None, 1, both, 0, MB, 2 * MB, 1.0, 3 * MB, 4 * MB, None) == INVALID


def test_empty_calls_do_nothing():
    assert call("apply", N=0) == _lib.SANA_OK
    assert call("norm", B=0) == _lib.SANA_OK


@pytest.mark.parametrize("args,status", [
    ((0, 64, 1e4, None, MB), INVALID), ((8, 20, 1e4, None, MB), UNSUPPORTED), ((8, 272, 1e4, None, MB), UNSUPPORTED),
    ((8, 64, 1.0, None, MB), INVALID), ((8, 64, float("nan"), None, MB), INVALID), ((8, 64, 1e4, None, None), INVALID),
    ((8, 64, 1e4, None, MB + 4), INVALID),
    ((8, 64, 1e4, (4, 2.0, 0, 0, 0, 0), MB), INVALID), ((8, 64, 1e4, (1, 0.5, 0, 0, 0, 0), MB), INVALID),
    ((8, 64, 1e4, (3, 2.0, 0, 32, 1, 0), MB), INVALID), ((8, 64, 1e4, (3, 2.0, 64, 1, 32, 0), MB), INVALID),
    ((8, 64, 1e4, (3, 2.0, 64, 32, 0, 0), MB), INVALID), ((8, 64, 1e4, (3, 2.0, 64, 32, 1, -1.0), MB), INVALID),
])
def test_bad_tables_are_refused(args, status):
    top, rot, theta, sc, table = args
    sc = None if sc is None else _lib.RotaryScaling(*sc)
    assert L.sana_rotary_table(top, rot, theta, sc, table, None) == status


def test_workspace_size_follows_the_shape():
    size = _lib.qk_norm_rope_bwd_workspace_size
    assert size(1, 1, 128) == 1024 and size(1, 0, 128) == 0
    assert size(2, 4000, 128) == size(4, 4000, 128) == 2 * 148 * 1024
