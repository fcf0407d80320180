"""Integers that do not fit the C ABI's int are refused by the binding: cut to 32 bits, a window of
2^32 would mean no limit and an offset of 2^32 position 0 (no GPU: CPU tensors stand for CUDA ones)."""

import pytest
import torch

from tests._sana import _lib, sana
from tests.test_strides_cpu import OnGpu

BIG = 1 << 32
bf16 = torch.bfloat16


def gpu(*shape):
    return OnGpu(torch.zeros(*shape, dtype=bf16))


@pytest.mark.parametrize("bad", [dict(window=BIG), dict(window=BIG + 4), dict(sinks=BIG), dict(sinks=-BIG),
                                 dict(block=BIG + 1), dict(window=1 << 31)])
def test_window_calls(bad):
    kw = {**dict(window=4, sinks=1, block=1), **bad}
    with pytest.raises(ValueError, match="C int"):
        _lib._window_shape(gpu(1, 8, 256), gpu(1, 8, 128), gpu(1, 8, 128), None, 2, 1, kw["window"], kw["sinks"],
                           kw["block"], None, 0.0)
    with pytest.raises(ValueError, match="C int"):
        sana.window_anchor_bwd_workspace_size(1, 8, 8, 2, 1, **kw)


@pytest.mark.parametrize("bad", [dict(window=BIG), dict(sinks=BIG + 1)])
def test_step(bad):
    kw = {**dict(window=4, sinks=1), **bad}
    with pytest.raises(ValueError, match="C int"):
        sana.window_anchor_decode(gpu(1, 1, 256), gpu(1, 1, 128), gpu(1, 1, 128), None, gpu(1, 16, 128), gpu(1, 16, 128),
                                  torch.zeros(1, dtype=torch.int32), 2, 1, **kw)
    with pytest.raises(ValueError, match="C int"):
        sana.window_anchor_decode_workspace_size(1, 1, 2, 1, 16, **kw)


def test_positions():
    rt = sana.Rotary.__new__(sana.Rotary)
    for offset in (BIG, BIG + 3, -BIG):
        with pytest.raises(ValueError, match="C int"):
            _lib._qk_call(gpu(1, 8, 256), None, rt, 2, 0, None, offset, None)
    rope = sana.Rope.__new__(sana.Rope)
    with pytest.raises(ValueError, match="C int"):
        _lib._qk_call(gpu(1, 8, 256), None, rope, 2, 0, None, 0, (BIG + 1, 2, 4))
    with pytest.raises(ValueError, match="C int"):
        sana.qk_norm_rope_bwd_workspace_size(1, BIG + 1, 128)


def test_tables():
    with pytest.raises(ValueError, match="C int"):
        sana.Rotary(BIG + 8, 64, device="cpu")
    with pytest.raises(ValueError, match="C int"):
        sana.Rotary(8, BIG + 64, device="cpu")
    with pytest.raises(ValueError, match="C int"):
        sana.Rotary(8, 64, scaling=("yarn", 2.0, BIG + 4096), device="cpu")
