"""With a video grid's tables rotary_apply is the anchors' own rotation (rope_apply), from any frame on.

The two evaluate x c - y s with one rounding of a product each, not of the same product, and one of the
sum: they differ by at most 4 * 2^-24 of the products' size, and in bf16 by one rounding each more."""

import ctypes

import pytest
import torch

from tests._sana import _lib, sana

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offset", [0, 2])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_grid_rotation_is_the_anchors(dtype, offset):
    T, H, W, heads, D, B = 3, 5, 7, 4, 128, 2
    gen = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(B, T * H * W, heads * D, generator=gen, device="cuda").to(dtype)
    rope = sana.Rope(T + offset, H, W, (22, 21, 21))
    got, _ = sana.rotary_apply(x, None, rope, heads, 0, grid=(T, H, W), offset=offset)
    if offset == 0:
        want = sana.rope_apply(x, rope, (T, H, W), heads)
    else:
        shape, want = _lib.make_shape(B, (T, H, W), heads, D, offset), torch.empty_like(x)
        _lib.check(_lib.lib.sana_rope_apply(ctypes.byref(shape), _lib._dtype_code(x), _lib._ptr(x),
                                            ctypes.byref(rope.struct), 1.0, _lib._ptr(want), _lib._stream()))
    sana.sync_status()
    pair = x.double().unflatten(2, (-1, 2)).abs().sum(-1, keepdim=True).expand(-1, -1, -1, 2).flatten(2)
    tol = 4 * 2.0 ** -24 * pair
    if dtype == torch.bfloat16:
        tol = tol + 2 * 2.0 ** -8 * want.double().abs()
    assert ((got.double() - want.double()).abs() <= tol).all()
    # the first frame of the offset call is not the first frame of the grid
    if offset:
        assert not torch.equal(got, sana.rotary_apply(x, None, rope, heads, 0, grid=(T, H, W))[0])
