"""A Rotary is whole when its constructor returns, like a Rope: another stream may use it at once."""

import pytest
import torch

from tests._sana import sana

pytestmark = pytest.mark.gpu


def test_a_table_built_behind_long_work_is_used_on_another_stream():
    D, n = 128, 1 << 15
    q = torch.randn(1, 64, D, device="cuda")
    want, _ = sana.rotary_apply(q, None, sana.Rotary(n, D), 1, 0, offset=n - 64)
    x = torch.randn(8192, 8192, device="cuda")
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        x = x @ x * 1e-4                 # some ten ms on the stream that builds the table
    held = sana.Rotary(n, D)
    with torch.cuda.stream(other):
        got, _ = sana.rotary_apply(q, None, held, 1, 0, offset=n - 64)
    torch.cuda.synchronize()
    sana.sync_status()
    assert torch.equal(got, want)


def test_a_table_may_be_built_in_a_capture():
    D = 128
    q = torch.randn(1, 16, D, device="cuda")
    want, _ = sana.rotary_apply(q, None, sana.Rotary(16, D), 1, 0)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        held = sana.Rotary(16, D)
        got, _ = sana.rotary_apply(q, None, held, 1, 0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
