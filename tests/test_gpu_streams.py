"""The stream that a call goes to is torch's current one, with either way of asking for it."""
import pytest
import torch

import w4a16_dequant_gemv_amd as w4
from w4a16_dequant_gemv_amd import api, kv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ask", [api._raw_stream, api._stream_of_object])
def test_calls_take_the_current_stream(ask, monkeypatch):
    monkeypatch.setattr(api, "_raw_stream", ask)
    monkeypatch.setattr(kv, "_raw_stream", ask)
    x = torch.ones((1, 128), dtype=torch.float16, device="cuda")
    for s in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            assert api._stream(x) == s.cuda_stream == ask(x.device.index)
    qw = w4.quantize_pack(torch.randn((64, 128), device="cuda"))
    cache = kv.PagedKVCache(2, 1, 64, 1, x.device, page=64)
    batch = kv.PagedBatch(*(torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([0, 1], [0], [[0]], [0])))
    k = torch.ones((1, 1, 64), dtype=torch.float16, device="cuda")
    want = w4.linear(x, qw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                        # a call on any other stream would not be in it
        y = w4.linear(x, qw)
        cache.append(k, 2 * k, batch)
        a = cache.attend(k, batch)
    for _ in range(3):
        y.zero_()
        a.zero_()
        cache.v_tail.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and (a == 2).all()
