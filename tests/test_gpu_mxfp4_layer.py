"""MXFP4 projections and the paged cache's attention over shared pages as a decoder layer
has them: queries, keys and values from one product, appended and rotated, attended, and
the output projection.  Every stage against the definition in 64 bits of what it was given."""
import numpy as np
import pytest
import torch

import mx4_ref
import paged_ref as ref
from gpu_util import to_dev
from shared_cases import Case
from test_gpu_mxfp4 import check_product, exact, operand
from test_gpu_paged_shared import Shared, weights
from w4a16_dequant_gemv_amd import kv, mxfp4

pytestmark = pytest.mark.gpu

# a few answers to one question, a step of drafted tokens behind three prompts, and a full step
LAYERS = [Case(128, 128, 8, 8, ((3, 4),), 100, 1, 2), Case(64, 64, 2, 8, ((6, 9), (5, 4), (2, 1)), 150, 3, 0),
          Case(128, 64, 2, 16, ((9, 70),), 90, 1, 0)]


@pytest.mark.parametrize("c", LAYERS)
def test_layer(c):
    hidden = 1024
    w = Shared(c)
    B, d, q_size, kv_size = len(w.seqs), c.d, c.n_q * c.d, c.n_kv * c.d
    wqkv, wqkv_values = operand(q_size + 2 * kv_size, hidden, 1)
    wo, wo_values = operand(hidden, q_size, 2)
    rope = kv.rope_table(w.table.shape[1] * c.page, d, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    prefix = w.prefix()
    T, new = sum(w.new), w.new
    x = torch.empty((T, hidden), dtype=torch.float16, device="cuda")
    batch = w.batch(new)
    positions = torch.empty(T, dtype=torch.int32, device="cuda")

    def layer():
        qkv = mxfp4.linear(x, wqkv)
        k, v = qkv[:, q_size:q_size + kv_size].view(T, -1, d), qkv[:, q_size + kv_size:].view(T, -1, d)
        q = w.cache.append(k, v, batch, q=qkv[:, :q_size].view(T, -1, d), rope=rope, positions=positions)
        a = w.cache.attend(q, batch, prefix=prefix)
        return qkv, q, a, mxfp4.linear(a.view(T, q_size), wo)

    def advance():
        held = [len(s) for s in w.seqs]
        batch.ctx_lens.copy_(to_dev(np.array(held, np.int32)))
        at = np.concatenate([h + np.arange(m) for h, m in zip(held, new)]).astype(np.int32)
        positions.copy_(to_dev(at))
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        return at

    def check(parts, at):
        qkv, q, a, y = parts
        check_product(qkv, mx4_ref.values(*mx4_ref.quantize(exact(x))), wqkv_values, "qkv")
        # keys, values and queries as the cache has to have them, from the qkv that the product gave
        host = qkv.cpu().numpy().reshape(T, -1, d)
        rq, rk = (ref.rotate(np.ascontiguousarray(t), rope.cpu().numpy(), at) for t in (host[:, :c.n_q], host[:, c.n_q:c.n_q + c.n_kv]))
        assert np.array_equal(q.cpu().numpy().view(np.int16), rq.view(np.int16))
        i = 0
        for s, m in zip(w.seqs, new):
            s.append(rk[i:i + m], host[i:i + m, c.n_q + c.n_kv:])
            i += m
        w.check(rq, a, weights=weights(c))
        check_product(y, mx4_ref.values(*mx4_ref.quantize(exact(a.view(T, q_size)))), wo_values, "output")

    for _ in range(2):
        at = advance()
        check(layer(), at)
    at = advance()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        parts = layer()
    for _ in range(3):                                         # the first one again appends what the warm-up did
        graph.replay()
        torch.cuda.synchronize()
        check(parts, at)
        torch.randn(1000, device="cuda").sum().item()
        at = advance()
