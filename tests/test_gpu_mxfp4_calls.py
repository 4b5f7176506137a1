"""MXFP4 as programs call it: captured steps, streams, workspaces, blocks that are no
numbers, extreme scales, operands and outputs beyond 4 GiB."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
from test_gpu_mxfp4 import check_product, check_quantized, exact, operand
from w4a16_dequant_gemv_amd import W4A16Error, mxfp4

pytestmark = pytest.mark.gpu

# (m, n_out, k): every kernel of the product, rows that end inside a stage and rows that do not
SIZES = [(1, 40, 288), (5, 100, 4096), (1, 100, 8160), (7, 90, 10016), (20, 130, 512), (70, 500, 800), (700, 3000, 544), (1000, 4001, 2080), (2000, 6001, 544),
         (2050, 5003, 1056), (2000, 8101, 800), (40, 302, 8000), (100, 71, 28640)]


def random(m, k, seed, dtype=torch.float16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((m, k), generator=g, device="cuda").to(dtype)


def bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_blocks_that_are_no_numbers(m, n, k):
    """An infinity or NaN in x spoils its row of y, a scale of 255 in W its column; nothing else changes."""
    qw, _ = operand(n, k, m)
    x = random(m, k, n)
    want = mxfp4.linear(x, qw)
    rows, cols = sorted({0, m // 2, m - 1}), sorted({n - 1, n // 3})
    for r, v, at in zip(rows, (float("inf"), float("nan"), -float("inf")), (k - 1, k // 2, 0)):
        x[r, at] = v
    for y in (mxfp4.linear(x, qw), mxfp4.matmul(mxfp4.quantize(x), qw)):
        assert torch.isnan(y[rows]).all()
        keep = torch.ones(m, dtype=torch.bool, device="cuda")
        keep[rows] = False
        assert torch.equal(bits(y[keep]), bits(want[keep]))
    blocks = qw.block_scales()
    blocks[cols[0], 0], blocks[cols[1], -1] = 255, 255
    bad = mxfp4.MXTensor.from_blocks(qw.codes, blocks)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[cols] = False
    y = mxfp4.matmul(mxfp4.quantize(random(m, k, n)), bad)
    assert torch.isnan(y[:, cols]).all() and torch.equal(bits(y[:, keep]), bits(want[:, keep]))


@pytest.mark.parametrize("m,n,k", SIZES)
def test_bytes_behind_the_last_block(m, n, k):
    """Scales behind a row's last block may hold anything."""
    qw, _ = operand(n, k, m)
    qx, _ = operand(m, k, n)
    want = mxfp4.matmul(qx, qw)
    for q in (qx, qw):
        if k % 256:
            q.scales[-1, :, k % 256 // 32:] = 255
    assert torch.equal(bits(mxfp4.matmul(qx, qw)), bits(want))
    assert torch.equal(mxfp4.dequantize(qx), mxfp4.dequantize(mxfp4.MXTensor.from_blocks(qx.codes, qx.block_scales())))


@pytest.mark.parametrize("m,n,k", SIZES)
def test_extreme_scales(m, n, k):
    """Powers of two that cancel leave y as it is; products out of the type's range are infinities."""
    (qx, _), (qw, _) = operand(m, k, n), operand(n, k, m)
    want = mxfp4.matmul(qx, qw)
    for by in (110, -110):
        move = lambda q, e: mxfp4.MXTensor.from_blocks(q.codes, (q.block_scales().int() + e).to(torch.uint8))
        assert torch.equal(bits(mxfp4.matmul(move(qx, by), move(qw, -by))), bits(want))
    big = mxfp4.MXTensor.from_blocks(torch.full_like(qx.codes, 0x77), torch.full_like(qx.block_scales(), 254))
    wide = mxfp4.MXTensor.from_blocks(torch.full_like(qw.codes, 0xFF), torch.full_like(qw.block_scales(), 254))
    for dtype in (torch.float16, torch.bfloat16):
        assert bool((mxfp4.matmul(big, wide, dtype) == -float("inf")).all())


def test_captured_steps():
    """Layers in one captured graph, of which those of a stream share a workspace, replayed with new inputs and the
    program's own work between the replays."""
    sizes = [(1, 4096, 1024), (8, 1000, 4096), (100, 700, 1024), (900, 3000, 544), (40, 300, 11008)]
    w = [operand(n, k, n)[0] for _, n, k in sizes]
    x = [random(m, k, m) for m, _, k in sizes]
    ws = torch.empty(max(mxfp4.workspace_size(*s) for s in sizes) + 16, dtype=torch.uint8, device="cuda")
    step = lambda: [mxfp4.linear(a, b, workspace=ws) for a, b in zip(x, w)] + [mxfp4.dequantize(mxfp4.quantize(x[2]), torch.float16)]
    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for i in range(5):
        for a in x:
            a.copy_(random(*a.shape, 50 + i))
        want = [mxfp4.linear(a, b) for a, b in zip(x, w)] + [mxfp4.dequantize(mxfp4.quantize(x[2]), torch.float16)]
        for o in got:
            o.zero_()
        ws.fill_(0xFF)
        torch.randn(4096, device="cuda").sum().item()
        g.replay()
        torch.cuda.synchronize()
        for o, y in zip(got, want):
            assert torch.equal(bits(o), bits(y)), i


def test_streams():
    """Calls on two streams at once, without workspaces of the caller's."""
    qw, _ = operand(300, 11008, 1)
    xs = [random(m, 11008, m) for m in (3, 40, 700, 2050)]
    want = [mxfp4.linear(x, qw) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            outs.append((i % 4, mxfp4.linear(xs[i % 4], qw)))
    torch.cuda.synchronize()
    for i, y in outs:
        assert torch.equal(bits(y), bits(want[i]))


def test_empty_and_refused():
    qw, _ = operand(10, 64, 1)
    none, _ = operand(0, 64, 1)
    x = random(4, 64, 1)
    assert mxfp4.linear(x[:0], qw).shape == (0, 10) and mxfp4.linear(x, none).shape == (4, 0)
    assert mxfp4.quantize(x[:0]).codes.shape == (0, 32) and mxfp4.dequantize(none).shape == (0, 64)
    assert mxfp4.matmul(none, qw).shape == (0, 10)
    one = torch.zeros((1, 4096), dtype=torch.float16, device="cuda")
    wide = torch.zeros((40, 4096), dtype=torch.float16, device="cuda")
    big, _ = operand(100, 4096, 1)
    ws = torch.empty(mxfp4.workspace_size(40, 100, 4096), dtype=torch.uint8, device="cuda")
    long, _ = operand(64, 28672, 1)
    wrong = mxfp4.MXTensor(qw.codes, qw.scales[:, :9].contiguous())
    for f in (lambda: mxfp4.linear(x.float(), qw), lambda: mxfp4.linear(x.cpu(), qw), lambda: mxfp4.linear(x[:, :32], qw),
              lambda: mxfp4.linear(x.T, qw), lambda: mxfp4.linear(x[0], qw), lambda: mxfp4.linear(x[:1].expand(4, 64), qw),
              lambda: mxfp4.linear(x, wrong), lambda: mxfp4.linear(x, qw, out=torch.empty((4, 10), device="cuda")),
              lambda: mxfp4.linear(x, qw, out=torch.empty((4, 11), dtype=torch.float16, device="cuda")),
              lambda: mxfp4.linear(x, qw, out=torch.empty((4, 10), dtype=torch.float16)),
              lambda: mxfp4.linear(x, qw, out=torch.empty((10, 4), dtype=torch.float16, device="cuda").T),
              lambda: mxfp4.linear(wide, big, workspace=ws[:-16]), lambda: mxfp4.linear(wide, big, workspace=ws.cpu()),
              lambda: mxfp4.linear(wide, big, workspace=ws[8:]), lambda: mxfp4.matmul(long, long, workspace=ws[:64]), lambda: mxfp4.matmul(qw, big), lambda: mxfp4.matmul(qw, qw, torch.float32),
              lambda: mxfp4.quantize(x[:, 1:33]), lambda: mxfp4.quantize(x.int()), lambda: mxfp4.quantize(x[:, :48]),
              lambda: mxfp4.quantize(x, out=big), lambda: mxfp4.dequantize(qw, torch.float64), lambda: mxfp4.dequantize(wrong),
              lambda: mxfp4.quantize(torch.zeros((4, 100), dtype=torch.float16, device="cuda")[:, :64])):
        with pytest.raises(W4A16Error):
            f()
    mxfp4.linear(wide, big, workspace=ws)
    own = torch.empty(mxfp4.workspace_size(64, 64, 28672, linear=False), dtype=torch.uint8, device="cuda")
    assert torch.equal(mxfp4.matmul(long, long, workspace=own), mxfp4.matmul(long, long))
    mxfp4.linear(one, big, workspace=ws[:0])                  # quantized on the way


def test_beyond_4_gib():
    """Offsets that 32 bits do not hold: x, the values that come back, codes, y."""
    g = torch.Generator(device="cuda").manual_seed(3)
    rows, k = 300001, 8192
    x = torch.empty((rows, k), dtype=torch.float16, device="cuda")
    x.view(-1)[:1 << 26].normal_(generator=g)
    x[-700:].normal_(generator=g)
    q = mxfp4.quantize(x)
    check_quantized(x[-600:], mxfp4.MXTensor(q.codes[-600:], q.scales[:, -600:].contiguous()), "the last rows")
    v = mxfp4.dequantize(q, torch.float16)
    del x
    last = mxfp4.MXTensor(q.codes[-600:].contiguous(), q.scales[:, -600:].contiguous())
    assert torch.equal(v[-600:], mxfp4.dequantize(last, torch.float16))
    del v, q
    n = 520001                                                # 8.5 GB of codes, just within the limit
    codes = torch.randint(0, 256, (n, k * 2), generator=g, dtype=torch.uint8, device="cuda")
    scales = torch.randint(118, 126, (n, k * 4 // 32), generator=g, dtype=torch.uint8, device="cuda")
    w = mxfp4.MXTensor.from_blocks(codes, scales)
    tail = ref.values(ref.unpack(codes[-300:].cpu().numpy()), scales[-300:].cpu().numpy())
    for m in (1, 70):
        qx, xv = operand(m, 4 * k, m)
        check_product(mxfp4.matmul(qx, w)[:, -300:], xv, tail, f"{m} rows")
    del w, codes, scales
    (qx, xv), (qw, wv) = operand(40000, 64, 1), operand(60000, 64, 2)       # 4.8 GB of y
    y = mxfp4.matmul(qx, qw)
    check_product(y[-300:, -700:], xv[-300:], wv[-700:], "y")
    check_product(y[20000:20300, :700], xv[20000:20300], wv[:700], "y")
