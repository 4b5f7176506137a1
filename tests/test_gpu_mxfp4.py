"""MXFP4 on the GPU: quantization and the way back bit for bit against the definition,
products against binary64."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
from w4a16_dequant_gemv_amd import mxfp4

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16, torch.float32]


def exact(t):
    return t.double().cpu().numpy()


def check_quantized(x, q, what=""):
    codes, scales = ref.quantize(exact(x))
    got_s = q.block_scales().cpu().numpy()
    bad = np.argwhere(got_s != scales)
    assert not len(bad), f"{what}: {len(bad)} scales differ, first at {bad[0]}: {got_s[tuple(bad[0])]}, {scales[tuple(bad[0])]}"
    assert np.array_equal(q.scales.cpu().numpy(), ref.laid(scales)), what
    got = ref.unpack(q.codes.cpu().numpy())
    keep = np.repeat(scales != 255, 32, 1)
    bad = np.argwhere((got != codes) & keep)
    assert not len(bad), (f"{what}: {len(bad)} codes differ, first at {bad[0]}: x = {exact(x)[tuple(bad[0])]!r}, "
                          f"{got[tuple(bad[0])]}, {codes[tuple(bad[0])]}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,k,stride", [(1, 32, 32), (1, 4096, 4096), (3, 64, 64), (7, 288, 320), (64, 256, 512),
                                           (129, 5024, 5024), (1000, 96, 96), (5, 11008, 22016)])
def test_quantize(dtype, rows, k, stride):
    g = torch.Generator(device="cuda").manual_seed(rows * k)
    x = (torch.randn((rows, stride), generator=g, device="cuda") * torch.exp2(
        torch.randint(-12, 12, (rows, 1), generator=g, device="cuda").float())).to(dtype)[:, :k]
    q = mxfp4.quantize(x)
    check_quantized(x, q)
    codes, scales = ref.quantize(exact(x))
    v = ref.values(codes, scales)
    for to in TYPES:
        assert np.array_equal(exact(mxfp4.dequantize(q, to)), exact(torch.from_numpy(v).to(to)), equal_nan=True), to
    out = mxfp4.MXTensor(torch.full_like(q.codes, 255), torch.full_like(q.scales, 255))
    assert mxfp4.quantize(x, out=out) is out
    assert torch.equal(out.codes, q.codes) and torch.equal(out.scales, q.scales)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_quantize_every_value(dtype):
    """Every pattern of 16 bits, beside each power of two that makes it large or small in its block."""
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16)
    x = bits.view(dtype)
    tops = [0.0, 1.0, 2.0**-14, 2.0**-20, 1000.0, 2.0**15] if dtype == torch.float16 else [0.0, 1.0, 2.0**-126, 2.0**-100, 2.0**120]
    for top in tops:
        y = x.clone().view(-1, 16)
        z = torch.cat([y, torch.full_like(y, top)], 1).contiguous()          # 16 values and 16 times the power
        check_quantized(z, mxfp4.quantize(z), f"{dtype}, {top}")


def test_quantize_borders_of_binary32():
    """Values at and next to the borders between codes, at scales from the smallest to the largest."""
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9999995, 4.0, 0.0, 2.0, 3.0], np.float32)
    near = np.concatenate([borders, np.nextafter(borders, np.float32(0)), np.nextafter(borders, np.float32(100))])
    near = np.concatenate([near, -near])
    rows = []
    for e in (-149, -140, -130, -127, -126, -125, -100, -1, 0, 1, 60, 120, 125):
        for v in near.reshape(-1, 28):
            block = np.zeros(32)
            block[:28], block[28:] = v, [4.0, -4.0, 4.0, -0.0]
            rows.append(np.ldexp(block, e).astype(np.float32))
    rows.append(np.zeros(32, np.float32))
    rows.append(-np.zeros(32, np.float32))
    rows.append(np.full(32, 2.0**-149, np.float32))
    rows.append(np.full(32, np.finfo(np.float32).max))
    for v in (np.inf, -np.inf, np.nan):
        r = np.ones(32, np.float32)
        r[5] = v
        rows.append(r)
    x = torch.from_numpy(np.stack(rows)).cuda()
    q = mxfp4.quantize(x)
    check_quantized(x, q)
    assert torch.isnan(mxfp4.dequantize(q)[-3:]).all()


def test_dequantize_every_code_and_scale():
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    scales = np.arange(256, dtype=np.uint8)[:, None]
    q = mxfp4.MXTensor.from_blocks(torch.from_numpy(ref.pack(codes)).cuda(), torch.from_numpy(scales).cuda())
    with np.errstate(over="ignore"):
        v = torch.from_numpy(ref.values(codes, scales))
    for to in TYPES:
        want = v.to(torch.float32).to(to) if to != torch.float32 else v.to(to)   # binary32 holds all but overflows
        got = mxfp4.dequantize(q, to).cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        same = (got == want) | torch.isnan(want)
        assert bool(same.all()), (to, np.argwhere(~same.numpy())[:3])
        assert torch.equal(torch.signbit(got)[:255], torch.signbit(want)[:255])


def operand(rows, k, seed, device="cuda"):
    """Random codes and scales over a few powers of two, as MXTensor and values."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (rows, k), dtype=np.uint8)
    scales = rng.integers(118, 126, (rows, k // 32), dtype=np.uint8)
    q = mxfp4.MXTensor.from_blocks(torch.from_numpy(ref.pack(codes)).to(device), torch.from_numpy(scales).to(device))
    return q, ref.values(codes, scales)


def check_product(y, x, w, what=""):
    want, tol = ref.product(x, w, torch.finfo(y.dtype).eps / 2)
    off = np.abs(exact(y) - want)
    bad = np.argwhere(~(off <= tol))
    assert not len(bad), f"{what}: {len(bad)} of {off.size} off, first at {bad[0]}: {exact(y)[tuple(bad[0])]}, {want[tuple(bad[0])]}"


SHAPES = [(1, 16, 32), (1, 1, 32), (2, 17, 64), (1, 4096, 4096), (5, 100, 288), (16, 64, 512), (17, 33, 992), (40, 300, 1024),
          (64, 128, 256), (65, 129, 5024), (130, 1000, 480), (256, 256, 256), (257, 511, 800), (300, 5003, 544),
          (513, 256, 2048), (1000, 520, 1504)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matmul(m, n, k, dtype):
    qx, x = operand(m, k, m + n)
    qw, w = operand(n, k, m + k + 1)
    guard = torch.full((m + 2, n), 7.0, dtype=dtype, device="cuda")
    y = mxfp4.matmul(qx, qw, dtype, out=guard[1:-1])
    check_product(y, x, w)
    assert bool((guard[0] == 7).all()) and bool((guard[-1] == 7).all())
    assert torch.equal(y, mxfp4.matmul(qx, qw, dtype))


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear(m, n, k):
    qw, w = operand(n, k, m + n)
    g = torch.Generator(device="cuda").manual_seed(m * n)
    for dtype, stride in ((torch.float16, k), (torch.bfloat16, k + 64)):
        x = (torch.randn((m, stride), generator=g, device="cuda") * 3).to(dtype)[:, :k]
        y = mxfp4.linear(x, qw)
        assert y.dtype == dtype
        codes, scales = ref.quantize(exact(x))
        check_product(y, ref.values(codes, scales), w)
        assert torch.equal(y, mxfp4.matmul(mxfp4.quantize(x), qw, dtype)), "linear is quantize and matmul"
        ws = torch.empty(mxfp4.workspace_size(m, n, k) + 16, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(y)
        assert mxfp4.linear(x, qw, out=out, workspace=ws) is out and torch.equal(out, y)


@pytest.mark.parametrize("m,n,k", ref.KERNELS)
def test_every_kernel(m, n, k):
    qw, w = operand(n, k, m + n)
    g = torch.Generator(device="cuda").manual_seed(n)
    for dtype in (torch.float16, torch.bfloat16):
        x = torch.randn((m, k), generator=g, device="cuda").to(dtype)
        y = mxfp4.linear(x, qw)
        check_product(y, ref.values(*ref.quantize(exact(x))), w, mxfp4.kernel_config(m, n, k, dtype))
        assert torch.equal(y, mxfp4.matmul(mxfp4.quantize(x), qw, dtype))


@pytest.mark.parametrize("seed", range(40))
def test_random_products(seed):
    """Sizes from one row, channel or block to some thousands, x in rows apart, y anywhere, a workspace of the caller's."""
    rng = np.random.default_rng(400 + seed)
    size = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    m, n, k = size(1, 3000), size(1, 9000), 32 * size(1, 900)
    while m * n * k > 2e9:
        m, n = max(1, m // 2), max(1, n * 2 // 3)
    dtype = (torch.float16, torch.bfloat16)[int(rng.integers(2))]
    apart, off = 8 * int(rng.integers(0, 5)), int(rng.integers(0, 3))
    print(m, n, k, dtype, mxfp4.kernel_config(m, n, k, dtype), flush=True)
    qw, w = operand(n, k, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((m, k + apart), generator=g, device="cuda").to(dtype)[:, :k]
    room = torch.full((m * n + 8,), 7.0, dtype=dtype, device="cuda")
    y = room[off:off + m * n].view(m, n)
    ws = torch.full((mxfp4.workspace_size(m, n, k) + 16,), 255, dtype=torch.uint8, device="cuda")
    mxfp4.linear(x, qw, out=y, workspace=ws)
    check_product(y, ref.values(*ref.quantize(exact(x))), w)
    assert bool((room[:off] == 7).all()) and bool((room[off + m * n:] == 7).all()) and bool((ws[-16:] == 255).all())
    assert torch.equal(y, mxfp4.matmul(mxfp4.quantize(x), qw, dtype))
