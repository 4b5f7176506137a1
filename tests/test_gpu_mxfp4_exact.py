"""MXFP4 products where binary32 has no rounding to do, so that the result is one number: every
block of a long k counts; and products of scales at the bottom, which the other operand's scales bring back."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
from test_gpu_mxfp4 import exact
from w4a16_dequant_gemv_amd import mxfp4

pytestmark = pytest.mark.gpu


def tensor(codes, scales):
    return mxfp4.MXTensor.from_blocks(torch.from_numpy(ref.pack(codes)).cuda(), torch.from_numpy(scales).cuda())


@pytest.mark.parametrize("m,n,k", ref.KERNELS + [(16, 100, 28672), (300, 200, 28640), (129, 70, 16416)])
def test_whole_numbers(m, n, k):
    """Values 0, +-1, +-2, +-4 at one scale: products are whole numbers of at most 16, their sums below 2^24 however
    they are ordered, so that the sum is exact and the output's rounding the only one.  A block that is left out or comes twice
    changes nearly every element, however long k is: its 32 products add up to 34 on average, and fp16 holds the sums to 1."""
    rng = np.random.default_rng(m + n + k)
    assert 16 * k < 1 << 24
    code = np.array([0, 2, 4, 6, 10, 12, 14], np.uint8)
    cx, cw = code[rng.integers(0, 7, (m, k))], code[rng.integers(0, 7, (n, k))]
    sx, sw = np.full((m, k // 32), 127, np.uint8), np.full((n, k // 32), 127, np.uint8)
    qx, qw = tensor(cx, sx), tensor(cw, sw)
    want = torch.from_numpy(ref.values(cx, sx)).cuda() @ torch.from_numpy(ref.values(cw, sw)).cuda().T   # exact in binary64
    for dtype in (torch.float16, torch.bfloat16):
        y = mxfp4.matmul(qx, qw, dtype)
        off = (y != want.to(torch.float32).to(dtype)).nonzero()
        assert not len(off), (mxfp4.kernel_config(m, n, k, dtype, linear=False), len(off), off[0].tolist())


@pytest.mark.parametrize("m,n,k", [(1, 40, 288), (5, 100, 4096), (20, 130, 512), (3, 40, 10016), (70, 500, 800), (1000, 401, 2080), (40, 302, 8000)])
@pytest.mark.parametrize("low", range(9))
def test_scales_at_the_bottom(m, n, k, low):
    """Codes of any kind under scale bytes 0 .. 8 of one operand, against bytes that make the two scales' product 2^-126, near
    it and up to 1.  Relative to the scales' product the values are those of scales of 1, so the tolerance is theirs (its last
    term, fp16's smallest step, becomes the output's: bfloat16's subnormal numbers are 2^-133 apart)."""
    rng = np.random.default_rng(m * 10 + low)
    cx, cw = rng.integers(0, 16, (m, k), dtype=np.uint8), rng.integers(0, 16, (n, k), dtype=np.uint8)
    for both in (128, 129, 133, 180, 254):
        for sx, sw in ((low, both - low), (both - low, low)):
            if max(sx, sw) > 254:
                continue
            bx, bw = np.full((m, k // 32), sx, np.uint8), np.full((n, k // 32), sw, np.uint8)
            y = exact(mxfp4.matmul(tensor(cx, bx), tensor(cw, bw), torch.bfloat16))
            x, w = ref.values(cx, bx), ref.values(cw, bw)
            want = x @ w.T
            tol = (k + 8) * 2.0**-23 * (np.abs(x) @ np.abs(w).T) + 2.0**-8 * np.abs(want) + 2.0**-133
            bad = np.argwhere(~(np.abs(y - want) <= tol))
            assert not len(bad), (sx, sw, len(bad), bad[0], y[tuple(bad[0])], want[tuple(bad[0])])


@pytest.mark.parametrize("m,k", [(1, 4096), (4, 4096), (40, 512)])
def test_small_x(m, k):
    """x whose blocks get scale byte 0 (subnormal bfloat16 among them), times W with large scales: the linear layer's own quantization."""
    rng = np.random.default_rng(m)
    x = torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32) * 2.0**-126).cuda().to(torch.bfloat16)
    cw, sw = rng.integers(0, 16, (64, k), dtype=np.uint8), np.full((64, k // 32), 250, np.uint8)
    codes, scales = ref.quantize(exact(x))
    assert (scales <= 1).all() and (codes & 7).any()
    v, w = ref.values(codes, scales), ref.values(cw, sw)
    y = exact(mxfp4.linear(x, tensor(cw, sw)))
    want, tol = ref.product(v, w, 2.0**-8)
    tol = tol - 2.0**-25 + 2.0**-133
    assert bool((np.abs(y - want) <= tol).all())
