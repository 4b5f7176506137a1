"""MXFP4's refusals, through the C ABI (every call carries an invalid argument, so nothing
is launched) and through the Python wrappers, and its definition in `mx4_ref`."""
import os
import re

import numpy as np
import pytest
import torch

import mx4_ref as ref
from mx4_ref import KERNELS
from w4a16_dequant_gemv_amd import _lib, mxfp4
from w4a16_dequant_gemv_amd._lib import Q4_ERR_ALIGN, Q4_ERR_NULL, Q4_ERR_SHAPE, W4A16Error

P = 0x10000
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def test_every_declared_symbol_is_exported(L):
    text = open(os.path.join(ROOT, "include", "mxfp4.h"), encoding="utf-8").read()
    names = set(re.findall(r"^\s*(?:int64_t|int)\s*(mx4_\w+)\s*\(", text, re.M))
    assert names == set(_lib.MX4_SIGNATURES)
    for n in names:
        assert hasattr(L, n)


def quantize(L, **kw):
    a = dict(x=P, type=0, rows=3, k=64, stride=64, codes=P, scales=P)
    a.update(kw)
    return L.mx4_quantize(a["x"], a["type"], a["rows"], a["k"], a["stride"], a["codes"], a["scales"], None)


def dequantize(L, **kw):
    a = dict(codes=P, scales=P, rows=3, k=64, type=0, out=P)
    a.update(kw)
    return L.mx4_dequantize(a["codes"], a["scales"], a["rows"], a["k"], a["type"], a["out"], None)


def matmul(L, **kw):
    a = dict(xc=P, xs=P, wc=P, ws=P, m=3, n=5, k=64, type=0, space=None, size=0, y=P)
    a.update(kw)
    return L.mx4_matmul(a["xc"], a["xs"], a["wc"], a["ws"], a["m"], a["n"], a["k"], a["type"], a["space"],
                        a["size"], a["y"], None)


def linear(L, **kw):
    a = dict(x=P, type=0, stride=4096, wc=P, ws=P, m=40, n=5, k=4096, space=P, size=1 << 20, y=P)
    a.update(kw)
    return L.mx4_linear(a["x"], a["type"], a["stride"], a["wc"], a["ws"], a["m"], a["n"], a["k"], a["space"], a["size"],
                        a["y"], None)


@pytest.mark.parametrize("call,bad,code", [
    (quantize, dict(x=None), Q4_ERR_NULL), (quantize, dict(codes=None), Q4_ERR_NULL), (quantize, dict(scales=None), Q4_ERR_NULL),
    (quantize, dict(type=3), Q4_ERR_SHAPE), (quantize, dict(type=-1), Q4_ERR_SHAPE), (quantize, dict(rows=0), Q4_ERR_SHAPE),
    (quantize, dict(rows=-5), Q4_ERR_SHAPE), (quantize, dict(rows=1 << 25), Q4_ERR_SHAPE), (quantize, dict(k=0), Q4_ERR_SHAPE),
    (quantize, dict(k=48), Q4_ERR_SHAPE), (quantize, dict(k=1 << 21, stride=1 << 21), Q4_ERR_SHAPE),
    (quantize, dict(rows=1 << 24, k=1 << 20, stride=1 << 20), Q4_ERR_SHAPE), (quantize, dict(stride=56), Q4_ERR_SHAPE),
    (quantize, dict(stride=66), Q4_ERR_SHAPE), (quantize, dict(stride=68), Q4_ERR_SHAPE),
    (quantize, dict(stride=1 << 60), Q4_ERR_SHAPE), (quantize, dict(type=2, stride=66), Q4_ERR_SHAPE),
    (quantize, dict(x=P + 8), Q4_ERR_ALIGN), (quantize, dict(codes=P + 8), Q4_ERR_ALIGN), (quantize, dict(scales=P + 4), Q4_ERR_ALIGN),
    (dequantize, dict(codes=None), Q4_ERR_NULL), (dequantize, dict(scales=None), Q4_ERR_NULL), (dequantize, dict(out=None), Q4_ERR_NULL),
    (dequantize, dict(type=3), Q4_ERR_SHAPE), (dequantize, dict(k=33), Q4_ERR_SHAPE), (dequantize, dict(rows=0), Q4_ERR_SHAPE),
    (dequantize, dict(out=P + 8), Q4_ERR_ALIGN), (dequantize, dict(codes=P + 4), Q4_ERR_ALIGN), (dequantize, dict(scales=P + 4), Q4_ERR_ALIGN),
    (matmul, dict(xc=None), Q4_ERR_NULL), (matmul, dict(xs=None), Q4_ERR_NULL), (matmul, dict(wc=None), Q4_ERR_NULL),
    (matmul, dict(ws=None), Q4_ERR_NULL), (matmul, dict(y=None), Q4_ERR_NULL), (matmul, dict(type=2), Q4_ERR_SHAPE),
    (matmul, dict(m=0), Q4_ERR_SHAPE), (matmul, dict(n=0), Q4_ERR_SHAPE), (matmul, dict(n=1 << 25), Q4_ERR_SHAPE),
    (matmul, dict(k=40), Q4_ERR_SHAPE), (matmul, dict(m=1 << 20, n=1 << 20), Q4_ERR_SHAPE), (matmul, dict(xc=P + 8), Q4_ERR_ALIGN),
    (matmul, dict(xs=P + 4), Q4_ERR_ALIGN), (matmul, dict(wc=P + 8), Q4_ERR_ALIGN), (matmul, dict(ws=P + 4), Q4_ERR_ALIGN),
    (matmul, dict(y=P + 1), Q4_ERR_ALIGN), (matmul, dict(m=64, k=28672), Q4_ERR_NULL),
    (matmul, dict(m=64, k=28672, space=P, size=16384), Q4_ERR_SHAPE), (matmul, dict(m=64, k=28672, space=P + 8, size=1 << 24), Q4_ERR_ALIGN),
    (linear, dict(x=None), Q4_ERR_NULL), (linear, dict(wc=None), Q4_ERR_NULL), (linear, dict(ws=None), Q4_ERR_NULL),
    (linear, dict(space=None), Q4_ERR_NULL), (linear, dict(y=None), Q4_ERR_NULL), (linear, dict(type=2), Q4_ERR_SHAPE),
    (linear, dict(m=0), Q4_ERR_SHAPE), (linear, dict(k=16, stride=16), Q4_ERR_SHAPE), (linear, dict(stride=4064), Q4_ERR_SHAPE),
    (linear, dict(stride=4100), Q4_ERR_SHAPE), (linear, dict(size=16), Q4_ERR_SHAPE), (linear, dict(size=-1), Q4_ERR_SHAPE),
    (linear, dict(x=P + 2), Q4_ERR_ALIGN), (linear, dict(wc=P + 8), Q4_ERR_ALIGN), (linear, dict(ws=P + 4), Q4_ERR_ALIGN),
    (linear, dict(space=P + 8), Q4_ERR_ALIGN), (linear, dict(y=P + 1), Q4_ERR_ALIGN)])
def test_refusals(L, call, bad, code):
    assert call(L, **bad) == code


def test_workspace_size(L):
    for bad in ((0, 5, 64), (3, 0, 64), (3, 5, 0), (3, 5, 48), (-1, 5, 64), (1 << 25, 5, 64)):
        assert L.mx4_linear_workspace_size(*bad) == 0 and L.mx4_matmul_workspace_size(*bad) == 0
    for m, n, k in ((17, 100, 4096), (33, 5, 288), (2048, 11008, 4096)):
        size = mxfp4.workspace_size(m, n, k)
        assert size >= m * k // 2 + -(-k // 256) * 8 * m
        assert linear(L, m=m, n=n, k=k, stride=k, size=size - 1) == Q4_ERR_SHAPE
        assert linear(L, m=m, n=n, k=k, stride=k, space=None) == Q4_ERR_NULL
    assert mxfp4.workspace_size(1, 4096, 4096) == 0          # quantized on the way
    assert mxfp4.workspace_size(2048, 11008, 4096, linear=False) == 0
    parts = mxfp4.workspace_size(64, 300, 28672, linear=False)
    assert parts >= 2 * 64 * 300 * 4 and mxfp4.workspace_size(64, 300, 28672) >= parts + 64 * 28672 * 17 // 32


def test_config_reports_every_kernel(L):
    """Each kernel that the rules can choose, at sizes that the GPU tests run."""
    names = {mxfp4.kernel_config(m, n, k, linear=linear) for m, n, k in KERNELS for linear in (True, False)}
    for want in ("mx4_rows_kernel<0, 1, 0, 2>", "mx4_rows_kernel<0, 1, 0, 4>", "mx4_quantize_kernel<0>, mx4_rows_kernel<0, 1, -1, 2>",
                 "mx4_quantize_kernel<0>, mx4_rows_kernel<0, 1, -1, 4>", "mx4_rows_kernel<0, 2, -1, 2>", "mx4_rows_kernel<0, 2, 0, 2>", "mx4_tile_kernel<0, 1, 1, 4, false>", "mx4_tile_kernel<0, 2, 1, 3, false>",
                 "mx4_tile_kernel<0, 2, 2, 3, false>", "mx4_tile_kernel<0, 2, 2, 2, false>", "mx4_tile_kernel<0, 3, 4, 2, false>",
                 "mx4_tile_kernel<0, 4, 4, 2, false>", "mx4_tile_kernel<0, 1, 1, 4, true>, mx4_join_kernel<0>"):
        assert want in names, want
    assert mxfp4.kernel_config(1, 64, 64, torch.bfloat16) == "mx4_rows_kernel<1, 1, 1, 2>"
    buf = __import__("ctypes").create_string_buffer(8)
    assert L.mx4_linear_config(1, 64, 64, 0, 1, None, 8) == Q4_ERR_NULL
    for bad in ((0, 64, 64, 0), (1, 64, 48, 0), (1, 64, 64, 2), (1, 1 << 25, 64, 0)):
        assert L.mx4_linear_config(*bad, 1, buf, 8) == Q4_ERR_SHAPE
    assert L.mx4_linear_config(1, 64, 64, 0, 1, buf, 0) == Q4_ERR_SHAPE
    assert L.mx4_linear_config(1, 64, 64, 0, 1, buf, 8) == 0 and buf.value == b"mx4_row"


def test_python_refuses():
    c, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((1, 4, 8), dtype=torch.uint8)
    q = mxfp4.MXTensor(c, s)
    for f in (lambda: mxfp4.quantize(torch.zeros(4, 64)), lambda: mxfp4.dequantize(q), lambda: mxfp4.matmul(q, q),
              lambda: mxfp4.linear(torch.zeros((4, 64), dtype=torch.float16), q), lambda: mxfp4.dequantize(c),
              lambda: mxfp4.MXTensor.from_blocks(c, torch.zeros((4, 3), dtype=torch.uint8)),
              lambda: mxfp4.MXTensor.from_blocks(c[:, :0], torch.zeros((4, 0), dtype=torch.uint8)),
              lambda: mxfp4.MXTensor.from_blocks(c.int(), torch.zeros((4, 2), dtype=torch.uint8)),
              lambda: mxfp4.MXTensor.from_blocks(c[:, :24], torch.zeros((4, 1), dtype=torch.uint8))):
        with pytest.raises(W4A16Error):
            f()


@pytest.mark.parametrize("rows,k", [(0, 32), (0, 512), (1, 32), (3, 256), (5, 288), (7, 11008)])
def test_order_of_scales(rows, k):
    rng = np.random.default_rng(k)
    s = rng.integers(0, 256, (rows, k // 32), dtype=np.uint8)
    q = mxfp4.MXTensor.from_blocks(torch.zeros((rows, k // 2), dtype=torch.uint8), torch.from_numpy(s))
    assert np.array_equal(q.scales.numpy(), ref.laid(s))
    assert np.array_equal(q.block_scales().numpy(), s)
    assert q.rows == rows and q.k == k and q.nbytes() == rows * k // 2 + q.scales.numel()


def test_reference_by_hand():
    """A block with every element, halves between them, and what is beyond the largest."""
    x = np.zeros((1, 32))
    x[0, :16] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, 0.26, 0.74, 1.74, 2.49, 3.49, 4.99, -7.5]
    codes, scales = ref.quantize(x)
    assert scales[0, 0] == 127
    assert ref.values(codes, scales)[0, :16].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 0, 0.5, 0.5, 1.5, 2, 3, 4, -6]
    codes, scales = ref.quantize(np.ldexp(x, 5))
    assert scales[0, 0] == 132 and np.array_equal(ref.values(codes, scales), np.ldexp(ref.values(*ref.quantize(x)), 5))
    assert np.array_equal(ref.unpack(ref.pack(codes)), codes)
