"""torch-facing wrappers over the MXFP4 entry points of libw4a16.so
(`include/mxfp4.h`): quantization of weights and activations to microscaled 4-bit
floating point, the way back, and the product of two quantized operands on the matrix
cores that take them as they are.

    w = mxfp4.quantize(weight)          # once
    y = mxfp4.linear(x, w)              # quantizes x and multiplies

Only argument marshalling happens here: tensors must already live on the GPU
and the library does all of the arithmetic on torch's current stream.
"""
from ctypes import create_string_buffer
from dataclasses import dataclass
from functools import lru_cache

import torch

from ._lib import W4A16Error, check, lib
from .api import _need, _raw_stream

BLOCK = 32                              # elements that share a scale
_HALVES = {torch.float16: 0, torch.bfloat16: 1}
_TYPES = {**_HALVES, torch.float32: 2}


@dataclass
class MXTensor:
    """A matrix [rows, k] in MXFP4 (the order of mxfp4.h).

    codes: uint8 [rows, k // 2]; element 2 i of a row in the low half of byte i.
    scales: uint8 [ceil(k / 256), rows, 8]; the scale 2^(s - 127) of elements
            32 b .. 32 b + 31 of a row at [b // 8, row, b % 8].
    """
    codes: torch.Tensor
    scales: torch.Tensor

    @property
    def rows(self):
        return self.codes.shape[0]

    @property
    def k(self):
        return self.codes.shape[1] * 2

    def nbytes(self):
        return self.codes.numel() + self.scales.numel()

    def block_scales(self):
        """The scales in the order of a checkpoint, uint8 [rows, k // 32]."""
        return self.scales.permute(1, 0, 2).flatten(1)[:, :self.k // BLOCK].contiguous()

    @classmethod
    def from_blocks(cls, codes, block_scales):
        """Codes [rows, k // 2] and scales [rows, k // 32] as a checkpoint has them."""
        if not isinstance(codes, torch.Tensor) or codes.dim() != 2 or codes.dtype != torch.uint8:
            raise W4A16Error("codes must be uint8 [rows, k // 2]")
        rows, blocks = codes.shape[0], codes.shape[1] // (BLOCK // 2)
        if not isinstance(block_scales, torch.Tensor) or block_scales.dtype != torch.uint8 or \
                not blocks or codes.shape[1] % (BLOCK // 2) or block_scales.shape != (rows, blocks):
            raise W4A16Error("block_scales must be uint8 [rows, k // 32], k a multiple of 32")
        s = torch.nn.functional.pad(block_scales, (0, -blocks % 8))
        return cls(codes.contiguous(), s.view(rows, -(-blocks // 8), 8).transpose(0, 1).contiguous())


def _parts(q, name):
    """Codes, scales, rows and k of an MXTensor whose tensors fit each other and are on one GPU."""
    if not isinstance(q, MXTensor):
        raise W4A16Error(f"{name} must be an MXTensor")
    c, s = q.codes, q.scales
    if not (isinstance(c, torch.Tensor) and c.is_cuda and c.dtype is torch.uint8 and c.dim() == 2 and c.is_contiguous()):
        raise W4A16Error(f"{name}.codes must be a contiguous uint8 GPU tensor [rows, k // 2]")
    rows, half = c.shape
    if not half or half % (BLOCK // 2):
        raise W4A16Error(f"{name}.codes must be [rows, k // 2], k a multiple of {BLOCK}, got {tuple(c.shape)}")
    shape = (half + 127) // 128, rows, 8
    if not (isinstance(s, torch.Tensor) and s.dtype is torch.uint8 and s.shape == shape and s.device == c.device
            and s.is_contiguous()):
        _need(s, torch.uint8, shape, f"{name}.scales")
        raise W4A16Error("all tensors must be on the same GPU")
    return c, s, rows, half * 2


def _rows_of(x, types):
    """Rows, k, row stride (they may be further apart than k) and type of x [rows, k]."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise W4A16Error("x must be a GPU tensor (there is no CPU implementation)")
    kind = types.get(x.dtype)
    if kind is None:
        raise W4A16Error(f"x must be one of {', '.join(str(t) for t in types)}, got {x.dtype}")
    if x.dim() != 2:
        raise W4A16Error(f"x must be [rows, k], got {tuple(x.shape)}")
    rows, k = x.shape
    if not k or k % BLOCK:
        raise W4A16Error(f"x must be [rows, k], k a multiple of {BLOCK}, got {tuple(x.shape)}")
    row, one = x.stride()
    if one != 1:
        raise W4A16Error("the elements of a row of x must lie side by side")
    return rows, k, row if rows > 1 else k, kind


def _output(out, like, shape, dtype):
    """`out` if it is one of these, or a new one on like's GPU."""
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    if not (isinstance(out, torch.Tensor) and out.dtype is dtype and out.shape == shape and out.device == like.device
            and out.is_contiguous()):
        _need(out, dtype, shape, "out")
        raise W4A16Error("all tensors must be on the same GPU")
    return out


def _call(name, gpu, *args):
    """A library call on torch's current stream of that GPU, made the current one."""
    fn = getattr(lib(), name)
    stream = _raw_stream(gpu)
    if torch.cuda.current_device() == gpu:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(gpu):
            rc = fn(*args, stream)
    if rc:
        check(rc, name)


def quantize(x, out=None):
    """fp16, bf16 or fp32 x [rows, k] -> MXTensor, bit-exact.  Rows may be further
    apart than k (a view into a fused projection's output), a multiple of 16 bytes."""
    rows, k, stride, kind = _rows_of(x, _TYPES)
    if out is None:
        codes = x.new_empty((rows, k // 2), dtype=torch.uint8)
        scales = x.new_empty((-(-k // 256), rows, 8), dtype=torch.uint8)
        out = MXTensor(codes, scales)
    else:
        codes, scales, *size = _parts(out, "out")
        if size != [rows, k] or codes.device != x.device:
            raise W4A16Error(f"out must be [{rows}, {k}] on x's GPU, got {size}")
    if rows:
        _call("mx4_quantize", x.get_device(), x.data_ptr(), kind, rows, k, stride, codes.data_ptr(), scales.data_ptr())
    return out


def dequantize(q, dtype=torch.float32, out=None):
    """MXTensor -> its values [rows, k] in fp32, fp16 or bf16, rounded once where the
    type does not hold them."""
    codes, scales, rows, k = _parts(q, "q")
    if dtype not in _TYPES:
        raise W4A16Error(f"dtype must be float32, float16 or bfloat16, got {dtype}")
    out = _output(out, codes, (rows, k), dtype)
    if rows:
        _call("mx4_dequantize", codes.get_device(), codes.data_ptr(), scales.data_ptr(), rows, k, _TYPES[dtype],
              out.data_ptr())
    return out


def _room(need, workspace, like):
    """(bytes, address) of the caller's workspace, or of a new one where one is needed."""
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device != like.device or not workspace.is_contiguous():
            raise W4A16Error("workspace must be a contiguous tensor on x's GPU")
        return workspace.numel() * workspace.element_size(), workspace.data_ptr(), workspace
    if not need:
        return 0, None, None
    workspace = like.new_empty(need, dtype=torch.uint8)
    return need, workspace.data_ptr(), workspace


def matmul(x, w, dtype=torch.float16, out=None, workspace=None):
    """y = x W^T of MXTensors x [m, k] and w [n_out, k], fp16 or bf16 [m, n_out].
    workspace: at least workspace_size(m, n_out, k, linear=False) bytes, as for `linear`."""
    xc, xs, m, k = _parts(x, "x")
    wc, ws, n, wk = _parts(w, "w")
    if k != wk:
        raise W4A16Error(f"x has rows of {k} elements, w of {wk}")
    if xc.device != wc.device:
        raise W4A16Error("all tensors must be on the same GPU")
    if dtype not in _HALVES:
        raise W4A16Error(f"dtype must be float16 or bfloat16, got {dtype}")
    out = _output(out, xc, (m, n), dtype)
    if m and n:
        size, at, _keep = _room(workspace_size(m, n, k, False), workspace, xc)
        _call("mx4_matmul", xc.get_device(), xc.data_ptr(), xs.data_ptr(), wc.data_ptr(), ws.data_ptr(), m, n, k,
              _HALVES[dtype], at, size, out.data_ptr())
    return out


def linear(x, w, out=None, workspace=None):
    """y = Q(x) W^T: fp16 or bf16 x [m, k] quantized to MXFP4 by rows of 32, times the
    MXTensor w [n_out, k]; y [m, n_out] has x's type.  workspace: at least
    workspace_size(m, n_out, k) bytes on the GPU, 16-byte aligned, for programs that keep
    one; calls that share it must not overlap."""
    wc, ws, n, wk = _parts(w, "w")
    m, k, stride, kind = _rows_of(x, _HALVES)
    if k != wk:
        raise W4A16Error(f"x has rows of {k} elements, w of {wk}")
    if x.device != wc.device:
        raise W4A16Error("all tensors must be on the same GPU")
    out = _output(out, x, (m, n), x.dtype)
    if m == 0 or n == 0:
        return out
    size, at, _keep = _room(workspace_size(m, n, k), workspace, wc)
    _call("mx4_linear", x.get_device(), x.data_ptr(), kind, stride, wc.data_ptr(), ws.data_ptr(), m, n, k, at, size,
          out.data_ptr())
    return out


def kernel_config(m, n_out, k, dtype=torch.float16, linear=True):
    """Names of the kernels that `linear` (or `matmul`) launches for these sizes, as
    profilers print them.  Nothing is launched; works without a GPU."""
    if dtype not in _HALVES:
        raise W4A16Error(f"dtype must be float16 or bfloat16, got {dtype}")
    name = create_string_buffer(128)
    check(lib().mx4_linear_config(m, n_out, k, _TYPES[dtype], 1 if linear else 0, name, len(name)), "mx4_linear_config")
    return name.value.decode()


@lru_cache(maxsize=4096)
def workspace_size(m, n_out, k, linear=True):
    """Bytes of `linear`'s (or `matmul`'s) workspace for x [m, k] and w [n_out, k]: room for the
    quantized x and for the sums of a long k's parts; 0 where a call needs neither."""
    return (lib().mx4_linear_workspace_size if linear else lib().mx4_matmul_workspace_size)(m, n_out, k)
