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

import torch

from ._lib import W4A16Error, check, lib
from .api import _need, _raw_stream, _same_device

BLOCK = 32                              # elements that share a scale
_TYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


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
        return self.scales.permute(1, 0, 2).reshape(self.rows, -1)[:, :self.k // BLOCK].contiguous()

    @classmethod
    def from_blocks(cls, codes, block_scales):
        """Codes [rows, k // 2] and scales [rows, k // 32] as a checkpoint has them."""
        if not isinstance(codes, torch.Tensor) or codes.dim() != 2 or codes.dtype != torch.uint8:
            raise W4A16Error("codes must be uint8 [rows, k // 2]")
        rows, blocks = codes.shape[0], codes.shape[1] // (BLOCK // 2)
        if not isinstance(block_scales, torch.Tensor) or block_scales.dtype != torch.uint8 or \
                codes.shape[1] % (BLOCK // 2) or block_scales.shape != (rows, blocks):
            raise W4A16Error("block_scales must be uint8 [rows, k // 32], k a multiple of 32")
        s = torch.nn.functional.pad(block_scales, (0, -blocks % 8))
        return cls(codes.contiguous(), s.view(rows, -1, 8).transpose(0, 1).contiguous())


def _scale_shape(rows, k):
    return -(-k // 256), rows, 8


def _check(q, name):
    """Raise unless q is an MXTensor whose tensors fit each other, and are on one GPU."""
    if not isinstance(q, MXTensor):
        raise W4A16Error(f"{name} must be an MXTensor")
    c, s = q.codes, q.scales
    if not (isinstance(c, torch.Tensor) and c.is_cuda and c.dtype is torch.uint8 and c.dim() == 2 and c.is_contiguous()
            and c.shape[1] and not c.shape[1] % (BLOCK // 2)):
        raise W4A16Error(f"{name}.codes must be a contiguous uint8 GPU tensor [rows, k // 2], k a multiple of {BLOCK}")
    shape = _scale_shape(c.shape[0], c.shape[1] * 2)
    if not (isinstance(s, torch.Tensor) and s.dtype is torch.uint8 and s.shape == shape and s.device == c.device
            and s.is_contiguous()):
        _need(s, torch.uint8, shape, f"{name}.scales")
        raise W4A16Error("all tensors must be on the same GPU")


def _rows_of(x, types):
    """The row stride of x [rows, k], whose rows may be further apart than k."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise W4A16Error("x must be a GPU tensor (there is no CPU implementation)")
    if x.dtype not in types:
        raise W4A16Error(f"x must be one of {', '.join(str(t) for t in types)}, got {x.dtype}")
    if x.dim() != 2 or x.shape[1] % BLOCK or not x.shape[1]:
        raise W4A16Error(f"x must be [rows, k], k a multiple of {BLOCK}, got {tuple(x.shape)}")
    row, one = x.stride()
    if one != 1:
        raise W4A16Error("the elements of a row of x must lie side by side")
    return row if x.shape[0] > 1 else x.shape[1]


def _call(name, device, *args):
    """A library call on torch's current stream of that GPU, made the current one."""
    fn = getattr(lib(), name)
    gpu = device.index
    stream = _raw_stream(gpu)
    if torch.cuda.current_device() == gpu:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(gpu):
            rc = fn(*args, stream)
    if rc:
        check(rc, name)


def _output(out, shape, dtype, like):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _need(out, dtype, shape, "out")
    _same_device(like, out)
    return out


def quantize(x, out=None):
    """fp16, bf16 or fp32 x [rows, k] -> MXTensor, bit-exact.  Rows may be further
    apart than k (a view into a fused projection's output), a multiple of 16 bytes."""
    stride = _rows_of(x, _TYPES)
    rows, k = x.shape
    if out is None:
        out = MXTensor(torch.empty((rows, k // 2), dtype=torch.uint8, device=x.device),
                       torch.empty(_scale_shape(rows, k), dtype=torch.uint8, device=x.device))
    else:
        _check(out, "out")
        _need(out.codes, torch.uint8, (rows, k // 2), "out.codes")
        _same_device(x, out.codes)
    if rows:
        _call("mx4_quantize", x.device, x.data_ptr(), _TYPES[x.dtype], rows, k, stride, out.codes.data_ptr(),
              out.scales.data_ptr())
    return out


def dequantize(q, dtype=torch.float32, out=None):
    """MXTensor -> its values [rows, k] in fp32, fp16 or bf16, rounded once where the
    type does not hold them."""
    _check(q, "q")
    if dtype not in _TYPES:
        raise W4A16Error(f"dtype must be float32, float16 or bfloat16, got {dtype}")
    out = _output(out, (q.rows, q.k), dtype, q.codes)
    if q.rows:
        _call("mx4_dequantize", out.device, q.codes.data_ptr(), q.scales.data_ptr(), q.rows, q.k, _TYPES[dtype],
              out.data_ptr())
    return out


def matmul(x, w, dtype=torch.float16, out=None):
    """y = x W^T of MXTensors x [m, k] and w [n_out, k], fp16 or bf16 [m, n_out]."""
    _check(x, "x")
    _check(w, "w")
    if x.k != w.k:
        raise W4A16Error(f"x has rows of {x.k} elements, w of {w.k}")
    _same_device(x.codes, w.codes)
    if dtype not in (torch.float16, torch.bfloat16):
        raise W4A16Error(f"dtype must be float16 or bfloat16, got {dtype}")
    out = _output(out, (x.rows, w.rows), dtype, x.codes)
    if x.rows and w.rows:
        _call("mx4_matmul", out.device, x.codes.data_ptr(), x.scales.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(),
              x.rows, w.rows, x.k, _TYPES[dtype], out.data_ptr())
    return out


def linear(x, w, out=None, workspace=None):
    """y = Q(x) W^T: fp16 or bf16 x [m, k] quantized to MXFP4 by rows of 32, times the
    MXTensor w [n_out, k]; y [m, n_out] has x's type.  workspace: at least
    workspace_size(m, k) bytes on the GPU, 16-byte aligned, for programs that keep one."""
    stride = _rows_of(x, (torch.float16, torch.bfloat16))
    _check(w, "w")
    m, k = x.shape
    if k != w.k:
        raise W4A16Error(f"x has rows of {k} elements, w of {w.k}")
    _same_device(x, w.codes)
    out = _output(out, (m, w.rows), x.dtype, x)
    if m == 0 or w.rows == 0:
        return out
    if workspace is None:
        workspace = torch.empty(workspace_size(m, k), dtype=torch.uint8, device=x.device)
    elif not isinstance(workspace, torch.Tensor) or workspace.device != x.device or not workspace.is_contiguous():
        raise W4A16Error("workspace must be a contiguous tensor on x's GPU")
    _call("mx4_linear", x.device, x.data_ptr(), _TYPES[x.dtype], stride, w.codes.data_ptr(), w.scales.data_ptr(), m,
          w.rows, k, workspace.data_ptr(), workspace.numel() * workspace.element_size(), out.data_ptr())
    return out


def kernel_config(m, n_out, k, dtype=torch.float16, linear=True):
    """Names of the kernels that `linear` (or `matmul`) launches for these sizes, as
    profilers print them.  Nothing is launched; works without a GPU."""
    if dtype not in (torch.float16, torch.bfloat16):
        raise W4A16Error(f"dtype must be float16 or bfloat16, got {dtype}")
    name = create_string_buffer(128)
    check(lib().mx4_linear_config(m, n_out, k, _TYPES[dtype], 1 if linear else 0, name, len(name)), "mx4_linear_config")
    return name.value.decode()


def workspace_size(m, k):
    """Bytes of `linear`'s workspace for x [m, k]."""
    return lib().mx4_linear_workspace_size(m, k)
