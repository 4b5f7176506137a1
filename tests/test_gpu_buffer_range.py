"""The range check of raw buffer loads, on which MXFP4's tiles rely: they put a stage's place in a row
into the scalar offset, end the buffer behind the tile's last row, and load stages that do not
exist from buffers of no bytes.  Every dword at or behind the end has to come as zero, the scalar
offset counted, however large it is."""
import ctypes
import os

import pytest
import torch

from w4a16_dequant_gemv_amd import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(build.TEST_LIB):
        build.build_test_kernels()
    lib = ctypes.CDLL(build.TEST_LIB)
    lib.buffer_range.argtypes = [ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_void_p]
    return lib


@pytest.mark.parametrize("records,soffset", [(512, 0), (520, 0), (1024, 512), (1000, 512), (1024, 1024), (1024, 2048), (0, 0), (0, 256),
                                             (0, 8192), (16384, 15872), (16384, 1 << 15)])
def test_scalar_offset_is_counted(L, records, soffset):
    words = torch.arange(1, (1 << 14) + 1, dtype=torch.int32, device="cuda")            # 64 KB: all that the lanes could address
    assert soffset + 1024 <= 4 * words.numel() and records <= 4 * words.numel()
    out = torch.full((256,), -1, dtype=torch.int32, device="cuda")
    assert L.buffer_range(words.data_ptr(), records, soffset, out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    at = torch.arange(256, dtype=torch.int32) + soffset // 4
    assert torch.equal(out.cpu(), torch.where(4 * at < records, at + 1, 0).int())
