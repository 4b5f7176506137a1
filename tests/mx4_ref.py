"""MXFP4 from its definition, in 64 bits with numpy: codes and scales of a matrix, the
values that they stand for, and products with the error that a kernel may have."""
import numpy as np

# Sizes (m, n_out, k) that between them are run by every kernel of the product.
KERNELS = [(1, 40, 288), (1, 100, 8160), (5, 100, 4096), (3, 40, 10016), (16, 256, 8192), (20, 130, 512), (20, 100, 2048), (70, 500, 800), (700, 3000, 544),
           (1000, 4001, 2080), (1111, 6000, 544), (2000, 6001, 544), (2050, 5003, 1056), (2000, 8101, 800), (40, 302, 8000), (100, 70, 28640),
           (64, 4096, 11008)]

VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def quantize(x):
    """x [rows, k] float64 (exact values of the input) -> codes uint8 [rows, k], scales uint8 [rows, k / 32]."""
    rows, k = x.shape
    y = x.reshape(rows, k // 32, 32)
    mag = np.abs(y)
    top = mag.max(-1)
    ok = np.isfinite(top)
    e = np.where(ok & (top > 0), np.frexp(np.where(ok, top, 1))[1] - 1 - 2, -127).clip(-127)
    a = np.ldexp(np.where(ok[..., None], mag, 0), -e[..., None])
    # the nearest value; from two as near the one with an even code
    d = np.abs(a[..., None] - VALUES) * 4 + (np.arange(8) % 2) * 2.0**-40
    code = np.where(a >= 6, 7, d.argmin(-1)).astype(np.uint8) | (np.signbit(y) << 3).astype(np.uint8)
    return code.reshape(rows, k), np.where(ok, e + 127, 255).astype(np.uint8)


def values(codes, scales):
    """codes [rows, k], scales [rows, k / 32] -> float64 [rows, k]."""
    rows, k = codes.shape
    v = VALUES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v.reshape(rows, k // 32, 32) * s[..., None]).reshape(rows, k)


def pack(codes):
    return codes[:, ::2] | codes[:, 1::2] << 4


def unpack(b):
    return np.stack((b & 15, b >> 4), -1).reshape(b.shape[0], 2 * b.shape[1])


def laid(scales):
    """[rows, k / 32] in the library's order [ceil(k / 256)][rows][8]."""
    rows, blocks = scales.shape
    s = np.zeros((rows, -(-blocks // 8) * 8), np.uint8)
    s[:, :blocks] = scales
    return np.ascontiguousarray(s.reshape(rows, -(-blocks // 8), 8).transpose(1, 0, 2))


def product(x, w, half_step):
    """x [m, k], w [n, k] float64 -> (x w^T, how far a kernel may be off): an addition in
    binary32, rounded or cut, loses less than 2^-23 of the largest partial sum, of which there are
    fewer than k + 8 (four bits of them joined at the end), then the output's own rounding."""
    y = x @ w.T
    return y, (x.shape[1] + 8) * 2.0**-23 * (np.abs(x) @ np.abs(w).T) + half_step * np.abs(y) + 2.0**-25
