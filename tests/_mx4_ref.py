"""The microscaled 4-bit format from its definition, in numpy and 64 bits: used by the tests alone."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantise(x, rand=None):
    """(codes uint8 [rows, blocks, 32], scale bytes int [rows, blocks]) of the rows of x (float64 values of any type)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = -(-cols // 32)
    b = np.zeros((rows, nb * 32))
    b[:, :cols] = x
    b = b.reshape(rows, nb, 32)
    bad = ~np.isfinite(b).all(2)
    a = np.where(bad[..., None], 0.0, np.abs(b))
    top = a.max(2)
    e = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127)  # floor(log2 top) - 2
    e = np.maximum(e, -127)
    if rand is not None:
        e = e + (np.ldexp(top, -e) > 6)
    t = np.ldexp(a, -e[..., None])
    code = np.zeros(t.shape, np.int64)
    if rand is None:
        for i in range(7):
            mid = (GRID[i] + GRID[i + 1]) / 2
            code += (t > mid) if i % 2 == 0 else (t >= mid)  # a tie goes to the even code
    else:
        r = np.zeros((rows, nb * 32))
        r[:, :cols] = rand
        r = r.reshape(t.shape)
        for i in range(7):
            code += (t - GRID[i]) / (GRID[i + 1] - GRID[i]) > (255.5 - r) / 256
    code = code | (np.signbit(b).astype(np.int64) << 3)
    code[bad] = 0
    return code.astype(np.uint8), np.where(bad, 255, e + 127)


def values(code, byte, cols):
    """The float64 matrix that codes and scale bytes stand for."""
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    v = np.where(byte[..., None] == 255, np.nan, np.ldexp(v, byte[..., None] - 127))
    return v.reshape(code.shape[0], -1)[:, :cols]


def layout(code, byte):
    """The bytes of the matrix as include/zr.h states them, element by element of the statement."""
    rows, nb = byte.shape
    tr, tc = -(-rows // 128), -(-nb * 32 // 256)
    out = np.zeros((tr, tc, 17408), np.uint8)
    r, j = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    ri, ji = r % 128, j % 8
    at = ri * 128 + (ji ^ (ri % 8)) * 16
    two = code[..., 0::2] | (code[..., 1::2] << 4)
    for k in range(16):
        out[r // 128, j // 8, at + k] = two[..., k]
    out[r // 128, j // 8, 16384 + (ji // 4) * 512 + (ri % 32) * 16 + (ri // 32) * 4 + ji % 4] = byte
    return out.reshape(-1)


def rounding(dtype, y):
    """Half a unit in the last place of a torch type at the magnitudes y: what one rounding to it may cost."""
    bits, low = {"torch.float32": (24, -126), "torch.bfloat16": (8, -126), "torch.float16": (11, -14)}[str(dtype)]
    e = np.maximum(np.frexp(np.abs(y))[1] - 1, low)
    return np.ldexp(1.0, e - bits)
