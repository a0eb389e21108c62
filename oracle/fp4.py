"""CPU oracle of the microscaled 4-bit floats (test infrastructure, NumPy).

Written from the definitions in ``include/eqat.h``: blocks, scales, codes and values, by
search for the nearest grid value in fp64 of the fp32 quantities that the definition
names.
"""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = {"mx": 32, "nv": 16}


def e4m3_values():
    """The 127 finite values of the e4m3 codes 0x00 .. 0x7E."""
    v = []
    for c in range(0x7F):
        e, m = c >> 3, c & 7
        v.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


def nearest(a, grid):
    """Index of the nearest value of an ascending grid for a >= 0, ties to the even index."""
    a = np.asarray(a, np.float64)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    return np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))


def tensor_scale(W):
    a = np.abs(np.asarray(W, np.float64))
    a = a[np.isfinite(a)]
    amax = a.max() if a.size else 0.0
    e = -100
    while e < 100 and amax > 2688.0 * 2.0 ** e:
        e += 1
    return np.float32(2.0 ** e)


def quantize(W, fmt, g=None):
    """(codes [N, K] in 0..15, scale bytes [N, G], values fp64 [N, K]) of fp32 W."""
    W = np.asarray(W, np.float32)
    N, K = W.shape
    b = BLOCK[fmt]
    x = W.reshape(N, K // b, b)
    with np.errstate(over="ignore", invalid="ignore"):
        if fmt == "nv":
            g = np.float32(1.0 if g is None else g)
            x = x * (np.float32(1.0) / g)
        bad = ~np.isfinite(x).all(2)
        amax = np.where(bad, np.float32(0), np.abs(x).max(2))
    if fmt == "nv":
        byte = nearest((amax / np.float32(6.0)).astype(np.float64), e4m3_values())
        s = e4m3_values()[byte]
        out = (s.astype(np.float32) * g).astype(np.float64)
        nan = 0x7F
    else:
        with np.errstate(divide="ignore"):
            e = np.where(amax > 0, np.frexp(amax.astype(np.float64))[1] - 3, -127)
        byte = np.maximum(e, -127) + 127
        s = 2.0 ** (byte - 127.0)
        out = s
        nan = 0xFF
    safe = np.where(s > 0, s, 1.0)[..., None]
    with np.errstate(invalid="ignore"):
        mag = np.where(s[..., None] > 0, np.abs(x).astype(np.float64) / safe, 0.0)
    mag = np.where(bad[..., None], 0.0, mag)
    code = nearest(mag, GRID) + 8 * (np.signbit(x) & ~bad[..., None])
    val = np.where(code >= 8, -1.0, 1.0) * GRID[code % 8] * out[..., None]
    val = np.where(bad[..., None], np.nan, val)
    return code.reshape(N, K), np.where(bad, nan, byte), val.reshape(N, K)


def tiles(scale_bytes):
    """Scale bytes [N, G] as the tiles [ceil(N/128), ceil(G/4), 512] (padding 0)."""
    N, G = scale_bytes.shape
    out = np.zeros((-(-N // 128), -(-G // 4), 512), np.uint8)
    for r in range(N):
        for j in range(G):
            out[r // 128, j // 4, 16 * (r % 32) + 4 * ((r % 128) // 32) + j % 4] = scale_bytes[r, j]
    return out


def pack(codes):
    """Codes [N, K] -> bytes [N, K/2]."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
