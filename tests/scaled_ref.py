"""Plain implementations of the block-scaled operators for the tests: numpy, fp64 unless a step of the
definition is itself in fp32 (the NVFP4 factors)."""
import numpy as np

NV, M8, M4 = 1, 2, 3
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127])


def block(fmt):
    return 16 if fmt == NV else 32


def col_tiles(fmt, n):
    return -(-(n // block(fmt)) // 4)


def nearest(table, a):
    """Index of the table value nearest to a >= 0, ties to the even index, saturating at the last."""
    i = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    lo, hi = a - table[i - 1], table[i] - a
    return np.where((hi < lo) | ((hi == lo) & (i % 2 == 0)), i, i - 1)


def encode(fmt, v):
    """Codes of v (already divided by the scale), sign in the top bit."""
    if fmt == M8:
        return (nearest(E4M3, np.abs(v)) | np.where(np.signbit(v), 128, 0)).astype(np.uint8)
    return (nearest(E2M1, np.abs(v)) | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def decode(fmt, c):
    if fmt == M8:
        return np.where(c & 128, -1.0, 1.0) * np.append(E4M3, np.nan)[c & 127]
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def scale_value(fmt, s):
    if fmt == NV:
        return np.append(E4M3, np.nan)[s & 127]
    return np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))


def quantise(fmt, v, g=None):
    """Codes [R, n] (one a byte), scale bytes [R, n / block], row factors (fp32) of fp32 rows v."""
    v = np.asarray(v, np.float32)
    R, n = v.shape
    b = v.reshape(R, -1, block(fmt))
    amax = np.abs(b).max(2)
    if fmt == NV:
        f = np.float32
        if g is None:
            g = np.maximum(np.abs(v).max(1) * f(1 / 2688), f(2.0 ** -110))
        g = np.broadcast_to(np.asarray(g, f), (R,))
        ginv = (f(1) / g)[:, None]
        s = nearest(E4M3, (amax * ginv * f(1 / 6)).astype(np.float64)).astype(np.uint8)
        sf = E4M3[s].astype(f)
        inv = np.where(sf > 0, ginv / np.where(sf > 0, sf, f(1)), f(0)).astype(f)
        return encode(NV, (b * inv[:, :, None]).astype(np.float64)).reshape(R, n), s, g
    top, top_exp = (1.75, 8) if fmt == M8 else (1.5, 2)
    m, e = np.frexp(amax.astype(np.float64))
    e = np.where(amax > 0, np.clip(e - 1 - top_exp + (2 * m > top), -127, 127), -127)
    return encode(fmt, b.astype(np.float64) * 2.0 ** -e[:, :, None].astype(np.float64)).reshape(R, n), (e + 127).astype(np.uint8), None


def dequantise(fmt, codes, scales, g=None):
    """fp64 values of codes [..., n] (one a byte) and scale bytes [..., n / block]."""
    v = decode(fmt, codes).reshape(*scales.shape, block(fmt)) * scale_value(fmt, scales)[..., None]
    v = v.reshape(codes.shape)
    return v if g is None else v * np.asarray(g, np.float64)[..., None]


def pack(fmt, codes):
    return codes if fmt == M8 else codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(fmt, packed):
    if fmt == M8:
        return packed
    return np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def scale_index(fmt, n, rows):
    """Byte index in the tiles of every block of the given scale rows: [len(rows), n / block]."""
    r, b = np.asarray(rows)[:, None], np.arange(n // block(fmt))[None, :]
    return ((r // 128) * col_tiles(fmt, n) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def scale_rows(offsets, R):
    """Scale row of each of R grouped rows; offsets: first row of each group."""
    out = np.empty(R, np.int64)
    ends = list(offsets[1:]) + [R]
    for g, (lo, hi) in enumerate(zip(offsets, ends)):
        out[lo:hi] = (lo // 128 + g) * 128 + np.arange(hi - lo)
    return out


def tile(fmt, scales, rows, row_tiles, fill=0):
    """Tiles of scale bytes [len(rows), n / block] placed at the given scale rows."""
    n = scales.shape[1] * block(fmt)
    out = np.full(row_tiles * col_tiles(fmt, n) * 512, fill, np.uint8)
    out[scale_index(fmt, n, rows)] = scales
    return out


def weight_tiles(fmt, scales, fill=0):
    """Tiles of a stack's scale bytes [G, N, n / block]."""
    G, N, nb = scales.shape
    rt = -(-N // 128)
    rows = (np.arange(G)[:, None] * rt * 128 + np.arange(N)[None, :]).reshape(-1)
    return tile(fmt, scales.reshape(G * N, nb), rows, G * rt, fill)


def silu(x):
    return x / (1 + np.exp(-np.clip(x, -700, 700)))


def bf16(a):
    """fp32 values rounded to bf16, as fp32."""
    a = np.ascontiguousarray(a, np.float32)
    u = a.view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint32) << 16).view(np.float32)
