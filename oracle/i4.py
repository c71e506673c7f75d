"""fp64 oracle of the 4-bit cache: 4-bit integers with one scale byte for 16
elements and one exponent byte for a vector, in pages.  Written from the
format's definition; numpy only.  (Attention: oracle/f8.py's, over rows().)"""

import numpy as np

BLOCK, GROUP = 16, 16


def _scale_values():
    """Value of every scale byte: 5 exponent bits (bias 15), 3 bits behind the point; exponent 0 is
    subnormal (step 2^-17)."""
    return np.array([(u % 8) * 2.0 ** -17 if u < 8 else (1 + u % 8 / 8) * 2.0 ** (u // 8 - 15) for u in range(256)])


SCALES = _scale_values()


def quantise(x):
    """x [..., d] -> (codes 0..15 uint8 [..., d], scale bytes [..., d/16], exponent bytes [...])."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    top = np.abs(x).max(-1)
    e = np.ones(top.shape)
    nz = top > 0
    e[nz] = np.maximum(1, np.ceil(np.log2(top[nz] / 240.0)) + 127)
    # (log2 may round across a power of two: settle it with exact comparisons)
    e = np.where(top > 240.0 * np.exp2(e - 127), e + 1, e)
    e = np.where((e > 1) & (top <= 240.0 * np.exp2(e - 128)), e - 1, e)
    y = (x * np.exp2(127 - e)[..., None]).reshape(*x.shape[:-1], -1, GROUP)
    g = np.abs(y).max(-1)
    fits = g[..., None] <= 7.5 * SCALES[1:161]
    assert fits[..., -1].all()
    u = np.where(g <= 2.0 ** -18, 0, 1 + fits.argmax(-1))
    s = np.where(u > 0, SCALES[u], 1.0)[..., None]
    n = np.where(u[..., None] > 0, np.clip(np.rint(y / s), -7, 7), 0) + 8
    return n.reshape(x.shape).astype(np.uint8), u.astype(np.uint8), np.where(bad, 255, e).astype(np.uint8)


def values(codes, scales, exps):
    """Codes, scale bytes and exponent bytes back to fp64 vectors."""
    s = np.where(exps == 255, np.nan, np.exp2(exps.astype(np.float64) - 127.0))
    return (codes.astype(np.float64) - 8) * np.repeat(SCALES[scales], GROUP, -1) * s[..., None]


def parts(pages, d):
    """Views of pages uint8 [blocks, heads, 18 d + 32]: (packed codes, scales, exponents) of keys and of values."""
    nb, h, _ = pages.shape
    cut = lambda at, w: pages[:, :, at:at + 16 * w].reshape(nb, h, BLOCK, w)  # noqa: E731
    return [(cut(8 * d * i, d // 2), cut(16 * d + d * i, d // 16), pages[:, :, 18 * d + 16 * i:18 * d + 16 * (i + 1)])
            for i in (0, 1)]


def store(pages, k, v, slots):
    """k, v [T, heads, d] into a copy of the pages."""
    d = k.shape[2]
    pages = pages.copy()
    for i, x in enumerate((k, v)):
        codes, scales, exps = quantise(x)
        packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
        for t, s in enumerate(slots):
            if s < 0 or s >= pages.shape[0] * BLOCK:
                continue
            b, r = divmod(int(s), BLOCK)
            for at, w, y in ((8 * d * i, d // 2, packed), (16 * d + d * i, d // 16, scales)):
                pages[b, :, at + r * w:at + (r + 1) * w] = y[t]
            pages[b, :, 18 * d + 16 * i + r] = exps[t]
    return pages


def rows(pages, table_row, n, d):
    """Keys and values fp64 [n, heads, d] of one sequence."""
    t = np.arange(n)
    b, r = table_row[t // BLOCK], t % BLOCK
    both = []
    for packed, scales, exps in parts(pages, d):
        p = packed[b, :, r]
        codes = np.stack([p & 15, p >> 4], -1).reshape(*p.shape[:-1], d)
        both.append(values(codes, scales[b, :, r], exps[b, :, r]))
    return both
