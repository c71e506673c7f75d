"""fp64 oracle of the 8-bit cache: e4m3 codes with one power-of-two scale per
vector, pages, and attention over the stored vectors.  Written from the format's
definition; numpy only."""

import numpy as np

BLOCK = 16


def _e4m3_values():
    """Value of every code: sign, 4 exponent bits (bias 7), 3 mantissa bits;
    exponent 0 is subnormal (step 2^-9), code 0x7F / 0xFF is NaN, no infinity."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = np.nan if (e, m) == (15, 7) else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        out[c] = -x if c & 128 else x
    return out


VALUES = _e4m3_values()


def e4m3_codes(x):
    """Nearest codes of |x| <= 448, ties to the even mantissa; the sign of zero is kept."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    _, e = np.frexp(np.where(a == 0, 1.0, a))  # a in [2^(e-1), 2^e)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    v = np.rint(a / step) * step
    c = np.searchsorted(VALUES[:127], v)  # the positive values ascend with the code
    assert np.array_equal(VALUES[c], v)
    return (c | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantise(x):
    """x [..., d] -> (codes uint8 [..., d], exponent bytes uint8 [...])."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x).all(-1)
    y = np.where(bad[..., None], 0.0, x)
    top = np.abs(y).max(-1)
    e = np.full(top.shape, -126.0)
    nz = top > 0
    e[nz] = np.maximum(np.ceil(np.log2(top[nz] / 448.0)), -126)
    # (log2 may round across a power of two: settle it with exact comparisons)
    e = np.where(nz & (top > 448.0 * np.exp2(e)), e + 1, e)
    e = np.where(nz & (e > -126) & (top <= 448.0 * np.exp2(e - 1)), e - 1, e)
    codes = e4m3_codes(y * np.exp2(-e)[..., None])
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8)
    return codes, np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, exps):
    """Codes and exponent bytes back to fp64 vectors."""
    s = np.where(exps == 255, np.nan, np.exp2(exps.astype(np.float64) - 127.0))
    return VALUES[codes] * s[..., None]


def parts(pages, d):
    """Views of pages uint8 [blocks, heads, 32 d + 32]: key codes and value
    codes [blocks, heads, 16, d], key and value exponents [blocks, heads, 16]."""
    nb, h, _ = pages.shape
    return (pages[:, :, :16 * d].reshape(nb, h, BLOCK, d), pages[:, :, 16 * d:32 * d].reshape(nb, h, BLOCK, d),
            pages[:, :, 32 * d:32 * d + 16], pages[:, :, 32 * d + 16:])


def store(pages, k, v, slots):
    """k, v [T, heads, d] into a copy of the pages."""
    d = k.shape[2]
    pages = pages.copy()
    for x, code_at, exp_at in ((k, 0, 32 * d), (v, 16 * d, 32 * d + 16)):
        codes, exps = quantise(x)
        for t, s in enumerate(slots):
            if s < 0 or s >= pages.shape[0] * BLOCK:
                continue
            b, r = divmod(int(s), BLOCK)
            pages[b, :, code_at + r * d:code_at + (r + 1) * d] = codes[t]
            pages[b, :, exp_at + r] = exps[t]
    return pages


def rows(pages, table_row, n, d):
    """Keys and values fp64 [n, heads, d] of one sequence."""
    kc, vc, ke, ve = parts(pages, d)
    t = np.arange(n)
    b, r = table_row[t // BLOCK], t % BLOCK
    return values(kc[b, :, r], ke[b, :, r]), values(vc[b, :, r], ve[b, :, r])


def attention(q, k, v, scale, limit=None):
    """q [n, Hq, d], k and v [m, Hkv, d] -> (out [n, Hq, d], lse [n, Hq],
    weight [n, Hq, d] = sum_t p_t |v_t|, the size of the summed terms).  Row i
    sees the first limit[i] keys (all of them by default); none: 0 and -inf."""
    n, hq, d = q.shape
    m, hkv, _ = k.shape
    out, lse, mag = np.zeros((n, hq, d)), np.full((n, hq), -np.inf), np.zeros((n, hq, d))
    limit = np.full(n, m) if limit is None else np.clip(limit, 0, m)
    for h in range(hq):
        kh, vh = k[:, h // (hq // hkv)], v[:, h // (hq // hkv)]
        z = (q[:, h] @ kh.T) * scale if m else np.zeros((n, 0))
        seen = np.arange(m)[None] < limit[:, None]
        z = np.where(seen, z, -np.inf)
        live = limit > 0
        if not live.any():
            continue
        top = z[live].max(-1, keepdims=True)
        p = np.exp(z[live] - top)
        tot = p.sum(-1, keepdims=True)
        lse[live, h] = (np.log(tot) + top)[:, 0]
        p /= tot
        # a key that is not seen contributes nothing, whatever its value is
        if np.isfinite(vh).all():
            out[live, h], mag[live, h] = p @ vh, p @ np.abs(vh)
        else:
            for i, row in enumerate(np.flatnonzero(live)):
                mm = limit[row]
                out[row, h], mag[row, h] = p[i, :mm] @ vh[:mm], p[i, :mm] @ np.abs(vh[:mm])
    return out, lse, mag
