"""Oracles of what a serving step does around the caches: norm with rotation of
query and key heads (fp64, angles reduced in exact rationals) and the plan of a
step (request by request).  numpy and the standard library only."""

from fractions import Fraction

import numpy as np

BLOCK = 16


def _two_pi(digits=60):
    """2 pi as a fraction, from 16 atan(1/5) - 4 atan(1/239)."""
    one = 10 ** (digits + 10)

    def atan_inv(n):
        s = t = one // n
        k, sign = 1, 1
        while t:
            t //= n * n
            k, sign = k + 2, -sign
            s += sign * (t // k)
        return s

    return Fraction(2 * (16 * atan_inv(5) - 4 * atan_inv(239)), one)


TWO_PI = _two_pi()


def angles(positions, inv_freq):
    """positions x inv_freq, reduced to (-pi, pi] without rounding before the last step."""
    out = np.zeros((len(positions), len(inv_freq)))
    for j, f in enumerate(inv_freq):
        turn = Fraction(float(f)) / TWO_PI
        for i, p in enumerate(positions):
            t = (turn * int(p)) % 1
            out[i, j] = float((t - 1 if 2 * t > 1 else t) * TWO_PI)
    return out


def powers(base, rot):
    return np.array([float(base) ** (-2.0 * i / rot) for i in range(rot // 2)])


def norm_rope(x, weight, positions, inv_freq, eps, interleaved=False, norm=True):
    """x [T, heads, d] -> (fp64 result, |a| + |b| of each element's pair after the norm)."""
    y = np.asarray(x, np.float64)
    d, rot = y.shape[-1], 2 * len(inv_freq)
    if norm:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        if weight is not None:
            y = y * np.asarray(weight, np.float64)
    out, size = y.copy(), np.abs(y)
    t = angles(positions, inv_freq)[:, None]
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    out[..., a] = y[..., a] * np.cos(t) - y[..., b] * np.sin(t)
    out[..., b] = y[..., b] * np.cos(t) + y[..., a] * np.sin(t)
    size[..., a] = size[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    assert size.shape[-1] == d
    return out, size


def plan(lens, new, table, free, next_free, n_tokens):
    """One step's plan, token by token: (table, slots, positions, kv_rows, seq_lens, cu_q, cu_k, next).  Packed
    keys keep a row for every new token of a request, served or not."""
    table = table.copy()
    cap = table.shape[1] * BLOCK
    slots, pos, rows = (np.full(n_tokens, x, np.int64) for x in (-1, 0, -1))
    seq, cu_q, cu_k = [], [0], [0]
    at = min(max(int(next_free), 0), len(free))
    for b, (have, n) in enumerate(zip(lens, new)):
        have, n = min(max(int(have), 0), cap), max(int(n), 0)
        t0 = cu_q[-1]
        n = min(n, n_tokens - t0)
        served = 0
        for i in range(n):
            p = have + i
            pos[t0 + i] = p
            if served < i or p >= cap:
                continue
            if p % BLOCK == 0:
                if at == len(free):
                    continue
                table[b, p // BLOCK] = free[at]
                at += 1
            block = int(table[b, p // BLOCK])
            slots[t0 + i] = block * BLOCK + p % BLOCK if block >= 0 else -1
            rows[t0 + i] = cu_k[-1] + p
            served += 1
        seq.append(have + served)
        cu_q.append(t0 + n)
        cu_k.append(cu_k[-1] + have + n)
    return table, slots, pos, rows, np.array(seq), np.array(cu_q), np.array(cu_k), at
