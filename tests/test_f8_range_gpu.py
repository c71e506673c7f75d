"""Decode over the 8-bit cache with scores far from zero, against the fp64 oracle."""

import numpy as np
import pytest

from oracle import f8
from test_f8_gpu import DT, _bound, _cache, _gpu, _np, _rng, _slots, _table

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _ranked(d, g, lens, kinds, size, qt, ot, seed, v_scales=(-12, 13)):
    """Decode with scores kind * about size^2 (not a power of two; scale 1) and value
    vectors of scales far apart: the mean of the values of a sequence's highest kind.
    The oracle's scores are 60 times the kind: e^-60 is nothing beside the largest."""
    rng = _rng(51, d, g, seed)
    table, blocks = _table(rng, lens)
    c = _cache(d, 1, g, blocks, len(lens), table.shape[1])
    n = sum(lens)
    kind = rng.choice(kinds, n)
    q, k = np.zeros((len(lens), g, d)), np.zeros((n, 1, d))
    q[..., 5] = size * 141 / 128
    k[:, 0, 5] = kind * size * 1.25
    v = rng.standard_normal((n, 1, d)) * 2.0 ** rng.integers(*v_scales, (n, 1, 1))
    c.store(_gpu(k, torch.float32), _gpu(v, torch.float32), _gpu(_slots(table, lens)))
    got = c.decode(_gpu(q, DT[qt]), _gpu(table), _gpu(np.array(lens, np.int32)), scale=1.0, out_dtype=DT[ot])
    assert c.device_error() == 0
    pages, gn = c.pages().cpu().numpy(), _np(got)
    q[..., 5], k[:, 0, 5] = 1, kind * 60
    at = 0
    for b, m in enumerate(lens):
        if m == 0:
            assert not gn[b].any()
            continue
        _, vb = f8.rows(pages, table[b], m, d)
        ref, _, mag = f8.attention(q[b:b + 1], k[at:at + m], vb, 1.0)
        tol = _bound(q[b:b + 1], k[at:at + m], vb, 1.0, mag, ref, "f32" in (qt, ot), got.dtype)[0]
        err = np.abs(gn[b] - ref[0])
        assert (err <= tol).all(), (b, m, err.max(), (err / tol).max())
        at += m


@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 11, 2.0 ** 13, 2.0 ** 17, 2.0 ** 45])
@pytest.mark.parametrize("d,g,lens,qt,ot", [
    (128, 4, [1, 40, 300, 0, 17], "bf16", "bf16"),
    (128, 8, [9000, 3], "f32", "f32"),
    (256, 5, [2500, 33], "bf16", "f32"),
    (256, 16, [200, 700], "bf16", "bf16"),
    (128, 2, [60] * 700, "bf16", "bf16"),     # whole units to warps
])
def test_value_scales_beside_large_scores(d, g, lens, qt, ot, size):
    for i, kinds in enumerate(([1.0], [-1.0], [-1, -1, -1, 0, 1.0])):
        _ranked(d, g, lens, kinds, size, qt, ot, i)


@pytest.mark.parametrize("size", [2.0 ** 51, 2.0 ** 60, 1.375 * 2.0 ** 62])
@pytest.mark.parametrize("d,g,lens,qt,ot", [
    (128, 4, [1, 40, 300, 0, 17], "bf16", "bf16"),
    (128, 8, [9000, 3], "f32", "f32"),
    (256, 16, [1, 700], "bf16", "f32"),
    (128, 2, [60] * 700, "bf16", "bf16"),
])
def test_scores_down_to_the_end_of_the_range(d, g, lens, qt, ot, size):
    """Every score of a sequence far below zero (2^102 .. 2^125): its values, not those of
    a sequence without a token."""
    for i, kinds in enumerate(([-1.0], [-1, -1, -0.25])):
        _ranked(d, g, lens, kinds, size, qt, ot, 10 + i)


@pytest.mark.parametrize("d,g,qt,ot", [(128, 4, "f32", "f32"), (128, 16, "bf16", "bf16"), (256, 8, "bf16", "f32")])
def test_exponent_byte_zero(d, g, qt, ot):
    """Pages that something else filled: the byte 0 is 2^-127 for keys, too."""
    rng = _rng(52, d, g)
    lens = [70, 5, 400]
    table, blocks = _table(rng, lens)
    c = _cache(d, 1, g, blocks, len(lens), table.shape[1])
    n = sum(lens)
    k, v = rng.standard_normal((n, 1, d)), rng.standard_normal((n, 1, d))
    slots = _slots(table, lens)
    c.store(_gpu(k, torch.float32), _gpu(v, torch.float32), _gpu(slots))
    host = c.pages().cpu().numpy()
    f8.parts(host, d)[2][slots // 16, 0, slots % 16] = rng.integers(0, 3, n)
    c.pages().copy_(_gpu(host))
    q = torch.from_numpy(rng.standard_normal((len(lens), g, d)) * 2.0 ** 121).to(DT[qt])
    got = c.decode(q.cuda(), _gpu(table), _gpu(np.array(lens, np.int32)), out_dtype=DT[ot])
    assert c.device_error() == 0
    for b, m in enumerate(lens):
        kb, vb = f8.rows(host, table[b], m, d)
        args = _np(q)[b:b + 1], kb, vb, 1 / np.sqrt(d)
        ref, _, mag = f8.attention(*args)
        tol = _bound(*args, mag, ref, "f32" in (qt, ot), got.dtype)[0]
        err = np.abs(_np(got)[b] - ref[0])
        assert (err <= tol).all(), (b, err.max(), (err / tol).max())


@pytest.mark.parametrize("d,hkv,g", [(128, 8, 1), (256, 4, 2), (128, 4, 12)])
def test_long_sums_are_rounded_not_cut_off(d, hkv, g):
    """fp32, positive values, many steps per warp: the outputs are right on average.
    What is rounded to nearest leaves no mean error; a tensor-core product may lose up to
    2^-23 of its own sum, and at most four are added up before the next rounding."""
    rng = _rng(53, d, g)
    lens = [40000, 39999]
    table, blocks = _table(rng, lens)
    c = _cache(d, hkv, hkv * g, blocks, 2, table.shape[1])
    n = sum(lens)
    gen = torch.Generator("cuda").manual_seed(53)
    k = torch.randn((n, hkv, d), generator=gen, device="cuda")
    v = torch.rand((n, hkv, d), generator=gen, device="cuda") + 0.5
    c.store(k, v, _gpu(_slots(table, lens)))
    q = torch.randn((2, hkv * g, d), generator=gen, device="cuda")
    got = _np(c.decode(q, _gpu(table), _gpu(np.array(lens, np.int32))))
    assert c.device_error() == 0
    pages = c.pages().cpu().numpy()
    for b, m in enumerate(lens):
        kb, vb = f8.rows(pages, table[b], m, d)
        ref, _, mag = f8.attention(_np(q)[b:b + 1], kb, vb, 1 / np.sqrt(d))
        tol = _bound(_np(q)[b:b + 1], kb, vb, 1 / np.sqrt(d), mag, ref, True, torch.float32)[0]
        assert (np.abs(got[b] - ref[0]) <= tol).all()
        mean = ((got[b] - ref[0]) / ref[0]).mean()
        assert abs(mean) <= 4 * 2.0 ** -23, (b, mean)
