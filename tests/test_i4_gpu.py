"""The 4-bit cache on the GPU against its fp64 oracle (oracle/i4.py).

Codes, scale and exponent bytes are equal bit for bit, and so are rows read back
(a code times a scale, rounded once).  Attention outputs lie within the bound of
the 8-bit cache's tests: the products run on operands that hold code times scale
exactly, so the roundings are the same.  Caches start filled with 0xFF (NaN
exponents, the largest codes), so anything read behind a sequence's end shows.
"""

import numpy as np
import pytest

import turboquant_bit_kv_tq_gb300 as tq
from oracle import f8, i4
from test_f8_gpu import CASES, DT, _bound, _gpu, _np, _rng, _slots, _table

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _cache(d, hkv, hq, blocks, batch, columns, fill=0xFF):
    c = tq.TQI4Cache(head_dim=d, num_kv_heads=hkv, num_q_heads=hq, num_blocks=blocks, max_batch=batch,
                     max_blocks_per_seq=columns)
    c.cache.fill_(fill)
    return c


# ------------------------------------------------------------------- store
def _vectors(rng, n, h, d, dtype):
    """Vectors of very different sizes, groups of very different sizes in one vector, zeros, one-element vectors,
    elements at the borders between two codes and next to them."""
    x = rng.standard_normal((n, h, d)) * np.exp(rng.uniform(-6, 6, (n, h, 1)))
    x *= np.exp(np.repeat(rng.uniform(-5, 0, (n, h, d // 16)), 16, -1))
    x[0::7] = 0
    x[1::7, :, 1:] = 0
    x[2::7] *= 2.0 ** np.repeat(rng.integers(-30, 1, x[2::7].shape[:2] + (d // 16,)), 16, -1)
    # multiples of half a step of a scale of four bits; the group's first element fixes the scale
    s = rng.integers(8, 16, x[3::7].shape[:2] + (d // 16, 1)) / 8
    y = rng.integers(-15, 16, x[3::7].shape[:2] + (d // 16, 16)) / 2 * s
    y[..., :1] = 7.5 * s
    x[3::7] = y.reshape(x[3::7].shape)
    t = torch.from_numpy(x).to(DT[dtype])
    if dtype == "f32":  # one unit of the last place to either side
        t[10::14] = torch.nextafter(t[10::14], torch.full_like(t[10::14], 1e9))
        t[3::14] = torch.nextafter(t[3::14], torch.full_like(t[3::14], -1e9))
    return t


@pytest.mark.parametrize("d,h,n,dtype", [(128, 8, 1, "bf16"), (128, 8, 37, "bf16"), (128, 3, 260, "f32"),
                                         (128, 1, 17, "f16"), (256, 4, 50, "bf16"), (256, 1, 133, "f32"),
                                         (256, 5, 18, "f16"), (128, 2, 2000, "bf16"), (128, 2, 2000, "f16")])
def test_store_bits(d, h, n, dtype):
    rng = _rng(61, d, h, n)
    blocks = n // 16 + 4
    c = _cache(d, h, h, blocks, 1, 1)
    before = c.pages().cpu().numpy()
    k, v = _vectors(rng, n, h, d, dtype), _vectors(rng, n, h, d, dtype)
    slots = rng.permutation(blocks * 16)[:n].astype(np.int64)
    slots[n // 2] = -1
    c.store(k.cuda(), v.cuda(), _gpu(slots))
    assert np.array_equal(c.pages().cpu().numpy(), i4.store(before, _np(k), _np(v), slots))
    assert c.device_error() == 0


def test_store_extremes_and_bad_vectors():
    d = 128
    x = np.zeros((12, 1, d), np.float32)
    x[0, 0, :20] = 3.4028234e38
    x[0, 0, 16] = 1e30
    x[1, 0, :2] = 2.0 ** -149, 2.0 ** -140
    x[2, 0, 3] = np.inf
    x[3, 0, 90] = np.nan
    x[4, 0, 127] = -np.inf
    x[5, 0, :3] = 1e-37, -1e-38, 1e-39
    x[6, 0, :] = -0.0
    x[7, 0, :4] = 240 * 2.0 ** 20, 1, -1, 241
    x[8, 0, :4] = np.float32(240) * (1 + 2.0 ** -23), 9, -9, 17
    x[9, 0, [0, 16, 17]] = 240, 2.0 ** -18, -(2.0 ** -19)              # a group at the border of no scale
    x[10, 0, [0, 16, 32]] = 240, np.float32(2.0 ** -18) * (1 + 2.0 ** -23), 7.5 * 2.0 ** -17  # and just above it
    x[11, 0, [0, 16]] = 3.4028234e38, 2.0 ** -149                      # below fp32's range beside the largest
    c = _cache(d, 1, 1, 1, 1, 1)
    before = c.pages().cpu().numpy()
    slots = np.arange(12, dtype=np.int64)
    c.store(_gpu(x), _gpu(x[::-1]), _gpu(slots))
    assert np.array_equal(c.pages().cpu().numpy(), i4.store(before, x, x[::-1], slots))


def test_store_rows_of_a_projection_and_bad_slots():
    rng = _rng(62)
    d, h, n = 128, 2, 21
    qkv = torch.randn((n, 4 + 2 * h, d), dtype=torch.bfloat16, device="cuda")
    k, v = qkv[:, 4:4 + h], qkv[:, 4 + h:]
    c = _cache(d, h, h, 3, 1, 1)
    before = c.pages().cpu().numpy()
    slots = rng.permutation(48)[:n].astype(np.int64)
    slots[[3, 4, 5]] = 48, -2, 1 << 40
    c.store(k, v, _gpu(slots))
    assert np.array_equal(c.pages().cpu().numpy(), i4.store(before, _np(k), _np(v), slots))
    assert c.device_error() == tq.TQ_DEVERR_SLOT and c.device_error() == 0
    c.store(k[:0], v[:0], _gpu(slots[:0]))  # no token: nothing


# -------------------------------------------------------------------- load
@pytest.mark.parametrize("d,h,lens,dtype", [(128, 8, [1], "bf16"), (128, 2, [0, 15, 16, 17, 0, 100], "f32"),
                                            (128, 3, [300, 1, 33], "f16"), (256, 4, [40, 0, 7], "bf16"),
                                            (256, 1, [18], "f32"), (128, 1, list(range(70)), "bf16")])
def test_load(d, h, lens, dtype):
    rng = _rng(63, d, h, len(lens))
    table, blocks = _table(rng, lens)
    c = _cache(d, h, h, blocks, len(lens) + 1, table.shape[1])
    n = sum(lens)
    k, v = rng.standard_normal((n, h, d)), rng.standard_normal((n, h, d)) * 3
    c.store(_gpu(k, torch.float32), _gpu(v, torch.float32), _gpu(_slots(table, lens)))
    room = 3
    starts = np.cumsum([0] + [m + room for m in lens]).astype(np.int32)
    ko = torch.full((int(starts[-1]) + 5, h, d), -7.0, dtype=DT[dtype], device="cuda")
    vo = ko.clone()
    c.load(_gpu(table), _gpu(np.array(lens, np.int32)), _gpu(starts), ko, vo)
    pages = c.pages().cpu().numpy()
    want_k, want_v = np.full(ko.shape, -7.0), np.full(vo.shape, -7.0)
    for b, m in enumerate(lens):
        want_k[starts[b]:starts[b] + m], want_v[starts[b]:starts[b] + m] = i4.rows(pages, table[b], m, d)
    # the values have 7 significant bits and ordinary exponents: exact in every dtype
    assert np.array_equal(_np(ko), want_k) and np.array_equal(_np(vo), want_v)
    assert c.device_error() == 0


def test_load_at_the_ends_of_the_range():
    d = 128
    x = np.zeros((4, 1, d), np.float32)
    x[0, 0, :32] = np.linspace(-3.4028234e38, 3.4028234e38, 32)
    x[1, 0, :32] = np.linspace(-1e-38, 1e-38, 32)
    x[2, 0, :32] = np.linspace(-1e-42, 1e-42, 32)
    x[3, 0, :32] = np.linspace(1e-3, 1e30, 32)
    c = _cache(d, 1, 1, 1, 1, 1)
    c.store(_gpu(x), _gpu(x), _gpu(np.arange(4, dtype=np.int64)))
    one = _gpu(np.array([4], np.int32))
    want, _ = i4.rows(c.pages().cpu().numpy(), np.zeros(1, np.int64), 4, d)
    for dtype in DT.values():
        k, v = torch.zeros((4, 1, d), dtype=dtype, device="cuda"), torch.zeros((4, 1, d), dtype=dtype, device="cuda")
        c.load(_gpu(np.zeros((1, 1), np.int32)), one, _gpu(np.zeros(1, np.int32)), k, v)
        assert torch.equal(k.cpu(), torch.from_numpy(want).to(dtype)) and torch.equal(k, v)


def test_load_reads_nan_vectors_and_refuses_bad_rows():
    d, h, lens = 128, 2, [20, 30]
    rng = _rng(64)
    table, blocks = _table(rng, lens)
    c = _cache(d, h, h, blocks, 2, table.shape[1])
    x = rng.standard_normal((50, h, d)).astype(np.float32)
    x[5, 1, 7] = np.inf
    c.store(_gpu(x), _gpu(x), _gpu(_slots(table, lens)))
    ko = torch.zeros((50, h, d), device="cuda")
    vo = torch.zeros_like(ko)
    c.load(_gpu(table), _gpu(np.array(lens, np.int32)), _gpu(np.array([0, 20], np.int32)), ko, vo)
    got = _np(ko)
    assert np.isnan(got[5, 1]).all() and np.isfinite(np.delete(got.reshape(100, d), 11, 0)).all()
    # rows outside the outputs, a bad block id and a length past the table: the rest is read
    ko.fill_(-7)
    t2 = table.copy()
    t2[1, 0] = blocks
    c.load(_gpu(t2), _gpu(np.array([20, 10 ** 6], np.int32)), _gpu(np.array([-3, 35], np.int32)), ko, vo)
    assert c.device_error() == tq.TQ_DEVERR_SEQLEN | tq.TQ_DEVERR_BLOCK | tq.TQ_DEVERR_CHUNK
    again = _np(ko)
    kept = np.nan_to_num(got[3:20], nan=-99.0)
    assert np.array_equal(np.nan_to_num(again[:17], nan=-99.0), kept) and (again[17:50] == -7).all()


# ------------------------------------------------------------------ decode
def _decode_case(d, hkv, g, lens, qt, seed, k_gain=1.0, v_scales=None, q_gain=1.0):
    rng = _rng(65, seed)
    hq = hkv * g
    table, blocks = _table(rng, lens)
    c = _cache(d, hkv, hq, blocks, len(lens), table.shape[1])
    n = sum(lens)
    k = rng.standard_normal((n, hkv, d)) * np.exp(0.5 * rng.standard_normal((hkv, d))) * k_gain
    v = rng.standard_normal((n, hkv, d))
    if v_scales is not None:
        v *= 2.0 ** rng.integers(*v_scales, (n, hkv, 1))
    c.store(_gpu(k, torch.float32), _gpu(v, torch.float32), _gpu(_slots(table, lens)))
    q = torch.from_numpy(rng.standard_normal((len(lens), hq, d)) * q_gain).to(DT[qt])
    return c, q, table


def _steps(q, k, v, exps, scale):
    """What the weights' steps add.  A weight p_t 2^e_t (e_t the value's exponent) goes in as one or two fp16 parts
    whose steps are 2^-24 at least, beside a largest weight of at least 2^4: it is off by up to 2^-29 of the
    sequence's largest, times |v_t| 2^-e_t.  (A 4-bit code of the largest can be 0: then that is all there is.)"""
    out = np.zeros((q.shape[1], v.shape[2]))
    g = q.shape[1] // k.shape[1]
    for h in range(q.shape[1]):
        z = k[:, h // g] @ q[0, h] * scale
        size = np.exp2(exps[:, h // g] - 127.0)
        most = (np.exp(z - z.max()) * size).max() / np.exp(z - z.max()).sum()
        out[h] = 2.0 ** -29 * most * (np.abs(v[:, h // g]) / size[:, None]).sum(0)
    return out


def _check_decode(c, q, table, lens, got, scale=0.0):
    d = c.cfg.head_dim
    pages = c.pages().cpu().numpy()
    sc = scale if scale > 0 else 1 / np.sqrt(d)
    qn, gn = _np(q), _np(got)
    precise = q.dtype == torch.float32 or got.dtype == torch.float32
    for b, n in enumerate(lens):
        if n == 0:
            assert not gn[b].any(), b
            continue
        k, v = i4.rows(pages, table[b], n, d)
        ref, _, mag = f8.attention(qn[b:b + 1], k, v, sc)
        t = np.arange(n)
        exps = i4.parts(pages, d)[1][2][table[b, t // 16], :, t % 16].astype(np.float64)
        tol = _bound(qn[b:b + 1], k, v, sc, mag, ref, precise, got.dtype)[0] + _steps(qn[b:b + 1], k, v, exps, sc)
        err = np.abs(gn[b] - ref[0])
        assert (err <= tol).all(), (b, n, err.max(), (err / tol).max())


def _lens(lens):
    return _gpu(np.array(lens, np.int32))


@pytest.mark.parametrize("d,hkv,g,lens,qt,ot", CASES)
def test_decode(d, hkv, g, lens, qt, ot):
    c, q, table = _decode_case(d, hkv, g, lens, qt, d + hkv * 7 + g)
    args = (q.cuda(), _gpu(table), _lens(lens))
    got = c.decode(*args, out_dtype=DT[ot])
    _check_decode(c, q, table, lens, got)
    again = c.decode(*args, out_dtype=DT[ot])
    assert torch.equal(got, again)  # joined in a fixed order
    assert c.device_error() == 0


@pytest.mark.parametrize("d,hkv,g,lens,qt,ot", [
    (128, 1, 12, [20000, 3], "f32", "f32"),              # parts joined in groups
    (256, 1, 16, [12000], "bf16", "bf16"),               # more parts than fit at a time
    (256, 1, 4, [31, 6000, 1, 300], "f16", "f32"),
    (128, 8, 4, [4000, 40, 0, 90, 17, 700, 64, 3000], "bf16", "bf16"),  # several units in a run
    (128, 4, 2, [257] * 130, "bf16", "bf16"),            # more units than blocks, too long for a warp
])
def test_decode_many_parts_and_units(d, hkv, g, lens, qt, ot):
    c, q, table = _decode_case(d, hkv, g, lens, qt, 3 * d + hkv + g)
    got = c.decode(q.cuda(), _gpu(table), _lens(lens), out_dtype=DT[ot])
    _check_decode(c, q, table, lens, got)
    assert c.device_error() == 0


def test_decode_more_sequences_than_blocks():
    rng = _rng(66)
    lens = [int(x) for x in rng.integers(0, 90, 700)]
    lens[0], lens[-1], lens[350] = 0, 0, 800
    c, q, table = _decode_case(128, 2, 4, lens, "bf16", 77)
    got = c.decode(q.cuda(), _gpu(table), _lens(lens))
    _check_decode(c, q, table, lens, got)


@pytest.mark.parametrize("d,g,ot", [(128, 4, "bf16"), (128, 16, "f32"), (256, 8, "f32")])
def test_decode_value_scales_far_apart(d, g, ot):
    """Value vectors 2^-40 .. 2^40, peaked and flat scores: no weight is lost beside a large scale."""
    lens = [600, 40]
    for gain in (0.05, 6.0):
        c, q, table = _decode_case(d, 1, g, lens, "f32", 9, k_gain=gain, v_scales=(-40, 41))
        got = c.decode(q.cuda(), _gpu(table), _lens(lens), out_dtype=DT[ot])
        _check_decode(c, q, table, lens, got)


@pytest.mark.parametrize("d,g,qt", [(128, 4, "bf16"), (128, 12, "f32"), (256, 4, "f32"), (256, 16, "bf16")])
def test_decode_groups_of_very_different_scales(d, g, qt):
    """Scales of one vector from the largest (32) down to the subnormal ones and to none."""
    rng = _rng(67, d, g)
    lens = [70, 300]
    table, blocks = _table(rng, lens)
    c = _cache(d, 1, g, blocks, 2, table.shape[1])
    n = sum(lens)
    kv = []
    for _ in range(2):
        x = rng.standard_normal((n, 1, d)) * np.repeat(2.0 ** rng.integers(-26, 1, (n, 1, d // 16)), 16, -1)
        x[..., 0] = 2
        kv.append(_gpu(x, torch.float32))
    c.store(*kv, _gpu(_slots(table, lens)))
    q = torch.from_numpy(rng.standard_normal((2, g, d))).to(DT[qt])
    got = c.decode(q.cuda(), _gpu(table), _lens(lens), out_dtype=torch.float32)
    _check_decode(c, q, table, lens, got)


@pytest.mark.parametrize("x", [-121, 118])
@pytest.mark.parametrize("d,lens", [(128, [9000, 40]), (256, [700, 3000])])
def test_decode_values_at_the_ends_of_the_range(d, lens, x):
    """Values near 2^x, all positive: the power of two of the output and the row
    sum meet at its end only.  In units of 2^x, beside the bound one rounding of
    an fp32 number that may be subnormal: 2^-150."""
    rng = _rng(68, d, x & 255)
    g, n = 4, sum(lens)
    table, blocks = _table(rng, lens)
    c = _cache(d, 1, g, blocks, len(lens), table.shape[1])
    k, v = 0.05 * rng.standard_normal((n, 1, d)), rng.uniform(0.5, 4, (n, 1, d)) * 2.0 ** x
    c.store(_gpu(k, torch.float32), _gpu(v, torch.float32), _gpu(_slots(table, lens)))
    q = rng.standard_normal((len(lens), g, d)).astype(np.float32)
    got = c.decode(_gpu(q), _gpu(table), _lens(lens))
    pages, sc = c.pages().cpu().numpy(), 1 / np.sqrt(d)
    for b, m in enumerate(lens):
        kb, vb = i4.rows(pages, table[b], m, d)
        vb = vb * 2.0 ** -x
        ref, _, mag = f8.attention(q[b:b + 1].astype(np.float64), kb, vb, sc)
        tol = _bound(q[b:b + 1].astype(np.float64), kb, vb, sc, mag, ref, True, got.dtype)[0] + 2.0 ** (-150 - x)
        err = np.abs(_np(got)[b] * 2.0 ** -x - ref[0])
        assert (err <= tol).all(), (b, m, err.max(), (err / tol).max())


def test_decode_queries_far_from_one_and_a_given_scale():
    for qt, gain in (("f32", 2.0 ** 90), ("f32", 2.0 ** -90), ("bf16", 2.0 ** 100), ("f16", 2.0 ** -14)):
        lens = [333]
        c, q, table = _decode_case(128, 1, 4, lens, qt, 10, q_gain=gain)
        scale = float(0.09 / gain)
        got = c.decode(q.cuda(), _gpu(table), _lens(lens), out_dtype=torch.float32, scale=scale)
        _check_decode(c, q, table, lens, got, scale=float(np.float32(scale)))


@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 13, 2.0 ** 45, 2.0 ** 60])
@pytest.mark.parametrize("d,g,lens,qt,ot", [(128, 4, [1, 40, 300, 0, 17], "bf16", "bf16"), (128, 8, [9000, 3], "f32", "f32"),
                                            (256, 5, [2500, 33], "bf16", "f32"), (128, 2, [60] * 700, "bf16", "bf16")])
def test_decode_value_scales_beside_large_scores(d, g, lens, qt, ot, size):
    """Scores of kind * about size^2 and value vectors of scales far apart: the mean of the values of a
    sequence's highest kind.  The oracle's scores are 60 times the kind; a lower kind's weight there is at most
    e^-60 each, where the call's is 0, so they may differ by m e^-60 max |v|: seen where 4-bit codes of the highest
    kind are 0."""
    for seed, kinds in enumerate(([1.0], [-1.0], [-1, -1, -1, 0, 1.0])):
        rng = _rng(69, d, g, seed)
        table, blocks = _table(rng, lens)
        c = _cache(d, 1, g, blocks, len(lens), table.shape[1])
        n = sum(lens)
        kind = rng.choice(kinds, n)
        q, k = np.zeros((len(lens), g, d)), np.zeros((n, 1, d))
        q[..., 5] = size * 141 / 128
        k[:, 0, 5] = kind * size * 1.25
        v = rng.standard_normal((n, 1, d)) * 2.0 ** rng.integers(-12, 13, (n, 1, 1))
        c.store(_gpu(k, torch.float32), _gpu(v, torch.float32), _gpu(_slots(table, lens)))
        got = c.decode(_gpu(q, DT[qt]), _gpu(table), _lens(lens), scale=1.0, out_dtype=DT[ot])
        assert c.device_error() == 0
        pages, gn = c.pages().cpu().numpy(), _np(got)
        q[..., 5], k[:, 0, 5] = 1, kind * 60
        at = 0
        for b, m in enumerate(lens):
            if m == 0:
                assert not gn[b].any()
                continue
            _, vb = i4.rows(pages, table[b], m, d)
            ref, _, mag = f8.attention(q[b:b + 1], k[at:at + m], vb, 1.0)
            tol = _bound(q[b:b + 1], k[at:at + m], vb, 1.0, mag, ref, "f32" in (qt, ot), got.dtype)[0]
            tol = tol + m * np.exp(-60) * np.abs(vb).max()
            err = np.abs(gn[b] - ref[0])
            assert (err <= tol).all(), (b, m, err.max(), (err / tol).max())
            at += m


def test_decode_bad_vectors_stay_in_their_head():
    rng = _rng(70)
    lens, d, hkv, g = [50, 50], 128, 4, 2
    table, blocks = _table(rng, lens)
    c = _cache(d, hkv, hkv * g, blocks, 2, table.shape[1])
    k, v = rng.standard_normal((100, hkv, d)), rng.standard_normal((100, hkv, d))
    k[3, 0, 0] = np.nan       # sequence 0, head 0
    v[7, 1, 5] = np.inf       # sequence 0, head 1
    c.store(_gpu(k, torch.float32), _gpu(v, torch.float32), _gpu(_slots(table, lens)))
    q = rng.standard_normal((2, hkv * g, d))
    q[1, 7, 2] = np.inf       # sequence 1, query head 7 (KV head 3)
    got = _np(c.decode(_gpu(q, torch.bfloat16), _gpu(table), _lens(lens)))
    bad = np.zeros((2, hkv * g), bool)
    bad[0, :4], bad[1, 7] = True, True
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()


def test_decode_bad_blocks_and_lengths():
    """A block id outside the pool is left out with its tokens; lengths are clamped to the table."""
    lens = [100, 60, 30]
    c, q, table = _decode_case(128, 2, 4, lens, "bf16", 31)
    bad = table.copy()
    bad[0, 2], bad[1, 0] = -1, c.cfg.num_blocks
    qg = q.cuda()
    got = c.decode(qg, _gpu(bad), _lens(lens))
    assert c.device_error() == tq.TQ_DEVERR_BLOCK and c.device_error() == 0
    pages = c.pages().cpu().numpy()
    for b, gone in ((0, range(32, 48)), (1, range(0, 16)), (2, ())):
        k, v = i4.rows(pages, table[b], lens[b], 128)
        keep = np.setdiff1d(np.arange(lens[b]), gone)
        ref, _, mag = f8.attention(_np(q[b:b + 1]), k[keep], v[keep], 1 / np.sqrt(128))
        tol = _bound(_np(q[b:b + 1]), k[keep], v[keep], 1 / np.sqrt(128), mag, ref, False, got.dtype)[0]
        assert (np.abs(_np(got)[b] - ref[0]) <= tol).all(), b
    full = 16 * table.shape[1]
    one = c.decode(qg[:1], _gpu(table), _lens([full]))
    over = c.decode(qg[:1], _gpu(table), _lens([full + 5]))
    assert c.device_error() == tq.TQ_DEVERR_SEQLEN
    assert torch.equal(torch.nan_to_num(one), torch.nan_to_num(over))
    assert not c.decode(qg[:1], _gpu(table), _lens([-4])).any() and c.device_error() == tq.TQ_DEVERR_SEQLEN


def test_rows_behind_the_end_and_other_rows_have_no_say():
    """The same sequence with other contents behind its last token and in other pages: the same bits."""
    lens = [37, 130, 16]
    outs = []
    for fill in (0xFF, 0x00, 0x7F, 0x88):
        rng = _rng(71)
        table, blocks = _table(rng, lens)
        c = _cache(128, 2, 8, blocks, 3, table.shape[1], fill)
        n = sum(lens)
        k, v = _gpu(rng.standard_normal((n, 2, 128)), torch.float32), _gpu(rng.standard_normal((n, 2, 128)), torch.float32)
        c.store(k, v, _gpu(_slots(table, lens)))
        q = _gpu(rng.standard_normal((3, 8, 128)), torch.bfloat16)
        outs.append(c.decode(q, _gpu(table), _lens(lens)))
    assert all(torch.equal(outs[0], o) for o in outs[1:]) and torch.isfinite(outs[0]).all()


def test_decode_queries_of_a_projection_streams_and_graphs():
    lens = [700, 33, 0]
    c, q, table = _decode_case(128, 2, 4, lens, "bf16", 32)
    wide = torch.zeros((3, 20, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, 5:13] = q.cuda()
    args = (wide[:, 5:13], _gpu(table), _lens(lens))
    want = c.decode(q.cuda(), *args[1:])
    assert torch.equal(c.decode(*args), want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = torch.full_like(want, 9)
    c.decode(*args, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.decode(*args, out=out)
    for n in ([700, 33, 0], [1, 2, 3], [400, 0, 20]):
        args[2].copy_(_lens(n))
        out.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        _check_decode(c, q, table, n, out)


def test_two_handles_on_two_streams():
    lens = [3000, 40]
    made = [_decode_case(128, 1, 4, lens, "bf16", 20 + i) for i in range(2)]
    args = [(q.cuda(), _gpu(t), _lens(lens)) for _, q, t in made]
    refs = [c.decode(*a) for (c, _, _), a in zip(made, args)]
    streams = [torch.cuda.Stream() for _ in made]
    outs = [torch.zeros_like(r) for r in refs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (c, _, _), a, s, o in zip(made, args, streams, outs):
            c.decode(*a, out=o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, r) for o, r in zip(outs, refs))


def test_cache_beyond_four_gigabytes():
    d, hkv = 128, 8
    page = 18 * d + 32
    blocks = (5 << 30) // (hkv * page)
    c = tq.TQI4Cache(head_dim=d, num_kv_heads=hkv, num_q_heads=32, num_blocks=blocks, max_batch=1,
                     max_blocks_per_seq=40, cache=torch.empty(blocks * hkv * page, dtype=torch.uint8, device="cuda"))
    n = 600
    table = np.arange(blocks - 40, blocks, dtype=np.int32)[None, ::-1].copy()
    rng = _rng(72)
    k, v = (_gpu(rng.standard_normal((n, hkv, d)), torch.bfloat16) for _ in range(2))
    c.store(k, v, _gpu(_slots(table, [n])))
    rows = (1 << 31) // (hkv * d) + 700  # output offsets past 2^31 elements
    ko = torch.empty((rows, hkv, d), dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(ko)
    c.load(_gpu(table), _lens([n]), _gpu(np.array([rows - n], np.int32)), ko, vo)
    for got, x in ((ko[-n:], k), (vo[-n:], v)):
        assert np.array_equal(_np(got), i4.values(*i4.quantise(_np(x))))
    q = torch.randn((1, 32, d), device="cuda").to(torch.bfloat16)
    got = c.decode(q, _gpu(table), _lens([n]))
    kn, vn = _np(ko[-n:]), _np(vo[-n:])
    ref, _, mag = f8.attention(_np(q), kn, vn, 1 / np.sqrt(d))
    assert (np.abs(_np(got) - ref) <= _bound(_np(q), kn, vn, 1 / np.sqrt(d), mag, ref, False, torch.bfloat16)).all()
    assert c.device_error() == 0


def test_refusals():
    c = _cache(128, 2, 8, 4, 2, 2)
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device="cuda")
    t, n = torch.zeros((2, 2), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    k = torch.zeros((2, 2, 128), dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    for error, call in [
        (ValueError, lambda: c.decode(q[:, :6], t, n)),
        (ValueError, lambda: c.decode(q.transpose(0, 1).contiguous().transpose(0, 1), t, n)),
        (ValueError, lambda: c.decode(q, t[:, :1], n)),
        (ValueError, lambda: c.decode(q, t[:1], n)),
        (ValueError, lambda: c.decode(q, t, n[:1])),
        (TypeError, lambda: c.decode(q, t.long(), n)),
        (TypeError, lambda: c.decode(q.double(), t, n)),
        (ValueError, lambda: c.decode(q, t, n, out=q[:1])),
        (ValueError, lambda: c.decode(q.cpu(), t, n)),
        (ValueError, lambda: c.store(k, k[:1], slots)),
        (ValueError, lambda: c.store(k, k, slots[:1])),
        (TypeError, lambda: c.store(k, k, slots.int())),
        (TypeError, lambda: c.store(k.int(), k.int(), slots)),
        (ValueError, lambda: c.store(k[:1].expand(2, 2, 128), k, slots)),
        (ValueError, lambda: c.load(t, n, n, k, k[:1])),
        (ValueError, lambda: c.load(t, n, n[:1], k, k)),
    ]:
        with pytest.raises(error):
            call()
    big = torch.zeros((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(tq.TQError) as e:  # more sequences than max_batch
        c.decode(big, torch.zeros((3, 2), dtype=torch.int32, device="cuda"),
                 torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert e.value.status == -1
    odd = torch.zeros(2 * 8 * 128 + 8, dtype=torch.bfloat16, device="cuda")[1:-7].view(2, 8, 128)
    with pytest.raises(tq.TQError) as e:
        c.decode(odd, t, n)
    assert e.value.status == -5
    with pytest.raises(ValueError):
        tq.TQI4Cache(head_dim=128, num_kv_heads=2, num_q_heads=8, num_blocks=4, max_blocks_per_seq=2, cache=c.cache[:-1])
    with pytest.raises(ValueError):
        tq.tq_i4_decode_attention(c.handle, c.cfg, q, c.cache[:-1], t, n, q.clone())


# ------------------------------------------------- other strides, shared blocks
@pytest.mark.parametrize("d,h,dtype", [(128, 3, "bf16"), (256, 1, "f32"), (128, 2, "f16")])
def test_rows_that_start_at_odd_multiples_of_sixteen_bytes(d, h, dtype):
    """Stored from and loaded to rows that 32-byte accesses cannot reach."""
    rng = _rng(73, d, h)
    n, pad = 45, 128 // torch.finfo(DT[dtype]).bits
    table, blocks = _table(rng, [n])
    wide = torch.zeros((n, h * d + pad), dtype=DT[dtype], device="cuda")
    k, v = (_gpu(rng.standard_normal((n, h, d)), DT[dtype]) for _ in range(2))
    views = []
    for x in (k, v):
        w = wide.clone()
        w[:, :h * d] = x.flatten(1)
        views.append(w[:, :h * d].unflatten(1, (h, d)))
    c = _cache(d, h, h, blocks, 1, table.shape[1])
    before = c.pages().cpu().numpy()
    slots = _slots(table, [n])
    c.store(*views, _gpu(slots))
    assert np.array_equal(c.pages().cpu().numpy(), i4.store(before, _np(k), _np(v), slots))
    outs = [torch.full((n * h * d + 2 * pad,), -7.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    ko, vo = (x[pad:-pad].view(n, h, d) for x in outs)
    c.load(_gpu(table), _lens([n]), _lens([0]), ko, vo)
    for got, want, whole in zip((ko, vo), i4.rows(c.pages().cpu().numpy(), table[0], n, d), outs):
        assert np.array_equal(_np(got), want) and (whole[:pad] == -7).all() and (whole[-pad:] == -7).all()


@pytest.mark.parametrize("d,g,qt,ot,most", [(128, 16, "bf16", "bf16", 50), (256, 4, "f32", "f32", 60),
                                            (256, 12, "bf16", "f32", 40), (128, 4, "f32", "bf16", 35)])
def test_many_short_sequences(d, g, qt, ot, most):
    """More units than blocks, whole ones to warps: one and two tiles of heads, two pages a step, both precisions."""
    rng = _rng(74, d, g)
    lens = [int(x) for x in rng.integers(0, most, 900)]
    lens[0], lens[1], lens[-1] = most, 0, 1
    c, q, table = _decode_case(d, 1, g, lens, qt, 78)
    got = c.decode(q.cuda(), _gpu(table), _lens(lens), out_dtype=DT[ot])
    _check_decode(c, q, table, lens, got)
    assert torch.equal(got, c.decode(q.cuda(), _gpu(table), _lens(lens), out_dtype=DT[ot])) and c.device_error() == 0


def test_sequences_that_share_blocks():
    """A common prefix in the same blocks, and a sequence that is another's beginning."""
    lens = [300, 200, 64]
    c, q, table = _decode_case(128, 2, 4, [300, 300, 300], "bf16", 79)
    table[1, :8], table[2, :4] = table[0, :8], table[0, :4]
    got = c.decode(q.cuda(), _gpu(table), _lens(lens))
    _check_decode(c, q, table, lens, got)
    alone = c.decode(q[2:].cuda(), _gpu(table[2:]), _lens(lens[2:]))
    _check_decode(c, q[2:], table[2:], lens[2:], alone)


def test_load_is_captured_and_replayed():
    lens = [70, 0, 33]
    c, q, table = _decode_case(128, 2, 2, [90, 90, 90], "bf16", 80)
    t, ld, starts = _gpu(table), _lens(lens), _lens([0, 100, 200])
    ko, vo = (torch.zeros((300, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.load(t, ld, starts, ko, vo)
    pages = c.pages().cpu().numpy()
    for lens in ([70, 0, 33], [1, 90, 16]):
        ld.copy_(_lens(lens))
        ko.fill_(-7)
        vo.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        want = np.full((2, 300, 2, 128), -7.0)
        for b, n in enumerate(lens):
            want[:, 100 * b:100 * b + n] = i4.rows(pages, table[b], n, 128)
        assert np.array_equal(_np(ko), want[0]) and np.array_equal(_np(vo), want[1])


@pytest.mark.parametrize("d,hkv,g,count,shortest,longest,qt,ot", [
    (128, 1, 4, 400, 150, 2000, "bf16", "bf16"),  # even runs: several units, and parts of them, each
    (128, 1, 12, 270, 150, 2000, "f32", "f32"),
    (256, 1, 4, 270, 150, 2000, "bf16", "f32"),
    (128, 8, 4, 57, 0, 300, "bf16", "bf16"),      # about as many units as blocks: a unit a run
    (128, 4, 2, 100, 0, 400, "f16", "f16"),       # runs of a few units' longest
    (256, 2, 20, 30, 0, 300, "bf16", "f32"),      # two units share a head's pages
    (128, 8, 4, 61, 0, 300, "bf16", "bf16"),      # more units than blocks: whole ones to blocks
    (128, 1, 16, 500, 0, 700, "f32", "bf16"),
    (256, 1, 4, 400, 0, 600, "bf16", "bf16"),
])
def test_how_units_are_dealt_out(d, hkv, g, count, shortest, longest, qt, ot):
    rng = _rng(75, d, hkv, g, count)
    lens = [int(x) for x in rng.integers(shortest, min(longest, shortest + 300), count)]
    lens[count // 2], lens[3] = longest, 1
    c, q, table = _decode_case(d, hkv, g, lens, qt, 81)
    args = (q.cuda(), _gpu(table), _lens(lens))
    got = c.decode(*args, out_dtype=DT[ot])
    _check_decode(c, q, table, lens, got)
    assert torch.equal(got, c.decode(*args, out_dtype=DT[ot])) and c.device_error() == 0
    # a sequence by itself: other runs, the same bounds
    one = slice(count // 2, count // 2 + 1)
    got = c.decode(*(x[one] for x in args), out_dtype=DT[ot])
    _check_decode(c, q[one], table[one], lens[one], got)


@pytest.mark.parametrize("d,h,count,longest", [(128, 2, 33, 90), (256, 1, 100, 60), (128, 1, 70, 1500)])
def test_load_of_many_sequences(d, h, count, longest):
    """More sequences than are looked at together, some of them empty, with gaps between their rows."""
    rng = _rng(76, d, count)
    lens = [int(x) for x in rng.integers(0, longest, count)]
    lens[0], lens[31], lens[32], lens[-1] = 0, longest, 0, 17
    c, _, table = _decode_case(d, h, 1, lens, "bf16", 82)
    gaps = rng.integers(0, 4, count)
    starts = np.concatenate([[2], 2 + np.cumsum(np.array(lens) + gaps)]).astype(np.int32)
    want = np.full((2, int(starts[-1]) + 3, h, d), -7.0)
    ko, vo = (_gpu(x, torch.float32) for x in want)
    c.load(_gpu(table), _lens(lens), _gpu(starts[:-1]), ko, vo)
    pages = c.pages().cpu().numpy()
    for b, n in enumerate(lens):
        want[:, starts[b]:starts[b] + n] = i4.rows(pages, table[b], n, d)
    assert np.array_equal(_np(ko), want[0]) and np.array_equal(_np(vo), want[1])
    assert c.device_error() == 0


def test_pages_whose_memory_is_exchanged():
    """The calls go by the cache tensor as it is now, not by the memory that it had when the handle was made."""
    c, cfg = _cache(128, 2, 4, 8, 2, 4, fill=0), dict(dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(97)
    k, v, q = (_gpu(rng.standard_normal((20, h, 128)), torch.bfloat16) for h in (2, 2, 4))
    slots, table, lens = _gpu(np.arange(20)), _gpu(np.arange(8, dtype=np.int32).reshape(2, 4)), _gpu(np.int32([20, 0]))
    old = c.cache.data  # (the same memory, which stays allocated)
    c.cache.data = torch.zeros_like(old)
    c.store(k, v, slots)
    assert not old.any()
    want = i4.store(np.zeros((8, 2, c.page_bytes), np.uint8), _np(k), _np(v), np.arange(20))
    assert np.array_equal(c.pages().cpu().numpy(), want)
    out = [torch.zeros((20, 2, 128), **cfg) for _ in range(2)]
    c.load(table, lens, _gpu(np.int32([0, 20])), *out)
    for x, y in zip(out, i4.rows(want, np.arange(4), 20, 128)):
        assert np.array_equal(_np(x), torch.from_numpy(y).to(torch.bfloat16).double().numpy())
    got = c.decode(q[:2], table, lens)
    c.cache.data = old
    old.copy_(torch.from_numpy(want.reshape(-1)))
    assert torch.equal(c.decode(q[:2], table, lens), got) and bool(got[0].any())
    for bad in (old[:-1], old.cpu(), torch.cat([old, old])[::2]):
        c.cache.data = bad
        for call in (lambda: c.store(k, v, slots), lambda: c.load(table, lens, lens, *out),
                     lambda: c.decode(q[:2], table, lens)):
            with pytest.raises(ValueError):
                call()
    c.cache.data = old
    assert torch.equal(c.decode(q[:2], table, lens), got) and c.device_error() == 0
