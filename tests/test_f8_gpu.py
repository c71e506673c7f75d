"""The 8-bit cache on the GPU against its fp64 oracle (oracle/f8.py).

Codes and exponent bytes are equal bit for bit, and so are rows read back (a
code times a power of two, rounded once).  Attention outputs lie within a bound
made of the roundings the kernel makes; see _bound().  Caches start filled with
0xFF (NaN codes, NaN scales), so anything read behind a sequence's end shows.
"""

import numpy as np
import pytest

import turboquant_bit_kv_tq_gb300 as tq
from oracle import f8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _rng(*seed):
    return np.random.default_rng(seed)


def _table(rng, lens, spare=3):
    need = [(n + 15) // 16 for n in lens]
    blocks = sum(need) + spare
    table = np.zeros((len(lens), max(1, max(need))), np.int32)
    perm = rng.permutation(blocks)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, blocks


def _cache(d, hkv, hq, blocks, batch, columns, fill=0xFF):
    c = tq.TQF8Cache(head_dim=d, num_kv_heads=hkv, num_q_heads=hq, num_blocks=blocks, max_batch=batch,
                     max_blocks_per_seq=columns)
    c.cache.fill_(fill)
    return c


def _slots(table, lens):
    return np.concatenate([table[b, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16
                           for b, n in enumerate(lens)] + [np.zeros(0, np.int64)])


def _gpu(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def _np(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------- store
def _vectors(rng, n, h, d, dtype):
    """Vectors of very different sizes, zeros, one-element vectors, values at the rounding borders."""
    x = rng.standard_normal((n, h, d)) * np.exp(rng.uniform(-6, 6, (n, h, 1)))
    x[0::7] = 0
    x[1::7, :, 1:] = 0
    x[2::7] = np.sign(x[2::7]) * rng.choice([1.0625, 1.1875, 448, 464, 1.75 * 2 ** 9, 0.875], x[2::7].shape)
    x[3::7] *= 2.0 ** rng.integers(-12, -3)
    return torch.from_numpy(x).to(DT[dtype])


@pytest.mark.parametrize("d,h,n,dtype", [(128, 8, 1, "bf16"), (128, 8, 37, "bf16"), (128, 3, 260, "f32"),
                                         (128, 1, 17, "f16"), (256, 4, 50, "bf16"), (256, 1, 33, "f32"),
                                         (256, 5, 18, "f16")])
def test_store_bits(d, h, n, dtype):
    rng = _rng(1, d, h, n)
    blocks = n // 16 + 4
    c = _cache(d, h, h, blocks, 1, 1)
    before = c.pages().cpu().numpy()
    k, v = _vectors(rng, n, h, d, dtype), _vectors(rng, n, h, d, dtype)
    slots = rng.permutation(blocks * 16)[:n].astype(np.int64)
    slots[n // 2] = -1
    c.store(k.cuda(), v.cuda(), _gpu(slots))
    want = f8.store(before, _np(k), _np(v), slots)
    assert np.array_equal(c.pages().cpu().numpy(), want)
    assert c.device_error() == 0


def test_store_extremes_and_bad_vectors():
    d = 128
    x = np.zeros((9, 1, d), np.float32)
    x[0, 0, :2] = 3.4028234e38, 1e30
    x[1, 0, :2] = 2.0 ** -149, 2.0 ** -140
    x[2, 0, 3] = np.inf
    x[3, 0, 90] = np.nan
    x[4, 0, 127] = -np.inf
    x[5, 0, :3] = 1e-37, -1e-38, 1e-39
    x[6, 0, :] = -0.0
    x[7, 0, :4] = 448 * 2.0 ** 20, 1, -1, 449
    x[8, 0, :4] = np.float32(448) * (1 + 2.0 ** -23), 9, -9, 17
    c = _cache(d, 1, 1, 1, 1, 1)
    before = c.pages().cpu().numpy()
    slots = np.arange(9, dtype=np.int64)
    c.store(_gpu(x), _gpu(x[::-1]), _gpu(slots))
    assert np.array_equal(c.pages().cpu().numpy(), f8.store(before, x, x[::-1], slots))


def test_store_rows_of_a_projection_and_bad_slots():
    rng = _rng(2)
    d, h, n = 128, 2, 21
    qkv = torch.randn((n, 4 + 2 * h, d), dtype=torch.bfloat16, device="cuda")
    k, v = qkv[:, 4:4 + h], qkv[:, 4 + h:]
    c = _cache(d, h, h, 3, 1, 1)
    before = c.pages().cpu().numpy()
    slots = rng.permutation(48)[:n].astype(np.int64)
    slots[[3, 4, 5]] = 48, -2, 1 << 40
    c.store(k, v, _gpu(slots))
    assert np.array_equal(c.pages().cpu().numpy(), f8.store(before, _np(k), _np(v), slots))
    assert c.device_error() == tq.TQ_DEVERR_SLOT and c.device_error() == 0
    c.store(k[:0], v[:0], _gpu(slots[:0]))  # no token: nothing


# -------------------------------------------------------------------- load
@pytest.mark.parametrize("d,h,lens,dtype", [(128, 8, [1], "bf16"), (128, 2, [0, 15, 16, 17, 0, 100], "f32"),
                                            (128, 3, [300, 1, 33], "f16"), (256, 4, [40, 0, 7], "bf16"),
                                            (256, 1, [18], "f32"), (128, 1, list(range(70)), "bf16")])
def test_load(d, h, lens, dtype):
    rng = _rng(3, d, h, len(lens))
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
        want_k[starts[b]:starts[b] + m], want_v[starts[b]:starts[b] + m] = f8.rows(pages, table[b], m, d)
    # the values have 4 significant bits and ordinary exponents: exact in every dtype
    assert np.array_equal(_np(ko), want_k) and np.array_equal(_np(vo), want_v)
    assert c.device_error() == 0


def test_load_reads_nan_vectors_and_refuses_bad_rows():
    d, h, lens = 128, 2, [20, 30]
    rng = _rng(4)
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
def _bound(q, k, v, scale, mag, ref, precise, out_dtype):
    """How far an output may be from the oracle's.

    Weights: fp16 (2^-11 of each), or two fp16 parts (2^-21); e^x in 2^-22 and
    its argument's rounding, 2^-22 of the largest |score| in log2 units.
    Scores: fp32 accumulation over d/16 tensor-core steps, at most two units of
    2^-23 of the running sum each, <= sum |q||k|; a query of two fp16 parts:
    2^-21 of that.  Sums over n tokens: a warp adds one 16-token step at a time
    (at most n/16 in a row), 2^-23 each, and a few joins.  fp16 weights below
    2^-14 keep an absolute half step 2^-25 beside a largest one of at least 1
    (the references are moved when it passes 2^12 and set it to 2^4).  Output
    rounding: eps/2.  Everything but the last scales the summed terms' size."""
    n, d = k.shape[0], k.shape[2]
    g = q.shape[1] // k.shape[1]
    kk = np.repeat(np.abs(k), g, 1)
    s = np.einsum("nhd,mhd->nhm", np.abs(q), kk).max(-1)[..., None] * scale  # natural units
    ds = s * ((d / 16) * 2.0 ** -22 + (2.0 ** -21 if precise else 0) + 3 * 2.0 ** -24)
    dw = (2.0 ** -21 if precise else 2.0 ** -11) + 2.0 ** -22 * (2 + s * 1.45)
    sums = (n / 16 + 16) * 2.0 ** -22
    rel = 2 * (ds + sums) + dw
    vmax = np.repeat(np.abs(v).max((0, 2)), g)[None, :, None]
    tiny = n * (0 if precise else 2.0 ** -25) * vmax / max(1, n) ** 0.5
    return rel * mag + torch.finfo(out_dtype).eps / 2 * np.abs(ref) + tiny + 1e-30


def _decode_case(d, hkv, g, lens, qt, ot, seed, k_gain=1.0, v_scales=None, scale=0.0, q_gain=1.0):
    rng = _rng(5, seed)
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


def _check_decode(c, q, table, lens, ot, got, scale=0.0):
    d = c.cfg.head_dim
    pages = c.pages().cpu().numpy()
    sc = scale if scale > 0 else 1 / np.sqrt(d)
    qn, gn = _np(q), _np(got)
    precise = q.dtype == torch.float32 or got.dtype == torch.float32
    for b, n in enumerate(lens):
        if n == 0:
            assert not gn[b].any(), b
            continue
        k, v = f8.rows(pages, table[b], n, d)
        ref, _, mag = f8.attention(qn[b:b + 1], k, v, sc)
        tol = _bound(qn[b:b + 1], k, v, sc, mag, ref, precise, got.dtype)[0]
        err = np.abs(gn[b] - ref[0])
        assert (err <= tol).all(), (b, n, err.max(), (err / tol).max())


CASES = [
    (128, 8, 4, [130], "bf16", "bf16"),
    (128, 2, 1, [1, 0, 15, 16, 17, 31, 32, 33], "bf16", "bf16"),
    (128, 1, 3, [2000], "f16", "f16"),
    (128, 1, 8, [5000, 1, 700], "bf16", "f32"),
    (128, 2, 12, [257, 64], "f32", "f32"),
    (128, 1, 16, [900, 0, 3], "bf16", "bf16"),
    (128, 1, 40, [150, 20], "bf16", "f32"),
    (256, 2, 8, [130, 1, 0, 999], "bf16", "bf16"),
    (256, 1, 5, [1500], "f32", "f32"),
    (256, 1, 16, [260, 17], "f16", "f16"),
    (256, 1, 11, [400, 33], "f32", "bf16"),
    (128, 1, 1, [1], "f32", "f16"),
    (128, 4, 2, list(range(60)), "bf16", "bf16"),
]


@pytest.mark.parametrize("d,hkv,g,lens,qt,ot", CASES)
def test_decode(d, hkv, g, lens, qt, ot):
    c, q, table = _decode_case(d, hkv, g, lens, qt, ot, d + hkv * 7 + g)
    args = (q.cuda(), _gpu(table), _gpu(np.array(lens, np.int32)))
    got = c.decode(*args, out_dtype=DT[ot])
    _check_decode(c, q, table, lens, ot, got)
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
    c, q, table = _decode_case(d, hkv, g, lens, qt, ot, 3 * d + hkv + g)
    got = c.decode(q.cuda(), _gpu(table), _gpu(np.array(lens, np.int32)), out_dtype=DT[ot])
    _check_decode(c, q, table, lens, ot, got)
    assert c.device_error() == 0


def test_decode_more_sequences_than_blocks():
    rng = _rng(6)
    lens = [int(x) for x in rng.integers(0, 90, 700)]
    lens[0], lens[-1], lens[350] = 0, 0, 800
    c, q, table = _decode_case(128, 2, 4, lens, "bf16", "bf16", 77)
    got = c.decode(q.cuda(), _gpu(table), _gpu(np.array(lens, np.int32)))
    _check_decode(c, q, table, lens, "bf16", got)


@pytest.mark.parametrize("d,g,ot", [(128, 4, "bf16"), (128, 16, "f32"), (256, 8, "f32")])
def test_decode_value_scales_far_apart(d, g, ot):
    """Value vectors 2^-40 .. 2^40, peaked and flat scores: no weight is lost beside a large scale."""
    for gain in (0.05, 6.0):
        c, q, table = _decode_case(d, 1, g, [600, 40], "f32", ot, 9, k_gain=gain, v_scales=(-40, 41))
        lens = [600, 40]
        got = c.decode(q.cuda(), _gpu(table), _gpu(np.array(lens, np.int32)), out_dtype=DT[ot])
        _check_decode(c, q, table, lens, ot, got)


@pytest.mark.parametrize("x", [-121, 118])
@pytest.mark.parametrize("d,lens", [(128, [9000, 40]), (256, [700, 3000])])
def test_decode_values_at_the_ends_of_the_range(d, lens, x):
    """Values near 2^x, all positive: the power of two of the output and the row
    sum meet at its end only.  In units of 2^x, beside the bound above one
    rounding of an fp32 number that may be subnormal: 2^-150."""
    rng = _rng(13, d, x & 255)
    g, n = 4, sum(lens)
    table, blocks = _table(rng, lens)
    c = _cache(d, 1, g, blocks, len(lens), table.shape[1])
    k, v = 0.05 * rng.standard_normal((n, 1, d)), rng.uniform(0.5, 4, (n, 1, d)) * 2.0 ** x
    c.store(_gpu(k, torch.float32), _gpu(v, torch.float32), _gpu(_slots(table, lens)))
    q = rng.standard_normal((len(lens), g, d)).astype(np.float32)
    got = c.decode(_gpu(q), _gpu(table), _gpu(np.array(lens, np.int32)))
    pages, sc = c.pages().cpu().numpy(), 1 / np.sqrt(d)
    for b, m in enumerate(lens):
        kb, vb = f8.rows(pages, table[b], m, d)
        vb = vb * 2.0 ** -x
        ref, _, mag = f8.attention(q[b:b + 1].astype(np.float64), kb, vb, sc)
        tol = _bound(q[b:b + 1].astype(np.float64), kb, vb, sc, mag, ref, True, got.dtype)[0] + 2.0 ** (-150 - x)
        err = np.abs(_np(got)[b] * 2.0 ** -x - ref[0])
        assert (err <= tol).all(), (b, m, err.max(), (err / tol).max())


def test_decode_queries_far_from_one_and_a_given_scale():
    for qt, gain in (("f32", 2.0 ** 90), ("f32", 2.0 ** -90), ("bf16", 2.0 ** 100), ("f16", 2.0 ** -14)):
        lens = [333]
        c, q, table = _decode_case(128, 1, 4, lens, qt, "f32", 10, q_gain=gain)
        scale = float(0.09 / gain)
        got = c.decode(q.cuda(), _gpu(table), _gpu(np.array(lens, np.int32)), out_dtype=torch.float32, scale=scale)
        _check_decode(c, q, table, lens, "f32", got, scale=float(np.float32(scale)))


def test_decode_bad_vectors_stay_in_their_head():
    rng = _rng(11)
    lens, d, hkv, g = [50, 50], 128, 4, 2
    table, blocks = _table(rng, lens)
    c = _cache(d, hkv, hkv * g, blocks, 2, table.shape[1])
    k, v = rng.standard_normal((100, hkv, d)), rng.standard_normal((100, hkv, d))
    k[3, 0, 0] = np.nan       # sequence 0, head 0
    v[7, 1, 5] = np.inf       # sequence 0, head 1
    c.store(_gpu(k, torch.float32), _gpu(v, torch.float32), _gpu(_slots(table, lens)))
    q = rng.standard_normal((2, hkv * g, d))
    q[1, 7, 0] = np.inf       # sequence 1, query head 7
    got = _np(c.decode(_gpu(q, torch.float32), _gpu(table), _gpu(np.array(lens, np.int32))))
    nan = np.isnan(got).any(-1)
    want = np.zeros((2, 8), bool)
    want[0, :4] = True
    want[1, 7] = True
    assert np.array_equal(nan, want) and np.isnan(got[want]).all()


def test_decode_bad_indices():
    lens = [100, 40, 16]
    c, q, table = _decode_case(128, 2, 4, lens, "bf16", "bf16", 12)
    t2 = table.copy()
    t2[0, 2], t2[1, :], t2[2, 0] = c.cfg.num_blocks, -5, 1 << 30
    got = _np(c.decode(q.cuda(), _gpu(t2), _gpu(np.array(lens, np.int32)), out_dtype=torch.float32))
    assert c.device_error() == tq.TQ_DEVERR_BLOCK
    pages = c.pages().cpu().numpy()
    k, v = f8.rows(pages, table[0], 100, 128)
    keep = np.r_[0:32, 48:100]
    ref, _, mag = f8.attention(_np(q)[:1], k[keep], v[keep], 1 / np.sqrt(128))
    assert (np.abs(got[0] - ref[0]) <= _bound(_np(q)[:1], k[keep], v[keep], 1 / np.sqrt(128), mag, ref, True,
                                              torch.float32)[0]).all()
    assert not got[1:].any()
    # lengths outside the table are clamped: -4 is none, one past it is all its columns
    got = c.decode(q.cuda(), _gpu(table), _gpu(np.array([-4, 10 ** 6, 16], np.int32)), out_dtype=torch.float32)
    assert c.device_error() & tq.TQ_DEVERR_SEQLEN
    assert not _np(got)[0].any()


def test_decode_strided_queries_streams_and_graphs():
    lens = [500, 33, 1200]
    c, q, table = _decode_case(128, 2, 4, lens, "bf16", "bf16", 13)
    td, ld = _gpu(table), _gpu(np.array(lens, np.int32))
    wide = torch.randn((3, 20, 128), device="cuda").to(torch.bfloat16)
    wide[:, 5:13] = q.cuda()
    ref = c.decode(q.cuda(), td, ld)
    assert torch.equal(c.decode(wide[:, 5:13], td, ld), ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(ref)
    c.decode(wide[:, 5:13], td, ld, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
    # a captured step, replayed with other lengths and other tokens in the same buffers
    k, v = (torch.randn((3, 2, 128), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    slots = _gpu(np.array([table[b, (n - 1) // 16] * 16 + (n - 1) % 16 for b, n in enumerate(lens)], np.int64))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.store(k, v, slots)
        c.decode(wide[:, 5:13], td, ld, out=out)
    for n in ([500, 33, 1200], [499, 0, 16], [1, 2, 3]):
        ld.copy_(torch.tensor(n, dtype=torch.int32))
        k.normal_()
        wide.normal_()
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, c.decode(wide[:, 5:13], td, ld))
        _check_decode(c, wide[:, 5:13], table, n, "bf16", got)


def test_decode_allocates_its_output_on_the_given_stream():
    """A block that the current stream still writes to is not handed to a call on another stream."""
    lens = [70, 33] * 60
    c, q, table = _decode_case(128, 2, 4, lens, "bf16", "bf16", 41)
    args = (q.cuda(), _gpu(table), _gpu(np.array(lens, np.int32)))
    want = c.decode(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.empty_like(want) for _ in range(200)]  # every free block of this size
    at = {x.data_ptr() for x in old}
    torch.cuda._sleep(20_000_000)  # about 10 ms
    for x in old:
        x.fill_(3)
    del old, x
    got = c.decode(*args, stream=side)
    assert got.data_ptr() not in at
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_two_handles_on_two_streams():
    lens = [3000, 40]
    made = [_decode_case(128, 1, 4, lens, "bf16", "bf16", 20 + i) for i in range(2)]
    args = [(q.cuda(), _gpu(t), _gpu(np.array(lens, np.int32))) for _, q, t in made]
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
    blocks = (5 << 30) // (hkv * (32 * d + 32))
    c = tq.TQF8Cache(head_dim=d, num_kv_heads=hkv, num_q_heads=32, num_blocks=blocks, max_batch=1,
                     max_blocks_per_seq=40, cache=torch.empty(blocks * hkv * (32 * d + 32), dtype=torch.uint8,
                                                              device="cuda"))
    n = 600
    table = np.arange(blocks - 40, blocks, dtype=np.int32)[None, ::-1].copy()
    rng = _rng(14)
    k, v = (_gpu(rng.standard_normal((n, hkv, d)), torch.bfloat16) for _ in range(2))
    c.store(k, v, _gpu(_slots(table, [n])))
    rows = (1 << 31) // (hkv * d) + 700  # output offsets past 2^31 elements
    ko = torch.empty((rows, hkv, d), dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(ko)
    ld = _gpu(np.array([n], np.int32))
    c.load(_gpu(table), ld, _gpu(np.array([rows - n], np.int32)), ko, vo)
    for got, x in ((ko[-n:], k), (vo[-n:], v)):
        assert np.array_equal(_np(got), f8.values(*f8.quantise(_np(x))))
    q = torch.randn((1, 32, d), device="cuda").to(torch.bfloat16)
    got = c.decode(q, _gpu(table), ld)
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
        tq.TQF8Cache(head_dim=128, num_kv_heads=2, num_q_heads=8, num_blocks=4, max_blocks_per_seq=2, cache=c.cache[:-1])
    with pytest.raises(ValueError):
        tq.tq_f8_decode_attention(c.handle, c.cfg, q, c.cache[:-1], t, n, q.clone())
