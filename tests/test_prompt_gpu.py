"""Prompt attention on the GPU against the fp64 oracle (oracle/f8.attention),
and as it is used: a prompt in chunks through the 8-bit cache, then decode."""

import numpy as np
import pytest

import turboquant_bit_kv_tq_gb300 as tq
from oracle import f8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _gpu(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def _np(t):
    return t.double().cpu().numpy()


def _starts(lens):
    return np.cumsum([0] + list(lens)).astype(np.int32)


def _bounds(q, k, scale, mag, ref, dtype, m):
    """How far outputs and lse may be from the oracle's.  Probabilities rounded to
    dtype (half a step each; fp16 ones below 2^-14 an absolute 2^-25 beside a
    largest of at least 1); scores accumulated in fp32 over d/16 tensor-core
    steps, two units of 2^-23 of sum |q||k| each; exponentials within 2^-22 and
    their argument's rounding; sums of m terms over 128 (64) keys at a time; one
    output rounding."""
    half = torch.finfo(dtype).eps / 2
    d, g = q.shape[2], q.shape[1] // k.shape[1]
    s = np.einsum("nhd,mhd->nhm", np.abs(q), np.repeat(np.abs(k), g, 1)).max(-1) * scale if m else np.zeros(q.shape[:2])
    ds = s * ((d / 16) * 2.0 ** -22 + 4 * 2.0 ** -24) + 2.0 ** -22 * (2 + 1.45 * s)
    sums = (m / 64 + 128) * 2.0 ** -23
    rel = half + 2 * (ds + sums)[..., None]
    tiny = 2.0 ** -25 * m ** 0.5 * (np.abs(mag).max() if m else 0)
    return rel * mag + half * np.abs(ref) + tiny + 1e-30, 2 * (ds + sums) + 2.0 ** -22 * (4 + s)


def _check(q, k, v, lq, lk, causal, out, lse, scale=None, skip=()):
    cq, ck = _starts(lq), _starts(lk)
    sc = 1 / np.sqrt(q.shape[2]) if scale is None else scale
    qn, kn, vn, on = _np(q), _np(k), _np(v), _np(out)
    ln = None if lse is None else _np(lse)
    for b, (n, m) in enumerate(zip(lq, lk)):
        if n == 0 or b in skip:
            continue
        qs, ks, vs = qn[cq[b]:cq[b + 1]], kn[ck[b]:ck[b + 1]], vn[ck[b]:ck[b + 1]]
        limit = np.arange(n) + 1 + m - n if causal else np.full(n, m)
        ref, z, mag = f8.attention(qs, ks, vs, sc, limit)
        seen = limit > 0
        tol, tz = _bounds(qs, np.nan_to_num(ks, nan=0, posinf=0, neginf=0), sc, np.nan_to_num(mag), np.nan_to_num(ref),
                          q.dtype, m)
        got = on[cq[b]:cq[b + 1]]
        bad = ~(np.abs(got - ref) <= tol) & np.isfinite(ref)
        assert not bad.any(), (b, n, m, np.argwhere(bad)[:4], np.nanmax(np.abs(got - ref)), np.nanmax(np.abs(got - ref) / tol))
        assert np.array_equal(np.isfinite(got), np.isfinite(ref)), (b, n, m)
        assert not got[~seen].any()
        if ln is not None:
            gz = ln[cq[b]:cq[b + 1]]
            assert np.isneginf(gz[~seen]).all()
            err = np.abs(gz[seen] - z[seen])
            assert (err <= tz[seen] + 2.0 ** -23 * np.abs(z[seen])).all(), (b, n, m, err.max())


def _case(d, g, h, lq, lk, dtype, seed, gain=1.0):
    rng = np.random.default_rng((7, d, g, h, seed))
    n, m = sum(lq), sum(lk)
    q = _gpu(rng.standard_normal((n, g * h, d)) * gain, DT[dtype])
    k = _gpu(rng.standard_normal((m, h, d)) * np.exp(0.5 * rng.standard_normal((h, d))), DT[dtype])
    v = _gpu(rng.standard_normal((m, h, d)), DT[dtype])
    p = tq.TQPrompt(head_dim=d, num_kv_heads=h, num_q_heads=g * h, dtype=DT[dtype], max_batch=len(lq) + 1,
                    max_tokens=max(1, n))
    return p, q, k, v, _gpu(_starts(lq)), _gpu(_starts(lk))


def _run(p, q, k, v, cq, ck, **kw):
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = p.attention(q, k, v, cq, ck, lse=lse, **kw)
    return out, lse


SHAPES = [
    (128, 1, 1, [1], [1]),
    (128, 4, 2, [5], [5]),
    (128, 4, 2, [31, 32, 33], [31, 32, 33]),
    (128, 1, 2, [127, 128, 129, 0, 1], [127, 128, 129, 0, 1]),
    (128, 1, 1, [255, 256, 257, 300], [255, 256, 257, 300]),
    (128, 8, 1, [700], [700]),
    (128, 3, 2, [200, 43], [200, 43]),
    (128, 5, 1, [60, 2], [60, 2]),
    (128, 16, 1, [50, 17], [50, 17]),
    (128, 40, 1, [7, 9], [7, 9]),
    (128, 128, 1, [3], [5]),
    (128, 4, 1, [40, 3, 64], [500, 1, 64]),            # chunks behind prefixes, fewer keys than queries
    (128, 2, 2, [130, 5, 260], [2, 0, 130]),           # rows that see nothing, no key at all
    (256, 1, 1, [1, 64, 65, 127, 128, 129], [1, 64, 65, 127, 128, 129]),
    (256, 8, 2, [100, 33], [100, 33]),
    (256, 4, 1, [400], [400]),
    (256, 3, 1, [10, 90, 0], [300, 90, 4]),
    (256, 2, 1, [200, 4], [3, 0]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,g,h,lq,lk", SHAPES)
def test_prompt(d, g, h, lq, lk, dtype, causal):
    p, q, k, v, cq, ck = _case(d, g, h, lq, lk, dtype, len(lq))
    out, lse = _run(p, q, k, v, cq, ck, causal=causal)
    assert p.device_error() == 0
    _check(q, k, v, lq, lk, causal, out, lse)
    again, _ = _run(p, q, k, v, cq, ck, causal=causal)
    assert torch.equal(out, again)


def test_long_prompt_and_many_short_ones():
    for d, g, h, lq in ((128, 4, 1, [3100]), (256, 2, 1, [1500]), (128, 4, 2, list(np.random.default_rng(3).integers(0, 150, 90)))):
        lq = [int(x) for x in lq]
        p, q, k, v, cq, ck = _case(d, g, h, lq, lq, "bf16", 11)
        out, lse = _run(p, q, k, v, cq, ck)
        assert p.device_error() == 0
        _check(q, k, v, lq, lq, True, out, lse)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,g,h,lq,lk,dtype", [
    (128, 4, 1, [5, 0, 40], [3000, 100, 2500], "bf16"),
    (128, 8, 2, [70], [4100], "f16"),
    (256, 8, 1, [17, 1], [2900, 3], "bf16"),
    (256, 1, 2, [33], [5000], "f16"),
    (128, 1, 1, [300], [2900], "bf16"),
    (128, 4, 1, [6], [0], "bf16"),
])
def test_few_rows_over_many_keys(d, g, h, lq, lk, dtype, causal):
    """The keys are cut into parts that other blocks take, and joined; rows behind the last sequence stay."""
    p, q, k, v, cq, ck = _case(d, g, h, lq, lk, dtype, 19)
    n, pad = sum(lq), 3
    q2 = torch.cat([q, torch.zeros((pad,) + q.shape[1:], device="cuda", dtype=q.dtype)])
    p = tq.TQPrompt(head_dim=d, num_kv_heads=h, num_q_heads=g * h, dtype=DT[dtype], max_batch=3, max_tokens=n + pad)
    out = torch.full(q2.shape, 5.0, device="cuda", dtype=q.dtype)
    lse = torch.full(q2.shape[:2], 7.0, device="cuda")
    p.attention(q2, k, v, cq, ck, out=out, lse=lse, causal=causal)
    assert p.device_error() == 0
    _check(q, k, v, lq, lk, causal, out[:n], lse[:n])
    assert (out[n:] == 5).all() and (lse[n:] == 7).all()
    again = out.clone()
    p.attention(q2, k, v, cq, ck, out=out, lse=lse, causal=causal)
    assert torch.equal(out, again)


def test_parts_with_values_a_row_does_not_see():
    lq, lk = 20, 4000
    p, q, k, v, cq, ck = _case(128, 4, 1, [lq], [lk], "bf16", 20)
    v[lk - 1, 0, 3] = float("inf")
    v[lk - 10, 0, 9] = float("nan")
    v[100, 0, 50] = float("-inf")  # seen by all
    out, _ = _run(p, q, k, v, cq, ck)
    got = _np(out)
    limit = np.arange(lq) + 1 + lk - lq
    clean = v.clone()
    for i, c in ((lk - 1, 3), (lk - 10, 9), (100, 50)):
        clean[i, 0, c] = 0
    ref, _, mag = f8.attention(_np(q), _np(k), _np(clean), 1 / np.sqrt(128), limit)
    tol, _ = _bounds(_np(q), _np(k), 1 / np.sqrt(128), mag, ref, q.dtype, lk)
    want = ref.copy()
    want[:, :, 50] = -np.inf
    want[limit > lk - 1, :, 3] = np.inf
    want[limit > lk - 10, :, 9] = np.nan
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isposinf(got), np.isposinf(want))
    assert np.array_equal(np.isneginf(got), np.isneginf(want)) and (np.abs(got[fin] - want[fin]) <= tol[fin]).all()


def test_peaked_scores_and_a_given_scale():
    # references move in nearly every tile: keys grow along the sequence
    lq = [600]
    p, q, k, v, cq, ck = _case(128, 4, 1, lq, lq, "bf16", 12, gain=3.0)
    k *= torch.linspace(0.2, 3.0, 600, device="cuda")[:, None, None].to(k.dtype)
    out, lse = _run(p, q, k, v, cq, ck)
    _check(q, k, v, lq, lq, True, out, lse)
    out, lse = _run(p, q, k, v, cq, ck, scale=0.25)
    _check(q, k, v, lq, lq, True, out, lse, scale=0.25)
    p, q, k, v, cq, ck = _case(256, 4, 1, lq, lq, "bf16", 13, gain=3.0)
    k *= torch.linspace(0.2, 3.0, 600, device="cuda")[:, None, None].to(k.dtype)
    out, lse = _run(p, q, k, v, cq, ck)
    _check(q, k, v, lq, lq, True, out, lse)


@pytest.mark.parametrize("d,h", [(128, 2), (256, 1)])
def test_rows_of_a_projection(d, h):
    lq = [70, 133]
    g = 4
    qkv = torch.randn((203, g * h + 2 * h, d), device="cuda").to(torch.bfloat16)
    q, k, v = qkv.split([g * h, h, h], 1)
    p = tq.TQPrompt(head_dim=d, num_kv_heads=h, num_q_heads=g * h, max_batch=2, max_tokens=203)
    cu = _gpu(_starts(lq))
    out, lse = _run(p, q, k, v, cu, cu)
    _check(q, k, v, lq, lq, True, out, lse)
    # a single row, whose stride says nothing
    one = torch.randn((1, 5 * h * d + 3), device="cuda").to(torch.bfloat16)[:, :h * d].view(1, h, d)
    cu = _gpu(_starts([1]))
    out, lse = _run(p, q[:1], one, one, cu, cu)
    _check(q[:1], one, one, [1], [1], True, out, lse)


@pytest.mark.parametrize("d", [128, 256])
def test_neighbours_and_rows_behind_the_last_sequence(d):
    """Infinities and NaN in another sequence's rows, and rows no sequence names."""
    lq, lk = [50, 90, 40], [75, 90, 201]
    p, q, k, v, cq, ck = _case(d, 2, 2, lq, lk, "bf16", 14)
    c = _starts(lk)
    k[c[1]:c[2]] = float("nan")
    v[c[1]:c[2]] = float("inf")
    v[c[1] + 3] = float("nan")
    pad = 9
    q2 = torch.cat([q, torch.full((pad,) + q.shape[1:], float("nan"), device="cuda").to(q.dtype)])
    k2 = torch.cat([k, torch.full((pad,) + k.shape[1:], float("nan"), device="cuda").to(k.dtype)])
    v2 = torch.cat([v, torch.full((pad,) + v.shape[1:], float("inf"), device="cuda").to(v.dtype)])
    p = tq.TQPrompt(head_dim=d, num_kv_heads=2, num_q_heads=4, max_batch=3, max_tokens=q2.shape[0])
    out = torch.full(q2.shape, 5.0, device="cuda", dtype=q.dtype)
    lse = torch.full(q2.shape[:2], 7.0, device="cuda")
    for causal in (True, False):
        p.attention(q2, k2, v2, cq, ck, out=out, lse=lse, causal=causal)
        _check(q, k, v, lq, lk, causal, out[:180], lse[:180], skip=(1,))
        assert torch.isnan(out[50:140]).all()
        assert (out[180:] == 5).all() and (lse[180:] == 7).all()


@pytest.mark.parametrize("d,g,lq,lk", [(128, 1, 300, 300), (128, 4, 150, 150), (128, 8, 40, 700), (256, 2, 200, 200),
                                       (256, 8, 20, 333)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_values_a_row_does_not_see(d, g, lq, lk, dtype):
    """Infinities and NaN in keys and values later than a row: no influence; the rows that see them get them."""
    p, q, k, v, cq, ck = _case(d, g, 2, [lq], [lk], dtype, 18)
    at = [lk - 1, lk - 3, lk - lq // 2, lk - lq + 2]
    v[at[0], 0, 5] = float("nan")
    v[at[1], 1, d - 1] = float("inf")
    v[at[2], 0, 0] = float("-inf")
    v[at[2] + 1, 0, 0] = float("inf")  # -inf, then NaN in the rows that see both
    v[at[3], 1, 77] = float("inf")
    k[at[1] + 1, 1, 3] = float("nan")  # the last rows of head 1
    out, lse = _run(p, q, k, v, cq, ck)
    got = _np(out)
    kn, vn, qn = _np(k), _np(v), _np(q)
    limit = np.arange(lq) + 1 + lk - lq
    clean = np.where(np.isfinite(vn), vn, 0.0)
    for h in range(2):
        sl = slice(h * g, (h + 1) * g)
        hurt = limit > at[1] + 1 if h == 1 else np.zeros(lq, bool)  # rows that see the NaN key
        ref, _, mag = f8.attention(qn[:, sl], np.nan_to_num(kn[:, h:h + 1]), clean[:, h:h + 1], 1 / np.sqrt(d), limit)
        tol, _ = _bounds(qn[:, sl], np.nan_to_num(kn[:, h:h + 1]), 1 / np.sqrt(d), mag, ref, q.dtype, lk)
        want = ref.copy()
        for key, col in np.argwhere(~np.isfinite(vn[:, h])):
            with np.errstate(invalid="ignore"):  # -inf + inf
                want[limit > key, :, col] += vn[key, h, col]
        want[hurt] = np.nan
        fin = np.isfinite(want)
        g_h = got[:, sl]
        assert np.array_equal(np.isnan(g_h), np.isnan(want)) and np.array_equal(g_h[~fin & ~np.isnan(want)],
                                                                               want[~fin & ~np.isnan(want)])
        assert (np.abs(g_h[fin] - want[fin]) <= tol[fin]).all()
    assert p.device_error() == 0


@pytest.mark.parametrize("d,g,h,lens,causal", [(128, 4, 4, [3000, 70, 1500], True), (256, 8, 3, [1300, 5, 900], True),
                                               (128, 2, 8, [700, 33, 300, 1000], False), (128, 1, 16, [2500], True)])
def test_rows_keep_their_bits_beside_values_that_are_not_finite(d, g, h, lens, causal):
    """Several items per block; some have such values, at their end, in the middle, in the
    last item of all: a row that sees none of its head is the same bit for bit, one that
    sees one has it in its column and the same bits in the others."""
    p, q, k, v, cq, ck = _case(d, g, h, lens, lens, "bf16", 19 + d + h)
    ref, _ = _run(p, q, k, v, cq, ck, causal=causal)
    rng = np.random.default_rng(d + h)
    n = sum(lens)
    bad = torch.zeros((n, h, d), dtype=torch.bool)
    for key in [0, n // 3, n // 2 + 1, n - 2, n - 1] if not causal else [n // 3, n // 2 + 1, n - 200, n - 2, n - 1]:
        bad[key, int(rng.integers(h)), int(rng.integers(d))] = True
    bad = bad.cuda()
    v2 = torch.where(bad, torch.tensor(float("inf"), dtype=v.dtype, device="cuda"), v)
    out, _ = _run(p, q, k, v2, cq, ck, causal=causal)
    sees = torch.zeros((n, h, d), dtype=torch.bool, device="cuda")  # [query row, KV head, column]
    at = 0
    for m in lens:
        part = bad[at:at + m]
        sees[at:at + m] = part.cumsum(0) > 0 if causal else part.any(0, keepdim=True)
        at += m
    sees = sees.repeat_interleave(g, 1)
    assert torch.equal(out[~sees], ref[~sees])
    assert not torch.isfinite(out[sees]).any() and sees.any()


def test_bad_starts_are_reported_and_stay_inside():
    p, q, k, v, cq, ck = _case(128, 2, 1, [40, 50], [40, 50], "bf16", 15)
    for bad_q, bad_k in (([0, 40, 200], [0, 40, 90]), ([0, 60, 40], [0, 40, 90]), ([0, 40, 90], [-5, 40, 90]),
                         ([0, 40, 90], [0, 40, 1 << 30])):
        p.attention(q, k, v, _gpu(np.array(bad_q, np.int32)), _gpu(np.array(bad_k, np.int32)))
        assert p.device_error() == tq.TQ_DEVERR_CHUNK
    out, lse = _run(p, q, k, v, cq, ck)
    _check(q, k, v, [40, 50], [40, 50], True, out, lse)


def test_streams_graphs_and_no_lse():
    lq = [90, 30]
    p, q, k, v, cq, ck = _case(128, 4, 2, lq, lq, "bf16", 16)
    ref, _ = _run(p, q, k, v, cq, ck)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(ref)
    p.attention(q, k, v, cq, ck, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.attention(q, k, v, cq, ck, out=out)
    for lens in ([90, 30], [1, 119], [120, 0]):
        q.normal_()
        v.normal_()
        cq.copy_(torch.from_numpy(_starts(lens)))
        ck.copy_(torch.from_numpy(_starts(lens)))
        graph.replay()
        torch.cuda.synchronize()
        _check(q, k, v, lens, lens, True, out, None)


def test_output_is_allocated_on_the_given_stream():
    p, q, k, v, cq, ck = _case(128, 4, 2, [90, 30], [90, 30], "bf16", 17)
    want = p.attention(q, k, v, cq, ck)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.empty_like(want) for _ in range(200)]  # every free block of this size
    torch.cuda._sleep(20_000_000)  # about 10 ms
    for x in old:
        x.fill_(3)
    del old, x
    got = p.attention(q, k, v, cq, ck, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("d,g", [(128, 4), (256, 8)])
def test_chunked_prompt_through_the_cache_then_decode(d, g):
    """Two prompts in chunks: read the prefix back, attend, store the chunk; then decode steps."""
    rng = np.random.default_rng((21, d))
    h, total, steps = 2, [150, 77], 3
    hq, dt = g * h, torch.bfloat16
    B, cap = 2, 16
    blocks = B * cap
    table = _gpu(rng.permutation(blocks).reshape(B, cap).astype(np.int32))
    tn = table.cpu().numpy()
    cache = tq.TQF8Cache(head_dim=d, num_kv_heads=h, num_q_heads=hq, num_blocks=blocks, max_batch=B, max_blocks_per_seq=cap)
    cache.cache.fill_(0xFF)
    p = tq.TQPrompt(head_dim=d, num_kv_heads=h, num_q_heads=hq, max_batch=B, max_tokens=256)
    new = [[_gpu(rng.standard_normal((n + steps, x, d)), dt) for x in (hq, h, h)] for n in total]
    done = [0, 0]
    slot = lambda b, t: tn[b, t // 16].astype(np.int64) * 16 + t % 16  # noqa: E731
    for chunk in ([64, 77], [50, 0], [36, 0]):
        q = torch.cat([new[b][0][done[b]:done[b] + chunk[b]] for b in range(B)])
        lk = [done[b] + chunk[b] for b in range(B)]
        ck = _starts(lk)
        k = torch.full((int(ck[-1]), h, d), float("nan"), device="cuda", dtype=dt)
        v = k.clone()
        cache.load(table, _gpu(np.array(done, np.int32)), _gpu(ck), k, v)
        for b in range(B):
            for dst, src in ((k, new[b][1]), (v, new[b][2])):
                dst[ck[b] + done[b]:ck[b + 1]] = src[done[b]:done[b] + chunk[b]]
        out, lse = _run(p, q, k, v, _gpu(_starts(chunk)), _gpu(ck))
        _check(q, k, v, chunk, lk, True, out, lse)
        slots = np.concatenate([slot(b, np.arange(done[b], lk[b])) for b in range(B)])
        cache.store(torch.cat([new[b][1][done[b]:lk[b]] for b in range(B)]),
                    torch.cat([new[b][2][done[b]:lk[b]] for b in range(B)]), _gpu(slots))
        done = lk
    pages_of = lambda: cache.pages().cpu().numpy()  # noqa: E731
    for s in range(steps):
        k = torch.stack([new[b][1][done[b]] for b in range(B)])
        v = torch.stack([new[b][2][done[b]] for b in range(B)])
        cache.store(k, v, _gpu(np.array([slot(b, np.int64(done[b])) for b in range(B)])))
        done = [n + 1 for n in done]
        q = torch.stack([new[b][0][done[b] - 1] for b in range(B)])
        got = _np(cache.decode(q, table, _gpu(np.array(done, np.int32))))
        pages = pages_of()
        for b in range(B):
            kk, vv = f8.rows(pages, tn[b], done[b], d)
            assert np.array_equal(kk[done[b] - 1], f8.values(*f8.quantise(_np(k[b]))))
            ref, _, mag = f8.attention(_np(q[b:b + 1]), kk, vv, 1 / np.sqrt(d))
            assert (np.abs(got[b] - ref[0]) <= 2.0 ** -10 * mag[0] + 2.0 ** -8 * np.abs(ref[0])).all()
    assert cache.device_error() == 0 and p.device_error() == 0


def test_refusals():
    p, q, k, v, cq, ck = _case(128, 2, 2, [8], [8], "bf16", 17)
    for error, call in [
        (TypeError, lambda: p.attention(q.half(), k, v, cq, ck)),
        (TypeError, lambda: p.attention(q, k, v.half(), cq, ck)),
        (ValueError, lambda: p.attention(q, k, v[:4], cq, ck)),
        (ValueError, lambda: p.attention(q[:, :3], k, v, cq, ck)),
        (ValueError, lambda: p.attention(q, k, v, cq, ck[:1])),
        (ValueError, lambda: p.attention(q, k, v, cq[:1], ck[:1])),
        (TypeError, lambda: p.attention(q, k, v, cq.long(), ck.long())),
        (ValueError, lambda: p.attention(q, k, v, cq, ck, out=q[:4])),
        (ValueError, lambda: p.attention(q, k, v, cq, ck, lse=torch.zeros((8, 3), device="cuda"))),
        (TypeError, lambda: p.attention(q, k, v, cq, ck, lse=torch.zeros((8, 4), device="cuda").half())),
        (ValueError, lambda: p.attention(q.cpu(), k, v, cq, ck)),
        (ValueError, lambda: p.attention(q.transpose(0, 1).contiguous().transpose(0, 1), k, v, cq, ck)),
    ]:
        with pytest.raises(error):
            call()
    with pytest.raises(tq.TQError) as e:  # more rows than max_tokens
        p.attention(torch.cat([q, q]), k, v, cq, ck)
    assert e.value.status == -1
    wide = torch.zeros(8 * 4 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(tq.TQError) as e:
        p.attention(wide[1:-7].view(8, 4, 128), k, v, cq, ck)
    assert e.value.status == -5
    for bad, status in [(dict(head_dim=64), -2), (dict(dtype=torch.float32), -2), (dict(num_q_heads=3), -1),
                        (dict(num_q_heads=258, num_kv_heads=2), -2), (dict(max_tokens=0), -1), (dict(max_batch=0), -1)]:
        with pytest.raises(tq.TQError) as e:
            tq.TQPrompt(**{**dict(head_dim=128, num_kv_heads=2, num_q_heads=4, max_batch=1, max_tokens=8), **bad})
        assert e.value.status == status, bad
