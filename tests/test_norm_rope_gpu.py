"""Norm with rotation on the GPU against its fp64 oracle (oracle/serve.py).

The bound.  The norm's factor: squares and their sum round at most 20 times (16 in
a lane, 4 or 5 exchanges) by 2^-24 of a sum of positive terms, half of which
reaches the root; rsqrt errs by 2^-22; with the products by it and by the weight an
element is off by at most 2^-24 (10 + 4 + 2) = 2^-20 of itself.  The angle is cut
off to 2^-32 of a turn (2^-29) and rounded to 2^-25 of half a turn (2^-23); sine
and cosine err by 2^-22 at most: together 2^-21.  The two products of a rotation
add 2^-23.  So 2^-19.3 of |a| + |b|, the elements of the pair; then half a step of
the output's type."""

import numpy as np
import pytest

import turboquant_bit_kv_tq_gb300 as tq
from oracle import serve

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _np(t):
    return t.double().cpu().numpy()


def _gpu(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def _check(got, x, w, pos, f, eps, interleaved=False, norm=True):
    want, size = serve.norm_rope(_np(x), None if w is None else _np(w), pos, f, eps, interleaved, norm)
    fin = torch.finfo(got.dtype)
    # (a subnormal of the type rounds by half its step, a result beyond it to an infinity)
    tol = 2.0 ** -19.3 * size + np.maximum(fin.eps / 2 * np.abs(want), fin.smallest_normal * fin.eps / 2) + 2.0 ** -149
    g = _np(got)
    assert np.isfinite(g).all()
    err = np.abs(g - want)
    assert (err <= tol).all(), (err.max(), (err / tol).max())


def _inputs(seed, n, hq, hk, d, dtype, wt=None, gain=1.0):
    rng = np.random.default_rng((81, seed))
    made = [_gpu(rng.standard_normal((n, h, d)) * gain * np.exp(rng.uniform(-3, 3, (n, h, 1))), DT[dtype])
            for h in (hq, hk, hk)]
    w = [_gpu(1 + 0.2 * rng.standard_normal(d), DT[wt or dtype]) for _ in range(2)]
    pos = rng.integers(-50, 1 << 20, n).astype(np.int32)
    return made, w, pos


@pytest.mark.parametrize("n,hq,hk,d,rot,dtype,wt,interleaved", [
    (1, 32, 8, 128, 128, "bf16", "bf16", False),
    (1, 1, 1, 128, 128, "f32", "f32", True),
    (37, 5, 1, 128, 64, "f16", "f32", False),
    (16, 8, 2, 256, 256, "bf16", "f32", False),
    (19, 3, 3, 256, 96, "f32", "bf16", True),
    (50, 4, 4, 128, 16, "bf16", "f16", False),
    (33, 2, 1, 256, 16, "f16", "f16", True),
    (9, 7, 2, 128, 0, "bf16", "bf16", False),
    (700, 32, 8, 128, 128, "bf16", "bf16", True),
    (1500, 12, 4, 256, 64, "f32", "f32", False),
    (5000, 3, 1, 128, 96, "bf16", "bf16", False),
    (2000, 64, 8, 128, 128, "bf16", "bf16", False),
    (3, 300, 2, 128, 128, "bf16", "bf16", False),
])
def test_norm_and_rotation(n, hq, hk, d, rot, dtype, wt, interleaved):
    (q, k, v), (wq, wk), pos = _inputs(n + hq, n, hq, hk, d, dtype, wt)
    h = tq.TQNormRope(head_dim=d, num_q_heads=hq, num_kv_heads=hk, rot_dim=rot, base=5e5, interleaved=interleaved)
    f = serve.powers(5e5, rot) if rot else np.zeros(0)
    qo, ko = h.apply(q, k, _gpu(pos), wq, wk)
    some = np.arange(n) if n < 60 else np.r_[0:20, n // 2:n // 2 + 9, n - 20:n]
    at = _gpu(some)
    eps = float(np.float32(1e-6))
    _check(qo[at], q[at], wq, pos[some], f, eps, interleaved)
    _check(ko[at], k[at], wk, pos[some], f, eps, interleaved)
    # keys and values to rows of longer buffers, some left out; other rows stay
    rng = np.random.default_rng((82, n))
    rows = rng.permutation(2 * n + 1)[:n].astype(np.int32)
    rows[::5] = -1
    long = [torch.full((2 * n + 1, hk, d), -7.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    out = h.apply(q, k, _gpu(pos), wq, wk, k_out=long[0], v=v, v_out=long[1], kv_rows=_gpu(rows))
    assert out[1] is long[0] and out[2] is long[1] and torch.equal(out[0], qo)
    want = [torch.full_like(long[0], -7.0) for _ in range(2)]
    live = _gpu(np.flatnonzero(rows >= 0))
    want[0][_gpu(rows[rows >= 0]).long()], want[1][_gpu(rows[rows >= 0]).long()] = ko[live], v[live]
    assert torch.equal(long[0], want[0]) and torch.equal(long[1], want[1])
    assert h.device_error() == 0


def test_far_positions_and_given_frequencies():
    rng = np.random.default_rng(83)
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1234567890, 10 ** 6 + 1, -77], np.int32)
    f = np.r_[rng.uniform(0, 3, 58), 6.5, 100.25, 1e-9, 0.0, -0.3, 2.0 ** 40 + 0.125]
    q, k = _gpu(rng.standard_normal((8, 2, 128)), torch.float32), _gpu(rng.standard_normal((8, 1, 128)), torch.float32)
    for interleaved in (False, True):
        h = tq.TQNormRope(head_dim=128, num_q_heads=2, num_kv_heads=1, inv_freq=f, interleaved=interleaved)
        qo, ko = h.apply(q, k, _gpu(pos))
        _check(qo, q, None, pos, f, float(np.float32(1e-6)), interleaved)
        _check(ko, k, None, pos, f, float(np.float32(1e-6)), interleaved)


def test_rotation_alone_and_one_weight():
    (q, k, _), (wq, _), pos = _inputs(5, 21, 4, 2, 128, "bf16")
    f = serve.powers(1e4, 128)
    h = tq.TQNormRope(head_dim=128, num_q_heads=4, num_kv_heads=2, norm=0)
    qo, ko = h.apply(q, k, _gpu(pos), wq)  # (weights are the norm's)
    _check(qo, q, None, pos, f, 0.0, norm=False)
    _check(ko, k, None, pos, f, 0.0, norm=False)
    h = tq.TQNormRope(head_dim=128, num_q_heads=4, num_kv_heads=2, eps=1e-3)
    qo, ko = h.apply(q, k, _gpu(pos), q_weight=wq)
    _check(qo, q, wq, pos, f, float(np.float32(1e-3)))
    _check(ko, k, None, pos, f, float(np.float32(1e-3)))


@pytest.mark.parametrize("dtype,gains", [("f32", (2.0 ** 100, 2.0 ** 120, 2.0 ** -70, 2.0 ** -120, 2.0 ** -135)),
                                         ("bf16", (2.0 ** 100, 2.0 ** 120, 2.0 ** -70, 2.0 ** -120)),
                                         ("f16", (2.0 ** 9, 2.0 ** -9))])
@pytest.mark.parametrize("d", [128, 256])
def test_squares_beyond_the_range(dtype, gains, d):
    """Elements whose squares over- or underflow, beside an ordinary eps, a tiny one and none."""
    pos = np.arange(6, dtype=np.int32)
    f = serve.powers(1e4, d)
    for gain in gains:
        for eps in (1e-6, 1e-35, 0.0):
            (q, k, _), (wq, wk), _ = _inputs(6, 6, 2, 1, d, dtype, gain=gain)
            q[2] = 0 if eps else q[1]
            h = tq.TQNormRope(head_dim=d, num_q_heads=2, num_kv_heads=1, eps=eps)
            qo, ko = h.apply(q, k, _gpu(pos), wq, wk)
            _check(qo, q, wq, pos, f, float(np.float32(eps)))
            _check(ko, k, wk, pos, f, float(np.float32(eps)))


def test_what_is_not_finite_stays_in_its_head():
    (q, k, _), (wq, wk), pos = _inputs(7, 9, 4, 2, 128, "bf16")
    h = tq.TQNormRope(head_dim=128, num_q_heads=4, num_kv_heads=2, rot_dim=64)
    clean = h.apply(q, k, _gpu(pos), wq, wk)
    q[3, 1, 5], k[4, 0, 100] = float("nan"), float("inf")
    got = h.apply(q, k, _gpu(pos), wq, wk)
    assert torch.isnan(got[0][3, 1]).all() and torch.isnan(got[1][4, 0, 100])
    for a, b, (t, hd) in ((got[0], clean[0], (3, 1)), (got[1], clean[1], (4, 0))):
        a[t, hd], b[t, hd] = 0, 0
        assert torch.equal(a, b)


@pytest.mark.parametrize("d,dtype,interleaved", [(128, "bf16", False), (256, "f32", True)])
def test_rows_of_a_projection_in_place_streams_and_graphs(d, dtype, interleaved):
    n, hq, hk = 45, 6, 2
    (q, k, v), (wq, wk), pos = _inputs(8, n, hq, hk, d, dtype)
    h = tq.TQNormRope(head_dim=d, num_q_heads=hq, num_kv_heads=hk, interleaved=interleaved)
    p = _gpu(pos)
    want = h.apply(q, k, p, wq, wk)
    qkv = torch.cat([q, k, v], 1)
    a, b, c = qkv.split([hq, hk, hk], 1)
    got = h.apply(a, b, p, wq, wk)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    keep = qkv.clone()
    h.apply(a, b, p, wq, wk, q_out=a, k_out=b)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(c, v)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = h.apply(q, k, p, wq, wk, v=v, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.apply(a, b, p, wq, wk, q_out=a, k_out=b)
    for _ in range(2):
        qkv.copy_(keep)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(c, v)


def test_outputs_are_allocated_on_the_given_stream():
    (q, k, _), (wq, wk), pos = _inputs(9, 60, 4, 4, 128, "bf16")
    h = tq.TQNormRope(head_dim=128, num_q_heads=4, num_kv_heads=4)
    p = _gpu(pos)
    want = h.apply(q, k, p, wq, wk)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.empty_like(q) for _ in range(200)]  # every free block of this size
    torch.cuda._sleep(20_000_000)  # about 10 ms
    for x in old:
        x.fill_(3)
    del old, x
    got = h.apply(q, k, p, wq, wk, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_outside_are_left_out_and_reported():
    (q, k, v), (wq, wk), pos = _inputs(10, 6, 2, 1, 128, "bf16")
    h = tq.TQNormRope(head_dim=128, num_q_heads=2, num_kv_heads=1)
    ko, vo = (torch.full((4, 1, 128), -7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rows = np.array([3, -1, 4, -2, 0, 2 ** 31 - 1], np.int32)
    h.apply(q, k, _gpu(pos), wq, wk, k_out=ko, v=v, v_out=vo, kv_rows=_gpu(rows))
    assert h.device_error() == tq.TQ_DEVERR_CHUNK and h.device_error() == 0
    assert torch.equal(vo[3], v[0]) and torch.equal(vo[0], v[4]) and (vo[1:3] == -7).all() and (ko[1:3] == -7).all()
    h.apply(q[:0], k[:0], _gpu(pos[:0]), wq, wk)  # no token: nothing


def test_many_vectors():
    """More vectors than 2^31 elements of output offsets."""
    n, hq, hk, d = 70000, 250, 1, 128
    q = torch.randn((1, hq, d), device="cuda").to(torch.bfloat16).expand(n, hq, d).contiguous()
    k = torch.randn((n, hk, d), device="cuda").to(torch.bfloat16)
    h = tq.TQNormRope(head_dim=d, num_q_heads=hq, num_kv_heads=hk)
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    h.apply(q, k, pos, q_out=q)
    assert torch.equal(q[0], q[-1]) and torch.equal(q[0], q[n // 2 + 1]) and bool((q == q[:1]).all())
    _check(q[:1], q[:1], None, [0], serve.powers(1e4, 128), 0.0, norm=True)


def test_refusals():
    (q, k, v), (wq, wk), pos = _inputs(11, 6, 2, 1, 128, "bf16")
    h = tq.TQNormRope(head_dim=128, num_q_heads=2, num_kv_heads=1)
    p = _gpu(pos)
    for error, call in [
        (TypeError, lambda: h.apply(q.half(), k, p)),
        (TypeError, lambda: h.apply(q, k, p, wq, wk.float())),
        (TypeError, lambda: h.apply(q, k, p.long())),
        (TypeError, lambda: h.apply(q, k, p, wq.int())),
        (ValueError, lambda: h.apply(q, k[:5], p)),
        (ValueError, lambda: h.apply(q, k, p[:5])),
        (ValueError, lambda: h.apply(q[:, :1], k, p)),
        (ValueError, lambda: h.apply(q, k, p, wq[:64])),
        (ValueError, lambda: h.apply(q, k, p, q_out=q[:3])),
        (ValueError, lambda: h.apply(q, k, p, k_out=torch.cat([k, k]))),
        (ValueError, lambda: h.apply(q, k, p, kv_rows=p)),
        (ValueError, lambda: h.apply(q, k, p, v=v[:4])),
        (ValueError, lambda: h.apply(q, k, p, v_out=v)),
        (ValueError, lambda: h.apply(q.cpu(), k, p)),
        (ValueError, lambda: h.apply(q, k, p.cpu())),
    ]:
        with pytest.raises(error):
            call()
    odd = torch.zeros(6 * 2 * 128 + 8, dtype=torch.bfloat16, device="cuda")[1:-7].view(6, 2, 128)
    with pytest.raises(tq.TQError) as e:
        h.apply(odd, k, p)
    assert e.value.status == -5
    with pytest.raises(tq.TQError) as e:
        tq.TQNormRope(head_dim=128, num_q_heads=2, num_kv_heads=1, inv_freq=np.full(64, np.nan))
    assert e.value.status == -1


# ------------------------------------------------------------- many tokens
# (from two pieces of 6 to 13 KB per SM on, rows go through shared memory)
@pytest.mark.parametrize("n,hq,hk,d,rot,dtype,interleaved", [
    (400, 24, 1, 128, 128, "bf16", False), (401, 23, 3, 128, 64, "bf16", True), (700, 90, 5, 128, 128, "f16", False),
    (400, 7, 2, 256, 96, "f32", True), (1300, 25, 2, 128, 16, "f32", False), (333, 12, 12, 256, 256, "bf16", False),
    (900, 3, 24, 128, 0, "bf16", False),
])
def test_many_tokens(n, hq, hk, d, rot, dtype, interleaved):
    (q, k, v), (wq, wk), pos = _inputs(n + hq, n, hq, hk, d, dtype, "f32")
    h = tq.TQNormRope(head_dim=d, num_q_heads=hq, num_kv_heads=hk, rot_dim=rot, base=5e5, interleaved=interleaved)
    f = serve.powers(5e5, rot) if rot else np.zeros(0)
    eps, p = float(np.float32(1e-6)), _gpu(pos)
    some = np.r_[0:9, n // 2:n // 2 + 9, n - 9:n]
    at = _gpu(some)
    qkv = torch.cat([q, k, v], 1)
    a, b, c = qkv.split([hq, hk, hk], 1)
    qo, ko = h.apply(a, b, p, wq, wk)
    _check(qo[at], q[at], wq, pos[some], f, eps, interleaved)
    _check(ko[at], k[at], wk, pos[some], f, eps, interleaved)
    # few of the same rows in a call of their own, which the other kernel takes
    part = h.apply(a[7:20], b[7:20], p[7:20], wq, wk)
    _check(part[0], q[7:20], wq, pos[7:20], f, eps, interleaved)
    _check(part[1], k[7:20], wk, pos[7:20], f, eps, interleaved)
    # rows of longer buffers, some left out, some outside
    rng = np.random.default_rng((84, n))
    rows = rng.permutation(2 * n)[:n].astype(np.int32)
    rows[::5], rows[3], rows[n - 2] = -1, 2 * n, -7
    long = [torch.full((2 * n, hk, d), -7.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    h.apply(a, b, p, wq, wk, k_out=long[0], v=c, v_out=long[1], kv_rows=_gpu(rows))
    assert h.device_error() == tq.TQ_DEVERR_CHUNK and h.device_error() == 0
    good = (rows >= 0) & (rows < 2 * n)
    want = [torch.full_like(long[0], -7.0) for _ in range(2)]
    want[0][_gpu(rows[good]).long()], want[1][_gpu(rows[good]).long()] = ko[_gpu(good)], v[_gpu(good)]
    assert torch.equal(long[0], want[0]) and torch.equal(long[1], want[1])
    # in place, captured and replayed
    keep = qkv.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        h.apply(a, b, p, wq, wk, q_out=a, k_out=b)
    for _ in range(2):
        qkv.copy_(keep)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, qo) and torch.equal(b, ko) and torch.equal(c, v)


@pytest.mark.parametrize("gain,eps", [(2.0 ** 120, 1e-6), (2.0 ** -70, 0.0), (2.0 ** -120, 1e-35), (1.0, 1e-6)])
def test_many_tokens_beyond_the_range_and_not_finite(gain, eps):
    n, hq, hk, d = 350, 24, 2, 128
    (q, k, _), (wq, wk), pos = _inputs(12, n, hq, hk, d, "f32", gain=gain)
    h = tq.TQNormRope(head_dim=d, num_q_heads=hq, num_kv_heads=hk, rot_dim=64, eps=eps)
    clean = h.apply(q, k, _gpu(pos), wq, wk)
    some, f = np.r_[0:4, n - 4:n], serve.powers(1e4, 64)
    _check(clean[0][_gpu(some)], q[_gpu(some)], wq, pos[some], f, float(np.float32(eps)))
    _check(clean[1][_gpu(some)], k[_gpu(some)], wk, pos[some], f, float(np.float32(eps)))
    q[3, 1, 5], k[344, 0, 100] = float("nan"), float("inf")
    got = h.apply(q, k, _gpu(pos), wq, wk)
    assert torch.isnan(got[0][3, 1]).all() and torch.isnan(got[1][344, 0, 100])
    for a, b, (t, hd) in ((got[0], clean[0], (3, 1)), (got[1], clean[1], (344, 0))):
        a[t, hd], b[t, hd] = 0, 0
        assert torch.equal(a, b)


@pytest.mark.parametrize("n", [21, 500])
def test_rows_that_start_at_odd_multiples_of_sixteen_bytes(n):
    (q, k, v), (wq, wk), pos = _inputs(13, n, 24, 2, 128, "bf16")
    h = tq.TQNormRope(head_dim=128, num_q_heads=24, num_kv_heads=2)
    want = h.apply(q, k, _gpu(pos), wq, wk, v=v)

    def apart(x):
        w = torch.zeros((n, x[0].numel() + 8), dtype=x.dtype, device="cuda")
        w[:, :-8] = x.flatten(1)
        return w, w[:, :-8].unflatten(1, x.shape[1:])

    ins, outs = [apart(x) for x in (q, k, v)], [apart(torch.zeros_like(x)) for x in (q, k, v)]
    h.apply(ins[0][1], ins[1][1], _gpu(pos), wq, wk, q_out=outs[0][1], k_out=outs[1][1], v=ins[2][1], v_out=outs[2][1])
    for (whole, got), x in zip(outs, want):
        assert torch.equal(got, x) and not whole[:, -8:].any()


def test_one_handle_on_two_streams():
    h = tq.TQNormRope(head_dim=128, num_q_heads=24, num_kv_heads=2)
    made = [_inputs(14 + i, n, 24, 2, 128, "bf16") for i, n in enumerate((600, 40))]
    args = [(q, k, _gpu(pos), wq, wk) for (q, k, _), (wq, wk), pos in made]
    want = [h.apply(*a) for a in args]
    outs = [[torch.zeros_like(x) for x in w] for w in want]
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    for _ in range(20):
        for a, o, s in zip(args, outs, streams):
            h.apply(*a, q_out=o[0], k_out=o[1], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for o, w in zip(outs, want) for x, y in zip(o, w))


def test_in_place_with_another_stride_is_refused():
    h = tq.TQNormRope(head_dim=128, num_q_heads=2, num_kv_heads=2)
    rows = torch.zeros(6, 1024, dtype=torch.bfloat16, device="cuda")
    apart = [rows[:, at:at + 256].view(6, 2, 128) for at in (0, 256, 512)]
    p = torch.arange(6, dtype=torch.int32, device="cuda")

    def near(x):
        return torch.as_strided(x, (6, 2, 128), (256, 128, 1))

    q, k, v = apart
    own = torch.zeros(6, 2, 128, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(q_out=near(q), k_out=k), dict(q_out=q, k_out=near(k)), dict(q_out=q, k_out=k, v=v, v_out=near(v))):
        with pytest.raises(tq.TQError) as e:
            h.apply(q, k, p, **kw)
        assert e.value.status == -1
    # (with the same stride, a single row, or the keys somewhere else it is a call like any other)
    h.apply(q, k, p, q_out=q, k_out=k, v=v, v_out=v)
    h.apply(q[:1], k[:1], p[:1], q_out=near(q)[:1], k_out=near(k)[:1])
    h.apply(q, k, p, q_out=q, k_out=own, kv_rows=p)
    torch.cuda.synchronize()
    assert h.device_error() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_frequencies_below_zero_are_as_exact_as_the_others(interleaved):
    """The bound: less than 2^-32 of a turn is cut off, and half a unit of 2^-64 of a turn a position (2^-34 at the
    farthest): 2^-29 together; fp32 rounds the reduced angle t by 2^-24 of itself, and a sine or cosine errs by two
    units at most, 2^-22 of itself.  So small sines show the angle itself, which a frequency of 53 bits behind the
    point would miss by up to 2^-20 at the farthest positions."""
    rng = np.random.default_rng(85)
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 77, 1234567890, -2000000011], np.int32)
    f = np.r_[0.3, 1e-3, 1e-6, 1e-9, 1e-12, 7e-16, 3e-16, 1e-17, 1e-30, 2.0 ** -54, 2.0 ** -60 * 6.28, 5.0,
              np.exp(rng.uniform(-35, 2, 52))]
    # (a pair's first element 1, its second 0: the outputs are cosines and sines)
    pair = torch.tensor([1.0, 0.0], device="cuda")
    q = (pair.repeat(64) if interleaved else pair.repeat_interleave(64)).expand(8, 1, 128).contiguous()
    for sign in (1.0, -1.0):
        h = tq.TQNormRope(head_dim=128, num_q_heads=1, num_kv_heads=1, inv_freq=sign * f, interleaved=interleaved, norm=0)
        y = _np(h.apply(q, q, _gpu(pos))[0]).reshape(8, *((64, 2) if interleaved else (2, 64)))
        c, s = (y[..., 0], y[..., 1]) if interleaved else (y[:, 0], y[:, 1])
        t = serve.angles(pos, sign * f)
        angle = 2.0 ** -29 + 2.0 ** -24 * np.abs(t)
        assert (np.abs(c - np.cos(t)) <= angle + 2.0 ** -22).all(), sign
        err = np.abs(s - np.sin(t)) / (angle + 2.0 ** -22 * np.abs(np.sin(t)))
        assert (err <= 1).all(), (sign, f[err.max(0).argmax()], err.max())


def test_rows_behind_two_to_the_31_elements():
    """Rows that differ, with positions of their own, at the ends and where an element's offset passes 2^31 (and 2^32
    bytes); outputs in memory of their own, the others' too."""
    n, hq, hk, d = 70000, 250, 1, 128
    row = hq * d
    q, out = (torch.zeros((n, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, k_out = (torch.zeros((n, hk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    edge = 2 ** 31 // row
    some = np.concatenate([np.arange(x - 2, x + 3) for x in (2, n - 3 - edge, edge // 2, edge, n - 3)])
    rng = np.random.default_rng(86)
    at, pos = _gpu(some), torch.zeros(n, dtype=torch.int32, device="cuda")
    q[at] = _gpu(rng.standard_normal((len(some), hq, d)), torch.bfloat16)
    k[at] = _gpu(rng.standard_normal((len(some), hk, d)), torch.bfloat16)
    p = rng.integers(1, 1 << 20, len(some)).astype(np.int32)
    pos[at] = _gpu(p)
    h = tq.TQNormRope(head_dim=d, num_q_heads=hq, num_kv_heads=hk)
    out.fill_(7)
    h.apply(q, k, pos, q_out=out, k_out=k_out)
    f, eps = serve.powers(1e4, 128), float(np.float32(1e-6))
    _check(out[at], q[at], None, p, f, eps)
    _check(k_out[at], k[at], None, p, f, eps)
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert not bool((out.amax((1, 2)) != 0)[rest].any()) and not bool((out.amin((1, 2)) != 0)[rest].any())
    # keys from the last row to the first and back: every row goes where it is sent
    rows = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")
    back = torch.zeros_like(k_out)
    h.apply(q, k, pos, q_out=q, k_out=back, kv_rows=rows)
    assert torch.equal(back.flip(0), k_out) and torch.equal(q, out)
    assert h.device_error() == 0
