"""Prompt attention: work items that follow one another in a block, and references
that move within one, against the fp64 oracle."""

import numpy as np
import pytest

import turboquant_bit_kv_tq_gb300 as tq
from test_prompt_gpu import DT, _case, _check, _gpu, _run, _starts

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _flush():
    """Everything out of L2, so that the call's copies come from memory."""
    torch.empty(256 << 20, dtype=torch.uint8, device="cuda").fill_(1)


@pytest.mark.parametrize("g,causal", [(4, True), (4, False), (1, True), (8, True)])
def test_short_chunks_over_keys_between_short_prompts(g, causal):
    """Many items per block at d = 128.  A chunk of at most 128 / g tokens leaves the
    second query tile without rows over two to four key tiles; the prompt after it is
    longer than a tile and ends within its first key tile, whose rows behind the last
    key are put to zero.  Those tiles wait for different things; the neighbours' values
    are NaN and infinite."""
    rng = np.random.default_rng((31, g, causal))
    tok, h, n = 128 // g, 8, 200
    lq, lk = [], []
    for i in range(n):
        if i % 2 == 0:
            lq.append(int(rng.integers(1, tok + 1)))
            lk.append(int(rng.integers(129, 401)))
        else:
            m = int(rng.integers(tok + 1, 128)) if tok < 127 else int(rng.integers(129, 250))
            lq.append(m)
            lk.append(m)
    p, q, k, v, cq, ck = _case(128, g, h, lq, lk, "bf16", 32)
    c = _starts(lk)
    hurt = list(range(5, n, 20))
    for b in hurt:
        v[c[b]:c[b + 1]] = float("inf")
        v[c[b]] = float("nan")
    ref = None
    for _ in range(12):
        _flush()
        out, lse = _run(p, q, k, v, cq, ck, causal=causal)
        assert p.device_error() == 0
        if ref is None:
            _check(q, k, v, lq, lk, causal, out, lse, skip=hurt)
            ref = out, lse
        assert torch.equal(out.nan_to_num(9.0, 9.0, 9.0), ref[0].nan_to_num(9.0, 9.0, 9.0)) and torch.equal(lse, ref[1])


def _steps(d, g, dtype, rows, levels, seed):
    """Rows over key tiles of 128 whose scores (scale 1) are levels[j] in tile j: one
    element of q and k carries them."""
    rng = np.random.default_rng((33, d, g, seed))
    m = 128 * len(levels)
    q = np.zeros((rows, g, d))
    k = np.zeros((m, 1, d))
    q[..., 0] = 1
    k[..., 0] = np.repeat(levels, 128)[:, None]
    p = tq.TQPrompt(head_dim=d, num_kv_heads=1, num_q_heads=g, dtype=DT[dtype], max_batch=1, max_tokens=rows)
    return p, _gpu(q, DT[dtype]), _gpu(k, DT[dtype]), rng, _gpu(_starts([rows])), _gpu(_starts([m]))


@pytest.mark.parametrize("d,g,rows", [(128, 4, 20), (128, 1, 200), (256, 4, 20), (256, 8, 50)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_reference_moves_twice_in_one_tile(d, g, rows, dtype):
    """Tile 1 lies 12 (or 9) log2 units above tile 0: the reference follows in tile 2.
    That one lies so far above that it is done again, and the reference moves a second
    time.  Only tile 0 has values, so a lost factor shows whole."""
    levels = [0, 8.5, 8.5 + 17] if dtype == "bf16" else [0, 6.25, 6.25 + 11]
    p, q, k, rng, cq, ck = _steps(d, g, dtype, rows, levels, rows)
    v = np.zeros((k.shape[0], 1, d))
    v[:128] = rng.uniform(1, 2, (128, 1, d)) * 2.0 ** 14
    v = _gpu(v, DT[dtype])
    out, lse = _run(p, q, k, v, cq, ck, causal=False, scale=1.0)
    assert p.device_error() == 0
    _check(q, k, v, [rows], [k.shape[0]], False, out, lse, scale=1.0)


def _fill_shared_memory(d, x):
    """Query tiles on every SM whose rows are x in element 0: what a later block finds in
    rows of shared memory that it does not load."""
    n = 256 * 152 * 2
    p = tq.TQPrompt(head_dim=d, num_kv_heads=1, num_q_heads=1, max_batch=1, max_tokens=n)
    q = torch.zeros((n, 1, d), device="cuda", dtype=torch.bfloat16)
    q[..., 0] = x
    one = torch.zeros((1, 1, d), device="cuda", dtype=torch.bfloat16)
    p.attention(q, one, one, _gpu(_starts([n])), _gpu(_starts([1])), causal=False)


@pytest.mark.parametrize("d,g", [(128, 3), (128, 5), (128, 40), (256, 3), (256, 40)])
def test_rows_that_no_token_has_do_not_steer_others(d, g):
    """128 % g rows of a query tile are not loaded.  Every tile's scores lie about 10 log2
    units above the last one's: a reference moves one tile late in every row, unless
    another row of the warp asks for more."""
    levels = [7.0 * j for j in range(6)]
    rows = 128 // g
    p, q, k, rng, cq, ck = _steps(d, g, "bf16", rows, levels, 34)
    k[..., 1:] = _gpu(0.25 * rng.standard_normal((k.shape[0], 1, d - 1)), k.dtype)
    q[..., 1:] = _gpu(0.25 * rng.standard_normal((rows, g, d - 1)), q.dtype)
    v = _gpu(rng.standard_normal(k.shape), k.dtype)
    outs = []
    for x in (0.0, 5.0, -3.0, 20.0):
        _fill_shared_memory(d, x)
        outs.append(_run(p, q, k, v, cq, ck, causal=False, scale=1.0))
    _check(q, k, v, [rows], [k.shape[0]], False, *outs[0], scale=1.0)
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.parametrize("d,g", [(128, 4), (256, 2)])
def test_queries_of_the_next_sequence_do_not_steer_a_row(d, g):
    """The rows behind a sequence's last are the next one's queries."""
    levels = [7.0 * j for j in range(6)]
    rows, m = 70 // g, 768
    p, q, k, rng, _, _ = _steps(d, g, "bf16", rows + 40, levels, 35)
    k[..., 1:] = _gpu(0.25 * rng.standard_normal((m, 1, d - 1)), k.dtype)
    q[:rows, :, 1:] = _gpu(0.25 * rng.standard_normal((rows, g, d - 1)), q.dtype)
    k = torch.cat([k, k[:5]])
    v = _gpu(rng.standard_normal(k.shape), k.dtype)
    p = tq.TQPrompt(head_dim=d, num_kv_heads=1, num_q_heads=g, max_batch=2, max_tokens=rows + 40)
    cq, ck = _gpu(_starts([rows, 40])), _gpu(_starts([m, 5]))
    outs = []
    for x in (0.0, 5.0, 20.0):
        q[rows:, :, 0] = x
        outs.append(_run(p, q, k, v, cq, ck, causal=False, scale=1.0))
    _check(q, k, v, [rows, 40], [m, 5], False, *outs[-1], scale=1.0)
    for out, lse in outs[1:]:
        assert torch.equal(out[:rows], outs[0][0][:rows]) and torch.equal(lse[:rows], outs[0][1][:rows])


@pytest.mark.parametrize("d,g", [(128, 4), (256, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scores_far_from_zero(d, g, dtype):
    """Scores 2^20 .. 2^21 plus a few halves, all exact in fp32: the softmax is that of
    the few halves.  Four tiles of small ones, then one key that weighs as much as they
    do together, so that what the references leave behind counts."""
    rows, m = 60, 768
    rng = np.random.default_rng((36, d))
    big = 2.0 ** 10 * (1 + rng.integers(0, 128, (rows, g)) / 128)
    x = 0.5 * rng.integers(-2, 3, m)
    x[530], x[700] = 6.5, 8.0
    q, k = np.zeros((rows, g, d)), np.zeros((m, 1, d))
    q[..., 1] = 1
    k[:, 0, 1] = x
    p = tq.TQPrompt(head_dim=d, num_kv_heads=1, num_q_heads=g, dtype=DT[dtype], max_batch=1, max_tokens=rows)
    v = _gpu(rng.standard_normal(k.shape), DT[dtype])
    near = _gpu(q, DT[dtype]), _gpu(k, DT[dtype])
    q[..., 0] = big
    k[..., 0] = 2.0 ** 10
    for sign in (1, -1):
        out, lse = _run(p, _gpu(sign * q, DT[dtype]), _gpu(sign * k if sign > 0 else np.where(np.arange(d) == 1, -k, k),
                                                         DT[dtype]), v, _gpu(_starts([rows])), _gpu(_starts([m])),
                        causal=False, scale=1.0)
        assert p.device_error() == 0
        _check(*near, v, [rows], [m], False, out, None, scale=1.0)
        # lse: the large part and ln of a sum, one rounding of the size of the large part each
        z = sign * big * 2.0 ** 10 + np.log(np.exp(x).sum())
        assert (np.abs(lse.double().cpu().numpy() - z) <= 3 * 2.0 ** -23 * 2 ** 21).all()
    # the first 300 keys far below: the references cross zero, then follow the few halves
    k[:300, 0, 0] *= -1
    out, _ = _run(p, _gpu(q, DT[dtype]), _gpu(k, DT[dtype]), v, _gpu(_starts([rows])), _gpu(_starts([m])), causal=False,
                  scale=1.0)
    _check(near[0], near[1][300:], v[300:], [rows], [m - 300], False, out, None, scale=1.0)


@pytest.mark.parametrize("d,g,lq,causal", [(128, 4, 60, False), (256, 2, 60, False), (128, 1, 300, True), (256, 1, 300, True)])
@pytest.mark.parametrize("dtype,size", [("bf16", 2.0 ** 17), ("bf16", 2.0 ** 40), ("f16", 2.0 ** 13), ("f16", 2.0 ** 15)])
def test_one_score_above_all_others(d, g, lq, causal, dtype, size):
    """Scores of about size^2 (not a power of two), 0 and their negative: a row's output is
    the mean of the values of its largest; a row that sees one key gets its value."""
    rng = np.random.default_rng((37, d, lq))
    m = 600 if not causal else lq
    kind = rng.choice([-1.0, -1.0, 0.0, 1.0], m)
    kind[:256] = np.minimum(kind[:256], 0)
    kind[:3] = -1
    q, k = np.zeros((lq, g, d)), np.zeros((m, 1, d))
    q[..., 3] = size * 141 / 128
    k[:, 0, 3] = kind * size * 159 / 128
    v = _gpu(rng.standard_normal(k.shape), DT[dtype])
    p = tq.TQPrompt(head_dim=d, num_kv_heads=1, num_q_heads=g, dtype=DT[dtype], max_batch=1, max_tokens=lq)
    out, lse = _run(p, _gpu(q, DT[dtype]), _gpu(k, DT[dtype]), v, _gpu(_starts([lq])), _gpu(_starts([m])), causal=causal,
                    scale=1.0)
    assert p.device_error() == 0
    # the same order with steps of 60: e^-60 is nothing beside the largest
    q[..., 3], k[:, 0, 3] = 1, kind * 60
    _check(_gpu(q, DT[dtype]), _gpu(k, DT[dtype]), v, [lq], [m], causal, out, None, scale=1.0)
    top = np.array([kind[:i + 1].max() for i in range(lq)]) if causal else np.full(lq, kind.max())
    z = top[:, None] * size * size * (141 / 128) * (159 / 128)
    assert (np.abs(lse.double().cpu().numpy() - z) <= 2.0 ** -22 * np.abs(z) + 8).all()


@pytest.mark.parametrize("d,g", [(128, 4), (256, 8)])
@pytest.mark.parametrize("dtype,size", [("bf16", 2.0 ** 30), ("f16", 2.0 ** 14)])
def test_large_scores_in_key_parts(d, g, dtype, size):
    """Few rows over many keys: parts with scores of size^2, of its negative and of small
    size, a few warps of them in the loop for large ones; captured and replayed."""
    rng = np.random.default_rng((38, d))
    lq, m = 20, 4500
    kind = np.full(m, -1.0)
    kind[1000:2500] = rng.choice([0.0, 1e-9], 1500)
    kind[3000:] = rng.choice([-1.0, 0.0], m - 3000)
    at = rng.choice(m, 3, replace=False)
    kind[at] = 1
    q, k = np.zeros((lq, g, d)), np.zeros((m, 1, d))
    q[..., 3] = size * 141 / 128
    q[10:] *= -1
    k[:, 0, 3] = kind * size * 159 / 128
    v = _gpu(rng.standard_normal(k.shape), DT[dtype])
    p = tq.TQPrompt(head_dim=d, num_kv_heads=1, num_q_heads=g, dtype=DT[dtype], max_batch=1, max_tokens=lq)
    args = _gpu(q, DT[dtype]), _gpu(k, DT[dtype]), v, _gpu(_starts([lq])), _gpu(_starts([m]))
    out, lse = _run(p, *args, causal=False, scale=1.0)
    assert p.device_error() == 0
    # the largest: kind 1, and for the negated queries kind -1
    top = np.where(np.arange(lq)[:, None] < 10, kind == 1, kind == -1)
    for i in (0, 10):
        near = np.zeros((10, g, d)), np.zeros((m, 1, d))
        near[0][..., 0] = 1
        near[1][:, 0, 0] = np.where(top[i], 0, -60)
        _check(_gpu(near[0], DT[dtype]), _gpu(near[1], DT[dtype]), v, [10], [m], False, out[i:i + 10], None, scale=1.0)
    graph = torch.cuda.CUDAGraph()
    again = torch.zeros_like(out)
    with torch.cuda.graph(graph):
        p.attention(*args, out=again, causal=False, scale=1.0)
    for _ in range(2):
        again.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, out)
