"""The plan of a step on the GPU against its oracle (oracle/serve.py), entry by
entry, and the plan in use: chunked prompts and a captured decode loop."""

import os
import subprocess
import sys

import numpy as np
import pytest

import turboquant_bit_kv_tq_gb300 as tq
from oracle import f8, i4, serve
from turboquant_bit_kv_tq_gb300 import workloads as wl

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ("slot_mapping", "positions", "kv_rows", "seq_lens", "cu_q", "cu_k", "next_free")


def _gpu(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype))).cuda()


def _run(lens, new, table, free, nxt, tokens, plan=None):
    """(device error, table after, outputs by name) of one call."""
    plan = plan or tq.TQPlan(max_batch=len(lens), max_blocks_per_seq=table.shape[1])
    out = plan.outputs(len(lens), tokens)
    for n in NAMES:
        getattr(out, n).fill_(-99)
    t = _gpu(table)
    plan.step(_gpu(lens), None if new is None else _gpu(new), t, _gpu(free), _gpu([nxt]), out)
    return plan.device_error(), t.cpu().numpy(), [getattr(out, n).cpu().numpy() for n in NAMES]


def _same(got, want):
    assert np.array_equal(got[1], want[0])
    for name, a, b in zip(NAMES, got[2], want[1:]):
        assert np.array_equal(a, np.atleast_1d(b)), name


def _case(seed, batch, longest, chunk, columns=None, spare=3, pad=0):
    rng = np.random.default_rng((91, seed))
    lens = rng.integers(0, longest + 1, batch)
    new = np.ones(batch, np.int64) if chunk == 0 else rng.integers(0, chunk + 1, batch)
    columns = columns or int(max(1, ((lens + new + 15) // 16).max()))
    have = (lens + 15) // 16
    taken = int(((lens + new + 15) // 16 - have).sum())
    perm = rng.permutation(int(have.sum()) + taken + spare + 2)
    table = np.full((batch, columns), -5)
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = perm[at:at + n]
        at += n
    return lens, new, table, perm[at:], 2, int(new.sum()) + pad


@pytest.mark.parametrize("batch,longest,chunk,pad", [(1, 0, 1, 0), (1, 15, 0, 0), (1, 16, 0, 3), (1, 100, 5000, 0),
                                                     (7, 40, 0, 5), (33, 300, 90, 0), (256, 1000, 0, 0), (257, 50, 33, 9),
                                                     (1000, 2000, 0, 24), (64, 8000, 2048, 100), (1500, 64, 40, 1),
                                                     (8192, 100, 3, 0), (3, 5, 0, 4000)])
def test_plan(batch, longest, chunk, pad):
    for seed in range(3):
        lens, new, table, free, nxt, tokens = _case(seed + batch, batch, longest, chunk, pad=pad)
        got = _run(lens, None if chunk == 0 else new, table, free, nxt, tokens)
        assert got[0] == 0
        _same(got, serve.plan(lens, new, table, free, nxt, tokens))


def test_nothing_new_and_no_rows():
    lens, table = [17, 0], np.array([[4, 5], [-1, -1]])
    got = _run(lens, [0, 0], table, [1], 0, 0)
    assert got[0] == 0
    _same(got, serve.plan(lens, [0, 0], table, [1], 0, 0))
    got = _run(lens, [0, 0], table, np.zeros(0), 0, 4)
    assert got[0] == 0
    _same(got, serve.plan(lens, [0, 0], table, [], 0, 4))


def test_what_does_not_fit_is_left_out():
    table = np.full((4, 4), -1)
    table[0, :2], table[1, :1], table[2, :4] = [8, 9], [7], [1, 2, 3, 4]
    lens = [30, 16, 60, 0]
    for new, free, nxt, tokens, error in [
        ([1, 1, 9, 3], [11, 12, 13], 0, 20, tq.TQ_DEVERR_SEQLEN),       # request 2 outgrows its row of the table
        ([5, 40, 2, 50], [11, 12, 13], 0, 120, tq.TQ_DEVERR_POOL),      # the list runs out inside request 1
        ([5, 3, 2, 50], [11, 12, 13], 3, 120, tq.TQ_DEVERR_POOL),       # it is empty
        ([5, 3, 2, 50], [11, 12, 13], 9, 120, tq.TQ_DEVERR_POOL),       # an entry behind its end
        ([5, 3, 2, 50], [11, 12, 13, 14, 15, 16], -2, 120, tq.TQ_DEVERR_POOL),
        ([5, 20, 2, 50], list(range(20, 40)), 1, 12, tq.TQ_DEVERR_CHUNK),  # fewer rows than tokens
        ([2 ** 31 - 1] * 4, list(range(20, 40)), 1, 30, tq.TQ_DEVERR_CHUNK),
        ([-3, 2, -(2 ** 31), 1], list(range(20, 40)), 1, 30, tq.TQ_DEVERR_SEQLEN),
    ]:
        got = _run(lens, new, table, free, nxt, tokens)
        _same(got, serve.plan(lens, new, table, free, nxt, tokens))
        assert got[0] & error and not got[0] & ~(error | tq.TQ_DEVERR_SEQLEN), (new, got[0])
    for bad in ([-1, 16, 60, 0], [30, 16, 65, 2 ** 31 - 1]):
        got = _run(bad, [1, 2, 3, 4], table, list(range(20, 40)), 0, 12)
        _same(got, serve.plan(bad, [1, 2, 3, 4], table, list(range(20, 40)), 0, 12))
        assert got[0] & tq.TQ_DEVERR_SEQLEN
    # ids are passed on; a negative one gives its tokens no slot
    got = _run([0, 3], [20, 2], np.array([[-1, -1], [-7, -1]]), [6, -4], 0, 22)
    _same(got, serve.plan([0, 3], [20, 2], np.array([[-1, -1], [-7, -1]]), [6, -4], 0, 22))


def test_many_refusals_at_random():
    """Short lists, tables and rows, all at once."""
    rng = np.random.default_rng(92)
    for i in range(40):
        batch = int(rng.integers(1, 600))
        lens, new, table, free, nxt, tokens = _case(100 + i, batch, 60, int(rng.integers(1, 50)))
        table = table[:, :max(1, table.shape[1] - int(rng.integers(0, 3)))].copy()
        free = free[:int(rng.integers(0, len(free) + 1))]
        tokens = max(0, tokens - int(rng.integers(0, 30)))
        got = _run(lens, new, table, free, nxt, tokens)
        _same(got, serve.plan(lens, new, table, free, nxt, tokens))


@pytest.mark.parametrize("batch,tokens", [(5, 5), (300, 300), (2000, 4000)])
def test_lengths_and_list_in_place_through_a_graph(batch, tokens):
    """A captured step that reads its own last lengths and list entry, replayed: as many steps as replays."""
    lens, new, table, free, nxt, _ = _case(7, batch, 100, 0, columns=12, spare=4 * batch)
    plan = tq.TQPlan(max_batch=batch, max_blocks_per_seq=12)
    out = plan.outputs(batch, tokens)
    t, fr = _gpu(table), _gpu(free)
    out.seq_lens.copy_(_gpu(lens))
    out.next_free.copy_(_gpu([nxt]))
    plan.step(out.seq_lens, None, t, fr, out.next_free, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.step(out.seq_lens, None, t, fr, out.next_free, out)
    for step in range(20):
        if step:
            graph.replay()
        want = serve.plan(lens, new, table, free, nxt, tokens)
        _same((0, t.cpu().numpy(), [getattr(out, n).cpu().numpy() for n in NAMES]), want)
        table, lens, nxt = want[0], want[4], want[7]
    assert plan.device_error() == 0


def test_given_stream():
    lens, new, table, free, nxt, tokens = _case(8, 40, 200, 30)
    plan = tq.TQPlan(max_batch=40, max_blocks_per_seq=table.shape[1])
    side = torch.cuda.Stream()
    args = (_gpu(lens), _gpu(new), _gpu(table), _gpu(free), _gpu([nxt]))
    torch.cuda.synchronize()
    out = plan.outputs(40, tokens, stream=side)
    assert plan.step(*args, out, stream=side) is out
    side.synchronize()
    _same((0, args[2].cpu().numpy(), [getattr(out, n).cpu().numpy() for n in NAMES]),
          serve.plan(lens, new, table, free, nxt, tokens))


def test_refusals():
    plan = tq.TQPlan(max_batch=2, max_blocks_per_seq=3)
    out = plan.outputs(2, 4)
    n, t, one = _gpu([1, 2]), _gpu(np.zeros((2, 3))), _gpu([0])
    free = _gpu([1, 2, 3])
    for error, call in [
        (ValueError, lambda: plan.step(n, n[:1], t, free, one, out)),
        (ValueError, lambda: plan.step(n, n, t[:, :2], free, one, out)),
        (ValueError, lambda: plan.step(n, n, t[:1], free, one, out)),
        (ValueError, lambda: plan.step(n, n, t, free, one[:0], out)),
        (ValueError, lambda: plan.step(n.cpu(), n, t, free, one, out)),
        (ValueError, lambda: plan.step(n, n, t.cpu(), free, one, out)),
        (TypeError, lambda: plan.step(n.long(), n, t, free, one, out)),
        (TypeError, lambda: plan.step(n, n, t, free.long(), one, out)),
        (ValueError, lambda: plan.step(_gpu([1, 2, 3]), None, _gpu(np.zeros((3, 3))), free, one, out)),
    ]:
        with pytest.raises(error):
            call()
    with pytest.raises(tq.TQError) as e:
        plan.step(_gpu([1, 2, 3]), None, _gpu(np.zeros((3, 3))), free, one, plan.outputs(3, 4))
    assert e.value.status == -1


# ------------------------------------------------------------- all together
@pytest.mark.parametrize("d,g,kind", [(128, 4, "i4"), (256, 2, "i4"), (128, 4, "f8")])
def test_serving_steps(d, g, kind):
    """Two prompts in chunks, then decode steps from a captured graph: plan, norm and rotation, stored prefix,
    prompt attention, store, decode.  Every step against the oracles on the same rows."""
    rng = np.random.default_rng((93, d, g))
    B, cap, h, steps = 3, 12, 2, 20
    hq, dt = g * h, torch.bfloat16
    blocks = B * cap
    rot, base = d // 2, 1e4
    oracle = i4 if kind == "i4" else f8
    make = tq.TQI4Cache if kind == "i4" else tq.TQF8Cache
    cache = make(head_dim=d, num_kv_heads=h, num_q_heads=hq, num_blocks=blocks, max_batch=B, max_blocks_per_seq=cap)
    cache.cache.fill_(0xFF)
    plan = tq.TQPlan(max_batch=B, max_blocks_per_seq=cap)
    rope = tq.TQNormRope(head_dim=d, num_q_heads=hq, num_kv_heads=h, rot_dim=rot, base=base)
    prompt = tq.TQPrompt(head_dim=d, num_kv_heads=h, num_q_heads=hq, max_batch=B, max_tokens=256)
    wq, wk = (_gpu(1 + 0.1 * rng.standard_normal(d), np.float32).to(dt) for _ in range(2))
    table = torch.zeros((B, cap), dtype=torch.int32, device="cuda")
    free = _gpu(rng.permutation(blocks))
    lens, nxt = _gpu(np.zeros(B)), _gpu([0])
    eps, f = float(np.float32(1e-6)), serve.powers(base, rot)

    def project(n):
        return _gpu(rng.standard_normal((n, hq + 2 * h, d)), np.float32).to(dt)

    def near(got, want, tol):
        assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()

    for chunk in ([64, 37, 0], [50, 0, 41], [0, 5, 3]):
        n = sum(chunk)
        out = plan.outputs(B, n + 7)  # a padded batch
        before = lens.cpu().numpy()
        plan.step(lens, _gpu(chunk), table, free, nxt, out)
        qkv = project(n + 7)
        q, k, v = qkv.split([hq, h, h], 1)
        ck = out.cu_k.cpu().numpy()
        kr = torch.full((int(ck[-1]), h, d), float("nan"), dtype=dt, device="cuda")
        vr = kr.clone()
        cache.load(table, lens, out.cu_k, kr, vr)
        qo, _, _ = rope.apply(q, k, out.positions, wq, wk, k_out=kr, v=v, v_out=vr, kv_rows=out.kv_rows)
        att = prompt.attention(qo, kr, vr, out.cu_q, out.cu_k)
        new_k = kr[out.kv_rows[:n].long()]
        cache.store(new_k, v[:n], out.slot_mapping[:n])
        lens, nxt = out.seq_lens, out.next_free
        assert not torch.isnan(kr).any()
        cq, pos = out.cu_q.cpu().numpy(), out.positions.cpu().numpy()
        want, size = serve.norm_rope(k[:n].double().cpu().numpy(), wk.double().cpu().numpy(), pos[:n], f, eps)
        # (bf16 has 8 significant bits: half a step is up to 2^-8 of the value)
        near(new_k, want, 2.0 ** -19.3 * size + 2.0 ** -8 * np.abs(want) + 1e-30)
        pages = cache.pages().cpu().numpy()
        for b in range(B):
            m, total = chunk[b], int(before[b]) + chunk[b]
            if m == 0:
                continue
            kb, vb = (x[ck[b]:ck[b + 1]].double().cpu().numpy() for x in (kr, vr))
            # the prefix is what the cache holds, the rest the chunk's own rows
            for x, y in zip((kb, vb), oracle.rows(pages, table[b].cpu().numpy(), total, d)):
                assert np.array_equal(x[:int(before[b])], y[:int(before[b])])
                assert np.array_equal(oracle.values(*oracle.quantise(x[int(before[b]):])), y[int(before[b]):])
            rows = qo[cq[b]:cq[b + 1]].double().cpu().numpy()
            ref, _, mag = f8.attention(rows, kb, vb, 1 / np.sqrt(d), np.arange(m) + int(before[b]) + 1)
            near(att[cq[b]:cq[b + 1]], ref, 2.0 ** -7 * mag + 2.0 ** -8 * np.abs(ref))

    # decode steps: one captured step, replayed; lengths and list entry go round in place
    out = plan.outputs(B, B)
    out.seq_lens.copy_(lens)
    out.next_free.copy_(nxt)
    qkv = torch.zeros((B, hq + 2 * h, d), dtype=dt, device="cuda")
    q, k, v = qkv.split([hq, h, h], 1)
    att = torch.zeros((B, hq, d), dtype=dt, device="cuda")
    saved = [x.clone() for x in (out.seq_lens, out.next_free, table)]

    def step():
        plan.step(out.seq_lens, None, table, free, out.next_free, out)
        rope.apply(q, k, out.positions, wq, wk, q_out=q, k_out=k)
        cache.store(k, v, out.slot_mapping)
        cache.decode(q, table, out.seq_lens, out=att)

    qkv.copy_(project(B))
    step()
    for x, y in zip((out.seq_lens, out.next_free, table), saved):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    at = lens.cpu().numpy().copy()
    for _ in range(steps):
        qkv.copy_(project(B))
        graph.replay()
        torch.cuda.synchronize()
        at += 1
        assert np.array_equal(out.seq_lens.cpu().numpy(), at) and np.array_equal(out.positions.cpu().numpy(), at - 1)
        pages, tn = cache.pages().cpu().numpy(), table.cpu().numpy()
        for b in range(B):
            kb, vb = oracle.rows(pages, tn[b], int(at[b]), d)
            assert np.array_equal(kb[-1], oracle.values(*oracle.quantise(k[b].double().cpu().numpy())))
            ref, _, mag = f8.attention(q[b:b + 1].double().cpu().numpy(), kb, vb, 1 / np.sqrt(d))
            near(att[b], ref[0], 2.0 ** -10 * mag[0] + 2.0 ** -8 * np.abs(ref[0]))
    used = table.cpu().numpy()
    ids = np.concatenate([used[b, :(int(at[b]) + 15) // 16] for b in range(B)])
    assert len(set(ids)) == len(ids) == int(out.next_free.item())  # no block twice
    assert cache.device_error() == 0 and plan.device_error() == 0 and rope.device_error() == 0


@pytest.mark.parametrize("d,kind,columns,spare,cut,served", [
    (128, "i4", 20, 3, 0, (30, 22, 2, 5)),   # the list runs out inside request 1; 2 and 3 have room in their blocks
    (128, "f8", 20, 0, 0, (0, 6, 2, 5)),     # it is empty
    (256, "i4", 4, 99, 0, (30, 38, 14, 5)),  # requests 1 and 2 outgrow their rows of the table
    (128, "i4", 4, 4, 7, (30, 38, 14, 0)),   # they do, and fewer rows than tokens
])
def test_a_chunk_of_which_only_a_part_fits(d, kind, columns, spare, cut, served):
    """The tokens of a chunk that got a slot attend to what lies before them, whatever of it was left out; the rest
    comes with the next step."""
    rng = np.random.default_rng((94, d, columns, spare))
    h, hq, dt, blocks = 2, 8, torch.bfloat16, 64
    make, oracle = (tq.TQI4Cache, i4) if kind == "i4" else (tq.TQF8Cache, f8)
    cache = make(head_dim=d, num_kv_heads=h, num_q_heads=hq, num_blocks=blocks, max_batch=4, max_blocks_per_seq=20)
    rope = tq.TQNormRope(head_dim=d, num_q_heads=hq, num_kv_heads=h)
    prompt = tq.TQPrompt(head_dim=d, num_kv_heads=h, num_q_heads=hq, max_batch=4, max_tokens=256)
    lens, chunk = np.array([16, 26, 46 if columns > 4 else 50, 11]), np.array([30, 50, 20, 5])
    free, table = rng.permutation(blocks), np.full((4, 20), -1)
    at = 0
    for b, n in enumerate((lens + 15) // 16):
        table[b, :n] = free[at:at + n]
        at += n
    old = [rng.standard_normal((int(lens.sum()), h, d)) for _ in range(2)]
    slots = np.concatenate([table[b, np.arange(n) // 16] * 16 + np.arange(n) % 16 for b, n in enumerate(lens)])
    cache.store(*(_gpu(x, np.float32).to(dt) for x in old), _gpu(slots, np.int64))
    wide = _gpu(table)
    for step in range(2):
        # (the second step has all the room it needs)
        cols = columns if step == 0 else 20
        plan = tq.TQPlan(max_batch=4, max_blocks_per_seq=cols)
        n = int(chunk.sum()) - (cut if step == 0 else 0)
        out, t = plan.outputs(4, n), wide[:, :cols].contiguous()
        plan.step(_gpu(lens), _gpu(chunk), t, _gpu(free[at:at + spare] if step == 0 else free[at:]), _gpu([0]), out)
        wide[:, :cols] = t
        assert bool(plan.device_error()) == (step == 0)
        got = _gpu(served) if step == 0 else _gpu(chunk)
        assert torch.equal(out.seq_lens, _gpu(lens) + got)
        q, k, v = _gpu(rng.standard_normal((n, hq + 2 * h, d)), np.float32).to(dt).split([hq, h, h], 1)
        cq, ck = out.cu_q.cpu().numpy(), out.cu_k.cpu().numpy()
        kr = torch.full((int(ck[-1]), h, d), float("nan"), dtype=dt, device="cuda")
        vr = kr.clone()
        cache.load(wide, _gpu(lens), out.cu_k, kr, vr)
        qo, _, _ = rope.apply(q, k, out.positions, k_out=kr, v=v, v_out=vr, kv_rows=out.kv_rows)
        att = prompt.attention(qo, kr, vr, out.cu_q, out.cu_k)
        for b, m in enumerate(got.tolist()):
            if m == 0:
                continue
            kb, vb = (x[ck[b]:ck[b] + lens[b] + m].double().cpu().numpy() for x in (kr, vr))
            assert np.isfinite(kb).all() and np.isfinite(vb).all()
            rows = qo[cq[b]:cq[b] + m].double().cpu().numpy()
            ref, _, mag = f8.attention(rows, kb, vb, 1 / np.sqrt(d), np.arange(m) + int(lens[b]) + 1)
            # (weights and outputs rounded to bf16: half a step is 2^-8 at most of either)
            err = np.abs(att[cq[b]:cq[b] + m].double().cpu().numpy() - ref)
            assert (err <= 2.0 ** -7 * mag + 2.0 ** -8 * np.abs(ref)).all(), (step, b, err.max())
        fits = out.slot_mapping >= 0
        assert int(fits.sum()) == int(got.sum())
        cache.store(kr[out.kv_rows.clamp(min=0).long()], v, out.slot_mapping)
        pages, tn = cache.pages().cpu().numpy(), wide.cpu().numpy()
        for b, m in enumerate(got.tolist()):  # what the prompt saw is what is stored
            if m == 0:
                continue
            x = oracle.rows(pages, tn[b], int(lens[b]) + m, d)[0]
            new = kr[ck[b] + lens[b]:ck[b] + lens[b] + m].double().cpu().numpy()
            assert np.array_equal(x[lens[b]:], oracle.values(*oracle.quantise(new)))
        lens, chunk, at = out.seq_lens.cpu().numpy(), chunk - got.cpu().numpy(), at + int(out.next_free)
    assert rope.device_error() == 0 and cache.device_error() == 0 and prompt.device_error() == 0


def test_sums_of_lengths_beyond_an_int_are_cut_off():
    """Two requests that fill their rows of the widest table; rows and positions behind 2^31 - 1 do not wrap."""
    columns = 2 ** 26 - 1
    table = torch.zeros((2, columns), dtype=torch.int32, device="cuda")
    plan = tq.TQPlan(max_batch=2, max_blocks_per_seq=columns)
    out, full = plan.outputs(2, 80), 16 * columns
    plan.step(_gpu([full, full - 1]), _gpu([40, 40]), table, _gpu([]), _gpu([0]), out)
    assert plan.device_error() == tq.TQ_DEVERR_SEQLEN
    assert out.cu_q.tolist() == [0, 40, 80] and out.seq_lens.tolist() == [full, full]
    assert out.cu_k.tolist() == [0, full + 40, 2 ** 31 - 1]
    assert out.slot_mapping.tolist() == [-1] * 40 + [15] + [-1] * 39
    assert out.kv_rows.tolist() == [-1] * 40 + [2 ** 31 - 1] + [-1] * 39


def test_batches_around_the_launch_limit_of_shared_memory():
    """Sums of 2448 .. 2457 requests take up to 48 KB with what the kernel has beside them, and more with it; each size
    in a process that has asked for no larger one."""
    call = ("import numpy as np, torch, turboquant_bit_kv_tq_gb300 as tq\n"
            "b = {}\n"
            "plan = tq.TQPlan(max_batch=b, max_blocks_per_seq=2)\n"
            "out = plan.outputs(b, b)\n"
            "table = torch.arange(2 * b, dtype=torch.int32, device='cuda').view(b, 2)\n"
            "lens = torch.arange(b, dtype=torch.int32, device='cuda') % 16 + 1\n"
            "zero = torch.zeros(1, dtype=torch.int32, device='cuda')\n"
            "plan.step(lens, None, table, torch.arange(2 * b, dtype=torch.int32, device='cuda'), zero, out)\n"
            "n = int((lens == 16).sum())\n"
            "assert plan.device_error() == 0 and int(out.next_free) == n\n"
            "assert torch.equal(out.seq_lens, lens + 1) and torch.equal(out.positions, lens)\n"
            "assert out.cu_k[-1] == (lens + 1).sum() and out.cu_q[-1] == b\n")
    for b in (2436, 2447, 2448, 2457, 2458):
        done = subprocess.run([sys.executable, "-c", call.format(b)], cwd=ROOT, capture_output=True, text=True)
        assert done.returncode == 0, (b, done.stderr[-2000:])


def test_outputs_whose_memory_is_exchanged():
    """A step writes its outputs where they are now, and refuses what they no longer can be."""
    lens, new, table, free, nxt, tokens = _case(9, 30, 100, 20)
    plan = tq.TQPlan(max_batch=30, max_blocks_per_seq=table.shape[1])
    out = plan.outputs(30, tokens)
    args = (_gpu(lens), _gpu(new), _gpu(table), _gpu(free), _gpu([nxt]))
    want = serve.plan(lens, new, table, free, nxt, tokens)
    old = [getattr(out, n).data for n in NAMES]  # (the same memory, which stays allocated)
    for x, n in zip(old, NAMES):
        x.fill_(-99)
        getattr(out, n).data = torch.full((x.shape[0] + 3,), -98, dtype=x.dtype, device="cuda")[:x.shape[0]]
    plan.step(*args, out)
    assert plan.device_error() == 0 and all(bool((x == -99).all()) for x in old)
    _same((0, args[2].cpu().numpy(), [getattr(out, n).cpu().numpy() for n in NAMES]), want)
    for x, n in zip(old, NAMES):
        good, other = getattr(out, n).data, torch.float32 if x.dtype != torch.int64 else torch.int32
        for bad in [x[1:], x.cpu(), x.to(other)] + [torch.cat([x, x])[::2]] * (x.shape[0] > 1):
            getattr(out, n).data = bad
            with pytest.raises((ValueError, TypeError)):
                plan.step(*args, out)
        getattr(out, n).data = good
    plan.step(_gpu(lens), *args[1:], out)
    _same((0, args[2].cpu().numpy(), [getattr(out, n).cpu().numpy() for n in NAMES]), want)


def test_positions_beyond_an_int_are_cut_off():
    """Tokens behind the end of the widest row of a table, which get no slot."""
    columns = 2 ** 27 - 1
    table = torch.zeros((1, columns), dtype=torch.int32, device="cuda")
    plan = tq.TQPlan(max_batch=1, max_blocks_per_seq=columns)
    out, full = plan.outputs(1, 40), 16 * columns
    plan.step(_gpu([full - 8]), _gpu([40]), table, _gpu([]), _gpu([0]), out)
    assert plan.device_error() == tq.TQ_DEVERR_SEQLEN and out.seq_lens.tolist() == [full]
    assert out.positions.tolist() == [min(full - 8 + i, 2 ** 31 - 1) for i in range(40)]
    assert out.slot_mapping.tolist() == [8 + i for i in range(8)] + [-1] * 32
    assert out.kv_rows.tolist() == [full - 8 + i for i in range(8)] + [-1] * 32


def test_decode_steps_over_the_rotated_codebooks_pages():
    """Plan, norm with rotation, store and decode of TurboQuant's own pages, which take contiguous rows: norm with
    rotation's outputs, the values' among them, out of a fused projection.  A captured step, bit for bit the calls on
    plain copies of the same rows with the oracle's slots."""
    w = wl.scaled(wl.config("llama8b_gqa4_b16_8k"), q_heads=8, kv_heads=2, batch=3)
    rng = np.random.default_rng(95)
    B, cap, hq, h, d, dt = 3, 6, 8, 2, 128, torch.bfloat16
    caches = [tq.TQCache(**wl.cache_config_kwargs(w, num_blocks=20, max_blocks=cap, max_batch=B, split_blocks=2))
              for _ in range(2)]
    rope = tq.TQNormRope(head_dim=d, num_q_heads=hq, num_kv_heads=h)
    plan = tq.TQPlan(max_batch=B, max_blocks_per_seq=cap)
    out = plan.outputs(B, B + 2)  # a padded batch: the rows behind the last token are stored nowhere
    out.seq_lens.copy_(_gpu([0, 0, 0]))
    out.next_free.zero_()
    host, free = np.full((B, cap), -1), rng.permutation(20)
    table, list_ = _gpu(np.zeros((B, cap))), _gpu(free)
    qkv = torch.zeros((B + 2, hq + 2 * h, d), dtype=dt, device="cuda")
    q, k, v = qkv.split([hq, h, h], 1)
    to = [torch.zeros((B + 2, n, d), dtype=dt, device="cuda") for n in (hq, h, h)]
    att = torch.zeros((B, hq, d), device="cuda")

    def step():
        plan.step(out.seq_lens, None, table, list_, out.next_free, out)
        rope.apply(q, k, out.positions, q_out=to[0], k_out=to[1], v=v, v_out=to[2])
        caches[0].store(to[1], to[2], out.slot_mapping)
        caches[0].decode(to[0][:B], table, out.seq_lens, out=att)

    step()  # (loads and sets up; its tokens, zeros, are written over)
    out.seq_lens.zero_()
    out.next_free.zero_()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    lens, nxt = [0] * B, 0
    for _ in range(40):
        qkv.copy_(_gpu(rng.standard_normal(qkv.shape), np.float32))
        graph.replay()
        host, slots, pos, _, lens, _, _, nxt = serve.plan(lens, [1] * B, host, free, nxt, B + 2)
        qo, ko = rope.apply(q.contiguous(), k.contiguous(), _gpu(pos))
        caches[1].store(ko[:B].contiguous(), v[:B].contiguous(), _gpu(slots[:B], np.int64))
        want = caches[1].decode(qo[:B].contiguous(), _gpu(np.maximum(host, 0)), _gpu(lens))
        assert torch.equal(att, want) and bool(torch.isfinite(att).all())
    assert torch.equal(caches[0].cache, caches[1].cache)
    assert all(c.device_error() == 0 for c in caches) and plan.device_error() == 0 and rope.device_error() == 0
