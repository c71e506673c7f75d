"""The examples of README.md, run as they stand."""

import os

import numpy as np
import pytest

from oracle import serve

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def _example(first):
    """The python block that begins with `first`."""
    blocks = [b.split("```")[0] for b in open(README).read().split("```python\n")[1:]]
    return [b for b in blocks if b.startswith(first)][0]


def test_decode_step_from_lengths_alone():
    import turboquant_bit_kv_tq_gb300 as tq

    rng = np.random.default_rng(98)
    batch = 3
    lens = np.array([16, 0, 37], np.int32)
    free = rng.permutation(60).astype(np.int32)
    table = np.full((batch, 512), -1, np.int32)
    table[0, :1], table[2, :3] = free[50], free[51:54]
    gpu = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    qkv = torch.randn((batch, 48, 128), device="cuda").to(torch.bfloat16)
    q, k, v = qkv.split([32, 8, 8], 1)
    ones = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    # memory that a careless example would read: neither these lengths nor this list entry
    for n in (batch, batch + 1, 1):
        waste = [torch.full((n,), 9, dtype=torch.int32, device="cuda") for _ in range(64)]
    del waste
    names = dict(tq=tq, torch=torch, batch=batch, lens=gpu(lens), first_free=gpu(np.array([2], np.int32)),
                 block_table=gpu(table), free_blocks=gpu(free), q=q, k=k, v=v, q_weight=ones, k_weight=ones)
    exec(_example("cache = tq.TQI4Cache"), names)
    want = serve.plan(lens, [1] * batch, table, free, 2, batch)
    out = names["out"]
    got = (names["block_table"], out.slot_mapping, out.positions, out.kv_rows, out.seq_lens, out.cu_q, out.cu_k, out.next_free)
    for a, b in zip(got, want):
        assert np.array_equal(a.cpu().numpy(), np.atleast_1d(b))
    assert torch.isfinite(names["step"].float()).all() and names["plan"].device_error() == 0
