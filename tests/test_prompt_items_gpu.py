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
