"""CPU checks of norm with rotation and of the step plan: the oracles against
plain computations, and the refusals that the host makes before anything
reaches CUDA."""

import os

import numpy as np
import pytest

import turboquant_bit_kv_tq_gb300 as tq
from oracle import serve

torch = pytest.importorskip("torch")

ROPE = dict(head_dim=128, num_kv_heads=2, num_q_heads=8)
PLAN = dict(max_batch=4, max_blocks_per_seq=6)


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(tq.library_path()):
        from turboquant_bit_kv_tq_gb300 import _build

        _build.build()
    tq.load_library()


def test_oracle_angles():
    assert abs(float(serve.TWO_PI) - 2 * np.pi) < 1e-15
    f = serve.powers(1e4, 64)
    near = serve.angles(np.arange(50), f)
    want = np.arange(50)[:, None] * f
    assert np.abs(np.sin(near) - np.sin(want)).max() < 1e-14
    # a frequency of an eighth of a turn and a half: positions far apart by whole turns agree
    g = [float(serve.TWO_PI) / 8]
    a = serve.angles([3, 3 + (1 << 20)], g)
    assert abs(a[0, 0] - a[1, 0]) < 1e-9 and abs(a[0, 0] - 3 * np.pi / 4) < 1e-14


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotation_depends_on_the_difference_of_positions(interleaved):
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 128))
    f = serve.powers(1e4, 96)
    dots = []
    for p in (0, 77, 100000):
        a, _ = serve.norm_rope(q, None, [p + 13], f, 0.0, interleaved)
        b, _ = serve.norm_rope(k, None, [p], f, 0.0, interleaved)
        dots.append((a * b).sum())
    assert np.ptp(dots) < 1e-10


def test_oracle_plan_by_hand():
    table = np.array([[7, -1, -1], [3, 4, -1], [-1, -1, -1]])
    t, s, p, r, n, cq, ck, at = serve.plan([16, 20, 0], [1, 13, 0], table, [9, 8, 5, 6], 1, 15)
    assert np.array_equal(t, [[7, 8, -1], [3, 4, 5], [-1, -1, -1]]) and at == 3
    assert list(s) == [128] + [64 + i for i in range(4, 16)] + [80, -1]
    assert list(p) == [16] + list(range(20, 33)) + [0] and list(r) == [16] + [17 + x for x in range(20, 33)] + [-1]
    assert list(n) == [17, 33, 0] and list(cq) == [0, 1, 14, 14] and list(ck) == [0, 17, 50, 50]


def test_bad_configs_are_refused():
    for bad, status in [(dict(head_dim=64), -2), (dict(rot_dim=24), -2), (dict(rot_dim=144), -1), (dict(rot_dim=-16), -1),
                        (dict(num_q_heads=0), -1), (dict(num_kv_heads=0), -1), (dict(eps=-1.0), -1),
                        (dict(eps=float("nan")), -1), (dict(base=0.0), -1), (dict(base=float("inf")), -1),
                        (dict(interleaved=2), -1), (dict(norm=-1), -1)]:
        with pytest.raises(tq.TQError) as e:
            tq.tq_norm_rope_sizes(tq.tq_norm_rope_config(**{**ROPE, **bad}))
        assert e.value.status == status, bad
    for bad, status in [(dict(max_batch=0), -1), (dict(max_blocks_per_seq=0), -1), (dict(max_batch=8193), -2),
                        (dict(max_batch=8192, max_blocks_per_seq=16384), -1)]:
        with pytest.raises(tq.TQError) as e:
            tq.tq_plan_sizes(tq.tq_plan_config(**{**PLAN, **bad}))
        assert e.value.status == status, bad
    assert tq.tq_plan_sizes(tq.tq_plan_config(max_batch=8192, max_blocks_per_seq=16383))["workspace_bytes"] > 0
    assert tq.tq_norm_rope_sizes(tq.tq_norm_rope_config(**ROPE, rot_dim=0))["workspace_bytes"] > 0


def test_null_arguments_are_refused():
    lib = tq.load_library()
    assert lib.tq_norm_rope_sizes(None, None) == -1 and lib.tq_plan_sizes(None, None) == -1
    assert lib.tq_norm_rope_create(None, None, None, None, None) == -1
    assert lib.tq_plan_create(None, None, None, None) == -1
    assert lib.tq_norm_rope(None, None, None, None, 1, 0, 0, 0, None, None, 0, None, None, 1, 1, None, None, None, 0, 0,
                            0, None) == -1
    assert lib.tq_plan_step(None, None, None, 1, None, 0, None, None, 1, None, None, None, None, None, None, None,
                            None) == -1
    assert lib.tq_norm_rope_get_device_error(None, None, None) == -1
    assert lib.tq_plan_get_device_error(None, None, None) == -1
    assert lib.tq_norm_rope_destroy(None) == 0 and lib.tq_plan_destroy(None) == 0


def test_bindings_check_before_any_call():
    cfg = tq.tq_norm_rope_config(**ROPE)
    q, k = torch.zeros((3, 8, 128)), torch.zeros((3, 2, 128))
    pos = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):  # CPU tensors never reach the library
        tq.tq_norm_rope(None, cfg, q, k, pos, q, k)
    with pytest.raises(TypeError):
        tq.tq_norm_rope(None, cfg, q, k.half(), pos, q, k)
    with pytest.raises(ValueError):
        tq.tq_norm_rope_create(cfg, None, inv_freq=np.ones(63))
    t = torch.zeros((2, 6), dtype=torch.int32)
    n, one = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        tq.tq_plan_step(None, tq.tq_plan_config(**PLAN), n, None, t, one, one, torch.zeros(2, dtype=torch.int64), n, n, n,
                        pos, pos, one)


def test_oracle_plan_of_which_only_a_part_fits():
    """Packed keys keep rows for tokens that got no slot: the last key stays that of the last token."""
    table = np.array([[7, -1, -1], [3, -1, -1]])
    t, s, p, r, n, cq, ck, at = serve.plan([14, 2], [9, 3], table, [], 0, 12)
    assert np.array_equal(t, table) and at == 0
    assert list(s) == [126, 127] + [-1] * 7 + [50, 51, 52] and list(p) == list(range(14, 23)) + [2, 3, 4]
    assert list(r) == [14, 15] + [-1] * 7 + [25, 26, 27]
    assert list(n) == [16, 5] and list(cq) == [0, 9, 12] and list(ck) == [0, 23, 28]
