"""CPU checks of the 4-bit cache: the oracle's format by brute force, the sizes,
and every refusal that the host makes before anything reaches CUDA."""

import os

import numpy as np
import pytest

import turboquant_bit_kv_tq_gb300 as tq
from oracle import i4

torch = pytest.importorskip("torch")

CFG = dict(head_dim=128, num_kv_heads=8, num_q_heads=32, num_blocks=10, max_batch=4, max_blocks_per_seq=4)


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(tq.library_path()):
        from turboquant_bit_kv_tq_gb300 import _build

        _build.build()
    tq.load_library()


def test_scale_bytes_are_fp16_numbers_cut_off():
    want = (np.arange(160, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(i4.SCALES[:160], want) and i4.SCALES[160] == 32


@pytest.mark.parametrize("top,byte", [(240.0, 127), (240.5, 128), (239.0, 127), (120.0, 126), (120.25, 127),
                                      (0.0, 1), (2.0 ** -149, 1), (3.4028234e38, 248), (2.0 ** 127, 247)])
def test_oracle_exponent_is_the_smallest_that_fits(top, byte):
    x = np.zeros((1, 128))
    x[0, 5] = -top
    codes, u, e = i4.quantise(x)
    assert e[0] == byte
    assert abs(i4.values(codes, u, e)[0, 5] + top) <= top / 14 + 2.0 ** -143


def test_oracle_scale_is_the_finest_that_keeps_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((400, 128)) * np.exp(rng.uniform(-12, 12, (400, 1))) * np.exp(rng.uniform(-3, 3, (400, 128)))
    codes, u, e = i4.quantise(x)
    y = (x * np.exp2(127.0 - e)[:, None]).reshape(400, 8, 16)
    s = i4.SCALES[u][..., None]
    # no element further than half a step, and the next finer scale would leave one so
    assert (np.abs(y - (codes.reshape(y.shape) - 8.0) * s) <= s / 2).all()
    g = np.abs(y).max(-1)
    assert (g[u > 1] > 7.5 * i4.SCALES[u[u > 1].astype(int) - 1]).all() and (u <= 160).all()
    assert codes.min() >= 1 and codes.max() <= 15


def test_oracle_marks_vectors_that_are_not_finite():
    x = np.ones((3, 128))
    x[0, 3], x[1, 100] = np.inf, np.nan
    codes, u, e = i4.quantise(x)
    assert list(e[:2]) == [255, 255] and (codes[:2] == 8).all() and not u[:2].any()
    back = i4.values(codes, u, e)
    assert np.isnan(back[:2]).all() and np.abs(back[2] - 1).max() <= 1 / 14


@pytest.mark.parametrize("d", [128, 256])
def test_sizes(d):
    s = tq.tq_i4_cache_sizes(tq.tq_i4_config(**{**CFG, "head_dim": d}))
    assert s["page_bytes"] == 18 * d + 32 and s["page_bytes"] % 16 == 0
    assert s["cache_bytes"] == 10 * 8 * s["page_bytes"]
    assert s["workspace_bytes"] > 0


def test_bad_configs_are_refused():
    for bad, status in [(dict(head_dim=64), -2), (dict(block_size=32), -2), (dict(num_q_heads=30), -1),
                        (dict(num_q_heads=4), -1), (dict(num_kv_heads=0), -1), (dict(num_blocks=0), -1),
                        (dict(num_blocks=1 << 31), -1), (dict(max_batch=0), -1), (dict(max_blocks_per_seq=0), -1),
                        (dict(max_blocks_per_seq=1 << 28), -1), (dict(max_batch=1 << 27), -1)]:
        with pytest.raises(tq.TQError) as e:
            tq.tq_i4_cache_sizes(tq.tq_i4_config(**{**CFG, **bad}))
        assert e.value.status == status, bad


def test_null_arguments_are_refused():
    lib = tq.load_library()
    assert lib.tq_i4_cache_sizes(None, None, None, None) == -1
    assert lib.tq_i4_cache_create(None, None, None, None) == -1
    assert lib.tq_i4_store(None, None, None, 1, 1024, 1024, 4, None, None, None) == -1
    assert lib.tq_i4_load(None, None, None, None, None, 1, 4, None, None, 1, None) == -1
    assert lib.tq_i4_decode_attention(None, None, 1, 4096, None, None, None, 0.0, 1, None, 1, None) == -1
    assert lib.tq_i4_get_device_error(None, None, None) == -1
    assert lib.tq_i4_cache_destroy(None) == 0


def test_binding_checks_before_any_call():
    cfg = tq.tq_i4_config(**CFG)
    k = torch.zeros((3, 8, 128), dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    i32 = dict(dtype=torch.int32)
    for call in [
        lambda: tq.tq_i4_store(None, cfg, k, k[:2], slots, None),
        lambda: tq.tq_i4_store(None, cfg, k, k.float(), slots, None),
        lambda: tq.tq_i4_store(None, cfg, k, k, slots, None),  # CPU tensors never reach the library
        lambda: tq.tq_i4_decode_attention(None, cfg, torch.zeros((3, 32, 128)), None, torch.zeros((3, 4), **i32),
                                          torch.zeros(3, **i32), torch.zeros((3, 32, 128))),
        lambda: tq.tq_i4_load(None, cfg, None, torch.zeros((3, 4), **i32), torch.zeros(3, **i32),
                              torch.zeros(3, **i32), k, k[:2]),
    ]:
        with pytest.raises(ValueError):
            call()
