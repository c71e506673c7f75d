"""CPU checks of the 8-bit cache: the oracle's format against torch's e4m3, the
sizes, and every refusal that the host makes before anything reaches CUDA."""

import os

import numpy as np
import pytest

import turboquant_bit_kv_tq_gb300 as tq
from oracle import f8

torch = pytest.importorskip("torch")

CFG = dict(head_dim=128, num_kv_heads=8, num_q_heads=32, num_blocks=10, max_batch=4, max_blocks_per_seq=4)


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(tq.library_path()):
        from turboquant_bit_kv_tq_gb300 import _build

        _build.build()
    tq.load_library()


def test_oracle_codes_match_torch():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000), f8.VALUES[:127],
                        (f8.VALUES[:126] + f8.VALUES[1:127]) / 2, 2.0 ** rng.uniform(-14, 8, 5000),
                        [0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(f8.e4m3_codes(x), want)
    assert np.array_equal(f8.VALUES[:127], torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("top,byte", [(448.0, 127), (449.0, 128), (447.0, 127), (224.0, 126), (224.5, 127), (1.75, 119),
                                      (0.0, 1), (2.0 ** -149, 1), (3.4028234e38, 247)])
def test_oracle_scale_is_the_smallest_that_fits(top, byte):
    x = np.zeros((1, 128))
    x[0, 5] = -top
    codes, e = f8.quantise(x)
    assert e[0] == byte
    assert top > 448 * 2.0 ** (byte - 128) or byte == 1
    assert abs(f8.VALUES[codes[0, 5]]) <= 448


def test_oracle_marks_vectors_that_are_not_finite():
    x = np.ones((3, 128))
    x[0, 3], x[1, 100] = np.inf, np.nan
    codes, e = f8.quantise(x)
    assert list(e[:2]) == [255, 255] and not codes[:2].any()
    assert np.isnan(f8.values(codes, e)[:2]).all() and np.array_equal(f8.values(codes, e)[2], x[2])


@pytest.mark.parametrize("d", [128, 256])
def test_sizes(d):
    s = tq.tq_f8_cache_sizes(tq.tq_f8_config(**{**CFG, "head_dim": d}))
    assert s["page_bytes"] == 32 * d + 32 and s["page_bytes"] % 16 == 0
    assert s["cache_bytes"] == 10 * 8 * s["page_bytes"]
    assert s["workspace_bytes"] > 0


def test_bad_configs_are_refused():
    for bad, status in [(dict(head_dim=64), -2), (dict(block_size=32), -2), (dict(num_q_heads=30), -1),
                        (dict(num_q_heads=4), -1), (dict(num_kv_heads=0), -1), (dict(num_blocks=0), -1),
                        (dict(num_blocks=1 << 31), -1), (dict(max_batch=0), -1), (dict(max_blocks_per_seq=0), -1),
                        (dict(max_blocks_per_seq=1 << 28), -1), (dict(max_batch=1 << 27), -1)]:
        with pytest.raises(tq.TQError) as e:
            tq.tq_f8_cache_sizes(tq.tq_f8_config(**{**CFG, **bad}))
        assert e.value.status == status, bad


def test_null_arguments_are_refused():
    lib = tq.load_library()
    assert lib.tq_f8_store(None, None, None, 1, 1024, 1024, 4, None, None, None) == -1
    assert lib.tq_f8_load(None, None, None, None, None, 1, 4, None, None, 1, None) == -1
    assert lib.tq_f8_decode_attention(None, None, 1, 4096, None, None, None, 0.0, 1, None, 1, None) == -1
    assert lib.tq_f8_get_device_error(None, None, None) == -1
    assert lib.tq_f8_cache_destroy(None) == 0


def test_binding_checks_before_any_call():
    cfg = tq.tq_f8_config(**CFG)
    k = torch.zeros((3, 8, 128), dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):  # shapes differ
        tq.tq_f8_store(None, cfg, k, k[:2], slots, None)
    with pytest.raises(ValueError):  # dtypes differ
        tq.tq_f8_store(None, cfg, k, k.float(), slots, None)
    with pytest.raises(ValueError):  # CPU tensors never reach the library
        tq.tq_f8_store(None, cfg, k, k, slots, None)
    q = torch.zeros((3, 32, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tq.tq_f8_decode_attention(None, cfg, q, None, torch.zeros((3, 4), dtype=torch.int32),
                                  torch.zeros(3, dtype=torch.int32), q)
    with pytest.raises(ValueError):
        tq.tq_f8_load(None, cfg, None, torch.zeros((3, 4), dtype=torch.int32), torch.zeros(3, dtype=torch.int32),
                      torch.zeros(3, dtype=torch.int32), k, k[:2])
