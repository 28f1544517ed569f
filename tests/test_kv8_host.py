"""CPU-side checks of the 8-bit cache: descriptions and arguments refused before any device work, and the
reference's own rounding against torch's conversion."""
import ctypes

import numpy as np
import pytest

from tests import kv8_ref


@pytest.fixture(scope="module")
def ff():
    from kv_cache_attention_ff_gb300 import build, ff as ffmod
    build.build()
    return ffmod


def _desc(ff, **kw):
    d = ff.KV8Desc()
    assert ff.lib().ff_kv8_desc_default(ctypes.byref(d)) == 0
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_defaults(ff):
    d = _desc(ff)
    assert (d.n_layers, d.batch, d.capacity, d.heads, d.kv_heads, d.head_dim, d.max_tokens) == \
        (1, 1, 31200, 12, 12, 128, 4680)
    assert ff.lib().ff_kv8_desc_default(None) == 1


@pytest.mark.parametrize("bad", [
    dict(head_dim=96), dict(heads=0), dict(kv_heads=0), dict(heads=12, kv_heads=5), dict(kv_heads=24),
    dict(capacity=0), dict(capacity=(1 << 30) + 1), dict(batch=0), dict(batch=65536), dict(n_layers=0),
    dict(max_tokens=0), dict(device=-1), dict(kv_heads=32768, heads=32768), dict(max_tokens=1 << 30),
])
def test_bad_descriptions_are_refused(ff, bad):
    d = _desc(ff, **bad)
    h = ctypes.c_void_p()
    assert ff.lib().ff_kv8_create(ctypes.byref(d), ctypes.byref(h)) == 1
    assert not h.value


def test_create_needs_an_out_pointer_and_a_description(ff):
    h = ctypes.c_void_p()
    assert ff.lib().ff_kv8_create(None, ctypes.byref(h)) == 1
    assert ff.lib().ff_kv8_create(ctypes.byref(_desc(ff)), None) == 1


def test_create_without_gpu_fails_cleanly(ff):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    h = ctypes.c_void_p()
    assert ff.lib().ff_kv8_create(ctypes.byref(_desc(ff)), ctypes.byref(h)) in (5, 7)
    assert not h.value
    with pytest.raises(ff.FFError):
        ff.KV8Cache(batch=1)
    with pytest.raises(TypeError):
        ff.KV8Cache(no_such_field=1)


def test_null_handles_are_refused(ff):
    lib, null, p = ff.lib(), ctypes.c_void_p(), ctypes.c_void_p(256)
    assert lib.ff_kv8_append(null, 0, 1, p, p, None, None, None) == 1
    assert lib.ff_kv8_load(null, 0, 1, None, p, p, None) == 1
    assert lib.ff_kv8_attn(null, 0, 1, p, None, 0, p, None, None, None, None) == 1
    assert lib.ff_kv8_evict(null, 0, null, 0, 1, 0, p, p, p, None) == 1
    assert lib.ff_kv8_layer_info(null, 0, None, None, None, None, None) == 1
    n = ctypes.c_size_t()
    assert lib.ff_kv8_bytes(null, ctypes.byref(n)) == 1
    assert lib.ff_kv8_error_poll(null) == 1
    assert lib.ff_kv8_destroy(null) == 0


def test_capacity_status_has_a_text(ff):
    assert b"capacity" in ff.lib().ff_status_string(8)
    assert ff.STATUS[8] == "FF_ERR_CAPACITY"


def test_reference_rounding_is_torchs():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(3)
    x = np.concatenate([rng.standard_normal(50000) * s for s in (1e-3, 0.02, 1.0, 100.0)]).astype(np.float32)
    x = np.concatenate([x, np.arange(-600, 600, dtype=np.float32) / 1024, np.float32([448, 447.9, -448, 0, -0.0])])
    got = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(kv8_ref.nearest8(x).astype(np.float32), got)


@pytest.mark.parametrize("top, e", [(448.0, 0), (449.0, 1), (1.0, -8), (0.875, -9), (0.876, -8), (0.0, -96), (2.0 ** -120, -96),
                                    (2.0 ** 127, 112)])
def test_reference_exponent(top, e):
    assert kv8_ref.exponent(np.array([0.0, -top])) == e
    if -96 < e < 112:
        assert top <= 448 * 2.0 ** e and top > 448 * 2.0 ** (e - 1)


@pytest.mark.parametrize("big", [
    dict(batch=65535, capacity=1 << 30, kv_heads=16384, heads=16384, max_tokens=1),  # 2^67 bytes of codes
    dict(batch=4096, capacity=1 << 30, kv_heads=1, heads=1, max_tokens=1),
])
def test_caches_beyond_any_memory_are_refused(ff, big):
    h = ctypes.c_void_p()
    assert ff.lib().ff_kv8_create(ctypes.byref(_desc(ff, **big)), ctypes.byref(h)) == 4
    assert not h.value
