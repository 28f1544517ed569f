"""CPU-side checks of the paged cache: descriptions and arguments refused before any device work, and the reference's own
plan."""
import ctypes
import random

import pytest

from tests.paged_ref import RefPaged


@pytest.fixture(scope="module")
def ff():
    from kv_cache_attention_ff_gb300 import build, ff as ffmod
    build.build()
    return ffmod


def _desc(ff, **kw):
    d = ff.PagedDesc()
    assert ff.lib().ff_paged_desc_default(ctypes.byref(d)) == 0
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_defaults(ff):
    d = _desc(ff)
    assert (d.n_layers, d.pages, d.page_rows, d.requests, d.capacity, d.heads, d.kv_heads, d.head_dim, d.max_rows) == \
        (1, 1950, 16, 1, 31200, 12, 12, 128, 4680)
    assert ff.lib().ff_paged_desc_default(None) == 1


@pytest.mark.parametrize("bad", [
    dict(head_dim=96), dict(heads=0), dict(kv_heads=0), dict(heads=12, kv_heads=5), dict(kv_heads=24), dict(pages=0),
    dict(capacity=0), dict(capacity=(1 << 30) + 1), dict(requests=0), dict(requests=8193), dict(n_layers=0),
    dict(max_rows=0), dict(device=-1), dict(page_rows=8), dict(page_rows=48), dict(page_rows=256), dict(page_rows=0),
    dict(max_rows=1 << 28),
])
def test_bad_descriptions_are_refused(ff, bad):
    h = ctypes.c_void_p()
    assert ff.lib().ff_paged_create(ctypes.byref(_desc(ff, **bad)), ctypes.byref(h)) == 1
    assert not h.value


@pytest.mark.parametrize("big", [
    dict(pages=1 << 30, page_rows=128),
    dict(pages=1 << 20, page_rows=128, heads=16, kv_heads=16),   # 2^31 rows of all heads
    dict(n_layers=1 << 20, pages=1 << 20),
    dict(requests=8192, capacity=1 << 30, page_rows=16, heads=1, kv_heads=1),  # 2^39 entries of tables
])
def test_caches_beyond_any_memory_are_refused(ff, big):
    h = ctypes.c_void_p()
    assert ff.lib().ff_paged_create(ctypes.byref(_desc(ff, **big)), ctypes.byref(h)) == 4
    assert not h.value


def test_create_needs_an_out_pointer_and_a_description(ff):
    h = ctypes.c_void_p()
    assert ff.lib().ff_paged_create(None, ctypes.byref(h)) == 1
    assert ff.lib().ff_paged_create(ctypes.byref(_desc(ff)), None) == 1


def test_create_without_gpu_fails_cleanly(ff):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    h = ctypes.c_void_p()
    assert ff.lib().ff_paged_create(ctypes.byref(_desc(ff)), ctypes.byref(h)) in (5, 7)
    assert not h.value
    with pytest.raises(ff.FFError):
        ff.PagedCache(pages=4)
    with pytest.raises(TypeError):
        ff.PagedCache(no_such_field=1)


def test_null_handles_are_refused(ff):
    lib, null, p = ff.lib(), ctypes.c_void_p(), ctypes.c_void_p(256)
    assert lib.ff_paged_plan(null, 1, None, p, None) == 1
    assert lib.ff_paged_store(null, 0, 1, p, p, None) == 1
    assert lib.ff_paged_attn(null, 0, 1, 1, p, p, None, None) == 1
    assert lib.ff_paged_info(null, None, None, None, None, None, None, None) == 1
    assert lib.ff_paged_layer_info(null, 0, None, None) == 1
    n = ctypes.c_size_t()
    assert lib.ff_paged_bytes(null, ctypes.byref(n)) == 1
    assert lib.ff_paged_error_poll(null) == 1
    assert lib.ff_paged_destroy(null) == 0


@pytest.mark.parametrize("seed", range(8))
def test_the_references_pages_are_each_one_requests(seed):
    """Whatever steps come, a page is on the stack or in one table, and what a step added comes off as it went on."""
    rng = random.Random(seed)
    ref = RefPaged(rng.choice([5, 40, 300]), rng.choice([16, 32, 64, 128]), rng.choice([1, 3, 17]), rng.choice([50, 700, 5000]))
    for _ in range(60):
        n = rng.choice([1, 9, 500])
        counts = [rng.choice([0, 1, 1, rng.randint(-2, 300)]) for _ in range(ref.requests)]
        start = None if rng.random() < 0.4 else [rng.choice([0, x, x - 1, x + 5, rng.randint(-1, x + 1)]) for x in ref.lengths]
        if start is not None:
            ref.plan(n, [0] * ref.requests, start)
        stack, lengths = list(ref.stack), list(ref.lengths)
        ref.plan(n, counts)
        mine = [int(ref.tables[r, j]) for r in range(ref.requests) for j in range(ref._pages(ref.lengths[r]))]
        assert sorted(mine + ref.stack) == list(range(ref.pages))
        assert all(0 <= x <= ref.capacity for x in ref.lengths) and sum(ref.news) <= ref.first[-1] <= n
        if rng.random() < 0.3:
            ref.plan(n, [0] * ref.requests, lengths)
            assert ref.stack == stack and ref.lengths == lengths
