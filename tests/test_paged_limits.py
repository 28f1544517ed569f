"""The paged cache's longest request: what its kernels' waits, sums and lists are good for."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def ff():
    from kv_cache_attention_ff_gb300 import build, ff as ffmod
    build.build()
    return ffmod


# A block of rows whose request is not cut passes through one CTA, a tile of 128 keys in some 2 us at most (two query
# tiles: 2600 clocks; K and V of 128 keys for every SM from memory: 1.5 us), and a warp without rows in four units waits
# for all of them: 2^24 keys take 1 s, 2^26 take the 4 s after which a wait gives up.
@pytest.mark.parametrize("capacity", [(1 << 24) + 1, 1 << 25, 1 << 28, 1 << 30])
def test_requests_longer_than_the_waits_allow_are_refused(ff, capacity):
    d = ff.PagedDesc()
    assert ff.lib().ff_paged_desc_default(ctypes.byref(d)) == 0
    d.capacity = capacity
    h = ctypes.c_void_p()
    assert ff.lib().ff_paged_create(ctypes.byref(d), ctypes.byref(h)) == 1
    assert not h.value


def test_the_longest_request_is_not_refused(ff):
    d = ff.PagedDesc()
    assert ff.lib().ff_paged_desc_default(ctypes.byref(d)) == 0
    d.capacity = 1 << 24
    h = ctypes.c_void_p()
    rc = ff.lib().ff_paged_create(ctypes.byref(d), ctypes.byref(h))
    assert rc in (0, 5, 7)  # a GPU that there is not, or another one
    if rc == 0:
        assert ff.lib().ff_paged_destroy(h) == 0
