"""The paged cache (ff_paged_*) against the 64-bit reference: plans, stored rows, attention of prompts, chunks and tokens,
whole runs of steps, graphs and refusals."""
import ctypes
import random

import numpy as np
import pytest

from tests.paged_ref import RefPaged

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ff():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_attention_ff_gb300 import build, ff as ffmod
    build.build()
    return ffmod


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def host(t):
    return t.detach().double().cpu().numpy()


def bf16(x):
    """x rounded to bf16 on the GPU, and those values in 64 bits."""
    t = torch.as_tensor(np.asarray(x, np.float32), device="cuda").to(torch.bfloat16)
    return t, host(t)


def make(ff, pages, page_rows, requests, capacity, heads, kv, d, max_rows, **kw):
    cache = ff.PagedCache(pages=pages, page_rows=page_rows, requests=requests, capacity=capacity, heads=heads, kv_heads=kv,
                          head_dim=d, max_rows=max_rows, **kw)
    return cache, RefPaged(pages, page_rows, requests, capacity, kv, d)


def shuffled(cache, ref, seed):
    """Pages in no order, as a pool in use has them."""
    order = np.random.default_rng(seed).permutation(ref.pages)
    cache.free.copy_(torch.as_tensor(order.astype(np.int32)))
    ref.stack = order.tolist()


def check_plan(cache, ref, n):
    assert cache.lengths.tolist() == ref.lengths
    assert cache.first.tolist() == ref.first
    assert cache.slots[:n].tolist() == ref.slots
    assert cache.positions[:n].tolist() == ref.positions
    assert int(cache.n_free) == len(ref.stack)
    assert cache.free[:len(ref.stack)].tolist() == ref.stack
    tables = cache.tables.cpu().numpy()
    for r, x in enumerate(ref.lengths):
        used = ref._pages(x)
        assert np.array_equal(tables[r, :used], ref.tables[r, :used])
    assert cache.error_poll() == (8 if ref.dropped else 0)


def plan(cache, ref, n, counts, start=None):
    cache.plan(n, i32(counts), start=None if start is None else i32(start))
    ref.plan(n, counts, start)
    check_plan(cache, ref, n)


def store(cache, ref, n, rng, layer=0, scale=1.0):
    shape = (n, cache.kv_heads, cache.head_dim)
    k, k64 = bf16(rng.standard_normal(shape) * scale)
    v, v64 = bf16(rng.standard_normal(shape))
    cache.store(layer, k, v)
    ref.store(k64, v64)


def check_attn(cache, ref, q, most=None, layer=0):
    """Runs the attention and compares everything that it may and may not write; returns (out, lse)."""
    n = len(q)
    q, q64 = bf16(q)
    out = torch.full_like(q, 7.0)
    lse = torch.full((n, cache.heads), 7.0, device="cuda")
    cache.attn(layer, q, out, most=most, lse=lse)
    want, want_lse, tol, ltol = ref.attn(q64, most)
    assert cache.error_poll() == 0
    got, got_lse = host(out), host(lse)
    there = ~np.isnan(want)
    assert np.all(got[~there] == 7.0) and np.all(got_lse[np.isnan(want_lse)] == 7.0)
    assert np.all(np.abs(got - want)[there] <= tol[there])
    there = ~np.isnan(want_lse)
    assert np.all(np.abs(got_lse - want_lse)[there] <= ltol[there])
    again = torch.full_like(q, 7.0)
    cache.attn(layer, q, again, most=most)  # without lse: the same bits
    assert torch.equal(again, out)
    return out, lse


# ---- plans -------------------------------------------------------------------


@pytest.mark.parametrize("pages, page_rows, requests, capacity", [
    (1, 16, 1, 16), (7, 16, 1, 100), (40, 32, 5, 333), (300, 64, 33, 5000), (2000, 16, 257, 700), (900, 128, 1024, 1000),
    (5000, 16, 1025, 2000), (9000, 16, 2600, 400),
])
def test_plans_follow_the_rule(ff, pages, page_rows, requests, capacity):
    rng = random.Random(pages)
    n_max = 3000
    cache, ref = make(ff, pages, page_rows, requests, capacity, 1, 1, 64, n_max)
    shuffled(cache, ref, pages)
    for step in range(25):
        n = rng.choice([1, 17, 800, n_max])
        kind = rng.random()
        most = 1 if kind < 0.3 else rng.choice([3, 40, 1000])
        counts = [rng.choice([0, 1, most, rng.randint(-2, most + 3)]) for _ in range(requests)]
        start = None
        if rng.random() < 0.6:
            start = [rng.choice([x, x, 0, x - 1, x - 20, rng.randint(-1, x + 2), 1 << 30]) for x in ref.lengths]
        plan(cache, ref, n, counts, start)
        if rng.random() < 0.3:  # the step is taken back: the stack is as before
            plan(cache, ref, 1, [0] * requests, [x - y for x, y in zip(ref.lengths, ref.news)])


def test_the_most_requests(ff):
    cache, ref = make(ff, 20000, 16, 8192, 64, 1, 1, 64, 20000)
    plan(cache, ref, 20000, [(r * 7) % 5 for r in range(8192)])
    plan(cache, ref, 20000, [1] * 8192, [x if r % 3 else 0 for r, x in enumerate(ref.lengths)])
    plan(cache, ref, 1, [0] * 8192, [0] * 8192)
    assert int(cache.n_free) == 20000


def test_rows_without_a_page_are_dropped_and_reported(ff):
    cache, ref = make(ff, 5, 16, 4, 64, 2, 1, 64, 200)
    plan(cache, ref, 200, [17, 40, 16, 3])   # 2 + 3 pages, then none
    assert ref.lengths == [17, 40, 0, 0] and ref.dropped
    rng = np.random.default_rng(0)
    store(cache, ref, 200, rng)
    check_attn(cache, ref, rng.standard_normal((200, 2, 64)))
    plan(cache, ref, 100, [14, 10, 1, 1])    # up to what their pages hold
    assert ref.lengths == [31, 48, 0, 0] and ref.dropped
    plan(cache, ref, 100, [40, 0, 0, 0], [31, 0, 0, 0])  # past the capacity
    assert ref.lengths == [64, 0, 0, 0] and ref.dropped
    plan(cache, ref, 20, [0, 15, 15, 0])     # past the packed rows
    assert ref.news == [0, 15, 0, 0] and ref.dropped


def test_whatever_the_tables_hold(ff):
    """Lengths, pages and stack that make no sense lead nowhere outside the pool."""
    cache, _ = make(ff, 6, 16, 3, 64, 2, 2, 64, 64)
    k, _ = bf16(np.ones((64, 2, 64)))
    q = k
    for lengths, table, n_free in ([(-5, 1 << 30, 64), 1 << 30, 1 << 30], [(64, 64, 64), -7, -3], [(1, 2, 1 << 29), 5, 0]):
        cache.lengths.copy_(i32(lengths))
        cache.tables.fill_(table)
        cache.free.fill_(table)
        cache.n_free.fill_(n_free)
        for counts, start in (([1, 30, 5], None), ([64, 64, 64], None), ([-9, 1 << 30, 3], None), ([0, 0, 0], i32([0, -1, 1 << 30]))):
            cache.plan(64, i32(counts), start=start)
            cache.store(0, k, k)
            cache.attn(0, q, torch.empty_like(q))
    torch.cuda.synchronize()
    cache.error_poll()
    assert 0 <= int(cache.n_free) <= 6 and int(cache.lengths.min()) >= 0 and int(cache.lengths.max()) <= 64
    assert int(cache.slots.max()) < 6 * 16


# ---- rows --------------------------------------------------------------------


@pytest.mark.parametrize("page_rows, kv, d, n", [(16, 1, 64, 1), (16, 3, 128, 77), (32, 8, 128, 300), (64, 5, 64, 200),
                                                 (128, 40, 128, 129)])
def test_rows_go_to_their_places_and_nowhere_else(ff, page_rows, kv, d, n):
    rng = np.random.default_rng(n)
    requests = 5
    cache, ref = make(ff, 60, page_rows, requests, 10 * page_rows, kv, kv, d, n + 9, n_layers=2)
    shuffled(cache, ref, n)
    for layer in (0, 1):
        for x in cache.layer(layer):
            x.fill_(3.0)
    ref.pool = {x: np.full_like(y, 3.0) for x, y in ref.pool.items()}
    counts = [n // 3, 0, n - n // 3 - n // 4, n // 4, 0]
    for again in range(3):
        plan(cache, ref, n + 9, counts)
        store(cache, ref, n + 9, rng, layer=1)
    k, v = cache.layer(1)
    assert np.array_equal(host(k).transpose(0, 2, 1, 3), ref.pool["k"])
    assert np.array_equal(host(v).transpose(0, 2, 1, 3), ref.pool["v"])
    assert all(bool((x == 3.0).all()) for x in cache.layer(0))


# ---- attention ---------------------------------------------------------------

CASES = [
    # page_rows, heads, kv_heads, d, rows held before, new rows, more rows of the buffers
    (16, 1, 1, 64, [0], [1], 0),                       # the first token
    (16, 2, 2, 128, [207], [1], 3),
    (16, 12, 12, 128, [2000], [1], 0),
    (32, 8, 2, 128, [0, 15, 16, 31, 32, 333, 1000], [1] * 7, 1),
    (64, 40, 8, 64, [700, 0, 5, 64, 63], [1, 5, 0, 2, 3], 6),
    (128, 6, 2, 128, [127, 128, 129, 3000], [8, 1, 7, 8], 0),    # 24 rows of a head
    (16, 32, 1, 64, [100, 17], [1, 1], 0),             # 32 rows
    (16, 33, 1, 64, [100, 17], [1, 1], 0),             # and one more
    (32, 130, 1, 64, [150, 3], [1, 2], 0),             # a group wider than a tile
    (16, 300, 2, 128, [40], [3], 0),
    (16, 2, 2, 64, [0], [208], 0),                     # prompts
    (16, 4, 4, 128, [0], [129], 2),
    (16, 8, 2, 64, [0] * 6, [1, 63, 64, 65, 333, 200], 5),
    (32, 5, 1, 128, [0, 0, 0], [300, 2, 31], 0),
    (64, 6, 2, 128, [0, 0], [257, 515], 1),
    (128, 7, 1, 64, [0, 0], [130, 40], 0),
    (16, 12, 12, 128, [0], [700], 0),
    (128, 3, 3, 128, [0, 0], [512, 256], 0),
    (16, 8, 2, 128, [500, 31, 0, 1000, 3], [100, 1, 40, 300, 0], 9),   # chunks and tokens
    (32, 10, 2, 64, [2000, 1, 999], [1, 130, 33], 0),
    (64, 16, 1, 128, [3000], [90], 0),
    (128, 4, 2, 128, [127, 255], [1, 128], 0),
    (16, 24, 2, 64, [5000, 20], [150, 3], 4),
    (16, 96, 2, 128, [70], [50], 0),                   # 48 rows of a token
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(ff, case):
    page_rows, heads, kv, d, held, new, more = CASES[case]
    rng = np.random.default_rng(case)
    rows = [x + y for x, y in zip(held, new)]
    pages = sum(-(-x // page_rows) for x in rows)
    n = max(max(1, sum(held)), sum(new) + more)
    cache, ref = make(ff, pages, page_rows, len(held), max(rows) + 5, heads, kv, d, n)
    shuffled(cache, ref, case)
    for x in cache.layer(0):  # what nobody stored is NaN
        x.fill_(float("nan"))
    if sum(held):
        plan(cache, ref, n, held)
        store(cache, ref, n, rng, scale=1.5)
    n = sum(new) + more
    plan(cache, ref, n, new)
    store(cache, ref, n, rng, scale=1.5)
    check_attn(cache, ref, rng.standard_normal((n, heads, d)))
    check_attn(cache, ref, rng.standard_normal((n, heads, d)), most=max(new))
    if max(new) > 1:
        check_attn(cache, ref, rng.standard_normal((n, heads, d)), most=max(1, max(new) // 2))


@pytest.mark.parametrize("d, scale", [(128, 30.0), (64, 1e3), (128, 3e4)])
@pytest.mark.parametrize("new", [[1, 3], [200, 90]])
def test_peaked_rows(ff, d, scale, new):
    """Scores of hundreds to billions: one key has all the weight, and nothing overflows."""
    rng = np.random.default_rng(int(scale))
    cache, ref = make(ff, 60, 16, 2, 800, 4, 2, d, 700)
    plan(cache, ref, 700, [300, 350])
    store(cache, ref, 700, rng, scale=scale)
    plan(cache, ref, sum(new), new)
    store(cache, ref, sum(new), rng, scale=scale)
    q, q64 = bf16(rng.standard_normal((sum(new), 4, d)) * scale)
    out, lse = torch.zeros_like(q), torch.zeros((sum(new), 4), device="cuda")
    cache.attn(0, q, out, lse=lse)
    want, want_lse, tol, ltol = ref.attn(q64)
    got, got_lse = host(out), host(lse)
    assert np.all(np.isfinite(got)) and np.all(np.isfinite(got_lse))
    assert np.all(np.abs(got_lse - want_lse) <= ltol)
    # where the scores' own errors leave the weights known
    known = ltol < 0.01
    assert np.all(np.abs(got - want)[known] <= tol[known])
    assert np.all(np.abs(got) <= 1.01 * np.abs(ref.pool["v"]).max())


@pytest.mark.parametrize("new", [[1, 1, 0], [40, 3, 0], [300, 1, 150]])
def test_what_no_row_may_see(ff, new):
    """NaN and infinities in the rows of other requests, behind the last row of a page, in free pages, in padded queries
    and in rows without a place."""
    rng = np.random.default_rng(3)
    held, n = [70, 333, 20], sum(new) + 6
    cache, ref = make(ff, 70, 16, 3, 700, 6, 2, 128, 600)
    shuffled(cache, ref, 1)
    plan(cache, ref, 600, held)
    store(cache, ref, 600, rng)
    plan(cache, ref, n, new)
    store(cache, ref, n, rng)
    q = rng.standard_normal((n, 6, 128))
    want, want_lse = check_attn(cache, ref, q)
    mine = np.zeros((70, 16), bool)
    for r in (0, 1):
        at = np.arange(ref.lengths[r])
        mine[ref.tables[r, at // 16], at % 16] = True
    foreign = torch.as_tensor(~mine, device="cuda")[:, None, :, None]
    for bad in (float("nan"), float("inf"), float("-inf")):
        for x in cache.layer(0):
            x.copy_(torch.where(foreign, torch.full_like(x, bad), x))
        dirty, _ = bf16(q)
        dirty[sum(new):] = bad
        out, lse = torch.full_like(want, 7.0), torch.full_like(want_lse, 7.0)
        cache.attn(0, dirty, out, lse=lse)
        m = new[0] + new[1]
        assert torch.equal(out[:m], want[:m]) and torch.equal(lse[:m], want_lse[:m])
        assert bool((out[sum(new):] == 7.0).all()) and bool((lse[sum(new):] == 7.0).all())


def test_values_that_are_not_finite_stay_with_their_request(ff):
    rng = np.random.default_rng(5)
    for new in ([1, 1], [100, 60]):
        cache, ref = make(ff, 40, 32, 2, 500, 4, 2, 64, 400)
        plan(cache, ref, 400, [150, 200])
        store(cache, ref, 400, rng)
        plan(cache, ref, sum(new), new)
        store(cache, ref, sum(new), rng)
        q, _ = bf16(rng.standard_normal((sum(new), 4, 64)))
        clean = torch.zeros_like(q)
        cache.attn(0, q, clean)
        page = int(ref.tables[0, 0])
        cache.layer(0)[1][page, 1, 3, 5] = float("inf")  # feature 5 of a row of request 0, kv head 1
        out = torch.zeros_like(q)
        cache.attn(0, q, out)
        same = torch.ones_like(q, dtype=torch.bool)
        same[:new[0], 2:, 5] = False
        assert torch.equal(out[same], clean[same])
        assert not bool(torch.isfinite(out[~same]).any())


def test_offsets_past_32_bits(ff):
    """A pool of 6 GB for K and V each: the request's pages lie at its end."""
    pages, kv, d, new = 180_000, 8, 128, 70
    cache, ref = make(ff, pages, 16, 2, 400, 16, kv, d, 400)
    ref.pool = {x: np.zeros((1, 1, kv, d)) for x in "kv"}
    order = np.arange(pages)  # the highest page on top
    cache.free.copy_(torch.as_tensor(order.astype(np.int32)))
    rng = np.random.default_rng(1)
    small = RefPaged(100, 16, 2, 400, kv, d)  # the same, of the last 100 pages
    small.stack = list(range(100))
    for counts in ([300, 40], [1, new]):
        n = sum(counts)
        cache.plan(n, i32(counts))
        small.plan(n, counts)
        assert cache.slots[:n].tolist() == [x + (pages - 100) * 16 for x in small.slots]
        store(cache, small, n, rng)
        check_attn(cache, small, rng.standard_normal((n, 16, d)))


# ---- a run ---------------------------------------------------------------------


@pytest.mark.parametrize("page_rows, heads, kv, d", [(16, 8, 2, 128), (64, 4, 4, 64)])
def test_a_run_of_steps(ff, page_rows, heads, kv, d):
    """Prompts come in, tokens are drafted and partly rejected, requests end and others take their pages: two layers,
    every step checked."""
    rng, draw = np.random.default_rng(9), random.Random(9)
    requests, layers = 6, 2
    cache, ref = make(ff, 900 // page_rows, page_rows, requests, 400, heads, kv, d, 500, n_layers=layers)
    refs = [ref, *[RefPaged(ref.pages, page_rows, requests, 400, kv, d) for _ in range(layers - 1)]]
    for step in range(14):
        start, counts = list(ref.lengths), [0] * requests
        for r in range(requests):
            kind = draw.random()
            if not start[r]:
                counts[r] = draw.choice([0, 1, 33, 150])   # a prompt, or none
            elif kind < 0.15:
                start[r], counts[r] = 0, draw.choice([0, 20, 100])  # it ends; another may come
            elif kind < 0.5:
                start[r], counts[r] = start[r] - draw.randint(0, min(start[r], 3)), draw.randint(1, 4)  # drafts rejected
            else:
                counts[r] = draw.choice([1, 1, 40])
        n = max(1, sum(counts) + draw.randint(0, 4))
        cache.plan(n, i32(counts), start=i32(start))
        for one in refs:
            one.plan(n, counts, start)
        check_plan(cache, ref, n)
        for layer, one in enumerate(refs):
            store(cache, one, n, rng, layer=layer)
            check_attn(cache, one, rng.standard_normal((n, heads, d)), most=max(1, max(counts)), layer=layer)


def test_a_recorded_step_follows_its_counts(ff):
    rng = np.random.default_rng(4)
    heads, kv, d, requests, n = 8, 2, 128, 4, 320
    cache, ref = make(ff, 120, 16, requests, 600, heads, kv, d, n)
    counts, start = i32([0] * requests), i32([0] * requests)
    k, v, q = (torch.zeros((n, x, d), dtype=torch.bfloat16, device="cuda") for x in (kv, kv, heads))
    out, lse = torch.zeros_like(q), torch.zeros((n, heads), device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cache.plan(n, counts, start=start)
        cache.store(0, k, v)
        cache.attn(0, q, out, lse=lse)
    for new, cut in (([200, 3, 0, 60], None), ([1, 1, 1, 1], None), ([1, 300, 2, 1], [201, 0, 1, 50]), ([0, 0, 0, 0], None)):
        cut = list(ref.lengths) if cut is None else cut
        counts.copy_(i32(new))
        start.copy_(i32(cut))
        values = [bf16(rng.standard_normal(x.shape)) for x in (k, v, q)]
        for to, (x, _) in zip((k, v, q), values):
            to.copy_(x)
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        ref.plan(n, new, cut)
        check_plan(cache, ref, n)
        ref.store(values[0][1], values[1][1])
        want, want_lse, tol, ltol = ref.attn(values[2][1])
        got, got_lse = host(out), host(lse)
        gone = np.isnan(want)
        assert np.all(got[gone] == 7.0) and np.all(np.abs(got - want)[~gone] <= tol[~gone])
        gone = np.isnan(want_lse)
        assert np.all(got_lse[gone] == 7.0) and np.all(np.abs(got_lse - want_lse)[~gone] <= ltol[~gone])


def test_calls_on_other_streams_wait_for_each_other(ff):
    rng = np.random.default_rng(6)
    cache, ref = make(ff, 400, 16, 4, 1600, 8, 2, 128, 1500)
    streams = [torch.cuda.Stream() for _ in range(3)]
    values = []
    for counts in ([700, 200, 1, 333], [1, 1, 1, 1], [3, 100, 0, 5]):
        n = sum(counts)
        values.append([bf16(rng.standard_normal((n, x, 128))) for x in (2, 2, 8)] + [i32(counts), counts, n])
    torch.cuda.synchronize()
    for (k, k64), (v, v64), (q, q64), device_counts, counts, n in values:
        out, lse = torch.full_like(q, 7.0), torch.full((n, 8), 7.0, device="cuda")
        torch.cuda.synchronize()
        cache.plan(n, device_counts, stream=streams[0])
        cache.store(0, k, v, stream=streams[1])
        cache.attn(0, q, out, lse=lse, stream=streams[2])
        streams[2].synchronize()
        ref.plan(n, counts)
        ref.store(k64, v64)
        want, _, tol, _ = ref.attn(q64)
        assert np.all(np.abs(host(out) - want) <= tol)


# ---- refusals ------------------------------------------------------------------


def test_bad_calls_are_refused(ff):
    cache, _ = make(ff, 10, 16, 3, 64, 4, 2, 64, 40)
    lib, h = ff.lib(), cache.handle
    P = ctypes.c_void_p
    counts = i32([1, 2, 3])
    q = torch.zeros((40, 4, 64), dtype=torch.bfloat16, device="cuda")
    k, v, out = torch.zeros_like(q[:, :2]).contiguous(), torch.zeros_like(q[:, :2]).contiguous(), torch.zeros_like(q)
    lse = torch.zeros((40, 4), device="cuda")
    c, qp, kp, vp, op, lp = (x.data_ptr() for x in (counts, q, k, v, out, lse))
    for n, start, cnt in ((0, None, c), (41, None, c), (-1, None, c), (6, None, None), (6, c + 2, c), (6, None, c + 1)):
        assert lib.ff_paged_plan(h, n, start, cnt, None) == 1
    for layer, n, a, b in ((-1, 6, kp, vp), (1, 6, kp, vp), (0, 0, kp, vp), (0, 41, kp, vp), (0, 6, None, vp), (0, 6, kp, None),
                           (0, 6, kp + 8, vp), (0, 6, kp, vp + 2)):
        assert lib.ff_paged_store(h, layer, n, a, b, None) == 1
    for layer, n, most, a, o, l in ((-1, 6, 1, qp, op, lp), (1, 6, 1, qp, op, lp), (0, 0, 1, qp, op, lp), (0, 41, 1, qp, op, lp),
                                    (0, 6, 0, qp, op, lp), (0, 6, -1, qp, op, lp), (0, 6, 1, None, op, lp), (0, 6, 1, qp, None, lp),
                                    (0, 6, 1, qp + 8, op, lp), (0, 6, 1, qp, op + 4, lp), (0, 6, 1, qp, op, lp + 2),
                                    (0, 6, 1, qp, qp, lp), (0, 6, 1, qp, qp + 16, lp), (0, 6, 1, qp, op, qp), (0, 6, 1, qp, op, op + 64)):
        assert lib.ff_paged_attn(h, layer, n, most, a, o, l, None) == 1
    with pytest.raises(TypeError):
        cache.plan(6, counts.long())
    with pytest.raises(TypeError):
        cache.plan(6, counts.cpu())
    with pytest.raises(ValueError):
        cache.plan(6, counts[:2])
    with pytest.raises(TypeError):
        cache.plan(6, i32([1, 0, 2, 0, 3, 0])[::2])
    with pytest.raises(ValueError):
        cache.store(0, k, v[:6])
    with pytest.raises(TypeError):
        cache.store(0, k.float(), v)
    with pytest.raises(TypeError):
        cache.store(0, q[:, :2], v)
    with pytest.raises(ValueError):
        cache.attn(0, q, out[:6])
    with pytest.raises(TypeError):
        cache.attn(0, q, out, lse=lse.double())
    with pytest.raises(ff.FFError):
        cache.attn(0, q, out, most=0)
    torch.cuda.synchronize()
    assert cache.lengths.tolist() == [0, 0, 0] and int(cache.n_free) == 10


def test_memory_limits_and_views(ff):
    with pytest.raises(ff.FFError) as e:
        ff.PagedCache(pages=1000, requests=2, max_bytes=1 << 20)
    assert e.value.status == 4
    cache = ff.PagedCache(pages=100, requests=2, capacity=50, heads=4, head_dim=64, max_rows=7)
    assert cache.bytes() >= 2 * 100 * 16 * 4 * 64 * 2
    k, v = cache.layer(0)
    assert k.shape == v.shape == (100, 4, 16, 64) and k.dtype == torch.bfloat16
    assert cache.tables.shape == (2, 4) and cache.slots.tolist() == [-1] * 7 and cache.free.tolist() == list(range(99, -1, -1))
    lengths = cache.lengths
    del cache, k, v
    assert lengths.tolist() == [0, 0]  # a view keeps the memory
