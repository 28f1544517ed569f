"""The 8-bit cache where it could go wrong: offsets past 32 bits, many sequences, wide groups, rows and queries that hold
NaN where nothing may look, graphs side by side, calls repeated at once."""
import gc

import numpy as np
import pytest

from tests.kv8_ref import RefCache, lse_tol, out_tol
from tests.test_gpu_kv8 import bf16, check_attn, check_cache, host, i32, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ff():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_attention_ff_gb300 import build, ff as ffmod
    build.build()
    return ffmod


@pytest.mark.parametrize("n", [3, 40])
def test_offsets_past_32_bits(ff, n):
    """2.2 million rows of 8 heads: 2.25 GB of codes for K and V each.  All rows but the last few are zeros, so that
    the softmax is known: each zero row has score 0."""
    rows, kv, d, tail = 2_200_003, 8, 128, 70
    cache = ff.KV8Cache(batch=1, capacity=rows + 100, heads=kv, kv_heads=kv, head_dim=d, max_tokens=n)
    k8, v8, ks, vs, lengths = cache.layer(0)
    ks.fill_(1.0)
    vs.fill_(1.0)
    lengths.fill_(rows - tail)
    rng = np.random.default_rng(n)
    k, k64 = bf16(rng.standard_normal((1, tail, kv, d)) * 2)
    v, v64 = bf16(rng.standard_normal((1, tail, kv, d)) * 8)
    cache.append(0, k, v)
    assert lengths.tolist() == [rows]
    # what was stored: the tail as the reference stores it behind 2200003 - 70 rows of scale 1
    ref = RefCache(1, 256, kv, d)
    at = (rows - tail) % 64
    ref.length[:] = at
    for x in "kv":
        ref.e[x][:, 0] = 0
    ref.append(k64, v64)
    kk, vv = torch.empty_like(k), torch.empty_like(v)
    cache.load(0, kk, vv, start=i32([rows - tail]))
    rk, rv = ref.load(tail, [at])
    assert np.array_equal(host(kk), rk) and np.array_equal(host(vv), rv)

    q, q64 = bf16(rng.standard_normal((1, n, kv, d)) * 2)
    out, lse = torch.zeros_like(q), torch.zeros((1, n, kv), device="cuda")
    w = torch.zeros((1, kv, rows + 100), device="cuda")
    cache.attn(0, q, out, lse=lse, weights=w)
    assert cache.error_poll() == 0
    s = np.einsum("nhd,thd->nht", q64[0], rk[0]) / np.sqrt(d)
    top = np.maximum(s.max(-1), 0.0)
    z = np.exp(s - top[..., None])
    total = z.sum(-1) + (rows - tail) * np.exp(-top)
    want = np.einsum("nht,thd->nhd", z, rv[0]) / total[..., None]
    spread = np.einsum("nht,thd->nhd", z, np.abs(rv[0])) / total[..., None]
    mag = (np.einsum("nhd,thd->nht", np.abs(q64[0]), np.abs(rk[0])) / np.sqrt(d)).max(-1)
    # the sum of the many equal rows is made of blocks' sums: at most 2^-24 for each of 2.2 million additions would be
    # 0.13; pieces of 32 to 128 keys are added up one after the other, 2^-24 each, and merged
    tol = out_tol(want, spread, mag, d, 0) + np.abs(want) * (rows / 32) * 2.0 ** -24
    assert np.all(np.abs(host(out)[0] - want) <= tol)
    want_lse = top + np.log(total)
    assert np.all(np.abs(host(lse)[0] - want_lse) <= lse_tol(mag, d) + np.abs(want_lse) * 2.0 ** -24 + rows / 32 * 2.0 ** -24)
    got = host(w[0, :, rows - tail:rows])
    want_w = (z / total[..., None]).sum(0)
    assert np.all(np.abs(got - want_w) <= want_w * (2 * lse_tol(mag.max(), d) + (n + rows / 32) * 2.0 ** -23))
    assert not bool(w[:, :, rows:].any())

    # the tail is the heaviest but for some of its rows; they move to the front of a small cache
    dst = ff.KV8Cache(batch=1, capacity=128, heads=kv, kv_heads=kv, head_dim=d, max_tokens=1)
    wout, kept = torch.zeros((1, kv, 128), device="cuda"), torch.zeros((1, kv, 100), dtype=torch.int32, device="cuda")
    weights = torch.zeros_like(w)
    weights[:, :, rows - tail:rows] = torch.rand((1, kv, tail), device="cuda") + 0.1
    cache.evict(0, dst, 0, 100, 5, weights, wout, kept)
    # 30 zero-weight rows fill the budget: the lowest ones
    want_kept = list(range(30)) + list(range(rows - tail, rows))
    assert all(row == want_kept for row in kept[0].tolist())
    dst.load(0, kk, vv, start=i32([30]))
    blocks = RefCache(1, 128, kv, d)
    blocks.append(np.concatenate([np.zeros((1, 30, kv, d)), rk], 1), np.concatenate([np.zeros((1, 30, kv, d)), rv], 1))
    wk, wv = blocks.load(tail, [30])
    assert np.array_equal(host(kk), wk) and np.array_equal(host(vv), wv)
    del cache, dst, k8, v8, ks, vs, lengths
    gc.collect()


WIDE = [
    # batch, n, heads, kv_heads, lengths, counts, causal
    (1, 1, 48, 1, [300], None, True),          # one token, 48 rows
    (1, 1, 130, 1, [150], None, True),         # a group wider than a tile of 128
    (2, 2, 160, 1, [200, 3], [2, 1], True),
    (1, 3, 66, 2, [129], None, True),          # 33 heads of a group: tiles of 3 tokens
    (2, 9, 20, 4, [700, 65], [9, 4], False),   # 45 rows
    (1, 600, 4, 2, [900], None, True),         # 1200 rows of a head
    (900, 1, 1, 1, None, None, True),          # more sequences than run at once
    (130, 2, 8, 8, None, None, True),
    (40, 3, 4, 1, None, None, False),
]


@pytest.mark.parametrize("case", range(len(WIDE)))
def test_wide_groups_and_many_sequences(ff, case):
    batch, n, heads, kv, lengths, counts, causal = WIDE[case]
    rng = np.random.default_rng(case)
    if lengths is None:
        lengths = rng.integers(0, 90, batch).tolist()
    m = max(lengths)
    cache, ref = make(ff, batch, m + 3, heads, kv, 64, max_tokens=n)
    k, k64 = bf16(rng.standard_normal((batch, m, kv, 64)))
    v, v64 = bf16(rng.standard_normal((batch, m, kv, 64)))
    cache.append(0, k, v, counts=i32(lengths))
    ref.append(k64, v64, None, lengths)
    check_attn(cache, ref, rng.standard_normal((batch, n, heads, 64)), causal=causal, counts=counts, weigh=True)


@pytest.mark.parametrize("n, heads, kv", [(6, 2, 2), (6, 8, 2), (60, 4, 2), (150, 1, 1)])
def test_padded_queries_may_hold_anything(ff, n, heads, kv):
    rng = np.random.default_rng(n)
    cache, ref = make(ff, 3, 300, heads, kv, 128, max_tokens=n)
    k, k64 = bf16(rng.standard_normal((3, 290, kv, 128)))
    cache.append(0, k, k, counts=i32([290, 100, 64]))
    ref.append(k64, k64, None, [290, 100, 64])
    counts = [n // 2, n, 1]
    q = rng.standard_normal((3, n, heads, 128))
    clean = check_attn(cache, ref, q, causal=True, counts=counts, weigh=True)
    dirty, _ = bf16(q)
    for b, c in enumerate(counts):
        dirty[b, c:] = float("nan")
    out = torch.full_like(dirty, 3.0)
    lse = torch.full((3, n, heads), 3.0, device="cuda")
    w = torch.zeros((3, kv, 300), device="cuda")
    cache.attn(0, dirty, out, causal=True, counts=i32(counts), lse=lse, weights=w)
    assert np.array_equal(host(out), clean)
    assert not bool(torch.isnan(lse).any()) and not bool(torch.isnan(w).any())
    # each valid query that sees a row (the last of a causal call, as many as rows are held) hands out one unit per head
    total = host(w).sum(-1)
    want = np.minimum(counts, [290, 100, 64])[:, None] * heads / kv
    assert np.all(np.abs(total - want) <= want * 2.0 ** -10)


@pytest.mark.parametrize("n", [1, 100])
def test_not_a_number_in_a_key_stays_with_those_who_see_it(ff, n):
    rng = np.random.default_rng(n)
    cache, _ = make(ff, 1, 400, 2, 2, 64, max_tokens=n)
    x = rng.standard_normal((1, 400, 2, 64)).astype(np.float32)
    v, _ = bf16(rng.standard_normal((1, 400, 2, 64)))
    outs = []
    for bad in (False, True):
        if bad:
            x[0, 399, 1, 7] = np.nan
        k, _ = bf16(x)
        cache.append(0, k, v, start=i32([0]))
        q, _ = bf16(np.random.default_rng(5).standard_normal((1, n, 2, 64)))
        out = torch.zeros_like(q)
        cache.attn(0, q, out, causal=True)
        outs.append(host(out))
    assert np.array_equal(outs[0][:, :, 0], outs[1][:, :, 0])        # the other head
    assert np.array_equal(outs[0][:, :-1], outs[1][:, :-1])          # queries before the row
    assert np.all(np.isnan(outs[1][0, -1, 1]))


def test_graphs_of_two_caches_side_by_side(ff):
    rng = np.random.default_rng(40)
    parts = []
    for i in range(2):
        cache, ref = make(ff, 2, 900, 4, 2, 64, max_tokens=50)
        k, k64 = bf16(rng.standard_normal((2, 800, 2, 64)))
        cache.append(0, k, k)
        ref.append(k64, k64)
        q, q64 = bf16(rng.standard_normal((2, 50 if i else 1, 4, 64)))
        out, w = torch.zeros_like(q), torch.zeros((2, 2, 900), device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cache.attn(0, q, out, weights=w)
        parts.append((cache, ref, q64, out, w, graph, torch.cuda.Stream()))
    turns = 20
    for _ in range(turns):
        for *_, graph, stream in parts:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for cache, ref, q64, out, w, *_ in parts:
        ro, _, rw, (spread, mag, wtol) = ref.attn(q64, weights=np.zeros((2, 2, 900)))
        assert np.all(np.abs(host(out) - ro) <= out_tol(ro, spread, mag, 64, 800))
        # one turn's bound for each, and an fp32 rounding of the running sum
        assert np.all(np.abs(host(w) - turns * rw) <= turns * (wtol + turns * 2.0 ** -23 * rw))
        assert cache.error_poll() == 0


def test_a_graph_between_eager_calls(ff):
    """Replays and eager calls in turn on one stream, append and attention of another shape among them."""
    rng = np.random.default_rng(41)
    cache, ref = make(ff, 1, 700, 2, 2, 64, max_tokens=40)
    k = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(0, k, k)
        cache.attn(0, q, out, causal=True)
    for turn in range(6):
        big, big64 = bf16(rng.standard_normal((1, 37, 2, 64)))
        bq, bq64 = bf16(rng.standard_normal((1, 37, 2, 64)))
        bout = torch.zeros_like(bq)
        cache.append(0, big, big)
        cache.attn(0, bq, bout, causal=True)
        ref.append(big64, big64)
        want = ref.attn(bq64, True)
        a, a64 = bf16(rng.standard_normal((1, 1, 2, 64)))
        e, e64 = bf16(rng.standard_normal((1, 1, 2, 64)))
        k.copy_(a), q.copy_(e)
        graph.replay()
        ref.append(a64, a64)
        for got, (ro, _, _, (spread, mag, _)) in ((bout, want), (out, ref.attn(e64, True))):
            assert np.all(np.abs(host(got) - ro) <= out_tol(ro, spread, mag, 64, 700))
    check_cache(cache, ref)


def test_lengths_that_are_out_of_range_count_as_the_bounds(ff):
    cache, _ = make(ff, 3, 100, 2, 2, 64, max_tokens=40)
    k, _ = bf16(np.random.default_rng(1).standard_normal((3, 100, 2, 64)))
    cache.append(0, k, k)
    q, _ = bf16(np.random.default_rng(2).standard_normal((3, 40, 2, 64)))
    for n in (1, 40):
        qn = q[:, :n].contiguous()
        want, got = torch.zeros_like(qn), torch.zeros_like(qn)
        cache.lengths(0).copy_(i32([100, 0, 100]))
        cache.attn(0, qn, want)
        cache.lengths(0).copy_(i32([2 ** 31 - 1, -7, 101]))
        cache.attn(0, qn, got)
        assert torch.equal(want.view(torch.int16), got.view(torch.int16))
    kk, vv = torch.empty_like(k), torch.empty_like(k)
    cache.load(0, kk, vv)
    assert not bool(kk[1].any()) and bool(kk[0].any())


def test_capacity_of_one_row(ff):
    cache, ref = make(ff, 1, 1, 3, 1, 64, max_tokens=60)
    k, k64 = bf16(np.random.default_rng(3).standard_normal((1, 1, 1, 64)))
    cache.append(0, k, k)
    ref.append(k64, k64)
    for n in (1, 60):
        check_attn(cache, ref, np.random.default_rng(n).standard_normal((1, n, 3, 64)), weigh=True, causal=n == 1)


def test_zero_rows_that_leave_a_block_of_huge_scale_stay_zeros(ff):
    """Rows 0..63 hold one value of 2^115 and zeros elsewhere; only zero rows are kept, whose block has the least scale."""
    (cache, ref), (dst, dref) = make(ff, 1, 128, 2, 2, 64), make(ff, 1, 64, 2, 2, 64)
    x = np.zeros((1, 64, 2, 64))
    x[0, 5, :, 7] = 2.0 ** 115
    k, k64 = bf16(x)
    cache.append(0, k, k)
    ref.append(k64, k64)
    w = np.ones((1, 2, 128), np.float32)
    w[0, :, 5] = 0.0
    wout = torch.empty((1, 2, 64), device="cuda")
    kept = torch.empty((1, 2, 20), dtype=torch.int32, device="cuda")
    cache.evict(0, dst, 0, 20, 10, torch.from_numpy(w).cuda(), wout, kept)
    ref.evict(w, 20, 10, dref)
    assert 5 not in kept.cpu().numpy()
    check_cache(dst, dref)


def test_each_threads_own_stream_is_a_stream_of_its_own(ff):
    """The handle 2 stands for another stream in every host thread: the second thread's call has to wait for the first's."""
    import threading
    cache, ref = make(ff, 1, 256, 2, 2, 64, max_tokens=4)
    rng = np.random.default_rng(7)
    k, k64 = bf16(rng.standard_normal((1, 200, 2, 64)))
    q, q64 = bf16(rng.standard_normal((1, 4, 2, 64)))
    out = torch.zeros_like(q)
    ref.append(k64, k64)
    torch.cuda.synchronize()
    failed = []

    def run(call):
        def body():
            try:
                call(torch.cuda.ExternalStream(2))
            except Exception as e:
                failed.append(e)
        t = threading.Thread(target=body)
        t.start()
        t.join()

    def first(stream):
        with torch.cuda.stream(stream):
            torch.cuda._sleep(50_000_000)
        cache.append(0, k, k, stream=stream)

    def second(stream):
        cache.attn(0, q, out, stream=stream)
        stream.synchronize()

    run(first)
    run(second)
    assert not failed
    want, _, _, (spread, mag, _) = ref.attn(q64)
    assert np.all(np.abs(host(out) - want) <= out_tol(want, spread, mag, 64, 200))


def test_overlapping_outputs_are_refused(ff):
    import ctypes
    cache, _ = make(ff, 1, 128, 2, 2, 64, max_tokens=4)
    lib, h = ff.lib(), cache.handle
    kv = torch.zeros((1, 8, 2, 64), dtype=torch.bfloat16, device="cuda")
    q, out = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((2, 2, 128), device="cuda")
    P = lambda t, off=0: ctypes.c_void_p(t.data_ptr() + off)
    assert lib.ff_kv8_load(h, 0, 4, None, P(kv), P(kv, 1008), None) == 1
    assert lib.ff_kv8_attn(h, 0, 4, P(q), None, 0, P(out), P(q), None, None, None) == 1          # lse over q
    assert lib.ff_kv8_attn(h, 0, 4, P(q), None, 0, P(out), P(out), None, None, None) == 1        # lse over out
    assert lib.ff_kv8_attn(h, 0, 4, P(q), None, 0, P(out), P(w), None, P(w), None) == 1          # weights over lse
    assert lib.ff_kv8_attn(h, 0, 4, P(q), None, 0, P(out), None, P(w, 4), P(w), None) == 1       # shifted weights
    assert lib.ff_kv8_attn(h, 0, 4, P(q), None, 0, P(w), None, None, P(w), None) == 1            # weights over out
    assert lib.ff_kv8_attn(h, 0, 4, P(q), None, 0, P(out), None, P(w, 1024), P(w), None) == 0    # side by side
    torch.cuda.synchronize()
    assert cache.error_poll() == 0


def _fill(ff, batch, m, heads, kv, d, n, lengths, seed, moving):
    """A cache whose blocks of 64 rows have very different magnitudes (of V: and so of the output's unit) and rising keys."""
    rng = np.random.default_rng(seed)
    cache, ref = make(ff, batch, m + 5, heads, kv, d, max_tokens=n)
    k, v = rng.standard_normal((batch, m, kv, d)), rng.standard_normal((batch, m, kv, d))
    if moving:
        block = np.arange(m) // 64
        v *= 2.0 ** rng.integers(-18, 19, block[-1] + 1)[block][None, :, None, None]
        k *= (0.2 + 3.0 * np.arange(m) / m)[None, :, None, None]
    kt, k64 = bf16(k)
    vt, v64 = bf16(v)
    cache.append(0, kt, vt, counts=i32(lengths))
    ref.append(k64, v64, None, lengths)
    return cache, ref, rng


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [32, 33, 100, 127, 128, 129, 256, 257])
@pytest.mark.parametrize("moving", [False, True])
def test_numbers_of_rows_around_the_forms(ff, d, rows, moving):
    """One query row a token, and sequences of 0 to 11 key tiles, whole and ragged."""
    lengths = [0, 1, 127, 128, 129, 256, 300, 640, 1399]
    cache, ref, rng = _fill(ff, len(lengths), 1399, 2, 2, d, rows, lengths, rows, moving)
    q = rng.standard_normal((len(lengths), rows, 2, d))
    check_attn(cache, ref, q, weigh=True)
    counts = [rows, 1, rows, 0, rows - 5, 31, rows, rows, rows - 1]
    check_attn(cache, ref, q, causal=True, counts=counts, weigh=True)


@pytest.mark.parametrize("batch, n, heads, kv, m", [
    (70, 20, 4, 2, 700),    # 420 items of 256 keys, one tile of rows each
    (33, 40, 12, 2, 300),   # two tiles, one of them ragged
    (1, 70, 8, 1, 20000),   # cut into ranges of rows
    (3, 300, 6, 1, 400),    # fewer items than run at once, many tiles
])
@pytest.mark.parametrize("causal", [False, True])
def test_weights_of_more_items_than_run_at_once(ff, batch, n, heads, kv, m, causal):
    lengths = np.random.default_rng(m).integers(0, m + 1, batch)
    lengths[0] = m
    counts = np.random.default_rng(n).integers(0, n + 1, batch)
    counts[0] = n
    if batch > 1:
        counts[1] = 0
    cache, ref, rng = _fill(ff, batch, m, heads, kv, 64, n, lengths.tolist(), n, False)
    q = rng.standard_normal((batch, n, heads, 64))
    check_attn(cache, ref, q, causal=causal, counts=counts.tolist(), weigh=True)
    a, b = torch.zeros((batch, kv, m + 5), device="cuda"), torch.zeros((batch, kv, m + 5), device="cuda")
    qt, _ = bf16(q)
    out = torch.empty_like(qt)
    for w in (a, b):  # a call repeated gives the same bits
        cache.attn(0, qt, out, causal=causal, counts=i32(counts.tolist()), weights=w)
    assert torch.equal(a, b)
