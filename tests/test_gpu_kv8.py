"""The 8-bit cache on the GPU against the 64-bit reference: stored rows and kept rows exactly, attention and weights
within bounds that are derived in kv8_ref."""
import ctypes

import numpy as np
import pytest

from tests import kv8_ref
from tests.kv8_ref import BLOCK, RefCache, lse_tol, out_tol

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ff():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_attention_ff_gb300 import build, ff as ffmod
    build.build()
    return ffmod


def bf16(x):
    """float array -> (bf16 CUDA tensor, its values in 64 bits)."""
    t = torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def host(t):
    return t.detach().double().cpu().numpy()


def make(ff, batch, capacity, heads, kv_heads, d, max_tokens=64, n_layers=1):
    c = ff.KV8Cache(batch=batch, capacity=capacity, heads=heads, kv_heads=kv_heads, head_dim=d, max_tokens=max_tokens,
                    n_layers=n_layers)
    return c, RefCache(batch, capacity, kv_heads, d)


def check_cache(cache, ref, layer=0):
    """Lengths, codes, scales and read-back of the held rows, exactly."""
    k8, v8, ks, vs, lengths = cache.layer(layer)
    assert lengths.tolist() == ref.length.tolist()
    for x, codes, scales in (("k", k8, ks), ("v", v8, vs)):
        val = host(codes.clone().view(torch.float8_e4m3fn))
        val = val.transpose(0, 1, 3, 2, 4).reshape(ref.batch, -1, ref.kv_heads, ref.d)
        for b in range(ref.batch):
            n = int(ref.length[b])
            t = -(-n // BLOCK)
            assert np.array_equal(host(scales)[b, :t], np.ldexp(1.0, ref.e[x][b, :t])), (x, b)
            assert np.array_equal(val[b, :n], ref.code[x][b, :n], equal_nan=True), (x, b)
    n = max(1, int(ref.length.max()))
    shape = (ref.batch, n, ref.kv_heads, ref.d)
    k = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, 7.0)
    cache.load(layer, k, v)
    rk, rv = ref.load(n)
    assert np.array_equal(host(k), rk, equal_nan=True) and np.array_equal(host(v), rv, equal_nan=True)


def check_attn(cache, ref, q, layer=0, causal=False, counts=None, weigh=False, seed=0):
    qt, q64 = bf16(q)
    out = torch.full_like(qt, 3.0)
    lse = torch.full(q.shape[:3], 3.0, device="cuda")
    rng = np.random.default_rng(seed)
    w_in = w = wt = None
    if weigh:
        w_in = rng.random((ref.batch, ref.kv_heads, ref.capacity)).astype(np.float32)
        wt = torch.full(w_in.shape, 3.0, device="cuda")
        w = torch.from_numpy(w_in).cuda()
    cache.attn(layer, qt, out, causal=causal, counts=i32(counts), lse=lse, weights=wt, weights_in=w)
    torch.cuda.synchronize()
    assert cache.error_poll() == 0
    ro, rl, rw, (spread, mag, wtol) = ref.attn(q64, causal, counts, w_in)
    o, l = host(out), host(lse)
    written = ~np.isnan(rl)
    assert np.all(o[~written] == 3.0) and np.all(l[~written] == 3.0)  # left as they were
    n_keys = int(ref.length.max())
    ro0 = np.where(np.isnan(ro), 3.0, ro)
    err, tol = np.abs(o - ro0), out_tol(ro0, spread, mag, ref.d, n_keys)
    assert np.all(err <= tol + 1e-30), (err.max(), (err - tol).max())
    empty = written & np.isinf(rl)
    assert np.all(o[empty] == 0.0) and np.all(np.isneginf(l[empty]))
    some = written & ~empty
    # the fp32 result itself: half a step of it
    assert np.all(np.abs(l[some] - rl[some]) <= lse_tol(mag[some], ref.d) + np.abs(rl[some]) * 2.0 ** -24)
    if weigh:
        got = host(wt)
        for b in range(ref.batch):
            n = int(ref.length[b])
            assert np.all(got[b, :, n:] == 3.0)
            assert np.all(np.abs(got[b, :, :n] - rw[b, :, :n]) <= wtol[b, :, :n] + 2.0 ** -23 * rw[b, :, :n])
    return o


# ------------------------------------------------------------------- storing


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch, kv_heads, capacity, runs", [
    (1, 1, 64, [1]),
    (1, 2, 100, [63, 1, 1, 35]),            # ends a block, starts one, stops at an odd capacity
    (2, 3, 300, [1, 1, 130, 64, 5]),
    (3, 1, 257, [257]),
    (1, 5, 1000, [500, 17, 200]),
])
def test_append_matches_the_reference(ff, d, batch, kv_heads, capacity, runs):
    rng = np.random.default_rng(d + capacity)
    cache, ref = make(ff, batch, capacity, kv_heads, kv_heads, d)
    for i, n in enumerate(runs):
        # later runs are louder, so that a block's scale grows under rows that it holds
        k, k64 = bf16(rng.standard_normal((batch, n, kv_heads, d)) * 3.0 ** i)
        v, v64 = bf16(rng.standard_normal((batch, n, kv_heads, d)) * 0.2 ** i)
        cache.append(0, k, v)
        ref.append(k64, v64)
        check_cache(cache, ref)
    assert cache.error_poll() == 0


def test_append_at_a_start_and_padded(ff):
    rng = np.random.default_rng(5)
    cache, ref = make(ff, 4, 200, 2, 2, 64)
    for start, counts in ((None, [70, 0, 33, 64]), ([10, 0, 33, 63], [70, 5, 0, 1]), ([500, -3, 20, 64], None),
                          (None, [-1, 99, 40, 0])):
        k, k64 = bf16(rng.standard_normal((4, 70, 2, 64)) * rng.choice([0.1, 1.0, 30.0]))
        v, v64 = bf16(rng.standard_normal((4, 70, 2, 64)))
        cache.append(0, k, v, start=i32(start), counts=i32(counts))
        ref.append(k64, v64, start, counts)
        check_cache(cache, ref)
    assert cache.error_poll() == 0


def test_append_twice_at_one_start_gives_the_same_bits(ff):
    # a chunk denoised again is stored again
    rng = np.random.default_rng(6)
    cache, _ = make(ff, 2, 200, 2, 2, 128)
    cache.append(0, bf16(rng.standard_normal((2, 50, 2, 128)))[0], bf16(rng.standard_normal((2, 50, 2, 128)))[0])
    k, v = bf16(20 * rng.standard_normal((2, 90, 2, 128)))[0], bf16(rng.standard_normal((2, 90, 2, 128)))[0]
    got = []
    for _ in range(2):
        cache.append(0, k, v, start=i32([50, 50]))
        got.append([x.clone() for x in cache.layer(0)])
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("d", [64, 128])
def test_append_of_special_values(ff, d):
    x = np.zeros((1, 320, 1, d), np.float32)
    x[0, 0:64] = np.random.default_rng(0).standard_normal((64, 1, d))
    x[0, 3, 0, 5], x[0, 4, 0, 6], x[0, 5, 0, 7] = np.inf, -np.inf, np.nan
    x[0, 64:128] = 0.0                      # nothing at all
    x[0, 128:192] = 2.0 ** -130             # subnormal bf16, below the least scale
    x[0, 192:256] = 3e38                    # above what the largest scale holds
    x[0, 256:320] = np.linspace(0, 448, 64)[:, None, None]  # ties and the type's own largest value
    cache, ref = make(ff, 1, 320, 1, 1, d)
    k, k64 = bf16(x)
    v, v64 = bf16(x[:, ::-1].copy())
    cache.append(0, k, v)
    with np.errstate(over="ignore"):
        ref.append(k64, v64)
    check_cache(cache, ref)


def test_rows_behind_the_new_ones_stay(ff):
    cache, _ = make(ff, 1, 128, 1, 1, 64)
    k8, v8 = cache.layer(0)[:2]
    k8.fill_(17)
    v8.fill_(18)
    one = torch.ones((1, 3, 1, 64), dtype=torch.bfloat16, device="cuda")
    cache.append(0, one, one)
    assert torch.all(k8[0, 0, 0, 3:] == 17) and torch.all(v8[0, 0, 0, 3:] == 18)
    assert torch.all(k8[0, 1] == 17) and torch.all(k8[0, 0, 0, :3] != 17)


def test_rows_past_the_capacity_are_dropped_and_reported(ff):
    rng = np.random.default_rng(8)
    cache, ref = make(ff, 2, 100, 1, 1, 64)
    for counts in ([90, 20], [20, 20]):
        k, k64 = bf16(rng.standard_normal((2, 90, 1, 64)))
        cache.append(0, k, k, counts=i32(counts))
        ref.append(k64, k64, None, counts)
        check_cache(cache, ref)
    assert ref.length.tolist() == [100, 40]
    assert ff.STATUS[cache.error_poll()] == "FF_ERR_CAPACITY"
    assert cache.error_poll() == 0


def test_load_from_a_start(ff):
    rng = np.random.default_rng(9)
    cache, ref = make(ff, 3, 200, 3, 3, 64)
    k, k64 = bf16(rng.standard_normal((3, 150, 3, 64)))
    cache.append(0, k, k, counts=i32([150, 7, 0]))
    ref.append(k64, k64, None, [150, 7, 0])
    for n, start in ((1, [149, 6, 0]), (70, [100, -5, 3]), (500, None), (9, [2 ** 31 - 5, -2 ** 31, 63])):
        out = [torch.full((3, n, 3, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        cache.load(0, *out, start=i32(start))
        for got, want in zip(out, ref.load(n, start)):
            assert np.array_equal(host(got), want)


# ------------------------------------------------------------------ attention

ATTN = [
    # batch, n, heads, kv_heads, lengths, counts, causal
    (1, 1, 1, 1, [1], None, True),
    (1, 1, 2, 2, [63], None, False),
    (2, 1, 4, 2, [64, 65], None, True),
    (3, 1, 5, 1, [0, 129, 1000], None, True),
    (4, 3, 6, 2, [3, 0, 2, 700], [3, 3, 3, 1], True),       # more queries than rows: some see nothing
    (2, 5, 16, 2, [333, 31], [5, 0], False),
    (1, 16, 1, 1, [257], None, True),
    (1, 17, 2, 1, [300], None, True),                       # 34 rows
    (2, 7, 9, 3, [90, 4097], None, False),
    (1, 40, 3, 3, [40], None, True),
    (1, 130, 2, 1, [513], None, True),                      # 260 rows: more than a tile of 256
    (2, 150, 3, 3, [640, 200], [150, 33], False),
    (1, 300, 1, 1, [300], None, True),
    (3, 100, 4, 2, [100, 50, 0], [100, 100, 20], True),
    (1, 129, 7, 1, [200], None, False),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention_matches_the_reference(ff, d, case):
    batch, n, heads, kv_heads, lengths, counts, causal = ATTN[case]
    rng = np.random.default_rng(100 * case + d)
    cap = max(max(lengths), 1) + 29
    cache, ref = make(ff, batch, cap, heads, kv_heads, d, max_tokens=n)
    # what lies behind the rows held must not matter: NaN codes, and scales as large as they come
    k8, v8, ks, vs, _ = cache.layer(0)
    k8.fill_(0x7f)
    v8.fill_(0xff)
    ks.fill_(2.0 ** 112)
    vs.fill_(2.0 ** 112)
    m = max(max(lengths), 1)
    k, k64 = bf16(rng.standard_normal((batch, m, kv_heads, d)) * rng.choice([0.3, 1.0, 2.0], (kv_heads, d)))
    v, v64 = bf16(rng.standard_normal((batch, m, kv_heads, d)) * np.exp(rng.standard_normal((batch, m, 1, 1))))
    cache.append(0, k, v, counts=i32(lengths))
    ref.append(k64, v64, None, lengths)
    q = rng.standard_normal((batch, n, heads, d)) * 1.5
    check_attn(cache, ref, q, causal=causal, counts=counts, weigh=case % 2 == 0, seed=case)
    check_attn(cache, ref, q, causal=causal, counts=counts, weigh=case % 2 == 1, seed=case)


@pytest.mark.parametrize("n", [1, 200])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_over_blocks_of_very_different_scales(ff, d, n):
    rng = np.random.default_rng(d + n)
    length = 700
    cache, ref = make(ff, 1, length, 2, 1, d, max_tokens=n)
    loud = np.repeat(rng.choice([-6.0, -2.0, 0.0, 3.0, 6.0], 11), 64)[:length]
    k, k64 = bf16(rng.standard_normal((1, length, 1, d)) * 2.0 ** (loud / 6)[None, :, None, None])
    v, v64 = bf16(rng.standard_normal((1, length, 1, d)) * 2.0 ** loud[None, :, None, None])
    cache.append(0, k, v)
    ref.append(k64, v64)
    check_attn(cache, ref, rng.standard_normal((1, n, 2, d)), weigh=True)


@pytest.mark.parametrize("n", [1, 200])
@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1.0, 1e4, 1e30])
def test_attention_of_queries_of_any_size(ff, n, scale):
    # a query's size is matched by the keys', so that the scores stay those of a model
    rng = np.random.default_rng(1)
    cache, ref = make(ff, 1, 300, 2, 2, 64, max_tokens=n)
    k, k64 = bf16(rng.standard_normal((1, 300, 2, 64)) * (1.0 / scale if 1e-20 < scale < 1e20 else 1.0))
    v, v64 = bf16(rng.standard_normal((1, 300, 2, 64)))
    cache.append(0, k, v)
    ref.append(k64, v64)
    q = rng.standard_normal((1, n, 2, 64)) * (scale if scale < 1e20 else 1.0)
    q[0, 0, 0, 0] = 0.0
    check_attn(cache, ref, q, weigh=True)


@pytest.mark.parametrize("n", [1, 200])
def test_one_key_far_above_the_others(ff, n):
    rng = np.random.default_rng(2)
    cache, ref = make(ff, 1, 500, 1, 1, 128, max_tokens=n)
    x = rng.standard_normal((1, 500, 1, 128))
    x[0, 311] *= 20
    k, k64 = bf16(x)
    v, v64 = bf16(rng.standard_normal((1, 500, 1, 128)))
    cache.append(0, k, v)
    ref.append(k64, v64)
    q = np.repeat(x[:, 311:312] * 0.4, n, axis=1)
    check_attn(cache, ref, q, weigh=True)


@pytest.mark.parametrize("n", [1, 150])
def test_not_a_number_stays_in_its_row(ff, n):
    rng = np.random.default_rng(3)
    cache, ref = make(ff, 2, 200, 2, 2, 64, max_tokens=n)
    x = rng.standard_normal((2, 200, 2, 64))
    k, k64 = bf16(x)
    cache.append(0, k, k)
    ref.append(k64, k64)
    q = rng.standard_normal((2, n, 2, 64))
    qt, _ = bf16(q)
    bad = qt.clone()
    bad[0, n - 1, 1, 3] = float("nan")
    outs = []
    for t in (qt, bad):
        out = torch.zeros_like(t)
        cache.attn(0, t, out)
        outs.append(host(out))
    assert np.all(np.isnan(outs[1][0, n - 1, 1]))
    outs[1][0, n - 1, 1] = outs[0][0, n - 1, 1]
    assert np.array_equal(outs[0], outs[1])


@pytest.mark.parametrize("n, heads, kv_heads, length", [(1, 8, 2, 9000), (3, 2, 2, 20000), (260, 4, 4, 5000)])
def test_a_call_repeated_gives_the_same_bits(ff, n, heads, kv_heads, length):
    rng = np.random.default_rng(4)
    cache, _ = make(ff, 2, length, heads, kv_heads, 128, max_tokens=n)
    k = torch.randn((2, length, kv_heads, 128), device="cuda").to(torch.bfloat16)
    cache.append(0, k, k.flip(1).contiguous(), counts=i32([length, length // 3]))
    q, _ = bf16(rng.standard_normal((2, n, heads, 128)))
    got = []
    for _ in range(3):
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
        w = torch.zeros((2, kv_heads, length), device="cuda")
        cache.attn(0, q, out, causal=True, lse=lse, weights=w)
        got.append((out, lse, w))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_weights_of_a_long_context_sum_to_the_queries(ff):
    n, heads, kv_heads, length = 33, 8, 2, 31200
    cache, _ = make(ff, 1, length, heads, kv_heads, 128, max_tokens=n)
    k = torch.randn((1, length, kv_heads, 128), device="cuda").to(torch.bfloat16)
    cache.append(0, k, k)
    q = torch.randn((1, n, heads, 128), device="cuda").to(torch.bfloat16)
    w = torch.zeros((1, kv_heads, length), device="cuda")
    for turns in (1, 2):  # accumulates in place
        cache.attn(0, q, torch.zeros_like(q), weights=w)
        total = host(w).sum(-1)
        # every probability is off by 2^-16 at most (scores of magnitude below 64)
        assert np.all(np.abs(total - turns * n * heads / kv_heads) <= turns * n * heads / kv_heads * 2.0 ** -10)


# ------------------------------------------------------------------- eviction


def check_evict(cache, ref, dst, dref, weights, n_keep, n_recent):
    wt = torch.from_numpy(np.asarray(weights, np.float32)).cuda()
    wout = torch.full((ref.batch, ref.kv_heads, dst.capacity), 9.0, device="cuda")
    kept = torch.full((ref.batch, ref.kv_heads, n_keep), 9, dtype=torch.int32, device="cuda")
    cache.evict(0, dst, 0, n_keep, n_recent, wt, wout, kept)
    rk, rw = ref.evict(np.asarray(weights, np.float32), n_keep, n_recent, dref)
    assert np.array_equal(kept.cpu().numpy(), rk)
    assert np.array_equal(host(wout), rw, equal_nan=True)
    check_cache(dst, dref)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths, n_keep, n_recent, kind", [
    ([0, 1, 2], 1, 0, "random"),
    ([200, 64, 5], 64, 10, "random"),
    ([200, 150, 199], 100, 100, "random"),      # the recent rows are the budget
    ([200, 150, 199], 130, 0, "ties"),
    ([200, 150, 199], 65, 1, "equal"),
    ([200, 150, 199], 65, 3, "special"),
    ([200, 150, 199], 200, 7, "random"),        # everything stays
    ([5000, 1025, 3000], 1024, 50, "ties"),
    ([9000, 8191, 2048], 4097, 1, "negative"),
])
def test_eviction_matches_the_reference(ff, d, lengths, n_keep, n_recent, kind):
    rng = np.random.default_rng(d + n_keep)
    m = max(lengths)
    cache, ref = make(ff, 3, m + 5, 2, 2, d)
    dst, dref = make(ff, 3, n_keep + 3, 4, 2, d)
    x = rng.standard_normal((3, m, 2, d)) * np.exp2(rng.integers(-4, 5, (3, m, 1, 1)) * (rng.random((3, m, 1, 1)) < 0.02))
    k, k64 = bf16(x)
    cache.append(0, k, k, counts=i32(lengths))
    ref.append(k64, k64, None, lengths)
    w = rng.random((3, 2, m + 5))
    if kind == "ties":
        w = rng.integers(0, 4, w.shape) / 4.0
    elif kind == "equal":
        w = np.full_like(w, 0.25)
    elif kind == "special":
        w = rng.choice([0.0, -0.0, np.inf, -np.inf, np.nan, 1.0, 1e-42, -1e-42], w.shape)
    elif kind == "negative":
        w = rng.standard_normal(w.shape) * 10.0 ** rng.integers(-30, 30, w.shape)
    check_evict(cache, ref, dst, dref, w.astype(np.float32), n_keep, n_recent)


def test_eviction_between_layers_of_one_handle(ff):
    rng = np.random.default_rng(11)
    cache, ref = make(ff, 2, 300, 2, 2, 64, n_layers=2)
    k, k64 = bf16(rng.standard_normal((2, 300, 2, 64)))
    cache.append(0, k, k)
    ref.append(k64, k64)
    w = torch.rand((2, 2, 300), device="cuda")
    wout, kept = torch.zeros_like(w), torch.zeros((2, 2, 90), dtype=torch.int32, device="cuda")
    cache.evict(0, cache, 1, 90, 20, w, wout, kept)
    dref = RefCache(2, 300, 2, 64)
    rk, rw = ref.evict(w.cpu().numpy(), 90, 20, dref)
    assert np.array_equal(kept.cpu().numpy(), rk) and np.array_equal(host(wout), rw)
    check_cache(cache, dref, layer=1)
    check_cache(cache, ref, layer=0)


# ---------------------------------------------------------------- together


@pytest.mark.parametrize("n", [1, 48])
def test_rollout_that_stays_at_a_budget(ff, n):
    """Append, attend with weights, evict, go on: as a long rollout uses them together."""
    rng = np.random.default_rng(n)
    budget, recent, heads, kv_heads, d = 150, 20, 4, 2, 64
    cap = budget + 3 * n
    cache, ref = make(ff, 2, cap, heads, kv_heads, d, max_tokens=n, n_layers=2)
    layer = 0
    w = torch.zeros((2, kv_heads, cap), device="cuda")
    for step in range(8):
        for _ in range(3):
            k, k64 = bf16(rng.standard_normal((2, n, kv_heads, d)))
            v, v64 = bf16(rng.standard_normal((2, n, kv_heads, d)))
            q, q64 = bf16(rng.standard_normal((2, n, heads, d)))
            out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
            before = host(w)
            cache.append(layer, k, v)
            cache.attn(layer, q, out, causal=True, lse=lse, weights=w)
            ref.append(k64, v64)
            ro, rl, rw, (spread, mag, wtol) = ref.attn(q64, True, None, before)
            assert np.all(np.abs(host(out) - ro) <= out_tol(ro, spread, mag, d, cap))
            assert np.all(np.abs(host(lse) - rl) <= lse_tol(mag, d) + np.abs(rl) * 2.0 ** -24)
            for b in range(2):
                m = int(ref.length[b])
                assert np.all(np.abs(host(w) - rw)[b, :, :m] <= wtol[b, :, :m] + 2.0 ** -23 * rw[b, :, :m])
        dref = RefCache(2, cap, kv_heads, d)
        keep = min(budget, cap)
        wout = torch.zeros_like(w)
        kept = torch.zeros((2, kv_heads, keep), dtype=torch.int32, device="cuda")
        cache.evict(layer, cache, 1 - layer, keep, recent, w, wout, kept)
        rk, rw = ref.evict(w.cpu().numpy(), keep, recent, dref)
        assert np.array_equal(kept.cpu().numpy(), rk) and np.array_equal(host(wout), rw)
        layer, ref, w = 1 - layer, dref, wout
        check_cache(cache, ref, layer)
    assert cache.error_poll() == 0


def test_loaded_rows_feed_the_framework_attention(ff):
    """A chunk over a cache gives what ff_attention_noalloc gives over the rows read back."""
    cache, _ = make(ff, 1, 700, 3, 3, 128, max_tokens=260)
    k = torch.randn((1, 700, 3, 128), device="cuda").to(torch.bfloat16)
    v = torch.randn_like(k)
    cache.append(0, k, v)
    q = torch.randn((1, 260, 3, 128), device="cuda").to(torch.bfloat16)
    out, other = torch.empty_like(q), torch.empty_like(q[0])
    cache.attn(0, q, out)
    kk, vv = torch.empty_like(k), torch.empty_like(v)
    cache.load(0, kk, vv)
    ff.attention_noalloc(q[0], kk[0], vv[0], other)
    # two roundings to bf16 (2^-8 each), and the other's probabilities in bf16
    spread = float(vv.abs().max())
    assert float((out[0].float() - other.float()).abs().max()) <= 3 * 2.0 ** -8 * spread


@pytest.mark.parametrize("n", [1, 70])
def test_captured_steps_follow_the_lengths(ff, n):
    rng = np.random.default_rng(20 + n)
    heads, kv_heads, d, cap = 4, 2, 64, 600
    cache, ref = make(ff, 2, cap, heads, kv_heads, d, max_tokens=n)
    shape = (2, n, kv_heads, d)
    k, v = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((2, n, heads, d), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
    w = torch.zeros((2, kv_heads, cap), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(0, k, v)
        cache.attn(0, q, out, causal=True, lse=lse, weights=w)
    assert cache.lengths(0).tolist() == [0, 0]
    for step in range(8):
        a, k64 = bf16(rng.standard_normal(shape))
        c, v64 = bf16(rng.standard_normal(shape))
        e, q64 = bf16(rng.standard_normal(q.shape))
        k.copy_(a), v.copy_(c), q.copy_(e)
        before = host(w)
        graph.replay()
        ref.append(k64, v64)
        ro, rl, rw, (spread, mag, wtol) = ref.attn(q64, True, None, before)
        assert np.all(np.abs(host(out) - ro) <= out_tol(ro, spread, mag, d, cap))
        for b in range(2):
            m = int(ref.length[b])
            assert np.all(np.abs(host(w) - rw)[b, :, :m] <= wtol[b, :, :m] + 2.0 ** -23 * rw[b, :, :m])
    check_cache(cache, ref)
    # calls outside the graph go on from there
    torch.cuda.synchronize()
    cache.append(0, k[:, :1].contiguous(), v[:, :1].contiguous())
    assert cache.lengths(0).tolist() == [8 * n + 1] * 2


def test_calls_on_other_streams_are_ordered(ff):
    rng = np.random.default_rng(30)
    cache, ref = make(ff, 1, 4000, 2, 2, 128, max_tokens=4)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    data = [bf16(rng.standard_normal((1, 400, 2, 128))) for _ in range(10)]
    q, q64 = bf16(rng.standard_normal((1, 4, 2, 128)))
    out = [torch.zeros_like(q) for _ in range(10)]
    torch.cuda.synchronize()
    for i, (k, _) in enumerate(data):
        cache.append(0, k, k, stream=s1)
        cache.attn(0, q, out[i], stream=s2)
    torch.cuda.synchronize()
    for i, (_, k64) in enumerate(data):
        ref.append(k64, k64)
        ro, _, _, (spread, mag, _) = ref.attn(q64)
        assert np.all(np.abs(host(out[i]) - ro) <= out_tol(ro, spread, mag, 128, 4000)), i
    check_cache(cache, ref)


# ------------------------------------------------------------------ refusals


def test_refusals(ff):
    cache, _ = make(ff, 2, 100, 4, 2, 64, max_tokens=8, n_layers=2)
    other, _ = make(ff, 2, 50, 4, 2, 64)
    lib, h, o = ff.lib(), cache.handle, other.handle
    kv = torch.zeros((2, 101, 2, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 9, 4, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    w, w2 = torch.zeros((2, 2, 100), device="cuda"), torch.zeros((2, 2, 100), device="cuda")
    kept = torch.zeros((2, 2, 100), dtype=torch.int32, device="cuda")
    P = lambda t, off=0: ctypes.c_void_p(t.data_ptr() + off)
    arg = 1
    assert lib.ff_kv8_append(h, 0, 0, P(kv), P(kv), None, None, None) == arg        # no rows
    assert lib.ff_kv8_append(h, 0, 101, P(kv), P(kv), None, None, None) == arg      # more than the capacity
    assert lib.ff_kv8_append(h, 2, 1, P(kv), P(kv), None, None, None) == arg        # no such layer
    assert lib.ff_kv8_append(h, -1, 1, P(kv), P(kv), None, None, None) == arg
    assert lib.ff_kv8_append(h, 0, 1, P(kv, 2), P(kv), None, None, None) == arg     # alignment
    assert lib.ff_kv8_append(h, 0, 1, None, P(kv), None, None, None) == arg
    assert lib.ff_kv8_load(h, 0, 0, None, P(kv), P(kv), None) == arg
    assert lib.ff_kv8_load(h, 0, 1 << 30, None, P(kv), P(kv), None) == arg
    assert lib.ff_kv8_attn(h, 0, 9, P(q), None, 0, P(out), None, None, None, None) == arg   # > max_tokens
    assert lib.ff_kv8_attn(h, 0, 0, P(q), None, 0, P(out), None, None, None, None) == arg
    assert lib.ff_kv8_attn(h, 0, 1, P(q), None, 2, P(out), None, None, None, None) == arg
    assert lib.ff_kv8_attn(h, 0, 1, P(q), None, 0, P(q), None, None, None, None) == arg     # out over q
    assert lib.ff_kv8_attn(h, 0, 1, P(q), None, 0, P(out), None, P(w), None, None) == arg   # weights_in alone
    assert lib.ff_kv8_evict(h, 0, h, 0, 10, 1, P(w), P(w2), P(kept), None) == arg           # onto itself
    assert lib.ff_kv8_evict(h, 0, o, 0, 51, 1, P(w), P(w2), P(kept), None) == arg           # over dst's capacity
    assert lib.ff_kv8_evict(h, 0, h, 1, 10, 11, P(w), P(w2), P(kept), None) == arg
    assert lib.ff_kv8_evict(h, 0, h, 1, 10, -1, P(w), P(w2), P(kept), None) == arg
    assert lib.ff_kv8_evict(h, 0, h, 1, 10, 1, P(w), P(w), P(kept), None) == arg            # weights_out over weights
    with pytest.raises(TypeError):
        cache.append(0, kv[:, :4].float(), kv[:, :4])
    with pytest.raises(TypeError):
        cache.attn(0, q[:, :4], out)                                                        # not contiguous
    with pytest.raises(ValueError):
        cache.append(0, kv[:, :4].contiguous(), kv[:, :5].contiguous())
    with pytest.raises(TypeError):
        cache.append(0, kv[:, :4].contiguous(), kv[:, :4].contiguous(), start=torch.zeros(2, device="cuda"))
    with pytest.raises(ff.FFError):
        cache.evict(0, cache, 0, 10, 1, w, w2, kept[..., :10].contiguous())
    big, _ = make(ff, 2, 100, 4, 4, 64)
    with pytest.raises(ff.FFError):
        cache.evict(0, big, 0, 10, 1, w, w2, kept[..., :10].contiguous())                   # other heads
    torch.cuda.synchronize()
    assert cache.lengths(0).tolist() == [0, 0] and cache.error_poll() == 0
    with pytest.raises(ff.FFError) as e:
        ff.KV8Cache(batch=1, capacity=1000, max_bytes=1000)
    assert e.value.code == "FF_ERR_OOM"


def test_views_keep_their_memory(ff):
    lengths = make(ff, 2, 100, 2, 2, 64)[0].lengths(0)  # the cache itself is let go
    import gc
    gc.collect()
    assert lengths.tolist() == [0, 0]


def test_current_device_and_sizes(ff):
    cache, _ = make(ff, 3, 130, 2, 2, 64, n_layers=4)
    k8, v8, ks, vs, lengths = cache.layer(3)
    assert k8.shape == (3, 3, 2, 64, 64) and ks.shape == (3, 3, 2) and lengths.shape == (3,)
    assert cache.bytes() >= 4 * 2 * k8.numel()
    assert torch.cuda.current_device() == 0
