"""Attention over blocks of V whose scales lie far apart: a query's result follows the scales of what it sees, and of
that only as far as it gives weight, in every form of the kernel (rows of a kv head: 1 to 32, to 128, more; whole
units and key ranges)."""
import numpy as np
import pytest

from tests.kv8_ref import BLOCK, RefCache, out_tol
from tests.test_gpu_kv8 import bf16, host, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROWS = [1, 8, 9, 25, 32, 33, 100, 128, 129, 300]


@pytest.fixture(scope="module")
def ff():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_attention_ff_gb300 import build, ff as ffmod
    build.build()
    return ffmod


def small_tol(ref, q64, causal):
    """What probabilities below f16's normal range add to out_tol.  A probability p_j is held as p_j * 2^(e_j + 5 - R) with
    2^e_j its block's scale and 2^R the output's unit, which is at most max_i p_i * 2^e_i over the keys that the row sees
    (the largest p so far counts as 1; all later rescaling is common).  Below the normal range it is off by at most half of
    2^-24, and it multiplies a code: 2^-25 * 2^(R - 5) * |code_j| each."""
    batch, n, heads, d = q64.shape
    group = heads // ref.kv_heads
    tol = np.zeros(q64.shape)
    for b in range(batch):
        length = int(ref.length[b])
        for h in range(ref.kv_heads):
            k, code = ref.values("k", b, h), np.abs(ref.code["v"][b, :length, h])
            e = np.repeat(ref.e["v"][b, :, h], BLOCK)[:length]
            sums = np.cumsum(code, 0)
            for g in range(h * group, (h + 1) * group):
                for i in range(n):
                    seen = max(0, length - n + i + 1) if causal else length
                    if seen:
                        s = k[:seen] @ q64[b, i, g] / np.sqrt(d)
                        lse = s.max() + np.log(np.exp(s - s.max()).sum())
                        level = ((s - lse) / np.log(2.0) + e[:seen]).max()
                        tol[b, i, g] = 2.0 ** (level - 30) * sums[seen - 1]
    return tol


def check(cache, ref, q, causal):
    """Output of the call, within the bounds of kv8_ref and of small_tol."""
    qt, q64 = bf16(q)
    out = torch.full_like(qt, 3.0)
    cache.attn(0, qt, out, causal=causal)
    torch.cuda.synchronize()
    assert cache.error_poll() == 0
    want, _, _, (spread, mag, _) = ref.attn(q64, causal)
    got = host(out)
    tol = out_tol(want, spread, mag, ref.d, int(ref.length.max())) + small_tol(ref, q64, causal)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0].tolist(), got[bad][0], want[bad][0], tol[bad][0])
    return out


def fill(ff, rng, rows, length, d, exps, shifts=None, spare=0):
    """A cache of one kv head: block b's V is N(0, 1) * 2^exps[b]; its keys are given shifts[b] less (log2) by a query
    of queries()."""
    cache, ref = make(ff, 1, length + spare, 1, 1, d, max_tokens=rows)
    block = np.arange(length) // BLOCK
    k = 0.5 * rng.standard_normal((1, length, 1, d))
    if shifts is not None:
        k -= (np.asarray(shifts, float)[block] * np.log(2.0) / (2.0 * np.sqrt(d)))[None, :, None, None]
    v = rng.standard_normal((1, length, 1, d)) * np.ldexp(1.0, np.asarray(exps)[block])[None, :, None, None]
    kt, k64 = bf16(k)
    vt, v64 = bf16(v)
    cache.append(0, kt, vt)
    ref.append(k64, v64)
    return cache, ref


def queries(rng, rows, d):
    return 2.0 + 0.5 * rng.standard_normal((1, rows, 1, d))


def stored_rows(rows):
    """Of a causal call: the first query sees 41 rows."""
    return rows + 40


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ratio", [20, 28, 40, 70, 100])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("spare", [0, 4000])
def test_a_louder_block_behind_what_a_query_sees(ff, rows, ratio, d, spare):
    rng = np.random.default_rng(1000 * rows + ratio + d)
    length = stored_rows(rows)
    for blocks in ([0, ratio], [0, ratio, -ratio // 2, 2]):
        exps = [blocks[b % len(blocks)] for b in range(-(-length // BLOCK))]
        cache, ref = fill(ff, rng, rows, length, d, exps, spare=spare)
        check(cache, ref, queries(rng, rows, d), True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("low, high", [(-90, 60), (-60, 100), (-95, 110)])
def test_scales_from_end_to_end_of_the_range(ff, rows, low, high, d):
    rng = np.random.default_rng(rows + d)
    length = stored_rows(rows)
    exps = [(low, high)[b % 2] for b in range(-(-length // BLOCK))]
    cache, ref = fill(ff, rng, rows, length, d, exps)
    check(cache, ref, queries(rng, rows, d), True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("ratio", [20, 40, 70, 100])
@pytest.mark.parametrize("beside", [6, 20, 45])
def test_a_louder_block_that_gets_hardly_any_weight(ff, rows, ratio, beside, d):
    """What the loud block contributes lies 2^beside below the others (about: a query's noise moves it)."""
    rng = np.random.default_rng(7 * rows + ratio + beside + d)
    shift = ratio + beside
    for exps, shifts in (([ratio, 0], [shift, 0]), ([0, ratio], [0, shift]),
                         ([ratio, 0, 0, 0, 0, 0, 0], [shift, 0, 0, 0, 0, 0, 0]),
                         ([0, 0, ratio, 3, -3, ratio // 2, 0], [5, 0, shift, 0, 2, ratio // 2 + beside, 0])):
        cache, ref = fill(ff, rng, rows, BLOCK * len(exps) - 7, d, exps, shifts)
        check(cache, ref, queries(rng, rows, d), False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", ROWS)
def test_levels_that_rise_and_fall(ff, rows, d):
    """Scales and scores of every block anywhere: the quiet blocks' weights make up for it, or do not."""
    for seed in range(4):
        rng = np.random.default_rng(100 * seed + rows + d)
        length = 1400 - seed
        exps = rng.integers(-40, 41, 22)
        shifts = np.maximum(exps + 40 + rng.integers(-12, 30, 22), 0)
        cache, ref = fill(ff, rng, rows, length, d, exps, shifts, spare=3000 * (seed % 2))
        q = queries(rng, rows, d)
        check(cache, ref, q, False)
        check(cache, ref, q, True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", ROWS)
def test_a_block_of_zeros_beside_others(ff, rows, d):
    """Zeros have the least scale, 2^-96: before and behind blocks of any other, with all the weight and with none."""
    rng = np.random.default_rng(rows + d)
    for exps in ([0, -1, 0], [50, -1, 0], [0, 50, -1]):
        cache, ref = make(ff, 1, 192, 1, 1, d, max_tokens=rows)
        for where in range(3):
            v = rng.standard_normal((1, 192, 1, d)) * np.ldexp(1.0, np.repeat(exps, 64))[None, :, None, None]
            v[:, where * 64:where * 64 + 64] = 0.0
            for shift in (0.0, 3.0, -3.0):
                k = 0.5 * rng.standard_normal((1, 192, 1, d))
                k[:, where * 64:where * 64 + 64] += shift
                kt, k64 = bf16(k)
                vt, v64 = bf16(v)
                cache.append(0, kt, vt, start=torch.zeros(1, dtype=torch.int32, device="cuda"))
                ref.append(k64, v64, [0])
                check(cache, ref, queries(rng, rows, d), False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", ROWS)
def test_hidden_blocks_change_no_bit(ff, rows, d):
    """Queries that see nothing of the last blocks give the same bits whatever these hold."""
    if rows == 1:
        rows = 2  # the last query sees everything
    length = stored_rows(rows)
    last = (length - 1) // BLOCK * BLOCK             # the first row of the last block
    see = length - rows + 1 + np.arange(rows)        # rows that each query sees
    if not (see <= last).any():
        length = last + 1                            # one row in the last block
        see = length - rows + 1 + np.arange(rows)
    rng = np.random.default_rng(rows + d)
    k = rng.standard_normal((1, length, 1, d))
    v = rng.standard_normal((1, length, 1, d))
    q, _ = bf16(rng.standard_normal((1, rows, 1, d)))
    for base in (0, -90):
        got = []
        for ratio in (0, 25, 60, 100, 190 if base else 110):
            cache, _ = make(ff, 1, length, 1, 1, d, max_tokens=rows)
            x = v * 2.0 ** base
            x[:, last:] *= 2.0 ** ratio
            cache.append(0, bf16(k)[0], bf16(x)[0])
            out = torch.zeros_like(q)
            cache.attn(0, q, out, causal=True)
            assert cache.error_poll() == 0
            got.append(out[0, torch.from_numpy(see <= last).cuda()].view(torch.int16))
        assert got[0].numel() and all(torch.equal(got[0], x) for x in got[1:])


def test_a_row_gives_the_same_in_every_form(ff):
    """One query, asked alone and with 31, 99 and 299 others beside it: a result of the same accuracy."""
    rng = np.random.default_rng(1)
    exps, shifts = [60, 0, 2, 90, -3, 0, 30], [80, 0, 1, 95, 3, 0, 70]
    cache, ref = fill(ff, rng, 300, 440, 64, exps, shifts)
    q = queries(rng, 300, 64)
    alone = host(check(cache, ref, q[:, :1], False))
    for rows in (32, 100, 300):
        many = host(check(cache, ref, q[:, :rows], False))
        want, _, _, (spread, mag, _) = ref.attn(bf16(q[:, :1])[1])
        tol = out_tol(want, spread, mag, 64, 440) + small_tol(ref, bf16(q[:, :1])[1], False)
        assert np.all(np.abs(many[:, :1] - alone) <= 2 * tol)


# One query row to 32 go through warps that take every fourth run of 32 keys.  With this many heads nothing is cut, so a
# warp meets blocks b, b + 2, b + 4, ..: pairs of blocks, in the tests below, whose scales and scores each are its own.
MANY = 920


def fill_pairs(ff, rng, rows, length, exps, shifts):
    """As fill(), with MANY kv heads, which share the pattern of scales and shifts but no value."""
    cache, ref = make(ff, 1, length, MANY, MANY, 64, max_tokens=rows)
    pair = np.arange(length) // (2 * BLOCK)
    k = 0.5 * rng.standard_normal((1, length, MANY, 64))
    k -= (np.asarray(shifts, float)[pair] * np.log(2.0) / 16.0)[None, :, None, None]
    v = rng.standard_normal((1, length, MANY, 64)) * np.ldexp(1.0, np.asarray(exps)[pair])[None, :, None, None]
    kt, k64 = bf16(k)
    vt, v64 = bf16(v)
    cache.append(0, kt, vt)
    ref.append(k64, v64)
    return cache, ref


@pytest.mark.parametrize("rows", [1, 3, 9, 25])
@pytest.mark.parametrize("exps, shifts", [
    ([100, 0, 0], [120, 0, 0]),             # loud without weight, then what counts
    ([90, 0, 85, 3], [130, 0, 100, 0]),
    ([-90, 60, -95], [0, 0, 0]),            # from the quietest to loud: more than 2^126 at once
    ([-90, 60, -90, -90], [0, 160, 0, 0]),  # the loud one without weight
    ([10, 30, 50, 70], [0, 20, 40, 60]),    # all of the same level
])
def test_one_warps_keys_of_any_scales(ff, rows, exps, shifts):
    rng = np.random.default_rng(rows + exps[0] % 7)
    cache, ref = fill_pairs(ff, rng, rows, 128 * len(exps) - 70, exps, shifts)
    q = 2.0 + 0.5 * rng.standard_normal((1, rows, MANY, 64))
    check(cache, ref, q, False)


@pytest.mark.parametrize("rows", [3, 9, 25])
@pytest.mark.parametrize("low, high", [(-90, 60), (0, 100), (-60, 112)])
def test_a_louder_pair_behind_what_a_query_sees(ff, rows, low, high):
    rng = np.random.default_rng(rows)
    cache, ref = fill_pairs(ff, rng, rows, 257 + rows // 2, [low, low, high], [0, 0, 0])
    check(cache, ref, 2.0 + 0.5 * rng.standard_normal((1, rows, MANY, 64)), True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("value", [1.75 * 2.0 ** 120, 2.0 ** 116, 2.0 ** -104])
def test_values_at_the_ends_of_what_is_held(ff, rows, value, d):
    """The largest magnitude that the cache holds, 448 * 2^112, in every row: their sum over the keys passes the fp32
    range where their mean does not.  And a magnitude near the least, 2^-9 * 2^-96."""
    rng = np.random.default_rng(rows)
    for heads, length, spare in ((1, 1500, 0), (1, 1500, 4000), (1, 300, 0), (MANY if d == 64 and rows < 32 else 2, 400, 0)):
        cache, _ = make(ff, 1, length + spare, heads, heads, d, max_tokens=rows)
        k = torch.from_numpy(rng.standard_normal((1, length, heads, d)).astype(np.float32)).to(torch.bfloat16).cuda()
        sign = torch.from_numpy(rng.choice([-1.0, 1.0], (1, 1, heads, d))).cuda()
        v = (sign * value).to(torch.bfloat16).expand_as(k).contiguous()
        cache.append(0, k, v)
        q, _ = bf16(rng.standard_normal((1, rows, heads, d)))
        for causal in (False, True):
            out = torch.zeros_like(q)
            cache.attn(0, q, out, causal=causal)
            assert cache.error_poll() == 0
            # all values of a feature are equal, and so is their mean.  bf16's half step; f16's of the probabilities, which
            # the sum does not share; the sums' 2^-24 a key
            err = (host(out) / value - host(sign)).__abs__().max()
            assert err <= 2.0 ** -8 + 1.01 * (2.0 ** -11 + length * 2.0 ** -24 + 2.0 ** -20)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 24, 2.0 ** 26, 2.0 ** 30, 2.0 ** 60, 2.0 ** 100])
def test_scores_of_any_size(ff, rows, size):
    """One key's score lies far above the others', by about `size`: the output is its row, in whichever tile it lies, and
    however large the maxima before it are."""
    rng = np.random.default_rng(rows)
    for best, sign in ((0, 1), (300, 1), (300, -1), (449, 1)):
        cache, _ = make(ff, 1, 450, 1, 1, 64, max_tokens=rows)
        x = -rng.choice([1.0, 2.0, 0.5], (1, 450, 1, 1)) * np.ones((1, 450, 1, 64))
        if sign < 0:
            x *= 4.0                  # all scores are negative: the best is the least of them in magnitude
        x[0, best] = sign * 1.5 if sign > 0 else -0.25
        side = np.sqrt(size / 64.0)   # of q and of k
        k, _ = bf16(x * 2.0 ** np.floor(np.log2(side)))
        v, v64 = bf16(rng.integers(-8, 9, (1, 450, 1, 64)) / 8.0)  # numbers of the cache
        cache.append(0, k, v)
        q, q64 = bf16((1.0 + 0.2 * rng.random((1, rows, 1, 64))) * side)
        out, lse = torch.zeros_like(q), torch.zeros((1, rows, 1), device="cuda")
        cache.attn(0, q, out, lse=lse)
        assert cache.error_poll() == 0
        kk, vv = torch.empty_like(k), torch.empty_like(v)
        cache.load(0, kk, vv)
        assert np.array_equal(host(vv), v64)
        assert np.all(np.abs(host(out)[0, :, 0] - v64[0, best, 0]) <= 2.0 ** -8 * np.abs(v64[0, best, 0]))
        top = (q64[0, :, 0] @ host(kk)[0, best, 0]) / 8.0
        assert np.all(np.abs(host(lse)[0, :, 0] - top) <= (64 + 8) * 2.0 ** -23 * np.abs(top))


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("masked", [64, 128, 320])
def test_keys_put_out_of_sight_by_a_feature(ff, rows, masked):
    """Some blocks' keys hold a large negative number where every query holds a positive one: scores of some -2^33, over
    whole tiles.  The rest is what it is without them."""
    rng = np.random.default_rng(rows + masked)
    length, d = 500, 64
    for first in (0, 128):
        hidden = np.arange(first, first + masked)
        seen = np.setdiff1d(np.arange(length), hidden)
        x = rng.standard_normal((1, length, 1, d))
        x[..., 0] = 0.0
        x[0, hidden, 0, 0] = -1.625 * 2.0 ** 25
        y = rng.standard_normal((1, length, 1, d))
        cache, _ = make(ff, 1, length, 1, 1, d, max_tokens=rows)
        kt, k64 = bf16(x)
        vt, v64 = bf16(y)
        cache.append(0, kt, vt)
        q = rng.standard_normal((1, rows, 1, d))
        q[..., 0] = 1.7265625 * 2.0 ** 10  # products of more bits than a score has
        qt, q64 = bf16(q)
        out, w = torch.zeros_like(qt), torch.zeros((1, 1, length), device="cuda")
        cache.attn(0, qt, out, weights=w)
        assert cache.error_poll() == 0
        ref = RefCache(1, len(seen), 1, d)  # `hidden` is made of whole blocks, so the others stay what they are
        ref.append(k64[:, seen], v64[:, seen])
        want, _, rw, (spread, mag, wtol) = ref.attn(q64, weights=np.zeros((1, 1, len(seen))))
        tol = out_tol(want, spread, mag, d, length) + small_tol(ref, q64, False)
        assert np.all(np.abs(host(out) - want) <= tol)
        assert not bool(w[0, 0, torch.from_numpy(hidden).cuda()].any())
        assert np.all(np.abs(host(w)[0, 0, seen] - rw[0, 0]) <= wtol[0, 0] + 2.0 ** -23 * rw[0, 0])
