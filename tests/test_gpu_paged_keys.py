"""The paged cache's attention over long contexts, key by key (tests/paged_keys.py): both kernels, cut and uncut ranges, pages
in no order, and the longest request."""
import numpy as np
import pytest

from tests.paged_keys import STAGE, count_errors, count_keys, features_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ff():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_attention_ff_gb300 import build, ff as ffmod
    build.build()
    return ffmod


def placed(ff, lengths, news, heads, kv, d, page_rows, seed=0, own_pages=None, capacity=None):
    """A cache that holds `lengths` rows of each request, `news` of them planned as a step; the pages lie in no order.
    own_pages: how many of a request's pages are its own (the last among them), the others being anybody's (default: all)."""
    rng = np.random.default_rng(seed)
    width = [-(-x // page_rows) for x in lengths]
    own = [x if own_pages is None else min(x, own_pages) for x in width]
    shared = 0 if own_pages is None else 400
    pages = sum(own) + shared + 5
    order = rng.permutation(pages).astype(np.int32)
    cache = ff.PagedCache(pages=pages, page_rows=page_rows, requests=len(lengths), capacity=capacity or max(lengths),
                          heads=heads, kv_heads=kv, head_dim=d, max_rows=sum(news) + 16)
    tables, at = [], shared
    for r, (x, mine) in enumerate(zip(width, own)):
        table = order[rng.integers(0, max(shared, 1), x)]
        table[np.append(rng.choice(x - 1, mine - 1, replace=False), x - 1)] = order[at:at + mine]
        at += mine
        cache.tables[r, :x] = torch.as_tensor(table, device="cuda")
        tables.append(table)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cache.lengths.copy_(i32(lengths))
    cache.free[:pages - at] = torch.as_tensor(order[at:], device="cuda")
    cache.n_free.fill_(pages - at)
    cache.plan(sum(news), i32(news), start=i32([x - y for x, y in zip(lengths, news)]))
    assert cache.lengths.tolist() == list(lengths) and cache.error_poll() == 0
    for r, table in enumerate(tables):
        assert np.array_equal(cache.tables[r, :len(table)].cpu().numpy(), table)
    return cache, tables, rng


def forms(cache, news):
    """`most` for which a call takes the token form (if it may) and the prompt form."""
    group = cache.heads // cache.kv_heads
    few = max(news) <= 8 // group
    return [*([max(news)] if few else []), max(max(news), 8 // group + 1)]


def count(cache, tables, rng, lengths, news):
    """Largest errors of out and lse over both forms, in units of what is allowed."""
    heads, kv, d, page_rows = cache.heads, cache.kv_heads, cache.head_dim, cache.page_rows
    feature = rng.integers(0, d, (cache.pages, kv, page_rows // STAGE))
    k, v = cache.layer(0)
    k.normal_()
    ones = torch.nn.functional.one_hot(torch.as_tensor(feature, device="cuda"), d).to(torch.bfloat16)
    v.copy_(ones.repeat_interleave(STAGE, dim=2))
    n = sum(news)
    q = torch.zeros((n, heads, d), dtype=torch.bfloat16, device="cuda")
    counts, seen = np.zeros((n, kv, d)), np.zeros((n, kv), np.int64)
    at = 0
    for table, length, new in zip(tables, lengths, news):
        for h in range(kv):
            stages = features_of(table, feature, page_rows, h)
            total = count_keys(stages, length, d)
            for i in range(new):  # row i sees `hidden` keys fewer
                hidden = new - 1 - i
                mine = total.copy()
                for key in range(length - hidden, length):
                    mine[stages[key // STAGE]] -= 1
                counts[at + i, h], seen[at + i, h] = mine, length - hidden
        at += new
    group = heads // kv
    counts, seen = counts.repeat(group, 1), seen.repeat(group, 1)
    worst = [0.0, 0.0]
    for most in forms(cache, news):
        out, lse = torch.full_like(q, 7.0), torch.full((n, heads), 7.0, device="cuda")
        cache.attn(0, q, out, most=most, lse=lse)
        errors = count_errors(out.double().cpu().numpy(), lse.double().cpu().numpy(), counts, seen)
        assert cache.error_poll() == 0
        worst = [max(x, y) for x, y in zip(worst, errors)]
    return worst


def plant(cache, tables, rng, lengths, news, passes):
    """Every query row finds its key wherever it is: over `passes` passes the keys go through the stages that are the
    request's own, first, last and other rows of them in turn."""
    heads, kv, d, page_rows = cache.heads, cache.kv_heads, cache.head_dim, cache.page_rows
    group, n = heads // kv, sum(news)
    # no other key's score is above 0, and theirs is 21^2 / sqrt(d) (39 or 55): with 2^24 others, e^39 / 2^24 = 2^32
    c = 21.0
    assert group <= d
    k, v = cache.layer(0)
    v.uniform_(0.5, 1.5)
    first = np.concatenate([[0], np.cumsum(news)])
    q = torch.zeros((n, heads, d), dtype=torch.bfloat16, device="cuda")
    for h in range(heads):
        q[:, h, h % group] = c
    times = np.bincount(np.concatenate(tables), minlength=cache.pages)
    use = [np.flatnonzero(times[t] == 1) for t in tables]  # pages that are the request's own
    for at in range(passes):
        k.zero_()
        page, head, row, feature, want = [], [], [], [], np.zeros((n, heads, 2), np.int64)
        for r, (length, new) in enumerate(zip(lengths, news)):
            if not new:
                continue
            seen = length - new + 1  # of the first row, so that all rows see it
            stages = np.concatenate([x * (page_rows // STAGE) + np.arange(page_rows // STAGE) for x in use[r]])
            stages = stages[stages * STAGE < seen]
            for h in range(kv):
                for g in range(group):
                    i = (at * kv + h) * group + g
                    stage = stages[i % len(stages)]
                    inside = (0, STAGE - 1, rng.integers(0, STAGE))[(i // len(stages) + at) % 3]
                    key = min(stage * STAGE + int(inside), seen - 1)
                    page.append(tables[r][key // page_rows])
                    head.append(h)
                    row.append(key % page_rows)
                    feature.append(g)
                    want[first[r]:first[r + 1], h * group + g] = page[-1], row[-1]
        index = [torch.as_tensor(np.array(x), dtype=torch.long, device="cuda") for x in (page, head, row, feature)]
        k[index[0], index[1], index[2], index[3]] = c
        want = torch.as_tensor(want, device="cuda")
        of = torch.arange(heads, device="cuda") // group
        expected = v[want[..., 0], of.expand(n, heads), want[..., 1]]
        for most in forms(cache, news):
            out = torch.full_like(q, 7.0)
            cache.attn(0, q, out, most=most)
            assert torch.equal(out, expected), (at, most, torch.nonzero((out != expected).any(-1))[:4].tolist())
    assert cache.error_poll() == 0


CASES = [
    # lengths, new rows, heads, kv_heads, d, page_rows
    ([31200], [1], 64, 8, 128, 16),
    ([31200], [1], 12, 12, 128, 16),
    ([31200, 20011, 5000, 333], [1, 1, 1, 1], 32, 8, 128, 16),
    ([40000], [4], 2, 1, 64, 128),
    ([60000, 17], [1, 1], 8, 1, 64, 32),
    ([31207, 9000], [3, 5], 40, 8, 64, 64),
    ([31200], [200], 4, 2, 128, 16),
    ([33333, 4000, 129], [70, 1, 129], 6, 2, 64, 32),
    ([20000] * 20, [9] * 20, 16, 8, 128, 64),   # blocks of rows that are not cut
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_every_key_is_counted_once(ff, case):
    lengths, news, heads, kv, d, page_rows = CASES[case]
    cache, tables, rng = placed(ff, lengths, news, heads, kv, d, page_rows, seed=case)
    out, lse = count(cache, tables, rng, lengths, news)
    assert out <= 1 and lse <= 1


@pytest.mark.parametrize("case", range(len(CASES)))
def test_a_row_finds_its_key_in_every_stage(ff, case):
    lengths, news, heads, kv, d, page_rows = CASES[case]
    cache, tables, rng = placed(ff, lengths, news, heads, kv, d, page_rows, seed=case)
    stages = max(lengths) // STAGE
    plant(cache, tables, rng, lengths, news, min(150, -(-3 * stages // heads)))


# 152 SMs list at most 4 * 304 / kv_heads + requests + 1 key ranges of few rows (the handle has room for no more): with more
# stages than that many ranges of 128 hold, whatever rule cuts them, a warp, which takes every fourth stage, has more than the
# 32 whose pages it holds, and with twice as many it takes pages twice on the way.
MANY = [
    # requests, keys, kv_heads, group, d, page_rows, refills
    (64, 12000, 8, 2, 128, 16, 1),
    (64, 16001, 8, 1, 64, 128, 2),
    (64, 16400, 8, 4, 128, 16, 2),
    (40, 18000, 8, 8, 64, 64, 1),
]


@pytest.mark.parametrize("case", range(len(MANY)))
def test_ranges_longer_than_a_warps_list_of_pages(ff, case):
    requests, keys, kv, group, d, page_rows, refills = MANY[case]
    lengths = [keys - 37 * r % 64 for r in range(requests)]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert sum(lengths) / STAGE / (4 * 2 * sms // kv + requests + 1) > 128 * refills
    news = [1] * requests
    cache, tables, rng = placed(ff, lengths, news, kv * group, kv, d, page_rows, seed=case)
    out, lse = count(cache, tables, rng, lengths, news)
    assert out <= 1 and lse <= 1
    plant(cache, tables, rng, lengths, news, -(-keys // STAGE // (kv * group)))


@pytest.mark.parametrize("heads, d, new", [(2, 64, 1), (2, 128, 70), (12, 64, 1)])
def test_the_longest_request(ff, heads, d, new):
    """2^24 rows over few pages that come again and again, beside a short request."""
    lengths, news = [1 << 24, 300], [new, 1]
    cache, tables, rng = placed(ff, lengths, news, heads, 1, d, 128, seed=d, own_pages=200, capacity=1 << 24)
    out, lse = count(cache, tables, rng, lengths, news)
    assert out <= 1 and lse <= 1
    plant(cache, tables, rng, lengths, news, 20)
    n = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    cache.plan(2, n)  # one row more has no place
    assert cache.error_poll() == 8 and cache.lengths.tolist() == [1 << 24, 301]
