"""The paged cache where it could go wrong: many key ranges of few rows, more requests and heads than run at once, buffers
larger than the step, random shapes, first calls inside a capture, graphs beside eager calls."""
import random
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest

from tests.test_gpu_paged import bf16, check_attn, check_plan, host, i32, make, plan, shuffled, store

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ff():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_attention_ff_gb300 import build, ff as ffmod
    build.build()
    return ffmod


def filled(ff, page_rows, heads, kv, d, held, new, more=0, seed=0):
    """A cache and its reference with `held` rows of every request, planned and stored, then the step of `new` ones."""
    rng = np.random.default_rng(seed)
    rows = [x + y for x, y in zip(held, new)]
    pages = max(1, sum(-(-x // page_rows) for x in rows))
    n = max(1, sum(new) + more)
    cache, ref = make(ff, pages, page_rows, len(held), max(rows) + 3, heads, kv, d, max(n, sum(held)))
    shuffled(cache, ref, seed)
    for x in cache.layer(0):
        x.fill_(float("nan"))
    if sum(held):
        plan(cache, ref, sum(held), held)
        store(cache, ref, sum(held), rng)
    plan(cache, ref, n, new)
    store(cache, ref, n, rng)
    return cache, ref, rng, n


LONG = [
    # page_rows, heads, kv_heads, d, held, new: few rows over long contexts, cut into many ranges
    (16, 1, 1, 64, [20000], [1]),
    (64, 2, 1, 128, [12345, 3], [1, 1]),
    (16, 8, 1, 128, [9001], [1]),
    (16, 9, 1, 128, [9001], [1]),
    (32, 10, 2, 128, [9000], [3]),
    (128, 5, 1, 64, [15000, 100], [5, 1]),
    (16, 40, 1, 128, [6000], [1]),
    (16, 3, 1, 64, [8000, 8000], [40, 3]),
    (32, 4, 2, 128, [7000], [150]),
    (16, 70, 1, 64, [5000], [1]),
    (16, 300, 1, 64, [3000], [1]),
    (128, 2, 2, 128, [127, 128, 5000], [1, 200, 9]),
]


@pytest.mark.parametrize("case", range(len(LONG)))
def test_long_contexts_of_few_rows(ff, case):
    page_rows, heads, kv, d, held, new = LONG[case]
    cache, ref, rng, n = filled(ff, page_rows, heads, kv, d, held, new, seed=case)
    check_attn(cache, ref, rng.standard_normal((n, heads, d)))
    check_attn(cache, ref, rng.standard_normal((n, heads, d)), most=max(new))


@pytest.mark.parametrize("requests, heads, kv, new", [(700, 2, 1, 1), (700, 4, 1, 30), (40, 12, 2, 20), (1100, 1, 1, 2), (3, 500, 500, 1),
                                                      (2, 500, 500, 40), (5, 1000, 250, 3)])
def test_more_work_than_runs_at_once(ff, requests, heads, kv, new):
    draw = random.Random(requests + heads)
    held = [draw.choice([0, 1, 16, draw.randint(0, 90)]) for _ in range(requests)]
    news = [draw.choice([0, 1, new, draw.randint(0, new)]) for _ in range(requests)]
    cache, ref, rng, n = filled(ff, 16, heads, kv, 64, held, news, more=3, seed=requests)
    check_attn(cache, ref, rng.standard_normal((n, heads, 64)))
    check_attn(cache, ref, rng.standard_normal((n, heads, 64)), most=max(1, *news))


@pytest.mark.parametrize("requests, heads, kv, long, new", [(250, 2, 1, [9000], 9), (400, 4, 2, [6000, 0, 3000], 9), (600, 20, 2, [5000], 3),
                                                            (60, 16, 8, [4000, 2500], 40), (57, 24, 8, [4000], 30), (450, 9, 1, [7000] * 3, 1)])
def test_one_context_much_longer_than_the_others(ff, requests, heads, kv, long, new):
    """Few blocks are cut among many that are not, in more rounds than the GPU holds at once."""
    draw = random.Random(requests)
    held = [draw.randint(0, 120) for _ in range(requests)]
    for x, at in zip(long, (requests // 2, 0, requests - 1)):
        held[at] = x
    news = [draw.choice([1, new, draw.randint(0, new)]) for _ in range(requests)]
    cache, ref, rng, n = filled(ff, 32, heads, kv, 64, held, news, seed=requests)
    check_attn(cache, ref, rng.standard_normal((n, heads, 64)))


@pytest.mark.parametrize("requests, heads, kv, d, held, new", [(160, 1, 1, 64, 3000, 1), (44, 8, 4, 128, 1500, 2), (20, 24, 8, 128, 2000, 20),
                                                               (310, 2, 1, 64, 1100, 9), (60, 6, 3, 64, 2500, 3), (153, 1, 1, 128, 700, 130)])
def test_steps_whose_last_round_is_not_full(ff, requests, heads, kv, d, held, new):
    """Equal blocks, a few more than run at once: the last ones are cut."""
    cache, ref, rng, n = filled(ff, 64, heads, kv, d, [held + i % 3 for i in range(requests)], [new] * requests, seed=requests)
    check_attn(cache, ref, rng.standard_normal((n, heads, d)))


@pytest.mark.parametrize("requests, heads, kv, new", [(1100, 1, 1, 1), (2100, 4, 2, 2), (1025, 8, 1, 1), (1024, 2, 2, 1)])
def test_long_contexts_among_many_tokens(ff, requests, heads, kv, new):
    """Some requests are cut, most are not, and there are more of them than threads list at once."""
    draw = random.Random(requests)
    held = [draw.randint(0, 20) for _ in range(requests)]
    for at in (5, 1000, requests - 1):
        held[at] = draw.randint(4000, 6000)
    news = [draw.randint(0, new) for _ in range(requests)]
    news[5] = news[1000] = news[-1] = new
    cache, ref, rng, n = filled(ff, 16, heads, kv, 64, held, news, seed=requests)
    check_attn(cache, ref, rng.standard_normal((n, heads, 64)), most=new)
    check_attn(cache, ref, rng.standard_normal((n, heads, 64)))


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(ff, seed):
    draw = random.Random(seed)
    page_rows, d = draw.choice([16, 32, 64, 128]), draw.choice([64, 128])
    kv, group = draw.choice([1, 2, 3, 5, 8]), draw.choice([1, 2, 3, 4, 5, 7, 8, 12, 17])
    requests = draw.choice([1, 2, 5, 9])
    held = [draw.choice([0, draw.randint(0, 40), draw.randint(0, 700)]) for _ in range(requests)]
    new = [draw.choice([0, 1, draw.randint(1, 9), draw.randint(1, 300)]) for _ in range(requests)]
    cache, ref, rng, n = filled(ff, page_rows, kv * group, kv, d, held, new, more=draw.randint(0, 9), seed=seed)
    check_attn(cache, ref, rng.standard_normal((n, kv * group, d)), most=draw.choice([None, max(1, *new)]))


@pytest.mark.parametrize("new", [[1, 1, 2], [30, 1, 140]])
def test_buffers_of_other_sizes_than_the_plan(ff, new):
    """Rows behind the step's are neither stored, whatever an earlier plan left in their slots, nor computed; a call with
    fewer rows than the plan computes those."""
    rng = np.random.default_rng(1)
    cache, ref = make(ff, 60, 16, 3, 300, 4, 2, 64, 400)
    plan(cache, ref, 400, [100, 150, 50])
    store(cache, ref, 400, rng)
    n = sum(new)
    plan(cache, ref, n, new)
    shape = (400, 2, 64)
    (k, k64), (v, v64) = bf16(rng.standard_normal(shape)), bf16(rng.standard_normal(shape))
    before = [x.clone() for x in cache.layer(0)]
    cache.store(0, k, v)
    ref.store(k64, v64)
    for x, name in zip(cache.layer(0), "kv"):
        at = np.arange(60 * 16)
        held = np.zeros(60 * 16, bool)
        for r, length in enumerate(ref.lengths):
            rows = np.arange(length)
            held[ref.tables[r, rows // 16] * 16 + rows % 16] = True
        got = host(x).transpose(0, 2, 1, 3).reshape(-1, 2, 64)
        assert np.array_equal(got[held], ref.pool[name].reshape(-1, 2, 64)[held])
        old = host(before["kv".index(name)]).transpose(0, 2, 1, 3).reshape(-1, 2, 64)
        assert np.array_equal(got[at[~held]], old[at[~held]])
    q, q64 = bf16(rng.standard_normal((400, 4, 64)))
    want, want_lse, tol, _ = ref.attn(q64)
    for rows in (400, n, n - 1, max(1, n // 2), 1):
        out, lse = torch.full_like(q, 7.0), torch.full((400, 4), 7.0, device="cuda")
        cache.attn(0, q[:rows], out[:rows], lse=lse[:rows], most=max(new))
        m = min(rows, n)
        assert bool((out[m:] == 7.0).all()) and bool((lse[m:] == 7.0).all())
        assert np.all(np.abs(host(out)[:m] - want[:m]) <= tol[:m])


def test_a_plan_from_the_lengths_themselves(ff):
    """`start` may be the cache's own lengths, and a call may follow before the one ahead of it has run."""
    rng = np.random.default_rng(2)
    cache, ref = make(ff, 40, 16, 3, 200, 2, 2, 64, 100)
    plan(cache, ref, 100, [40, 0, 20])
    for counts in ([1, 5, 0], [2, 2, 2], [0, 0, 1]):
        cache.plan(10, i32(counts), start=cache.lengths)
        ref.plan(10, counts)
    check_plan(cache, ref, 10)
    store(cache, ref, 10, rng)


def test_an_empty_step_does_nothing(ff):
    cache, ref = make(ff, 4, 16, 2, 32, 4, 2, 128, 50)
    q = torch.randn(50, 4, 128, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 3.0)
    kv = torch.ones(50, 2, 128, dtype=torch.bfloat16, device="cuda")
    cache.store(0, kv, kv)           # before the first plan
    cache.attn(0, q, out)
    plan(cache, ref, 50, [0, 0])
    cache.store(0, kv, kv)
    cache.attn(0, q, out)
    cache.attn(0, q, out, most=1)
    assert bool((out == 3.0).all()) and not any(bool(x.any()) for x in cache.layer(0))
    assert cache.error_poll() == 0


def test_graphs_and_eager_steps_side_by_side(ff):
    """Two recorded steps of different sizes, replayed in turn with eager ones in between, all on one stream."""
    rng = np.random.default_rng(8)
    cache, ref = make(ff, 300, 32, 3, 900, 4, 2, 128, 300)
    steps = {}
    for name, n, most in (("tokens", 4, 1), ("prompts", 300, 300)):
        st = dict(n=n, counts=i32([0, 0, 0]), k=torch.zeros(n, 2, 128, dtype=torch.bfloat16, device="cuda"),
                  q=torch.zeros(n, 4, 128, dtype=torch.bfloat16, device="cuda"))
        st["v"], st["out"], st["graph"] = torch.zeros_like(st["k"]), torch.zeros_like(st["q"]), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(st["graph"]):
            cache.plan(n, st["counts"])
            cache.store(0, st["k"], st["v"])
            cache.attn(0, st["q"], st["out"], most=most)
        steps[name] = st
    for name, counts in (("prompts", [200, 30, 0]), ("tokens", [1, 1, 0]), ("eager", [1, 0, 60]), ("tokens", [1, 1, 1]),
                         ("prompts", [3, 100, 1]), ("tokens", [0, 1, 1])):
        st = steps.get(name) or dict(steps["prompts"], n=sum(counts))
        n = st["n"]
        (k, k64), (v, v64), (q, q64) = (bf16(rng.standard_normal((n, x, 128))) for x in (2, 2, 4))
        if name == "eager":
            out = torch.full_like(q, 7.0)
            cache.plan(n, i32(counts))
            cache.store(0, k, v)
            cache.attn(0, q, out, most=max(counts))
        else:
            for to, x in ((st["k"], k), (st["v"], v), (st["q"], q)):
                to.copy_(x)
            st["counts"].copy_(i32(counts))
            out = st["out"].fill_(7.0)
            st["graph"].replay()
        ref.plan(n, counts)
        ref.store(k64, v64)
        want, _, tol, _ = ref.attn(q64)
        got, there = host(out), ~np.isnan(want)
        assert np.all(got[~there] == 7.0) and np.all(np.abs(got - want)[there] <= tol[there])
    check_plan(cache, ref, 4)


SCRIPT = """
import torch
from kv_cache_attention_ff_gb300 import ff
dev = torch.device("cuda:0")
gen = torch.Generator(device=dev).manual_seed(3)
draw = lambda *s: torch.randn(*s, device=dev, generator=gen).to(torch.bfloat16)
R, H, KV, D, N = 3, 6, 2, {d}, 400
counts = [torch.tensor(x, dtype=torch.int32, device=dev) for x in ([300, 1, 90], [1, 1, 1], [40, 1, 2])]
inputs = [(draw(N, KV, D), draw(N, KV, D), draw(N, H, D)) for _ in counts]

def state():
    return (ff.PagedCache(pages=90, page_rows=16, requests=R, capacity=500, heads=H, kv_heads=KV, head_dim=D, max_rows=N),
            [torch.zeros(N, H, D, dtype=torch.bfloat16, device=dev) for _ in counts], torch.zeros(N, H, device=dev))

def calls(cache, outs, lse):
    for c, most, (k, v, q), out in zip(counts, (300, 1, 40), inputs, outs):
        cache.plan(N, c)
        cache.store(0, k, v)
        cache.attn(0, q, out, most=most, lse=lse)

a, b = state(), state()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls(*a)
graph.replay()
calls(*b)
torch.cuda.synchronize()
assert a[0].error_poll() == 0 and b[0].error_poll() == 0
assert a[0].lengths.tolist() == [341, 3, 93]
flat = lambda s: [*s[1], s[2], *s[0].layer(0), s[0].tables, s[0].slots, s[0].free]
for x, y in zip(flat(a), flat(b)):
    assert torch.equal(x, y)
print("same")
"""


@pytest.mark.parametrize("d", [64, 128])
def test_the_first_calls_are_captured(d):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cache_attention_ff_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(d=d)], cwd=Path(__file__).resolve().parent.parent,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout + r.stderr


def test_most_beyond_what_a_step_can_have(ff):
    """A cache for single tokens holds no room for the results of prompts; `most` may still be anything."""
    rng = np.random.default_rng(5)
    cache, ref = make(ff, 700, 16, 2, 9000, 4, 2, 128, 2)
    cache.lengths.copy_(i32([9000 - 1, 40]))
    order = torch.arange(700, dtype=torch.int32, device="cuda")
    cache.tables[0, :563], cache.tables[1, :3] = order[:563], order[563:566]
    cache.n_free.fill_(700 - 566)
    cache.free[:134] = order[566:]
    ref.lengths, ref.stack = [8999, 40], list(range(566, 700))
    ref.tables[0, :563], ref.tables[1, :3] = np.arange(563), np.arange(563, 566)
    for name, x in zip("kv", cache.layer(0)):
        y, y64 = bf16(rng.standard_normal((700, 2, 16, 128)))
        x.copy_(y)
        ref.pool[name] = y64.transpose(0, 2, 1, 3).copy()
    plan(cache, ref, 2, [1, 1])
    store(cache, ref, 2, rng)
    for most in (1, 2, 5, 1 << 30):
        check_attn(cache, ref, rng.standard_normal((2, 4, 128)), most=most)
