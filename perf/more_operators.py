"""The operators of the paged key/value cache: planning a step, storing rows, and attention over pages.

A pool of pages is shared by requests of different lengths.  A page holds page_rows rows of every kv head:
    k, v      bf16   [pages, kv_heads, page_rows, head_dim]
    tables    int32  [requests, most pages of one]: the pages of each request, in order
    lengths   int32  [requests], the rows held
    free      int32  [pages], a stack of the n_free[0] pages that no request has
The new rows of a step lie packed, one request after the other: q [n, heads, head_dim], k and v [n, kv_heads, head_dim].

  plan   cuts request r to start[r] rows (where start is given), then adds counts[r] new ones.  Pages that nobody needs
         any more go onto the stack (the j-th of them to free[n_free + all - 1 - j]), then the pages that are needed
         come off it, requests in order; a row for which no page is left has no place.  Gives
             first      int32 [requests + 1]: where the rows of each request begin
             slots      int32 [n]: page * page_rows + row of every new row's place, -1 where it has none
             positions  int32 [n]: its index in the request, 0 where it has no place
  store  puts row i of k and v into slots[i], for every kv head.
  attn   out = softmax(q k^T / sqrt(head_dim)) v over the rows held, causal: of the c new rows of a request that now
         holds L, row i sees rows 0 .. L - c + i.  lse is the natural logarithm of the softmax sum.  Query heads share
         the kv heads in groups.  Rows of q behind the last request are left as they were.
"""
import math

import torch

own = False


def _attn(name, requests, new, length, heads, kv_heads, d, page, ragged, what):
    """what: "token" (`new` tokens at most each), "prompt" (whole prompts), "chunk" (`new` rows behind a prefix; every
    second request has one token instead)."""
    return dict(name=name, op="attn", what=what, requests=requests, new=new, length=length, heads=heads,
                kv_heads=kv_heads, d=d, page=page, ragged=ragged)


def _store(name, requests, new, length, kv_heads, d, page, ragged):
    return dict(name=name, op="store", what="chunk" if new > 1 else "token", requests=requests, new=new, length=length,
                heads=kv_heads, kv_heads=kv_heads, d=d, page=page, ragged=ragged)


def _plan(name, requests, new, length, page):
    return dict(name=name, op="plan", what="plan", requests=requests, new=new, length=length, heads=1, kv_heads=1, d=64,
                page=page, ragged=True)


def listed():
    return [
        # one token of a small model behind a short context: nothing but latency
        _attn("token_tiny", 1, 1, 208, 2, 2, 64, 16, False, "token"),
        # one token against the context of a 480p chunk (20 frames of 1560 tokens, 12 heads)
        _attn("token_480p", 1, 1, 31200, 12, 12, 128, 16, False, "token"),
        # one token each of a served batch, grouped heads, requests of very different lengths
        _attn("token_batch", 64, 1, 8190, 32, 8, 128, 16, True, "token"),
        # up to five drafted tokens of eight requests, large pages
        _attn("drafts", 8, 5, 20011, 40, 8, 128, 64, True, "token"),
        # a few short prompts of a small model
        _attn("prompts_tiny", 5, 0, 333, 8, 2, 64, 32, True, "prompt"),
        # prompts of different lengths in one step, grouped heads
        _attn("prompts", 12, 0, 4680, 32, 8, 128, 16, True, "prompt"),
        # one long prompt: ten frames of 480p, 12 heads
        _attn("prompt_480p", 1, 0, 15600, 12, 12, 128, 128, False, "prompt"),
        # a step of everything: prompts that continue behind a prefix, and single tokens of other requests
        _attn("chunks", 10, 1560, 12480, 40, 8, 128, 32, True, "chunk"),
        # a decoding step of a served batch: one token each, a page here and there
        _plan("plan_tokens", 128, 0, 8190, 16),
        # a fifth of the requests end and prompts come in their place
        _plan("plan_prompts", 300, 1111, 8190, 16),
        # a token of a served batch
        _store("store_token", 64, 1, 8190, 8, 128, 16, True),
        # chunks of 1560 rows and single tokens, 40 kv heads
        _store("store_chunks", 6, 1560, 12480, 40, 128, 32, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    d = rng.choice([64, 128])
    page = rng.choice([16, 16, 32, 64, 128])
    kind = rng.choice(["token", "token", "draft", "prompt", "prompt", "chunk", "plan", "store"])
    kv = rng.choice([1, 2, 3, 4, 8, 12, 40])
    group = rng.choice([1, 1, 2, 3, 4, 5, 8])
    requests = 1 if rng.random() < 0.3 else _log(rng, 1, 65)
    ragged = rng.random() < 0.7
    if kind == "plan":
        return _plan("", _log(rng, 1, 500), _log(rng, 1, 2000), _log(rng, 1, 20000), page)
    if kind in ("token", "draft"):
        new = 1 if kind == "token" else rng.randint(2, 8)
        length = max(new, min(_log(rng, 1, 60000), 1_200_000 // (requests * kv)))
        return _attn("", requests, new, length, kv * group, kv, d, page, ragged, "token")
    requests = min(requests, 16)
    if kind == "store":
        new = _log(rng, 1, 4680)
        length = max(new, min(_log(rng, new, 31200), 1_200_000 // (requests * kv)))
        new = min(new, max(1, 190_000 // (requests * kv)))
        return _store("", requests, new, length, kv, d, page, ragged)
    pairs = 1_000_000_000 // (requests * kv * group)
    if kind == "prompt":
        length = min(_log(rng, 1, 12000), math.isqrt(2 * pairs), 1_200_000 // (requests * kv))
        return _attn("", requests, 0, length, kv * group, kv, d, page, ragged, "prompt")
    new = min(_log(rng, 9, 2000), math.isqrt(pairs))
    length = max(new, min(_log(rng, new, 31200), pairs // new, 1_200_000 // (requests * kv)))
    return _attn("", requests, new, length, kv * group, kv, d, page, ragged, "chunk")


# ---- inputs ----------------------------------------------------------------


def _lengths(c):
    """Rows held when the step is over (plan: before it): the longest first, the others anywhere below it.  One slot of
    four or more is idle."""
    got = []
    for b in range(c["requests"]):
        x = c["length"]
        if c["ragged"] and b:
            x = 1 + (x - 1) * ((b * 7919 + 3) % 101) // 101
        got.append(x)
    if c["requests"] >= 4:
        got[3] = 0
    return got


def _counts(c):
    """New rows of the step."""
    got = []
    for b, x in enumerate(_lengths(c)):
        if c["what"] == "plan":  # a prompt in an idle slot, else a token; now and then a slot stays idle
            got.append(1 + c["new"] * ((b * 37 + 5) % 97) // 97 if _ended(c, b) and b % 15 != 7 else min(x, 1))
        elif c["what"] == "prompt":
            got.append(x)
        elif c["what"] == "chunk":
            got.append(min(x, c["new"] if b % 2 == 0 else 1))
        else:
            got.append(min(x, 1 + (b * 3 + c["new"] - 1) % c["new"]))
    return got


def _ended(c, b):
    return c["what"] == "plan" and c["new"] > 0 and b % 5 == 2


def _held(c):
    """Rows held before the step."""
    if c["op"] == "plan":
        return [0 if _ended(c, b) else x for b, x in enumerate(_lengths(c))]
    return [x - y for x, y in zip(_lengths(c), _counts(c))]


def _pages(c, rows):
    return [-(-x // c["page"]) for x in rows]


def _after(c):
    return [x + y for x, y in zip(_held(c), _counts(c))]


def _n(c):
    """Rows of the packed buffers: a few more than the step has, as buffers of a recorded step are."""
    return -(-sum(_counts(c)) // 8) * 8


def prepare(case, seed):
    c = case
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    held, counts, after, n = _held(c), _counts(c), _after(c), _n(c)
    need = _pages(c, after)
    pool = sum(need) + sum(need) // 10 + 3
    width = max(max(need), 1) + 2
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    st = dict(case=c, dev=dev, n=n, width=width, pool=pool, start=i32(held), counts=i32(counts), none=i32([0] * len(held)),
              most=max(max(counts), 1))
    # pages as a pool in use has them: in no order
    order = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    given = held if c["op"] == "plan" else after
    tables = torch.zeros((c["requests"], width), dtype=torch.int32, device=dev)
    at = 0
    for b, x in enumerate(_pages(c, given)):
        tables[b, :x] = order[at:at + x]
        at += x
    st["tables"], st["lengths"], st["n_free"] = tables, i32(given), i32([pool - at])
    st["free"] = torch.zeros(pool, dtype=torch.int32, device=dev)
    st["free"][:pool - at] = order[at:]
    st["first"] = i32([0] * (c["requests"] + 1))
    st["slots"], st["positions"] = i32([0] * n), i32([0] * n)
    if c["op"] != "plan":
        _plain_plan(st, st["start"], st["counts"])
        shape = (pool, c["kv_heads"], c["page"], c["d"])
        loud = 0.5 + 1.5 * torch.rand((c["kv_heads"], 1, c["d"]), generator=gen, device=dev) ** 4
        st["k_pool"] = torch.randn(shape, generator=gen, device=dev).mul_(loud).to(torch.bfloat16)
        st["v_pool"] = torch.randn(shape, generator=gen, device=dev).to(torch.bfloat16)
    if c["op"] == "store":
        rows = (n, c["kv_heads"], c["d"])
        st["k"], st["v"] = (torch.randn(rows, generator=gen, device=dev).to(torch.bfloat16) for _ in range(2))
    if c["op"] == "attn":
        shape = (n, c["heads"], c["d"])
        st["q"] = (1.3 * torch.randn(shape, generator=gen, device=dev)).to(torch.bfloat16)
        st["out"] = torch.zeros(shape, dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.zeros(shape[:2], dtype=torch.float32, device=dev)
    if own:
        from kv_cache_attention_ff_gb300 import ff
        cache = ff.PagedCache(pages=pool, page_rows=c["page"], requests=c["requests"], capacity=width * c["page"],
                              heads=c["heads"], kv_heads=c["kv_heads"], head_dim=c["d"], max_rows=n)
        cache.tables.copy_(st["tables"])
        cache.lengths.copy_(st["lengths"])
        cache.free.copy_(st["free"])
        cache.n_free.copy_(st["n_free"])
        if c["op"] != "plan":
            cache.plan(n, st["counts"], start=st["start"])
            k, v = cache.layer(0)
            k.copy_(st["k_pool"])
            v.copy_(st["v_pool"])
            del st["k_pool"], st["v_pool"]
        st["cache"] = cache
        torch.cuda.synchronize()
    return st


# ---- the plain forms ---------------------------------------------------------


def _plain_plan(st, start, counts):
    c, dev, n, width = st["case"], st["dev"], st["n"], st["width"]
    page, pool = c["page"], st["pool"]
    length = st["lengths"].long()
    kept = torch.minimum(start.long().clamp(min=0), length)
    first = torch.zeros(c["requests"] + 1, dtype=torch.long, device=dev)
    first[1:] = counts.long().clamp(0, n).cumsum(0)
    first.clamp_(max=n)
    want = (kept + first[1:] - first[:-1]).clamp(max=width * page)
    had, need = (length + page - 1) // page, (want + page - 1) // page
    j = torch.arange(width, device=dev)
    # pages onto the stack
    back = (j >= need[:, None]) & (j < had[:, None])
    n_back = back.sum()
    top = st["n_free"].long() + n_back
    at = torch.where(back, top - 1 - (back.flatten().cumsum(0).view_as(back) - 1), torch.full_like(back, pool, dtype=torch.long))
    free = torch.cat([st["free"], st["free"][:1]])
    free.scatter_(0, at.flatten(), st["tables"].flatten())
    # and off it
    taken = (need - had).clamp(min=0)
    got = torch.minimum(taken, (top - (taken.cumsum(0) - taken)).clamp(min=0))
    mine = (j >= had[:, None]) & (j < (had + got)[:, None])
    at = (top - mine.flatten().cumsum(0)).view_as(mine).clamp(0, pool)
    st["tables"].copy_(torch.where(mine, free[at], st["tables"]))
    st["free"].copy_(free[:pool])
    st["n_free"].copy_(top - got.sum())
    length = torch.where(taken > 0, torch.minimum(want, (had + got) * page), want)
    st["lengths"].copy_(length)
    st["first"].copy_(first)
    # the rows' places
    i = torch.arange(n, device=dev)
    r = torch.searchsorted(first[1:], i, right=True).clamp(max=c["requests"] - 1)
    position = kept[r] + i - first[r]
    placed = (i < first[-1]) & (position < length[r])
    position = torch.where(placed, position, torch.zeros_like(position))
    slot = st["tables"][r, position // page].long() * page + position % page
    st["slots"].copy_(torch.where(placed, slot, torch.full_like(slot, -1)))
    st["positions"].copy_(position)


def _plain_store(st):
    # rows without a place go to one more slot at the end
    c, rows = st["case"], st["pool"] * st["case"]["page"]
    at = torch.where(st["slots"] >= 0, st["slots"].long(), torch.full_like(st["slots"], rows, dtype=torch.long))
    got = []
    for new, name in ((st["k"], "k_pool"), (st["v"], "v_pool")):
        x = st[name].transpose(1, 2).reshape(rows, c["kv_heads"], c["d"])
        x = torch.cat([x, x[:1]])
        x[at] = new
        x = x[:rows].reshape(st["pool"], c["page"], c["kv_heads"], c["d"]).transpose(1, 2)
        st[name].copy_(x)
        got.append(st[name])
    return got


def _plain_tokens(st):
    """All requests at once, padded to the longest."""
    c, dev, R = st["case"], st["dev"], st["case"]["requests"]
    rows, new = c["length"], st["most"]
    group, d = c["heads"] // c["kv_heads"], c["d"]
    length, first = st["lengths"].long(), st["first"].long()
    count = first[1:] - first[:-1]
    tables = st["tables"][:, :-(-rows // c["page"])].long()
    k, v = (st[x][tables].float().transpose(1, 2).reshape(R, c["kv_heads"], -1, d)[:, :, :rows] for x in ("k_pool", "v_pool"))
    i = torch.arange(new, device=dev)
    valid = i < count[:, None]
    at = torch.where(valid, first[:-1, None] + i, torch.full_like(count[:, None] + i, st["n"]))  # one row more for the rest
    q = torch.cat([st["q"], st["q"][:1]])[at].float()
    q = q.reshape(R, new, c["kv_heads"], group, d).permute(0, 2, 3, 1, 4).reshape(R, c["kv_heads"], group * new, d)
    s = torch.matmul(q, k.transpose(2, 3)).reshape(R, c["kv_heads"], group, new, rows) * (1.0 / math.sqrt(d))
    seen = torch.where(valid, (length - count)[:, None] + i + 1, torch.zeros_like(at))
    s.masked_fill_((torch.arange(rows, device=dev) >= seen[..., None])[:, None, None], -math.inf)
    some = (seen > 0)[:, None, None, :, None]
    m = torch.where(some, s.amax(-1, keepdim=True), torch.zeros_like(s[..., :1]))
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(R, c["kv_heads"], group * new, rows), torch.where((torch.arange(rows, device=dev) < length[:, None])[:, None, :, None], v, torch.zeros_like(v)))
    o = o.reshape(R, c["kv_heads"], group, new, d) / torch.where(some, l, torch.ones_like(l))
    o = o.permute(0, 3, 1, 2, 4).reshape(R, new, c["heads"], d).to(torch.bfloat16)
    lse = (m + torch.log(l))[..., 0].permute(0, 3, 1, 2).reshape(R, new, c["heads"])
    out, to_lse = torch.cat([st["out"], st["out"][:1]]), torch.cat([st["lse"], st["lse"][:1]])
    out[at], to_lse[at] = o, lse
    return [out[:st["n"]], to_lse[:st["n"]]]


def _plain_prompts(st):
    """One request after the other, as many heads at a time as 4 GB of scores hold."""
    c, dev = st["case"], st["dev"]
    group, d = c["heads"] // c["kv_heads"], c["d"]
    out, to_lse = st["out"].clone(), st["lse"].clone()
    at = 0
    for b, (length, count) in enumerate(zip(_after(c), _counts(c))):
        if not count:
            continue
        pages = st["tables"][b, :-(-length // c["page"])].long()
        k, v = (st[x][pages].float().transpose(0, 1).reshape(c["kv_heads"], -1, d)[:, :length] for x in ("k_pool", "v_pool"))
        q = st["q"][at:at + count].float().transpose(0, 1)  # [heads, count, d]
        hidden = torch.arange(length, device=dev) > (torch.arange(count, device=dev) + length - count)[:, None]
        step = max(1, 1_000_000_000 // (count * length))
        for h in range(0, c["heads"], step):
            of = torch.arange(h, min(h + step, c["heads"]), device=dev) // group
            s = torch.matmul(q[h:h + step], k[of].transpose(1, 2)).mul_(1.0 / math.sqrt(d)).masked_fill_(hidden, -math.inf)
            m = s.amax(-1, keepdim=True)
            p = s.sub_(m).exp_()
            l = p.sum(-1, keepdim=True)
            out[at:at + count, h:h + step] = (torch.matmul(p, v[of]) / l).transpose(0, 1).to(torch.bfloat16)
            to_lse[at:at + count, h:h + step] = (m + torch.log(l))[..., 0].T
        at += count
    return [out, to_lse]


# ---- one pass ------------------------------------------------------------------


def run(st):
    c = st["case"]
    if c["op"] == "plan":
        # the step before is taken back (its tokens were drafts, its prompts have ended), then comes the next
        if own:
            cache = st["cache"]
            cache.plan(st["n"], st["none"], start=st["start"])
            cache.plan(st["n"], st["counts"])
            return [cache.tables, cache.lengths, cache.first, cache.slots, cache.positions, cache.n_free]
        _plain_plan(st, st["start"], st["none"])
        _plain_plan(st, st["lengths"], st["counts"])
        return [st[x] for x in ("tables", "lengths", "first", "slots", "positions", "n_free")]
    if c["op"] == "store":
        if own:
            st["cache"].store(0, st["k"], st["v"])
            return list(st["cache"].layer(0))
        return _plain_store(st)
    if own:
        st["cache"].attn(0, st["q"], st["out"], most=st["most"], lse=st["lse"])
        return [st["out"], st["lse"]]
    return _plain_tokens(st) if c["what"] == "token" else _plain_prompts(st)


def work(case):
    c = case
    after, counts, n = _after(c), _counts(c), _n(c)
    row = c["kv_heads"] * 2 * c["d"] * 2  # bytes of K and V
    if c["op"] == "plan":
        moved = sum(x - y for x, y in zip(_pages(c, after), _pages(c, _held(c))))
        # two calls: lengths, counts, starts and first of each; slots and positions; pages off the stack and onto it
        return {"bytes": 2 * (c["requests"] * 20 + n * 8) + moved * 16, "flops": 2 * n}
    if c["op"] == "store":
        return {"bytes": sum(counts) * (2 * row + 4), "flops": 0}
    pairs = sum(m * (x - m) + m * (m + 1) // 2 for x, m in zip(after, counts))
    held = sum(x for x, m in zip(after, counts) if m)
    return {"bytes": held * row + sum(counts) * c["heads"] * (4 * c["d"] + 4), "flops": 4 * c["d"] * pairs * c["heads"]}


# ---- the definitions in 64 bits --------------------------------------------------


def exact(case, seed):
    """The definitions in 64 bits, one request and head after the other; None for the plans, which are whole numbers."""
    global own
    c, was = case, own
    if c["op"] == "plan":
        return None
    own = False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    at, page, d = 0, c["page"], c["d"]
    if c["op"] == "store":
        got = [st[x].double() for x in ("k_pool", "v_pool")]
        for b, (length, count) in enumerate(zip(_after(c), _counts(c))):
            table = st["tables"][b].tolist()
            done = 0
            while done < count:  # as far as the page goes
                position = length - count + done
                rows = min(count - done, page - position % page)
                for to, x in zip(got, (st["k"], st["v"])):
                    to[table[position // page], :, position % page:position % page + rows] = \
                        x[at + done:at + done + rows].double().transpose(0, 1)
                done += rows
            at += count
        return got
    group = c["heads"] // c["kv_heads"]
    out, lse = st["out"].double(), st["lse"].double()
    for b, (length, count) in enumerate(zip(_after(c), _counts(c))):
        if not count:
            continue
        table = st["tables"][b, :-(-length // page)].tolist()
        for h in range(c["kv_heads"]):
            k, v = (torch.cat([st[x][t, h] for t in table]).double()[:length] for x in ("k_pool", "v_pool"))
            for g in range(h * group, (h + 1) * group):
                for i in range(0, count, 2048):  # queries
                    m = min(2048, count - i)
                    seen = length - count + i + m
                    s = (st["q"][at + i:at + i + m, g].double() @ k[:seen].T).div_(math.sqrt(d))
                    s += torch.full_like(s, -math.inf).triu_(seen - m + 1)
                    top = torch.logsumexp(s, 1)
                    lse[at + i:at + i + m, g] = top
                    out[at + i:at + i + m, g] = s.sub_(top[:, None]).exp_() @ v[:seen]
        at += count
    return [out, lse]
