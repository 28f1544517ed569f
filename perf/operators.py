"""The operators of the 8-bit key/value cache: appending rows, reading rows back, attention
(with the weight that every key received, where asked), and eviction by accumulated weight.

The cache of one layer holds, for every sequence b, blocks of 64 tokens:
    k8, v8            e4m3 codes   [batch, blocks, kv_heads, 64, head_dim]
    k_scale, v_scale  fp32         [batch, blocks, kv_heads], powers of two
    lengths           int32        [batch], the rows held
A row stands for code * scale.  The scale of a block is 2^e for the smallest e with
(largest finite magnitude of its rows) <= 448 * 2^e, e kept within -96 .. 112.

  append  rows start[b] .. start[b] + counts[b] - 1 take the codes of the new k, v (bf16).  The rows of
          the first block that lie before start[b] stay, and the block's scale is the larger of theirs
          and the one that the new rows need.  lengths[b] becomes start[b] + counts[b].
  load    the values of rows start[b] .. start[b] + n - 1 as bf16; rows that are not held are zeros.
  attn    out = softmax(q k^T / sqrt(head_dim)) v over the rows held; with `causal`, query i of counts[b]
          sees rows 0 .. lengths[b] - counts[b] + i.  A query that sees nothing gives 0 and lse -inf;
          queries from counts[b] on are left as they were.  Query heads share the kv heads in groups.
          weights[b, h, j] = weights_in[b, h, j] + what row j received from all queries of the group.
  evict   of every (sequence, kv head): the last n_recent rows and the rows of largest weight before
          them, n_keep in all (the lower row first among equals), moved into another layer in order.
"""
import math

import torch

own = False

BLOCK = 64
E_MIN, E_MAX = -96, 112


def _attn(name, batch, n, heads, kv_heads, d, length, ragged, causal, padded, weigh):
    return dict(name=name, op="attn", batch=batch, n=n, heads=heads, kv_heads=kv_heads, d=d, length=length,
                ragged=ragged, causal=causal, padded=padded, weigh=weigh)


def _append(name, batch, n, kv_heads, d, length, ragged, padded):
    return dict(name=name, op="append", batch=batch, n=n, heads=kv_heads, kv_heads=kv_heads, d=d, length=length,
                ragged=ragged, padded=padded)


def _evict(name, batch, kv_heads, d, length, ragged, keep, recent):
    return dict(name=name, op="evict", batch=batch, n=1, heads=kv_heads, kv_heads=kv_heads, d=d, length=length,
                ragged=ragged, keep=keep, recent=recent)


def listed():
    return [
        # one token of a small model over a short cache: nothing but latency
        _attn("token_tiny", 1, 1, 2, 2, 64, 208, False, True, False, False),
        # one token against the context of a 480p chunk (20 frames of 1560 tokens, 12 heads)
        _attn("token_480p", 1, 1, 12, 12, 128, 31200, False, True, False, False),
        # one token each of a served batch, grouped heads, sequences of very different lengths
        _attn("token_batch", 32, 1, 32, 8, 128, 8190, True, True, False, False),
        # five drafted tokens of four sequences, with the weights that an eviction will go by
        _attn("draft_weigh", 4, 5, 40, 8, 128, 20011, True, True, True, True),
        # a ragged batch of prompts, causal, into empty caches
        _attn("prompts", 3, 1111, 8, 2, 64, 1111, True, True, True, False),
        # one frame of a chunk against eight frames, with weights
        _attn("frame_weigh", 1, 1560, 12, 12, 128, 12480, False, False, False, True),
        # the 1.3B 480p renderer call: 4680 queries, 31200 keys
        _attn("chunk_480p", 1, 4680, 12, 12, 128, 31200, False, False, False, False),
        # a token of a served batch
        _append("append_token", 32, 1, 8, 128, 8190, True, False),
        # a chunk of three frames behind 17 frames, 40 heads: starts inside a block
        _append("append_chunk", 1, 4680, 40, 128, 31200, False, False),
        # half of a 480p context goes
        _evict("evict_480p", 1, 12, 128, 31200, False, 15600, 1560),
        # a served batch back to a budget
        _evict("evict_batch", 16, 8, 64, 8190, True, 1000, 100),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    d = rng.choice([64, 128])
    kind = rng.choice(["token", "token", "few", "chunk", "chunk", "append", "evict"])
    kv = rng.choice([1, 2, 3, 4, 8, 12, 40])
    group = rng.choice([1, 1, 2, 3, 4, 5, 8])
    batch = 1 if rng.random() < 0.4 else _log(rng, 1, 33)
    if kind in ("token", "few"):
        n = 1 if kind == "token" else rng.randint(2, 40)
        length = min(_log(rng, max(n, 1), 60000), 1_200_000 // (batch * kv))
        return _attn_drawn(batch, max(1, min(n, length)), kv * group, kv, d, length, rng)
    if kind == "chunk":
        batch = min(batch, 4)
        n = min(_log(rng, 41, 4700), math.isqrt(1_000_000_000 // (batch * kv * group)))
        length = max(n, min(_log(rng, n, 31200), 1_000_000_000 // (batch * kv * group * n), 1_200_000 // (batch * kv)))
        return _attn_drawn(batch, n, kv * group, kv, d, length, rng)
    if kind == "append":
        n = _log(rng, 1, 4680)
        length = max(n, min(_log(rng, n, 31200), 1_200_000 // (batch * kv)))
        n = min(n, max(1, 190_000 // (batch * kv)))
        return _append("", batch, n, kv, d, length, rng.random() < 0.5, rng.random() < 0.3) | {"name": ""}
    length = max(2, min(_log(rng, 60, 60000), 1_200_000 // (batch * kv)))
    keep = rng.randint(1, length)
    return _evict("", batch, kv, d, length, rng.random() < 0.5, keep, rng.randint(0, keep)) | {"name": ""}


def _attn_drawn(batch, n, heads, kv, d, length, rng):
    return _attn("", batch, n, heads, kv, d, length, rng.random() < 0.5, rng.random() < 0.6, rng.random() < 0.3,
                 rng.random() < 0.4)


# ---- inputs ----------------------------------------------------------------


def _lengths(c):
    """Rows held when the pass is over (attn, append) or before it (evict): the longest first, the others anywhere
    below it; in a ragged attention batch of four or more one sequence holds nothing."""
    got = []
    for b in range(c["batch"]):
        x = c["length"]
        if c["ragged"] and b:
            x = 1 + (x - 1) * ((b * 7919 + 3) % 101) // 101
        got.append(x)
    if c["ragged"] and c["batch"] >= 4 and c["op"] == "attn":
        got[3] = 0
    return got


def _counts(c):
    """New rows of every sequence: at most n and at most what it holds; fewer in a padded batch."""
    return [min(x, c["n"] if not (c["padded"] and b) else (c["n"] * (17 - (b * 31 + 7) % 17)) // 17)
            for b, x in enumerate(_lengths(c))]


def _pow2(amax):
    """2^e for the smallest e with amax <= 448 * 2^e, within the bounds."""
    m, e = torch.frexp(amax.float())  # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    return torch.ldexp(torch.ones_like(m), e)


def _codes(x, scale):
    """e4m3 codes of x / scale (nearest, ties to even), saturating."""
    return (x.float() / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _rows(c, n, gen, dev, keys):
    """bf16 rows as a model makes them: a few loud channels in keys, a slow drift along the sequence."""
    x = torch.randn((c["batch"], n, c["kv_heads"], c["d"]), generator=gen, device=dev)
    if keys:
        x = x * (0.5 + 1.5 * torch.rand((c["kv_heads"], c["d"]), generator=gen, device=dev) ** 4)
    x = x * torch.exp(0.4 * torch.sin(torch.arange(n, device=dev) / 97.0))[None, :, None, None]
    return x.to(torch.bfloat16)


def _packed(x, capacity):
    """Codes and scales of rows [batch, n, kv_heads, d] laid out in blocks, capacity rows."""
    b, n, h, d = x.shape
    blocks = -(-capacity // BLOCK)
    full = torch.zeros((b, blocks * BLOCK, h, d), dtype=x.dtype, device=x.device)
    full[:, :n] = x
    full = full.reshape(b, blocks, BLOCK, h, d).transpose(2, 3).contiguous()
    scale = _pow2(full.abs().amax((3, 4)))
    return _codes(full, scale[..., None, None]), scale


def _capacity(c):
    return -(-(c["length"] + BLOCK + (c["n"] if c["op"] == "append" and c["padded"] else 0)) // BLOCK) * BLOCK


def _read_back(c):
    """Rows read back after an append: every sequence's touched blocks, from the start of the first one."""
    return c["n"] + BLOCK - 1


def prepare(case, seed):
    c = case
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    lengths, cap = _lengths(c), _capacity(c)
    held = lengths
    st = dict(case=c, dev=dev, capacity=cap)
    if c["op"] != "evict":
        counts = _counts(c)
        st["count_of"] = torch.tensor(counts, dtype=torch.int32, device=dev)
        st["counts"] = None if min(counts) == c["n"] else st["count_of"]
    if c["op"] == "append":
        held = [x - y for x, y in zip(lengths, counts)]
        st["start"] = torch.tensor(held, dtype=torch.int32, device=dev)
        st["k"], st["v"] = _rows(c, c["n"], gen, dev, True), _rows(c, c["n"], gen, dev, False)
    st["lengths"] = torch.tensor(held, dtype=torch.int32, device=dev)
    st["k8"], st["k_scale"] = _packed(_rows(c, c["length"], gen, dev, True), cap)
    st["v8"], st["v_scale"] = _packed(_rows(c, c["length"], gen, dev, False), cap)
    shape = (c["batch"], c["n"], c["heads"], c["d"])
    if c["op"] == "attn":
        st["q"] = (1.3 * torch.randn(shape, generator=gen, device=dev)).to(torch.bfloat16)
        st["out"] = torch.zeros(shape, dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.zeros(shape[:3], dtype=torch.float32, device=dev)
        if c["weigh"]:
            w = torch.rand((c["batch"], c["kv_heads"], cap), generator=gen, device=dev)
            st["weights_in"] = w * (torch.arange(cap, device=dev) < st["lengths"][:, None, None])
            st["weights"] = st["weights_in"].clone()
    elif c["op"] == "append":
        st["first"] = st["start"] // BLOCK * BLOCK
        rows = (c["batch"], _read_back(c), c["kv_heads"], c["d"])
        st["k_out"] = torch.zeros(rows, dtype=torch.bfloat16, device=dev)
        st["v_out"] = torch.zeros(rows, dtype=torch.bfloat16, device=dev)
    else:
        # accumulated weights: most of the mass on a few rows, many small ones equal to each other
        u = torch.rand((c["batch"], c["kv_heads"], cap), generator=gen, device=dev)
        w = torch.where(u < 0.3, torch.full_like(u, 0.0625), torch.exp(6.0 * u) / 40.0)
        st["weights"] = w * (torch.arange(cap, device=dev) < st["lengths"][:, None, None])
        st["keep_cap"] = -(-c["keep"] // BLOCK) * BLOCK
        shape = (c["batch"], c["kv_heads"])
        st["kept"] = torch.zeros((*shape, c["keep"]), dtype=torch.int32, device=dev)
        st["weights_out"] = torch.zeros((*shape, st["keep_cap"]), dtype=torch.float32, device=dev)
        rows = (c["batch"], c["keep"], c["kv_heads"], c["d"])
        st["k_out"] = torch.zeros(rows, dtype=torch.bfloat16, device=dev)
        st["v_out"] = torch.zeros(rows, dtype=torch.bfloat16, device=dev)
    if own:
        from kv_cache_attention_ff_gb300 import ff
        desc = dict(batch=c["batch"], heads=c["heads"], kv_heads=c["kv_heads"], head_dim=c["d"])
        st["cache"] = ff.KV8Cache(capacity=cap, max_tokens=c["n"], **desc)
        k8, v8, k_scale, v_scale, length = st["cache"].layer(0)
        k8.copy_(st["k8"].view(torch.uint8))
        v8.copy_(st["v8"].view(torch.uint8))
        k_scale.copy_(st["k_scale"])
        v_scale.copy_(st["v_scale"])
        length.copy_(st["lengths"])
        if c["op"] == "evict":
            st["kept_cache"] = ff.KV8Cache(capacity=st["keep_cap"], max_tokens=1, **desc)
        torch.cuda.synchronize()
        for name in ("k8", "v8", "k_scale", "v_scale"):
            del st[name]
    return st


# ---- the plain forms ---------------------------------------------------------


def _values(k8, scale):
    """fp32 values [batch, kv_heads, rows, d] of codes in blocks."""
    x = k8.float() * scale[..., None, None]
    b, blocks, h, _, d = x.shape
    return x.transpose(1, 2).reshape(b, h, blocks * BLOCK, d)


def _plain_attn(st):
    c, dev = st["case"], st["dev"]
    group, rows = c["heads"] // c["kv_heads"], c["length"]
    k = _values(st["k8"], st["k_scale"])[:, :, :rows]
    v = _values(st["v8"], st["v_scale"])[:, :, :rows]
    q = st["q"].float().reshape(c["batch"], c["n"], c["kv_heads"], group, c["d"]).permute(0, 2, 3, 1, 4)
    s = torch.matmul(q.reshape(c["batch"], c["kv_heads"], group * c["n"], c["d"]), k.transpose(2, 3))
    s = s.reshape(c["batch"], c["kv_heads"], group, c["n"], rows) * (1.0 / math.sqrt(c["d"]))
    i = torch.arange(c["n"], device=dev)
    length, count = st["lengths"][:, None], st["count_of"][:, None]
    seen = (length - count + i + 1 if c["causal"] else length + 0 * i).clamp(min=0)  # [batch, n]
    seen = torch.where(i < count, seen, torch.zeros_like(seen))[:, None, None, :, None]
    hidden = torch.arange(rows, device=dev) >= seen
    s.masked_fill_(hidden, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(seen > 0, m, torch.zeros_like(m))
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(seen > 0, l, torch.ones_like(l))
    o = torch.matmul(p.reshape(c["batch"], c["kv_heads"], group * c["n"], rows), v)
    o = o.reshape(c["batch"], c["kv_heads"], group, c["n"], c["d"]).permute(0, 3, 1, 2, 4)
    o = o.reshape(c["batch"], c["n"], c["heads"], c["d"])
    lse = torch.where(seen > 0, m + torch.log(l), torch.full_like(l, -math.inf))[..., 0]
    lse = lse.permute(0, 3, 1, 2).reshape(c["batch"], c["n"], c["heads"])
    valid = (i < count)[:, :, None]
    got = [torch.where(valid[..., None], o.to(torch.bfloat16), st["out"]), torch.where(valid, lse, st["lse"])]
    if c["weigh"]:
        w = st["weights_in"].clone()
        w[:, :, :rows] += p.sum((2, 3))
        got.append(w)
    return got


def _plain_load(k8, scale, lengths, start, n):
    row = start[:, None].long() + torch.arange(n, device=k8.device)
    held = row < lengths[:, None]
    row = torch.where(held, row, torch.zeros_like(row))
    b = torch.arange(k8.shape[0], device=k8.device)[:, None]
    x = k8.view(torch.uint8)[b, row // BLOCK, :, row % BLOCK].view(torch.float8_e4m3fn)
    x = x.float() * scale[b, row // BLOCK][..., None]
    return torch.where(held[:, :, None, None], x, torch.zeros_like(x)).to(torch.bfloat16)


def _plain_append(st):
    c, dev = st["case"], st["dev"]
    blocks = (c["n"] + 2 * BLOCK - 2) // BLOCK  # as many as the new rows may touch
    start, count = st["start"].long(), st["count_of"].long()
    b = torch.arange(c["batch"], device=dev)[:, None]
    at = start[:, None] // BLOCK + torch.arange(blocks, device=dev)  # [batch, blocks]
    touched = ((at * BLOCK < (start + count)[:, None]) & (count > 0)[:, None])[..., None]
    before = (at * BLOCK < start[:, None])[..., None]
    row = at[:, :, None] * BLOCK + torch.arange(BLOCK, device=dev)
    fresh = (row >= start[:, None, None]) & (row < (start + count)[:, None, None])
    source = (row - start[:, None, None]).clamp(0, c["n"] - 1)
    for new, codes, scales in ((st["k"], "k8", "k_scale"), (st["v"], "v8", "v_scale")):
        x = new.float()[b[:, :, None], source]  # [batch, blocks, 64, kv_heads, d]
        x = torch.where(fresh[..., None, None], x, torch.zeros_like(x)).transpose(2, 3)
        bits, old_scale = st[codes].view(torch.uint8)[b, at], st[scales][b, at]
        scale = _pow2(x.abs().amax((3, 4)))
        scale = torch.where(before, torch.maximum(scale, old_scale), scale)
        old = bits.view(torch.float8_e4m3fn).float() * (old_scale / scale)[..., None, None]
        x = torch.where(fresh[:, :, None, :, None], x / scale[..., None, None], old).clamp(-448.0, 448.0)
        # rows past the new ones stay as they were
        code = x.to(torch.float8_e4m3fn).view(torch.uint8)
        written = (row < (start + count)[:, None, None])[:, :, None, :, None] & touched[..., None, None]
        st[codes].view(torch.uint8)[b, at] = torch.where(written, code, bits)
        st[scales][b, at] = torch.where(touched, scale, old_scale)
    st["lengths"] = st["start"] + st["count_of"]
    got = [_plain_load(st[codes], st[scales], st["lengths"], st["first"], _read_back(c))
           for codes, scales in (("k8", "k_scale"), ("v8", "v_scale"))]
    return [*got, st["lengths"]]


def _plain_evict(st):
    c, dev = st["case"], st["dev"]
    cap, keep = st["capacity"], c["keep"]
    j = torch.arange(cap, device=dev)
    length = st["lengths"].long()[:, None, None]
    recent = (j >= length - c["recent"]) & (j < length)
    key = torch.where(recent, torch.full_like(st["weights"], math.inf), st["weights"])
    key = torch.where(j < length, key, torch.full_like(key, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.where(j[:keep] < length, order, torch.full_like(order, cap)).sort(-1).values
    count = length.clamp(max=keep)
    held = j[:keep] < count
    at = torch.where(held, kept, torch.zeros_like(kept))
    weights = torch.zeros_like(st["weights_out"])
    weights[..., :keep] = torch.where(held, st["weights"].gather(-1, at), torch.zeros_like(weights[..., :keep]))
    got = [torch.where(held, kept, torch.full_like(kept, -1)).to(torch.int32), weights,
           count[:, 0, 0].to(torch.int32)]
    for codes, scales in (("k8", "k_scale"), ("v8", "v_scale")):
        x = _values(st[codes], st[scales])  # [batch, h, rows, d]
        x = x.gather(2, at[..., None].expand(-1, -1, -1, c["d"]))
        x = torch.where(held[..., None], x, torch.zeros_like(x))
        x = torch.nn.functional.pad(x, (0, 0, 0, st["keep_cap"] - keep))
        x = x.reshape(c["batch"], c["kv_heads"], -1, BLOCK, c["d"])
        scale = _pow2(x.abs().amax((3, 4)))[..., None, None]
        x = (_codes(x, scale).float() * scale).reshape(c["batch"], c["kv_heads"], st["keep_cap"], c["d"])
        got.append(x[:, :, :keep].transpose(1, 2).to(torch.bfloat16))
    return got


# ---- one pass ------------------------------------------------------------------


def run(st):
    c = st["case"]
    if not own:
        return {"attn": _plain_attn, "append": _plain_append, "evict": _plain_evict}[c["op"]](st)
    cache = st["cache"]
    if c["op"] == "attn":
        if c["weigh"]:
            cache.attn(0, st["q"], st["out"], causal=c["causal"], counts=st["counts"], lse=st["lse"],
                       weights=st["weights"], weights_in=st["weights_in"])
            return [st["out"], st["lse"], st["weights"]]
        cache.attn(0, st["q"], st["out"], causal=c["causal"], counts=st["counts"], lse=st["lse"])
        return [st["out"], st["lse"]]
    if c["op"] == "append":
        cache.append(0, st["k"], st["v"], start=st["start"], counts=st["counts"])
        cache.load(0, st["k_out"], st["v_out"], start=st["first"])
        return [st["k_out"], st["v_out"], cache.lengths(0)]
    kept = st["kept_cache"]
    cache.evict(0, kept, 0, c["keep"], c["recent"], st["weights"], st["weights_out"], st["kept"])
    kept.load(0, st["k_out"], st["v_out"])
    return [st["kept"], st["weights_out"], kept.lengths(0), st["k_out"], st["v_out"]]


def work(case):
    c = case
    lengths = _lengths(c)
    row = c["kv_heads"] * 2 * c["d"]  # values of K and V in a row of the cache
    held = sum(lengths)
    scales = sum(-(-x // BLOCK) for x in lengths) * c["kv_heads"] * 2 * 4
    if c["op"] == "attn":
        counts = _counts(c)
        queries = sum(counts) * c["heads"]
        pairs = 0
        for x, m in zip(lengths, counts):
            pairs += sum(max(0, x - m + i + 1) for i in range(m)) if c["causal"] else x * m
        weigh = held * c["kv_heads"] * 8 if c["weigh"] else 0
        return {"bytes": held * row + scales + queries * (4 * c["d"] + 4) + weigh, "flops": 4 * c["d"] * pairs * c["heads"]}
    if c["op"] == "append":
        counts = _counts(c)
        values = c["batch"] * _read_back(c) * row
        return {"bytes": sum(counts) * row * 3 + values * 2, "flops": values * 2}
    kept = sum(min(x, c["keep"]) for x in lengths)
    return {"bytes": held * c["kv_heads"] * 4 + kept * row * (1 + 1 + 2) + kept * c["kv_heads"] * 8,
            "flops": held * c["kv_heads"] + kept * row * 2}


# ---- the definitions in 64 bits --------------------------------------------------


def _nearest8(x):
    """x (64 bits, at most 448 in magnitude after clamping) rounded to the nearest e4m3 number, ties to even."""
    x = x.clamp(-448.0, 448.0)
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _block_scale(rows):
    """The scale of a block from its values in 64 bits."""
    top = float(rows.abs().max()) if rows.numel() else 0.0
    return 2.0 ** max(E_MIN, min(E_MAX, math.ceil(math.log2(top / 448.0)))) if top else 2.0 ** E_MIN


def _exact_append(c, st):
    got = []
    for new, codes, scales, out in ((st["k"], "k8", "k_scale", "k_out"), (st["v"], "v8", "v_scale", "v_out")):
        rows = torch.zeros(st[out].shape, dtype=torch.float64, device=st["dev"])
        for b, (length, count) in enumerate(zip(_lengths(c), _counts(c))):
            start, first = length - count, (length - count) // BLOCK * BLOCK
            for t in range(first, length, BLOCK):
                stay = max(start - t, 0)
                end = min(length, t + BLOCK)
                for h in range(c["kv_heads"]):
                    old = st[codes][b, t // BLOCK, h, :stay].double() * float(st[scales][b, t // BLOCK, h])
                    x = new[b, t + stay - start:end - start, h].double()
                    scale = _block_scale(x)
                    if stay:
                        scale = max(scale, float(st[scales][b, t // BLOCK, h]))
                    x = torch.cat([old, x]) if count else old
                    rows[b, t - first:t - first + len(x), h] = _nearest8(x / scale) * scale
        got.append(rows)
    return [*got, None]


def _exact_evict(c, st):
    got = [torch.zeros(st[a].shape, dtype=torch.float64, device=st["dev"]) for a in ("weights_out", "k_out", "v_out")]
    for b, length in enumerate(_lengths(c)):
        for h in range(c["kv_heads"]):
            w = st["weights"][b, h, :length].double()
            kept = torch.arange(length, device=st["dev"])
            if length > c["keep"]:
                old = length - c["recent"]
                top = torch.sort(-w[:old], stable=True).indices[:c["keep"] - c["recent"]]
                kept = torch.cat([top.sort().values, kept[old:]])
            got[0][b, h, :len(kept)] = w[kept]
            for to, codes, scales in ((got[1], "k8", "k_scale"), (got[2], "v8", "v_scale")):
                x = (st[codes][b, :, h].double() * st[scales][b, :, h].double()[:, None, None]).reshape(-1, c["d"])[kept]
                for t in range(0, len(kept), BLOCK):
                    scale = _block_scale(x[t:t + BLOCK])
                    to[b, t:min(t + BLOCK, len(kept)), h] = _nearest8(x[t:t + BLOCK] / scale) * scale
    return [None, got[0], None, got[1], got[2]]


def exact(case, seed):
    """The definitions in 64 bits, one head after the other; None where whole numbers come back, and for cases of many blocks."""
    global own
    c, was = case, own
    own = False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if c["op"] != "attn":
        blocks = c["batch"] * c["kv_heads"] * (c["n"] // BLOCK + 2 if c["op"] == "append" else c["keep"] // BLOCK + 1)
        if blocks > 15000:
            return None
        return _exact_append(c, st) if c["op"] == "append" else _exact_evict(c, st)
    out, lse = st["out"].double(), st["lse"].double()
    w = st["weights_in"].double() if c["weigh"] else None
    group = c["heads"] // c["kv_heads"]
    for b, (length, count) in enumerate(zip(_lengths(c), _counts(c))):
        if not count:
            continue
        for h in range(c["kv_heads"]):
            k, v = (st[a][b, :, h].double().mul(st[s][b, :, h].double()[:, None, None]).reshape(-1, c["d"])[:length]
                    for a, s in (("k8", "k_scale"), ("v8", "v_scale")))
            for g in range(h * group, (h + 1) * group):
                s = (st["q"][b, :count, g].double() @ k.T).div_(math.sqrt(c["d"]))
                if c["causal"]:
                    s += torch.full_like(s, -math.inf).triu_(length - count + 1)
                top = torch.logsumexp(s, 1)
                p = s.sub_(top[:, None]).exp_()
                lse[b, :count, g] = top
                out[b, :count, g] = p @ v
                if w is not None:
                    w[b, h, :length] += p.sum(0)
    return [out, lse] if w is None else [out, lse, w]
