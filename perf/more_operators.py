"""Prompts and shared prefixes over a paged cache: what is measured of them, and their plain forms.

Two operators beside the attention of single tokens over the cache:

  prompt_attn    causal attention of every request's new tokens (a whole prompt, a further chunk of one, a single
                 token), packed one request behind the other, over the request's rows in the pages
  prefix_attn    attention of one new token a row over a prefix that many rows share, and the row's own pages

``run`` computes them in elementary torch operations, in 32 bits and rounded once at the end, or (``own``) calls
this repository's package.  ``exact`` computes them in 64 bits, a head of a request or of a row at a time.
"""
import random

import torch

own = False

# ------------------------------------------------------------------------------------------------ cases


def _prompt(name, fresh, lo, hi, heads, kv_heads, hd, page, chunks=0, chunk=0, clo=0, chi=0, decode=0, dlo=0, dhi=0, idle=0,
            pad=0, window=0, sink=False, head_major=False):
    """fresh prompts of lo to hi tokens, `chunks` of about `chunk` tokens behind clo to chi earlier ones, `decode` single
    tokens behind dlo to dhi, `idle` requests without a token, `pad` rows behind the last."""
    return dict(name=name, op="prompt_attn", fresh=fresh, lo=lo, hi=hi, heads=heads, kv_heads=kv_heads, hd=hd, page=page,
                chunks=chunks, chunk=chunk, clo=clo, chi=chi, decode=decode, dlo=dlo, dhi=dhi, idle=idle, pad=pad,
                window=window, sink=sink, head_major=head_major)


def _prefix(name, n, prefixes, plen, lo, hi, heads, kv_heads, hd, page, window=0, sink=False, head_major=False):
    """n rows over `prefixes` prefixes, the longest of plen rows, each with lo to hi rows of its own."""
    return dict(name=name, op="prefix_attn", n=n, prefixes=prefixes, plen=plen, lo=lo, hi=hi, heads=heads,
                kv_heads=kv_heads, hd=hd, page=page, window=window, sink=sink, head_major=head_major)


def listed():
    return [
        # one short question: the latency of the whole chain of loads
        _prompt("prompt 1 x 17", 1, 17, 17, 16, 4, 64, 16),
        # a prefill step of a chat server: prompts of very different lengths, four query heads to a key head
        _prompt("prompt 12 ragged gqa", 12, 100, 4000, 32, 8, 128, 16),
        # one long document
        _prompt("prompt 16k", 1, 16384, 16384, 64, 8, 128, 64),
        # chunked prefill: few new tokens behind much that the cache already holds, odd sizes
        _prompt("prompt chunks", 0, 0, 0, 32, 4, 128, 32, chunks=6, chunk=389, clo=5000, chi=30000),
        # wide heads, a key head for each query head, a sliding window with sinks, odd pages, pages stored a head at a time
        _prompt("prompt window mha 256", 5, 1, 6001, 16, 16, 256, 17, idle=1, window=1000, sink=True, head_major=True),
        # a mixed step: decodes beside two prompt chunks, five query heads to a key head, a head size off the powers of two
        _prompt("prompt mixed step", 1, 700, 700, 40, 8, 80, 16, chunks=1, chunk=513, clo=3000, chi=3000, decode=64, dlo=1,
                dhi=5000, idle=3, pad=19),
        # two turns behind a short system prompt
        _prefix("prefix 2 x 500", 2, 1, 500, 20, 31, 16, 4, 64, 16),
        # a chat server's batch behind one long system prompt
        _prefix("prefix 64 x 8k", 64, 1, 8192, 40, 700, 32, 8, 128, 16),
        # many questions about one document: the largest
        _prefix("prefix 256 x 32k", 256, 1, 32768, 100, 2000, 64, 8, 128, 64),
        # three prefixes of odd lengths, one of them empty, wide heads, a window that ends inside the prefix, sinks
        _prefix("prefix groups window 192", 45, 3, 7001, 0, 3500, 20, 4, 192, 17, window=4096, sink=True, head_major=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    """One more case of the same ranges: one token to long prompts, rows and prefixes, any page and head layout."""
    hd = rng.choice([64, 64, 72, 80, 96, 128, 128, 192, 256])
    kv = rng.choice([1, 2, 4, 8, 16])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 20])
    page = rng.choice([1, 8, 16, 17, 32, 64, 128, 256])
    window = rng.choice([0, 0, 0, _log(rng, 1, 8192)])
    kw = dict(window=window, sink=rng.random() < 0.4, head_major=rng.random() < 0.4)
    row = kv * hd * 4  # bytes of a row's keys and values
    if rng.random() < 0.6:
        hi = 1
        while hi < 16384 and (2 * hi) ** 2 * kv * g * hd < 5e11 and 2 * hi * row * (1 + g) < 2e9:
            hi *= 2
        kind = rng.choice(["fresh", "chunks", "mixed"])
        top = _log(rng, 1, hi)
        fresh = 0 if kind == "chunks" else _log(rng, 1, max(1, min(24, (hi * hi) // (top * top))))
        chunk = _log(rng, 1, 600)
        back = _log(rng, 1, max(2, min(32000, int(5e11 / (600 * 8 * kv * g * hd)), 800_000_000 // (8 * row))))
        chunks = 0 if kind == "fresh" else rng.randint(1, 8)
        decode = rng.randint(1, 48) if kind == "mixed" else 0
        dhi = _log(rng, 1, max(2, min(8000, 400_000_000 // (max(1, decode) * row))))
        return _prompt("", fresh, _log(rng, 1, top), top, kv * g, kv, hd, page, chunks=chunks, chunk=chunk,
                       clo=_log(rng, 1, back), chi=back, decode=decode, dlo=0, dhi=dhi, idle=rng.choice([0, 0, 2]),
                       pad=rng.choice([0, 0, rng.randint(1, 40)]), **kw)
    n = _log(rng, 1, 256)
    hi = _log(rng, 1, max(2, min(4000, 600_000_000 // (n * row))))
    plen = _log(rng, 1, max(2, min(32768, int(1e11 / (n * kv * g * hd)), 400_000_000 // row)))
    return _prefix("", n, rng.choice([1, 1, 1, 2, 5]), plen, rng.choice([0, _log(rng, 1, hi)]), hi, kv * g, kv, hd, page, **kw)


def _lengths(n, lo, hi):
    """n lengths from lo to hi, evenly spread over their logarithm (zero and one included where lo is 0)."""
    if n <= 1:
        return [hi] * n
    a = max(lo, 1)
    v = [int(round(a * (hi / a) ** (i / (n - 1)))) if hi >= a else hi for i in range(n)]
    if lo == 0:
        v[0] = 0
    return v


def _shuffled(v, seed):
    v = list(v)
    random.Random(seed).shuffle(v)
    return v


def _requests(c):
    """(new tokens, rows after the step) of every request of a prompt case."""
    a = [(max(x, 1), max(x, 1)) for x in _lengths(c["fresh"], c["lo"], c["hi"])]
    new = [max(1, c["chunk"] - 3 * i) for i in range(c["chunks"])]
    a += [(x, b + x) for x, b in zip(new, _lengths(c["chunks"], c["clo"], c["chi"]))]
    a += [(1, b + 1) for b in _lengths(c["decode"], c["dlo"], c["dhi"])]
    return a + [(0, 40 * i) for i in range(c["idle"])]


def _prefix_lengths(c):
    """Rows of each prefix: the first has plen, the last none if there are three or more."""
    k = c["prefixes"]
    v = [max(1, (c["plen"] * (k - i)) // k) for i in range(k)]
    if k >= 3:
        v[-1] = 0
    return v


def _prefix_rows(c):
    """First row of each prefix's batch, and the end of the last."""
    k = c["prefixes"]
    return [(c["n"] * i) // k for i in range(k)] + [c["n"]]


# ------------------------------------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(torch.bfloat16)


def _pages(g, c, n_pages):
    """A cache tensor [page][row][head][feature]; head_major: stored with a head's rows of a page side by side."""
    if c["head_major"]:
        return _bf(g, n_pages, c["kv_heads"], c["page"], c["hd"]).transpose(1, 2)
    return _bf(g, n_pages, c["page"], c["kv_heads"], c["hd"])


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(g, counts, spare):
    """Block tables for lists of page counts (one list a table) over one pool, with spare pages, and the pool's size."""
    total = sum(map(sum, counts))
    perm = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    tables, used = [], 0
    for per in counts:
        width = max(per) + 2
        t = torch.zeros(len(per), width, dtype=torch.int32, device="cuda")
        t[torch.arange(width, device="cuda")[None, :] < _i32(per)[:, None]] = perm[used:used + sum(per)]
        used += sum(per)
        tables.append(t)
    return tables, total + spare


def prepare(case, seed):
    g, page = _gen(seed), case["page"]
    H, hd = case["heads"], case["hd"]
    sink = torch.randn(H, generator=g, device="cuda") if case["sink"] else None
    if case["op"] == "prompt_attn":
        reqs = _shuffled(_requests(case), seed)
        new, rows = [x for x, _ in reqs], [y for _, y in reqs]
        (table,), n_pages = _tables(g, [[-(-y // page) for y in rows]], 5)
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        n = cu[-1] + case["pad"]
        # the query heads of a fused projection's rows, read as a strided view
        q = _bf(g, n, (H + 2 * case["kv_heads"]) * hd, scale=1.5)[:, :H * hd].view(n, H, hd)
        return dict(case, q=q, k=_pages(g, case, n_pages), v=_pages(g, case, n_pages), table=table, cu=_i32(cu), length=_i32(rows),
                    at=cu, rows=rows, sink_w=sink, scale=hd ** -0.5, out=torch.zeros(n, H, hd, dtype=torch.bfloat16, device="cuda"),
                    lse=torch.zeros(n, H, device="cuda"))
    lens = _shuffled(_lengths(case["n"], case["lo"], case["hi"]), seed)
    plens = _prefix_lengths(case)
    (table, prefix), n_pages = _tables(g, [[-(-x // page) for x in lens], [-(-x // page) for x in plens]], 5)
    return dict(case, q=_bf(g, case["n"], H, hd, scale=1.5), k=_pages(g, case, n_pages), v=_pages(g, case, n_pages), table=table,
                pos=_i32([x - 1 for x in lens]), prefix=prefix, prefix_len=_i32(plens), cu=_i32(_prefix_rows(case)),
                at=_prefix_rows(case), rows=lens, plens=plens, sink_w=sink, scale=hd ** -0.5)


# ------------------------------------------------------------------------------------------------ run

_context = None


def _ctx():
    """The library context that a program keeps."""
    global _context
    if _context is None:
        import compressed_sparse_attention_attn_gb300 as csa
        _context = csa.Context(dict(dim=512, n_heads=1, head_dim=512, rope_dim=64, q_rank=64, o_rank=64, groups=1,
                                    window=128, eps=1e-6, index_heads=0, index_hd=0, index_topk=0, cand_block=64,
                                    max_seq=16, max_tokens=1, max_batch=1, rope_theta=10000.0,
                                    compress_rope_theta=10000.0, rope_factor=1.0, beta_fast=32.0, beta_slow=1.0))
    return _context


def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _cache(s):
    import compressed_sparse_attention_attn_gb300 as csa
    if "cache" not in s:
        s["cache"] = csa.PagedCache(s["k"], s["v"])
    return s["cache"]


def _own_prompt(s):
    o, lse = _ctx().prompt_attn(s["q"], _cache(s), s["table"], s["cu"], s["length"], s["scale"], sink=s["sink_w"],
                                window=s["window"], out=s["out"], lse=s["lse"])
    return {"o": o, "lse": lse}


def _own_prefix(s):
    o, lse = _ctx().prefix_attn(s["q"], _cache(s), s["table"], s["pos"], s["prefix"], s["prefix_len"], s["scale"],
                                cu=s["cu"] if s["prefixes"] > 1 else None, sink=s["sink_w"], window=s["window"], with_lse=True)
    return {"o": o, "lse": lse}


def _gather(pages, table, n, page):
    """Rows 0 .. n-1 behind a table row, in 32 bits: [kv][n][hd]."""
    p = torch.arange(n, device=table.device)
    return pages[table.long()[p // page], p % page].float().transpose(0, 1)


def _softmax(score, sink):
    """Weights over the last axis of [kv][g][...][rows], their sum without and with the sink's term, and the maximum."""
    top = score.amax(-1, keepdim=True)
    if sink is not None:
        sink = sink.view(sink.shape + (1,) * (score.dim() - 2))
        top = torch.maximum(top, sink)
    top = top.masked_fill(top == float("-inf"), 0.0)  # (a row without a position: its weights are all 0)
    weight = (score - top).exp()
    total = weight.sum(-1, keepdim=True)
    below = total if sink is None else total + (sink - top).exp()
    return weight, total, below.masked_fill(below == 0, 1.0), top


def _attend(q, keys, values, seen, s):
    """q [t][H][hd] over rows [kv][n][hd] that `seen` [t][n] marks: o [t][H][hd], lse [t][H]."""
    t, H, hd = q.shape
    kv = s["kv_heads"]
    qs = q.float().view(t, kv, H // kv, hd).permute(1, 2, 0, 3).reshape(kv, -1, hd)
    score = (torch.matmul(qs, keys.transpose(1, 2)) * s["scale"]).view(kv, H // kv, t, -1).masked_fill(~seen, float("-inf"))
    weight, total, below, top = _softmax(score, None if s["sink_w"] is None else s["sink_w"].view(kv, H // kv))
    o = torch.matmul(weight.view(kv, (H // kv) * t, -1), values).view(kv, H // kv, t, hd) / below
    lse = (top + total.log()).squeeze(-1)
    return o.permute(2, 0, 1, 3).reshape(t, H, hd).to(torch.bfloat16), lse.permute(2, 0, 1).reshape(t, H)


def _plain_prompt(s):
    """A request at a time, its rows gathered through the table, its tokens in blocks that bound the scores' memory."""
    for r, (a, b, n) in enumerate(zip(s["at"], s["at"][1:], s["rows"])):
        if a == b:
            continue
        keys, values = (_gather(s[x], s["table"][r], n, s["page"]) for x in "kv")
        step = max(1, (1 << 28) // (s["heads"] * n))
        for t0 in range(a, b, step):
            t1 = min(b, t0 + step)
            pos = (torch.arange(t0, t1, device="cuda") + (n - b))[:, None]
            j = torch.arange(n, device="cuda")[None, :]
            seen = (j <= pos) & (j > pos - s["window"]) if s["window"] else j <= pos
            s["out"][t0:t1], s["lse"][t0:t1] = _attend(s["q"][t0:t1], keys, values, seen, s)
    return {"o": s["out"], "lse": s["lse"]}


def _plain_prefix(s):
    """A prefix at a time: the scores of all its rows over the prefix in one product, those over the rows' own pages in
    another (padded to the longest), one softmax over both."""
    H, hd, kv = s["heads"], s["hd"], s["kv_heads"]
    o = torch.empty_like(s["q"])
    lse = torch.empty(s["n"], H, device="cuda")
    for i, (a, b, L) in enumerate(zip(s["at"], s["at"][1:], s["plens"])):
        keys, values = (_gather(s[x], s["prefix"][i], L, s["page"]) for x in "kv")
        step = max(1, (1 << 28) // max(1, H * L, 2 * kv * hd * max(s["rows"][a:b], default=0)))
        for t0 in range(a, b, step):
            t1 = min(b, t0 + step)
            t, pos, m = t1 - t0, s["pos"][t0:t1].long()[:, None], max(1, *s["rows"][t0:t1])
            q = s["q"][t0:t1].float().view(t, kv, H // kv, hd)
            first = pos + L + 1 - s["window"] if s["window"] else torch.zeros_like(pos)  # over prefix and own rows together
            at = torch.arange(m, device="cuda").expand(t, m)
            seen = (at <= pos) & (at + L >= first)
            page_id = s["table"][t0:t1].long().gather(1, at // s["page"])
            mine, held = (s[x][page_id, at % s["page"]].float().permute(0, 2, 1, 3) for x in "kv")  # [t][kv][m][hd]
            one = torch.matmul(q.permute(1, 2, 0, 3).reshape(kv, H // kv * t, hd), keys.transpose(1, 2)).view(kv, H // kv, t, L)
            one = one.masked_fill(torch.arange(L, device="cuda")[None, :] < first, float("-inf"))
            two = torch.matmul(q, mine.transpose(2, 3)).masked_fill(~seen[:, None, None], float("-inf")).permute(1, 2, 0, 3)
            weight, total, below, top = _softmax(torch.cat([one, two], -1) * s["scale"],
                                                 None if s["sink_w"] is None else s["sink_w"].view(kv, H // kv))
            x = torch.matmul(weight[..., :L].reshape(kv, H // kv * t, L), values).view(kv, H // kv, t, hd)
            x = x + torch.matmul(weight[..., L:].permute(2, 0, 1, 3), held * seen[:, None, :, None]).permute(1, 2, 0, 3)
            o[t0:t1] = (x / below).permute(2, 0, 1, 3).reshape(t, H, hd).to(torch.bfloat16)
            lse[t0:t1] = (top + total.log()).squeeze(-1).permute(2, 0, 1).reshape(t, H)
    return {"o": o, "lse": lse}


_plain = {"prompt_attn": _plain_prompt, "prefix_attn": _plain_prefix}
_own = {"prompt_attn": _own_prompt, "prefix_attn": _own_prefix}


# ------------------------------------------------------------------------------------------------ work


def _pairs(new, rows, window):
    """Rows attended by a request's tokens in all, and those that any of them attends."""
    first = rows - new
    if not window:
        return new * first + new * (new + 1) // 2, rows if new else 0
    full = max(0, min(new, rows - window))  # tokens with a whole window before them
    part = new - full
    return full * window + part * first + part * (part + 1) // 2, min(rows, window + new - 1) if new else 0


def work(c):
    row, H, hd = c["kv_heads"] * c["hd"] * 4, c["heads"], c["hd"]
    if c["op"] == "prompt_attn":
        reqs = _requests(c)
        pairs = [_pairs(x, y, c["window"]) for x, y in reqs]
        seen, n = sum(p[1] for p in pairs), sum(x for x, _ in reqs)
        return {"bytes": seen * row + n * H * (4 * hd + 4) + sum(-(-p[1] // c["page"]) * 4 for p in pairs) + 8 * len(reqs),
                "flops": 4 * H * hd * sum(p[0] for p in pairs)}
    lens, plens, at, w = _lengths(c["n"], c["lo"], c["hi"]), _prefix_lengths(c), _prefix_rows(c), c["window"]
    mine = sum(min(x, w) if w else x for x in lens)
    both = prefix = 0
    for a, b, L in zip(at, at[1:], plens):  # (in the order before the lengths are dealt out: the same in the mean)
        seen = [min(L, max(0, w - x)) if w else L for x in lens[a:b]]
        both += sum(seen)
        prefix += max(seen, default=0)
    return {"bytes": (mine + prefix) * row + c["n"] * H * (4 * hd + 4) + 4 * (-(-(mine + prefix) // c["page"]) + c["n"]),
            "flops": 4 * H * hd * (mine + both)}


# ------------------------------------------------------------------------------------------------ exact


def _exact_rows(s, o, lse, t, h0, q, k, v, first, last):
    """Heads h0 .. of tokens t: q [tokens][g][hd] over rows k, v [n][hd], those from first to last (each [tokens])."""
    g = q.shape[1]
    z = torch.einsum("tgd,nd->tgn", q, k) * s["scale"]
    j = torch.arange(k.shape[0], device="cuda")
    z.masked_fill_(((j < first[:, None]) | (j > last[:, None]))[:, None, :], float("-inf"))
    e = torch.logsumexp(z, -1)
    lse[t, h0:h0 + g] = e
    if s["sink_w"] is not None:
        e = torch.logaddexp(e, s["sink_w"][h0:h0 + g].double())
    z -= e.masked_fill(e == float("-inf"), 0.0)[..., None]
    o[t, h0:h0 + g] = torch.einsum("tgn,nd->tgd", z.exp_(), v)


def exact(case, seed):
    """The same outputs from the definition in 64 bits."""
    if work(case)["flops"] > 2e12:  # (more than 20 seconds)
        return None
    s = prepare(case, seed)
    N, H, hd = s["q"].shape
    kv, page = s["kv_heads"], s["page"]
    g = H // kv
    o = torch.zeros(N, H, hd, dtype=torch.float64, device="cuda")
    lse = torch.zeros(N, H, dtype=torch.float64, device="cuda")

    def rows(table, n, h):
        j = torch.arange(n, device="cuda")
        at = table[j // page].long() * page + j % page
        return (s[x].select(2, h).reshape(-1, hd)[at].double() for x in "kv")

    def of_head(t, h):
        return s["q"][t, h * g:(h + 1) * g].double()

    if s["op"] == "prompt_attn":
        for r, n in enumerate(s["rows"]):
            a, b = s["at"][r], s["at"][r + 1]
            for h in range(kv if b > a else 0):
                k, v = rows(s["table"][r], n, h)
                for t0 in range(a, b, max(1, (1 << 26) // (g * n))):
                    t = slice(t0, min(b, t0 + max(1, (1 << 26) // (g * n))))
                    last = torch.arange(t.start, t.stop, device="cuda") + n - b
                    first = last + 1 - s["window"] if s["window"] else torch.zeros_like(last)
                    _exact_rows(s, o, lse, t, h * g, of_head(t, h), k, v, first, last)
        return {"o": o, "lse": lse}
    for i, L in enumerate(s["plens"]):
        for h in range(kv):
            shared = [x for x in rows(s["prefix"][i], L, h)]
            for t in range(s["at"][i], s["at"][i + 1]):
                k, v = (torch.cat([x, y]) for x, y in zip(shared, rows(s["table"][t], s["rows"][t], h)))
                last = torch.tensor([k.shape[0] - 1], device="cuda")
                first = last + 1 - s["window"] if s["window"] else torch.zeros_like(last)
                if k.shape[0] == 0:
                    lse[t, h * g:(h + 1) * g] = float("-inf")
                    continue
                _exact_rows(s, o, lse, slice(t, t + 1), h * g, of_head(slice(t, t + 1), h), k, v, first, last)
    return {"o": o, "lse": lse}
