"""The operators of a continuous batch over a paged cache: what is measured of them, and their plain forms.

Three operators that a server calls in turn, once a step:

  page_step      block tables, slot maps and positions of the step's tokens, built on the GPU from the
                 requests' lengths and a pool of free pages
  qk_norm_rope   RMSNorm of each head's query and key and the position rotation, the key and value rows
                 written to their slots of the paged cache
  paged_attn     attention of one new token a row over the paged cache

``run`` computes them in elementary torch operations, in 32 bits and rounded once at the end, or (``own``) calls
this repository's package.  ``exact`` computes them in 64 bits, a request or a head at a time.
"""
import random

import torch

own = False

# ------------------------------------------------------------------------------------------------ cases


def _attn(name, n, lo, hi, heads, kv_heads, hd, page, latent=False, window=0, sink=False, head_major=False):
    return dict(name=name, op="paged_attn", n=n, lo=lo, hi=hi, heads=heads, kv_heads=kv_heads, hd=hd, page=page,
                latent=latent, window=window, sink=sink, head_major=head_major)


def _norm(name, n, heads, kv_heads, hd, rd, page, first, latent=False, half=False, last=True, norm=True, pad=0):
    return dict(name=name, op="qk_norm_rope", n=n, heads=heads, kv_heads=kv_heads, hd=hd, rd=rd, page=page,
                first=first, latent=latent, half=half, last=last, norm=norm, pad=pad)


def _step(name, decode, chunks, chunk, ended, idle, lo, hi, page, pad):
    return dict(name=name, op="page_step", decode=decode, chunks=chunks, chunk=chunk, ended=ended, idle=idle, lo=lo,
                hi=hi, page=page, pad=pad)


def listed():
    return [
        # one short chat turn: the latency of the whole chain of loads
        _attn("attn 1 x 37", 1, 37, 37, 16, 4, 64, 16),
        # a serving batch in mid-conversation, ragged, four query heads to a key head
        _attn("attn 32 ragged gqa", 32, 300, 4000, 32, 8, 128, 16),
        # a few long documents, ragged; the cache is far larger than L2
        _attn("attn 4 x 64k gqa", 4, 50000, 65536, 64, 8, 128, 64),
        # wide heads, a key head for each query head, a sliding window with sinks, odd pages, pages stored a head at a
        # time, an empty row
        _attn("attn window mha 256", 48, 0, 9000, 16, 16, 256, 17, window=1000, sink=True, head_major=True),
        # the layer's own heads (64 x 512 over one latent row that is key and value), 32 x 1 at about p = 1000
        _attn("attn latent decode", 32, 800, 1001, 64, 1, 512, 64, latent=True, sink=True),
        # the same over 16384 rows, 64 x 1: the largest
        _attn("attn latent long", 64, 12000, 16384, 64, 1, 512, 64, latent=True, sink=True),
        # a decode step's rows: 32 tokens, half layout over the whole head
        _norm("norm decode 32", 32, 32, 8, 128, 128, 16, 2000, half=True),
        # a prefill chunk at the layer's head shapes: 64 x 512, the last 64 turned, one latent row a token
        _norm("norm latent 4096", 4096, 64, 1, 512, 64, 64, 0, latent=True),
        # a mixed step of odd size: part of a 96-wide head turned, padded rows at the end
        _norm("norm odd 1537", 1537, 24, 6, 96, 48, 17, 30000, half=True, last=False, pad=23),
        # 64 requests that decode, some of them over a page's end
        _step("step decode 64", 64, 0, 0, 0, 0, 1, 4000, 16, 0),
        # a large mixed step: decodes, prefill chunks, requests that ended or wait, a padded batch
        _step("step mixed 1500", 1200, 24, 1000, 176, 100, 0, 8000, 32, 900),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    """One more case of the same ranges: one token to long caches, any page, head layout and padding."""
    op = rng.choice(["attn", "attn", "latent", "norm", "norm", "step"])
    if op == "attn":
        n, hd = _log(rng, 1, 96), rng.choice([64, 80, 96, 128, 192, 256])
        kv = rng.choice([1, 2, 3, 4, 8, 16])
        g = rng.choice([1, 2, 4, 5, 7, 8, 16, 20])
        top = max(2, min(65536, 800_000_000 // (n * kv * hd * 4)))
        hi = _log(rng, 1, top)
        window = rng.choice([0, 0, 0, _log(rng, 1, 8192)])
        return _attn("", n, rng.choice([0, _log(rng, 1, hi)]), hi, kv * g, kv, hd, rng.choice([1, 8, 16, 17, 32, 64, 128]),
                     window=window, sink=rng.random() < 0.4, head_major=rng.random() < 0.4)
    if op == "latent":
        n = _log(rng, 1, 96)
        hi = _log(rng, 1, max(2, min(65536, 900_000_000 // (n * 1024))))
        return _attn("", n, _log(rng, 1, hi), hi, rng.choice([16, 32, 40, 64, 128]) if n * hi < 400_000 else 64, 1, 512,
                     rng.choice([16, 17, 32, 64, 128]), latent=True, window=rng.choice([0, 0, _log(rng, 1, 4096)]),
                     sink=rng.random() < 0.7)
    if op == "norm":
        hd = rng.choice([64, 80, 96, 128, 192, 256, 512])
        latent = hd == 512 or rng.random() < 0.2
        kv = 1 if latent else rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 5, 8, 16])
        n = _log(rng, 1, max(2, min(16384, 120_000_000 // ((heads + 2 * kv) * hd))))
        rd = rng.choice([hd, hd, 16 * rng.randint(1, hd // 16), 16 * rng.randint(1, hd // 16), 2 * rng.randint(1, hd // 2)])
        return _norm("", n, heads, kv, hd, rd, rng.choice([1, 16, 17, 64]), _log(rng, 1, 60000), latent=latent,
                     half=rng.random() < 0.5, last=rng.random() < 0.5, norm=rng.random() < 0.8,
                     pad=rng.choice([0, 0, rng.randint(1, 40)]))
    return _step("", _log(rng, 1, 2000), rng.randint(0, 30), _log(rng, 1, 1200), rng.randint(0, 200), rng.randint(0, 100),
                 0, _log(rng, 1, 9000), rng.choice([1, 16, 17, 32, 64]) if rng.random() < 0.8 else 128,
                 rng.choice([0, rng.randint(1, 1000)]))


def _lengths(n, lo, hi):
    """n lengths from lo to hi, evenly spread over their logarithm (zero and one included where lo is 0)."""
    if n == 1:
        return [hi]
    a = max(lo, 1)
    v = [int(round(a * (hi / a) ** (i / (n - 1)))) if hi >= a else hi for i in range(n)]
    if lo == 0:
        v[0] = 0
    return v


def _order(n, seed):
    at = list(range(n))
    random.Random(seed).shuffle(at)
    return at


# ------------------------------------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(torch.bfloat16)


def _pages(g, n_pages, page, kv_heads, hd, head_major):
    """A cache tensor [page][row][head][feature]; head_major: stored with a head's rows of a page side by side."""
    if head_major:
        return _bf(g, n_pages, kv_heads, page, hd).transpose(1, 2)
    return _bf(g, n_pages, page, kv_heads, hd)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    return {"paged_attn": _prepare_attn, "qk_norm_rope": _prepare_norm, "page_step": _prepare_step}[case["op"]](case, seed)


def _prepare_attn(c, seed):
    g = _gen(seed)
    lens = _lengths(c["n"], c["lo"], c["hi"])
    lens = [lens[i] for i in _order(c["n"], seed)]
    page, per = c["page"], [-(-x // c["page"]) for x in lens]
    width, total = max(per) + 2, sum(per)
    n_pages = total + 5
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(c["n"], width, dtype=torch.int32, device="cuda")
    mask = torch.arange(width, device="cuda")[None, :] < _i32(per)[:, None]
    table[mask] = perm[:total]
    k = _pages(g, n_pages, page, c["kv_heads"], c["hd"], c["head_major"])
    v = None if c["latent"] else _pages(g, n_pages, page, c["kv_heads"], c["hd"], c["head_major"])
    return dict(c, q=_bf(g, c["n"], c["heads"], c["hd"], scale=1.5), k=k, v=v, table=table,
                pos=_i32([x - 1 for x in lens]),
                sink_w=torch.randn(c["heads"], generator=g, device="cuda") if c["sink"] else None,
                rows=min(max(lens), c["window"] or max(lens)), scale=c["hd"] ** -0.5)


def _prepare_norm(c, seed):
    g = _gen(seed)
    n, H, kv, hd, rd, page = c["n"], c["heads"], c["kv_heads"], c["hd"], c["rd"], c["page"]
    # the rows of one projection: query heads, key heads, value heads side by side, read as strided views
    x = _bf(g, n, (H + (1 if c["latent"] else 2) * kv) * hd, scale=2.0)
    q = x[:, :H * hd].view(n, H, hd)
    k = x[:, H * hd:(H + kv) * hd].view(n, kv, hd)
    v = None if c["latent"] else x[:, (H + kv) * hd:].view(n, kv, hd)
    n_pages = -(-n // page) + 3
    slot = torch.randperm(n_pages * page, generator=g, device="cuda")[:n].to(torch.int32)
    top = c["first"] + n
    pos = (c["first"] + torch.randperm(n, generator=g, device="cuda")).to(torch.int32)
    live = n - min(c["pad"], n - 1)
    slot[live:] = -1
    pos[live:] = -1
    inv = 10000.0 ** (-2.0 * torch.arange(rd // 2, device="cuda", dtype=torch.float64) / rd)
    a = torch.arange(top, device="cuda", dtype=torch.float64)[:, None] * inv
    tab = torch.stack([a.cos(), a.sin()], -1).float().contiguous()
    w = lambda: 1.0 + 0.1 * torch.randn(hd, generator=g, device="cuda")  # noqa: E731
    return dict(c, q=q, k=k, v=v, pos=pos, slot=slot, tab=tab, at=hd - rd if c["last"] else 0, eps=1e-6,
                q_norm=w() if c["norm"] else None, k_norm=w() if c["norm"] else None,
                q_out=torch.zeros(n, H, hd, dtype=torch.bfloat16, device="cuda"),
                k_pages=_pages(g, n_pages, page, kv, hd, False),
                v_pages=None if c["latent"] else _pages(g, n_pages, page, kv, hd, False))


def _step_lengths(c):
    """(length, new tokens) of every request of a step: decodes, chunks (the first of them into an empty request),
    ended requests (-1) and idle ones."""
    n = c["decode"] + c["chunks"] + c["ended"] + c["idle"]
    lens = _lengths(n, c["lo"], c["hi"])
    lens = [lens[i] for i in _order(n, 7)]
    new = [1] * c["decode"] + [max(1, c["chunk"] - 7 * i) for i in range(c["chunks"])] + [-1] * c["ended"] + [0] * c["idle"]
    for i in range(c["decode"], c["decode"] + c["chunks"], 2):
        lens[i] = 0
    return lens, new


def _prepare_step(c, seed):
    g = _gen(seed)
    lens, new = _step_lengths(c)
    order = _order(len(lens), seed)
    lens, new, page = [lens[i] for i in order], [new[i] for i in order], c["page"]
    have = [-(-x // page) for x in lens]
    need = sum(-(-(x + a) // page) - h for x, a, h in zip(lens, new, have) if a > 0)
    width = max(-(-(x + max(a, 0)) // page) for x, a in zip(lens, new)) + 3
    n_pages = sum(have) + need + 11
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    mask = torch.arange(width, device="cuda")[None, :] < _i32(have)[:, None]
    table[mask] = perm[:sum(have)]
    free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    head, count = n_pages // 3, n_pages - sum(have)
    free[(head + torch.arange(count, device="cuda")) % n_pages] = perm[sum(have):]
    n = sum(max(a, 0) for a in new) + c["pad"]
    e = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(c, new=_i32(new), length=_i32(lens), table=table, free=free, state=_i32([head, count]), tok_req=e(n),
                tok_pos=e(n), tok_slot=e(n), cu=e(len(lens) + 1), length_out=e(len(lens)), state_out=e(2), info=e(4))


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


def _own_attn(s):
    import compressed_sparse_attention_attn_gb300 as csa
    if "cache" not in s:
        s["cache"] = csa.PagedCache(s["k"], s["v"])
    o, lse = _ctx().paged_attn(s["q"], s["cache"], s["table"], s["pos"], s["scale"], sink=s["sink_w"],
                               window=s["window"], with_lse=True)
    return {"o": o, "lse": lse}


def _own_norm(s):
    import compressed_sparse_attention_attn_gb300 as csa
    if "cache" not in s:
        s["cache"] = csa.PagedCache(s["k_pages"], s["v_pages"])
    _ctx().qk_norm_rope(s["q"], s["k"], s["v"], s["cache"], s["pos"], s["slot"], tab=s["tab"], rd=s["rd"],
                        rope_at=s["at"], half=s["half"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=s["eps"],
                        q_out=s["q_out"])
    return {"q": s["q_out"], "k": s["k_pages"], "v": s["v_pages"]}


def _own_step(s):
    import compressed_sparse_attention_attn_gb300 as csa
    csa.page_step(s["new"], s["length"], s["table"], s["free"], s["state"], s["page"], s["tok_req"], s["tok_pos"],
                  s["tok_slot"], s["cu"], length_out=s["length_out"], state_out=s["state_out"], info=s["info"])
    return _step_outputs(s)


def _step_outputs(s):
    return {k: s[k] for k in ("tok_req", "tok_pos", "tok_slot", "cu", "table", "free", "length_out", "state_out", "info")}


def _plain_attn(s):
    """Rows gathered through the table (padded to the longest), scores, a masked softmax with the sink in its
    denominator, and the weighted sum."""
    q, pos, page, kv = s["q"], s["pos"].long(), s["page"], s["kv_heads"]
    n, H, hd = q.shape
    first = (pos + 1 - s["window"]).clamp(min=0) if s["window"] else torch.zeros_like(pos)
    at = first[:, None] + torch.arange(s["rows"], device=q.device)
    valid = at <= pos[:, None]
    at = torch.where(valid, at, torch.zeros_like(at))
    page_id = s["table"].long().gather(1, at // page)
    keys = s["k"][page_id, at % page].float()  # [n][rows][kv][hd]
    values = keys if s["v"] is None else s["v"][page_id, at % page].float()
    values = values * valid[:, :, None, None]
    score = torch.matmul(q.float().view(n, kv, H // kv, hd), keys.permute(0, 2, 3, 1)) * s["scale"]
    score = score.masked_fill(~valid[:, None, None, :], float("-inf"))
    top = score.amax(-1, keepdim=True)
    if s["sink_w"] is not None:
        top = torch.maximum(top, s["sink_w"].view(1, kv, H // kv, 1))
    top = top.masked_fill(top == float("-inf"), 0.0)  # (a row without a position: its weights are all 0)
    weight = (score - top).exp()
    total = weight.sum(-1, keepdim=True)
    below = total if s["sink_w"] is None else total + (s["sink_w"].view(1, kv, H // kv, 1) - top).exp()
    below = below.masked_fill(below == 0, 1.0)
    o = torch.matmul(weight, values.permute(0, 2, 1, 3)) / below
    return {"o": o.reshape(n, H, hd).to(torch.bfloat16), "lse": (top + total.log()).reshape(n, H)}


def _plain_rows(x, w, s, live):
    """Normed and turned rows of x [n][heads][hd] in 32 bits."""
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * w
    at, rd = s["at"], s["rd"]
    cs = s["tab"][s["pos"].clamp(min=0).long()][:, None]  # [n][1][rd/2][2]
    part = y[..., at:at + rd]
    a, b = (part[..., :rd // 2], part[..., rd // 2:]) if s["half"] else (part[..., 0::2], part[..., 1::2])
    re, im = a * cs[..., 0] - b * cs[..., 1], a * cs[..., 1] + b * cs[..., 0]
    turned = torch.cat([re, im], -1) if s["half"] else torch.stack([re, im], -1).flatten(-2)
    return torch.cat([y[..., :at], turned, y[..., at + rd:]], -1).to(torch.bfloat16)


def _plain_norm(s):
    live = (s["pos"] >= 0)[:, None, None]
    s["q_out"].copy_(torch.where(live, _plain_rows(s["q"], s["q_norm"], s, live), s["q_out"]))
    kept = s["slot"] >= 0
    slot = s["slot"][kept].long()
    page_id, row = slot // s["page"], slot % s["page"]
    s["k_pages"][page_id, row] = _plain_rows(s["k"], s["k_norm"], s, live)[kept]
    if s["v"] is not None:
        s["v_pages"][page_id, row] = s["v"][kept]
    return {"q": s["q_out"], "k": s["k_pages"], "v": s["v_pages"]}


def _plain_step(s):
    new, length, table, free, page = s["new"].long(), s["length"].long(), s["table"], s["free"], s["page"]
    n_pages, width, n, R = free.numel(), table.shape[1], s["tok_req"].numel(), new.numel()
    head, count = s["state"][0].long(), s["state"][1].long()
    add = new.clamp(min=0)
    have = (length + page - 1) // page
    need = (length + add + page - 1) // page - have
    back = torch.where(new < 0, have, torch.zeros_like(have))
    cu = torch.cat([torch.zeros_like(add[:1]), add.cumsum(0)])
    taken, returned = need.cumsum(0), back.cumsum(0)
    # tokens
    t = torch.arange(n, device=new.device)
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=R - 1)
    live = t < cu[-1]
    pos = length[r] + t - cu[r]
    p = pos // page
    fresh = free[(head + (taken - need)[r] + p - have[r]) % n_pages].long()
    held = table[r, p.clamp(0, width - 1)].long()
    slot = torch.where(p >= have[r], fresh, held) * page + pos % page
    s["tok_req"].copy_(torch.where(live, r, -1))
    s["tok_pos"].copy_(torch.where(live, pos, -1))
    s["tok_slot"].copy_(torch.where(live, slot, -1))
    # released pages go behind the last free one
    k = (torch.arange(n_pages, device=new.device) - head - count) % n_pages
    rr = torch.searchsorted(returned, k, right=True).clamp(max=R - 1)
    j = (k - (returned - back)[rr]).clamp(0, width - 1)
    old_free = free.clone()
    free.copy_(torch.where(k < returned[-1], table[rr, j], free))
    # pages taken
    col = torch.arange(width, device=new.device)[None, :]
    mine = (col >= have[:, None]) & (col < (have + need)[:, None])
    table.copy_(torch.where(mine, old_free[(head + (taken - need)[:, None] + col - have[:, None]) % n_pages], table))
    s["cu"].copy_(cu)
    s["length_out"].copy_(torch.where(new < 0, torch.zeros_like(length), length + add))
    s["state_out"].copy_(torch.stack([(head + taken[-1]) % n_pages, count - taken[-1] + returned[-1]]))
    s["info"].copy_(torch.stack([cu[-1], taken[-1], returned[-1], torch.zeros_like(head)]))
    return _step_outputs(s)


_plain = {"paged_attn": _plain_attn, "qk_norm_rope": _plain_norm, "page_step": _plain_step}
_own = {"paged_attn": _own_attn, "qk_norm_rope": _own_norm, "page_step": _own_step}


# ------------------------------------------------------------------------------------------------ work


def work(c):
    if c["op"] == "paged_attn":
        lens = _lengths(c["n"], c["lo"], c["hi"])
        rows = sum(min(x, c["window"] or x) for x in lens)
        pages = sum(-(-min(x, c["window"] or x) // c["page"]) for x in lens)
        row = c["kv_heads"] * c["hd"] * 2 * (1 if c["latent"] else 2)
        return {"bytes": rows * row + c["n"] * c["heads"] * (4 * c["hd"] + 4) + 4 * pages + 4 * c["n"],
                "flops": 4 * rows * c["heads"] * c["hd"]}
    if c["op"] == "qk_norm_rope":
        live = c["n"] - min(c["pad"], c["n"] - 1)
        heads = c["heads"] + c["kv_heads"] * (1 if c["latent"] else 2)
        return {"bytes": live * (4 * heads * c["hd"] + 4 * c["rd"]) + 8 * c["n"],
                "flops": live * (c["heads"] + c["kv_heads"]) * (6 * c["hd"] + 3 * c["rd"])}
    lens, new = _step_lengths(c)
    have = [-(-x // c["page"]) for x in lens]
    moved = sum(-(-(x + a) // c["page"]) - h if a > 0 else (h if a < 0 else 0) for x, a, h in zip(lens, new, have))
    tokens = sum(max(a, 0) for a in new) + c["pad"]
    return {"bytes": 16 * len(lens) + 12 * tokens + 8 * moved + 40, "flops": 8 * tokens}


# ------------------------------------------------------------------------------------------------ exact


def exact(case, seed):
    """The same outputs from the definitions in 64 bits, a request (or a token's heads) at a time."""
    s = prepare(case, seed)
    if case["op"] == "paged_attn":
        return _exact_attn(s)
    if case["op"] == "qk_norm_rope":
        return _exact_norm(s)
    return None


def _exact_attn(s):
    n, H, hd = s["q"].shape
    g = H // s["kv_heads"]
    o = torch.zeros(n, H, hd, dtype=torch.float64, device="cuda")
    lse = torch.full((n, H), float("-inf"), dtype=torch.float64, device="cuda")
    last = s["pos"].tolist()
    for i in range(n):
        first = max(0, last[i] + 1 - s["window"]) if s["window"] else 0
        rows = range(first, last[i] + 1)
        if not rows:
            continue
        p = torch.arange(first, last[i] + 1, device="cuda")
        ids = s["table"][i, p // s["page"]].long()
        k = s["k"][ids, p % s["page"]].double()
        v = k if s["v"] is None else s["v"][ids, p % s["page"]].double()
        for h in range(s["kv_heads"]):
            qh = s["q"][i, h * g:(h + 1) * g].double()
            z = qh @ k[:, h].T * s["scale"]
            e = torch.logsumexp(z, 1)
            lse[i, h * g:(h + 1) * g] = e
            if s["sink_w"] is not None:
                e = torch.logaddexp(e, s["sink_w"][h * g:(h + 1) * g].double())
            o[i, h * g:(h + 1) * g] = torch.exp(z - e[:, None]) @ v[:, h]
    return {"o": o, "lse": lse}


def _exact_norm(s):
    half, at, h2 = s["half"], s["at"], s["rd"] // 2
    i = torch.arange(h2, device="cuda")
    lo, hi = (at + i, at + i + h2) if half else (at + 2 * i, at + 2 * i + 1)

    def rows(x, w):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[-1] + s["eps"]) * w.double()
        cos, sin = (s["tab"][s["pos"].clamp(min=0).long(), :, k].double()[:, None, :] for k in (0, 1))
        a, b = y[..., lo].clone(), y[..., hi].clone()
        y[..., lo] = a * cos - b * sin
        y[..., hi] = b * cos + a * sin
        return y

    q = s["q_out"].double()
    live = s["pos"] >= 0
    q[live] = rows(s["q"], s["q_norm"])[live]
    k = s["k_pages"].double()
    kept = s["slot"] >= 0
    at_slot = s["slot"][kept].long()
    k.view(-1, *k.shape[2:])[at_slot] = rows(s["k"], s["k_norm"])[kept]
    if s["v"] is None:
        return {"q": q, "k": k, "v": None}
    v = s["v_pages"].double()
    v.view(-1, *v.shape[2:])[at_slot] = s["v"].double()[kept]
    return {"q": q, "k": k, "v": v}
