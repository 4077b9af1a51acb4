"""Attention of prompts and of rows that share a prefix over a paged cache, on the GPU against plain 64-bit forms, and runs of
the paged calls together.

Tolerances, from the roundings alone, as those of single tokens over the cache: half a step of the result, 2^-8 |want|; an error d
of a score moves the result by at most 2 d A with A = sum_j w_j |V_j|, d at most (hd + 8) 2^-24 sum |q K| scale (one rounding a
product and a sum) plus 2^-21 (the exponential) plus rows x 2^-24 (the row's sum); a weight below f32's smallest normal number
may be 0.  The weights enter their product as one bf16 term, at most 2^-8 off, and the denominator adds up the same terms: the
result moves by at most 2^-8 sum_j w_j |V_j - O| <= 2^-8 (A + |want|).  A row's own part of a prefix batch has two terms (2^-16).
"""
import math

import numpy as np
import pytest
import torch

from test_paged import Batch, Pool, close_rows, csa, ctx, gen, i32, make_ctx, randn, ref_rows, rope_tab  # noqa: F401

pytestmark = pytest.mark.gpu


def ref(q, K, V, kv, scale, sink, first, last):
    """(O, lse, tolerance of O, of lse): q [t][H][hd] over rows first[t] .. last[t] of K, V [n][kv][hd], in 64 bits."""
    t, H, hd = q.shape
    g, n = H // kv, K.shape[0]
    O = torch.zeros(t, H, hd, dtype=torch.float64, device="cuda")
    lse = torch.full((t, H), float("-inf"), dtype=torch.float64, device="cuda")
    tol, tol_l = torch.zeros_like(O), torch.zeros_like(lse)
    if n == 0 or t == 0:
        return O, lse, tol, tol_l
    j = torch.arange(n, device="cuda")
    seen = (j >= first[:, None]) & (j <= last[:, None])
    rows = seen.sum(1)
    for h in range(kv):
        hs = slice(h * g, (h + 1) * g)
        qd, Kd, Vd = q[:, hs].double(), K[:, h].double(), V[:, h].double()
        S = torch.einsum("tgd,nd->tgn", qd, Kd) * scale
        S = S.masked_fill(~seen[:, None], float("-inf"))
        e = torch.logsumexp(S, -1)
        den = e if sink is None else torch.logaddexp(e, sink[hs].double())
        w = torch.exp(S - den.masked_fill(den == float("-inf"), 0.0)[..., None])
        Kabs = torch.einsum("tgd,nd->tgn", qd.abs(), Kd.abs()).masked_fill(~seen[:, None], 0.0).amax(-1)
        d = (hd + 8) * 2.0 ** -24 * Kabs * abs(scale) + 2.0 ** -21 + (rows * 2.0 ** -24)[:, None]
        O[:, hs] = torch.einsum("tgn,nd->tgd", w, Vd)
        A = torch.einsum("tgn,nd->tgd", w, Vd.abs())
        least = 2.0 ** -126 * torch.einsum("tn,nd->td", seen.double(), Vd.abs())[:, None]
        lse[:, hs] = e
        tol[:, hs] = 2.0 ** -8 * O[:, hs].abs() + (2 * d[..., None] + 2.0 ** -8) * A + 2.0 ** -8 * O[:, hs].abs() + 2 * least
        tol_l[:, hs] = d + 2.0 ** -22 * (1 + e.abs())
    return O, lse, tol, tol_l


def close(o, lse, want, what):
    O, e, tol, tol_l = want
    err = (o.double() - O).abs()
    fits = not err.isnan().any().item() and (err <= tol).all().item()
    assert fits, "%s: off by %g, %g too much" % (what, err.max(), (err - tol).max())
    if lse is not None:
        none = e == float("-inf")
        fits = torch.equal(lse[none].double(), e[none]) and ((lse.double() - e).abs()[~none] <= tol_l[~none]).all().item()
        assert fits, "%s: lse off by %g" % (what, (lse.double() - e).abs()[~none].max())


def cus(new):
    return np.concatenate([[0], np.cumsum(new)]).tolist()


def check_prompt(b, new, q, o, lse, sink=None, window=0, scale=None, lens=None, only=None):
    """Request r's new[r] newest tokens, packed, against its rows; rows behind the last request's are not looked at."""
    cu = cus(new)
    for r, n in enumerate(b.lens if lens is None else lens):
        if new[r] == 0 or (only is not None and r not in only):
            continue
        a, e = cu[r], cu[r + 1]
        for t0 in range(a, e, 512):
            t = slice(t0, min(e, t0 + 512))
            last = torch.arange(t.start, t.stop, device="cuda") + n - e
            first = (last + 1 - window).clamp(min=0) if window else torch.zeros_like(last)
            close(o[t], None if lse is None else lse[t],
                  ref(q[t], b.rows_k[r][:n], b.rows_v[r][:n], b.kv, b.scale if scale is None else scale, sink, first, last),
                  "request %d, tokens from %d" % (r, t0 - a))


def prompt(csa, ctx, b, new, pad=0, sink=None, window=0, **kw):
    n = sum(new) + pad
    q = b.queries(n)
    out = torch.full((n, b.H, b.hd), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, b.H), 3.0, device="cuda")
    ctx.prompt_attn(q, csa.PagedCache(b.k, b.v), b.table, i32(cus(new)), i32(b.lens), b.scale, sink=sink, window=window, out=out,
                    lse=lse, **kw)
    assert (out[n - pad:] == 3).all() and (lse[n - pad:] == 3).all()
    return q, out, lse


# every kind of request: whole prompts, chunks behind earlier rows, single tokens, none
LENS = [1, 0, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 40, 500, 257, 9]
NEW = [1, 0, 2, 15, 3, 17, 63, 1, 65, 127, 128, 129, 300, 0, 131, 255, 1]
SHAPES = [  # H, kv, hd, page, latent, order, window, sink
    (4, 4, 64, 16, False, "nhd", 0, False),
    (8, 2, 64, 16, False, "hnd", 0, True),
    (32, 8, 128, 16, False, "nhd", 0, False),
    (7, 1, 128, 17, False, "nhd", 100, True),
    (16, 1, 128, 1, False, "hnd", 0, False),
    (20, 1, 128, 64, False, "nhd", 0, True),
    (40, 2, 64, 32, False, "nhd", 70, False),
    (3, 3, 80, 16, False, "nhd", 0, False),
    (10, 2, 96, 8, False, "hnd", 1, True),
    (6, 3, 192, 128, False, "nhd", 0, False),
    (6, 2, 136, 16, False, "nhd", 33, True),
    (16, 16, 256, 17, False, "hnd", 64, True),
    (10, 2, 248, 48, False, "nhd", 0, False),
    (8, 1, 256, 16, True, "nhd", 0, False),
    (12, 2, 128, 256, True, "hnd", 0, False),
    (5, 1, 8, 16, False, "nhd", 0, False),
    (130, 1, 72, 16, False, "nhd", 0, True),
    (257, 1, 64, 24, False, "nhd", 200, False),
]


@pytest.mark.parametrize("H,kv,hd,page,latent,order,window,sink", SHAPES)
def test_prompt(csa, ctx, H, kv, hd, page, latent, order, window, sink):
    b = Batch(LENS, H, kv, hd, page, latent, order, seed=H * hd)
    sw = torch.randn(H, generator=b.g, device="cuda") if sink else None
    q, o, lse = prompt(csa, ctx, b, NEW, pad=3, sink=sw, window=window)
    check_prompt(b, NEW, q, o, lse, sw, window)
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd", [(8, 2, 128), (4, 4, 64), (10, 1, 256), (9, 3, 192), (6, 2, 96)])
@pytest.mark.parametrize("lens,new", [
    ([1], [1]), ([40], [40]), ([3000], [3000]), ([20000], [1]), ([9000], [70]), ([9000, 1, 0, 1, 4000], [300, 1, 0, 0, 1]),
    ([1] * 700, [1] * 700), (list(range(300)), [min(i, 5) for i in range(300)]), ([700] * 40, [1, 17] * 20)])
def test_prompt_lengths(csa, ctx, H, kv, hd, lens, new):
    """One prompt alone, few tokens behind much, many short requests; the same bits again, whatever finished first."""
    b = Batch(lens, H, kv, hd, 16, seed=len(lens) + hd)
    q, o, lse = prompt(csa, ctx, b, new)
    check_prompt(b, new, q, o, lse)
    cache, cu, length = csa.PagedCache(b.k, b.v), i32(cus(new)), i32(lens)
    for _ in range(3):
        o2, lse2 = ctx.prompt_attn(q, cache, b.table, cu, length, b.scale, with_lse=True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(ctx.prompt_attn(q, cache, b.table, cu, length, b.scale), o)
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd,window", [(8, 2, 128, 0), (16, 2, 256, 700), (20, 4, 80, 5000)])
@pytest.mark.parametrize("seed", range(4))
def test_prompt_uneven(csa, ctx, H, kv, hd, window, seed):
    """Long and short, whole and in part, in any order."""
    rng = np.random.default_rng(100 * hd + seed)
    lens = [int(rng.choice([0, 1, 3, 16, 33, 97, 200])) for _ in range(int(rng.integers(2, 30)))]
    for _ in range(int(rng.integers(1, 4))):
        lens.insert(int(rng.integers(0, len(lens) + 1)), int(rng.integers(500, 7000)))
    new = [int(rng.integers(0, min(x, 900) + 1)) for x in lens]
    b = Batch(lens, H, kv, hd, int(rng.choice([5, 16, 64])), seed=seed)
    sink = torch.randn(H, generator=b.g, device="cuda")
    q, o, lse = prompt(csa, ctx, b, new, pad=int(rng.integers(0, 50)), sink=sink, window=window)
    check_prompt(b, new, q, o, lse, sink, window)
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd", [(8, 2, 128), (20, 4, 80), (16, 2, 256), (4, 4, 64), (6, 2, 192)])
def test_prompt_cold(csa, ctx, H, kv, hd):
    """Every call on another batch than the one before, with nothing of it in L2: what a stage still holds of an earlier one, or
    shares of an earlier call, may not be taken for what is on its way."""
    batches = []
    for seed in range(4):
        rng = np.random.default_rng(1000 * hd + seed)
        lens = [int(rng.choice([1, 3, 16, 33, 97, 200])) for _ in range(int(rng.integers(8, 30)))]
        for _ in range(3):
            lens.insert(int(rng.integers(0, len(lens) + 1)), int(rng.integers(500, 3000)))
        new = [int(rng.integers(1, min(x, 700) + 1)) for x in lens]
        b = Batch(lens, H, kv, hd, int(rng.choice([5, 16, 64])), seed=seed)
        q = b.queries(sum(new))
        batches.append((b, new, q, (q, csa.PagedCache(b.k, b.v), b.table, i32(cus(new)), i32(lens), b.scale)))
    flush = torch.empty(96 << 20, device="cuda")
    for turn in range(3):
        for b, new, q, args in batches:
            flush.fill_(float("nan"))
            o, lse = ctx.prompt_attn(*args, with_lse=True)
            if turn == 0:
                check_prompt(b, new, q, o, lse)
                b.want = o, lse
            assert torch.equal(o, b.want[0]) and torch.equal(lse, b.want[1])
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd", [(8, 2, 128), (4, 1, 256)])
def test_prompt_strided_rows_and_in_place(csa, ctx, H, kv, hd):
    """Rows of a wider buffer, whose other columns stay, and the result over q itself."""
    lens, new = [70, 300, 9], [70, 120, 2]
    b = Batch(lens, H, kv, hd, 16, seed=3)
    N = sum(new) + 2
    wide = randn(b.g, N, H * hd + 64, scale=1.5)
    q = wide[:, 8:8 + H * hd].view(N, H, hd)
    buf = torch.full((N, H * hd + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :H * hd].view(N, H, hd)
    args = (csa.PagedCache(b.k, b.v), b.table, i32(cus(new)), i32(lens), b.scale)
    o, lse = ctx.prompt_attn(q, *args, out=out, with_lse=True)
    assert o is out and (buf[:, H * hd:] == 3).all() and (out[-2:] == 3).all()
    check_prompt(b, new, q, out, lse)
    keep = wide.clone()
    got = ctx.prompt_attn(q, *args, out=q)
    assert got is q and torch.equal(q[:-2], out[:-2]) and torch.equal(wide[-2:], keep[-2:])
    assert torch.equal(wide[:, :8], keep[:, :8]) and torch.equal(wide[:, 8 + H * hd:], keep[:, 8 + H * hd:])
    assert ctx.status() == 0


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_rows_that_heads_and_pages_share(csa, ctx, hd):
    """A cache with strides of 0: one key head for all, one page, one row of a page."""
    H, kv, page = 8, 4, 16
    b = Batch([70, 300, 33], H, kv, hd, page, seed=hd)
    new, cu = [70, 200, 1], i32([0, 70, 270, 271])
    q = b.queries(271)
    pos, prefix_len = i32([69, -1, 32]), i32([290])
    k, v = b.k.nan_to_num(0.5), b.v.nan_to_num(0.5)
    for shared in ([t[:, :, 1:2].expand_as(t) for t in (k, v)], [t[3:4].expand_as(t) for t in (k, v)], [t[:, 2:3].expand_as(t) for t in (k, v)]):
        whole, flat = csa.PagedCache(*(t.contiguous() for t in shared)), csa.PagedCache(*shared)
        for f in (lambda c: ctx.prompt_attn(q, c, b.table, cu, i32(b.lens), b.scale, with_lse=True),
                  lambda c: ctx.prefix_attn(q[:3].contiguous(), c, b.table, pos, b.table[1:2].contiguous(), prefix_len, b.scale,
                                            with_lse=True)):
            (o, lse), (o2, lse2) = f(whole), f(flat)
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd", [(8, 2, 128), (16, 2, 64), (6, 1, 256), (18, 2, 128)])
def test_prompt_single_tokens_in_place(csa, ctx, H, kv, hd):
    """Decodes and prompts whose results take the place of their queries."""
    lens, new = [6000, 40, 1, 333, 9000, 64], [1, 40, 1, 100, 1, 0]
    b = Batch(lens, H, kv, hd, 16, seed=3 * hd)
    q = b.queries(sum(new) + 2)
    o, lse = ctx.prompt_attn(q, csa.PagedCache(b.k, b.v), b.table, i32(cus(new)), i32(lens), b.scale, with_lse=True)
    for _ in range(5):
        p = q.clone()
        o2, lse2 = ctx.prompt_attn(p, csa.PagedCache(b.k, b.v), b.table, i32(cus(new)), i32(lens), b.scale, out=p, with_lse=True)
        n = sum(new)
        assert o2 is p and torch.equal(p[:n], o[:n]) and torch.equal(lse2[:n], lse[:n]) and torch.equal(p[n:], q[n:])
    check_prompt(b, new, q, o, lse)
    assert ctx.status() == 0


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_prompt_extreme_scores(csa, ctx, hd):
    """Scores of +-thousands, a scale of either sign and of 0, sinks far above and below and infinite."""
    H, kv, lens, new = 8, 2, [200, 64, 1], [200, 10, 1]
    b = Batch(lens, H, kv, hd, 16, seed=8)
    q = b.queries(sum(new))
    args = (q, csa.PagedCache(b.k, b.v), b.table, i32(cus(new)), i32(lens))
    for scale in (40.0, -40.0, 0.0, 1e-3):
        for sink in (None, torch.full((H,), -1e4, device="cuda"), torch.full((H,), 50.0, device="cuda")):
            o, lse = ctx.prompt_attn(*args, scale, sink=sink, with_lse=True)
            check_prompt(b, new, q, o, lse, sink, scale=scale)
    assert (ctx.prompt_attn(*args, b.scale, sink=torch.full((H,), float("inf"), device="cuda")) == 0).all()
    o = ctx.prompt_attn(*args, b.scale, sink=torch.full((H,), float("-inf"), device="cuda"))
    check_prompt(b, new, q, o, None)


def test_prompt_growing_scores(csa, ctx):
    """Maxima that grow along the row, by little and by much, so that sums so far are rescaled again and again."""
    H, kv, hd, n = 4, 2, 128, 1500
    b = Batch([n], H, kv, hd, 16, seed=4)
    for step in (0.01, 0.3):
        grow = torch.arange(n, device="cuda").float() * step
        b.rows_k[0][:] = (torch.randn(n, kv, hd, generator=b.g, device="cuda") * 0.1).to(torch.bfloat16)
        b.rows_k[0][:, :, 0] = grow[:, None].to(torch.bfloat16)
        p = torch.arange(n, device="cuda")
        b.k[b.table[0].long()[p // 16], p % 16] = b.rows_k[0]
        q = b.queries(n, 0.5)
        q[..., 0] = 1.0
        o, lse = ctx.prompt_attn(q, csa.PagedCache(b.k, b.v), b.table, i32([0, n]), i32([n]), 1.0, with_lse=True)
        check_prompt(b, [n], q, o, lse, scale=1.0)


@pytest.mark.parametrize("hd", [64, 128, 192, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_prompt_values_that_are_not_finite(csa, ctx, hd, bad):
    """A NaN or an infinity reaches the tokens that attend its row, in its feature, and no others; as a key their whole head."""
    H, kv, lens, new, page = 8, 2, [300, 700, 40], [300, 450, 40], 16
    g = H // kv
    b = Batch(lens, H, kv, hd, page, seed=2)
    q = b.queries(sum(new))
    for window in (0, 150):
        def run():
            return ctx.prompt_attn(q, csa.PagedCache(b.k, b.v), b.table, i32(cus(new)), i32(lens), b.scale, window=window,
                                   with_lse=True)
        want, want_lse = run()
        for r, p in ((0, 0), (0, 131), (0, 299), (1, 100), (1, 255), (1, 256), (1, 600)):
            at = (int(b.table[r, p // page]), p % page)
            t = torch.arange(sum(new), device="cuda")
            pos = t - cus(new)[r + 1] + lens[r]
            hit = (t >= cus(new)[r]) & (t < cus(new)[r + 1]) & (pos >= p)
            if window:
                hit &= pos < p + window
            keep = b.v[at].clone()
            b.v[at][1, 3] = bad
            o, lse = run()
            b.v[at] = keep
            assert torch.equal(o[~hit], want[~hit]) and torch.equal(lse, want_lse)
            assert not o[hit][:, g:, 3].isfinite().any()
            rest = [d for d in range(hd) if d != 3]
            assert torch.equal(o[hit][:, :, rest], want[hit][:, :, rest]) and torch.equal(o[hit][:, :g], want[hit][:, :g])
            keep = b.k[at].clone()
            b.k[at][1] = float("nan")
            o, lse = run()
            b.k[at] = keep
            assert torch.equal(o[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
            assert o[hit][:, g:].isnan().all() and lse[hit][:, g:].isnan().all() and torch.equal(o[hit][:, :g], want[hit][:, :g])
    # everywhere at once: more bad rows than any list of them holds
    b.v.view(torch.int16)[..., 1] = torch.tensor([bad], dtype=torch.bfloat16).view(torch.int16).item()
    o, _ = run()
    assert not o[..., 1].isfinite().any() and torch.equal(o[..., 2:], want[..., 2:]) and torch.equal(o[..., 0], want[..., 0])
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd,page", [(8, 1, 128, 16), (16, 2, 64, 17), (9, 1, 128, 16), (24, 8, 256, 8), (18, 2, 192, 64),
                                          (5, 1, 80, 1), (17, 1, 256, 16)])
@pytest.mark.parametrize("window,sink", [(0, False), (150, True)])
def test_prompt_single_tokens(csa, ctx, H, kv, hd, page, window, sink):
    """Decoding requests alone, one behind padding, among chunks and prompts, on both sides of 8 heads a key head; the rows
    that a window hides hold nothing that counts."""
    for lens, new, pad in (([700], [1], 0), ([700], [1], 5), ([1], [1], 3), ([1, 2, 33, 0, 5000, 64, 65], [1] * 3 + [0] + [1] * 3, 2),
                           ([900, 3, 1, 400, 2000, 17], [1, 3, 1, 200, 1, 0], 0), ([129] * 90, [1, 2, 1] * 30, 7)):
        b = Batch(lens, H, kv, hd, page, seed=len(lens) * hd + pad)
        sw = torch.randn(H, generator=b.g, device="cuda") if sink else None
        q, o, lse = prompt(csa, ctx, b, new, pad=pad, sink=sw, window=window)
        check_prompt(b, new, q, o, lse, sw, window)
        if not window:
            continue
        pages = {}  # (the rows before every window, not finite)
        for r, n in enumerate(lens):
            for j in range(max(0, n - new[r] - window + 1)):
                pages.setdefault(int(b.table[r, j // page]), []).append(j % page)
        for at, rows in pages.items():
            b.k[at, rows], b.v[at, rows] = float("nan"), float("inf")
        o2, lse2 = ctx.prompt_attn(q, csa.PagedCache(b.k, b.v), b.table, i32(cus(new)), i32(lens), b.scale, sink=sw, window=window,
                                   with_lse=True)
        n = sum(new)
        assert torch.equal(o2[:n], o[:n]) and torch.equal(lse2[:n], lse[:n])
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv", [(8, 2), (9, 1)])
def test_prompt_single_token_errors(csa, ctx, H, kv):
    """A decoding request's length, page or place that cannot be: recorded, its row left or what is there attended, and no other's."""
    lens, new = [300, 64, 50, 90], [1, 1, 20, 1]
    b = Batch(lens, H, kv, 128, 16, seed=77)
    q, cache = b.queries(sum(new) + 2), csa.PagedCache(b.k, b.v)

    def run(table=b.table, cu=cus(new), lens=lens):
        out, lse = torch.full_like(q, 3.0), torch.full(q.shape[:2], 3.0, device="cuda")
        ctx.prompt_attn(q, cache, table, i32(cu), i32(lens), b.scale, out=out, lse=lse)
        return out, lse

    for le, row, rest in (([300, 0, 50, 90], 1, [0, 2, 3]), ([-5, 64, 50, 90], 0, [1, 2, 3])):
        o, lse = run(lens=le)
        assert ctx.status() == -1 and ctx.status() == 0
        assert (o[row] == 3).all() and (lse[row] == 3).all()
        check_prompt(b, new, q, o, lse, only=rest)
    o, lse = run(cu=[0, 1, 2, 22, q.shape[0] + 1])
    assert ctx.status() == -1 and ctx.status() == 0
    assert (o[22:] == 3).all() and (lse[22:] == 3).all()
    check_prompt(b, new, q, o, lse, only=[0, 1, 2])
    o, lse = run(table=b.table[:, :10].contiguous())  # 300 positions in 160: those
    assert ctx.status() == -1 and ctx.status() == 0
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    close(o[:1], lse[:1], ref(q[:1], b.rows_k[0][:160], b.rows_v[0][:160], kv, b.scale, None, zero, zero + 159), "past the table")
    check_prompt(b, new, q, o, lse, only=[1, 2, 3])
    t = b.table.clone()
    t[3, 0] = -1  # no page: its rows are left out
    o, lse = run(table=t)
    assert ctx.status() == -1 and ctx.status() == 0
    close(o[22:23], lse[22:23], ref(q[22:23], b.rows_k[3][16:90], b.rows_v[3][16:90], kv, b.scale, None, zero, zero + 73), "no page")
    check_prompt(b, new, q, o, lse, only=[0, 1, 2])


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_prompt_caller_errors(csa, ctx, hd):
    """Each is recorded, and nothing else of the call suffers."""
    H, kv, page = 8, 2, 16
    lens, new = [48, 400, 48], [48, 200, 5]
    b = Batch(lens, H, kv, hd, page, seed=9)
    q = b.queries(sum(new) + 4)
    cache = csa.PagedCache(b.k, b.v)
    cu = cus(new)

    def run(table=b.table, cu=cu, lens=lens):
        out, lse = torch.full_like(q, 3.0), torch.full(q.shape[:2], 3.0, device="cuda")
        ctx.prompt_attn(q, cache, table, i32(cu), i32(lens), b.scale, out=out, lse=lse)
        return out, lse

    for bad in (-1, b.n_pages, 2 ** 31 - 1):  # a page outside the pool: its rows are left out
        t = b.table.clone()
        t[1, 3] = bad
        o, lse = run(t)
        assert ctx.status() == -1 and ctx.status() == 0
        check_prompt(b, new, q, o, lse, only=[0, 2])
        keep = torch.cat([torch.arange(48), torch.arange(64, 400)]).cuda()
        last = torch.arange(200, device="cuda") + 200 - 16
        close(o[48:248], lse[48:248], ref(q[48:248], b.rows_k[1][keep], b.rows_v[1][keep], kv, b.scale, None,
                                          torch.zeros_like(last), last), "bad page")
    # lengths below the new tokens, tokens past N, borders that fall: the request's rows are left as they were
    N = q.shape[0]
    for c, le, rows in (([0, 48, 248, 253], [48, 199, 48], (48, 248)), ([0, 48, 248, 253], [48, -1, 48], (48, 248)),
                        ([0, 48, 248, N + 1], lens, (248, N)), ([-1, 48, 248, 253], lens, (0, 48))):
        o, lse = run(cu=c, lens=le)
        assert ctx.status() == -1 and ctx.status() == 0
        assert (o[rows[0]:rows[1]] == 3).all() and (lse[rows[0]:rows[1]] == 3).all()
        check_prompt(b, new, q, o, lse, only=[r for r in range(3) if cu[r] >= rows[1] or cu[r + 1] <= rows[0]])
    o, lse = run(cu=[0, 48, 40, 253])
    assert ctx.status() == -1 and ctx.status() == 0
    check_prompt(b, new, q, o, lse, only=[0])
    # a length past the table: its rows there alone
    t = b.table[:, :10].contiguous()
    o, lse = run(t)
    assert ctx.status() == -1 and ctx.status() == 0
    last = torch.arange(200, device="cuda") + 200
    close(o[48:248], lse[48:248], ref(q[48:248], b.rows_k[1][:160], b.rows_v[1][:160], kv, b.scale, None, torch.zeros_like(last),
                                      last), "past the table")
    check_prompt(b, new, q, o, lse, only=[0, 2])


@pytest.mark.parametrize("window", [0, 1000])
def test_prompt_rows_up_to_2_31(csa, ctx, window):
    """Tokens at the last positions that a table may hold: all scores 0, all values of a feature the same power of two."""
    H, kv, hd, page, n = 4, 2, 64, 2 ** 20, 300
    width = (2 ** 31 - 1) // page
    rows = width * page + (0 if window else -width * page + 2 ** 22)
    row = 2.0 ** (torch.arange(hd, device="cuda") % 5 - 2)
    k = row.to(torch.bfloat16).expand(2, page, kv, hd).contiguous()
    table = (torch.arange(width, device="cuda", dtype=torch.int32) % 2)[None].contiguous()
    q = torch.zeros(n, H, hd, dtype=torch.bfloat16, device="cuda")
    o, lse = ctx.prompt_attn(q, csa.PagedCache(k), table, i32([0, n]), i32([rows]), 1.0, window=window, with_lse=True)
    assert torch.equal(o, row.to(torch.bfloat16).expand(n, H, hd))
    want = torch.log((torch.arange(n, device="cuda") + rows - n + 1).clamp(max=window or rows).double())[:, None]
    assert ((lse.double() - want).abs() <= 640 * 2.0 ** -24 + 2.0 ** -21 * want).all()
    assert ctx.status() == 0


def test_prompt_far_offsets(csa, ctx):
    """A pool above 2^31 elements, and tokens that lie 2^30 elements apart."""
    page, kv, hd, H = 64, 8, 128, 32
    n_pages = 2 ** 31 // (page * kv * hd) + 40
    k = torch.zeros(n_pages, page, kv, hd, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    b = Batch([200], H, kv, hd, page, seed=10)
    ids = torch.tensor([n_pages - 1, 3, n_pages - 20, n_pages - 2], device="cuda")
    src = b.table[0, :4].long()
    k[ids], v[ids] = b.k[src], b.v[src]
    wide = torch.zeros(3, 2 ** 30, dtype=torch.bfloat16, device="cuda")
    q = wide[:, :H * hd].view(3, H, hd)
    q.copy_(b.queries(3))
    args = (csa.PagedCache(k, v), ids.to(torch.int32)[None].contiguous(), i32([0, 3]), i32([200]), b.scale)
    o, lse = ctx.prompt_attn(q, *args, with_lse=True)
    check_prompt(b, [3], q, o, lse)
    assert torch.equal(ctx.prompt_attn(q, *args, out=q), o)
    o2 = ctx.prefix_attn(o, csa.PagedCache(k, v), i32([[3]] * 3), i32([-1] * 3), args[1], i32([200]), b.scale)
    last = torch.full((3,), 199, device="cuda")
    close(o2, None, ref(o, b.rows_k[0], b.rows_v[0], kv, b.scale, None, last * 0, last), "prefix")
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd", [(8, 2, 128), (16, 1, 256), (4, 2, 64)])
def test_weights_add_up_to_one(csa, ctx, H, kv, hd):
    """A feature that is the same in all rows comes back as it is: the denominator adds up what the weights are rounded to for their
    product.  Every 40th row scores higher by so much that a weight of the others, 1.003875 / 2, lies just below a
    border of bf16's and loses 2^-8.04 of itself: with the weights as they were in the denominator, 1.9921875 would become
    1.984375.  The f32 errors of a sum of 4000 products are at most 2^-12 of it, half a step is 2^-9.  lse is of the
    weights as they were."""
    n, page, scale, same = 4000, 16, 0.68928, 255 / 128
    k = torch.full((n // page, page, kv, hd), same, dtype=torch.bfloat16, device="cuda")
    k[..., 0] = 0
    k.view(n, kv, hd)[20::40, :, 0] = 1
    v = k.clone()
    q = torch.zeros(n, H, hd, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    table = torch.arange(n // page, device="cuda", dtype=torch.int32)[None]
    cache = csa.PagedCache(k, v)
    o, lse = ctx.prompt_attn(q, cache, table, i32([0, n]), i32([n]), scale, with_lse=True)
    assert (o[..., 1:].float() == same).all()
    rows = torch.arange(1, n + 1, device="cuda").double()
    high = ((rows - 21).div(40, rounding_mode="floor") + 1).clamp(min=0)
    want = torch.log(high * math.exp(scale) + rows - high)[:, None]
    assert ((lse.double() - want).abs() <= 2.0 ** -20 * (1 + want) + n * 2.0 ** -24).all()
    o, lse = ctx.prefix_attn(q[:8], cache, table.expand(8, -1).contiguous(), i32([-1, 0, 39, 40, 400, 800, 1000, 3999]), table,
                             i32([n]), scale, with_lse=True)
    assert (o[..., 1:].float() == same).all() and ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd", [(8, 2, 128), (20, 1, 256), (12, 4, 64)])
def test_prompt_streams_contexts_and_graphs(csa, ctx, H, kv, hd):
    """Two contexts at once on two streams; two captured graphs of one context replayed by turns while lengths change."""
    lens, new = [3000, 900, 25, 2500], [1, 700, 25, 300]
    b = Batch(lens, H, kv, hd, 16, seed=11)
    q = b.queries(sum(new))
    cache, cu, length = csa.PagedCache(b.k, b.v), i32(cus(new)), i32(lens)
    want = ctx.prompt_attn(q, cache, b.table, cu, length, b.scale)
    other = make_ctx(csa)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got.append(ctx.prompt_attn(q, cache, b.table, cu, length, b.scale, stream=s1))
        got.append(other.prompt_attn(q, cache, b.table, cu, length, b.scale, stream=s2))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
    other.close()
    cus_ = [cu, i32([0, 0, 5, 5, 9])]
    lengths = [length, i32([7, 900, 3, 64])]
    outs = [torch.zeros_like(q) for _ in range(2)]
    graphs = []
    for c, le, o in zip(cus_, lengths, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ctx.prompt_attn(q, cache, b.table, c, le, b.scale, out=o)
        graphs.append(g)
    for step in range(4):
        if step == 2:
            cus_[0].copy_(i32([0, 500, 501, 501, 502]))
            lengths[0].copy_(i32([500, 1, 0, 2001]))
        wants = []
        for c, le, o in zip(cus_, lengths, outs):
            o.zero_()
            wants.append(ctx.prompt_attn(q, cache, b.table, c, le, b.scale, out=torch.zeros_like(q)))
        for g in graphs:
            g.replay()
        assert all(torch.equal(o, w) for o, w in zip(outs, wants))
    assert ctx.status() == 0


# ------------------------------------------------------------------------------------------ shared prefixes

class Prefixes:
    """Own rows of each request and rows of each prefix over one pool; what nobody holds is NaN."""

    def __init__(self, own, plens, H, kv, hd, page, latent=False, order="nhd", seed=0):
        b = Batch(list(own) + list(plens), H, kv, hd, page, latent, order, seed)
        n = len(own)
        self.b, self.own, self.plens, self.n = b, list(own), list(plens), n
        self.table, self.prefix = b.table[:n].contiguous(), b.table[n:].contiguous()
        self.k, self.v, self.scale = b.k, b.v, b.scale

    def check(self, q, o, lse, pos, group, req=None, sink=None, window=0, scale=None):
        for n in range(len(pos)):
            b, L = self.b, self.plens[group[n]]
            r, p = (n if req is None else req[n]), self.n + group[n]
            K = torch.cat([b.rows_k[p], b.rows_k[r][:pos[n] + 1]])
            V = torch.cat([b.rows_v[p], b.rows_v[r][:pos[n] + 1]])
            last = torch.tensor([L + pos[n]], device="cuda")
            first = (last + 1 - window).clamp(min=0) if window else last * 0
            close(o[n:n + 1], None if lse is None else lse[n:n + 1],
                  ref(q[n:n + 1], K, V, b.kv, b.scale if scale is None else scale, sink, first, last), "row %d" % n)


OWN = [1, 0, 2, 15, 16, 17, 63, 64, 65, 127, 129, 300]


@pytest.mark.parametrize("H,kv,hd,page,latent,order,window,sink", SHAPES)
@pytest.mark.parametrize("plens", [[333], [200, 0, 65]])
def test_prefix(csa, ctx, H, kv, hd, page, latent, order, window, sink, plens):
    P = Prefixes(OWN, plens, H, kv, hd, page, latent, order, seed=H * hd)
    sw = torch.randn(H, generator=P.b.g, device="cuda") if sink else None
    N = len(OWN)
    q = P.b.queries(N)
    cu = None if len(plens) == 1 else [0, 5, 9, N]
    group = [0] * N if cu is None else [0] * 5 + [1] * 4 + [2] * 3
    pos = [x - 1 for x in OWN]
    o, lse = ctx.prefix_attn(q, csa.PagedCache(P.k, P.v), P.table, i32(pos), P.prefix, i32(plens), P.scale,
                             cu=None if cu is None else i32(cu), sink=sw, window=window, with_lse=True)
    P.check(q, o, lse, pos, group, None, sw, window)
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd", [(8, 2, 128), (16, 16, 64), (12, 1, 256), (9, 3, 192)])
@pytest.mark.parametrize("n,own,plen", [(1, 5, 1), (1, 0, 20000), (2, 3000, 9000), (70, 40, 2000), (300, 3, 777), (33, 200, 0), (5, 0, 0)])
def test_prefix_lengths(csa, ctx, H, kv, hd, n, own, plen):
    """One row, many, none of their own, no prefix; the same bits again."""
    P = Prefixes([max(0, own - i % 7) for i in range(n)], [plen], H, kv, hd, 16, seed=n + hd)
    q = P.b.queries(n)
    pos = [x - 1 for x in P.own]
    args = (csa.PagedCache(P.k, P.v), P.table, i32(pos), P.prefix, i32([plen]), P.scale)
    o, lse = ctx.prefix_attn(q, *args, with_lse=True)
    P.check(q, o, lse, pos, [0] * n)
    for _ in range(3):
        o2, lse2 = ctx.prefix_attn(q, *args, with_lse=True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    mine = q.clone()
    assert ctx.prefix_attn(mine, *args, out=mine) is mine and torch.equal(mine, o)
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd", [(8, 2, 128), (4, 1, 256)])
def test_prefix_rows_of_requests(csa, ctx, H, kv, hd):
    """Several rows of one request, padding in all its forms, strided rows, windows that end inside the prefix and behind it."""
    P = Prefixes([70, 300, 9], [500, 90], H, kv, hd, 16, seed=3)
    req = [2, 1, 1, 1, -1, 0, 2, 0, 2, 1, 0]
    pos = [3, 0, 299, 150, 5, 69, 8, -1, -2, 298, 7]
    cu, N = [1, 4, 10], len(req)  # (row 0 and row 10 are nobody's)
    group = [0] * 4 + [1] * 7
    wide = randn(P.b.g, N, H * hd + 64, scale=1.5)
    q = wide[:, 8:8 + H * hd].view(N, H, hd)
    sink = torch.randn(H, generator=P.b.g, device="cuda")
    live = [n for n in range(1, 10) if req[n] >= 0 and pos[n] >= -1]
    for window in (0, 1, 60, 200, 430):
        buf = torch.full((N, H * hd + 16), 3.0, dtype=torch.bfloat16, device="cuda")
        out = buf[:, :H * hd].view(N, H, hd)
        lse = torch.full((N, H), 3.0, device="cuda")
        ctx.prefix_attn(q, csa.PagedCache(P.k, P.v), P.table, i32(pos), P.prefix, i32([500, 90]), P.scale, cu=i32(cu), req=i32(req),
                        sink=sink, window=window, out=out, lse=lse)
        P.check(q[live], out[live], lse[live], [pos[n] for n in live], [group[n] for n in live], [req[n] for n in live], sink, window)
        for n in set(range(N)) - set(live):
            assert (out[n] == 3).all() and (lse[n] == 3).all()
        assert (buf[:, H * hd:] == 3).all() and ctx.status() == 0


@pytest.mark.parametrize("hd", [64, 256])
def test_prefix_extreme_scores(csa, ctx, hd):
    H, kv, own = 8, 2, [60, 1, 0, 300]
    P = Prefixes(own, [200], H, kv, hd, 16, seed=8)
    pos = [x - 1 for x in own]
    q = P.b.queries(4)
    args = (q, csa.PagedCache(P.k, P.v), P.table, i32(pos), P.prefix, i32([200]))
    for scale in (40.0, -40.0, 0.0, 1e-3):
        for sink in (None, torch.full((H,), -1e4, device="cuda"), torch.full((H,), 50.0, device="cuda")):
            o, lse = ctx.prefix_attn(*args, scale, sink=sink, with_lse=True)
            P.check(q, o, lse, pos, [0] * 4, None, sink, scale=scale)
    assert (ctx.prefix_attn(*args, P.scale, sink=torch.full((H,), float("inf"), device="cuda")) == 0).all()


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prefix_values_that_are_not_finite(csa, ctx, hd, bad):
    """In the prefix: the rows of that prefix whose window reaches it; in a request's own rows: that request's."""
    H, kv, own, page = 8, 2, [300, 40, 0, 90, 5, 7], 16
    g = H // kv
    P = Prefixes(own, [500, 300], H, kv, hd, page, seed=2)
    q = P.b.queries(6)
    pos = torch.tensor([x - 1 for x in own])

    def run(window):
        return ctx.prefix_attn(q, csa.PagedCache(P.k, P.v), P.table, i32(pos.tolist()), P.prefix, i32([500, 300]), P.scale,
                               cu=i32([0, 4, 6]), window=window, with_lse=True)

    for window, at in ((0, 3), (0, 499), (200, 490), (200, 330), (450, 100)):
        want, want_lse = run(window)
        hit = torch.tensor([n < 4 and (not window or 500 + int(pos[n]) < at + window) for n in range(6)]).cuda()
        where = (int(P.prefix[0, at // page]), at % page)
        keep = P.v[where].clone()
        P.v[where][1, 3] = bad
        o, lse = run(window)
        P.v[where] = keep
        assert torch.equal(o[~hit], want[~hit]) and torch.equal(lse, want_lse) and torch.equal(o[:, :g], want[:, :g])
        assert not o[hit][:, g:, 3].isfinite().any()
        rest = [d for d in range(hd) if d != 3]
        assert torch.equal(o[..., rest], want[..., rest])
    where = (int(P.table[3, 2]), 4)
    P.v[where][1, 3] = bad
    o, _ = run(0)
    want, _ = run(0)
    assert not o[3, g:, 3].isfinite().any() and o[[0, 1, 2, 4, 5]].isfinite().all()
    assert ctx.status() == 0


def test_prefix_caller_errors(csa, ctx):
    H, kv, hd, page = 8, 2, 128, 16
    P = Prefixes([48, 48, 48], [96], H, kv, hd, page, seed=9)
    q = P.b.queries(3)
    cache = csa.PagedCache(P.k, P.v)

    def run(table=P.table, pos=(47, 47, 47), prefix=P.prefix, plen=(96,), **kw):
        out = torch.full_like(q, 3.0)
        ctx.prefix_attn(q, cache, table, i32(list(pos)), prefix, i32(list(plen)), P.scale, out=out, **kw)
        return out

    keep = torch.cat([torch.arange(32), torch.arange(48, 96)]).cuda()
    for bad in (-1, P.b.n_pages, 2 ** 31 - 1):
        t = P.prefix.clone()
        t[0, 2] = bad
        o = run(prefix=t)
        assert ctx.status() == -1 and ctx.status() == 0
        K, V = P.b.rows_k[3], P.b.rows_v[3]
        P.b.rows_k[3], P.b.rows_v[3], P.plens[0] = K[keep], V[keep], 80
        P.check(q, o, None, [47] * 3, [0] * 3)
        P.b.rows_k[3], P.b.rows_v[3], P.plens[0] = K, V, 96
    o = run(req=i32([0, 3, 2]))
    assert ctx.status() == -1 and (o[1] == 3).all()
    P.check(q[[0, 2]], o[[0, 2]], None, [47] * 2, [0] * 2, [0, 2])
    o = run(plen=(-5,))
    assert ctx.status() == -1
    want = ctx.paged_attn(q, cache, P.table, i32([47] * 3), P.scale)
    assert ((o.double() - want.double()).abs() <= 2.0 ** -7 * want.double().abs()).all()  # (two roundings of nearly the same)
    o = run(prefix=P.prefix[:, :4].contiguous())
    assert ctx.status() == -1
    P.b.rows_k[3], P.b.rows_v[3], P.plens[0] = P.b.rows_k[3][:64], P.b.rows_v[3][:64], 64
    P.check(q, o, None, [47] * 3, [0] * 3)
    for cu in ([0, 2, 1], [-1, 1, 3], [0, 2, 4]):  # the second, the first, the second prefix's rows are left as they were
        o = run(prefix=P.prefix.expand(2, -1).contiguous(), plen=(64, 64), cu=i32(cu))
        assert ctx.status() == -1 and ctx.status() == 0
        rows = [0, 1] if cu[0] == 0 else [1, 2]
        P.check(q[rows], o[rows], None, [47] * 2, [0] * 2, rows)
        assert (o[2 if cu[0] == 0 else 0] == 3).all()


def test_prefix_replayed(csa, ctx):
    """Two graphs of one context by turns, prefix lengths and positions changed between."""
    H, kv, hd = 8, 2, 128
    P = Prefixes([300, 0, 64, 2000], [3000, 500], H, kv, hd, 16, seed=5)
    q = P.b.queries(4)
    cache = csa.PagedCache(P.k, P.v)
    pos = [i32([299, -1, 63, 1999]), i32([0, -2, 5, 700])]
    plen, cu = [i32([3000, 500]), i32([9, 0])], [i32([0, 1, 4]), i32([0, 3, 4])]
    outs, graphs = [torch.zeros_like(q) for _ in range(2)], []

    def run(i, out):
        return ctx.prefix_attn(q, cache, P.table, pos[i], P.prefix, plen[i], P.scale, cu=cu[i], out=out)

    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(i, outs[i])
        graphs.append(g)
    for step in range(4):
        if step == 2:
            pos[0].copy_(i32([20, -1, 3, 0]))  # (request 1 has no rows of its own)
            plen[0].copy_(i32([1, 499]))
        want = [run(i, torch.zeros_like(q)) for i in range(2)]
        for i in range(2):
            outs[i].zero_()
            graphs[i].replay()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = ctx.prefix_attn(q, cache, P.table, pos[1], P.prefix, plen[1], P.scale, cu=cu[1], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got[[0, 2, 3]], want[1][[0, 2, 3]]) and ctx.status() == 0


def test_workspace(csa, ctx):
    """More rows of a prefix batch than the context's workspace holds shares for: refused, and nothing is written."""
    H, hd, N = 64, 128, 4096
    b = Batch([40], H, 8, hd, 16)
    q = torch.full((N, H, hd), 3.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(csa.CsaError, match="workspace") as e:
        ctx.prefix_attn(q, csa.PagedCache(b.k, b.v), b.table, i32([39] * N), b.table, i32([40]), 0.1, req=i32([0] * N), out=q)
    assert e.value.code == -2
    torch.cuda.synchronize()
    assert (q == 3).all() and ctx.status() == 0


@pytest.mark.parametrize("hd", [64, 256])
def test_prompt_last_positions(csa, ctx, hd):
    """Tokens whose tile of positions ends past 2^31: a NaN behind a token's position does not reach it there either."""
    H, kv, page, n = 2, 1, 2 ** 16, 200
    width = (2 ** 31 - 1) // page
    rows, window = width * page, 90
    k = torch.ones(2, page, kv, hd, dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    table = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    v[1, page - 100, 0, 5] = float("nan")
    q = torch.zeros(n, H, hd, dtype=torch.bfloat16, device="cuda")
    o = ctx.prompt_attn(q, csa.PagedCache(k, v), table, i32([0, n]), i32([rows]), 1.0, window=window)
    pos = torch.arange(n, device="cuda") - n + page
    hit = (pos >= page - 100) & (pos < page - 100 + window)
    assert o[hit][..., 5].isnan().all() and (o[~hit] == 1).all()
    o[..., 5] = 1
    assert (o == 1).all() and ctx.status() == 0


def test_no_tokens(csa, ctx):
    b = Batch([40], 8, 2, 64, 16)
    cache, none = csa.PagedCache(b.k, b.v), i32([])
    e = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = ctx.prompt_attn(e, cache, b.table, i32([0, 0]), i32([40]), 0.1, with_lse=True)
    assert o.shape == (0, 8, 64) and lse.shape == (0, 8)
    o, lse = ctx.prefix_attn(e, cache, b.table, none, b.table, i32([40]), 0.1, with_lse=True)
    assert o.shape == (0, 8, 64) and lse.shape == (0, 8)
    # nothing but padding
    q = b.queries(3)
    out = torch.full_like(q, 3.0)
    ctx.prompt_attn(q, cache, b.table, i32([0, 0]), i32([-7]), 0.1, out=out)
    ctx.prefix_attn(q, cache, b.table, i32([-2] * 3), b.table, i32([40]), 0.1, req=i32([0] * 3), out=out)
    assert (out == 3).all() and ctx.status() == 0


# ------------------------------------------------------------------------------------------ together

@pytest.mark.parametrize("H,kv,hd,page", [(16, 4, 128, 16), (10, 2, 80, 17)])
def test_prompts_then_decodes_in_a_graph(csa, ctx, H, kv, hd, page):
    """A server's steps: page_step in place, projection, qk_norm_rope into the pages, prompt_attn for whatever tokens the step has
    (prompts, chunks, decodes), captured once and replayed; then a decode step of all behind a shared prefix.  Every
    attention against its 64-bit form over the rows that the steps wrote."""
    dim, N, R, n_pages, width = 256, 700, 5, 120, 60
    g = gen(21)
    lens = [0, 0, 0, 0, 0]
    pool = Pool(n_pages, page, lens, 3)
    table, free, state, length = i32(pool.table(width)), i32(pool.ring(5)), i32([5, len(pool.free)]), i32(lens)
    new, cu = i32([1] * R), i32([0] * (R + 1))
    maps = [torch.empty(N, dtype=torch.int32, device="cuda") for _ in range(3)]
    cache = csa.PagedCache(randn(g, n_pages, page, kv, hd), randn(g, n_pages, page, kv, hd))
    W = randn(g, (H + 2 * kv) * hd, dim, scale=dim ** -0.5)
    x = randn(g, N, dim)
    qn, kn = (1 + 0.1 * torch.randn(hd, generator=g, device="cuda") for _ in range(2))
    tab = rope_tab(1500, hd)
    sink = torch.randn(H, generator=g, device="cuda")
    y = torch.empty(N, (H + 2 * kv) * hd, dtype=torch.bfloat16, device="cuda")
    q = torch.full((N, H, hd), 5.0, dtype=torch.bfloat16, device="cuda")
    o = torch.full((N, H, hd), 5.0, dtype=torch.bfloat16, device="cuda")
    scale = hd ** -0.5

    def step():
        csa.page_step(new, length, table, free, state, page, *maps, cu)
        ctx.linear(x, W, out=y)
        yq, yk, yv = (y[:, a * hd:e * hd].view(N, e - a, hd) for a, e in ((0, H), (H, H + kv), (H + kv, H + 2 * kv)))
        ctx.qk_norm_rope(yq, yk, yv, cache, maps[1], maps[2], tab=tab, rd=hd, half=True, q_norm=qn, k_norm=kn, q_out=q)
        ctx.prompt_attn(q, cache, table, cu, length, scale, sink=sink, out=o)

    def rows(ids, n):
        j = torch.arange(n, device="cuda")
        ids = torch.tensor(ids, device="cuda", dtype=torch.long)
        return (t[ids[j // page], j % page] for t in (cache.k, cache.v))

    graph = torch.cuda.CUDAGraph()
    before = [t.clone() for t in (table, free, state, length, cache.k, cache.v)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()  # warm-up, undone below
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for t, t0 in zip((table, free, state, length, cache.k, cache.v), before):
        t.copy_(t0)
    q.fill_(5.0)
    o.fill_(5.0)
    for st in ([300, 17, 0, 129, 1], [250, 1, 200, 1, 1], [1, 1, 1, -1, 33], [0] * R, [1, 1, 1, 90, 1]):
        new.copy_(i32(st))
        x.copy_(randn(g, N, dim))
        o_before = o.clone()
        graph.replay()
        torch.cuda.synchronize()
        toks, _, _ = pool.step(st)
        n = len(toks)
        assert length.tolist() == pool.lens and cu.tolist() == cus([max(s, 0) for s in st])
        pos = maps[1][:n]
        if n:
            close_rows(q[:n], ref_rows(y[:n, :H * hd].view(n, H, hd), qn, ctx.cfg.eps, tab, pos, hd, 0, True), "q")
        assert torch.equal(o[n:], o_before[n:])
        for r in range(R):
            a, e = int(cu[r]), int(cu[r + 1])
            if e > a:
                K, V = rows(pool.pages[r], pool.lens[r])
                last = pos[a:e].long()
                close(o[a:e], None, ref(q[a:e], K, V, kv, scale, sink, last * 0, last), "request %d" % r)
    # requests 1 to 4 answer behind request 0's rows as their prefix
    lens = pool.lens
    got, lse = ctx.prefix_attn(q[:4], cache, table, i32([x - 1 for x in lens[1:]]), table[:1], length[:1], scale, req=i32([1, 2, 3, 4]),
                               sink=sink, with_lse=True)
    for i in range(4):
        (K0, V0), (K1, V1) = rows(pool.pages[0], lens[0]), rows(pool.pages[i + 1], lens[i + 1])
        last = torch.tensor([lens[0] + lens[i + 1] - 1], device="cuda")
        close(got[i:i + 1], lse[i:i + 1], ref(q[i:i + 1], torch.cat([K0, K1]), torch.cat([V0, V1]), kv, scale, sink, last * 0, last),
              "answer %d" % i)
    # and the prefix's own split makes no difference to what paged_attn gives over the same rows in one table
    assert ctx.status() == 0
