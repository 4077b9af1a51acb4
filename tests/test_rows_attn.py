"""csa_prompt_attn and csa_prefix_attn on the GPU: values that are not finite behind long windows, calls right behind the
kernels that write their inputs, single tokens among many others and behind padding, lse where it is small,
the largest prefix batches, prefixes against the same rows in one table, bad values among own rows.

What a call leaves is compared bit for bit with what it leaves without the value: the sums of the other rows and features do not
change with it.
"""
import pytest
import torch

from test_paged import Batch, csa, ctx, gen, i32, randn  # noqa: F401
from test_prompt import Prefixes, check_prompt, close, cus, prompt, ref

pytestmark = pytest.mark.gpu


class Far:
    """1.2 million positions over eight pages by turns, of which two more pages hold a place each."""

    page, width, N, H, window = 4096, 300, 320, 128, 2 ** 20

    def __init__(self, hd, places):
        g = gen(hd)
        self.hd, self.rows = hd, self.page * self.width
        self.k, self.v = (randn(g, 8 + len(places), self.page, 1, hd) for _ in range(2))
        self.table = (torch.arange(self.width, device="cuda", dtype=torch.int32) % 8)[None].contiguous()
        for i, p in enumerate(places):
            self.table[0, p // self.page] = 8 + i
        self.q = randn(g, self.N, self.H, hd)

    def check(self, run, i, place, bad, hit):
        """The value at `place`, in the i-th page of its own, reaches the rows of `hit` in its feature, and nothing else."""
        want, want_lse = run()
        assert want.isfinite().all()
        at = (8 + i, place % self.page, 0, 3)
        keep = self.v[at].clone()
        self.v[at] = bad
        o, lse = run()
        self.v[at] = keep
        assert torch.equal(o[~hit], want[~hit]) and torch.equal(lse, want_lse)
        assert not o[hit][..., 3].isfinite().any()
        rest = [d for d in range(self.hd) if d != 3]
        assert torch.equal(o[..., rest], want[..., rest])


@pytest.mark.parametrize("hd", [64, 128, 192, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prefix_bad_value_in_a_long_window(csa, ctx, hd, bad):
    """More items than CTAs, windows of a million positions that begin at five different ones: a value at their edge, and one that
    every row attends."""
    first = Far.page * Far.width - Far.window  # of a row without rows of its own
    places = [first + 2, 700000]
    F = Far(hd, places)
    own = torch.arange(F.N, device="cuda", dtype=torch.int32) % 5 - 1
    args = (F.q, csa.PagedCache(F.k, F.v), F.table.expand(F.N, -1)[:, :1].contiguous(), own, F.table, i32([F.rows]), hd ** -0.5)
    for i, place in enumerate(places):
        hit = first + own + 1 <= place
        F.check(lambda: ctx.prefix_attn(*args, window=F.window, with_lse=True), i, place, bad, hit)
    assert ctx.status() == 0


@pytest.mark.parametrize("hd", [64, 128, 192, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
def test_prompt_bad_value_in_a_long_window(csa, ctx, hd, bad):
    """More items than CTAs, windows of a million positions: a value where the first ones begin, one in the middle of all, one
    among the tokens' own rows."""
    rows, w, N = Far.page * Far.width, Far.window, Far.N
    places = [rows - N + 101 - w, 700000, rows - 200]
    F = Far(hd, places)
    pos = torch.arange(N, device="cuda") + rows - N
    args = (F.q, csa.PagedCache(F.k, F.v), F.table, i32([0, N]), i32([rows]), hd ** -0.5)
    for i, place in enumerate(places):
        hit = (pos >= place) & (pos - w < place)
        F.check(lambda: ctx.prompt_attn(*args, window=w, with_lse=True), i, place, bad, hit)
    assert ctx.status() == 0


@pytest.mark.parametrize("hd", [64, 80, 192, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prefix_bad_values_in_every_tile(csa, ctx, hd, bad):
    """A feature without one finite value, in windows that begin in the prefix: the other features keep their bits."""
    own = [300, 40, 0, 90, 5, 7, 0, 1]
    P = Prefixes(own, [5000], 8, 2, hd, 16, seed=4)
    q = P.b.queries(8)

    def run():
        return ctx.prefix_attn(q, csa.PagedCache(P.k, P.v), P.table, i32([x - 1 for x in own]), P.prefix, i32([5000]), P.scale,
                               window=4000, with_lse=True)

    want, want_lse = run()
    P.v.view(torch.int16)[..., 1] = torch.tensor([bad], dtype=torch.bfloat16).view(torch.int16).item()
    o, lse = run()
    assert not o[..., 1].isfinite().any() and torch.equal(lse, want_lse)
    assert torch.equal(o[..., 2:], want[..., 2:]) and torch.equal(o[..., 0], want[..., 0])
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd", [(8, 2, 128), (4, 4, 64), (16, 2, 256), (18, 2, 128)])
def test_inputs_written_by_the_kernel_before(csa, ctx, H, kv, hd):
    """Calls in one graph, the inputs of each (queries, lengths, places, tables, a row of the cache) written by the kernels right before
    it: every call finds its own, not those of the call before."""
    lens, new = [3000, 900, 25, 2500, 64], [[1, 40, 1, 0, 1], [1, 1, 25, 300, 1], [0, 1, 1, 1, 64]]
    b = Batch(lens, H, kv, hd, 16, seed=hd)
    cache, N, R = csa.PagedCache(b.k, b.v), 400, len(lens)
    g = gen(hd + 1)
    steps = []
    for i, n in enumerate(new):
        order = torch.randperm(R, generator=torch.Generator().manual_seed(i)).tolist()
        length = [lens[r] - 3 * i for r in order]
        n = [min(a, x) for a, x in zip(n, length)]
        steps.append(dict(q=randn(g, N, H, hd), row=randn(g, kv, hd), table=b.table[order].contiguous(), cu=i32(cus(n)),
                          length=i32(length), pos=i32([x - 1 for x in length]), plen=i32([lens[i % R]])))
    now = {k: torch.empty_like(v) for k, v in steps[0].items()}
    last = cache.v[int(b.table[0, 0]), 0]

    def calls(s, o, p):
        for k, v in s.items():
            now[k].copy_(v)
        last.copy_(now["row"])
        ctx.prompt_attn(now["q"], cache, now["table"], now["cu"], now["length"], b.scale, out=o)
        now["q"].copy_(s["q"].flip(0))
        last.copy_(s["row"] * 2)
        ctx.prefix_attn(now["q"][:R], cache, now["table"], now["pos"], now["table"][:1], now["plen"], b.scale, out=p)

    def outs():
        return [(torch.zeros(N, H, hd, dtype=torch.bfloat16, device="cuda"), torch.zeros(R, H, hd, dtype=torch.bfloat16, device="cuda"))
                for _ in steps]

    want, got = outs(), outs()
    for s, (o, p) in zip(steps, want):
        torch.cuda.synchronize()
        calls(s, o, p)
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for s, (o, p) in zip(steps, got):
            calls(s, o, p)
    for _ in range(20):
        for o, p in got:
            o.zero_(), p.zero_()
        graph.replay()
        assert all(torch.equal(x, y) for a, e in zip(got, want) for x, y in zip(a, e))
    assert ctx.status() == -1 and ctx.status() == 0  # (prefixes that are longer than the pages behind them: recorded, left out)


@pytest.mark.parametrize("H,kv,hd", [(8, 2, 128), (4, 4, 64), (16, 2, 256), (9, 1, 128), (6, 2, 192)])
@pytest.mark.parametrize("lens,new", [([900], [1]), ([1], [1]), ([40], [17]), ([300, 64, 5000, 7], [1, 1, 1, 1]),
                                      ([700, 0, 2000, 130], [1, 0, 300, 1]), ([150, 90], [150, 20]), ([6000], [33])])
def test_padding_changes_no_bit(csa, ctx, H, kv, hd, lens, new):
    """The same batch with no padding rows, with a few, and with thousands, as a graph captured at its largest step has them."""
    b = Batch(lens, H, kv, hd, 16, seed=hd)
    n, cu, length, cache = sum(new), i32(cus(new)), i32(lens), csa.PagedCache(b.k, b.v)
    q = b.queries(n + 6000)
    o, lse = ctx.prompt_attn(q[:n], cache, b.table, cu, length, b.scale, with_lse=True)
    check_prompt(b, new, q, o, lse)
    for pad in (1, 511, 6000):
        out, lse2 = torch.full_like(q[:n + pad], 3.0), torch.full((n + pad, H), 3.0, device="cuda")
        ctx.prompt_attn(q[:n + pad], cache, b.table, cu, length, b.scale, out=out, lse=lse2)
        assert torch.equal(out[:n], o) and torch.equal(lse2[:n], lse) and (out[n:] == 3).all() and (lse2[n:] == 3).all()
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd,page", [(8, 2, 128, 16), (16, 2, 64, 17), (4, 4, 256, 16), (18, 2, 128, 16)])
@pytest.mark.parametrize("window", [0, 600])
def test_single_tokens_beside_long_chunks(csa, ctx, H, kv, hd, page, window):
    """Decodes, short and long, in a batch of more than 512 tokens a request: on either side of 8 heads a key head."""
    lens, new = [5000, 3400, 1, 33, 9000], [1, 2900, 1, 1, 1]
    b = Batch(lens, H, kv, hd, page, seed=hd)
    sink = torch.randn(H, generator=b.g, device="cuda")
    q, o, lse = prompt(csa, ctx, b, new, pad=2, sink=sink, window=window)
    check_prompt(b, new, q, o, lse, sink, window)
    assert ctx.status() == 0


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_lse_of_one_score_and_a_little(csa, ctx, hd):
    """Two scores, 0 and -x: lse = log(1 + e^-x).  With w = e^-x the sum 1 + w is off by half a step of 1 (2^-24), by w 2^-22 (the power)
    and by w x 2^-22 (the score in base 2, two roundings), and lse again by a step of the logarithm's and two roundings, 2^-22 of it."""
    n, page = 120, 16
    gap = 1 + torch.arange(n, device="cuda").float() / 16  # (exact in bf16 up to 8 bits of it: what the rows hold is read back)
    k = torch.zeros(n + 1, page, 1, hd, dtype=torch.bfloat16, device="cuda")
    k[:n, 1, 0, 0] = -gap.to(torch.bfloat16)
    x = -k[:n, 1, 0, 0].double()
    q = torch.zeros(2 * n, 1, hd, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    w = torch.exp(-x)
    want = torch.log1p(w)
    tol = 2.0 ** -24 + w * (1 + x) * 2.0 ** -22 + want * 2.0 ** -22
    table = torch.arange(n, device="cuda", dtype=torch.int32)[:, None]
    cache = csa.PagedCache(k, torch.ones_like(k))
    _, lse = ctx.prompt_attn(q, cache, table, i32(list(range(0, 2 * n + 1, 2))), i32([2] * n), 1.0, with_lse=True)
    assert (lse[0::2, 0] == 0).all() and ((lse[1::2, 0].double() - want).abs() <= tol).all()
    _, lse = ctx.prefix_attn(q[:n], cache, table, i32([-1] * n), table, i32([2] * n), 1.0, cu=i32(list(range(n + 1))), with_lse=True)
    assert ((lse[:, 0].double() - want).abs() <= tol).all()
    o, lse = ctx.prefix_attn(q[:n], cache, table, i32([1] * n), i32([[n]]), i32([1]), 1.0, with_lse=True)  # 0, and 0 and -x of its own
    assert (o == 1).all() and ((lse[:, 0].double() - torch.log1p(1 + w)).abs() <= tol + 2.0 ** -22).all() and ctx.status() == 0


@pytest.mark.parametrize("hd,thousand", [(64, 330), (128, 130), (192, 61), (256, 66)])
def test_prefix_rows_that_fit_the_workspace(csa, ctx, hd, thousand):
    """The most rows by the header's sum, and 64 rows more, which are refused before anything is written."""
    H, kv = 64, 8
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    room = (128 << 20) - (256 << 10) - (24 << 20) - sms * 2 * (256 if hd < 256 else 128) * (4 * hd + 16)
    N = (room - (64 << 10)) // (H * (4 * hd + 8))  # (and the plan, below 64 KiB)
    assert sms != 152 or abs(N * H / 1000 - thousand) < 2
    b = Batch([40, 70], H, kv, hd, 16, seed=hd)
    q = b.queries(N + 64)
    args = (csa.PagedCache(b.k, b.v), b.table)
    more = (b.table[1:2].contiguous(), i32([70]), b.scale)
    pos, req = torch.arange(N + 64, dtype=torch.int32, device="cuda") % 41 - 1, torch.zeros(N + 64, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 3.0)
    with pytest.raises(csa.CsaError, match="workspace") as e:
        ctx.prefix_attn(q, *args, pos, *more, req=req, out=out)
    torch.cuda.synchronize()
    assert e.value.code == -2 and (out == 3).all()
    o, lse = ctx.prefix_attn(q[:N], *args, pos[:N], *more, req=req[:N], with_lse=True)
    for n in (0, 1, 40, N // 2, N - 41, N - 1):
        p = int(pos[n])
        K, V = (torch.cat([rows[1], rows[0][:p + 1]]) for rows in (b.rows_k, b.rows_v))
        last = torch.tensor([70 + p], device="cuda")
        close(o[n:n + 1], lse[n:n + 1], ref(q[n:n + 1], K, V, kv, b.scale, None, last * 0, last), "row %d" % n)
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd,page,window", [(8, 2, 128, 16, 0), (4, 4, 64, 8, 200), (9, 1, 128, 16, 330), (16, 2, 256, 32, 0),
                                                 (6, 2, 192, 16, 90)])
def test_prefix_and_own_rows_in_one_table(csa, ctx, H, kv, hd, page, window):
    """Prefix and own pages one behind the other in a table are rows of paged_attn: the same results, whichever way they are split.
    Both are within the tolerance of prefix_attn's one bf16 term of the 64-bit form, so they are within twice that of each other."""
    own, plen = [1, 0, 2, 15, 16, 17, 100, 300], 20 * page
    P = Prefixes(own, [plen], H, kv, hd, page, seed=hd + page)
    n, pos = len(own), [x - 1 for x in own]
    q, sink = P.b.queries(n), torch.randn(H, generator=P.b.g, device="cuda")
    cache = csa.PagedCache(P.k, P.v)
    o, lse = ctx.prefix_attn(q, cache, P.table, i32(pos), P.prefix, i32([plen]), P.scale, sink=sink, window=window, with_lse=True)
    joined = torch.cat([P.prefix[:, :20].expand(n, -1), P.table], 1).contiguous()
    o2, lse2 = ctx.paged_attn(q, cache, joined, i32([plen + x for x in pos]), P.scale, sink=sink, window=window, with_lse=True)
    for i in range(n):
        K, V = (torch.cat([rows[n], rows[i][:pos[i] + 1]]) for rows in (P.b.rows_k, P.b.rows_v))
        last = torch.tensor([plen + pos[i]], device="cuda")
        first = (last + 1 - window).clamp(min=0) if window else last * 0
        want, e, tol, tol_l = ref(q[i:i + 1], K, V, kv, P.scale, sink, first, last)
        close(o[i:i + 1], lse[i:i + 1], (want, e, tol, tol_l), "prefix_attn, row %d" % i)
        close(o2[i:i + 1], lse2[i:i + 1], (want, e, tol, tol_l), "paged_attn, row %d" % i)
        assert ((o[i:i + 1].double() - o2[i:i + 1].double()).abs() <= 2 * tol).all()
        assert ((lse[i:i + 1].double() - lse2[i:i + 1].double()).abs() <= 2 * tol_l).all()
    assert ctx.status() == 0


@pytest.mark.parametrize("hd", [64, 128, 192, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("window", [0, 60, 400])
def test_prefix_bad_value_among_own_rows(csa, ctx, hd, bad, window):
    """It reaches its request's rows that attend it, in its feature of its kv head's heads; all else keeps its bits."""
    H, kv, own, page = 8, 2, [300, 40, 0, 90, 5, 7], 16
    g = H // kv
    P = Prefixes(own, [500, 300], H, kv, hd, page, seed=2)
    req = [0, 1, 2, 3, 3, 3, 4, 5]
    pos = [299, 39, -1, 89, 35, 36, 4, 6]
    q = P.b.queries(len(req))

    def run():
        return ctx.prefix_attn(q, csa.PagedCache(P.k, P.v), P.table, i32(pos), P.prefix, i32([500, 300]), P.scale, cu=i32([0, 5, 8]),
                               req=i32(req), window=window, with_lse=True)

    want, want_lse = run()
    assert want.isfinite().all()
    at = 36
    P.v[int(P.table[3, at // page]), at % page][1, 3] = bad
    hit = torch.tensor([r == 3 and p >= at and (not window or p < at + window) for r, p in zip(req, pos)], device="cuda")
    assert hit.tolist() == [False] * 3 + [True, False, True] + [False] * 2
    o, lse = run()
    assert torch.equal(lse, want_lse) and torch.equal(o[~hit], want[~hit]) and torch.equal(o[:, :g], want[:, :g])
    rest = [d for d in range(hd) if d != 3]
    assert torch.equal(o[..., rest], want[..., rest]) and not o[hit][:, g:, 3].isfinite().any()
    assert ctx.status() == 0
