"""The paged-cache operators on the GPU, against plain 64-bit forms: csa_page_step (token maps and block
tables), csa_qk_norm_rope (head norms, rotation, cache write), csa_paged_attn (single tokens over the pages),
and a run of the three together in a captured graph.

Tolerances, from the roundings alone.  A bf16 result is off by at most half a step, 2^-8 |want|.  Norm and
rotation: at most about 50 f32 roundings in a row (the sum of squares of a lane's vectors and five
shuffles, the root, the division, two products, the turn), each 2^-24 of the two values of a pair: 2^-17 of
the row's largest value covers them.  Attention: an error d of a score changes a weight by the factor
e^(+-d), so the result moves by at most 2 d A with A_d = sum_j w_j |V_jd|; d is at most (hd + 8) 2^-24
sum_d |q_d K_jd| scale (one rounding a product and a sum) plus 2^-21 (the exponential) and the row sum adds rows
2^-24.  A weight below f32's smallest normal number may be 0, which moves the result by at most 2^-126 sum_j |V_jd|.
Where the weights are rounded for the matrix product the result moves by that rounding times A: 2^-16
for two bf16 terms, 2^-8 for one (head_dim above 256).
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def csa():
    import compressed_sparse_attention_attn_gb300 as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def ctx(csa):
    return make_ctx(csa)


def make_ctx(csa):
    from csa_inputs import Geometry
    return csa.Context(Geometry(dim=64, max_tokens=1, max_batch=1, max_seq=16).as_dict())


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------ page_step

class Pool:
    """The allocator as lists."""

    def __init__(self, n_pages, page, lens, seed):
        rng = np.random.default_rng(seed)
        ids = rng.permutation(n_pages).tolist()
        self.page, self.n_pages = page, n_pages
        self.lens = list(lens)
        self.pages = [[ids.pop() for _ in range(-(-x // page))] for x in lens]
        self.free = ids

    def step(self, new):
        took, back, toks = 0, 0, []
        pool = list(self.free)
        released = []
        for r, a in enumerate(new):
            if a < 0:
                released += self.pages[r]
                back += len(self.pages[r])
                self.pages[r], self.lens[r] = [], 0
                continue
            for i in range(a):
                p = self.lens[r] + i
                if p // self.page >= len(self.pages[r]):
                    self.pages[r].append(pool.pop(0))
                    took += 1
                toks.append((r, p, self.pages[r][p // self.page] * self.page + p % self.page))
            self.lens[r] += max(a, 0)
        self.free = pool + released
        return toks, took, back

    def table(self, width):
        t = np.full((len(self.lens), width), -7, np.int32)
        for r, p in enumerate(self.pages):
            t[r, :len(p)] = p
        return t

    def ring(self, head):
        f = np.full(self.n_pages, -9, np.int32)
        for i, p in enumerate(self.free):
            f[(head + i) % self.n_pages] = p
        return f


def check_step(csa, lens, new_steps, page, n_pages, width, N, head, seed=0, in_place=True):
    pool = Pool(n_pages, page, lens, seed)
    R = len(lens)
    table, free, state = i32(pool.table(width)), i32(pool.ring(head)), i32([head, len(pool.free)])
    length = i32(lens)
    maps = [torch.full((N,), -5, dtype=torch.int32, device="cuda") for _ in range(3)]
    cu = torch.full((R + 1,), -5, dtype=torch.int32, device="cuda")
    for new in new_steps:
        old = table.cpu().numpy()
        toks, took, back = pool.step(new)
        outs = {} if in_place else dict(length_out=torch.empty_like(length), state_out=torch.empty_like(state))
        info = csa.page_step(i32(new), length, table, free, state, page, *maps, cu, **outs)
        if not in_place:
            length, state = outs["length_out"], outs["state_out"]
        head = (head + took) % n_pages
        assert info.tolist() == [len(toks), took, back, 0]
        want = np.full((3, N), -1, np.int64)
        if toks:
            want[:, :len(toks)] = np.array(toks).T
        for k in range(3):
            assert np.array_equal(maps[k].cpu().numpy(), want[k])
        assert length.tolist() == pool.lens and state.tolist() == [head, len(pool.free)]
        assert cu.tolist() == np.concatenate([[0], np.cumsum(np.maximum(new, 0))]).tolist()
        got, now = table.cpu().numpy(), pool.table(width)
        for r in range(R):  # (an ended request's entries stay as they were)
            assert np.array_equal(got[r][:len(pool.pages[r])], now[r][:len(pool.pages[r])])
            if new[r] >= 0:
                assert np.array_equal(got[r][len(pool.pages[r]):], old[r][len(pool.pages[r]):])
        ring = free.cpu().numpy()
        assert [ring[(head + i) % n_pages] for i in range(len(pool.free))] == pool.free


@pytest.mark.parametrize("page", [1, 16, 17, 128])
@pytest.mark.parametrize("in_place", [True, False])
def test_page_step_small(csa, page, in_place):
    """Empty, one-token and page-border requests; ends, waits, a step of nothing; pages released in one step serve
    the next; the ring wraps."""
    lens = [0, 1, page - 1, page, page + 1, 3 * page, 0, 5]
    steps = [[1] * 8, [0, 3, 1, 1, page, -1, 0, 2 * page + 1], [0] * 8, [-1, -1, 0, 1, 0, 1, -1, 1], [1] * 8, [-1] * 8, [2] * 8]
    need = sum(-(-(x + 5 + 3 * page) // page) for x in lens)
    check_step(csa, lens, steps, page, need, 3 * page + 12, 6 * page + 12, need - 2, in_place=in_place)


@pytest.mark.parametrize("R,N,page", [(1, 1, 16), (1, 5000, 16), (300, 300, 16), (1025, 4500, 32), (5000, 9000, 7), (14000, 20000, 64)])
def test_page_step_sizes(csa, R, N, page):
    rng = np.random.default_rng(R)
    lens = rng.integers(0, 6 * page, R).tolist()
    steps = []
    for _ in range(2):
        new = rng.integers(-1, 2, R)
        new[rng.integers(0, R)] = max(0, N - int(np.maximum(new, 0).sum()) - R) // 2 + 1
        steps.append(new.tolist())
    n_pages = sum(-(-x // page) for x in lens) + 2 * (N + R)
    check_step(csa, lens, steps, page, n_pages, (6 * page + 2 * N) // page + 3, N, n_pages // 2, seed=R)


@pytest.mark.parametrize("case,bit", [("tokens", 1), ("one request's tokens", 1), ("negative length", 2), ("width", 2),
                                      ("held past width", 2), ("pool", 4), ("state", 8), ("count", 8), ("overfull", 8)])
def test_page_step_errors_change_nothing(csa, case, bit):
    page, n_pages, width, N = 4, 10, 3, 8
    length, new = [3, 4, 0], [1, 1, 2]
    state, ring = [2, 6], list(range(10))
    if case == "tokens":
        new = [1, 4, 4]
    elif case == "one request's tokens":
        new = [1, 2 ** 31 - 1, 0]
    elif case == "negative length":
        length = [3, -1, 0]
    elif case == "width":
        length = [3, 12, 0]
    elif case == "held past width":
        length, new = [3, 13, 0], [1, 0, 0]
    elif case == "pool":
        state = [2, 1]
    elif case == "state":
        state = [10, 4]
    elif case == "count":
        state = [0, 11]
    elif case == "overfull":
        state, new = [0, 10], [-1, 0, 0]
    t = i32(np.arange(9).reshape(3, 3))
    L, S, F = i32(length), i32(state), i32(ring)
    maps = [torch.full((N,), 5, dtype=torch.int32, device="cuda") for _ in range(3)]
    cu = i32([9, 9, 9, 9])
    info = csa.page_step(i32(new), L, t, F, S, page, *maps, cu)
    assert info.tolist() == [0, 0, 0, bit]
    assert L.tolist() == length and S.tolist() == state and F.tolist() == ring
    assert t.tolist() == np.arange(9).reshape(3, 3).tolist() and cu.tolist() == [0] * 4
    assert all((m == -1).all() for m in maps)


def test_page_step_bad_entries_give_no_slot(csa):
    """A table entry or a free page outside the pool: its tokens get slot -1, the others theirs."""
    t, F = i32([[99, 0], [3, 0], [0, 0]]), i32([-4, 5, 6, 7, 0, 0, 0, 0])
    L, S = i32([2, 2, 0]), i32([0, 4])
    maps = [torch.empty(4, dtype=torch.int32, device="cuda") for _ in range(3)]
    info = csa.page_step(i32([1, 1, 2]), L, t, F, S, 4, *maps)
    assert info.tolist() == [4, 1, 0, 0]
    assert maps[0].tolist() == [0, 1, 2, 2] and maps[1].tolist() == [2, 2, 0, 1] and maps[2].tolist() == [-1, 14, -1, -1]


# ------------------------------------------------------------------------------------------ qk_norm_rope

def rope_tab(rows, rd, base=10000.0):
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * base ** (
        -torch.arange(0, rd, 2, device="cuda", dtype=torch.float64) / max(rd, 1))
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def ref_rows(x, w, eps, tab, pos, rd, at, half):
    y = x.double()
    if w is not None:
        y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + eps) * w.double()
    if rd:
        i = torch.arange(rd // 2, device="cuda")
        lo, hi = (at + i, at + i + rd // 2) if half else (at + 2 * i, at + 2 * i + 1)
        cs = tab.double()[pos.long().clamp(min=0)][:, None]
        a, b = y[..., lo].clone(), y[..., hi].clone()
        y[..., lo] = a * cs[..., 0] - b * cs[..., 1]
        y[..., hi] = a * cs[..., 1] + b * cs[..., 0]
    return y


def close_rows(got, want, what):
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -17 * want.abs().amax(-1, keepdim=True)
    d = (got.double() - want).abs()
    assert (d <= tol).all(), "%s: off by %g where %g is allowed" % (what, (d - tol).max().item(), tol.flatten()[(d - tol).argmax()].item())


NORM = [  # N, H, kv, hd, rd, at, half, norm, v, slots, page, order
    (1, 1, 1, 64, 64, 0, False, True, True, True, 16, "nhd"),
    (5, 4, 2, 128, 128, 0, True, True, True, True, 16, "hnd"),
    (33, 8, 1, 512, 64, 448, False, True, False, True, 64, "nhd"),
    (7, 3, 3, 80, 32, 48, True, True, True, True, 1, "hnd"),
    (9, 5, 1, 96, 20, 2, True, True, True, True, 17, "nhd"),
    (9, 5, 1, 96, 22, 10, False, False, True, False, 4, "nhd"),
    (3, 2, 1, 8, 8, 0, False, True, True, True, 3, "nhd"),
    (3, 2, 2, 24, 2, 22, True, True, True, True, 3, "hnd"),
    (6, 2, 1, 1024, 512, 256, True, True, False, True, 8, "nhd"),
    (6, 2, 1, 576, 64, 512, False, True, True, True, 8, "nhd"),
    (4, 2, 1, 256, 0, 0, False, True, True, True, 8, "nhd"),
    (4, 2, 2, 192, 192, 0, True, False, True, False, 8, "hnd"),
    (300, 24, 8, 128, 64, 0, True, True, True, True, 16, "nhd"),
]


@pytest.mark.parametrize("N,H,kv,hd,rd,at,half,norm,has_v,slots,page,order", NORM)
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_rope(csa, ctx, N, H, kv, hd, rd, at, half, norm, has_v, slots, page, order, in_place):
    g = gen(N * hd + rd)
    x = randn(g, N, (H + 2 * kv) * hd + 8, scale=3.0)  # a fused projection's rows, with something behind them
    x[0, :hd] = 0  # a head of zeros
    q = x[:, :H * hd].view(N, H, hd)
    k = x[:, H * hd:(H + kv) * hd].view(N, kv, hd)
    v = x[:, (H + kv) * hd:(H + 2 * kv) * hd].view(N, kv, hd) if has_v else None
    n_pages = -(-N // page) + 2
    pages = lambda: randn(g, n_pages, page, kv, hd) if order == "nhd" else randn(g, n_pages, kv, page, hd).transpose(1, 2)  # noqa: E731
    kp, vp = pages(), pages() if has_v else None
    slot = torch.randperm(n_pages * page, generator=g, device="cuda")[:N].to(torch.int32) if slots else None
    pos = torch.randint(0, 900, (N,), generator=g, device="cuda").to(torch.int32)
    tab = rope_tab(900, rd) if rd else None
    if N > 2:
        pos[N // 2] = -1  # padding
        if slots:
            slot[0] = -1  # a query alone
    w = lambda: 1 + 0.2 * torch.randn(hd, generator=g, device="cuda") if norm else None  # noqa: E731
    qw, kw = w(), w()
    live = pos >= 0
    x0, kp0, vp0 = x.clone(), kp.clone(), None if vp is None else vp.clone()
    wq = ref_rows(q, qw, 1e-6, tab, pos, rd, at, half)
    wk = ref_rows(k, kw, 1e-6, tab, pos, rd, at, half)
    out = q if in_place else torch.full((N, H, hd), 9.0, dtype=torch.bfloat16, device="cuda")
    got = ctx.qk_norm_rope(q, k, v, csa.PagedCache(kp, vp), pos, slot, tab=tab, rd=rd, rope_at=at, half=half,
                           q_norm=qw, k_norm=kw, eps=1e-6, q_out=out)
    assert got is out
    close_rows(out[live], wq[live], "q")
    old = x0[:, :H * hd].view(N, H, hd) if in_place else torch.full_like(out, 9.0)
    assert torch.equal(out[~live], old[~live])
    kept = live & (slot >= 0) if slots else live
    at_row = (slot if slots else torch.arange(N, device="cuda")).long()
    close_rows(kp[at_row[kept] // page, at_row[kept] % page], wk[kept], "k")
    other = torch.ones(n_pages * page, dtype=torch.bool, device="cuda")
    other[at_row[kept]] = False
    r = torch.arange(n_pages * page, device="cuda")[other]
    assert torch.equal(kp[r // page, r % page], kp0[r // page, r % page])
    if has_v:
        vv = x0[:, (H + kv) * hd:(H + 2 * kv) * hd].view(N, kv, hd)
        assert torch.equal(vp[at_row[kept] // page, at_row[kept] % page], vv[kept])
        assert torch.equal(vp[r // page, r % page], vp0[r // page, r % page])
    assert torch.equal(x[:, (H if in_place else 0) * hd:], x0[:, (H if in_place else 0) * hd:])
    assert ctx.status() == 0


def test_norm_rope_keys_only_and_large_values(csa, ctx):
    """Without queries; values whose squares are far from 1 (1e15, 1e-15) norm as the formula says."""
    g = gen(4)
    k = torch.randn(6, 2, 64, generator=g, device="cuda")
    k[1] *= 1e15
    k[2] *= 1e-15
    k = k.to(torch.bfloat16)
    cache = csa.PagedCache(torch.zeros(6, 1, 2, 64, dtype=torch.bfloat16, device="cuda"))
    pos, w = i32([0, 1, 2, 3, 4, 5]), torch.ones(64, device="cuda")
    tab = rope_tab(6, 64)
    assert ctx.qk_norm_rope(None, k, None, cache, pos, tab=tab, rd=64, k_norm=w, eps=1e-6) is None
    close_rows(cache.k[:, 0], ref_rows(k, w, 1e-6, tab, pos, 64, 0, False), "k")


def test_norm_rope_bad_positions_and_slots(csa, ctx):
    """A position past the table or a slot outside the pool skips its token and sets the status word."""
    g = gen(5)
    assert ctx.status() == 0
    for pos, slot in (([0, 8, 2], [0, 1, 2]), ([0, 1, 2], [0, 12, 2]), ([0, 1, 2], [0, -2, 2])):
        q, k = randn(g, 3, 2, 64), randn(g, 3, 1, 64)
        kp = torch.full((3, 4, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        out = torch.full_like(q, 7.0)
        ctx.qk_norm_rope(q, k, None, csa.PagedCache(kp), i32(pos), i32(slot), tab=rope_tab(8, 64), rd=64, q_out=out)
        assert (out[1] == 7).all() and not (out[0] == 7).any() and (kp.view(12, 64)[1] == 5).all()
        assert ctx.status() == csa._abi.CSA_OK - 1 and ctx.status() == 0


# ------------------------------------------------------------------------------------------ paged_attn

class Batch:
    """Requests of the given lengths over shuffled pages; rows behind a request's last and pages of nobody hold NaN."""

    def __init__(self, lens, H, kv, hd, page, latent=False, order="nhd", seed=0, scale_q=1.5):
        g = gen(seed)
        self.lens, self.H, self.kv, self.hd, self.page = lens, H, kv, hd, page
        per = [-(-x // page) for x in lens]
        self.n_pages = sum(per) + 3
        perm = torch.randperm(self.n_pages, generator=g, device="cuda").tolist()
        width = max(per + [1]) + 1
        table = np.full((len(lens), width), -3, np.int32)

        def pages():
            t = torch.full((self.n_pages, page, kv, hd) if order == "nhd" else (self.n_pages, kv, page, hd), float("nan"),
                           dtype=torch.bfloat16, device="cuda")
            return t if order == "nhd" else t.transpose(1, 2)

        self.k, self.v = pages(), None if latent else pages()
        self.rows_k, self.rows_v = [], []
        at = 0
        for r, x in enumerate(lens):
            ids = perm[at:at + per[r]]
            at += per[r]
            table[r, :per[r]] = ids
            K = randn(g, x, kv, hd)
            V = K if latent else randn(g, x, kv, hd)
            self.rows_k.append(K)
            self.rows_v.append(V)
            if x:
                p = torch.arange(x, device="cuda")
                idt = torch.tensor(ids, device="cuda")[p // page]
                self.k[idt, p % page] = K
                if not latent:
                    self.v[idt, p % page] = V
        self.table = i32(table)
        self.g = g
        self.scale = hd ** -0.5

    def queries(self, n, scale=1.5):
        return randn(self.g, n, self.H, self.hd, scale=scale)


def ref_attn(q, K, V, kv, scale, sink):
    """(O, lse, A, d) of one row's heads over rows K, V [x][kv][hd] in 64 bits: A, d as the tolerances use them."""
    H, hd = q.shape
    g = H // kv
    if K.shape[0] == 0:
        z = torch.zeros(H, hd, dtype=torch.float64, device="cuda")
        return z, torch.full((H,), float("-inf"), dtype=torch.float64, device="cuda"), z, torch.zeros(H, 1, dtype=torch.float64, device="cuda")
    qd = q.double().view(kv, g, hd)
    Kd, Vd = K.double().permute(1, 0, 2), V.double().permute(1, 0, 2)
    S = qd @ Kd.transpose(1, 2) * scale
    lse = torch.logsumexp(S, -1)
    den = lse if sink is None else torch.logaddexp(lse, sink.double().view(kv, g))
    w = torch.exp(S - den[..., None])
    d = (hd + 8) * 2.0 ** -24 * (qd.abs() @ Kd.abs().transpose(1, 2)).amax(-1) * abs(scale) + 2.0 ** -21 + K.shape[0] * 2.0 ** -24
    A = w @ Vd.abs()
    least = 2.0 ** -126 * Vd.abs().sum(1, keepdim=True).expand_as(A)  # (2 d + ...) A + least, kept in A's place: d >= 2^-21
    return (w @ Vd).reshape(H, hd), lse.reshape(H), (A + least * 2.0 ** 21).reshape(H, hd), d.reshape(H, 1)


def check_rows(b, q, o, lse, pos, req=None, sink=None, window=0, scale=None):
    for n in range(len(pos)):
        r = n if req is None else req[n]
        lo = max(0, pos[n] + 1 - window) if window else 0
        K, V = b.rows_k[r][lo:pos[n] + 1], b.rows_v[r][lo:pos[n] + 1]
        want, wl, A, d = ref_attn(q[n], K, V, b.kv, b.scale if scale is None else scale, sink)
        w_round = 2.0 ** -8 if b.hd > 256 else 2.0 ** -16
        tol = 2.0 ** -8 * want.abs() + (2 * d + w_round) * A
        err = (o[n].double() - want).abs()
        assert not err.isnan().any() and (err <= tol).all(), "row %d (%d rows): off by %g where %g is allowed" % (
            n, K.shape[0], err.max().item(), tol.flatten()[(err - tol).argmax()].item())
        if lse is not None:
            if K.shape[0] == 0:
                assert (lse[n] == float("-inf")).all()
            else:
                assert ((lse[n].double() - wl).abs() <= d[:, 0] + 2.0 ** -22 * (1 + wl.abs())).all(), "lse of row %d" % n


LENS = [1, 0, 2, 15, 16, 17, 63, 64, 65, 100, 129, 500]
ATTN = [  # H, kv, hd, page, latent, order, window, sink
    (4, 4, 64, 16, False, "nhd", 0, False),
    (8, 2, 64, 16, False, "hnd", 0, True),
    (32, 8, 128, 16, False, "nhd", 0, False),
    (7, 1, 128, 17, False, "nhd", 100, True),
    (16, 1, 128, 1, False, "hnd", 0, False),
    (20, 1, 128, 64, False, "nhd", 0, True),
    (40, 2, 64, 32, False, "nhd", 70, False),
    (3, 3, 80, 16, False, "nhd", 0, False),
    (10, 2, 96, 8, False, "hnd", 0, True),
    (6, 3, 192, 128, False, "nhd", 0, False),
    (16, 16, 256, 17, False, "hnd", 64, True),
    (8, 1, 256, 16, True, "nhd", 0, False),
    (5, 1, 8, 16, False, "nhd", 0, False),
    (64, 1, 512, 64, True, "nhd", 0, True),
    (16, 1, 512, 16, True, "nhd", 0, False),
    (128, 1, 512, 64, True, "nhd", 130, True),
    (40, 2, 512, 17, True, "hnd", 0, True),
    (3, 3, 320, 1, True, "nhd", 0, False),
    (70, 1, 264, 32, True, "nhd", 0, True),
]


@pytest.mark.parametrize("H,kv,hd,page,latent,order,window,sink", ATTN)
def test_paged_attn(csa, ctx, H, kv, hd, page, latent, order, window, sink):
    b = Batch(LENS, H, kv, hd, page, latent, order, seed=H * hd)
    pos = [x - 1 for x in LENS]
    q = b.queries(len(LENS))
    sw = torch.randn(H, generator=b.g, device="cuda") if sink else None
    o, lse = ctx.paged_attn(q, csa.PagedCache(b.k, b.v), b.table, i32(pos), b.scale, sink=sw, window=window, with_lse=True)
    check_rows(b, q, o, lse, pos, None, sw, window)
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd,latent", [(8, 2, 128, False), (16, 16, 64, False), (64, 1, 512, True), (12, 1, 256, False)])
@pytest.mark.parametrize("lens", [[1], [40], [3000], [20000], [5000, 1, 0, 1, 9000], [1] * 700, list(range(300))])
def test_paged_attn_lengths(csa, ctx, H, kv, hd, latent, lens):
    """One row alone, long rows split over the device beside short ones, many short rows."""
    b = Batch(lens, H, kv, hd, 16, latent, seed=len(lens) + hd)
    pos = [x - 1 for x in lens]
    q = b.queries(len(lens))
    cache = csa.PagedCache(b.k, b.v)
    o, lse = ctx.paged_attn(q, cache, b.table, i32(pos), b.scale, with_lse=True)
    check_rows(b, q, o, lse, pos)
    # the same bits again, whatever finished first
    for _ in range(3):
        o2, lse2 = ctx.paged_attn(q, cache, b.table, i32(pos), b.scale, with_lse=True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd,latent", [(8, 2, 128, False), (64, 1, 512, True)])
def test_paged_attn_rows_of_requests(csa, ctx, H, kv, hd, latent):
    """Several rows of one request at different positions, padding rows and an empty row; a strided q and out."""
    b = Batch([70, 300, 9], H, kv, hd, 16, latent, seed=3)
    req = [1, 1, 1, -1, 0, 2, 0, 2, 1]
    pos = [0, 299, 150, 5, 69, 8, -1, -2, 298]
    N = len(req)
    wide = randn(b.g, N, H * hd + 64, scale=1.5)
    q = wide[:, 8:8 + H * hd].view(N, H, hd)
    buf = torch.full((N, H * hd + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :H * hd].view(N, H, hd)
    lse = torch.full((N, H), 3.0, device="cuda")
    sink = torch.randn(H, generator=b.g, device="cuda")
    ctx.paged_attn(q, csa.PagedCache(b.k, b.v), b.table, i32(pos), b.scale, req=i32(req), sink=sink, out=out, lse=lse)
    live = [n for n in range(N) if req[n] >= 0 and pos[n] >= -1]
    check_rows(b, q[live], out[live], lse[live], [pos[n] for n in live], [req[n] for n in live], sink)
    for n in set(range(N)) - set(live):
        assert (out[n] == 3).all() and (lse[n] == 3).all()
    assert (buf[:, H * hd:] == 3).all() and ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd,latent", [(8, 2, 128, False), (64, 1, 512, True)])
def test_paged_attn_extreme_scores(csa, ctx, H, kv, hd, latent):
    """Scores of +-thousands, all of them far below zero, sinks far above and below; an infinite sink takes everything."""
    b = Batch([200, 64, 1], H, kv, hd, 16, latent, seed=8)
    pos = [199, 63, 0]
    q = b.queries(3)
    cache = csa.PagedCache(b.k, b.v)
    for scale in (40.0, -40.0, 0.0, 1e-3):
        for sink in (None, torch.full((H,), -1e4, device="cuda"), torch.full((H,), 50.0, device="cuda")):
            o, lse = ctx.paged_attn(q, cache, b.table, i32(pos), scale, sink=sink, with_lse=True)
            check_rows(b, q, o, lse, pos, None, sink, scale=scale)
    o = ctx.paged_attn(q, cache, b.table, i32(pos), b.scale, sink=torch.full((H,), float("inf"), device="cuda"))
    assert (o == 0).all()
    o = ctx.paged_attn(q, cache, b.table, i32(pos), b.scale, sink=torch.full((H,), float("-inf"), device="cuda"))
    check_rows(b, q, o, None, pos)


@pytest.mark.parametrize("H,kv,hd,latent", [(8, 2, 128, False), (64, 1, 512, True)])
def test_paged_attn_bad_pages_and_requests(csa, ctx, H, kv, hd, latent):
    """A page id outside the pool leaves its rows out, a request outside the table its row as it was, a position
    past the table the rows past it; each sets the status word."""
    page = 16
    b = Batch([48, 48, 48], H, kv, hd, page, latent, seed=9)
    q = b.queries(3)
    cache = csa.PagedCache(b.k, b.v)
    for bad in (-1, b.n_pages, 2 ** 31 - 1):
        t = b.table.clone()
        t[1, 1] = bad
        o, lse = ctx.paged_attn(q, cache, t, i32([47, 47, 47]), b.scale, with_lse=True)
        keep = torch.cat([torch.arange(16), torch.arange(32, 48)]).cuda()
        full_k, full_v = b.rows_k[1], b.rows_v[1]
        b.rows_k[1], b.rows_v[1] = full_k[keep], full_v[keep]
        check_rows(b, q, o, lse, [47, 31, 47])
        b.rows_k[1], b.rows_v[1] = full_k, full_v
        assert ctx.status() == -1 and ctx.status() == 0
    out = torch.full_like(q, 3.0)
    ctx.paged_attn(q, cache, b.table, i32([47, 47, 47]), b.scale, req=i32([0, 3, 2]), out=out)
    assert (out[1] == 3).all() and ctx.status() == -1
    check_rows(b, q[[0, 2]], out[[0, 2]], None, [47, 47], [0, 2])
    t = b.table[:, :3].contiguous()
    o = ctx.paged_attn(q, cache, t, i32([47, 60, 2 ** 31 - 1]), b.scale)
    assert ctx.status() == -1 and ctx.status() == 0
    check_rows(b, q, o, None, [47, 47, 47])


def test_paged_attn_far_pages(csa, ctx):
    """A pool above 2^31 elements: page offsets need 64 bits."""
    page, kv, hd, H = 64, 8, 128, 32
    n_pages = 2 ** 31 // (page * kv * hd) + 40
    k = torch.zeros(n_pages, page, kv, hd, dtype=torch.bfloat16, device="cuda")
    b = Batch([200], H, kv, hd, page, seed=10)
    ids = torch.tensor([n_pages - 1, 3, n_pages - 20, n_pages - 2], device="cuda")
    v = torch.zeros_like(k)
    src = b.table[0, :4].long()
    k[ids], v[ids] = b.k[src], b.v[src]
    q = b.queries(1)
    o, lse = ctx.paged_attn(q, csa.PagedCache(k, v), ids.to(torch.int32)[None].contiguous(), i32([199]), b.scale, with_lse=True)
    check_rows(b, q, o, lse, [199])
    # and writing there
    x = randn(b.g, 2, kv, hd)
    slot = i32([(n_pages - 3) * page + 5, 7])
    ctx.qk_norm_rope(None, x, x, csa.PagedCache(k, v), i32([0, 0]), slot)
    assert torch.equal(k[n_pages - 3, 5], x[0]) and torch.equal(v[0, 7], x[1]) and ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd,latent", [(8, 2, 128, False), (64, 1, 512, True)])
def test_paged_attn_streams_and_contexts(csa, ctx, H, kv, hd, latent):
    """Two contexts at once on two streams, and calls on a stream that is not the current one."""
    b = Batch([4000, 900, 2500], H, kv, hd, 16, latent, seed=11)
    pos = [3999, 899, 2499]
    q = b.queries(3)
    cache, p = csa.PagedCache(b.k, b.v), i32(pos)
    want = ctx.paged_attn(q, cache, b.table, p, b.scale)
    other = make_ctx(csa)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got.append(ctx.paged_attn(q, cache, b.table, p, b.scale, stream=s1))
        got.append(other.paged_attn(q, cache, b.table, p, b.scale, stream=s2))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
    other.close()


@pytest.mark.parametrize("H,kv,hd,page,order,window,pad", [
    (16, 2, 512, 24, "nhd", 0, 0), (32, 2, 512, 8, "hnd", 50, 0), (8, 4, 384, 48, "hnd", 100, 8), (64, 1, 512, 128, "nhd", 300, 0),
    (64, 1, 512, 4, "nhd", 0, 0), (9, 3, 288, 12, "nhd", 33, 8), (200, 1, 512, 40, "hnd", 0, 24), (65, 1, 448, 96, "nhd", 1, 64)])
def test_paged_attn_latent_pages(csa, ctx, H, kv, hd, page, order, window, pad):
    """Latent rows in pages of many sizes, several kv heads, windows that begin inside a tile, rows that lie apart."""
    lens = [1, 0, 47, 48, 49, 95, 96, 97, 300, 1000]
    b = Batch(lens, H, kv, hd, page, True, order, seed=hd + page)
    if pad:  # a cache with room between its rows
        wide = torch.full(b.k.shape[:3] + (hd + pad,), float("nan"), dtype=torch.bfloat16, device="cuda")
        k = wide[..., 8:8 + hd] if pad > 8 else wide[..., :hd]
        k.copy_(b.k)
    else:
        k = b.k
    pos = [x - 1 for x in lens]
    q = b.queries(len(lens))
    sink = torch.randn(H, generator=b.g, device="cuda")
    o, lse = ctx.paged_attn(q, csa.PagedCache(k), b.table, i32(pos), b.scale, sink=sink, window=window, with_lse=True)
    check_rows(b, q, o, lse, pos, None, sink, window)
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd,latent", [(8, 2, 128, False), (4, 4, 256, False), (32, 2, 256, False), (6, 3, 64, False),
                                            (64, 1, 512, True), (66, 1, 264, True)])
@pytest.mark.parametrize("seed", range(4))
def test_paged_attn_uneven_rows(csa, ctx, H, kv, hd, latent, seed):
    """Few long rows among many short, empty and padding ones, in any order."""
    rng = np.random.default_rng(100 * hd + seed)
    lens = [int(rng.choice([0, 1, 3, 16, 33, 97, 200])) for _ in range(int(rng.integers(3, 60)))]
    for _ in range(int(rng.integers(1, 4))):
        lens.insert(int(rng.integers(0, len(lens) + 1)), int(rng.integers(500, 9000)))
    b = Batch(lens, H, kv, hd, int(rng.choice([5, 16, 64])), latent, seed=seed)
    N = len(lens)
    pos = [x - 1 if rng.random() > 0.2 else -2 for x in lens]
    q = b.queries(N)
    out = torch.full((N, H, hd), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, H), 3.0, device="cuda")
    ctx.paged_attn(q, csa.PagedCache(b.k, b.v), b.table, i32(pos), b.scale, out=out, lse=lse)
    live = [n for n in range(N) if pos[n] >= -1]
    check_rows(b, q[live], out[live], lse[live], [pos[n] for n in live], live)
    for n in set(range(N)) - set(live):
        assert (out[n] == 3).all() and (lse[n] == 3).all()
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd,latent", [(640, 1, 512, True), (130, 1, 512, True), (64, 1, 512, True), (256, 1, 128, False),
                                            (96, 32, 64, False)])
@pytest.mark.parametrize("N", [20, 32, 33])
def test_paged_attn_few_live_rows(csa, ctx, H, kv, hd, latent, N):
    """Mostly padding: few rows over many head groups, one row past the others' length by far."""
    lens = [0] * N
    lens[2], lens[N // 2], lens[N - 1] = 2500, 1, 300
    b = Batch(lens, H, kv, hd, 16, latent, seed=N)
    pos = [x - 1 if x else -5 for x in lens]
    q = b.queries(N)
    out = torch.full((N, H, hd), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, H), 3.0, device="cuda")
    ctx.paged_attn(q, csa.PagedCache(b.k, b.v), b.table, i32(pos), b.scale, out=out, lse=lse)
    live = [n for n in range(N) if lens[n]]
    check_rows(b, q[live], out[live], lse[live], [pos[n] for n in live], live)
    for n in set(range(N)) - set(live):
        assert (out[n] == 3).all() and (lse[n] == 3).all()
    # nothing but padding
    out.fill_(3.0)
    ctx.paged_attn(q, csa.PagedCache(b.k, b.v), b.table, i32([-2] * N), b.scale, out=out)
    assert (out == 3).all() and ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd,latent", [(8, 2, 128, False), (20, 1, 256, False), (64, 1, 512, True)])
def test_paged_attn_replayed_and_in_place(csa, ctx, H, kv, hd, latent):
    """Two captured graphs of one context replayed by turns while positions change, and the result over q itself."""
    lens = [3000, 1, 0, 700, 64]
    b = Batch(lens, H, kv, hd, 16, latent, seed=5)
    q = b.queries(len(lens))
    cache = csa.PagedCache(b.k, b.v)
    p1, p2 = i32([x - 1 for x in lens]), i32([-1, 0, -2, 5, 63])
    outs = [torch.zeros_like(q) for _ in range(2)]
    graphs = []
    for p, o in zip((p1, p2), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ctx.paged_attn(q, cache, b.table, p, b.scale, out=o)
        graphs.append(g)
    for step in range(4):
        if step == 2:
            p1.copy_(i32([1500, 0, -1, 699, 2]))
        want = []
        for p, o in zip((p1, p2), outs):
            o.zero_()
            want.append(ctx.paged_attn(q, cache, b.table, p, b.scale, out=torch.zeros_like(q)))
        for g in graphs:
            g.replay()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    pos = [x - 1 for x in lens]
    want, lse = ctx.paged_attn(q, cache, b.table, i32(pos), b.scale, with_lse=True)
    check_rows(b, q, want, lse, pos)
    mine = q.clone()
    got = ctx.paged_attn(mine, cache, b.table, i32(pos), b.scale, out=mine)
    assert got is mine and torch.equal(mine, want)
    assert ctx.status() == 0


def test_empty_batches(csa, ctx):
    """No tokens: nothing happens, whatever an empty tensor's pointer is."""
    b = Batch([40], 8, 2, 64, 16)
    cache = csa.PagedCache(b.k, b.v)
    none = i32([])
    e = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = ctx.paged_attn(e, cache, b.table, none, 0.1, req=none, with_lse=True)
    assert o.shape == (0, 8, 64) and lse.shape == (0, 8)
    kv = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    k0 = b.k.clone()
    assert ctx.qk_norm_rope(e, kv, kv, cache, none, none, tab=rope_tab(8, 64), rd=64).shape == (0, 8, 64)
    assert torch.equal(k0.nan_to_num(7.0), b.k.nan_to_num(7.0))
    length, state = i32([5]), i32([0, 2])
    info = csa.page_step(i32([0]), length, b.table, i32([1, 2]), state, 16, none, none, none)
    assert info.tolist() == [0, 0, 0, 0] and length.tolist() == [5] and ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd,latent", [(8, 2, 128, False), (16, 1, 256, True), (64, 1, 512, True), (70, 1, 320, True)])
def test_paged_attn_weights_add_up_to_one(csa, ctx, H, kv, hd, latent):
    """A feature that is the same in all rows comes back as it is: what the weights are rounded to for their product
    is what the denominator adds up.  Every 40th row scores higher than the others by so much that a weight of the
    others, 2^-0.99442 = 1.003875 / 2, lies just below a border of bf16's (1 + 2^-8) / 2 and loses 2^-8.04 of itself:
    with the weights as they were in the denominator, 1.9921875 would become 1.984375.  The f32 errors of a sum of 4000
    products are at most 2^-12 of it, half a step is 2^-9.  lse is of the weights as they were."""
    lens, page, scale, same = [40, 4000, 1, 160], 16, 0.68928, 255 / 128
    R, per = len(lens), 4000 // 16
    k = torch.full((R * per, page, kv, hd), same, dtype=torch.bfloat16, device="cuda")
    k[..., 0] = 0
    k.view(R, per * page, kv, hd)[:, 20::40, :, 0] = 1
    v = None if latent else k.clone()
    q = torch.zeros(R, H, hd, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    table = torch.arange(R * per, device="cuda", dtype=torch.int32).view(R, per)
    o, lse = ctx.paged_attn(q, csa.PagedCache(k, v), table, i32([x - 1 for x in lens]), scale, with_lse=True)
    assert (o[..., 1:].float() == same).all()
    for r, n in enumerate(lens):
        high = len(range(20, n, 40))
        want = math.log(high * math.exp(scale) + n - high)
        assert ((lse[r].double() - want).abs() <= 2.0 ** -20 * (1 + want) + n * 2.0 ** -24).all()
    assert ctx.status() == 0


# ------------------------------------------------------------------------------------------ kernels by size, alignment and heads

@pytest.mark.parametrize("R,width,N", [(300, 1100, 900), (257, 1025, 2048), (256, 1100, 300), (2049, 40, 2048), (2048, 40, 2049)])
def test_page_step_long_tables(csa, R, width, N):
    """Both sides of the rule for one CTA or eight: by the tables' width, the requests and the tokens."""
    rng = np.random.default_rng(R + width)
    lens = rng.integers(0, 30 * 16, R)
    lens[rng.integers(0, R, 5)] = (width - 3) * 16 + 7 if width > 100 else 37 * 16
    steps = []
    for _ in range(2):
        new = rng.integers(-1, 2, R)
        new[np.cumsum(np.maximum(new, 0)) > N - 20] = 0
        new[3] = 20
        steps.append(new.tolist())
    lens[3] = 5
    n_pages = int(sum(-(-x // 16) for x in lens)) + 2 * (N + R)
    check_step(csa, lens.tolist(), steps, 16, n_pages, width, N, n_pages - 5, seed=R)


@pytest.mark.parametrize("case,bit", [("tokens", 1), ("negative length", 2), ("width", 2), ("pool", 4), ("state", 8), ("overfull", 8)])
@pytest.mark.parametrize("in_place", [True, False])
def test_page_step_errors_over_eight_ctas_change_nothing(csa, case, bit, in_place):
    """An error in the middle of a large step: nothing of it is done by any CTA."""
    R, N, page, width, n_pages = 3000, 5000, 4, 30, 60000
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 100, R)
    new = rng.integers(-1, 3, R)
    lens[1700], new[1700] = 17, 1
    held = int(sum(-(-x // page) for x in lens))
    head, count = 39000, n_pages - held
    if case == "tokens":
        new[1700] = N
        lens[1700] = 0
        width = 1300
    elif case == "negative length":
        lens[1700] = -2
    elif case == "width":
        lens[1700] = width * page
    elif case == "pool":
        count = 10
    elif case == "state":
        head = n_pages
    elif case == "overfull":
        count = n_pages - 5
    t = torch.randint(0, n_pages, (R, width), dtype=torch.int32, device="cuda")
    F = torch.randperm(n_pages, device="cuda").to(torch.int32)
    L, S = i32(lens), i32([head, count])
    keep = [x.clone() for x in (t, F, L, S)]
    maps = [torch.full((N,), 5, dtype=torch.int32, device="cuda") for _ in range(3)]
    cu = torch.full((R + 1,), 9, dtype=torch.int32, device="cuda")
    outs = {} if in_place else dict(length_out=torch.full_like(L, 3), state_out=torch.full_like(S, 3))
    info = csa.page_step(i32(new), L, t, F, S, page, *maps, cu, **outs)
    assert info.tolist() == [0, 0, 0, bit]
    assert all(torch.equal(a, b) for a, b in zip((t, F, L, S), keep))
    if not in_place:
        assert torch.equal(outs["length_out"], L) and torch.equal(outs["state_out"], S)
    assert (cu == 0).all() and all((m == -1).all() for m in maps)


@pytest.mark.parametrize("hd,rd,at", [(64, 64, 0), (128, 64, 64), (80, 32, 48), (256, 256, 0), (512, 64, 448), (576, 64, 512)])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("off", [(1, 0), (0, 2), (3, 2), (2, 2)])
def test_norm_rope_tables_of_any_alignment(csa, ctx, hd, rd, at, half, off):
    """Weights that start on any 4 bytes and angles on any 8 of their buffers."""
    N, H, kv, page = 11, 3, 2, 8
    g = gen(hd + off[0])
    q, k, v = randn(g, N, H, hd), randn(g, N, kv, hd), randn(g, N, kv, hd)
    wbuf = 1 + 0.2 * torch.randn(2 * hd + 8, generator=g, device="cuda")
    qw, kw = wbuf[off[0]:off[0] + hd], wbuf[hd + 4 + off[0]:2 * hd + 4 + off[0]]
    tbuf = torch.empty(90 * rd + 4, device="cuda")
    tab = tbuf[off[1]:off[1] + 90 * rd].view(90, rd // 2, 2)
    tab.copy_(rope_tab(90, rd))
    pos = torch.randint(0, 90, (N,), generator=g, device="cuda").to(torch.int32)
    slot = torch.randperm(16, generator=g, device="cuda")[:N].to(torch.int32)
    kp, vp = (torch.zeros(2, page, kv, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = ctx.qk_norm_rope(q, k, v, csa.PagedCache(kp, vp), pos, slot, tab=tab, rd=rd, rope_at=at, half=half, q_norm=qw,
                           k_norm=kw, eps=1e-6)
    s = slot.long()
    close_rows(out, ref_rows(q, qw, 1e-6, tab, pos, rd, at, half), "q")
    close_rows(kp[s // page, s % page], ref_rows(k, kw, 1e-6, tab, pos, rd, at, half), "k")
    assert torch.equal(vp[s // page, s % page], v) and ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd,latent", [(48, 2, 64, False), (100, 1, 64, True), (33, 1, 64, False), (51, 3, 128, False),
                                            (64, 1, 256, True), (17, 1, 256, False)])
def test_paged_attn_many_heads_a_kv_head(csa, ctx, H, kv, hd, latent):
    """Head groups past the first, the last of them partly filled."""
    lens = [1, 0, 70, 333, 2000, 5]
    b = Batch(lens, H, kv, hd, 16, latent, seed=H)
    pos = [x - 1 for x in lens]
    q = b.queries(len(lens))
    sink = torch.randn(H, generator=b.g, device="cuda")
    o, lse = ctx.paged_attn(q, csa.PagedCache(b.k, b.v), b.table, i32(pos), b.scale, sink=sink, with_lse=True)
    check_rows(b, q, o, lse, pos, None, sink)
    assert ctx.status() == 0


@pytest.mark.parametrize("H,kv,hd,latent", [(8, 2, 128, False), (24, 2, 64, False), (4, 1, 256, True), (64, 1, 512, True)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_paged_attn_values_that_are_not_finite(csa, ctx, H, kv, hd, latent, bad):
    """A NaN or an infinity in an attended row: results that it enters are not finite, every other request's are as without
    it, and so are those of rows that end before it."""
    lens = [300, 2500, 40, 2500]
    b = Batch(lens, H, kv, hd, 16, latent, seed=2)
    q = b.queries(6)
    cache = csa.PagedCache(b.k, b.v)
    req, pos = [0, 1, 2, 3, 1, 1], [299, 2499, 39, 2499, 1199, 2000]
    args = (q, cache, b.table, i32(pos), b.scale)
    want, want_lse = ctx.paged_attn(*args, req=i32(req), with_lse=True)
    page, at = int(b.table[1, 1200 // 16]), 1200 % 16
    if latent:
        b.k[page, at, 0, 3] = bad
    else:
        b.v[page, at, 1, 3] = bad
    o, lse = ctx.paged_attn(*args, req=i32(req), with_lse=True)
    hit = [1, 5]
    kept = [n for n in range(6) if n not in hit]
    assert torch.equal(o[kept], want[kept]) and torch.equal(lse[kept], want_lse[kept])
    if latent:  # (the row's score is an infinity or NaN too: it takes the whole head, or leaves it but for the feature)
        assert not o[hit][..., 3].isfinite().any()
        nan_head = lse[hit].isnan() | lse[hit].isposinf()
        assert o[hit].isnan()[nan_head].all()
    else:
        g = H // kv
        assert not o[hit][:, g:, 3].isfinite().any() and torch.equal(lse[hit], want_lse[hit])
        rest = [d for d in range(hd) if d != 3]
        assert torch.equal(o[hit][:, :, rest], want[hit][:, :, rest]) and torch.equal(o[hit][:, :g], want[hit][:, :g])
    # a key: the whole head
    if not latent:
        b.v[page, at, 1, 3] = 0
        b.k[page, at, 1, :] = float("nan")
        o, lse = ctx.paged_attn(*args, req=i32(req), with_lse=True)
        assert o[hit][:, g:].isnan().all() and lse[hit][:, g:].isnan().all() and torch.equal(o[hit][:, :g], want[hit][:, :g])
        assert torch.equal(o[kept], want[kept])
    assert ctx.status() == 0


# ------------------------------------------------------------------------------------------ at the bounds

@pytest.mark.parametrize("H,kv,hd,page", [(1, 1, 64, 16), (12, 1, 128, 17), (2, 1, 512, 16), (2, 1, 512, 17)])
def test_paged_attn_rows_up_to_2_31(csa, ctx, H, kv, hd, page):
    """One row over the most positions that a table may hold (the table names the same pages again and again): the
    last unit ends past 2^31.  All scores are 0 and all values of a feature the same power of two, so that the
    result is that value and every sum before the shares are joined is exact; up to 640 roundings of the joins'
    sums move lse by at most 640 x 2^-24."""
    width = (2 ** 31 - 1) // page
    rows = width * page
    n_pages = 1024
    row = 2.0 ** (torch.arange(hd, device="cuda") % 5 - 2)
    k = row.to(torch.bfloat16).expand(n_pages, page, kv, hd).contiguous()
    table = (torch.arange(width, device="cuda", dtype=torch.int32) % n_pages)[None]
    q = torch.zeros(1, H, hd, dtype=torch.bfloat16, device="cuda")
    o, lse = ctx.paged_attn(q, csa.PagedCache(k), table, i32([rows - 1]), 1.0, with_lse=True)
    assert torch.equal(o, row.to(torch.bfloat16).expand(1, H, hd))
    assert ((lse.double() - math.log(rows)).abs() <= 640 * 2.0 ** -24 + 2.0 ** -21 * math.log(rows)).all()
    assert ctx.status() == 0


@pytest.mark.parametrize("in_place", [True, False])
def test_page_step_as_many_tokens_as_can_be_counted(csa, in_place):
    """Twice 2^30 - 2 new tokens on pages that the requests hold already, N at its bound: one request's fit, two's do not."""
    N = 2 ** 30 - 1
    page = N
    maps = [torch.empty(N, dtype=torch.int32, device="cuda") for _ in range(3)]
    for new, err in (([N - 1, N - 1], 1), ([N - 1, 1], 0)):
        t, L, S, F = i32([[0], [0]]), i32([1, 1]), i32([0, 0]), i32([7])
        cu = i32([9, 9, 9])
        outs = {} if in_place else dict(length_out=i32([5, 5]), state_out=i32([5, 5]))
        info = csa.page_step(i32(new), L, t, F, S, page, *maps, cu, **outs)
        got_l, got_s = (L, S) if in_place else (outs["length_out"], outs["state_out"])
        assert info.tolist() == ([0, 0, 0, 1] if err else [N, 0, 0, 0])
        assert got_l.tolist() == ([1, 1] if err else [N, 2]) and got_s.tolist() == [0, 0]
        assert cu.tolist() == ([0, 0, 0] if err else [0, N - 1, N])
        assert t.tolist() == [[0], [0]] and F.tolist() == [7]
        if err:
            assert all(bool((m == -1).all()) for m in maps)
        else:
            assert [int(m[N - 1]) for m in maps] == [1, 1, 1] and [int(m[N - 2]) for m in maps] == [0, N - 1, N - 1]


# ------------------------------------------------------------------------------------------ together

@pytest.mark.parametrize("latent", [False, True])
def test_steps_in_a_graph(csa, ctx, latent):
    """Decode steps of a batch as they are served: page_step in place, projection, qk_norm_rope into the pages, paged_attn,
    captured once and replayed while requests grow over page ends, wait and end; every stage against its own
    64-bit form on what it was given, over an allocator in plain Python."""
    H, kv, hd, page, rd = (64, 1, 512, 16, 64) if latent else (16, 4, 128, 16, 128)
    dim, N = 256, 12
    g = gen(21)
    lens = [0, 1, 15, 16, 17, 40, 200, 31]
    R, n_pages, width = len(lens), 40, 16
    pool = Pool(n_pages, page, lens, 3)
    table, free, state, length = i32(pool.table(width)), i32(pool.ring(5)), i32([5, len(pool.free)]), i32(lens)
    new = i32([1] * R)
    maps = [torch.empty(N, dtype=torch.int32, device="cuda") for _ in range(3)]
    kp = randn(g, n_pages, page, kv, hd)
    vp = None if latent else randn(g, n_pages, page, kv, hd)
    cache = csa.PagedCache(kp, vp)
    parts = 1 if latent else 2
    W = randn(g, (H + parts * kv) * hd, dim, scale=dim ** -0.5)
    x = randn(g, N, dim)
    qn, kn = (1 + 0.1 * torch.randn(hd, generator=g, device="cuda") for _ in range(2))
    tab = rope_tab(400, rd)
    sink = torch.randn(H, generator=g, device="cuda")
    y = torch.empty(N, (H + parts * kv) * hd, dtype=torch.bfloat16, device="cuda")
    q = torch.full((N, H, hd), 5.0, dtype=torch.bfloat16, device="cuda")
    o = torch.full((N, H, hd), 5.0, dtype=torch.bfloat16, device="cuda")
    info = torch.empty(4, dtype=torch.int32, device="cuda")

    def step():
        csa.page_step(new, length, table, free, state, page, *maps, info=info)
        ctx.linear(x, W, out=y)
        yq = y[:, :H * hd].view(N, H, hd)
        yk = y[:, H * hd:(H + kv) * hd].view(N, kv, hd)
        yv = None if latent else y[:, (H + kv) * hd:].view(N, kv, hd)
        ctx.qk_norm_rope(yq, yk, yv, cache, maps[1], maps[2], tab=tab, rd=rd, half=not latent, q_norm=qn, k_norm=kn, q_out=q)
        ctx.paged_attn(q, cache, table, maps[1], hd ** -0.5, req=maps[0], sink=sink, out=o)

    steps = [[1] * R, [1, 0, 1, 1, -1, 1, 1, 2], [1, 3, -1, 1, 2, 0, 1, 1], [0] * R, [1] * R]
    graph = torch.cuda.CUDAGraph()
    before = [t.clone() for t in (table, free, state, length, kp)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()  # warm-up, undone below
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for t, t0 in zip((table, free, state, length, kp), before):
        t.copy_(t0)
    q.fill_(5.0)
    o.fill_(5.0)
    for st in steps:
        new.copy_(i32(st))
        x.copy_(randn(g, N, dim))
        q_before, o_before = q.clone(), o.clone()
        graph.replay()
        torch.cuda.synchronize()
        toks, took, back = pool.step(st)
        n = len(toks)
        assert info.tolist() == [n, took, back, 0] and length.tolist() == pool.lens
        assert [maps[k][:n].tolist() for k in range(3)] == [[t[k] for t in toks] for k in range(3)]
        pos = maps[1][:n]
        close_rows(q[:n], ref_rows(y[:n, :H * hd].view(n, H, hd), qn, ctx.cfg.eps, tab, pos, rd, hd - rd, not latent), "q")
        slot = maps[2][:n].long()
        close_rows(kp[slot // page, slot % page],
                   ref_rows(y[:n, H * hd:(H + kv) * hd].view(n, kv, hd), kn, ctx.cfg.eps, tab, pos, rd, hd - rd, not latent), "k")
        assert torch.equal(q[n:], q_before[n:]) and torch.equal(o[n:], o_before[n:])
        for i, (r, p, _) in enumerate(toks):
            ids = torch.tensor(pool.pages[r], device="cuda")
            j = torch.arange(p + 1, device="cuda")
            K = kp[ids[j // page], j % page]
            V = K if latent else vp[ids[j // page], j % page]
            want, _, A, d = ref_attn(q[i], K, V, kv, hd ** -0.5, sink)
            tol = 2.0 ** -8 * want.abs() + (2 * d + (2.0 ** -8 if latent else 2.0 ** -16)) * A
            assert ((o[i].double() - want).abs() <= tol).all()
    assert ctx.status() == 0
