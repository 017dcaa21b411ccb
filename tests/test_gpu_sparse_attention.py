"""GPU: page bounds and page selection against their definitions in whole numbers, attention over the selected pages against
64 bits (test_gpu_tree_attention.py says where its tolerance comes from)."""
import math

import numpy as np
import pytest
import torch

import _decode_ref
import _step_ref as ref
import block_scaled_fp8_weight_gb300 as bsf8
from test_gpu_tree_attention import Problem

pytestmark = pytest.mark.gpu

INDEX = 10


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def random_cache(r, pages, H, page, D, low=20, high=250):
    """Any codes but NaN, any exponents whose values bf16 holds without rounding."""
    good = np.concatenate([np.arange(0, 127), np.arange(128, 255)]).astype(np.uint8)
    code = lambda: good[r.integers(0, 254, size=(pages, H, page, D))]  # noqa: E731
    byte = lambda: r.integers(low, high, size=(pages, H, page, D // 32)).astype(np.uint8)  # noqa: E731
    return [code(), byte(), code(), byte()]


def fresh_bounds(r, pages, H, page, D):
    """Bounds full of arbitrary bytes."""
    return bsf8.PageBounds(torch.from_numpy(r.integers(-128, 128, size=(pages, H, 2, D)).astype(np.int8)).cuda(),
                           torch.from_numpy(r.integers(0, 256, size=(pages, H, D // 32)).astype(np.uint8)).cuda(), page)


@pytest.mark.parametrize("D,H,page,B,most", [(64, 1, 16, 1, 1), (128, 8, 64, 3, 5), (256, 2, 48, 5, 9), (64, 5, 1024, 2, 2),
                                             (128, 2, 16, 70, 30), (128, 1, 32, 1024, 3), (128, 3, 64, 1, 400)])
def test_bounds(bsf8_lib, D, H, page, B, most):
    """Pages that became full, bit for bit; every other page's bounds stay."""
    r = np.random.default_rng(D + B)
    pages = B * most + 2
    data = random_cache(r, pages, H, page, D)
    data[1][:, :, :, 0] = np.maximum(data[1][:, :, :, 0], 120) - 0  # a block of alike exponents
    data[1][::2] = np.clip(data[1][::2], 118, 126)                 # pages as they are in earnest
    data[0][1, :, :, :32] = 0                                      # zeros
    data[0][-1, :, :, :32] = 0x80
    if pages > 4:
        data[1][2, 0, page - 1, 0] = 255                           # a block marked NaN
        data[0][3, H - 1, 0, 5], data[1][3, H - 1, 0, 0] = 0x7E, 254  # 448 * 2^127
    table = r.permutation(pages)[:B * most].reshape(B, most)
    end = r.integers(0, most * page + 1, size=B)
    end[0] = most * page
    start = np.minimum(end, r.integers(0, most * page + 1, size=B)) if B > 1 else end * 0
    cache = bsf8.KVCache(*(torch.from_numpy(t).cuda() for t in data))
    b = fresh_bounds(r, pages, H, page, D)
    want, byte = b.codes.cpu().numpy().copy(), b.exps.cpu().numpy().copy()
    touched = np.concatenate([table[i, start[i] // page:end[i] // page] for i in range(B)])
    want[touched], byte[touched] = ref.bounds(data[0][touched], data[1][touched])
    bsf8.kv_bounds(cache, b, i32(table), i32(end), start=i32(start) if B > 1 else None)
    assert np.array_equal(b.exps.cpu().numpy(), byte) and np.array_equal(b.codes.cpu().numpy(), want)
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("D,H,page,B,most", [(64, 10, 16, 100, 40), (64, 5, 48, 60, 70), (128, 8, 16, 64, 40), (256, 8, 16, 33, 41),
                                             (64, 3, 16, 100, 41)])
def test_bounds_of_many_short_pages(bsf8_lib, D, H, page, B, most):
    """More pages than warps: some to a warp at once, the last ones fewer, bad entries and marked blocks among them."""
    r = np.random.default_rng(D + B + page)
    pages = B * most + 1
    data = random_cache(r, pages, H, page, D, 110, 130)
    data[1][r.integers(0, pages, 50), r.integers(0, H, 50), r.integers(0, page, 50), r.integers(0, D // 32, 50)] = 255
    table = r.permutation(pages)[:B * most].reshape(B, most)
    given = table.copy()
    wrong = r.integers(0, B * most, 40)
    given.reshape(-1)[wrong] = np.where(wrong % 2, -1 - wrong, pages + wrong)
    cache = bsf8.KVCache(*(torch.from_numpy(t).cuda() for t in data))
    b = fresh_bounds(r, pages, H, page, D)
    want, byte = b.codes.cpu().numpy().copy(), b.exps.cpu().numpy().copy()
    touched = np.delete(table.reshape(-1), wrong)
    want[touched], byte[touched] = ref.bounds(data[0][touched], data[1][touched])
    bsf8.kv_bounds(cache, b, i32(given), i32([most * page] * B))
    assert np.array_equal(b.exps.cpu().numpy(), byte) and np.array_equal(b.codes.cpu().numpy(), want)
    assert bsf8.device_status() == INDEX


def test_bounds_bound_the_keys(bsf8_lib):
    """q . k of every key is below the page's sum."""
    r = np.random.default_rng(3)
    data = random_cache(r, 6, 2, 32, 128, 118, 126)
    cache = bsf8.KVCache(*(torch.from_numpy(t).cuda() for t in data))
    b = bsf8.PageBounds.empty(cache)
    bsf8.kv_bounds(cache, b, i32(np.arange(6)[None]), i32([192]))
    k = _decode_ref.decode(data[0], data[1])
    c = b.codes.cpu().numpy() * np.repeat(2.0 ** (b.exps.cpu().numpy().astype(float) - 127), 32, -1)[:, :, None]
    for _ in range(20):
        q = r.standard_normal(128)
        top = np.maximum(q, 0) * c[:, :, 0] + np.minimum(q, 0) * c[:, :, 1]
        assert np.all((k @ q).max(-1) <= top.sum(-1) + 1e-9)


def test_bad_lengths_and_pages_of_bounds(bsf8_lib):
    r = np.random.default_rng(4)
    data = random_cache(r, 5, 1, 16, 64)
    cache = bsf8.KVCache(*(torch.from_numpy(t).cuda() for t in data))
    for table, start, end, good in (([[0, 9, 1]], [0], [48], [0, 1]), ([[0, -1, 1]], [0], [48], [0, 1]),
                                    ([[0, 1, 2], [3, 4, 0]], [0, -1], [32, 48], [0, 1]),
                                    ([[0, 1, 2], [3, 4, 0]], [0, 20], [48, 10], [0, 1, 2]),
                                    ([[0, 1, 2], [3, 4, 0]], [0, 0], [16, 49], [0])):
        b = fresh_bounds(r, 5, 1, 16, 64)
        want, byte = b.codes.cpu().numpy().copy(), b.exps.cpu().numpy().copy()
        want[good], byte[good] = ref.bounds(data[0][good], data[1][good])
        bsf8.kv_bounds(cache, b, i32(table), i32(end), start=i32(start))
        assert np.array_equal(b.exps.cpu().numpy(), byte) and np.array_equal(b.codes.cpu().numpy(), want)
        assert bsf8.device_status() == INDEX


class Choice:
    """Requests over a pool of pages with bounds of any kind, and queries."""

    def __init__(self, seed, ctx, T, Hq, H, D, page, keep, sink=0, recent=0, nodes=None, scale=1.0, spread=4, ld=0):
        r = np.random.default_rng(seed)
        self.ctx, self.T, self.Hq, self.H, self.D, self.page = ctx, T, Hq, H, D, page
        self.keep, self.sink, self.recent = keep, sink, recent
        B = len(ctx)
        self.nodes = [T] * B if nodes is None else nodes
        need = [max(1, -(-(c + T) // page)) for c in ctx]
        pages = sum(need) + 2
        order = r.permutation(pages)
        self.table = np.full((B, max(need) + 1), -7)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.codes = r.integers(-127, 128, size=(pages, H, 2, D)).astype(np.int8)
        self.exps = r.integers(124 - spread, 125, size=(pages, H, D // 32)).astype(np.uint8)
        q = (r.standard_normal((B, T, Hq * D + ld)) * scale).astype(np.float32)
        self.q = torch.from_numpy(q).to(torch.bfloat16).cuda()[:, :, :Hq * D].unflatten(2, (Hq, D))

    def check(self, status=0, **kw):
        bounds = bsf8.PageBounds(torch.from_numpy(self.codes).cuda(), torch.from_numpy(self.exps).cuda(), self.page)
        pages, kept = bsf8.select_pages(self.q, bounds, i32(self.table), i32(self.ctx), self.keep, nodes=i32(self.nodes),
                                        sink=self.sink, recent=self.recent, **kw)
        q = self.q.double().cpu().numpy()
        for b, (c, n) in enumerate(zip(self.ctx, self.nodes)):
            want, k = ref.select(q[b], self.codes, self.exps, self.table[b], c, n, self.page, self.keep, self.sink, self.recent,
                                 pages.shape[2])
            assert np.array_equal(pages[b].cpu().numpy(), want), b
            assert int(kept[b]) == k
        assert bsf8.device_status() == status
        return pages, kept


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,Hq,H,page", [(1, 1, 1, 16), (1, 8, 2, 64), (5, 14, 2, 48), (33, 3, 3, 16), (1, 16, 1, 32), (256, 16, 1, 64)])
@pytest.mark.parametrize("keep,sink,recent", [(1, 0, 0), (5, 1, 2), (64, 0, 3), (7, 7, 0), (130, 2, 2)])
def test_selection(bsf8_lib, D, T, Hq, H, page, keep, sink, recent):
    """Lengths around the pages' ends and around `keep` pages, none at all, some hundred pages."""
    ctx = [0, 1, page - 1, page, keep * page, keep * page + page, keep * page + 2 * page - 1, 301 * page + 3]
    r = np.random.default_rng(T)
    Choice(D + keep, ctx, T, Hq, H, D, page, keep, sink, recent, nodes=[int(n) for n in r.integers(1, T + 1, size=len(ctx))]).check()


@pytest.mark.parametrize("n,keep", [(9000, 64), (9000, 8999), (49152, 700), (2049, 1000)])
@pytest.mark.parametrize("H", [1, 5])
def test_selection_of_many_pages(bsf8_lib, n, keep, H):
    Choice(n + H, [n * 16 + 5], 1, 2 * H, H, 64, 16, keep, 1, 2).check(max_len=n * 16 + 6)


@pytest.mark.parametrize("D,n,keep", [(128, 45000, 300), (256, 42000, 41000), (128, 40950, 5)])
def test_selection_of_many_pages_of_larger_heads(bsf8_lib, D, n, keep):
    Choice(n, [n * 16 + 5, 40], 2, 3, 1, D, 16, keep, 1, 2).check(max_len=n * 16 + 8)


def test_selection_for_many_requests(bsf8_lib):
    r = np.random.default_rng(2)
    Choice(5, [int(c) for c in r.integers(0, 5000, size=300)], 1, 8, 4, 128, 16, 20, 1, 1).check()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("full,keep", [(33, 32), (40, 3), (257, 31), (2049, 2000)])
def test_selection_of_a_few_pages_again_and_again(bsf8_lib, D, full, keep):
    """Warps whose pages end early, or that have none, ask for copies that write zeros where the keys are counted and listed
    next: hundreds of calls give the same pages."""
    c = Choice(D + full, [full * 16 + 3] * 40, 1, 4, 2, D, 16, keep)
    want = c.check()[0]
    bounds = bsf8.PageBounds(torch.from_numpy(c.codes).cuda(), torch.from_numpy(c.exps).cuda(), 16)
    table, ctx = i32(c.table), i32(c.ctx)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        differ += (bsf8.select_pages(c.q, bounds, table, ctx, keep)[0] != want).sum()
    assert int(differ) == 0 and bsf8.device_status() == 0


def test_equal_scores_go_to_the_lowest_index(bsf8_lib):
    c = Choice(6, [16 * 700, 16 * 33], 1, 2, 2, 64, 16, 31)
    c.codes[:] = c.codes[:1]
    c.exps[:] = 120
    c.check()
    c.codes[:, 0] = np.arange(len(c.codes))[:, None, None] % 3  # a few scores, often each
    c.check()
    c.q = c.q * 0  # all scores 0, of either sign
    c.codes = np.random.default_rng(1).integers(-127, 128, size=c.codes.shape).astype(np.int8)
    c.check()


def test_queries_and_bounds_at_their_ends(bsf8_lib):
    """Infinite and NaN query elements count as 0; tiny, huge and very uneven queries; pages with NaN come first;
    exponents over their whole range; a request without nodes."""
    c = Choice(7, [16 * 90 + 1] * 6, 3, 4, 2, 128, 16, 20, 1, 1, nodes=[3, 3, 3, 3, 0, 2])
    c.q[0, 0, 0, 3], c.q[0, 1, 1, 9], c.q[0, 2, 3] = math.inf, -math.inf, math.nan
    c.q[1] = math.nan
    c.q[2] = c.q[2] * 2.0 ** 120
    c.q[3] = c.q[3] * 2.0 ** -120
    c.q[5, 0] = c.q[5, 0] * 2.0 ** -14
    c.check()
    r = np.random.default_rng(8)
    c.exps[r.random(c.exps.shape) < 0.05] = 255
    c.check()  # on average 36 pages a head hold one: more than `keep`
    c.keep = 70
    c.check()
    c.exps = r.integers(0, 250, size=c.exps.shape).astype(np.uint8)
    c.check()
    c.exps = r.integers(0, 4, size=c.exps.shape).astype(np.uint8)
    c.check()


@pytest.mark.parametrize("full,keep", [(90, 20), (3000, 2500), (300, 1)])
def test_scores_that_are_nan_count_as_infinite(bsf8_lib, monkeypatch, full, keep):
    """Bounds that kv_bounds does not write: sums of exponent 2^127 that overflow downwards beside blocks of byte 255.  Their
    pages come first, `keep` of them at most, and nothing is written behind a row of the list."""
    c = Choice(15, [16 * full + 2], 2, 4, 2, 256, 16, keep)
    c.q[:, 1] = -c.q[:, 0]  # sums of both signs, of almost 2^14, in all channels
    c.q[:] = torch.where(c.q < 0, -255 / 128, 255 / 128).to(c.q.dtype)
    r = np.random.default_rng(15)
    down = r.random(len(c.codes)) < 0.6
    c.codes[down, :, 0], c.codes[down, :, 1] = -128, 127
    c.exps[down] = 254
    c.exps[down, :, 7] = 255
    plain = ref.scores

    def scores(*a):
        with np.errstate(all="ignore"):
            f = plain(*a)
        assert np.isnan(f).sum() > full // 3
        return np.where(np.isnan(f), np.inf, f)
    monkeypatch.setattr(ref, "scores", scores)
    c.check()


def test_query_rows_with_a_stride(bsf8_lib):
    Choice(9, [16 * 50, 16 * 80 + 7], 4, 6, 3, 64, 16, 12, ld=40).check()


def test_bad_lengths_and_pages_of_a_selection(bsf8_lib):
    c = Choice(10, [16 * 40], 2, 2, 1, 64, 16, 10)
    c.table[0, 5] = len(c.codes)  # its score is the lowest of all
    want = c.table[0, :40].tolist()
    bounds = bsf8.PageBounds(torch.from_numpy(c.codes).cuda(), torch.from_numpy(c.exps).cuda(), 16)
    pages, kept = bsf8.select_pages(c.q, bounds, i32(c.table), i32(c.ctx), 10)
    assert bsf8.device_status() == INDEX and len(c.codes) not in pages[0, 0, :10].tolist()
    pages, kept = bsf8.select_pages(c.q, bounds, i32(c.table), i32(c.ctx), 40)  # all stay: the attention will find it
    assert pages[0, 0, :40].tolist() == want
    assert bsf8.device_status() == 0
    c.table[0, 5] = 0
    for ctx, nodes in (([-1], [2]), ([16 * 42], [2]), ([640], [3]), ([640], [-1]), ([2 ** 31 - 1], [2])):
        pages, kept = bsf8.select_pages(c.q, bounds, i32(c.table), i32(ctx), 10, nodes=i32(nodes), max_len=642)
        assert bsf8.device_status() == INDEX
        assert 0 <= int(kept[0]) <= 160 + 15


def bounds_of(p, cache):
    b = bsf8.PageBounds.empty(cache)
    bsf8.kv_bounds(cache, b, i32(np.where(p.table == 1 << 30, 0, p.table)), i32(p.ctx))
    return b


def check_sparse(p, pages, out, lse):
    """Attention of Problem p over these pages in 64 bits, a head at a time."""
    g = p.Hq // p.Hkv
    out, lse, pages = out.double().cpu(), lse.double().cpu(), pages.cpu().numpy()
    for b in range(p.B):
        n, full, rest = int(p.nodes[b]), int(p.ctx[b]) // p.page, int(p.ctx[b]) % p.page
        assert not out[b, n:].any() and torch.all(lse[b, n:] == -math.inf)
        for h in range(p.Hkv):
            own = pages[b, h][pages[b, h] >= 0]
            tail = -(-(rest + n) // p.page)
            c = (len(own) - tail) * p.page + rest
            s = np.arange(c + n)
            pg, off = own[s // p.page], s % p.page
            k = _decode_ref.decode(p.data[0][pg, h, off], p.data[1][pg, h, off])
            v = _decode_ref.decode(p.data[2][pg, h, off], p.data[3][pg, h, off])
            q = p.q[b, :n, h * g:(h + 1) * g].double().numpy().reshape(n * g, p.D)
            see = np.concatenate([np.ones((n, c), bool), p.see[b, :n, :n]], 1)
            want, wl, mass, reach = _decode_ref.attention(q, k, v, np.repeat(see, g, 0), p.D ** -0.5)
            got = out[b, :n, h * g:(h + 1) * g].reshape(n * g, p.D)
            tol = want.abs() * 2.0 ** -8 + mass * (2.0 ** -9 + 2.0 ** -11 + 2.0 ** -14 + 2.0 ** -15 * reach[:, None])
            tol = tol + (c + n) * 2.0 ** -40 * np.nanmax(np.abs(v), initial=0.0)
            assert ((got - want).abs() <= tol).all(), (b, h)
            gl = lse[b, :n, h * g:(h + 1) * g].reshape(n * g)
            assert torch.all((gl - wl).abs() <= 2.0 ** -14 + 2.0 ** -16 * reach + 2.0 ** -22 * wl.abs())


@pytest.mark.parametrize("D,Hq,Hkv,T,page,keep", [(64, 4, 2, 1, 16, 3), (128, 8, 2, 1, 64, 40), (128, 14, 2, 9, 32, 9), (256, 3, 3, 2, 48, 5),
                                                  (64, 16, 1, 33, 16, 70), (128, 4, 4, 200, 64, 4), (256, 16, 2, 1, 128, 2)])
def test_attention_over_selected_pages(bsf8_lib, D, Hq, Hkv, T, page, keep):
    ctx = [0, 5, page, keep * page - 1, keep * page + 3, 5000 + 3 * page, 3000]
    r = np.random.default_rng(T)
    p = Problem(D + T, len(ctx), T, Hq, Hkv, D, page, ctx, nodes=r.integers(1, T + 1, size=len(ctx)), mask="tree" if T > 1 else None)
    cache = p.cache()
    mask = None if p.mask is None else torch.from_numpy(p.mask).cuda()
    pages, kept = bsf8.select_pages(p.q.cuda(), bounds_of(p, cache), i32(p.table), i32(p.ctx), keep, nodes=i32(p.nodes),
                                    sink=1, recent=1)
    lse = torch.empty((p.B, T, Hq), device="cuda")
    out = bsf8.sparse_attention(p.q.cuda(), cache, pages, kept, nodes=i32(p.nodes), mask=mask, lse=lse)
    check_sparse(p, pages, out, lse)
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("T,D,page", [(1, 128, 64), (7, 64, 16), (40, 128, 32)])
def test_all_pages_selected_is_tree_attention(bsf8_lib, T, D, page):
    """Bit for bit: the same tiles in the same order."""
    p = Problem(3, 3, T, 8, 2, D, page, [4000, 77, 0], mask="tree" if T > 1 else None)
    want, wl = p.run(max_len=4000 + T)
    cache = p.cache()
    pages, kept = bsf8.select_pages(p.q.cuda(), bounds_of(p, cache), i32(p.table), i32(p.ctx), 4000 // page)
    assert kept.tolist() == [4000, 77, 0]
    lse = torch.empty((3, T, 8), device="cuda")
    mask = None if p.mask is None else torch.from_numpy(p.mask).cuda()
    out = bsf8.sparse_attention(p.q.cuda(), cache, pages, kept, mask=mask, lse=lse, max_len=4000 + T)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, wl)


def test_the_best_pages_find_a_planted_key(bsf8_lib):
    """A key that a query looks for, in one page of hundreds: its page is among the few kept, and the output is its value's."""
    r = np.random.default_rng(12)
    p = Problem(12, 1, 1, 4, 1, 128, 64, [30000], mask=None, qscale=4.0)
    at = 17003
    q = p.q[0, 0, 2].double().numpy()  # one of the group's heads
    page, off = p.table[0, at // 64], at % 64
    code, byte = _decode_ref.quantise(np.float32(q * 40)[None])
    p.data[0][page, 0, off], p.data[1][page, 0, off] = code[0], byte[0]
    cache = p.cache()
    pages, kept = bsf8.select_pages(p.q.cuda(), bounds_of(p, cache), i32(p.table), i32(p.ctx), 12)
    assert int(page) in pages[0, 0].tolist() and int(kept[0]) == 12 * 64 + 30000 % 64
    out = bsf8.sparse_attention(p.q.cuda(), cache, pages, kept)
    v = _decode_ref.decode(p.data[2][page, 0, off], p.data[3][page, 0, off])
    assert np.abs(out[0, 0, 2].double().cpu().numpy() - v).max() <= np.abs(v).max() * 2.0 ** -6


def test_selection_and_attention_in_a_graph(bsf8_lib):
    p = Problem(13, 2, 5, 4, 2, 128, 32, [2000, 900])
    cache, b = p.cache(), None
    b = bounds_of(p, cache)
    q, table, ctx = p.q.cuda(), i32(np.where(p.table == 1 << 30, 0, p.table)), i32(p.ctx)
    mask = torch.from_numpy(p.mask).cuda()

    def step():
        bsf8.kv_bounds(cache, b, table, ctx)
        pages, kept = bsf8.select_pages(q, b, table, ctx, 20, sink=1)
        return bsf8.sparse_attention(q, cache, pages, kept, mask=mask)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for s in (1.0, -1.0, 3.0):
        q.copy_(p.q.cuda() * s)
        g.replay()
        assert torch.equal(out, step())


def test_refused_tensors(bsf8_lib):
    p = Problem(14, 2, 1, 4, 2, 64, 16, [100, 50])
    cache = p.cache()
    b = bounds_of(p, cache)
    q, table, ctx = p.q.cuda(), i32(np.where(p.table == 1 << 30, 0, p.table)), i32(p.ctx)
    pages, kept = bsf8.select_pages(q, b, table, ctx, 3)
    for bad in (lambda: bsf8.select_pages(q[..., :32], b, table, ctx, 3), lambda: bsf8.select_pages(q, b, table[:1], ctx, 3),
                lambda: bsf8.select_pages(q, b, table, ctx[:1], 3), lambda: bsf8.sparse_attention(q, cache, pages[:, :1], kept),
                lambda: bsf8.sparse_attention(q, cache, table, ctx), lambda: bsf8.kv_bounds(cache, b, table, ctx[:1]),
                lambda: bsf8.sparse_attention(q, cache, pages, kept[:1])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: bsf8.select_pages(q.float(), b, table, ctx, 3), lambda: bsf8.select_pages(q, b, table.long(), ctx, 3),
                lambda: bsf8.select_pages(q, b, table, ctx, 3.5)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: bsf8.select_pages(q, b, table, ctx, 0), lambda: bsf8.select_pages(q, b, table, ctx, 3, sink=4),
                lambda: bsf8.kv_bounds(cache, bsf8.PageBounds(b.codes, b.exps, 32), table, ctx)):
        with pytest.raises(bsf8.Bsf8Error):
            bad()
