"""GPU: attention of token trees over the paged cache against a plain 64-bit implementation.

Tolerance, from how the result is formed (per output, with A = sum p |v| of the row):
  * one rounding to bf16: half a step, at most 2^-8 of the value (and 2^-9 of A covers values
    that nearly cancel);
  * each p rounded to 11 bits before it meets its value: 2^-11 A; values rebuilt exactly within
    2^21 of the largest of their tile, below that 2^-25 of it;
  * a score summed in fp32 over D <= 256 products: off by at most D 2^-24 sum |q k| scale, which
    moves its p by as much, relatively, and the sum of the p's likewise: 2 * 2^-16 reach * A;
  * a p below 2^-29 of the row's largest loses bits, and below 2^-40 all of them: at most 2^-40 of
    the largest value a key;
  * sums over the keys in fp32, at most 2^-14 A for the lengths here."""
import math

import numpy as np
import pytest
import torch

import _decode_ref as ref
import block_scaled_fp8_weight_gb300 as bsf8

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Problem:
    """A cache of random keys and values (exponents spread over `spread` powers of two), its unused
    slots full of arbitrary bytes, NaN codes and infinite scales among them."""

    def __init__(self, seed, B, T, Hq, Hkv, D, page, ctx, nodes=None, mask="tree", spread=3, qscale=1.0, extra=0):
        r = self.r = np.random.default_rng(seed)
        self.B, self.T, self.Hq, self.Hkv, self.D, self.page = B, T, Hq, Hkv, D, page
        self.ctx = np.asarray(ctx)
        self.nodes = np.full(B, T) if nodes is None else np.asarray(nodes)
        need = [max(1, -(-int(c + T) // page)) for c in self.ctx]
        tp, pages = max(need) + extra, sum(need) + 3
        order = r.permutation(pages)
        self.table = np.full((B, tp), 1 << 30)  # entries that no slot needs: far outside
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.data = [r.integers(0, 256, size=(pages, Hkv, page, n), dtype=np.uint8) for n in (D, D // 32, D, D // 32)]
        good = np.concatenate([np.arange(0, 127), np.arange(128, 255)]).astype(np.uint8)
        for b in range(B):
            s = np.arange(self.ctx[b] + self.nodes[b])
            pg, off = self.table[b, s // page], s % page
            for j in (0, 2):
                self.data[j][pg, :, off] = good[r.integers(0, 254, size=(len(s), Hkv, D))]
                self.data[j + 1][pg, :, off] = r.integers(121 - spread, 122, size=(len(s), Hkv, D // 32))
        self.q = torch.from_numpy((r.standard_normal((B, T, Hq, D)) * qscale / 8).astype(np.float32)).to(torch.bfloat16)
        if mask == "tree":
            self.see = np.stack([ref.tree(r, T)[1] for _ in range(B)])
        elif mask == "random":
            self.see = r.random((B, T, T)) < 0.4
        else:
            self.see = np.broadcast_to(np.tril(np.ones((T, T), bool)), (B, T, T))
        self.mask = None if mask is None else ref.mask_words(self.see)

    def cache(self):
        return bsf8.KVCache(*(torch.from_numpy(t).cuda() for t in self.data))

    def run(self, cache=None, **kw):
        lse = torch.full((self.B, self.T, self.Hq), 123.0, device="cuda")
        out = bsf8.tree_attention(kw.pop("q", self.q.cuda()), cache or self.cache(), i32(self.table), i32(self.ctx),
                                  nodes=i32(self.nodes), mask=None if self.mask is None else torch.from_numpy(self.mask).cuda(),
                                  lse=lse, **kw)
        return out, lse

    def check(self, out, lse, scale=None, max_len=None):
        scale = self.D ** -0.5 if scale is None else scale
        g = self.Hq // self.Hkv
        out, lse = out.double().cpu(), lse.double().cpu()
        for b in range(self.B):
            c, n = int(self.ctx[b]), int(self.nodes[b])
            assert not out[b, n:].any() and torch.all(lse[b, n:] == -math.inf)
            if n == 0:
                continue
            s = np.arange(c + n)
            pg, off = self.table[b, s // self.page], s % self.page
            see = np.concatenate([np.ones((n, c), bool), self.see[b, :n, :n]], 1)
            for h in range(self.Hkv):
                k = ref.decode(self.data[0][pg, h, off], self.data[1][pg, h, off])
                v = ref.decode(self.data[2][pg, h, off], self.data[3][pg, h, off])
                q = self.q[b, :n, h * g:(h + 1) * g].double().numpy().reshape(n * g, self.D)
                want, wl, mass, reach = ref.attention(q, k, v, np.repeat(see, g, 0), scale)
                got = out[b, :n, h * g:(h + 1) * g].reshape(n * g, self.D)
                gl = lse[b, :n, h * g:(h + 1) * g].reshape(n * g)
                assert torch.equal(torch.isnan(got), torch.isnan(want)), (b, h)
                tol = want.abs() * 2.0 ** -8 + mass * (2.0 ** -9 + 2.0 ** -11 + 2.0 ** -14 + 2.0 ** -15 * reach[:, None])
                tol = tol + (c + n) * 2.0 ** -40 * np.nanmax(np.abs(v), initial=0.0)
                ok = torch.isnan(want) | ((got - want).abs() <= tol)
                assert ok.all(), (b, h, float(((got - want).abs() / tol).nan_to_num(0).max()))
                none = torch.isinf(wl)
                assert torch.equal(none, gl == -math.inf)
                fine = ~none & ~torch.isnan(wl)
                assert torch.equal(torch.isnan(wl), torch.isnan(gl))
                assert torch.all((gl - wl).abs()[fine] <= (2.0 ** -14 + 2.0 ** -16 * reach + 2.0 ** -22 * wl.abs())[fine])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,T,page", [(1, 1, 1, 16), (8, 2, 1, 64), (14, 2, 5, 48), (32, 2, 9, 16), (12, 3, 33, 32),
                                           (16, 1, 1, 128), (20, 1, 64, 16)])
def test_matches_64_bits(bsf8_lib, D, Hq, Hkv, T, page):
    """Contexts around the pages' and the tiles' ends, and none at all."""
    ctx = [0, 1, 15, 16, 63, 64, 127, 128, 129, 300]
    p = Problem(D + T, len(ctx), T, Hq, Hkv, D, page, ctx, mask="tree" if T > 1 else None)
    p.check(*p.run())
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("ctx,B", [(5000, 1), (20011, 2), (777, 40)])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 4, 1, 128), (7, 14, 2, 64), (40, 16, 2, 128), (3, 4, 2, 256)])
def test_long_contexts_split_over_the_sms(bsf8_lib, ctx, B, T, Hq, Hkv, D):
    r = np.random.default_rng(ctx)
    c = [ctx] if B == 1 else np.concatenate([[ctx, 0], r.integers(0, ctx, size=B - 2)])
    p = Problem(ctx + T, B, T, Hq, Hkv, D, 64, c, nodes=r.integers(1, T + 1, size=B), qscale=2.0)
    a = p.run()
    p.check(*a)
    b = p.run()
    assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(a, b))  # bit for bit
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("T", [2, 31, 32, 33, 100, 256])
def test_masks_of_any_shape(bsf8_lib, T):
    """Random masks: rows that see no node; with no context, rows that see nothing at all; chains."""
    for seed, ctx in ((1, [0, 0, 3]), (2, [130, 1, 64])):
        p = Problem(seed + T, 3, T, 4, 2, 64, 16, ctx, nodes=[T, max(1, T - 3), T], mask="random")
        p.see[:, 0] = False
        p.see[1] = False
        p.mask = ref.mask_words(p.see)
        p.check(*p.run())
        p = Problem(seed + T, 3, T, 6, 1, 128, 48, ctx, nodes=[T, 0, T // 2], mask=None)
        p.check(*p.run())
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_nan_reaches_only_the_rows_that_see_it(bsf8_lib, D):
    p = Problem(11, 2, 8, 4, 2, D, 16, [40, 5])
    at = {}
    for b, node in ((0, 3), (1, 6)):
        s = int(p.ctx[b]) + node
        at[b] = (p.table[b, s // 16], s % 16)
    # a key block of node 3 of request 0, head 0; a value block of node 6 of request 1, head 1
    p.data[0][at[0][0], 0, at[0][1], 32:64], p.data[1][at[0][0], 0, at[0][1], 1] = 0x7F, 255
    p.data[2][at[1][0], 1, at[1][1], 0:32], p.data[3][at[1][0], 1, at[1][1], 0] = 0x7F, 255
    out, lse = p.run()
    p.check(out, lse)
    for t in range(8):
        assert torch.isnan(out[0, t, :2]).all() == bool(p.see[0, t, 3]) and not torch.isnan(out[0, t, 2:]).any()
        assert torch.isnan(out[1, t, 2:, :32]).all() == bool(p.see[1, t, 6])
        assert not torch.isnan(out[1, t, 2:, 32:]).any() and not torch.isnan(out[1, t, :2]).any()
    # in the context every row sees it
    p = Problem(12, 1, 3, 4, 2, D, 16, [40])
    pg, off = p.table[0, 20 // 16], 20 % 16
    p.data[2][pg, 0, off, D - 32:], p.data[3][pg, 0, off, -1] = 0x7F, 255
    out, lse = p.run()
    p.check(out, lse)
    assert torch.isnan(out[0, :, :2, D - 32:]).all() and not torch.isnan(out[0, :, :2, :D - 32]).any()


def test_wide_ranges(bsf8_lib):
    """Exponents spread over 2^14 between blocks and tokens; scales at both ends of what softmax
    needs; scores so large that one key takes all; queries of zeros."""
    for seed, kw, scale in ((1, dict(spread=14), None), (2, dict(qscale=40.0), 1.0), (3, dict(qscale=1e-3), 1e-3),
                            (4, dict(qscale=0.0), None)):
        p = Problem(seed, 3, 6, 8, 2, 128, 32, [500, 33, 0], **kw)
        p.check(*p.run(scale=scale), scale=scale)
    # a few tokens' values 2^16 above the others', at probabilities near 0
    p = Problem(6, 1, 4, 4, 1, 64, 16, [200], mask=None, spread=0)
    s = np.array([7, 130])
    p.data[3][p.table[0, s // 16], :, s % 16] += 16
    p.data[0][p.table[0, s // 16], :, s % 16] = 0x7E | 128
    p.q = p.q.abs() * 8  # their keys point away from every query
    p.check(*p.run(scale=0.02), scale=0.02)
    assert bsf8.device_status() == 0


def test_strided_queries_and_one_request(bsf8_lib):
    """q as a view of a projection's output; max_len tighter than the table; a table with more pages."""
    p = Problem(21, 3, 4, 6, 2, 128, 16, [100, 3, 59], extra=5)
    wide = torch.randn(3 * 4, 6 * 128 + 256, device="cuda").to(torch.bfloat16)
    wide[:, 64:64 + 768] = p.q.cuda().view(12, 768)
    q = wide[:, 64:64 + 768].unflatten(1, (6, 128)).unflatten(0, (3, 4))
    a = p.run(q=q, max_len=104)
    p.check(*a)
    b = p.run()
    assert bsf8.device_status() == 0
    assert torch.allclose(a[0].float(), b[0].float(), atol=2 ** -6, rtol=2 ** -6)


def test_bad_lengths_and_pages_are_reported(bsf8_lib):
    """A request longer than max_len is cut there, a page outside the cache counts as not seen; both are
    reported, and the other requests are right."""
    p = Problem(31, 3, 2, 4, 2, 64, 16, [100, 50, 70])
    good, _ = p.run()
    assert bsf8.device_status() == 0
    p.run(max_len=80)
    assert bsf8.device_status() == 10
    keep = p.table[1, 1]
    p.table[1, 1] = -7
    out, _ = p.run()
    assert bsf8.device_status() == 10
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    # the rows that are left: slots 0 .. 15 and 32 .. 51
    q = Problem(31, 3, 2, 4, 2, 64, 16, [100, 50, 70])
    k, v = q.data[0], q.data[2]
    s = np.concatenate([np.arange(16), np.arange(32, 52)])
    pg, off = q.table[1, s // 16], s % 16
    see = np.concatenate([np.ones((2, 34), bool), q.see[1]], 1)
    for h in range(2):
        kk, vv = ref.decode(k[pg, h, off], q.data[1][pg, h, off]), ref.decode(v[pg, h, off], q.data[3][pg, h, off])
        want, _, mass, reach = ref.attention(q.q[1, :, 2 * h:2 * h + 2].double().numpy().reshape(4, 64), kk, vv,
                                             np.repeat(see, 2, 0), 1 / 8)
        got = out[1, :, 2 * h:2 * h + 2].double().cpu().reshape(4, 64)
        assert torch.all((got - want).abs() <= want.abs() * 2.0 ** -8 + mass * (2.0 ** -8 + 2.0 ** -15 * reach[:, None]))
    q.table[1, 1] = keep
    q.ctx = np.array([100, -4, 70])
    out, _ = q.run()
    assert bsf8.device_status() == 10
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])


def test_in_a_graph_with_a_given_workspace(bsf8_lib):
    """Captured with append before it: replays follow the lengths in device memory."""
    p = Problem(41, 2, 3, 8, 2, 128, 16, [20, 400])
    cache, table, ctx, nodes = p.cache(), i32(p.table), i32(p.ctx), i32(p.nodes)
    q, mask = p.q.cuda(), torch.from_numpy(p.mask).cuda()
    ws = torch.empty(max(16, bsf8.tree_attention_workspace_bytes(2, 3, 8, 2, 128)), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(2, 3, 8, device="cuda")
    call = lambda: bsf8.tree_attention(q, cache, table, ctx, nodes=nodes, mask=mask, out=out, lse=lse, workspace=ws,  # noqa: E731
                                       max_len=410)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for c in ([20, 400], [0, 17], [3, 399]):
        p.ctx = np.array(c)
        ctx.copy_(i32(c))
        # the nodes' rows move with the context: check against what lies there now
        g.replay()
        torch.cuda.synchronize()
        if c == [3, 399]:
            want, wl = p.run()
            assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, wl)
        else:
            p.check(out, lse)
    assert bsf8.device_status() == 0


def test_a_table_with_room_for_more_than_2_30_tokens(bsf8_lib):
    """The default max_len is then 2^30; the requests' own lengths are what counts."""
    p = Problem(51, 1, 3, 4, 2, 64, 1024, [2500], extra=(1 << 20) + 61)
    assert p.table.shape[1] * 1024 > 1 << 30
    p.check(*p.run())
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("extra", [0, 300])  # with room for more than 2048 tokens: the kernel for few rows at dim 128
@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 4, 2, 128), (3, 4, 2, 128), (5, 2, 2, 64), (4, 8, 1, 256), (40, 8, 2, 128),
                                        (20, 12, 3, 64), (70, 2, 1, 256)])
def test_infinite_and_nan_queries(bsf8_lib, T, Hq, Hkv, D, extra):
    """q . k of such a head is an infinity or NaN for every key, so its softmax is NaN: output and lse, where it sees
    anything.  Every other head's are the same bits as without."""
    p = Problem(D + T, 3, T, Hq, Hkv, D, 16, [700, 0, 130], extra=extra, mask="random")
    p.see[1, T // 2] = False                                # sees nothing: no context, no node
    p.mask = ref.mask_words(p.see)
    good, lse0 = p.run()
    q, bad = p.q.clone(), torch.zeros(3, T, Hq, dtype=torch.bool)
    for b, t, h, c, x in ((0, 0, 0, 5, math.inf), (0, T - 1, Hq - 1, D - 1, -math.inf), (1, T // 2, 0, 0, math.inf),
                          (2, T // 2, 1, 17, math.nan), (2, 0, Hq - 1, D // 2, math.inf)):
        q[b, t, h, c] = x
        bad[b, t, h] = True
    sees = torch.tensor(p.ctx > 0)[:, None] | torch.from_numpy(p.see.any(2))
    out, lse = p.run(q=q.cuda())
    out, lse, good, lse0 = out.cpu(), lse.cpu(), good.cpu(), lse0.cpu()
    want = bad & sees[..., None]
    assert torch.isnan(out[want]).all() and torch.isnan(lse[want]).all()
    assert torch.equal(out[~want].view(torch.int16), good[~want].view(torch.int16)) and torch.equal(lse[~want], lse0[~want])
    assert not out[1, T // 2].any() and torch.all(lse[1, T // 2] == -math.inf)
    # keys that all point away from the infinite channel
    p.data[0][:, :, :, 5] |= 0x80
    p.data[0][:, :, :, 5] &= 0xFE
    out, lse = p.run(q=q.cuda())
    assert torch.isnan(out[0, 0, 0]).all() and torch.isnan(lse[0, 0, 0])
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("extra", [0, 300])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 4, 2, 128), (3, 2, 1, 128), (5, 2, 2, 64), (4, 8, 1, 256), (40, 8, 2, 128),
                                        (33, 4, 1, 64), (70, 2, 1, 256)])
@pytest.mark.parametrize("scale", [3e4, 1e7, 1e9, 1e18, 1e30])
@pytest.mark.parametrize("away", [False, True])
def test_huge_scores(bsf8_lib, T, Hq, Hkv, D, scale, extra, away):
    """Scores of up to 1e31, of either sign: one key takes all where no other is within what fp32 sums tell apart
    (D 2^-24 of sum |q k| scale, for each of the two, and that again), and the lse is its score.  The output is the
    key's value, off by p's rounding to 11 bits and its own to bf16."""
    p = Problem(7 * D + T, 3, T, Hq, Hkv, D, 16, [2300, 40, 129], extra=extra)
    if away:  # every key points away from every query
        p.q = p.q.abs()
        p.data[0] |= 0x80
        p.data[0][p.data[0] == 0xFF] = 0xFE
    out, lse = p.run(scale=scale)
    out, lse, g, clear = out.double().cpu(), lse.double().cpu(), Hq // Hkv, 0
    for b in range(3):
        c = int(p.ctx[b])
        s = np.arange(c + T)
        pg, off = p.table[b, s // 16], s % 16
        see = torch.from_numpy(np.concatenate([np.ones((T, c), bool), p.see[b]], 1))
        for h in range(Hq):
            k, v = (torch.from_numpy(ref.decode(p.data[j][pg, h // g, off], p.data[j + 1][pg, h // g, off])) for j in (0, 2))
            q = p.q[b, :, h].double()
            x = (q @ k.T * scale).masked_fill(~see, -math.inf)
            grain = 4 * D * 2.0 ** -24 * (q.abs() @ k.abs().T * scale).amax(1)
            top, at = x.topk(2, 1)
            one = top[:, 0] - top[:, 1] > grain + 200
            clear += int(one.sum())
            want = v[at[:, 0]]
            assert torch.all((out[b, :, h] - want).abs()[one] <= (want.abs() * (2.0 ** -8 + 2.0 ** -10))[one]), (b, h)
            assert torch.all((lse[b, :, h] - top[:, 0]).abs()[one] <= (grain + 2.0 ** -22 * top[:, 0].abs())[one]), (b, h)
            # the others: between the values, at the score
            assert torch.isfinite(out[b, :, h]).all() and torch.all((lse[b, :, h] - top[:, 0]).abs() <= grain + 8 + 2.0 ** -22 * top[:, 0].abs())
            assert torch.all(out[b, :, h].abs() <= v.abs().amax() * (1 + 2.0 ** -7))
    assert clear > 3 * T * Hq // 2
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("extra", [0, 300])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 4, 2, 128), (3, 2, 1, 128), (5, 2, 2, 64), (4, 8, 1, 256), (40, 8, 2, 128)])
@pytest.mark.parametrize("byte", [3, 12, 30, 236])
def test_the_smallest_and_largest_values(bsf8_lib, T, Hq, Hkv, D, extra, byte):
    """Values about 2^-116 up to 2^117, over a short context, a long one and one that no block holds alone.  The
    tolerance is check's, with half a step of bf16's subnormal numbers (2^-134), as many channels hold next to nothing."""
    p = Problem(byte + D + T, 4, T, Hq, Hkv, D, 32, [4, 300, 2000, 4500], extra=extra)
    for b in range(4):
        s = np.arange(int(p.ctx[b]) + T)
        pg, off = p.table[b, s // 32], s % 32
        p.data[3][pg, :, off] = p.data[3][pg, :, off] - 121 + byte
    out = p.run()[0].double().cpu()
    for b in range(4):
        c = int(p.ctx[b])
        s = np.arange(c + T)
        pg, off = p.table[b, s // 32], s % 32
        see = np.concatenate([np.ones((T, c), bool), p.see[b]], 1)
        for h in range(Hq):
            k, v = (ref.decode(p.data[j][pg, h * Hkv // Hq, off], p.data[j + 1][pg, h * Hkv // Hq, off]) for j in (0, 2))
            want, _, mass, reach = ref.attention(p.q[b, :, h].double(), k, v, see, D ** -0.5)
            tol = want.abs() * 2.0 ** -8 + mass * (2.0 ** -9 + 2.0 ** -11 + 2.0 ** -14 + 2.0 ** -15 * reach[:, None])
            tol = tol + (c + T) * 2.0 ** -40 * np.abs(v).max() + 2.0 ** -134
            assert torch.all((out[b, :, h] - want).abs() <= tol), (b, h, float(((out[b, :, h] - want).abs() / tol).max()))
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("byte", [0, 3, 121])
@pytest.mark.parametrize("Hq,D", [(4, 128), (40, 128), (4, 64)])
def test_long_segments_in_one_block(bsf8_lib, Hq, D, byte):
    """More requests than blocks, each of 131072 tokens (the table names two pages over and over, so that every key counts
    512 times): a softmax's sum of 2^17 and values down to 2^-127 of a code, in one block's registers."""
    B, page, ctx = 200, 128, 131072
    p = Problem(byte + Hq + D, 1, 1, Hq, 1, D, page, [2 * page - 1], mask=None, spread=0)
    p.data[3][:] = byte
    table = np.tile(p.table[0, :2], ctx // page // 2 + 1)[None].repeat(B, 0)
    q = p.q.cuda().expand(B, 1, Hq, D).contiguous()
    out = bsf8.tree_attention(q, p.cache(), i32(table), i32([ctx - 1] * B)).double().cpu()
    s = np.arange(2 * page)
    pg, off = p.table[0, s // page], s % page
    k, v = (ref.decode(p.data[j][pg, 0, off], p.data[j + 1][pg, 0, off]) for j in (0, 2))
    want, _, mass, reach = ref.attention(p.q[0, 0].double(), k, v, np.ones((Hq, 2 * page), bool), D ** -0.5)
    # 2^12 steps of 32 keys, each sum off by at most 2^-23 of itself
    tol = want.abs() * 2.0 ** -8 + mass * (2.0 ** -9 + 2.0 ** -11 + 2.0 ** -11 + 2.0 ** -15 * reach[:, None]) + 2.0 ** -134
    assert torch.all((out[:, 0] - want).abs() <= tol), float(((out[:, 0] - want).abs() / tol).max())
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("extra", [0, 300])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(4, 4, 2, 128), (8, 1, 1, 128), (5, 2, 2, 64), (4, 8, 1, 256), (40, 8, 2, 128)])
def test_values_of_any_range(bsf8_lib, T, Hq, Hkv, D, extra):
    """Value exponents spread over 2^34, and one node's 2^12 above all others: each value is held to 2^-24 of the largest
    one of its request and head, whether a row sees that or not, and its product with p to 2^-35 of it a key."""
    p = Problem(3 * D + T, 3, T, Hq, Hkv, D, 16, [500, 33, 0], extra=extra)
    p.see[:, T - 1, :] = False
    p.see[:, T - 1, T - 1] = True   # one row sees that node alone, no other row sees it
    p.see[:, :T - 1, T - 1] = False
    p.mask = ref.mask_words(p.see)
    for b in range(3):
        c = int(p.ctx[b])
        s = np.arange(c + T)
        pg, off = p.table[b, s // 16], s % 16
        p.data[3][pg, :, off] = p.r.integers(80, 115, size=(c + T, Hkv, D // 32))
        p.data[3][pg[-1], :, off[-1]] = 126
    out = p.run()[0].double().cpu()
    for b in range(3):
        c = int(p.ctx[b])
        s = np.arange(c + T)
        pg, off = p.table[b, s // 16], s % 16
        see = np.concatenate([np.ones((T, c), bool), p.see[b]], 1)
        for h in range(Hq):
            k, v = (ref.decode(p.data[j][pg, h * Hkv // Hq, off], p.data[j + 1][pg, h * Hkv // Hq, off]) for j in (0, 2))
            want, _, mass, reach = ref.attention(p.q[b, :, h].double(), k, v, see, D ** -0.5)
            tol = want.abs() * 2.0 ** -8 + mass * (2.0 ** -9 + 2.0 ** -11 + 2.0 ** -14 + 2.0 ** -15 * reach[:, None])
            tol = tol + np.abs(v).max() * (2.0 ** -24 + (c + T) * 2.0 ** -35)
            assert torch.all((out[b, :, h] - want).abs() <= tol), (b, h, float(((out[b, :, h] - want).abs() / tol).max()))
    assert bsf8.device_status() == 0
