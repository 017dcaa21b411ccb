"""GPU: what the attention kernels' own structure can get wrong: few rows of a request and head, many
short requests in one block's share, the same call again and again with no pause, waits that run out.
Formula and tolerances are those of the other attention tests; the kernel for up to 8 rows at dim 128
rounds p to 11 bits as well, above 2^-31 of its reference."""
import numpy as np
import pytest
import torch

import _decode_ref as ref
import block_scaled_fp8_weight_gb300 as bsf8
from test_gpu_tree_attention import Problem, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 48, 128])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 3, 3), (2, 8, 2), (8, 1, 1), (5, 3, 1), (3, 10, 2), (16, 1, 1), (4, 4, 1)])
def test_few_rows(bsf8_lib, T, Hq, Hkv, page):
    """Contexts from none to several tiles, trees and masks that leave rows empty, requests without nodes."""
    ctx = [0, 1, 15, 16, 127, 128, 129, 255, 700, 1500]
    nodes = [max(0, T - i % 3) for i in range(len(ctx))]
    for mask in ("tree", "random", None):
        p = Problem(7 * T + page, len(ctx), T, Hq, Hkv, 128, page, ctx, nodes=nodes, mask=mask, spread=5)
        if mask == "random":
            p.see[:, 0] = False
            p.mask = ref.mask_words(p.see)
        p.check(*p.run())
    assert bsf8.device_status() == 0


def test_few_rows_nan_in_values_and_a_bad_page(bsf8_lib):
    """NaN value blocks and a page outside the cache amid a long context: the other heads, requests and
    channel blocks are untouched."""
    p = Problem(3, 3, 2, 4, 2, 128, 32, [1000, 300, 5])
    good, _ = p.run()
    pg, off = p.table[0, 500 // 32], 500 % 32
    p.data[2][pg, 1, off, 64:96], p.data[3][pg, 1, off, 2] = 0x7F, 255
    out, lse = p.run()
    p.check(out, lse)
    assert torch.isnan(out[0, :, 2:, 64:96]).all() and torch.equal(out[0, :, :2], good[0, :, :2])
    assert torch.equal(out[0, :, 2:, :64], good[0, :, 2:, :64]) and torch.equal(out[1:], good[1:])
    assert bsf8.device_status() == 0
    p.table[0, 500 // 32] = 1 << 29
    out, _ = p.run()
    assert bsf8.device_status() == 10
    assert torch.isfinite(out).all() and torch.equal(out[1:], good[1:])


@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 4, 4, 128), (4, 4, 1, 128), (1, 4, 2, 64), (9, 8, 1, 128), (20, 8, 1, 256)])
def test_many_short_requests(bsf8_lib, T, Hq, Hkv, D):
    """More requests than blocks, a few long ones among them: shares of many segments, some of one tile."""
    r = np.random.default_rng(D + T)
    B = 400
    ctx = r.integers(0, 200, size=B)
    ctx[[5, 250]] = 3000
    nodes = r.integers(0, T + 1, size=B)
    p = Problem(D + 2 * T, B, T, Hq, Hkv, D, 16, ctx, nodes=nodes)
    p.check(*p.run())
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 8, 2, 128), (4, 8, 2, 128), (1, 8, 2, 64), (16, 8, 2, 128), (33, 8, 1, 128),
                                        (2, 8, 2, 256)])
def test_same_bits_again_and_again(bsf8_lib, T, Hq, Hkv, D):
    """Calls back to back (each starts while the one before ends): every one the same bits."""
    r = np.random.default_rng(T + D)
    p = Problem(5 * T + D, 24, T, Hq, Hkv, D, 32, r.integers(0, 2500, size=24), nodes=r.integers(1, T + 1, size=24))
    cache, table, ctx, nodes = p.cache(), i32(p.table), i32(p.ctx), i32(p.nodes)
    q, mask = p.q.cuda(), torch.from_numpy(p.mask).cuda()
    out = torch.empty(20, *q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(20, *q.shape[:3], device="cuda")
    call = lambda i: bsf8.tree_attention(q, cache, table, ctx, nodes=nodes, mask=mask, out=out[i], lse=lse[i])  # noqa: E731
    call(0)
    torch.cuda.synchronize()
    p.check(out[0], lse[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(1, 20):
            call(i)
    for _ in range(5):
        out[1:] = 0
        graph.replay()
        torch.cuda.synchronize()
        assert bsf8.device_status() == 0
        assert torch.equal(out[1:].view(torch.int16), out[:1].expand(19, -1, -1, -1, -1).contiguous().view(torch.int16))
        assert torch.equal(lse[1:], lse[:1].expand(19, -1, -1, -1).contiguous())


@pytest.mark.parametrize("T,D", [(1, 128), (4, 128), (1, 64), (40, 128), (3, 256)])
def test_timeout_is_reported_without_hanging(bsf8_lib, T, D):
    """With the test-only option that suppresses loads every wait of the kernel runs out after the shortened
    bound; it returns and the status says so.  The next call is right again."""
    p = Problem(T + D, 2, T, 4, 1, D, 16, [300, 40])
    assert bsf8.device_status() == 0
    old = bsf8.get_option(bsf8.OPT_WAIT_TIMEOUT_NS)
    try:
        bsf8.set_option(bsf8.OPT_WAIT_TIMEOUT_NS, 2_000_000)     # 2 ms
        bsf8.set_option(bsf8.OPT_DEBUG_SKIP_LOADS, 1)
        p.run()
        assert bsf8.device_status() == 7
    finally:
        bsf8.set_option(bsf8.OPT_DEBUG_SKIP_LOADS, 0)
        bsf8.set_option(bsf8.OPT_WAIT_TIMEOUT_NS, old)
    p.check(*p.run())
    assert bsf8.device_status() == 0


# ---- up to 8 rows where requests may be longer than 2048 tokens (`extra`: room in the table): keys and
# channels fill the matrix instruction there, at dim 128

@pytest.mark.parametrize("page", [16, 48, 128])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 3, 3), (2, 8, 2), (8, 1, 1), (4, 2, 1), (3, 4, 2), (1, 8, 1), (7, 1, 1)])
def test_few_rows_in_a_long_table(bsf8_lib, T, Hq, Hkv, page):
    """Contexts from none to many tiles, trees and masks that leave rows empty, requests without nodes."""
    ctx = [0, 1, 15, 16, 127, 128, 129, 255, 700, 3100]
    nodes = [max(0, T - i % 3) for i in range(len(ctx))]
    for mask in ("tree", "random", None):
        p = Problem(11 * T + page, len(ctx), T, Hq, Hkv, 128, page, ctx, nodes=nodes, mask=mask, spread=5)
        if mask == "random":
            p.see[:, 0] = False
            p.mask = ref.mask_words(p.see)
        p.check(*p.run())
    assert bsf8.device_status() == 0


def test_few_rows_nan_and_bad_pages_in_a_long_table(bsf8_lib):
    p = Problem(4, 3, 2, 4, 2, 128, 32, [1000, 300, 5], extra=70)
    good, _ = p.run()
    pg, off = p.table[0, 500 // 32], 500 % 32
    p.data[2][pg, 1, off, 64:96], p.data[3][pg, 1, off, 2] = 0x7F, 255     # a value block
    node = int(p.ctx[1]) + 1
    pk, ok = p.table[1, node // 32], node % 32
    p.data[0][pk, 0, ok, 0:32], p.data[1][pk, 0, ok, 0] = 0x7F, 255        # a node's key block
    out, lse = p.run()
    p.check(out, lse)
    assert torch.isnan(out[0, :, 2:, 64:96]).all() and torch.equal(out[0, :, :2], good[0, :, :2])
    assert torch.equal(out[0, :, 2:, :64], good[0, :, 2:, :64]) and torch.equal(out[2], good[2])
    assert torch.equal(out[1, 0, :2].isnan().any(), torch.tensor(bool(p.see[1, 0, 1]), device="cuda"))
    assert torch.isnan(out[1, 1, :2]).all() and not torch.isnan(out[1, :, 2:]).any()
    assert bsf8.device_status() == 0
    p.table[0, 500 // 32] = 1 << 29
    out, _ = p.run()
    assert bsf8.device_status() == 10
    assert torch.isfinite(out[0]).all() and torch.equal(out[2], good[2])


def test_few_rows_wide_ranges_in_a_long_table(bsf8_lib):
    for seed, kw, scale in ((1, dict(spread=14), None), (2, dict(qscale=40.0), 1.0), (3, dict(qscale=1e-3), 1e-3),
                            (4, dict(qscale=0.0), None)):
        p = Problem(seed, 3, 2, 8, 2, 128, 32, [500, 33, 0], extra=70, **kw)
        p.check(*p.run(scale=scale), scale=scale)
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 4, 4), (4, 2, 1), (1, 8, 1)])
def test_many_requests_in_a_long_table(bsf8_lib, T, Hq, Hkv):
    """More requests than blocks, a few long ones among them, calls back to back: shares of many segments,
    some of one tile; every call the same bits."""
    r = np.random.default_rng(Hq)
    B = 400
    ctx = r.integers(0, 200, size=B)
    ctx[[5, 250]] = 5000
    nodes = r.integers(0, T + 1, size=B)
    p = Problem(3 * T + Hq, B, T, Hq, Hkv, 128, 16, ctx, nodes=nodes)
    cache, table, c, n = p.cache(), i32(p.table), i32(p.ctx), i32(p.nodes)
    q, mask = p.q.cuda(), torch.from_numpy(p.mask).cuda()
    out = torch.empty(12, *q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(12, *q.shape[:3], device="cuda")
    call = lambda i: bsf8.tree_attention(q, cache, table, c, nodes=n, mask=mask, out=out[i], lse=lse[i])  # noqa: E731
    call(0)
    torch.cuda.synchronize()
    p.check(out[0], lse[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(1, 12):
            call(i)
    for _ in range(5):
        out[1:] = 0
        graph.replay()
        torch.cuda.synchronize()
        assert bsf8.device_status() == 0
        assert torch.equal(out[1:].view(torch.int16), out[:1].expand(11, -1, -1, -1, -1).contiguous().view(torch.int16))


def test_few_rows_timeout_in_a_long_table(bsf8_lib):
    p = Problem(9, 2, 1, 4, 1, 128, 16, [3000, 40])
    old = bsf8.get_option(bsf8.OPT_WAIT_TIMEOUT_NS)
    try:
        bsf8.set_option(bsf8.OPT_WAIT_TIMEOUT_NS, 2_000_000)     # 2 ms
        bsf8.set_option(bsf8.OPT_DEBUG_SKIP_LOADS, 1)
        p.run()
        assert bsf8.device_status() == 7
    finally:
        bsf8.set_option(bsf8.OPT_DEBUG_SKIP_LOADS, 0)
        bsf8.set_option(bsf8.OPT_WAIT_TIMEOUT_NS, old)
    p.check(*p.run())
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("T,Hq,D", [(3, 4, 128), (16, 4, 128), (30, 4, 128), (9, 4, 64), (33, 4, 64), (9, 4, 256), (40, 4, 256)])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4])
def test_the_last_tiles_value_exponent(bsf8_lib, T, Hq, D, tiles):
    """Shares of 1 to 4 tiles a block, each tile with a value exponent of its own, so that a block's last tile
    has another largest exponent than those before it: the outputs are scaled by the last one's.  The same
    call again and again gives the same bits."""
    keys = 64 if D == 256 else 128
    p = Problem(tiles + T + D, 1, T, Hq, 1, D, 128, [152 * tiles * keys - T - 5], spread=0)
    s = np.arange(int(p.ctx[0]) + T)
    steps = np.arange(len(s) // keys + 1) * 5 % 16
    p.data[3][p.table[0, s // 128], 0, s % 128] = (106 + steps[s // keys])[:, None]
    cache, args = p.cache(), (i32(p.table), i32(p.ctx))
    q, mask = p.q.cuda(), torch.from_numpy(p.mask).cuda()
    p.check(*p.run(cache=cache))
    out = torch.empty(10, *q.shape, dtype=torch.bfloat16, device="cuda")
    for i in range(10):
        bsf8.tree_attention(q, cache, *args, mask=mask, out=out[i])
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), out[:1].expand_as(out).contiguous().view(torch.int16))
    assert bsf8.device_status() == 0
