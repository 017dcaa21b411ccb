"""GPU: the paged cache -- append (norm, rotation, quantisation), read back, commit -- against
plain 64-bit implementations."""
import numpy as np
import pytest
import torch

import _decode_ref as ref
import block_scaled_fp8_weight_gb300 as bsf8

pytestmark = pytest.mark.gpu


def bf16(r, *shape, scale=1.0):
    return torch.from_numpy((r.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def make_cache(r, pages, heads, dim, page_size):
    """A cache full of arbitrary bytes (NaN codes and byte 255 among them)."""
    b = lambda *s: torch.from_numpy(r.integers(0, 256, size=s, dtype=np.uint8)).cuda()  # noqa: E731
    return bsf8.KVCache(b(pages, heads, page_size, dim), b(pages, heads, page_size, dim // 32),
                        b(pages, heads, page_size, dim), b(pages, heads, page_size, dim // 32))


def arrays(cache):
    return [t.cpu().numpy().copy() for t in (cache.k8, cache.kexp, cache.v8, cache.vexp)]


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def place(table, req, slot, page_size):
    table = table.cpu().numpy()
    return table[req, slot // page_size], slot % page_size


@pytest.mark.parametrize("D,Hq,Hkv,page,N", [(64, 3, 1, 16, 1), (128, 8, 2, 48, 37), (256, 5, 5, 64, 130),
                                             (128, 32, 8, 16, 700), (64, 14, 2, 32, 2500)])
def test_append_without_norm_or_rotation_is_bit_exact(bsf8_lib, D, Hq, Hkv, page, N):
    """Values and unrotated keys: codes and exponents are those of the definition, bit for bit;
    queries pass unchanged; nothing else in the cache moves.  q, k, v are views of one tensor."""
    r = np.random.default_rng(D + N)
    B = 3
    per = -(-N // B)
    tp = -(-(per + 5) // page)
    cache = make_cache(r, B * tp + 2, Hkv, D, page)
    before = arrays(cache)
    table = i32(r.permutation(B * tp + 2)[:B * tp].reshape(B, tp))
    x = bf16(r, N, (Hq + 2 * Hkv) * D + 8)
    mag = torch.from_numpy(2.0 ** r.integers(-20, 20, size=(N, x.shape[1])).astype(np.float32))
    x = (x.float() * mag).to(torch.bfloat16)
    x[0, Hq * D:Hq * D + 32] = 0  # a block of zeros
    xd = x.cuda()
    cut = lambda a, h: xd[:, a:a + h * D].unflatten(1, (h, D))  # noqa: E731
    q, k, v = cut(0, Hq), cut(Hq * D, Hkv), cut((Hq + Hkv) * D, Hkv)
    req = np.arange(N) % B
    slot = np.arange(N) // B + 2
    out = bsf8.qkv_append(q, k, v, cache, table, i32(req), i32(slot))
    assert torch.equal(out.view(torch.int16), q.contiguous().view(torch.int16))
    pg, off = place(table, req, slot, page)
    want = before
    few = np.unique(np.concatenate([np.arange(min(N, 40)), np.arange(N)[-40:]]))
    got = arrays(cache)
    for j, t in ((0, k), (2, v)):
        rows = t.float().cpu().numpy().astype(np.float64)
        c, e = ref.quantise(rows[few])
        assert np.array_equal(got[j][pg[few], :, off[few]], c)
        assert np.array_equal(got[j + 1][pg[few], :, off[few]], e)
        # all of them: half a step of e4m3 at the block's scale (normal: 2^-4 of the value;
        # subnormal: half of 2^-9), and the scale no larger than it has to be
        val = ref.decode(got[j][pg, :, off], got[j + 1][pg, :, off])
        amax = np.abs(rows.reshape(N, Hkv, -1, 32)).max(-1)
        sc = 2.0 ** (got[j + 1][pg, :, off].astype(np.float64) - 127)
        assert np.all(448 * sc >= amax) and np.all((224 * sc < amax) | (got[j + 1][pg, :, off] == 0))
        assert np.all(np.abs(val - rows) <= np.maximum(np.abs(rows) / 16, np.repeat(sc, 32, -1) * 2.0 ** -10))
        for w in (j, j + 1):
            want[w][pg, :, off] = got[w][pg, :, off]
    for a, b in zip(want, got):
        assert np.array_equal(a, b)  # every other row is as it was
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("D,Hq,Hkv,rot,inter,norm", [
    (128, 4, 2, 128, False, True), (128, 4, 2, 128, True, True), (64, 3, 1, 32, False, True),
    (64, 2, 2, 16, True, False), (256, 5, 1, 64, False, True), (256, 2, 2, 256, False, False),
    (128, 7, 3, 0, False, True), (256, 3, 1, 256, True, True)])
@pytest.mark.parametrize("N", [1, 45, 1300])
def test_append_norm_and_rotation(bsf8_lib, D, Hq, Hkv, rot, inter, norm, N):
    """Queries within one bf16 rounding of the 64-bit result (half a step, 2^-9 of the value, plus
    fp32 arithmetic: 2^-17 of the row's largest); keys within one e4m3 rounding of it."""
    r = np.random.default_rng(rot + N)
    page, P = 32, 300
    q, k, v = bf16(r, N, Hq, D, scale=3.0).cuda(), bf16(r, N, Hkv, D).cuda(), bf16(r, N, Hkv, D).cuda()
    cache = make_cache(r, -(-N // page), Hkv, D, page)
    table = i32(r.permutation(-(-N // page))[None])
    qn, kn = (1 + 0.3 * bf16(r, D).float()).to(torch.bfloat16).cuda(), (1 + 0.3 * bf16(r, D).float()).to(torch.bfloat16).cuda()
    pos = r.integers(0, P, size=N)
    cs = None
    if rot:
        ang = np.arange(P)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
        cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    out = bsf8.qkv_append(q, k, v, cache, table, i32(np.zeros(N)), i32(np.arange(N)), pos=i32(pos) if rot else None,
                          cos_sin=None if cs is None else torch.from_numpy(cs).cuda(), q_norm=qn if norm else None,
                          k_norm=kn if norm else None, eps=1e-5, interleaved=inter)
    f64 = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    wq = ref.norm_rotate(f64(q), f64(qn) if norm else None, cs, pos, inter, 1e-5)
    wk = ref.norm_rotate(f64(k), f64(kn) if norm else None, cs, pos, inter, 1e-5)
    top = np.abs(wq).max(-1, keepdims=True)
    assert np.all(np.abs(f64(out) - wq) <= np.abs(wq) * 2.0 ** -8 + top * 2.0 ** -17)
    pg, off = place(table, np.zeros(N, int), np.arange(N), page)
    c8, ce, w8, we = arrays(cache)
    got, e = ref.decode(c8[pg, :, off], ce[pg, :, off]), ce[pg, :, off]
    sc = np.repeat(2.0 ** (e.astype(np.float64) - 127), 32, -1)
    top = np.abs(wk).max(-1, keepdims=True)
    assert np.all(np.abs(got - wk) <= np.maximum(np.abs(wk) / 16, sc * 2.0 ** -10) * (1 + 2.0 ** -10) + top * 2.0 ** -17)
    amax = np.abs(wk.reshape(N, Hkv, -1, 32)).max(-1)
    s2 = 2.0 ** (e.astype(np.float64) - 127)
    assert np.all(448 * s2 >= amax * (1 - 2.0 ** -17)) and np.all(224 * s2 < amax * (1 + 2.0 ** -17))
    # values are neither normed nor rotated
    val = ref.decode(w8[pg, :, off], we[pg, :, off])
    sv = np.repeat(2.0 ** (we[pg, :, off].astype(np.float64) - 127), 32, -1)
    assert np.all(np.abs(val - f64(v)) <= np.maximum(np.abs(f64(v)) / 16, sv * 2.0 ** -10))
    assert bsf8.device_status() == 0


def test_append_special_values(bsf8_lib):
    """Infinities and NaN make their 32-channel block NaN and no other; zeros keep their sign; the
    largest and the smallest bf16 magnitudes; rows of zeros through the norm."""
    r = np.random.default_rng(5)
    D, page, N = 128, 16, 6
    k, v = bf16(r, N, 1, D), bf16(r, N, 1, D)
    v[0, 0, 40] = float("inf")
    v[1, 0, 100] = float("nan")
    v[2, 0, :32] = 0.0
    v[2, 0, 5] = -0.0
    v[3, 0, 32:64] = torch.tensor(0x7F7F, dtype=torch.int16).view(torch.bfloat16)   # the largest
    v[4, 0, 64:96] = torch.tensor(0x0001, dtype=torch.int16).view(torch.bfloat16)   # the smallest
    k[5] = 0
    cache = make_cache(r, 1, 1, D, page)
    table = i32([[0]])
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    bsf8.qkv_append(None, k.cuda(), v.cuda(), cache, table, i32([0] * N), i32(range(N)), k_norm=w)
    c8, ce, w8, we = arrays(cache)
    c, e = ref.quantise(v.float().numpy().astype(np.float64))
    assert np.array_equal(w8[0, :, :N].transpose(1, 0, 2), c) and np.array_equal(we[0, :, :N].transpose(1, 0, 2), e)
    assert list(we[0, 0, 0]).count(255) == 1 and we[0, 0, 1, 3] == 255
    assert not c8[0, 0, 5].any()
    ko, vo = bsf8.kv_read(cache, table, i32([0] * N), i32(range(N)))
    nan = torch.isnan(vo.cpu()[:, 0])
    want = torch.zeros(N, D, dtype=torch.bool)
    want[0, 32:64] = True
    want[1, 96:] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("D,Hkv,page,N", [(64, 1, 16, 1), (128, 3, 48, 333), (256, 2, 1024, 77), (128, 8, 16, 3001)])
def test_read_is_bit_exact(bsf8_lib, D, Hkv, page, N):
    """Every byte pair: bf16(code * 2^(byte - 127)); k or v alone gives the same rows."""
    r = np.random.default_rng(N)
    pages = 9
    cache = make_cache(r, pages, Hkv, D, page)
    table = i32(r.integers(0, pages, size=(4, 3)))
    req, slot = r.integers(0, 4, size=N), r.integers(0, 3 * page, size=N)
    slot[::17] = -1
    k, v = bsf8.kv_read(cache, table, i32(req), i32(slot))
    pg, off = place(table, req, np.maximum(slot, 0), page)
    data = arrays(cache)
    for got, j in ((k, 0), (v, 2)):
        want = ref.decode(data[j][pg, :, off], data[j + 1][pg, :, off])
        want[slot < 0] = 0
        with np.errstate(over="ignore"):
            want = torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16)
        g = got.cpu()
        assert torch.equal(torch.isnan(g), torch.isnan(want))
        assert torch.equal(g.nan_to_num(0), want.nan_to_num(0))
    lib, st = bsf8.load(), cache._struct()
    import ctypes
    only = torch.empty_like(k)
    for args, whole in (((only.data_ptr(), None), k), ((None, only.data_ptr()), v)):
        only.zero_()
        assert lib.bsf8_kv_read(ctypes.byref(st), table.data_ptr(), 4, 3, i32(req).data_ptr(), i32(slot).data_ptr(),
                                *args, N, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(only.view(torch.int16), whole.view(torch.int16))
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("D,Hkv,page,B,T", [(64, 1, 16, 1, 1), (128, 8, 16, 5, 8), (256, 3, 48, 3, 33), (64, 2, 64, 40, 256)])
def test_commit_moves_the_kept_nodes(bsf8_lib, D, Hkv, page, B, T):
    r = np.random.default_rng(T)
    ctx = r.integers(0, 70, size=B)
    tp = -(-(70 + T) // page)
    cache = make_cache(r, B * tp, Hkv, D, page)
    table = i32(r.permutation(B * tp).reshape(B, tp))
    path, count = np.full((B, T), -1), np.zeros(B, int)
    for b in range(B):
        n = int(r.integers(0, T)) if b else T - 1  # the first keeps all but one
        way = [0] + sorted(r.choice(np.arange(1, T), n, replace=False).tolist()) if T > 1 else [0]
        path[b, :len(way)], count[b] = way, len(way)
    want = arrays(cache)
    old = [t.copy() for t in want]
    for b in range(B):
        for i in range(count[b]):
            a, z = ctx[b] + path[b, i], ctx[b] + i
            pa, pz = int(table[b, a // page]), int(table[b, z // page])
            for o, w in zip(old, want):
                w[pz, :, z % page] = o[pa, :, a % page]
    bsf8.kv_commit(cache, table, i32(ctx), i32(path), i32(count))
    for a, b in zip(want, arrays(cache)):
        assert np.array_equal(a, b)
    assert bsf8.device_status() == 0


def test_bad_indices_are_skipped_and_reported(bsf8_lib):
    """Requests, slots, pages and positions outside their tables: the row is skipped, the status word
    says so, and every other row is right."""
    r = np.random.default_rng(9)
    D, page, N = 64, 16, 8
    cache = make_cache(r, 4, 1, D, page)
    before = arrays(cache)
    table = i32([[0, 1], [2, 99]])
    k, v, q = (bf16(r, N, 1, D).cuda() for _ in range(3))
    req = [0, 5, 0, 1, 1, -1, 0, 0]
    slot = [3, 3, 32, 16, 5, 1, -1, 7]
    pos = [0, 0, 0, 0, 0, 0, 0, 50]
    cs = torch.zeros(10, 16, device="cuda")
    cs[:, :8] = 1
    out = torch.full((N, 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    bsf8.qkv_append(q, k, v, cache, table, i32(req), i32(slot), pos=i32(pos), cos_sin=cs, out=out)
    assert bsf8.device_status() == 10 and bsf8.device_status() == 0
    assert torch.equal(out[:7], q[:7]) and torch.all(out[7] == 7)  # a bad position leaves the token out
    got = arrays(cache)
    for j, t in ((0, k), (2, v)):
        c, e = ref.quantise(t.float().cpu().numpy().astype(np.float64))
        before[j][0, :, 3], before[j + 1][0, :, 3] = c[0], e[0]
        before[j][2, :, 5], before[j + 1][2, :, 5] = c[4], e[4]
    for a, b in zip(before, got):
        assert np.array_equal(a, b)
    ko, vo = bsf8.kv_read(cache, table, i32(req), i32(slot))
    assert bsf8.device_status() == 10
    for n in (1, 2, 3, 5, 6):
        assert not ko[n].any() and not vo[n].any()
    assert torch.equal(torch.isnan(ko[0]), torch.isnan(ko[0])) and ko[4].any()
    bsf8.kv_commit(cache, table, i32([0, 14]), i32([[0, 3], [0, 2]]), i32([2, 2]))  # slot 16 of request 1: page 99
    assert bsf8.device_status() == 10
    before[0][0, :, 1], before[1][0, :, 1], before[2][0, :, 1], before[3][0, :, 1] = (
        before[0][0, :, 3], before[1][0, :, 3], before[2][0, :, 3], before[3][0, :, 3])
    for a, b in zip(before, arrays(cache)):
        assert np.array_equal(a, b)


def test_empty_calls_and_side_stream(bsf8_lib):
    r = np.random.default_rng(1)
    cache = make_cache(r, 2, 2, 64, 16)
    before = arrays(cache)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    z = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    table = i32([[0, 1]])
    assert bsf8.qkv_append(z, z, z, cache, table, none, none).shape == (0, 2, 64)
    k, v = bsf8.kv_read(cache, table, none, none)
    assert k.shape == v.shape == (0, 2, 64)
    x = bf16(r, 20, 2, 64).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bsf8.qkv_append(None, x, x, cache, table, i32([0] * 20), i32(range(20)))
        k, v = bsf8.kv_read(cache, table, i32([0] * 20), i32(range(20)))
    side.synchronize()
    assert torch.equal(k.view(torch.int16), v.view(torch.int16))
    c, e = ref.quantise(x.float().cpu().numpy().astype(np.float64))
    assert torch.equal(k.cpu().double(), torch.from_numpy(ref.decode(c, e)))
    assert not np.array_equal(before[0], arrays(cache)[0])


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
def test_calls_run_where_the_tensors_are(bsf8_lib):
    """Tensors on a device that is not the current one: the calls run there, on its current stream, and the
    current device is as before."""
    from test_gpu_tree_attention import Problem
    p = Problem(1, 2, 3, 4, 2, 128, 16, [100, 7])
    want = p.run()
    other = torch.device("cuda", 1)
    move = lambda *t: [x.to(other) for x in t]  # noqa: E731
    c = p.cache()
    cache = bsf8.KVCache(*move(c.k8, c.kexp, c.v8, c.vexp))
    table, ctx, nodes, q, mask = move(i32(p.table), i32(p.ctx), i32(p.nodes), p.q.cuda(), torch.from_numpy(p.mask).cuda())
    assert torch.cuda.current_device() == 0
    out = bsf8.tree_attention(q, cache, table, ctx, nodes=nodes, mask=mask)
    assert torch.cuda.current_device() == 0 and out.device == other
    assert torch.equal(out.cpu().view(torch.int16), want[0].cpu().view(torch.int16))
    req, slot = torch.zeros(5, dtype=torch.int32, device=other), torch.arange(5, dtype=torch.int32, device=other)
    x = torch.randn(5, 2, 128, device=other).to(torch.bfloat16)
    bsf8.qkv_append(None, x, x, cache, table, req, slot)
    k, v = bsf8.kv_read(cache, table, req, slot)
    path = torch.tensor([[0, 2, -1]] * 2, dtype=torch.int32, device=other)
    bsf8.kv_commit(cache, table, ctx, path, torch.tensor([2, 2], dtype=torch.int32, device=other))
    prob = torch.full((2, 3, 5), 0.2, device=other)
    tree = torch.tensor([[-1, 0, 0]] * 2, dtype=torch.int32, device=other)
    count = bsf8.verify_tree(prob, tree.clamp(min=0), tree, torch.zeros(2, 3, device=other), q=prob)[1]
    assert torch.equal(k, v) and count.device == other and torch.cuda.current_device() == 0


@pytest.mark.parametrize("D,Hkv,page", [(64, 1, 16), (128, 8, 16), (256, 3, 48)])
def test_commit_of_paths_that_leave_node_0_out(bsf8_lib, D, Hkv, page):
    """Every entry moves, the first one too: paths that start past node 0, that keep all nodes, none, one."""
    r = np.random.default_rng(D)
    paths = [[1, 2], [3], [5, 6, 20], [0, 1, 2, 3], [0, 7, 8], [], list(range(1, 21)), [20]]
    B, T = len(paths), 21
    ctx = r.integers(0, 70, size=B)
    tp = -(-(70 + T) // page)
    cache = make_cache(r, B * tp, Hkv, D, page)
    table = i32(r.permutation(B * tp).reshape(B, tp))
    want = arrays(cache)
    old = [t.copy() for t in want]
    for b, way in enumerate(paths):
        for i, node in enumerate(way):
            a, z = ctx[b] + node, ctx[b] + i
            for o, w in zip(old, want):
                w[int(table[b, z // page]), :, z % page] = o[int(table[b, a // page]), :, a % page]
    bsf8.kv_commit(cache, table, i32(ctx), i32([way + [-1] * (T - len(way)) for way in paths]), i32([len(w) for w in paths]))
    for a, b in zip(want, arrays(cache)):
        assert np.array_equal(a, b)
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("path,count,moved", [
    ([1, 2, 4], 4, [(1, 0), (2, 1), (4, 2)]),     # a count above T: cut to it
    ([1, 2, 4], -1, []),                          # below 0
    ([0, 3, 3], 3, [(3, 1)]),                     # the same node twice
    ([0, 4, 2], 3, [(4, 1)]),                     # backwards
    ([-1, 1, 4], 3, [(4, 2)]),                    # no node, and the one after it in its place already
    ([0, 0, 2], 3, [])])
def test_commit_reports_bad_counts_and_paths(bsf8_lib, path, count, moved):
    """What is wrong is left out and reported; the rest moves, and so do other requests' nodes."""
    r = np.random.default_rng(3)
    D, page = 64, 16
    cache = make_cache(r, 4, 2, D, page)
    want = arrays(cache)
    old = [t.copy() for t in want]
    table, ctx = np.array([[0, 2], [3, 1]]), [13, 2]
    for b, steps in ((0, moved), (1, [(2, 1)])):
        for node, i in steps:
            a, z = ctx[b] + node, ctx[b] + i
            for o, w in zip(old, want):
                w[table[b, z // page], :, z % page] = o[table[b, a // page], :, a % page]
    bsf8.kv_commit(cache, i32(table), i32(ctx), i32([path, [0, 2, -1]]), i32([count, 2]))
    assert bsf8.device_status() == 10
    for a, b in zip(want, arrays(cache)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("D,rot", [(64, 32), (128, 64), (256, 64), (128, 0)])
@pytest.mark.parametrize("inter", [False, True])
def test_infinities_outside_the_rotation_stay(bsf8_lib, D, rot, inter):
    """Channels past `rot` are not rotated: infinities there come out of the queries as they went in; inside, a pair
    with one is what the formula gives."""
    r = np.random.default_rng(rot + D)
    N = 40
    q, k = bf16(r, N, 3, D), bf16(r, N, 1, D)
    for n in range(N):
        q[n, n % 3, rot + n % (D - rot)] = float("inf") if n % 2 else -float("inf")
    if rot:
        q[7, 0, 3] = float("inf")
    cache = make_cache(r, 4, 1, D, 16)
    pos = r.integers(1, 50, size=N)
    ang = np.arange(50)[:, None] * 10000.0 ** (-np.arange(max(rot, 2) // 2) / (max(rot, 2) // 2))
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    out = bsf8.qkv_append(q.cuda(), k.cuda(), k.cuda(), cache, i32([[0, 1, 2]]), i32([0] * N), i32(range(N)),
                          pos=i32(pos) if rot else None, cos_sin=torch.from_numpy(cs).cuda() if rot else None, interleaved=inter)
    with np.errstate(invalid="ignore"):
        want = ref.norm_rotate(q.float().numpy(), None, cs if rot else None, pos, inter, 0.0)
    got = out.float().cpu().numpy()
    assert np.array_equal(got[..., rot:], want[..., rot:])
    big = ~np.isfinite(want[..., :rot])
    assert np.array_equal(np.isnan(want[..., :rot]), np.isnan(got[..., :rot])) and np.array_equal(big, ~np.isfinite(got[..., :rot]))
    assert bsf8.device_status() == 0


def test_arguments_that_have_no_value_are_refused(bsf8_lib):
    """What Python cannot read as a truth value or a number raises its own error, and nothing is written."""
    r = np.random.default_rng(6)
    cache = make_cache(r, 1, 1, 64, 16)
    before = arrays(cache)
    x, table, at = bf16(r, 3, 1, 64).cuda(), i32([[0]]), (i32([0] * 3), i32(range(3)))
    with pytest.raises(RuntimeError, match="more than one value"):
        bsf8.qkv_append(x, x, x, cache, table, *at, interleaved=torch.zeros(2))
    with pytest.raises(TypeError, match="real number"):
        bsf8.qkv_append(x, x, x, cache, table, *at, eps="1e-6")
    with pytest.raises(TypeError):
        bsf8.tree_attention(x.view(1, 3, 1, 64), cache, table, i32([0]), max_len=1.5)
    with pytest.raises(TypeError, match="real number"):
        bsf8.tree_attention(x.view(1, 3, 1, 64), cache, table, i32([0]), scale="0.1")
    torch.cuda.synchronize()
    for a, b in zip(before, arrays(cache)):
        assert np.array_equal(a, b)


def test_outputs_that_do_not_fit_raise_torchs_own_error(bsf8_lib):
    r = np.random.default_rng(7)
    cache = make_cache(r, 1, 8, 256, 16)
    n = torch.cuda.get_device_properties(0).total_memory // (8 * 256 * 2) + 1  # tokens: keys alone are more than the card
    at = torch.zeros(n, dtype=torch.int32, device="cuda")
    with pytest.raises(torch.cuda.OutOfMemoryError):
        bsf8.kv_read(cache, i32([[0]]), at, at)
    del at
    k, v = bsf8.kv_read(cache, i32([[0]]), i32([0]), i32([3]))
    assert k.shape == (1, 8, 256) and bsf8.device_status() == 0
