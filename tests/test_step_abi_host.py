"""Host-side refusals of the operators around a decode step: each invalid argument gives its documented status before
any CUDA call (fake device addresses are only ever paired with an invalid argument)."""
import ctypes

import pytest

import block_scaled_fp8_weight_gb300 as bsf8
from block_scaled_fp8_weight_gb300 import build as bsf8_build
from block_scaled_fp8_weight_gb300.decode import _CacheStruct

OK, SHAPE, ALIGN, STRIDE, WORKSPACE, NULL, CUDA, TIMEOUT, DEVICE, VALUE, INDEX = range(11)
A = 0x10000  # a 16-byte aligned fake device address
NAN, INF = float("nan"), float("inf")


class Bounds(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("exps", ctypes.c_void_p), ("pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("heads", ctypes.c_int), ("dim", ctypes.c_int)]


@pytest.fixture(scope="module")
def lib():
    bsf8_build.build()
    return bsf8.load()


def cache(**kw):
    d = dict(k8=A, kexp=A, v8=A, vexp=A, pages=8, page_size=16, heads=2, dim=128)
    d.update(kw)
    return ctypes.byref(_CacheStruct(**d))


def bounds(**kw):
    d = dict(codes=A, exps=A, pages=8, page_size=16, heads=2, dim=128)
    d.update(kw)
    return ctypes.byref(Bounds(**d))


BAD_BOUNDS = [(dict(codes=0), NULL), (dict(exps=0), NULL), (dict(pages=0), SHAPE), (dict(page_size=8), SHAPE),
              (dict(page_size=40), SHAPE), (dict(page_size=2048), SHAPE), (dict(heads=0), SHAPE), (dict(dim=96), SHAPE),
              (dict(codes=A + 8), ALIGN), (dict(exps=A + 2), ALIGN), (dict(exps=A + 4, dim=256), ALIGN), (dict(pages=1 << 30, heads=2), SHAPE)]


def test_plan_refusals(lib):
    def f(**kw):
        d = dict(table=A, table_pages=4, page_size=16, held=A, free=A, count=A, pool=8, lens=A, add=A, done=A, req=A, slot=A,
                 start=A, granted=A, B=3, N=5)
        d.update(kw)
        return lib.bsf8_kv_plan(*d.values(), None)
    for name in ("table", "held", "free", "count", "lens", "add", "req", "slot", "start", "granted"):
        assert f(**{name: 0}) == NULL, name
        assert f(**{name: A + 2}) == ALIGN, name
    assert f(done=A + 2) == ALIGN
    for kw in (dict(B=0), dict(B=1025), dict(N=-1), dict(N=(1 << 30) + 1), dict(pool=0), dict(table_pages=0), dict(page_size=8),
               dict(page_size=24), dict(page_size=2048), dict(table_pages=1 << 27), dict(table_pages=1 << 21, B=1024)):
        assert f(**kw) == SHAPE, kw


def test_bounds_refusals(lib):
    f = lambda c=None, v=None, table=A, tp=4, start=A, end=A, B=2: lib.bsf8_kv_bounds(  # noqa: E731
        c or cache(), v or bounds(), table, tp, start, end, B, None)
    for bad, status in BAD_BOUNDS:
        assert f(v=bounds(**bad)) == status, bad
    for bad in (dict(pages=9), dict(page_size=32), dict(heads=1), dict(dim=64)):
        assert f(v=bounds(**bad)) == SHAPE, bad
    assert f(cache(dim=96)) == SHAPE and f(cache(k8=0)) == NULL and f(cache(kexp=A + 4)) == ALIGN
    assert f(table=0) == NULL and f(end=0) == NULL and f(B=0) == SHAPE and f(B=1025) == SHAPE and f(tp=0) == SHAPE
    assert f(start=A + 1) == ALIGN and f(end=A + 2) == ALIGN and f(B=1024, tp=1 << 21) == SHAPE


def select(lib, v=None, **kw):
    d = dict(q=A, ldq=512, table=A, table_pages=4, ctx=A, nodes=A, max_len=64, keep=3, sink=1, recent=2, pages=A, kept=A, B=2,
             T=3, Hq=4)
    d.update(kw)
    return lib.bsf8_select_pages(d["q"], d["ldq"], v or bounds(), d["table"], d["table_pages"], d["ctx"], d["nodes"],
                                 d["max_len"], d["keep"], d["sink"], d["recent"], d["pages"], d["kept"], d["B"], d["T"],
                                 d["Hq"], None)


def test_select_refusals(lib):
    for bad, status in BAD_BOUNDS:
        assert select(lib, bounds(**bad)) == status, bad
    for name in ("q", "table", "ctx", "pages", "kept"):
        assert select(lib, **{name: 0}) == NULL, name
    for kw in (dict(B=0), dict(B=1025), dict(T=0), dict(T=257), dict(Hq=0), dict(Hq=3), dict(max_len=0), dict(max_len=65),
               dict(table_pages=0), dict(keep=0), dict(keep=49153), dict(T=256, Hq=34, ldq=34 * 128),
               dict(table_pages=49154, max_len=49153 * 16)):
        assert select(lib, **kw) == SHAPE, kw
    for kw in (dict(sink=-1), dict(recent=-1), dict(sink=2, recent=2), dict(sink=4), dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1)):
        assert select(lib, **kw) == VALUE, kw
    assert select(lib, ldq=504) == STRIDE and select(lib, ldq=516) == ALIGN
    for name in ("q", "table", "ctx", "nodes", "pages", "kept"):
        assert select(lib, **{name: A + 2}) == ALIGN, name


def test_select_width(lib):
    f = lib.bsf8_select_width
    for T in (1, 2, 16, 17, 33, 256):
        for P in (16, 48, 64, 1024):
            # the most pages that a rest of 0 .. P - 1 tokens and T nodes take
            assert f(T, P, 5) == 5 + max(-(-(r + T) // P) for r in range(P))
    assert f(0, 16, 5) == f(257, 16, 5) == f(1, 8, 5) == f(1, 16, 0) == f(1, 16, 49153) == f(1, 24, 3) == 0


def test_sparse_attention_refusals(lib):
    """As tree_attention's; the width bounds max_len."""
    def f(c=None, **kw):
        d = dict(q=A, ldq=512, pages=A, width=4, kept=A, nodes=A, mask=A, scale=0.1, max_len=64, out=A, lse=A, B=2, T=3, Hq=4,
                 ws=A, wsb=1 << 40)
        d.update(kw)
        return lib.bsf8_sparse_attention(d["q"], d["ldq"], c or cache(), d["pages"], d["width"], d["kept"], d["nodes"], d["mask"],
                                         d["scale"], d["max_len"], d["out"], d["lse"], d["B"], d["T"], d["Hq"], d["ws"],
                                         d["wsb"], None)
    for name in ("q", "pages", "kept", "out"):
        assert f(**{name: 0}) == NULL, name
    for kw in (dict(B=0), dict(B=1025), dict(T=0), dict(T=257), dict(Hq=3), dict(max_len=0), dict(max_len=65), dict(width=0)):
        assert f(**kw) == SHAPE, kw
    assert f(scale=0.0) == VALUE and f(ldq=504) == STRIDE and f(pages=A + 2) == ALIGN and f(cache(dim=32)) == SHAPE
    need = lib.bsf8_tree_attention_workspace_bytes(2, 3, 4, 2, 128)
    assert f(ws=0) == WORKSPACE and f(wsb=need - 1) == WORKSPACE and f(ws=A + 4) == ALIGN


def test_sampling_refusals(lib):
    def tokens(**kw):
        d = dict(logits=A, bf16=0, ld=100, u=A, t=A, k=A, tp=A, mp=A, token=A, p=A, N=2, V=100)
        d.update(kw)
        return lib.bsf8_sample_tokens(*d.values(), None)

    def probs(**kw):
        d = dict(logits=A, bf16=1, ld=100, t=A, k=A, tp=A, mp=A, p=A, N=2, V=100)
        d.update(kw)
        return lib.bsf8_token_probs(*d.values(), None)
    for f in (tokens, probs):
        assert f(logits=0) == NULL and f(p=0) == NULL
        for kw in (dict(N=-1), dict(N=(1 << 20) + 1), dict(V=0), dict(V=(1 << 20) + 1)):
            assert f(**kw) == SHAPE, kw
        assert f(ld=99) == STRIDE and f(logits=A + 8) == ALIGN and f(N=0) == OK
        for name in ("t", "k", "tp", "mp", "p"):
            assert f(**{name: A + 2}) == ALIGN, name
    assert tokens(u=0) == NULL and tokens(token=0) == NULL and tokens(u=A + 1) == ALIGN and tokens(token=A + 2) == ALIGN
    assert probs(p=A + 8) == ALIGN


def test_norm_refusals(lib):
    def f(**kw):
        d = dict(x=A, ldx=256, res=A, ldr=256, fp32=0, post=A, gate=A, kind=1, ldg=256, scale=1.0, w=A, eps=1e-6, r=A, h=A, M=3,
                 H=256)
        d.update(kw)
        return lib.bsf8_residual_norm(*d.values(), None)
    assert f(x=0) == NULL and f(r=0, h=0) == NULL and f(w=0) == NULL and f(gate=0) == NULL
    for kw in (dict(M=-1), dict(H=0), dict(H=4), dict(H=260), dict(H=32776)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(scale=NAN), dict(scale=INF), dict(scale=-INF), dict(kind=4),
               dict(kind=-1)):
        assert f(**kw) == VALUE, kw
    for kw in (dict(ldx=248), dict(ldr=248), dict(kind=3, ldg=248), dict(kind=2, ldg=0)):
        assert f(**kw) == STRIDE, kw
    for kw in (dict(x=A + 8), dict(ldx=260), dict(res=A + 8), dict(ldr=260), dict(fp32=1, ldr=258), dict(post=A + 2), dict(w=A + 8),
               dict(r=A + 8), dict(h=A + 4), dict(gate=A + 8), dict(kind=3, ldg=260), dict(kind=2, gate=A + 1)):
        assert f(**kw) == ALIGN, kw
    assert f(M=0) == OK


def test_binding_refuses_cpu_tensors_and_wrong_types():
    torch = pytest.importorskip("torch")
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        bsf8.sample_tokens(torch.zeros(2, 5), torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA tensor"):
        bsf8.token_probs(torch.zeros(2, 5))
    with pytest.raises(ValueError, match="CUDA tensor"):
        bsf8.residual_norm(torch.zeros(2, 8, dtype=torch.bfloat16), None, None)
    with pytest.raises(ValueError, match="CUDA tensor"):
        bsf8.kv_plan(bsf8.PageBook.empty(2, 3, 4, device="cpu"), i, i, page_size=16, tokens=4)
    with pytest.raises(TypeError, match="logits must be a torch.Tensor"):
        bsf8.sample_tokens([1.0], None)
    cache_ = bsf8.KVCache.empty(2, 1, 64, 16, device="cpu")
    bounds_ = bsf8.PageBounds.empty(cache_)
    assert bounds_.codes.shape == (2, 1, 2, 64) and bounds_.exps.shape == (2, 1, 2) and bounds_.page_size == 16
    with pytest.raises(ValueError, match="CUDA tensor"):
        bsf8.kv_bounds(cache_, bounds_, torch.zeros((1, 2), dtype=torch.int32), i[:1])
    with pytest.raises(ValueError, match="codes must be"):
        bsf8.select_pages(torch.zeros(1, 1, 1, 64), bsf8.PageBounds(cache_.k8[0], bounds_.exps, 16), i[None], i[:1], 3)
