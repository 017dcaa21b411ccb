"""Host-side refusals of the decode operators: each invalid argument gives its documented status
before any CUDA call (fake device addresses are only ever paired with an invalid argument)."""
import ctypes

import pytest

import block_scaled_fp8_weight_gb300 as bsf8
from block_scaled_fp8_weight_gb300 import build as bsf8_build
from block_scaled_fp8_weight_gb300.decode import _CacheStruct

OK, SHAPE, ALIGN, STRIDE, WORKSPACE, NULL, CUDA, TIMEOUT, DEVICE, VALUE, INDEX = range(11)
A = 0x10000  # a 16-byte aligned fake device address


@pytest.fixture(scope="module")
def lib():
    bsf8_build.build()
    return bsf8.load()


def cache(**kw):
    d = dict(k8=A, kexp=A, v8=A, vexp=A, pages=8, page_size=16, heads=2, dim=128)
    d.update(kw)
    return ctypes.byref(_CacheStruct(**d))


BAD_CACHES = [(dict(k8=0), NULL), (dict(vexp=0), NULL), (dict(pages=0), SHAPE), (dict(page_size=8), SHAPE),
              (dict(page_size=40), SHAPE), (dict(page_size=2048), SHAPE), (dict(heads=0), SHAPE), (dict(dim=96), SHAPE),
              (dict(dim=512), SHAPE), (dict(k8=A + 8), ALIGN), (dict(kexp=A + 4), ALIGN),
              (dict(pages=1 << 26, page_size=64), SHAPE)]


def append(lib, c=None, **kw):
    d = dict(q=A, k=A, v=A, ldq=512, ldk=256, ldv=256, q_out=A, table=A, requests=3, table_pages=4, req=A, slot=A, pos=A,
             cos_sin=A, positions=10, rot=64, interleaved=0, q_norm=A, k_norm=A, eps=1e-6, N=5, Hq=4)
    d.update(kw)
    return lib.bsf8_qkv_append(d["q"], d["k"], d["v"], d["ldq"], d["ldk"], d["ldv"], d["q_out"], c or cache(), d["table"],
                               d["requests"], d["table_pages"], d["req"], d["slot"], d["pos"], d["cos_sin"], d["positions"],
                               d["rot"], d["interleaved"], d["q_norm"], d["k_norm"], d["eps"], d["N"], d["Hq"], None)


def test_append_refusals(lib):
    for bad, status in BAD_CACHES:
        assert append(lib, cache(**bad)) == status, bad
    for name in ("q", "k", "v", "q_out", "table", "req", "slot", "pos", "cos_sin"):
        assert append(lib, **{name: 0}) == NULL, name
    assert append(lib, N=-1) == SHAPE and append(lib, Hq=-1) == SHAPE and append(lib, requests=0) == SHAPE
    assert append(lib, table_pages=0) == SHAPE and append(lib, rot=8) == SHAPE and append(lib, rot=144) == SHAPE
    assert append(lib, rot=-16) == SHAPE and append(lib, positions=0) == SHAPE
    assert append(lib, eps=-1.0) == VALUE and append(lib, eps=float("nan")) == VALUE and append(lib, eps=float("inf")) == VALUE
    assert append(lib, ldq=504) == STRIDE and append(lib, ldk=248) == STRIDE and append(lib, ldv=0) == STRIDE
    assert append(lib, ldq=516) == ALIGN and append(lib, ldk=258) == ALIGN
    for name in ("q", "k", "v", "q_out", "cos_sin", "q_norm", "k_norm"):
        assert append(lib, **{name: A + 8}) == ALIGN, name
    assert append(lib, slot=A + 2) == ALIGN
    assert append(lib, N=0) == OK  # nothing to do


def test_read_refusals(lib):
    f = lambda c=None, table=A, n=3, tp=4, req=A, slot=A, k=A, v=A, N=5: lib.bsf8_kv_read(  # noqa: E731
        c or cache(), table, n, tp, req, slot, k, v, N, None)
    for bad, status in BAD_CACHES:
        assert f(cache(**bad)) == status, bad
    assert f(table=0) == NULL and f(req=0) == NULL and f(slot=0) == NULL and f(k=0, v=0) == NULL
    assert f(N=-1) == SHAPE and f(n=0) == SHAPE and f(tp=0) == SHAPE
    assert f(k=A + 8) == ALIGN and f(v=A + 2) == ALIGN and f(req=A + 1) == ALIGN
    assert f(N=0) == OK


def attention(lib, c=None, **kw):
    d = dict(q=A, ldq=512, table=A, table_pages=4, ctx=A, nodes=A, mask=A, scale=0.1, max_len=64, out=A, lse=A, B=2, T=3,
             Hq=4, ws=A, wsb=1 << 40)
    d.update(kw)
    return lib.bsf8_tree_attention(d["q"], d["ldq"], c or cache(), d["table"], d["table_pages"], d["ctx"], d["nodes"],
                                   d["mask"], d["scale"], d["max_len"], d["out"], d["lse"], d["B"], d["T"], d["Hq"], d["ws"],
                                   d["wsb"], None)


def test_attention_refusals(lib):
    for bad, status in BAD_CACHES:
        assert attention(lib, cache(**bad)) == status, bad
    for name in ("q", "table", "ctx", "out"):
        assert attention(lib, **{name: 0}) == NULL, name
    for kw in (dict(B=0), dict(B=1025), dict(T=0), dict(T=257), dict(Hq=0), dict(Hq=3), dict(max_len=0), dict(max_len=65),
               dict(table_pages=0)):
        assert attention(lib, **kw) == SHAPE, kw
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert attention(lib, scale=s) == VALUE
    assert attention(lib, ldq=504) == STRIDE and attention(lib, ldq=516) == ALIGN
    assert attention(lib, q=A + 2) == ALIGN and attention(lib, out=A + 8) == ALIGN and attention(lib, mask=A + 2) == ALIGN
    need = lib.bsf8_tree_attention_workspace_bytes(2, 3, 4, 2, 128)
    if need:
        assert attention(lib, ws=0) == WORKSPACE and attention(lib, wsb=need - 1) == WORKSPACE
        assert attention(lib, ws=A + 4) == ALIGN
    for bad in ((0, 3, 4, 2, 128), (2, 0, 4, 2, 128), (2, 3, 4, 3, 128), (2, 3, 4, 2, 100), (2, 300, 4, 2, 128)):
        assert lib.bsf8_tree_attention_workspace_bytes(*bad) == 0


def test_attention_refuses_more_work_than_it_can_count(lib):
    """Key tiles with a segment's start and end, over all requests, heads and row tiles, are counted in 31 bits.  (A
    scale of 0, refused after that, shows that the last call inside the bound is not.)"""
    def f(tiles, dim, heads, T, page=16, scale=0.0):
        keys = 64 if dim == 256 else 128
        return attention(lib, cache(dim=dim, heads=heads, page_size=page), B=1024, T=T, Hq=heads, ldq=heads * dim,
                         max_len=tiles * keys, table_pages=tiles * keys // page, scale=scale)
    assert f(26, 64, 65536, 1) == VALUE                                      # 2^26 segments of 26 + 5 places
    assert f(27, 64, 65536, 1) == SHAPE == f(27, 64, 65536, 1, scale=0.1)    # of 27 + 5: 2^31
    assert f(122, 256, 16384, 1) == VALUE and f(123, 256, 16384, 1) == SHAPE
    assert f(58, 64, 16384, 256) == VALUE and f(59, 64, 16384, 256) == SHAPE  # two row tiles
    # up to 8 rows at dim 128 and more than 2048 tokens: 4 a segment
    assert f(59, 128, 32768, 1) == VALUE and f(60, 128, 32768, 1) == SHAPE


def test_attention_refuses_contexts_past_2_30_tokens(lib):
    """Past that the kernels' 31-bit slots and their division of 16-token groups by pages would leave the
    block table."""
    f = lambda n, scale: attention(lib, cache(page_size=1024), max_len=n, table_pages=(1 << 20) + 64, scale=scale)  # noqa: E731
    assert f(1 << 30, 0.0) == VALUE  # inside: the scale is what is wrong
    for n in ((1 << 30) + 1, (1 << 30) + 65536):
        assert f(n, 0.0) == SHAPE == f(n, 0.1)


def test_verify_refusals(lib):
    def f(**kw):
        d = dict(p=A, q=A, ld=100, tokens=A, parent=A, u=A, nodes=A, path=A, count=A, token=A, B=2, T=3, V=100)
        d.update(kw)
        return lib.bsf8_verify_tree(*d.values(), None)
    for name in ("p", "tokens", "parent", "u", "path", "count", "token"):
        assert f(**{name: 0}) == NULL, name
    for kw in (dict(B=0), dict(B=65536), dict(T=0), dict(T=257), dict(V=0), dict(V=(1 << 20) + 1)):
        assert f(**kw) == SHAPE, kw
    assert f(ld=99) == STRIDE and f(p=A + 4) == ALIGN and f(q=A + 8) == ALIGN and f(u=A + 2) == ALIGN


def test_commit_refusals(lib):
    f = lambda c=None, table=A, tp=4, ctx=A, path=A, count=A, B=2, T=3: lib.bsf8_kv_commit(  # noqa: E731
        c or cache(), table, tp, ctx, path, count, B, T, None)
    for bad, status in BAD_CACHES:
        assert f(cache(**bad)) == status, bad
    assert f(table=0) == NULL and f(ctx=0) == NULL and f(path=0) == NULL and f(count=0) == NULL
    assert f(B=0) == SHAPE and f(T=0) == SHAPE and f(T=257) == SHAPE and f(tp=0) == SHAPE
    assert f(ctx=A + 2) == ALIGN


def test_index_status_has_a_name(lib):
    assert lib.bsf8_strerror(INDEX) != b"unknown status"
    assert bsf8.STATUS[INDEX] == "ERR_INDEX"


def test_binding_refuses_cpu_tensors_and_bad_shapes():
    torch = pytest.importorskip("torch")
    z = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    c = bsf8.KVCache(z(2, 1, 16, 64), z(2, 1, 16, 2), z(2, 1, 16, 64), z(2, 1, 16, 2))
    t = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        bsf8.kv_read(c, t, t[0], t[0])
    with pytest.raises(ValueError, match="vexp must have shape"):
        bsf8.KVCache(z(2, 1, 16, 64), z(2, 1, 16, 2), z(2, 1, 16, 64), z(2, 1, 16, 4))._struct()
    with pytest.raises(ValueError, match="CUDA tensor"):
        bsf8.verify_tree(torch.zeros(1, 2, 3), t, t, torch.zeros(1, 2))
