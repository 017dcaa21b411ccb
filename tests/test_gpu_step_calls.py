"""GPU: the operators around a decode step in the calls that programs make of them all: captured at their first call, on two
streams at once, over pages that requests share, and past 2^31 elements."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import block_scaled_fp8_weight_gb300 as bsf8

pytestmark = pytest.mark.gpu

FIRST = """
import torch
import block_scaled_fp8_weight_gb300 as bsf8

g = torch.Generator(device="cuda").manual_seed(1)
rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
whole = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
B, heads, D, page, pool = 200, 2, 128, 16, 8192
cache = bsf8.KVCache.empty(pool, heads, D, page)
cache.k8.copy_(torch.randint(0, 120, cache.k8.shape, generator=g, device="cuda"))
cache.v8.copy_(torch.randint(0, 120, cache.v8.shape, generator=g, device="cuda"))
cache.kexp.fill_(120)
cache.vexp.fill_(120)
table = torch.randperm(pool, generator=g, device="cuda").int()[:B * 40].view(B, 40).contiguous()
ctx = torch.randint(1, 600, (B,), generator=g, device="cuda").int()
q = rand(B, 1, 8, D).bfloat16()
x, r, w = rand(900, 2048).bfloat16(), rand(900, 2048), rand(2048).bfloat16()
logits, u = rand(40, 40000), torch.rand(40, generator=g, device="cuda")
k, p = whole([30] * 40), torch.full((40,), 0.9, device="cuda")
book = bsf8.PageBook.empty(B, 40, pool)
lens, add = torch.zeros_like(ctx), ctx.clone()
bounds = bsf8.PageBounds.empty(cache)


def step():
    plan = bsf8.kv_plan(book, lens, add, page_size=page, tokens=100000, done=torch.ones_like(lens))
    bsf8.kv_bounds(cache, bounds, table, ctx)
    pages, kept = bsf8.select_pages(q, bounds, table, ctx, 12, sink=1, recent=1, nodes=torch.zeros_like(lens))
    o = bsf8.sparse_attention(q, cache, pages, kept, nodes=torch.zeros_like(lens))
    h = bsf8.residual_norm(x, r, w, post_weight=w, gate=w)
    t = bsf8.sample_tokens(logits, u, top_k=k) + bsf8.sample_tokens(logits[:3], u[:3], top_p=p[:3]) + bsf8.sample_tokens(logits.bfloat16(), u)
    return (*plan, pages, kept, o, *h, *t, bsf8.token_probs(logits, top_p=p))


bsf8.residual_norm(x[:0], r[:0], w)  # what the binding loads; no kernel runs
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
first = [t.clone() for t in out]
graph.replay()
for a, b, c in zip(out, first, step()):
    assert torch.equal(a, b) and torch.equal(a, c)
assert bsf8.device_status() == 0
print("the same")
"""


def test_captured_at_their_first_call(bsf8_lib):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "the same", r.stdout + r.stderr


def test_two_streams_at_once(bsf8_lib):
    """Each stream's calls beside the other's: nothing is shared between two calls."""
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    sets = []
    for n in (5, 60):
        x = rand(40 * n, 5120).bfloat16()
        logits, u = rand(n, 60000), torch.rand(n, generator=g, device="cuda")
        p, k = torch.full((n,), 0.8, device="cuda"), torch.arange(1, n + 1, dtype=torch.int32, device="cuda") * 9
        cache = bsf8.KVCache.empty(512, 2, 64, 32)
        cache.k8.copy_(torch.randint(0, 120, cache.k8.shape, generator=g, device="cuda"))
        cache.kexp.fill_(121)
        b = bsf8.PageBounds.empty(cache)
        table = torch.randperm(512, generator=g, device="cuda").int()[:n * 8].view(n, 8).contiguous()
        ctx = torch.full((n,), 250, dtype=torch.int32, device="cuda")
        q, none = rand(n, 1, 4, 64).bfloat16(), torch.zeros_like(ctx)
        book = bsf8.PageBook.empty(n, 8, 512)

        def step(x=x, logits=logits, u=u, p=p, k=k, cache=cache, b=b, table=table, ctx=ctx, q=q, none=none, book=book):
            plan = bsf8.kv_plan(book, none, ctx, page_size=32, tokens=20000, done=ctx)
            bsf8.kv_bounds(cache, b, table, ctx)
            return (*plan, *bsf8.residual_norm(x, x.float(), x[0], post_weight=x[1]), *bsf8.sample_tokens(logits, u, top_p=p),
                    *bsf8.sample_tokens(logits, u, top_k=k), bsf8.token_probs(logits, top_k=k, top_p=p),
                    *bsf8.select_pages(q, b, table, ctx, 3, nodes=none))
        sets.append((step, step(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for step, want, s in sets:
            with torch.cuda.stream(s):
                outs.append((want, step()))
    torch.cuda.synchronize()
    for want, got in outs:
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert bsf8.device_status() == 0


def test_pages_that_requests_share(bsf8_lib):
    """Requests with the same first pages: bounds written by each, selected and read by each as if they were its own."""
    g = torch.Generator(device="cuda").manual_seed(4)
    cache = bsf8.KVCache.empty(64, 2, 128, 16)
    for t in (cache.k8, cache.v8):
        t.copy_(torch.randint(0, 120, t.shape, generator=g, device="cuda") + 128 * torch.randint(0, 2, t.shape, generator=g, device="cuda"))
    cache.kexp.fill_(119)
    cache.vexp.fill_(119)
    own = torch.arange(64, dtype=torch.int32, device="cuda").view(2, 32)
    shared = own[:1].repeat(5, 1)
    shared[1:, 20:] = own[1, :12]
    ctx = torch.full((5,), 32 * 16 - 3, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 1, 8, 128, generator=g, device="cuda").bfloat16().expand(5, 1, 8, 128).contiguous()
    b = bsf8.PageBounds.empty(cache)
    bsf8.kv_bounds(cache, b, shared, ctx)
    pages, kept = bsf8.select_pages(q, b, shared, ctx, 9, recent=1)
    o = bsf8.sparse_attention(q, cache, pages, kept)
    for i in (0, 3):
        again = bsf8.PageBounds.empty(cache)
        bsf8.kv_bounds(cache, again, shared[i:i + 1], ctx[:1])
        alone, n = bsf8.select_pages(q[:1], again, shared[i:i + 1], ctx[:1], 9, recent=1)
        assert torch.equal(alone[0], pages[i]) and torch.equal(n[0], kept[i])
        assert torch.allclose(bsf8.sparse_attention(q[:1], cache, alone, n)[0].float(), o[i].float(), rtol=2.0 ** -7, atol=1e-6)
    assert torch.equal(pages[1], pages[4]) and torch.equal(o[1], o[4])


def test_past_two_to_the_31_elements(bsf8_lib):
    """The last rows of tensors of more elements than 31 bits count are those of a call of their own."""
    M, H = 70001, 32768
    x = torch.zeros(M, H, device="cuda", dtype=torch.bfloat16)
    x[-2:] = torch.randn(2, H, device="cuda")
    w = torch.randn(H, device="cuda").bfloat16()
    h, r = bsf8.residual_norm(x, x, w)
    a, b = bsf8.residual_norm(x[-2:], x[-2:], w)
    assert torch.equal(h[-2:], a) and torch.equal(r[-2:], b) and not h[:-2].any()
    del x, h, r
    N, V = 2060, 1 << 20
    x = torch.full((N, V), float("-inf"), device="cuda", dtype=torch.bfloat16)
    x[:, 7] = 0.0
    x[-1] = torch.randn(V, device="cuda")
    u = torch.full((N,), 0.4, device="cuda")
    token, p = bsf8.sample_tokens(x, u)
    one, q = bsf8.sample_tokens(x[-1:].clone(), u[:1])
    assert (token[:-1] == 7).all() and (p[:-1] == 1).all() and int(token[-1]) == int(one) and float(p[-1]) == float(q)
    p = bsf8.token_probs(x)
    assert torch.equal(p[-1:], bsf8.token_probs(x[-1:].clone())) and (p[:-1, 7] == 1).all() and not p[:-1, 8:].any()


def test_lengths_that_no_call_takes(bsf8_lib):
    """max_len outside 31 bits and below -1 is a ValueError, as it always was for tree_attention; what only the library refuses
    is a Bsf8Error."""
    cache = bsf8.KVCache.empty(4, 1, 64, 16)
    b = bsf8.PageBounds.empty(cache)
    q = torch.zeros(1, 1, 1, 64, device="cuda", dtype=torch.bfloat16)
    table, ctx = torch.zeros((1, 4), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    calls = (lambda n: bsf8.tree_attention(q, cache, table, ctx, max_len=n),
             lambda n: bsf8.sparse_attention(q, cache, table[:, None], ctx, max_len=n),
             lambda n: bsf8.select_pages(q, b, table, ctx, 2, max_len=n))
    for f in calls:
        for n in (-2, -2 ** 31 + 1, -2 ** 31, 2 ** 31, -2 ** 40, 2 ** 40):
            with pytest.raises(ValueError):
                f(n)
        for n in (-1, 0, 65):
            with pytest.raises(bsf8.Bsf8Error):
                f(n)
        with pytest.raises(OverflowError):
            f(2 ** 70)
        with pytest.raises(TypeError):
            f(3.5)


def test_a_plan_of_many_tokens(bsf8_lib):
    N = (1 << 27) + 3
    book = bsf8.PageBook.empty(3, 1 << 15, 1 << 15)
    lens, add = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 5, 0], [1 << 20, 70000, 1]))
    req, slot, start, granted = bsf8.kv_plan(book, lens, add, page_size=64, tokens=N)
    assert granted.tolist() == add.tolist() and start.tolist() == [0, 1 << 20, (1 << 20) + 70000, (1 << 20) + 70001]
    n = int(start[-1])
    assert torch.equal(slot[:1 << 20], torch.arange(1 << 20, dtype=torch.int32, device="cuda"))
    assert slot[1 << 20:n].tolist() == list(range(5, 70005)) + [0] and int(req[n - 1]) == 2
    assert (slot[n:] == -1).all() and not req[n:].any()
    assert book.held.tolist() == [1 << 14, -(-70005 // 64), 1] and np.array_equal(book.table[0, :1 << 14].cpu().numpy(), np.arange(1 << 14))
