"""GPU: sampling and processed distributions against the definition in whole numbers, and that against the softmax."""
import numpy as np
import pytest
import torch

import _step_ref as ref
import block_scaled_fp8_weight_gb300 as bsf8

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def f32(v):
    return torch.tensor(np.asarray(v, np.float32), device="cuda")


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def check(x, u, t=None, k=None, tp=None, mp=None):
    """Tokens exactly, probabilities to 2^-22 of themselves (four roundings of 2^-24)."""
    kw = dict(temperature=None if t is None else f32(t), top_k=None if k is None else i32(k),
              top_p=None if tp is None else f32(tp), min_p=None if mp is None else f32(mp))
    token, p = bsf8.sample_tokens(x, f32(u), **kw)
    q = bsf8.token_probs(x, **kw)
    xs = x.float().cpu().numpy()
    q, token, p = q.cpu().numpy().astype(np.float64), token.cpu().numpy(), p.cpu().numpy().astype(np.float64)
    for n in range(len(xs)):
        at = lambda v, d: d if v is None else np.asarray(v)[n]  # noqa: E731
        w = ref.kept(xs[n], float(np.float32(at(t, 1.0))), int(at(k, 0)), float(np.float32(at(tp, 1.0))), float(np.float32(at(mp, 0.0))))
        want = ref.draw(w, np.float32(u[n]))
        assert token[n] == want, (n, token[n], want)
        share = w / max(1, int(w.sum()))
        assert np.all(np.abs(q[n] - share) <= share * 2.0 ** -22), n
        assert abs(p[n] - (share[want] if want >= 0 else 0)) <= (share[want] if want >= 0 else 0) * 2.0 ** -22
    assert bsf8.device_status() == 0


HOW = {"plain": {}, "hot": dict(t=1.9), "cold": dict(t=0.05), "k": dict(k=40), "k1": dict(k=1), "k600": dict(k=600),
       "p": dict(tp=0.9), "p0": dict(tp=0.0), "tiny p": dict(tp=1e-7), "min": dict(mp=0.05), "k+p": dict(k=50, tp=0.8, t=0.7),
       "k+min": dict(k=700, mp=0.001), "all": dict(k=300, tp=0.95, mp=0.002, t=1.3), "greedy": dict(t=0.0), "min+p": dict(mp=0.01, tp=0.6)}


@pytest.mark.parametrize("N,V,ld", [(1, 1, 1), (3, 7, 7), (2, 1000, 1003), (5, 4096, 4096), (3, 4097, 4100), (2, 50257, 50257),
                                    (3, 32000, 32064), (1, 131072, 131072), (1, 1 << 20, 1 << 20)])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("how", list(HOW))
def test_sampling(bsf8_lib, N, V, ld, bf16, how):
    if V >= 1 << 20 and how not in ("plain", "k", "all"):
        pytest.skip("the largest row with a few of them only")
    r = np.random.default_rng(V + len(how))
    x = torch.from_numpy((r.standard_normal((N, ld)) * 2.5 + 5 * (r.random((N, ld)) > 0.999)).astype(np.float32)).cuda()
    if bf16:
        x = x.to(torch.bfloat16)  # ties, at every border
    u = r.random(N).astype(np.float32)
    check(x[:, :V], u, **{a: [v] * N for a, v in HOW[how].items()})


@pytest.mark.parametrize("V", [2049, 2113, 4435, 8192, 8193, 9000])
@pytest.mark.parametrize("bf16", [False, True])
def test_many_of_a_short_row(bsf8_lib, V, bf16):
    """k about the maxima that a row has, the elements that are sorted, and the row's finite elements."""
    r = np.random.default_rng(V)
    ks = [60, 250, 257, 500, 530, 700, 840, 900, 1100, 1300, 1800, 1952, 1953, 2047, 2048]
    N = len(ks)
    x = torch.from_numpy((r.standard_normal((N, V)) * 2.5).astype(np.float32)).cuda()
    x[3, 400:] = float("-inf")  # 500 of 400
    x[7] = x[7].mul(2).round()  # few values
    x[9] *= 1e-30
    x[11, 5] = 1e30
    if bf16:
        x = x.to(torch.bfloat16)
    u = r.random(N).astype(np.float32)
    check(x, u, k=ks)
    check(x, u, k=ks, tp=[0.9] * N, mp=[1e-4] * N)


@pytest.mark.parametrize("V", [2500, 20000, 70001])
@pytest.mark.parametrize("bf16", [False, True])
def test_the_cut_among_many_alike(bsf8_lib, V, bf16):
    """top-p that ends among hundreds or thousands of one logit, of two next to each other, and of a few."""
    r = np.random.default_rng(V)
    ps = [0.02, 0.2, 0.35, 0.5, 0.51, 0.7, 0.8, 0.9, 0.97, 0.999, 0.9999, 1e-7]
    alike = [1, 20, 31, 33, 300, 700, 1500, 2040, 2049, 2300, 900, 64]
    x = np.full((len(ps), V), -9.0, np.float32)
    for i, n in enumerate(alike):
        at = r.permutation(V)
        x[i, at[:n]] = 2.0
        x[i, at[n:n + n // 2]] = 2.0 - 2.0 ** -7  # the bf16 value below it
        x[i, at[:5]] += r.random(5).astype(np.float32) * 3
    x = torch.from_numpy(x).cuda()
    if bf16:
        x = x.to(torch.bfloat16)
    u = r.random(len(ps)).astype(np.float32)
    check(x, u, tp=ps)
    check(x, u, tp=ps[::-1], mp=[1e-3] * len(ps), t=[0.8] * len(ps))


def test_rows_ask_for_different_things(bsf8_lib):
    r = np.random.default_rng(1)
    N, V = 64, 3001
    x = torch.from_numpy((r.standard_normal((N, V)) * 3).astype(np.float32)).cuda()
    check(x, r.random(N), t=r.choice([0.0, 0.3, 1.0, 2.0, -1.0, NAN], N), k=r.choice([-1, 0, 1, 2, 5, 40, 513, 3000, 3001, 9999], N),
          tp=r.choice([0.0, 0.3, 0.9, 0.999999, 1.0, 1.5, -0.5, NAN], N), mp=r.choice([0.0, -1.0, 0.2, 1.0, 2.0, NAN, 1e-6], N))


def test_ends_of_the_numbers(bsf8_lib):
    """Rows of nothing, of one value, with infinities and NaN, huge and tiny distances and temperatures."""
    V = 777
    x = np.zeros((16, V), np.float32)
    x[0] = -INF
    x[1] = NAN
    x[2] = INF
    x[3, 5] = x[3, 600] = INF
    x[4] = -INF
    x[4, 776] = -3e38
    x[5, ::2] = 3e38
    x[5, 1::2] = -3e38
    x[6] = NAN
    x[6, 3] = 0.0
    x[7] = 1e-30 * np.arange(V)
    x[8] = 40 * np.log(2) * np.linspace(0, 1, V)       # weights down to the last one
    x[9, ::3] = -0.0
    x[10] = np.float32(7.25)
    x[11] = -INF
    x[12] = np.arange(V) * 1e4
    x[13] = 2.0 ** -20 * np.arange(V)                  # all within one step of the histogram
    x[14] = -np.arange(V) * 0.01
    x[15] = np.where(np.arange(V) % 7 == 0, -INF, 1.0)
    d = torch.from_numpy(x).cuda()
    r = np.random.default_rng(3)
    for t in (1.0, 0.0, INF, 1e-30, 1e30, 1e-45, 50.0):
        for kw in ({}, dict(k=[3] * 16), dict(tp=[0.5] * 16), dict(k=[500] * 16, tp=[0.999] * 16), dict(mp=[0.5] * 16)):
            check(d, r.random(16), t=[t] * 16, **kw)


def test_the_draw_at_its_ends(bsf8_lib):
    r = np.random.default_rng(5)
    x = torch.from_numpy((r.standard_normal((1, 5000)) * 2).astype(np.float32)).cuda().expand(8, 5000).contiguous()
    check(x, [0.0, 1 - 2.0 ** -24, 1.0, 2.0, -1.0, NAN, INF, 2.0 ** -24], tp=[0.9] * 8)


def close_logits(r, N, V, n, top, far, few_values=False):
    """Rows whose largest logit is `top`, with n logits about 0 that it is one rounded distance away from, of either sign, the
    rest at `far`."""
    x = np.full((N, V), far, np.float32)
    for i in range(N):
        at = r.permutation(V)
        small = r.integers(-40, 41, size=n) if few_values else r.permutation(2 * n) - n
        x[i, at[:n]] = small[:n] * np.float32(2.0 ** -50)
        x[i, at[n]] = top
    return torch.from_numpy(x).cuda()


def test_a_larger_logit_at_the_same_rounded_distance_comes_first(bsf8_lib):
    """10 - 2^-31 and 10 - 2^-30 are one number in fp32: the order is the logits'."""
    for bf16 in (False, True):
        for V in (64, 3000, 9000):
            x = torch.full((2, V), -5.0, device="cuda")
            x[:, 0], x[:, 1], x[:, 2], x[:, 3], x[:, 4] = 10.0, 2.0 ** -31, 2.0 ** -30, -0.0, 0.0
            if bf16:
                x = x.to(torch.bfloat16)
            for k in (2, 3, 4, 5):
                check(x, [0.99999994, 0.3], k=[k] * 2)
                check(x, [0.99999994, 0.3], k=[k] * 2, t=[30.0] * 2, tp=[0.9] * 2)


@pytest.mark.parametrize("V,n", [(100, 60), (2048, 1500), (2500, 700), (8000, 4000), (5000, 3000), (40000, 900), (40000, 30000),
                                 (131072, 100000)])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("few_values", [False, True])
def test_the_cut_among_logits_at_one_rounded_distance(bsf8_lib, V, n, bf16, few_values):
    """By k: in the sort, among all of a short row, by digits; by top-p; by one after the other."""
    r = np.random.default_rng(V + n)
    ks = sorted({2, 5, n // 7 + 2, n // 3, n // 2, n - 1, n, min(n, 1900)})
    N = len(ks)
    x = close_logits(r, N, V, n, 10.0, -900.0, few_values)
    if bf16:
        x = x.to(torch.bfloat16)
    u = r.random(N).astype(np.float32)
    u[::2] = 0.99999994
    t = [20.0] * N  # the logits about 0 weigh 0.6 of the largest, those at -900 nothing
    check(x, u, t=t, k=ks)
    ps = np.linspace(0.01, 0.99, N)
    check(x, u, t=t, tp=ps)
    check(x, u, t=t, tp=ps, mp=[0.5] * N)
    check(x, u, t=t, k=ks, tp=ps[::-1])


@pytest.mark.parametrize("value", [0.0, -5.5])
def test_ties_go_to_the_lowest_index(bsf8_lib, value):
    """A row of equal logits over many blocks: top-k and top-p cut inside it."""
    V = 40003
    x = torch.full((5, V), value, device="cuda")
    x[1, 20000:] = value + 1
    x[2, ::2] = value + 1
    for k in (1, 2, 511, 513, 4096, 20002, 20003, 30000, V - 1):
        check(x, [0.999] * 5, k=[k] * 5)
    for p in (0.1, 0.5, 0.75):
        check(x, [0.999] * 5, tp=[p] * 5)
        check(x, [0.999] * 5, tp=[p] * 5, k=[25000] * 5)


def test_weights_are_the_softmax(bsf8_lib):
    """2^-16 of it: y's rounding (three of 2^-24 of y <= 40, times ln 2), the polynomial's 2^-21.9, the same in the sum, and
    2^-40 of the largest a token that is cut off."""
    r = np.random.default_rng(7)
    for V, t in ((9, 1.0), (5000, 0.6), (128000, 1.7)):
        x = (r.standard_normal((2, V)) * 4).astype(np.float32)
        p = bsf8.token_probs(torch.from_numpy(x).cuda(), temperature=f32([t] * 2)).cpu().numpy().astype(np.float64)
        z = x.astype(np.float64) / float(np.float32(t))
        e = np.exp(z - z.max(1, keepdims=True))
        want = e / e.sum(1, keepdims=True)
        assert np.all(np.abs(p - want) <= want * 2.0 ** -16 + want.max(1, keepdims=True) * 2.0 ** -40 * (1 + want * V))


def test_draws_follow_the_distribution(bsf8_lib):
    """65536 even steps of u over one row: each token's count is its share of them, off by one at most at either end of
    its run."""
    r = np.random.default_rng(8)
    x = torch.from_numpy(r.standard_normal((1, 50)).astype(np.float32)).cuda()
    n = 65536
    token, p = bsf8.sample_tokens(x.expand(n, 50).contiguous(), torch.arange(n, device="cuda") / n)
    q = bsf8.token_probs(x)[0]
    count = torch.bincount(token.long(), minlength=50)
    assert ((count - q * n).abs() <= 1.01).all()
    assert torch.equal(p, q[token.long()])


def test_sampling_in_a_graph_and_on_a_side_stream(bsf8_lib):
    r = np.random.default_rng(11)
    x = torch.from_numpy((r.standard_normal((3, 9001)) * 3).astype(np.float32)).cuda()
    u, t, k, tp = f32([0.1, 0.5, 0.9]), f32([1.0, 0.5, 0.0]), i32([0, 30, 0]), f32([0.9, 1.0, 1.0])
    want = bsf8.sample_tokens(x, u, temperature=t, top_k=k, top_p=tp)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = bsf8.sample_tokens(x, u, temperature=t, top_k=k, top_p=tp)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        token, p = bsf8.sample_tokens(x, u, temperature=t, top_k=k, top_p=tp)
        q = bsf8.token_probs(x, temperature=t, top_k=k, top_p=tp)
    for _ in range(3):
        x.copy_(torch.from_numpy((r.standard_normal((3, 9001)) * 3).astype(np.float32)))
        g.replay()
        want = bsf8.sample_tokens(x, u, temperature=t, top_k=k, top_p=tp)
        assert torch.equal(token, want[0]) and torch.equal(p, want[1])
        assert torch.equal(q, bsf8.token_probs(x, temperature=t, top_k=k, top_p=tp))


def test_refused_tensors(bsf8_lib):
    x, u = torch.zeros(4, 64, device="cuda"), torch.zeros(4, device="cuda")
    f = bsf8.sample_tokens
    for bad in (lambda: f(x.half(), u), lambda: f(x, u.double()), lambda: f(x, u, top_k=u), lambda: f(x, u, temperature=i32([1] * 4)),
                lambda: f(x, u, temperature=1.0)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: f(x[None], u), lambda: f(x.T, u), lambda: f(x, u[:3]), lambda: f(x, u, top_p=u[:1]), lambda: f(x.cpu(), u),
                lambda: bsf8.token_probs(x, out=x[:2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(bsf8.Bsf8Error):
        f(x[:, 1:], u)  # not 16-byte aligned
    token, p = f(x[:0], u[:0])
    assert token.shape == p.shape == (0,) and bsf8.token_probs(x[:0]).shape == (0, 64)
