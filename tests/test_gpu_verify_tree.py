"""GPU: verification of drafted trees, equal to Python's integers in every output."""
import numpy as np
import pytest
import torch

import _decode_ref as ref
import block_scaled_fp8_weight_gb300 as bsf8

pytestmark = pytest.mark.gpu


def problem(r, B, T, V, sharp=2.0, near=0.5):
    x = r.standard_normal((B, T, V)) * sharp
    soft = lambda y: (lambda e: e / e.sum(-1, keepdims=True))(np.exp(y - y.max(-1, keepdims=True)))  # noqa: E731
    p = soft(x).astype(np.float32)
    q = soft(x + near * r.standard_normal((B, T, V))).astype(np.float32)
    parent = np.zeros((B, T), np.int32)
    tok = np.zeros((B, T), np.int32)
    for b in range(B):
        parent[b] = ref.tree(r, T)[0]
        for i in range(1, T):
            w = q[b, parent[b, i]].astype(np.float64)
            tok[b, i] = r.choice(V, p=w / w.sum())
    u = (r.integers(0, 1 << 24, size=(B, T)) / float(1 << 24)).astype(np.float32)
    return p, q, tok, parent, u


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def compare(p, q, tok, parent, u, nodes=None, got=None):
    B, T, V = p.shape
    if got is None:
        got = bsf8.verify_tree(dev(p), dev(tok), dev(parent), dev(u), q=None if q is None else dev(q),
                               nodes=None if nodes is None else dev(np.asarray(nodes, np.int32)))
    path, count, token = (t.cpu().numpy() for t in got)
    for b in range(B):
        n = T if nodes is None else int(nodes[b])
        want = ref.verify(p[b], None if q is None else q[b], tok[b].tolist(), parent[b].tolist(), u[b], n)
        assert (path[b].tolist(), int(count[b]), int(token[b])) == want, b


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (2, 2, 3), (1, 6, 50257), (7, 9, 1000), (40, 16, 257), (3, 64, 513), (2, 256, 130),
                                   (160, 3, 33), (1, 4, 8191)])
def test_equal_to_integers(bsf8_lib, B, T, V, drawn):
    r = np.random.default_rng(B * 1000 + T + V)
    p, q, tok, parent, u = problem(r, B, T, V)
    compare(p, q if drawn else None, tok, parent, u, nodes=r.integers(1, T + 1, size=B))
    assert bsf8.device_status() == 0


@pytest.mark.parametrize("near", [0.0, 0.2, 3.0])
def test_many_walks(bsf8_lib, near):
    """Drafts equal to, near and far from the target: long walks, many rejections in a row."""
    r = np.random.default_rng(3)
    p, q, tok, parent, u = problem(r, 300, 12, 37, near=near)
    compare(p, q, tok, parent, u)
    parent[:] = np.where(np.arange(12) > 0, 0, -1)  # all children of the root: rejections pile up
    for b in range(300):
        tok[b] = r.choice(37, size=12, p=(lambda w: w / w.sum())(q[b, 0].astype(np.float64)))
    compare(p, q, tok, parent, u)
    compare(p, None, tok, parent, u)


def test_long_walks_over_large_rows(bsf8_lib):
    """Several sums a walk, each over the blocks of a cluster: far drafts (rejections in a row), near
    ones, and every request at another length."""
    r = np.random.default_rng(12)
    for near, V in ((0.3, 33001), (2.5, 40000)):
        p, q, tok, parent, u = problem(r, 12, 10, V, near=near)
        compare(p, q, tok, parent, u, nodes=r.integers(5, 11, size=12))
    # many requests at once: the same walks give the same answers
    P, Q = np.tile(p, (25, 1, 1)), np.tile(q, (25, 1, 1))
    tile = lambda x: np.tile(x, (25, 1))  # noqa: E731
    path, count, token = bsf8.verify_tree(dev(P), dev(tile(tok)), dev(tile(parent)), dev(tile(u)), q=dev(Q))
    for t in (path.view(25, 12, 10), count.view(25, 12), token.view(25, 12)):
        assert torch.equal(t, t[:1].expand_as(t))


def test_edges(bsf8_lib):
    """One-hot rows, rows of zeros and NaN, u = 0 and the largest u, tokens the target excludes."""
    V, T = 11, 4
    rows = np.zeros((8, T, V), np.float32)
    q = np.full((8, T, V), 1 / V, np.float32)
    tok = np.tile(np.array([0, 3, 5, 7], np.int32), (8, 1))
    parent = np.tile(np.array([-1, 0, 0, 1], np.int32), (8, 1))
    u = np.full((8, T), 0.5, np.float32)
    rows[0, :, 3] = 1                 # certain: kept
    rows[1, :, 10] = 1                # the drafts are excluded
    rows[2] = 0                       # no mass at all: V - 1
    rows[3] = np.nan                  # NaN counts as 0
    rows[4] = 1 / V
    u[4] = 0
    rows[5] = 1 / V
    u[5] = 1 - 2.0 ** -24
    rows[6, :, 0] = 1e-13             # below the fixed point's grain
    rows[7] = q[7]
    u[7] = 1.0                        # out of range: counts as the largest
    want_u = u.copy()
    want_u[7] = 1 - 2.0 ** -24
    for drawn in (True, False):
        got = bsf8.verify_tree(dev(rows), dev(tok), dev(parent), dev(u), q=dev(q) if drawn else None)
        compare(rows, q if drawn else None, tok, parent, want_u, got=got)


def test_strided_rows_and_determinism(bsf8_lib):
    """Rows with a stride that is no multiple of four elements; the same call twice."""
    r = np.random.default_rng(8)
    p, q, tok, parent, u = problem(r, 4, 5, 1001)
    buf = [torch.zeros(4, 5, 1003, device="cuda") for _ in range(2)]
    for t, x in zip(buf, (p, q)):
        t[..., :1001] = dev(x)
        t[..., 1001:] = 0.5           # between the rows: not to be counted
    a = bsf8.verify_tree(buf[0][..., :1001], dev(tok), dev(parent), dev(u), q=buf[1][..., :1001])
    compare(p, q, tok, parent, u, got=a)
    b = bsf8.verify_tree(buf[0][..., :1001], dev(tok), dev(parent), dev(u), q=buf[1][..., :1001])
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_the_kept_tokens_follow_the_target(bsf8_lib):
    """The first new token's frequencies over 200000 draws are the target's: each within six standard
    deviations of a binomial share."""
    r = np.random.default_rng(2)
    V, T, B, rounds = 7, 3, 50000, 4
    p, q, _, _, _ = problem(r, 1, T, V, sharp=1.0, near=1.5)
    P, Q = np.repeat(p, B, 0), np.repeat(q, B, 0)
    hits = np.zeros(V)
    for _ in range(rounds):
        tok = r.choice(V, size=(B, T), p=(lambda w: w / w.sum())(q[0, 0].astype(np.float64))).astype(np.int32)
        parent = np.tile(np.array([-1, 0, 0], np.int32), (B, 1))
        u = (r.integers(0, 1 << 24, size=(B, T)) / float(1 << 24)).astype(np.float32)
        path, count, token = bsf8.verify_tree(dev(P), dev(tok), dev(parent), dev(u), q=dev(Q))
        path, count, token = path.cpu().numpy(), count.cpu().numpy(), token.cpu().numpy()
        first = np.where(count > 1, tok[np.arange(B), np.maximum(path[:, 1], 0)], token)
        hits += np.bincount(first, minlength=V)
    n = rounds * B
    want = p[0, 0].astype(np.float64) / p[0, 0].astype(np.float64).sum()
    assert np.all(np.abs(hits / n - want) <= 6 * np.sqrt(want * (1 - want) / n))


def test_bad_nodes_are_never_kept(bsf8_lib):
    r = np.random.default_rng(4)
    p, q, tok, parent, u = problem(r, 3, 5, 50)
    parent[0, 2], tok[1, 1], parent[2, 4] = 3, 50, -5
    got = bsf8.verify_tree(dev(p), dev(tok), dev(parent), dev(u), q=dev(q), nodes=dev(np.array([5, 5, 9], np.int32)))
    assert bsf8.device_status() == 10
    tok2, par2 = tok.copy(), parent.copy()
    par2[0, 2], par2[1, 1], par2[2, 4] = -9, -9, -9
    tok2[1, 1] = 0
    compare(p, q, tok2, par2, u, got=got)


@pytest.mark.parametrize("rejections,V", [(18, 986896), (64, 266306)])
def test_rows_far_from_a_distribution(bsf8_lib, rejections, V):
    """Elements of 1 each: the mass left is nearly V 2^40 after every rejection, and what the one drafted token has
    given up, 2^40 (1 + (rejections - 1)(V - 1)) = 2^64, is more than 64 bits hold.  Nothing is left of it."""
    assert (rejections - 1) * (V - 1) + 1 == 1 << 24
    T = rejections + 1
    p, q = (torch.ones(1, T, V, device="cuda") for _ in range(2))
    p[..., 0] = 0.5
    q[..., 1:] = 0
    u = torch.full((1, T), 0.75, device="cuda")
    zeros = torch.zeros(1, T, dtype=torch.int32, device="cuda")
    for u0 in (0.0, 0.5):
        u[0, 0] = u0
        path, count, token = bsf8.verify_tree(p, zeros, zeros, u, q=q)
        assert path.tolist() == [[0] + [-1] * (T - 1)] and count.tolist() == [1]
        # the lowest x whose x elements of 1 pass u0 (V - 1)
        assert token.tolist() == [int(u0 * (V - 1)) + 1]
    assert bsf8.device_status() == 0
