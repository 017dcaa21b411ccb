"""Plain implementations of the operators around a decode step (pages and slots, page bounds and selection,
sampling, residual with norms), written from their definitions in include/bsf8.h: whole numbers as Python
integers, values in 64 bits."""
import math

import numpy as np

from _decode_ref import decode

ONE = 1 << 40
F = np.float32


def plan(table, held, free, count, lens, add, done, page_size, tokens):
    """The books after the call and (req, slot, start, granted), by one request after another."""
    B, most = table.shape
    table, held, free = table.copy(), list(held), free.copy()
    for b in range(B):
        if done is not None and done[b]:
            for i in range(held[b]):
                free[count] = table[b, i]
                count += 1
            held[b] = 0
    req, slot, start, granted = [], [], [0], []
    top, asked, needed, taken = count, 0, 0, 0
    for b in range(B):
        n, a = int(lens[b]), int(add[b])
        if n < 0 or a < 0 or n + a > most * page_size:
            n = a = 0
        need = max(0, -(-(n + a) // page_size) - held[b]) if a > 0 else 0
        asked, needed = asked + a, needed + need
        if asked > tokens or (need and needed > top):
            need = a = 0
        for _ in range(need):
            table[b, held[b]] = free[top - 1 - taken]
            held[b] += 1
            taken += 1
        req += [b] * a
        slot += range(n, n + a)
        start.append(start[-1] + a)
        granted.append(a)
    pad = tokens - len(req)
    return dict(table=table, held=np.array(held), free=free, count=top - taken, req=np.array(req + [0] * pad),
                slot=np.array(slot + [-1] * pad), start=np.array(start), granted=np.array(granted))


def bounds(codes, exps):
    """Bounds of pages [n, heads, page, D]: int8 codes [n, heads, 2, D], bytes [n, heads, D / 32]."""
    k = decode(codes, exps)
    n, H, _, D = k.shape
    out, byte = np.zeros((n, H, 2, D), np.int8), np.zeros((n, H, D // 32), np.uint8)
    for i in np.ndindex(n, H, D // 32):
        x = k[i[0], i[1], :, 32 * i[2]:32 * i[2] + 32]
        if (exps[i[0], i[1], :, i[2]] == 255).any() or not np.abs(x).max() < 2.0 ** 128:
            byte[i] = 255
            continue
        a = np.abs(x).max()
        e = max(-127, math.frexp(a / 127)[1] - 2 if a else -127)
        while 127 * 2.0 ** e < a:
            e += 1
        byte[i] = e + 127
        out[i[0], i[1], 0, 32 * i[2]:32 * i[2] + 32] = np.ceil(x.max(0) / 2.0 ** e)
        out[i[0], i[1], 1, 32 * i[2]:32 * i[2] + 32] = np.floor(x.min(0) / 2.0 ** e)
    return out, byte


def query_sums(q):
    """Integer sums [2][D] of the rows' positive and negative parts; q float64 [R, D]."""
    q = np.where(np.isfinite(q), q, 0.0)
    a = np.abs(q).max() if q.size else 0.0
    k = max(-100, math.frexp(a)[1] - 1 if a > 0 else -100)
    n = np.rint(q * 2.0 ** (17 - k)).astype(np.int64)
    up, dn = n.clip(min=0).sum(0), n.clip(max=0).sum(0)
    s = max(0, int(max(up.max(), -dn.min())).bit_length() - 14)
    r = (1 << s) >> 1
    return (up + r) >> s, (dn + r) >> s


def scores(q, codes, exps):
    """fp32 scores of pages from codes [n, 2, D] and bytes [n, D / 32] of one head."""
    up, dn = query_sums(q)
    with np.errstate(over="ignore"):
        S = (codes[:, 0].astype(np.int64) * up + codes[:, 1].astype(np.int64) * dn).reshape(len(codes), -1, 32).sum(-1)
    f = (S.astype(F) * F(2.0 ** -27)) * np.ldexp(F(1), np.minimum(exps.astype(int), 254) - 127).astype(F)
    f = np.where(exps == 255, F(np.inf), f)
    while f.shape[1] > 1:
        f = f[:, 0::2] + f[:, 1::2]
    return f[:, 0]


def select(q, codes, exps, table, ctx, nodes, page_size, keep, sink, recent, width):
    """(pages [heads][width], kept) of one request; q float64 [T, Hq, D]."""
    Hkv, D = codes.shape[1], codes.shape[3]
    g = q.shape[1] // Hkv
    full = ctx // page_size
    n = min(keep, full)
    out = np.full((Hkv, width), -1)
    for h in range(Hkv):
        best = np.arange(full)
        if full > keep:
            f = scores(q[:nodes, h * g:(h + 1) * g].reshape(-1, D), codes[table[:full], h], exps[table[:full], h])
            f[:sink] = np.inf
            f[full - recent:] = np.inf
            best = np.sort(np.lexsort((np.arange(full), -f.astype(np.float64)))[:keep])
        tail = np.arange(full, -(-(ctx + nodes) // page_size))
        at = np.concatenate([best, tail])
        out[h, :len(at)] = table[at]
    return out, n * page_size + ctx % page_size


EXP2 = [F(c) for c in (-0.0009449035860598087, 0.00920579768717289, -0.0552973598241806, 0.2401801496744156,
                       -0.6931437253952026, 1.0)]


def weights(x, t):
    """Python integers: the weights of a row of logits (float32)."""
    x = np.where(np.isnan(x), F(-np.inf), x.astype(F))
    top = x.max()
    w = np.zeros(len(x), np.int64)
    if top == -np.inf:
        return w, x
    with np.errstate(all="ignore"):
        rate = F(1.4426950408889634) / F(t) if t > 0 else F(np.inf)
        y = (top - x) * rate
        y = np.where(x == top, F(0), y)
        near = y <= 40
        n = np.floor(np.where(near, y, 0)).astype(F)
        f = np.where(near, y, 0).astype(F) - n
        p = np.full(len(x), EXP2[0])
        for c in EXP2[1:]:
            p = (p * f).astype(F)
            p = (p + c).astype(F)
        w = ((p * F(1 << 24)).astype(np.int64) << 16) >> n.astype(np.int64)
    return np.where(near, w, 0), x


def kept(x, t=1.0, k=0, tp=1.0, mp=0.0):
    """Weights of the tokens that stay (0 for the others)."""
    w, x = weights(x, t)
    order = np.lexsort((np.arange(len(x)), -x.astype(np.float64)))
    v = w[order]
    if k <= 0 or k > len(x):
        k = len(x)
    if not t >= 2.0 ** -126:
        k = 1
    v[k:] = 0
    least = max(1, math.ceil((min(max(float(F(mp)), 0.0), 1.0) if mp == mp else 0.0) * ONE))
    v = np.where(v >= least, v, 0)
    if tp < 1:
        total = sum(int(a) for a in v)
        cut = max(1, int(max(float(F(tp)), 0.0) * (1 << 24)) * total >> 24)
        v = np.where(np.cumsum(v) - v < cut, v, 0)
    out = np.zeros(len(x), np.int64)
    out[order] = v
    return out


def draw(w, u):
    """The token that u picks from the weights, -1 where there are none."""
    total = int(w.sum())
    if total == 0:
        return -1
    u = min(max(float(u), 0.0), 1 - 2.0 ** -24) if u == u else 0.0
    return int(np.searchsorted(np.cumsum(w), int(u * (1 << 24)) * total >> 24, side="right"))


def norm(x, residual, weight, post, gate, scale, eps):
    """float64 (h, r) and, for r, the sum of the magnitudes that go into it."""
    z = x
    if post is not None:
        z = z / np.sqrt((z ** 2).mean(-1, keepdims=True) + eps) * post
    if gate is not None:
        z = z * gate
    r = residual + scale * z
    mass = np.abs(residual) + np.abs(scale * z)
    with np.errstate(invalid="ignore", divide="ignore"):
        k = 1 / np.sqrt((r ** 2).mean(-1, keepdims=True) + eps)
    return r * k * weight, r, mass, k * np.abs(weight)
