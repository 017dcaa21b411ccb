"""Plain 64-bit implementations of the decode operators, written from their definitions in
include/bsf8.h (numpy and torch float64; nothing of the library)."""
import math

import numpy as np
import torch

ONE = 1 << 40


def e4m3_values():
    """Value of each of the 256 e4m3 codes."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if (c & 127) == 127:
            x = math.nan
        v[c] = -x if c & 128 else x
    return v


TABLE = e4m3_values()


def decode(codes, exps):
    """float64 values of uint8 codes [..., D] with exponent bytes [..., D / 32] (numpy)."""
    with np.errstate(invalid="ignore"):
        scale = np.where(exps == 255, np.inf, 2.0 ** (exps.astype(np.float64) - 127))
        return TABLE[codes] * np.repeat(scale, 32, axis=-1)


def block_exponents(x):
    """Exponent byte of each 32-channel block: the smallest e >= -127 with 448 * 2^e >= amax."""
    amax = np.abs(x.reshape(*x.shape[:-1], -1, 32)).max(-1)
    e = np.full(amax.shape, -127)
    for i in np.ndindex(amax.shape):
        if not np.isfinite(amax[i]):
            e[i] = 128
            continue
        while 448.0 * 2.0 ** float(e[i]) < amax[i]:
            e[i] += 1 if e[i] > -127 or amax[i] < 448.0 * 2.0 ** -120 else max(1, int(math.floor(math.log2(amax[i] / 448))) + 126)
    return (e + 127).astype(np.uint8)


def quantise(x):
    """(codes, exponent bytes) of float64 rows [..., D] that are exact in fp32."""
    e = block_exponents(x)
    y = x.reshape(*x.shape[:-1], -1, 32)
    grid = np.concatenate([TABLE[:127], TABLE[128:255]])
    order = np.argsort(grid[:127])
    mags = grid[:127][order]
    codes = np.zeros(y.shape, np.uint8)
    for i in np.ndindex(e.shape):
        if e[i] == 255:
            codes[i] = 0x7F
            continue
        z = np.abs(y[i]) / 2.0 ** (float(e[i]) - 127)
        hi = np.searchsorted(mags, z).clip(0, 126)
        lo = (hi - 1).clip(0)
        dh, dl = mags[hi] - z, z - mags[lo]
        pick = np.where((dh < dl) | ((dh == dl) & (order[hi] % 2 == 0)), hi, lo)
        codes[i] = order[pick].astype(np.uint8) | np.where(np.signbit(y[i]), 128, 0).astype(np.uint8)
    return codes.reshape(x.shape), e


def norm_rotate(x, w, cos_sin, pos, interleaved, eps):
    """float64 rows [N, heads, D]: norm by weight w (or None), then the rotation."""
    y = np.asarray(x, np.float64).copy()
    if w is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    if cos_sin is not None:
        rot = cos_sin.shape[1]
        z = y.copy()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c = cos_sin[pos, i].astype(np.float64)[:, None]
            s = cos_sin[pos, rot // 2 + i].astype(np.float64)[:, None]
            z[..., a] = y[..., a] * c - y[..., b] * s
            z[..., b] = y[..., b] * c + y[..., a] * s
        y = z
    return y


def tree(r, T, width=3):
    """Parents of a random token tree (node 0 the root) and its ancestor matrix."""
    parent = [-1] + [int(r.integers(max(0, i - 2 * width), i)) for i in range(1, T)]
    see = np.zeros((T, T), bool)
    for i in range(T):
        if i:
            see[i] = see[parent[i]]
        see[i, i] = True
    return parent, see


def mask_words(see):
    """bool [B, T, T] -> int32 [B, T, ceil(T / 32)]."""
    B, T, _ = see.shape
    W = (T + 31) // 32
    pad = np.zeros((B, T, W * 32), np.uint64)
    pad[..., :T] = see
    words = (pad.reshape(B, T, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return words.astype(np.uint32).view(np.int32)


def attention(q, k, v, see, scale):
    """One request and cache head in float64: q [R, D] rows, k and v [L, D], see [R, L].
    Returns out [R, D], lse [R], and per row: sum p |v| and the largest sum |q| |k| it sees."""
    q, k, v = (torch.as_tensor(t, dtype=torch.float64) for t in (q, k, v))
    see = torch.as_tensor(see)
    any_ = see.any(1)
    x = (q @ k.T) * scale
    x = x.masked_fill(~see, -math.inf)
    m = x.amax(1, keepdim=True).nan_to_num(neginf=0.0) if len(k) else torch.zeros(len(q), 1, dtype=torch.float64)
    p = torch.where(see, torch.exp(x - m), 0.0)
    total = p.sum(1, keepdim=True)
    pn = torch.where(any_[:, None], p / total, 0.0)
    vs = torch.where(torch.isnan(v), 0.0, v)
    out = pn @ vs
    # a NaN value reaches the rows that see it, and no others
    bad = (see.double() @ torch.isnan(v).double()) > 0
    out = torch.where(bad, math.nan, out)
    lse = torch.where(any_, (m + torch.log(total)).squeeze(1), -math.inf)
    mass = pn @ vs.abs()
    reach = ((q.abs() @ k.abs().T) * scale).masked_fill(~see, 0).amax(1) if len(k) else torch.zeros(len(q))
    return out, lse, mass, reach


def fix(p):
    return int(min(max(float(p), 0.0), 1.0) * ONE) if not math.isnan(float(p)) else 0


def verify(p, q, tok, parent, u, n):
    """One request by Python integers: p, q [T][V] (q None), returns (path, count, token)."""
    V = p.shape[1]
    U = [int(float(x) * (1 << 24)) for x in u]
    fixed = lambda row: [fix(x) for x in row]  # noqa: E731
    cur, path = 0, [0]
    R, Z = fixed(p[0]), ONE
    for i in range(1, n):
        if parent[i] != cur:
            continue
        x = tok[i]
        Q = [0] * V
        if q is None:
            Q[x] = ONE
        else:
            Q = fixed(q[cur])
        Q = [a * Z // ONE for a in Q]
        if U[i] * Q[x] // (1 << 24) < R[x]:
            cur = i
            path.append(i)
            R, Z = fixed(p[i]), ONE
        else:
            R = [max(a - b, 0) for a, b in zip(R, Q)]
            Z = sum(R)
    if sum(R) == 0:
        R = fixed(p[cur])
    at, run = U[0] * sum(R) // (1 << 24), 0
    token = V - 1
    for x in range(V):
        run += R[x]
        if run > at:
            token = x
            break
    return path + [-1] * (len(tok) - len(path)), len(path), token
