"""The workloads that the decode operators are timed and checked on: cache append, cache read,
tree attention, draft verification and cache commit.

Each case is one call of a speculative decoding step (or of the prompt pass before it) over a paged
cache whose keys and values are kept as e4m3 codes with one power-of-two exponent byte per 32 channels.
`run` computes a case with elementary torch operations in 32 bits (`own` false) or with this
package's kernels (`own` true); `exact` computes it in 64 bits, written apart from both.
"""
import math
import random

import numpy as np
import torch

own = False

ONE = 1 << 40  # a probability of 1 in the fixed point that the verification is defined in


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # --- qkv_append, then the written rows read back (what a prompt's own attention reads)
        # a verify pass of seven requests, nine nodes each: small, its latency counts
        dict(name="append-verify", op="append", B=7, T=9, Hq=32, Hkv=8, D=128, page=16, rot=128, inter=False, norm=True),
        # a long prompt of one request, cut by no round number
        dict(name="append-prompt", op="append", B=1, T=8191, Hq=32, Hkv=8, D=128, page=64, rot=64, inter=True, norm=True),
        # --- kv_read: a short prefix; a long context handed to another engine
        dict(name="read-short", op="read", N=257, B=3, Hkv=4, D=64, page=16),
        dict(name="read-long", op="read", N=65536, B=9, Hkv=8, D=128, page=32),
        # --- tree_attention
        # one user, one token: the smallest call
        dict(name="decode-one", op="attention", B=1, T=1, Hq=32, Hkv=8, D=128, page=16, ctx=1000, tree=False),
        # a full batch of single tokens with contexts of every length
        dict(name="decode-batch", op="attention", B=64, T=1, Hq=32, Hkv=8, D=128, page=64, ctx=16384, tree=False),
        # drafted trees for a few users: 23 nodes, 7 query heads a cache head
        dict(name="tree-ragged", op="attention", B=16, T=23, Hq=28, Hkv=4, D=128, page=16, ctx=8192, tree=True),
        # big trees over very long contexts: the products weigh most
        dict(name="tree-long", op="attention", B=2, T=64, Hq=32, Hkv=4, D=128, page=64, ctx=131072, tree=True),
        # --- verify_tree: a chain for one user (odd vocabulary); trees for a full batch
        dict(name="verify-chain", op="verify", B=1, T=6, V=50257, q=True, width=1),
        dict(name="verify-batch", op="verify", B=64, T=16, V=131072, q=True, width=3),
        # --- kv_commit: the kept nodes of one layer
        dict(name="commit-one", op="commit", B=1, T=8, Hkv=8, D=128, page=16, ctx=300),
        dict(name="commit-batch", op="commit", B=192, T=64, Hkv=8, D=128, page=64, ctx=400),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention", "attention", "verify", "commit"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "append":
        group = rng.choice([1, 3, 4, 7, 8])
        B = _log(rng, 1, 48)
        most = max(1, 8191 * 40 * 128 // (Hkv * (group + 2) * D * B))
        return dict(op=op, B=B, T=_log(rng, 1, min(most, 6000)), Hq=Hkv * group, Hkv=Hkv, D=D, page=page,
                    rot=rng.choice([0, 32, D // 2, D]), inter=rng.random() < 0.5, norm=rng.random() < 0.7)
    if op == "read":
        return dict(op=op, N=_log(rng, 1, 65536 * 8 * 128 // (Hkv * D)), B=rng.randint(1, 30), Hkv=Hkv, D=D, page=page)
    if op == "attention":
        group = rng.choice([1, 2, 4, 5, 8, 16])
        T = rng.choice([1, 1, rng.randint(2, 16), rng.randint(17, 64)])
        B = _log(rng, 1, 64)
        # at most the bytes of decode-batch and the products of tree-long
        most = min(64 * 9000 * 8 * 128 // (B * Hkv * D), 2 * 64 * 32 * 128 * 131072 // (B * T * Hkv * group * D))
        return dict(op=op, B=B, T=T, Hq=Hkv * group, Hkv=Hkv, D=D, page=page,
                    ctx=_log(rng, 1, max(2, min(most, 131072))), tree=T > 1 and rng.random() < 0.7)
    if op == "verify":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, T=rng.randint(1, 16), V=_log(rng, 1000, 131072), q=rng.random() < 0.7,
                    width=rng.choice([1, 2, 3]))
    return dict(op=op, B=_log(rng, 1, 192), T=rng.randint(1, 64), Hkv=Hkv, D=min(D, 128), page=page, ctx=_log(rng, 1, 400))


# ------------------------------------------------------------------------------------ inputs

def _block_exponent(amax):
    """Exponent byte of a 32-channel block: e + 127 with the smallest e >= -127 that has 448 * 2^e >= amax."""
    return ((amax.view(torch.int32) + 0x1FFFFF) >> 23).sub(8).clamp_(0, 254)


def _power(e):
    """2^(e - 127) of exponent bytes, as fp32 (byte 0 is the subnormal 2^-127)."""
    return (e.to(torch.int32) << 23).clamp_(min=0x400000).view(torch.float32)


def _quantise(x):
    """fp32 [..., D] -> e4m3 codes (uint8) and exponent bytes [..., D / 32]."""
    y = x.unflatten(-1, (-1, 32))
    e = _block_exponent(y.abs().amax(-1))
    codes = (y * _power(254 - e).unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.flatten(-2), e.to(torch.uint8)


def _decode(codes, exps):
    """The fp32 values that codes and exponent bytes stand for."""
    y = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
    return (y * _power(exps).unsqueeze(-1)).flatten(-2)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _pool(g, lens, page, Hkv, D, most=0):
    """A cache for requests of `lens` tokens (or of `most` each), its pages handed out in random order, and
    its block table."""
    need = [max(1, -(-n // page)) for n in lens]
    pages = max(sum(need), len(lens) * -(-most // page))
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32, device="cuda")
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    # a few channels are several times larger than the others, as keys' channels are
    gain = 1 + 5 * (torch.rand((Hkv, 1, D), generator=g, device="cuda") > 0.96)
    data = []
    for s in (gain, 1.0):
        k8 = torch.empty((pages, Hkv, page, D), dtype=torch.uint8, device="cuda")
        ke = torch.empty((pages, Hkv, page, D // 32), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 27) // (Hkv * page * D))
        for i in range(0, pages, step):
            x = torch.randn((min(step, pages - i), Hkv, page, D), generator=g, device="cuda")
            x = (x * s).to(torch.bfloat16).float()
            k8[i:i + step], ke[i:i + step] = _quantise(x)
        data += [k8, ke]
    return data, table


def _tree(r, T, width):
    """A token tree: each node's parent comes before it and has at most `width` children; node 0 is the root."""
    parent, kids = [-1], [0] * T
    for i in range(1, T):
        open_ = [j for j in range(max(0, i - 2 * width), i) if kids[j] < width]
        j = r.choice(open_) if open_ else i - 1
        kids[j] += 1
        parent.append(j)
    return parent


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c, r, g = dict(case), random.Random(seed), _gen(seed)
    s = {"op": c["op"], "case": c}
    bf = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    if c["op"] == "append":
        B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
        ctx = [r.randint(0, 300) for _ in range(B)]
        s["cache"], s["table"] = _pool(g, [n + T for n in ctx], c["page"], Hkv, D)
        # the projection's output: q, k and v of a token side by side
        x = bf(B * T, (Hq + 2 * Hkv) * D) * 2
        s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
        s["req"] = torch.arange(B, device="cuda", dtype=torch.int32).repeat_interleave(T)
        s["slot"] = (_ints(ctx)[:, None] + torch.arange(T, device="cuda", dtype=torch.int32)).flatten()
        # a node's position is its depth, shared by its siblings; a prompt's tokens follow each other
        if T <= 64:
            depth = []
            for _ in range(B):
                parent, d = _tree(r, T, 2), [0] * T
                for i in range(1, T):
                    d[i] = d[parent[i]] + 1
                depth += d
            s["pos"] = (_ints(ctx).repeat_interleave(T) + _ints(depth)).to(torch.int32)
        else:
            s["pos"] = s["slot"].clone()
        s["qn"] = s["kn"] = s["cs"] = None
        if c["norm"]:
            s["qn"], s["kn"] = (1 + 0.2 * bf(D)), (1 + 0.2 * bf(D))
        if c["rot"]:
            h = c["rot"] // 2
            f = 10000.0 ** (-torch.arange(h, device="cuda", dtype=torch.float32) / h)
            a = torch.arange(301 + T, device="cuda", dtype=torch.float32)[:, None] * f
            s["cs"] = torch.cat([a.cos(), a.sin()], 1)
    elif c["op"] == "read":
        N, B = c["N"], c["B"]
        per = [N // B + (i < N % B) for i in range(B)]
        s["cache"], s["table"] = _pool(g, [max(1, n) for n in per], c["page"], c["Hkv"], c["D"])
        s["req"] = torch.repeat_interleave(torch.arange(B, device="cuda", dtype=torch.int32), _ints(per))
        s["slot"] = torch.cat([torch.arange(n, device="cuda", dtype=torch.int32) for n in per])
    elif c["op"] == "attention":
        B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
        ctx = [c["ctx"] if B <= 2 else r.randint(1, c["ctx"]) for _ in range(B)]
        nodes = [T if B == 1 or T == 1 else r.randint(max(1, T // 2), T) for _ in range(B)]
        s["cache"], s["table"] = _pool(g, [n + T for n in ctx], c["page"], Hkv, D)
        s["q"] = bf(B, T, Hq, D) * 1.5
        s["ctx"], s["nodes"], s["max_len"] = _ints(ctx), _ints(nodes), max(ctx) + T
        s["mask"] = None
        if c["tree"]:
            W = -(-T // 32)
            m = np.zeros((B, T, W), np.uint32)
            for b in range(B):
                parent = _tree(r, T, 3)
                for i in range(T):
                    if i:
                        m[b, i] = m[b, parent[i]]
                    m[b, i, i // 32] |= np.uint32(1 << (i % 32))
            s["mask"] = torch.from_numpy(m.view(np.int32)).cuda()
    elif c["op"] == "verify":
        B, T, V = c["B"], c["T"], c["V"]
        base = torch.randn((B, T, V), generator=g, device="cuda") * 2.5
        s["p"] = torch.softmax(base, -1)
        # the draft model's probabilities are near the target's
        base += 0.7 * torch.randn((B, T, V), generator=g, device="cuda")
        q = torch.softmax(base, -1)
        del base
        parent = _ints([_tree(r, T, c["width"]) for _ in range(B)])
        s["parent"], s["nodes"] = parent, _ints([r.randint((T + 1) // 2, T) for _ in range(B)])
        # a node's token is drawn from its parent's row of the draft; node 0 is the last token kept
        at = (torch.rand((B, T), generator=g, device="cuda") * 0.999).unsqueeze(-1)
        tok = torch.zeros((B, T), dtype=torch.int32, device="cuda")
        for b in range(B):
            cum = q[b].double().cumsum(-1)[parent[b].clamp(min=0).long()].float()
            tok[b] = torch.searchsorted(cum, at[b]).squeeze(-1).clamp(max=V - 1).to(torch.int32)
        s["tok"], s["q"] = tok, q if c["q"] else None
        s["u"] = torch.rand((B, T), generator=g, device="cuda")
    else:
        B, T = c["B"], c["T"]
        ctx = [r.randint(max(0, c["ctx"] // 2), c["ctx"]) for _ in range(B)]
        s["cache"], s["table"] = _pool(g, [n + T for n in ctx], c["page"], c["Hkv"], c["D"], c["ctx"] + T)
        path, count = [], []
        for _ in range(B):
            # a way from the root down a tree
            way = [0] + sorted(r.sample(range(1, T), min(T - 1, r.randint(0, 7))))
            count.append(len(way))
            path.append(way + [-1] * (T - len(way)))
        s["ctx"], s["path"], s["count"] = _ints(ctx), _ints(path), _ints(count)
    return s


# ------------------------------------------------------------------------------------ plain forms

def _rows(s, req, slot):
    """Page and offset of (request, slot) pairs."""
    page = s["cache"][0].shape[2]
    return s["table"][req.long(), (slot // page).long()].long(), (slot % page).long()


def _norm_rotate(x, w, cs, pos, inter, eps=1e-6):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + eps) * w.float()
    if cs is None:
        return y
    rot = cs.shape[1]
    cos, sin = (t.unsqueeze(1) for t in cs[pos.long()].chunk(2, -1))
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., :rot // 2], y[..., rot // 2:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _plain_append(s):
    inter = s["case"]["inter"]
    k8, ke, v8, ve = s["cache"]
    q = _norm_rotate(s["q"], s["qn"], s["cs"], s["pos"], inter).to(torch.bfloat16)
    k = _norm_rotate(s["k"], s["kn"], s["cs"], s["pos"], inter)
    page, off = _rows(s, s["req"], s["slot"])
    k8[page, :, off], ke[page, :, off] = _quantise(k)
    v8[page, :, off], ve[page, :, off] = _quantise(s["v"].float())
    k, v = _plain_read(s)
    return {"q": q, "k": k, "v": v}


def _plain_read(s):
    k8, ke, v8, ve = s["cache"]
    page, off = _rows(s, s["req"], s["slot"])
    k = _decode(k8[page, :, off], ke[page, :, off])
    v = _decode(v8[page, :, off], ve[page, :, off])
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _plain_attention(s):
    k8, ke, v8, ve = s["cache"]
    q, ctx, nodes = s["q"], s["ctx"], s["nodes"]
    B, T, Hq, D = q.shape
    Hkv, page = k8.shape[1], k8.shape[2]
    n = -(-s["max_len"] // page)
    pages = s["table"][:, :n].long()
    gather = lambda t: t[pages].transpose(1, 2).flatten(2, 3)  # noqa: E731   [B, Hkv, n * page, ...]
    L = n * page
    at = torch.arange(L, device=q.device)
    j = at - ctx[:, None]                                        # the node a slot holds, negative: context
    if s["mask"] is None:
        tree = j[:, None, :] <= torch.arange(T, device=q.device)[:, None]
    else:
        bits = (s["mask"].unsqueeze(-1) >> torch.arange(32, device=q.device)) & 1
        bits = bits.flatten(2)[..., :T]
        tree = bits.gather(2, j.clamp(0, T - 1)[:, None, :].expand(B, T, L)) > 0
    seen = (j < 0)[:, None, :] | (tree & (j < nodes[:, None])[:, None, :])
    seen &= (torch.arange(T, device=q.device) < nodes[:, None])[:, :, None]
    qf = q.float().view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [B, Hkv, T * g, D]
    x = torch.matmul(qf, _decode(gather(k8), gather(ke)).transpose(-1, -2)) * (1 / math.sqrt(D))
    x = x.unflatten(2, (T, -1)).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m.masked_fill(m == -math.inf, 0)).exp_().flatten(2, 3)
    y = torch.matmul(x, _decode(gather(v8), gather(ve)))
    total = x.sum(-1, keepdim=True)
    y = y / total.masked_fill(total == 0, 1)
    return y.unflatten(2, (T, -1)).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(torch.bfloat16)


def _fix(p):
    return (p.clamp(0, 1) * float(ONE)).long()


def _times(a, z):
    """floor(a * z / 2^40) for a <= 2^40 and z < 2^42."""
    return (a * (z >> 20) + ((a * (z & 0xFFFFF)) >> 20)) >> 20


def _part(u, z):
    """floor(u * z / 2^24) for u < 2^24."""
    return (z >> 24) * u + (((z & 0xFFFFFF) * u) >> 24)


def _plain_verify(s):
    p, q, tok, parent, nodes = s["p"], s["q"], s["tok"].long(), s["parent"], s["nodes"]
    B, T, V = p.shape
    U = (s["u"] * float(1 << 24)).long()
    b = torch.arange(B, device=p.device)
    cur = torch.zeros(B, dtype=torch.int64, device=p.device)
    count = torch.ones(B, dtype=torch.int64, device=p.device)
    path = torch.full((B, T + 1), -1, dtype=torch.int64, device=p.device)
    path[:, 0] = 0
    R, Z = _fix(p[:, 0]), torch.full((B,), ONE, dtype=torch.int64, device=p.device)
    # the walk goes from node to node; all requests take a step at once
    for i in range(1, T):
        asked = (parent[:, i] == cur) & (i < nodes)
        x = tok[:, i:i + 1]
        Q = torch.zeros_like(R).scatter_(1, x, ONE) if q is None else _fix(q[b, cur])
        Q = _times(Q, Z[:, None])
        yes = asked & (_part(U[:, i:i + 1], Q.gather(1, x)) < R.gather(1, x)).squeeze(1)
        no = asked & ~yes
        R = torch.where(no[:, None], (R - Q).clamp(min=0), R)
        R = torch.where(yes[:, None], _fix(p[:, i]), R)
        Z = torch.where(yes, ONE, torch.where(no, R.sum(1), Z))
        cur = torch.where(yes, i, cur)
        path[b, torch.where(yes, count, T)] = i
        count = count + yes
    total = R.sum(1, keepdim=True)
    R = torch.where(total > 0, R, _fix(p[b, cur]))
    cum = R.cumsum(1)
    at = _part(U[:, :1], cum[:, -1:])
    token = (cum <= at).sum(1).clamp(max=V - 1)
    path = torch.where(torch.arange(T, device=p.device) < count[:, None], path[:, :T], -1)
    return {"path": path.to(torch.int32), "count": count.to(torch.int32), "token": token.to(torch.int32)}


def _held(s):
    """The cache's codes, as the numbers they are, and its exponent bytes."""
    k8, ke, v8, ve = s["cache"]
    return [k8.view(torch.float8_e4m3fn), ke, v8.view(torch.float8_e4m3fn), ve]


def _plain_commit(s):
    B, T = s["path"].shape
    i = torch.minimum(torch.arange(T, device="cuda", dtype=torch.int32), s["count"][:, None] - 1)
    req = torch.arange(B, device="cuda").repeat_interleave(T)
    src = _rows(s, req, (s["ctx"][:, None] + s["path"].gather(1, i.long())).flatten())
    dst = _rows(s, req, (s["ctx"][:, None] + i).flatten())
    for t in s["cache"]:
        t[dst[0], :, dst[1]] = t[src[0], :, src[1]]
    return _held(s)


def run(s):
    if not own:
        return {"append": _plain_append, "read": _plain_read, "attention": _plain_attention,
                "verify": _plain_verify, "commit": _plain_commit}[s["op"]](s)
    import block_scaled_fp8_weight_gb300 as bsf8
    op = s["op"]
    if op == "verify":
        path, count, token = bsf8.verify_tree(s["p"], s["tok"], s["parent"], s["u"], q=s["q"], nodes=s["nodes"])
        return {"path": path, "count": count, "token": token}
    cache = bsf8.KVCache(*s["cache"])
    if op == "append":
        q = bsf8.qkv_append(s["q"], s["k"], s["v"], cache, s["table"], s["req"], s["slot"], pos=s["pos"],
                            q_norm=s["qn"], k_norm=s["kn"], cos_sin=s["cs"], interleaved=s["case"]["inter"])
        k, v = bsf8.kv_read(cache, s["table"], s["req"], s["slot"])
        return {"q": q, "k": k, "v": v}
    if op == "read":
        return bsf8.kv_read(cache, s["table"], s["req"], s["slot"])
    if op == "attention":
        return bsf8.tree_attention(s["q"], cache, s["table"], s["ctx"], nodes=s["nodes"], mask=s["mask"],
                                   max_len=s["max_len"])
    bsf8.kv_commit(cache, s["table"], s["ctx"], s["path"], s["count"])
    return _held(s)


# ------------------------------------------------------------------------------------ work

def work(case):
    c = case
    row = lambda heads, byte: heads * c["D"] * byte  # noqa: E731
    held = 1 + 1 / 32  # bytes a cached value
    if c["op"] == "append":
        n = c["B"] * c["T"]
        b = row(c["Hq"], 4) + 2 * row(c["Hkv"], 2 + held) + 2 * row(c["Hkv"], held + 2) + 12
        return {"bytes": n * (b + 4 * c["rot"]), "flops": 10 * n * (c["Hq"] + 2 * c["Hkv"]) * c["D"]}
    if c["op"] == "read":
        return {"bytes": c["N"] * (2 * row(c["Hkv"], held + 2) + 8), "flops": 2 * c["N"] * c["Hkv"] * c["D"]}
    if c["op"] == "attention":
        # contexts are uniform in 1 .. ctx past two requests, nodes in T/2 .. T
        mean = c["ctx"] if c["B"] <= 2 else (c["ctx"] + 1) / 2
        t = c["T"] if c["B"] == 1 or c["T"] == 1 else (max(1, c["T"] // 2) + c["T"]) / 2
        keys = c["B"] * (mean + t)
        return {"bytes": keys * 2 * row(c["Hkv"], held) + c["B"] * c["T"] * row(c["Hq"], 4),
                "flops": 4 * keys * t * c["Hq"] * c["D"]}
    if c["op"] == "verify":
        # one row of the target a request, and of the draft's where it has one
        return {"bytes": c["B"] * (c["V"] * 4 * (2 if c["q"] else 1) + 20 * c["T"]), "flops": 4 * c["B"] * c["V"]}
    kept = 1 + min(c["T"] - 1, 7) / 2
    return {"bytes": c["B"] * (4 * c["T"] + 2 * kept * 2 * row(c["Hkv"], held)), "flops": 0}


# ------------------------------------------------------------------------------------ 64 bits

def _value(code, exp):
    """What e4m3 codes with exponent bytes stand for, in 64 bits, from the formats' definitions."""
    c = code.to(torch.int64)
    sign, e, m = 1 - 2 * (c >> 7), (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2((e - 7).double()))
    scale = torch.exp2(exp.double() - 127).repeat_interleave(32, -1)
    return sign * mag * scale


def _exact_append(s, c):
    """Keys and values are held against what they are before their codes are rounded: the codes' own
    rounding is a part of either side's error."""
    def turn(x, w):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.double()
        R = c["rot"]
        if R:
            z = y.clone()
            for i in range(R // 2):
                a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, i + R // 2)
                co = s["cs"][s["pos"].long(), i].double()[:, None]
                si = s["cs"][s["pos"].long(), i + R // 2].double()[:, None]
                z[..., a] = y[..., a] * co - y[..., b] * si
                z[..., b] = y[..., a] * si + y[..., b] * co
            y = z
        return y
    return {"q": turn(s["q"], s["qn"]), "k": turn(s["k"], s["kn"]), "v": s["v"].double()}


def _exact_read(s, c):
    P = c["page"]
    req, slot = s["req"].long(), s["slot"].long()
    page = s["table"][req, slot // P].long()
    k8, ke, v8, ve = s["cache"]
    out = []
    for code, exp in ((k8, ke), (v8, ve)):
        flat, fe = code.transpose(1, 2).flatten(0, 1), exp.transpose(1, 2).flatten(0, 1)
        out.append(_value(flat[page * P + slot % P], fe[page * P + slot % P]))
    return tuple(out)


def _exact_attention(s, c):
    B, T, Hq, D = s["q"].shape
    Hkv, P, G = c["Hkv"], c["page"], Hq // c["Hkv"]
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    k8, ke, v8, ve = s["cache"]
    mask = None if s["mask"] is None else s["mask"].cpu().numpy().view(np.uint32)
    for b in range(B):
        n, t = int(s["ctx"][b]), int(s["nodes"][b])
        pages = s["table"][b, :-(-(n + t) // P)].long()
        see = np.ones((t, n + t), bool)
        for i in range(t):
            for j in range(t):
                see[i, n + j] = j <= i if mask is None else bool(mask[b, i, j // 32] >> np.uint32(j % 32) & np.uint32(1))
        see = torch.from_numpy(see).cuda()
        for h in range(Hkv):
            k = _value(k8[pages, h].flatten(0, 1)[:n + t], ke[pages, h].flatten(0, 1)[:n + t])
            v = _value(v8[pages, h].flatten(0, 1)[:n + t], ve[pages, h].flatten(0, 1)[:n + t])
            for g in range(G):
                x = s["q"][b, :t, h * G + g].double() @ k.T / D ** 0.5
                x[~see] = -math.inf
                out[b, :t, h * G + g] = torch.softmax(x, -1) @ v
    return out


def _exact_commit(s, c):
    P = c["page"]
    table, path = s["table"].cpu().numpy(), s["path"].cpu().numpy()
    held = [t.clone() for t in s["cache"]]
    for b in range(c["B"]):
        n = int(s["ctx"][b])
        for i in range(int(s["count"][b])):
            a, z = n + int(path[b, i]), n + i
            for old, new in zip(s["cache"], held):
                new[table[b, z // P], :, z % P] = old[table[b, a // P], :, a % P]
    plain = torch.full_like(held[1], 127)  # the codes' own values
    return [_value(held[0], plain), held[1], _value(held[2], plain), held[3]]


def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers, defined in integers
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attention": _exact_attention,
            "commit": _exact_commit}[case["op"]](s, case)
