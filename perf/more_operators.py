"""The workloads that the second set of decode operators is timed and checked on: page and slot plans,
page bounds, attention over selected pages, sampling and processed distributions, residual with norms.

Each case is one call of a decode step (or of the prompt pass before it).  `run` computes a case with
elementary torch operations in 32 bits, or in integers where the operator is defined in integers (`own`
false), or with this package's kernels (`own` true); `exact` computes it in 64 bits, written apart from
both.
"""
import math
import random

import numpy as np
import torch

own = False

ONE = 1 << 40  # the weight of a row's largest logit
LOG2E = 1.4426950408889634
# 2^-f on [0, 1), fitted to it by least squares reweighted towards the largest relative error
EXP2 = (-0.6931437253952026, 0.2401801496744156, -0.0552973598241806, 0.00920579768717289, -0.0009449035860598087)


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # --- kv_plan: a verify pass of seven requests, nine nodes each (rarely a page is taken);
        dict(name="plan-verify", op="plan", B=7, page=16, most=9, long=0, ctx=300, done=0.0),
        # a full batch, half of it leaving, prompts coming in their place beside single tokens
        dict(name="plan-batch", op="plan", B=1024, page=16, most=1, long=700, ctx=2000, done=0.5),
        # --- kv_bounds: single tokens of a batch, of which a few fill their page; a long prompt
        dict(name="bounds-step", op="bounds", B=64, Hkv=8, D=128, page=64, ctx=1000, add=1),
        dict(name="bounds-prompt", op="bounds", B=3, Hkv=8, D=128, page=64, ctx=0, add=21843),
        # --- select_pages, then sparse_attention over what it gives: one user with a long context
        dict(name="sparse-one", op="sparse", B=1, T=1, Hq=32, Hkv=8, D=128, page=64, ctx=131072, keep=64, tree=False),
        # a batch of single tokens, contexts of every length
        dict(name="sparse-batch", op="sparse", B=32, T=1, Hq=32, Hkv=8, D=128, page=64, ctx=65536, keep=48, tree=False),
        # drafted trees, small pages, 7 query heads a cache head
        dict(name="sparse-tree", op="sparse", B=5, T=13, Hq=28, Hkv=4, D=128, page=32, ctx=40000, keep=100, tree=True),
        # --- sample_tokens: one user's token (odd vocabulary); a batch whose requests ask for different things
        dict(name="sample-one", op="sample", N=1, V=50257, bf16=False, how="k+p"),
        dict(name="sample-batch", op="sample", N=192, V=131072, bf16=True, how="mixed"),
        # --- token_probs: what draft verification takes, for trees of six nodes of eight requests
        dict(name="probs-trees", op="probs", N=48, V=131072, bf16=False, how="mixed"),
        # --- residual_norm: a verify pass's rows; a prompt's
        dict(name="norm-verify", op="norm", M=6, H=5120, gate="none", post=False, fp32=False),
        dict(name="norm-prompt", op="norm", M=8191, H=5120, gate="channel", post=True, fp32=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "bounds", "sparse", "sparse", "sample", "sample", "probs", "norm"])
    D, Hkv, page = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 3, 4, 8]), rng.choice([16, 32, 48, 64, 128])
    if op == "plan":
        return dict(op=op, B=_log(rng, 1, 1024), page=page, most=rng.choice([1, 1, rng.randint(2, 64)]),
                    long=rng.choice([0, _log(rng, 10, 700)]), ctx=_log(rng, 16, 2000), done=rng.choice([0.0, 0.1, 0.5, 1.0]))
    if op == "bounds":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, Hkv=Hkv, D=D, page=page, ctx=_log(rng, 1, 1000),
                    add=_log(rng, 1, max(2, 65529 * 8 * 128 // (B * Hkv * D))))
    if op == "sparse":
        group, T, B = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 1, rng.randint(2, 32)]), _log(rng, 1, 32)
        most = 32 * 32768 * 8 * 128 // (B * Hkv * D)
        ctx = _log(rng, 1, min(131072, most))
        return dict(op=op, B=B, T=T, Hq=Hkv * group, Hkv=Hkv, D=D, page=page, ctx=ctx,
                    keep=max(3, min(_log(rng, 3, 200), 4096 // page * 2)), tree=T > 1 and rng.random() < 0.7)
    if op in ("sample", "probs"):
        V = _log(rng, 1000, 131072)
        return dict(op=op, N=_log(rng, 1, (192 if op == "sample" else 48) * 131072 // V if V > 32768 else 192), V=V,
                    bf16=rng.random() < 0.5, how=rng.choice(["plain", "greedy", "k", "p", "k+p", "min", "mixed", "mixed"]))
    H = 8 * _log(rng, 8, 2048)
    return dict(op=op, M=_log(rng, 1, max(2, min(16384, 8191 * 5120 // H))), H=H, fp32=rng.random() < 0.5, post=rng.random() < 0.5,
                gate=rng.choice(["none", "channel", "token", "full"]))


# ------------------------------------------------------------------------------------ inputs

def _power(e):
    """2^(e - 127) of exponent bytes, as fp32 (byte 0 is the subnormal 2^-127)."""
    return (e.to(torch.int32) << 23).clamp_(min=0x400000).view(torch.float32)


def _quantise(x):
    """fp32 [..., D] -> e4m3 codes (uint8) and exponent bytes [..., D / 32]: the smallest e >= -127 with 448 * 2^e >= amax."""
    y = x.unflatten(-1, (-1, 32))
    e = ((y.abs().amax(-1).view(torch.int32) + 0x1FFFFF) >> 23).sub(8).clamp_(0, 254)
    codes = (y * _power(254 - e).unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.flatten(-2), e.to(torch.uint8)


def _decode(codes, exps):
    """The fp32 values that codes and exponent bytes stand for."""
    y = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
    return (y * _power(exps).unsqueeze(-1)).flatten(-2)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pool(g, lens, page, Hkv, D, most=0):
    """A cache for requests of `lens` tokens (or of `most` each), its pages handed out in random order, and its block table."""
    need = [max(1, -(-n // page)) for n in lens]
    pages = max(sum(need), len(lens) * -(-most // page))
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32, device="cuda")
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    # a few channels of the keys are several times larger than the others; a page's keys have something in common
    gain = 1 + 5 * (torch.rand((Hkv, 1, D), generator=g, device="cuda") > 0.96)
    data = []
    for s in (gain, None):
        c8 = torch.empty((pages, Hkv, page, D), dtype=torch.uint8, device="cuda")
        ce = torch.empty((pages, Hkv, page, D // 32), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 27) // (Hkv * page * D))
        for i in range(0, pages, step):
            n = min(step, pages - i)
            x = torch.randn((n, Hkv, page, D), generator=g, device="cuda")
            if s is not None:
                x = (x + 0.7 * torch.randn((n, Hkv, 1, D), generator=g, device="cuda")) * s
            c8[i:i + n], ce[i:i + n] = _quantise(x.to(torch.bfloat16).float())
        data += [c8, ce]
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


def prepare(case, seed):
    c, r, g = dict(case), random.Random(seed), _gen(seed)
    s = {"op": c["op"], "case": c}
    bf = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    if c["op"] == "plan":
        B, P = c["B"], c["page"]
        done = [r.random() < c["done"] for _ in range(B)]
        old = [r.randint(0, c["ctx"]) for _ in range(B)]                  # cached before
        held = [-(-n // P) for n in old]
        add = [r.randint(1, c["most"]) for _ in range(B)]
        lens = list(old)
        for b in range(B):
            if done[b]:  # its row goes to a new request: a prompt, where there are any
                lens[b] = 0
                add[b] = r.randint(1, c["long"]) if c["long"] else add[b]
        # a token budget a tenth over the mean; pages for almost all: a crowded batch's last requests may have to wait
        tokens = int(1.1 * B * ((1 - c["done"]) * (1 + c["most"]) / 2 + c["done"] * (1 + (c["long"] or c["most"])) / 2)) + c["most"]
        width = -(-(c["ctx"] + max(c["most"], c["long"])) // P)
        pool = B * width
        back = sum(h for h, d in zip(held, done) if d)
        want = sum(max(0, -(-(n + a) // P) - (0 if d else h)) for n, a, h, d in zip(lens, add, held, done))
        free = min(pool - sum(held), max(0, int(want * 0.98) + 1 - back))
        order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        table[torch.arange(width, device="cuda") < _ints(held)[:, None]] = order[:sum(held)]
        stack = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
        stack[:free] = order[sum(held):sum(held) + free]
        s.update(table=table, held=_ints(held), free=stack, count=_ints([free]), lens=_ints(lens), add=_ints(add),
                 done=_ints([int(d) for d in done]), tokens=tokens)
    elif c["op"] == "bounds":
        B = c["B"]
        start = [r.randint(0, c["ctx"]) for _ in range(B)]
        end = [n + (c["add"] if c["add"] == 1 or B == 1 else r.randint(1, c["add"])) for n in start]
        s["cache"], s["table"] = _pool(g, end, c["page"], c["Hkv"], c["D"], c["ctx"] + c["add"])
        pages = s["cache"][0].shape[0]
        # the bounds of the pages' earlier contents
        s["codes"] = torch.randint(-127, 128, (pages, c["Hkv"], 2, c["D"]), generator=g, device="cuda").to(torch.int8)
        s["exps"] = torch.randint(100, 130, (pages, c["Hkv"], c["D"] // 32), generator=g, device="cuda").to(torch.uint8)
        s["start"], s["end"] = _ints(start), _ints(end)
    elif c["op"] == "sparse":
        B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
        ctx = [c["ctx"] if B == 1 else r.randint(1, c["ctx"]) for _ in range(B)]
        nodes = [T if B == 1 or T == 1 else r.randint(max(1, T // 2), T) for _ in range(B)]
        s["cache"], s["table"] = _pool(g, [n + T for n in ctx], c["page"], Hkv, D)
        pages = s["cache"][0].shape[0]
        s["codes"] = torch.zeros((pages, Hkv, 2, D), dtype=torch.int8, device="cuda")
        s["exps"] = torch.zeros((pages, Hkv, D // 32), dtype=torch.uint8, device="cuda")
        _write_bounds(s, torch.arange(pages, device="cuda"))  # of all pages: what the steps before have kept up to date
        s["q"] = bf(B, T, Hq, D) * 1.5
        s["ctx"], s["nodes"] = _ints(ctx), _ints(nodes)
        s["mask"] = None
        if c["tree"]:
            m = np.zeros((B, T, -(-T // 32)), np.uint32)
            for b in range(B):
                parent = _tree(r, T, 3)
                for i in range(T):
                    if i:
                        m[b, i] = m[b, parent[i]]
                    m[b, i, i // 32] |= np.uint32(1 << (i % 32))
            s["mask"] = torch.from_numpy(m.view(np.int32)).cuda()
    elif c["op"] in ("sample", "probs"):
        N, V = c["N"], c["V"]
        # logits of a language model: most far below the best few
        x = torch.randn((N, V), generator=g, device="cuda") * 2.5
        x += 6 * (torch.rand((N, V), generator=g, device="cuda") > 0.9995)
        s["x"] = x.to(torch.bfloat16) if c["bf16"] else x
        how = [c["how"] if c["how"] != "mixed" else r.choice(["plain", "greedy", "k", "p", "k+p", "min", "k+p"]) for _ in range(N)]
        has = lambda *names: c["how"] in names + ("mixed",)  # noqa: E731
        floats = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
        s["t"] = floats([0.0 if h == "greedy" else r.uniform(0.5, 1.2) for h in how])
        s["k"] = _ints([r.choice([20, 40, 64, r.randint(2, 1000)]) if "k" in h else 0 for h in how]) if has("k", "k+p") else None
        s["p"] = floats([r.uniform(0.7, 0.98) if "p" in h.split("+") else 1.0 for h in how]) if has("p", "k+p") else None
        s["m"] = floats([r.uniform(0.01, 0.2) if h == "min" else 0.0 for h in how]) if has("min") else None
        s["u"] = torch.rand((N,), generator=g, device="cuda")
    else:
        M, H = c["M"], c["H"]
        s["x"], s["w"] = bf(M, H) * 3, 1 + 0.2 * bf(H)
        s["r"] = bf(M, H) * 2
        if c["fp32"]:
            s["r"] = s["r"].float() + 0.01 * torch.randn((M, H), generator=g, device="cuda")
        s["post"] = 1 + 0.2 * bf(H) if c["post"] else None
        s["gate"] = {"none": lambda: None, "channel": lambda: bf(H), "token": lambda: bf(M, 1), "full": lambda: bf(M, H)}[c["gate"]]()
        s["scale"] = round(r.uniform(0.2, 1.5), 3)
    return s


# ------------------------------------------------------------------------------------ plain forms

def _part(u, z):
    """floor(u * z / 2^24) for u < 2^24."""
    return (z >> 24) * u + (((z & 0xFFFFFF) * u) >> 24)


def _plain_plan(s):
    P = s["case"]["page"]
    table, held, free, count = s["table"], s["held"].long(), s["free"], s["count"].long()
    B, most = table.shape
    lens, add, done = s["lens"].long(), s["add"].long(), s["done"] > 0
    i = torch.arange(most, device=table.device)
    back = (i < held[:, None]) & done[:, None]      # the pages that come back, row after row
    pages = table[back]
    free[count + torch.arange(pages.numel(), device=table.device)] = pages
    count = count + pages.numel()
    held = torch.where(done, 0, held)
    need = torch.where(add > 0, ((lens + add + P - 1) // P - held).clamp(min=0), 0)
    upto = need.cumsum(0)
    fits = ((need == 0) | (upto <= count)) & (add.cumsum(0) <= s["tokens"])
    granted = torch.where(fits, add, 0)
    need = torch.where(fits, need, 0)
    # the j-th page taken is the j-th from the top of the stack
    new = (i >= held[:, None]) & (i < (held + need)[:, None])
    used = need.sum()
    table[new] = free[count - 1 - torch.arange(int(used), device=table.device)]
    s["held"].copy_(held + need)
    s["count"].copy_(count - used)
    start = torch.cat([torch.zeros(1, dtype=torch.int64, device=table.device), granted.cumsum(0)])
    n = torch.arange(s["tokens"], device=table.device)
    req = torch.searchsorted(start[1:], n, right=True).clamp(max=B - 1)
    real = n < start[-1]
    slot = torch.where(real, lens[req] + n - start[req], -1)
    return [t.to(torch.int32) for t in (torch.where(real, req, 0), slot, start, granted)]


def _plan_outputs(s, out):
    """The plan and the pages' books.  Table entries past a request's pages and the stack above its count keep what
    they held."""
    return list(out) + [s["table"], s["held"], s["free"], s["count"]]


def _write_bounds(s, pages):
    """The bounds of these pages, all heads: maxima rounded up, minima down."""
    k = _decode(s["cache"][0][pages], s["cache"][1][pages])                          # [n, heads, page, D]
    b = torch.stack([k.amax(2), k.amin(2)], 2).unflatten(-1, (-1, 32))               # [n, heads, 2, D / 32, 32]
    # the smallest e >= -127 with 127 * 2^e >= amax, over 32 channels of both
    e = (((b.abs().amax(-1).amax(2).view(torch.int32) + 0x1FFFF) >> 23) - 6).clamp_(min=0)
    b = b * _power(254 - e)[:, :, None, :, None]
    b[:, :, 0].ceil_()
    b[:, :, 1].floor_()
    s["codes"][pages], s["exps"][pages] = b.flatten(-2).to(torch.int8), e.to(torch.uint8)


def _plain_bounds(s):
    P = s["case"]["page"]
    i = torch.arange(s["table"].shape[1], device="cuda")  # pages that became full
    full = (i >= (s["start"] // P)[:, None]) & (i < (s["end"] // P)[:, None])
    _write_bounds(s, s["table"][full].long())
    return [s["codes"], s["exps"]]


SINK, RECENT = 1, 2  # the first page and the last two full ones are always kept


def _plain_select(s):
    c, q, ctx, nodes = s["case"], s["q"], s["ctx"].long(), s["nodes"]
    B, T, Hq, D = q.shape
    Hkv, P, keep = c["Hkv"], c["page"], c["keep"]
    real = (torch.arange(T, device=q.device) < nodes[:, None])[:, :, None, None, None]
    x = torch.where(real, q.float().view(B, T, Hkv, Hq // Hkv, D), 0)
    top = x.abs().amax((1, 3, 4)).clamp(min=2.0 ** -100)                             # [B, Hkv]
    k = (top.view(torch.int32) >> 23) - 127
    n = torch.round(torch.ldexp(x, (17 - k)[:, None, :, None, None])).long()
    Q = torch.stack([n.clamp(min=0).sum((1, 3)), n.clamp(max=0).sum((1, 3))], 2)     # [B, Hkv, 2, D]
    bits = torch.frexp(Q.abs().amax((2, 3)).double()).exponent
    sh = (bits - 14).clamp(min=0).long()[:, :, None, None]
    Q = (Q + ((1 << sh) >> 1)) >> sh
    full = ctx // P
    F = int(s["table"].shape[1])
    i = torch.arange(F, device=q.device)
    table = s["table"].long()
    code, e = s["codes"][table], s["exps"][table]                                     # [B, F, Hkv, 2, D], [B, F, Hkv, D / 32]
    S = (code.int() * Q[:, None].int()).unflatten(-1, (-1, 32)).sum((3, 5))           # [B, F, Hkv, D / 32]
    f = S.float() * 2.0 ** -27 * _power(e)
    while f.shape[-1] > 1:                                                            # in pairs
        f = f[..., 0::2] + f[..., 1::2]
    score = f.squeeze(-1).transpose(1, 2)
    always = (i < SINK) | (i >= full[:, None] - RECENT)
    score = torch.where(always[:, None], math.inf, score)
    score = torch.where((i < full[:, None])[:, None], score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices
    n = torch.minimum(full, torch.tensor(keep, device=q.device))                      # [B]
    width = keep + (2 * P - 2 + T) // P
    j = torch.arange(width, device=q.device)
    best = order[..., :keep]
    best = torch.nn.functional.pad(best, (0, keep - best.shape[-1]), value=F)
    best = torch.where(torch.arange(keep, device=q.device) < n[:, None, None], best, F).sort(-1).values
    tail = full[:, None] + j - n[:, None]                                             # [B, width]
    last = (ctx + nodes + P - 1) // P
    at = torch.where(j < n[:, None, None], torch.nn.functional.pad(best, (0, width - keep)),
                     torch.where(tail < last[:, None], tail, F)[:, None].expand(B, Hkv, width))
    held = torch.nn.functional.pad(table, (0, 1), value=-1)
    pages = held[:, None].expand(B, Hkv, F + 1).gather(2, at)
    return pages.to(torch.int32), (n * P + ctx % P).to(torch.int32)


def _plain_attention(s, pages, ctx):
    """Attention over a block table for each head."""
    k8, ke, v8, ve = s["cache"]
    q, nodes = s["q"], s["nodes"]
    B, T, Hq, D = q.shape
    Hkv, page = k8.shape[1], k8.shape[2]
    h = torch.arange(Hkv, device=q.device)[:, None]
    gather = lambda t: t[pages.clamp(min=0).long(), h].flatten(2, 3)  # noqa: E731   [B, Hkv, n * page, ...]
    L = pages.shape[2] * page
    j = torch.arange(L, device=q.device) - ctx[:, None]
    if s["mask"] is None:
        tree = j[:, None, :] <= torch.arange(T, device=q.device)[:, None]
    else:
        bits = ((s["mask"].unsqueeze(-1) >> torch.arange(32, device=q.device)) & 1).flatten(2)[..., :T]
        tree = bits.gather(2, j.clamp(0, T - 1)[:, None, :].expand(B, T, L)) > 0
    seen = (j < 0)[:, None, :] | (tree & (j < nodes[:, None])[:, None, :])
    seen &= (torch.arange(T, device=q.device) < nodes[:, None])[:, :, None]
    qf = q.float().view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    x = torch.matmul(qf, _decode(gather(k8), gather(ke)).transpose(-1, -2)) * (1 / math.sqrt(D))
    x = x.unflatten(2, (T, -1)).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m.masked_fill(m == -math.inf, 0)).exp_().flatten(2, 3)
    y = torch.matmul(x, _decode(gather(v8), gather(ve)))
    total = x.sum(-1, keepdim=True)
    y = y / total.masked_fill(total == 0, 1)
    return y.unflatten(2, (T, -1)).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(torch.bfloat16)


def _plain_sparse(s):
    pages, kept = _plain_select(s)
    return {"pages": pages, "kept": kept, "out": _plain_attention(s, pages, kept)}


def _weights(s):
    """Each logit's weight in the fixed point that the sampling is defined in."""
    x = s["x"].float()
    x = torch.where(x.isnan(), -math.inf, x)
    top = x.amax(-1, keepdim=True)
    t = s["t"][:, None]
    rate = torch.where(t > 0, torch.full_like(t, LOG2E) / t, math.inf)
    y = (top - x) * rate
    n = y.floor()
    f = y - n
    p = torch.full_like(f, EXP2[4])
    for a in (EXP2[3], EXP2[2], EXP2[1], EXP2[0], 1.0):
        p = p * f
        p = p + a
    near = y <= 40
    w = ((torch.where(near, p, 0) * 2.0 ** 24).long() << 16) >> torch.where(near, n, 40).long()
    w = torch.where(near, w, 0)
    w = torch.where(x == top, ONE, w)
    return torch.where(x == -math.inf, 0, w), x


def _plain_kept(s):
    """The weights of the tokens that stay, 0 for the others."""
    w, x = _weights(s)
    N, V = x.shape
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    v = w.gather(1, order)
    k = torch.full((N,), V, device=x.device) if s["k"] is None else torch.where(s["k"] > 0, s["k"], V)
    k = torch.where(s["t"] > 0, k, 1)
    v = torch.where(torch.arange(V, device=x.device) < k[:, None], v, 0)
    if s["m"] is not None:
        v = torch.where(v >= (s["m"].clamp(0, 1) * float(ONE)).ceil().long()[:, None], v, 0)
    if s["p"] is not None:
        total = v.sum(-1)
        cut = _part((s["p"].clamp(0, 1) * float(1 << 24)).long(), total).clamp(min=1)
        v = torch.where((v.cumsum(-1) - v < cut[:, None]) | (s["p"] >= 1)[:, None], v, 0)
    return torch.zeros_like(w).scatter_(1, order, v)


def _plain_sample(s):
    w = _plain_kept(s)
    cum = w.cumsum(-1)
    at = _part((s["u"] * float(1 << 24)).long()[:, None], cum[:, -1:])
    token = (cum <= at).sum(-1, keepdim=True)
    some = cum[:, -1:] > 0
    p = w.gather(1, torch.where(some, token, 0)).double() / cum[:, -1:].clamp(min=1)
    return {"token": torch.where(some, token, -1).squeeze(1).to(torch.int32), "p": p.squeeze(1).float()}


def _plain_probs(s):
    w = _plain_kept(s)
    total = w.sum(-1, keepdim=True).clamp(min=1)
    return (w.double() / total).float()


def _plain_norm(s):
    z = s["x"].float()
    if s["post"] is not None:
        z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + 1e-6) * s["post"].float()
    if s["gate"] is not None:
        z = z * s["gate"].float()
    r = s["r"].float() + s["scale"] * z
    h = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + 1e-6) * s["w"].float()
    return {"h": h.to(torch.bfloat16), "r": r.to(s["r"].dtype)}


def run(s):
    op = s["op"]
    if not own:
        if op == "plan":
            return _plan_outputs(s, _plain_plan(s))
        return {"bounds": _plain_bounds, "sparse": _plain_sparse, "sample": _plain_sample, "probs": _plain_probs,
                "norm": _plain_norm}[op](s)
    import block_scaled_fp8_weight_gb300 as bsf8
    c = s["case"]
    if op == "plan":
        book = bsf8.PageBook(s["table"], s["held"], s["free"], s["count"])
        return _plan_outputs(s, bsf8.kv_plan(book, s["lens"], s["add"], page_size=c["page"], tokens=s["tokens"], done=s["done"]))
    if op == "bounds":
        bounds = bsf8.PageBounds(s["codes"], s["exps"], c["page"])
        bsf8.kv_bounds(bsf8.KVCache(*s["cache"]), bounds, s["table"], s["end"], start=s["start"])
        return [s["codes"], s["exps"]]
    if op == "sparse":
        bounds = bsf8.PageBounds(s["codes"], s["exps"], c["page"])
        pages, kept = bsf8.select_pages(s["q"], bounds, s["table"], s["ctx"], c["keep"], nodes=s["nodes"], sink=SINK, recent=RECENT)
        out = bsf8.sparse_attention(s["q"], bsf8.KVCache(*s["cache"]), pages, kept, nodes=s["nodes"], mask=s["mask"])
        return {"pages": pages, "kept": kept, "out": out}
    if op == "sample":
        token, p = bsf8.sample_tokens(s["x"], s["u"], temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["m"])
        return {"token": token, "p": p}
    if op == "probs":
        return bsf8.token_probs(s["x"], temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["m"])
    h, r = bsf8.residual_norm(s["x"], s["r"], s["w"], post_weight=s["post"], gate=s["gate"], scale=s["scale"])
    return {"h": h, "r": r}


# ------------------------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "plan":
        # what requests add, and the pages that change hands, in the mean
        each = (1 + c["most"]) / 2
        new = (1 + c["long"]) / 2 if c["long"] else each
        tokens = c["B"] * ((1 - c["done"]) * each + c["done"] * new)
        moved = c["B"] * c["done"] * (c["ctx"] / 2 + new) / c["page"]
        return {"bytes": 8 * tokens + 8 * moved + 24 * c["B"], "flops": 0}
    if c["op"] == "bounds":
        add = c["add"] if c["add"] == 1 or c["B"] == 1 else (1 + c["add"]) / 2
        pages = c["B"] * add / c["page"] * c["Hkv"]
        return {"bytes": 8 * c["B"] + pages * (c["page"] * c["D"] * (1 + 1 / 32) + c["D"] * (2 + 1 / 32)),
                "flops": 2 * pages * c["page"] * c["D"]}
    if c["op"] == "sparse":
        # contexts are uniform in 1 .. ctx past one request, nodes in T/2 .. T
        mean = c["ctx"] if c["B"] == 1 else (c["ctx"] + 1) / 2
        t = c["T"] if c["B"] == 1 or c["T"] == 1 else (max(1, c["T"] // 2) + c["T"]) / 2
        P, most = c["page"], c["keep"] * c["page"]
        keys = min(mean, most) if c["B"] == 1 or c["ctx"] <= most else most - most * most / (2 * c["ctx"])
        keys = c["B"] * (keys + P / 2 + t)
        pages = c["B"] * mean / P * c["Hkv"]
        return {"bytes": pages * c["D"] * (2 + 1 / 32) + keys * 2 * c["Hkv"] * c["D"] * (1 + 1 / 32) +
                c["B"] * (4 * mean / P + c["T"] * c["Hq"] * c["D"] * 4),
                "flops": 4 * keys * t * c["Hq"] * c["D"] + 4 * pages * c["D"]}
    if c["op"] in ("sample", "probs"):
        n = c["N"] * c["V"]
        return {"bytes": n * ((2 if c["bf16"] else 4) + (4 if c["op"] == "probs" else 0)) + 28 * c["N"], "flops": 14 * n}
    n = c["M"] * c["H"]
    gate = {"none": 0, "channel": 2 * c["H"], "token": 2 * c["M"], "full": 2 * n}[c["gate"]]
    return {"bytes": n * (4 + (8 if c["fp32"] else 4)) + gate + c["H"] * (4 if c["post"] else 2), "flops": 10 * n}


# ------------------------------------------------------------------------------------ 64 bits

def _value(code, exp):
    """What e4m3 codes with exponent bytes stand for, in 64 bits, from the formats' definitions."""
    c = code.to(torch.int64)
    sign, e, m = 1 - 2 * (c >> 7), (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2((e - 7).double()))
    return sign * mag * torch.exp2(exp.double() - 127).repeat_interleave(32, -1)


def _exact_sparse(s, c):
    B, T, Hq, D = s["q"].shape
    Hkv, P, G = c["Hkv"], c["page"], Hq // c["Hkv"]
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    k8, ke, v8, ve = s["cache"]
    mask = None if s["mask"] is None else s["mask"].cpu().numpy().view(np.uint32)
    for b in range(B):
        n, t = int(s["ctx"][b]), int(s["nodes"][b])
        full = n // P
        pages = s["table"][b, :-(-(n + t) // P)].long()
        see = np.ones((t, t), bool)
        for i in range(t):
            for j in range(t):
                see[i, j] = j <= i if mask is None else bool(mask[b, i, j // 32] >> np.uint32(j % 32) & np.uint32(1))
        see = torch.from_numpy(see).cuda()
        for h in range(Hkv):
            q = s["q"][b, :t, h * G:(h + 1) * G].double().reshape(-1, D)
            a = float(q.abs().max())
            z = torch.round(q * 2.0 ** (17 - math.floor(math.log2(a)))) if a > 0 else q * 0
            up, dn = z.clamp(min=0).sum(0).cpu(), z.clamp(max=0).sum(0).cpu()
            sh = max(0, int(max(up.max(), -dn.min())).bit_length() - 14)
            both = [[(int(v) + (1 << sh >> 1)) >> sh for v in w] for w in (up, dn)]
            f = s["codes"][pages[:full], h].double() * torch.tensor(both, dtype=torch.float64, device="cuda")
            f = f.sum(1).unflatten(-1, (-1, 32)).sum(-1)                   # whole numbers below 2^27
            f = f.float().cpu().numpy() * np.float32(2.0 ** -27) * np.exp2(s["exps"][pages[:full], h].double().cpu().numpy() - 127).astype(np.float32)
            while f.shape[1] > 1:
                f = f[:, ::2] + f[:, 1::2]
            f = f[:, 0]
            f[:SINK] = np.inf
            f[max(0, full - RECENT):] = np.inf
            best = np.sort(np.lexsort((np.arange(full), -f))[:c["keep"]])
            mine = torch.cat([pages[torch.from_numpy(best).cuda()], pages[full:]])
            ctx = len(best) * P + n % P
            k = _value(k8[mine, h].flatten(0, 1)[:ctx + t], ke[mine, h].flatten(0, 1)[:ctx + t])
            v = _value(v8[mine, h].flatten(0, 1)[:ctx + t], ve[mine, h].flatten(0, 1)[:ctx + t])
            x = (q @ k.T / D ** 0.5).unflatten(0, (t, G))
            x[..., ctx:][~see[:, None, :].expand(t, G, t)] = -math.inf
            out[b, :t, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
    return {"pages": None, "kept": None, "out": out}


def _exact_probs(s, c):
    """The softmax over the tokens that stay; which ones do, and which one is drawn, is defined in whole numbers."""
    N, V = s["x"].shape
    x = s["x"].double()
    t = s["t"].tolist()

    def weigh(i):
        z = s["x"][i].float().cpu().numpy()
        if not t[i] > 0:
            return np.where(z == z.max(), ONE, 0)
        y = (z.max() - z) * (np.float32(LOG2E) / np.float32(t[i]))
        f, a = y - np.floor(y), np.float32(EXP2[-1])
        for b in EXP2[-2::-1] + (1.0,):
            a = a * f + np.float32(b)
        return np.where(y > 40, 0, ((a * np.float32(1 << 24)).astype(np.int64) << 16) >> np.minimum(np.floor(y), 40).astype(np.int64))
    out = torch.zeros((N, V), dtype=torch.float64, device="cuda")
    drawn = []
    for i in range(N):
        order = np.lexsort((np.arange(V), -x[i].cpu().numpy()))
        k = int(s["k"][i]) if s["k"] is not None else 0
        stay = order[:1 if not t[i] > 0 else k if k > 0 else V]
        v = weigh(i)[stay]
        if s["m"] is not None:
            m = math.ceil(min(max(float(s["m"][i]), 0.0), 1.0) * ONE)
            stay, v = stay[v >= m], v[v >= m]
        p = float(s["p"][i]) if s["p"] is not None else 1.0
        if p < 1:
            cut = max(1, int(max(p, 0.0) * (1 << 24)) * int(v.sum()) >> 24)
            less = np.cumsum(v) - v < cut
            stay, v = stay[less], v[less]
        if c["op"] == "sample":
            at, upto = np.argsort(stay), int(float(s["u"][i]) * (1 << 24)) * int(v.sum()) >> 24
            drawn.append(int(stay[at][np.searchsorted(np.cumsum(v[at]), upto, side="right")]))
        stay = torch.from_numpy(stay).cuda()
        out[i, stay] = torch.softmax(x[i, stay] / (t[i] if t[i] > 0 else 1.0), 0)
    if c["op"] == "sample":
        return {"token": None, "p": out.gather(1, torch.tensor(drawn, device="cuda")[:, None]).squeeze(1)}
    return out


def _exact_norm(s, c):
    z = s["x"].double()
    if s["post"] is not None:
        z = z / torch.sqrt(z.square().mean(1, True) + 1e-6) * s["post"].double()
    if s["gate"] is not None:
        z = s["gate"].double() * z
    r = s["r"].double() + z * s["scale"]
    return {"h": r / torch.sqrt(r.square().mean(1, True) + 1e-6) * s["w"].double(), "r": r}


def exact(case, seed):
    if case["op"] in ("plan", "bounds"):
        return None  # whole numbers, defined in integers
    s = prepare(case, seed)
    return {"sparse": _exact_sparse, "sample": _exact_probs, "probs": _exact_probs, "norm": _exact_norm}[case["op"]](s, case)
