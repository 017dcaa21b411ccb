"""Speculative decoding with the package's operators, end to end: one attention layer and a vocabulary
head with random weights, a cheap draft (the head on the tokens' embeddings alone), two requests of
different lengths.

    python examples/speculative_step.py [--steps 16] [--sample]

Each step drafts a tree of eight nodes a request, runs it through the layer in one pass

    gemm -> qkv_append -> tree_attention -> gemm -> gemm (head)

then verify_tree decides which nodes stay and draws the next token, and kv_commit moves the kept
nodes' keys and values together.  Without --sample the target is greedy, and each token is compared
with the best one of a plain pass over the request's tokens on a fresh cache (the two differ only in
which kernels sum what: a token may be another where the best two are that close).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp8_weight_gb300 as bsf8  # noqa: E402

HIDDEN, HQ, HKV, D, ROT, VOCAB, PAGE = 1024, 8, 2, 128, 64, 8192, 64
PARENT = [-1, 0, 0, 1, 1, 2, 3, 4]  # the drafted tree: node 0 is the last token kept


def twin(N, K, g):
    """A random [N, K] weight in its e4m3 + ue8m0 form, of about 1 / sqrt(K)."""
    w8 = torch.randint(0, 256, (1, N, K), generator=g, device="cuda").to(torch.uint8)
    w8 = (w8 & 0x80) | (w8 & 0x7F).clamp_(max=0x48)  # up to 4
    ex = torch.full((1, N // 32, K // 32), 127 - (K.bit_length() - 1) // 2, dtype=torch.uint8, device="cuda")
    return w8, ex


class Model:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.emb = torch.randn((VOCAB, HIDDEN), generator=g, device="cuda").to(torch.bfloat16)
        self.qkv, self.out = twin((HQ + 2 * HKV) * D, HIDDEN, g), twin(HIDDEN, HQ * D, g)
        self.head = twin(VOCAB, HIDDEN, g)
        self.norm = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]
        a = torch.arange(4096, device="cuda")[:, None] * 10000.0 ** (-torch.arange(ROT // 2, device="cuda") / (ROT // 2))
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float()

    def logits(self, h):
        h = (h.float() * torch.rsqrt(h.float().square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)
        return bsf8.gemm(h, *self.head).squeeze(1).float()

    def draft(self, tokens):
        """The draft's distribution after each token: no layer, only the embedding."""
        return torch.softmax(self.logits(self.emb[tokens.flatten()]), -1).unflatten(0, tokens.shape)

    def forward(self, tokens, cache, table, ctx, depth, mask=None):
        """Tokens [B, T] at slots ctx + 0 .. T - 1 and positions ctx + depth -> logits [B, T, VOCAB]."""
        B, T = tokens.shape
        h = self.emb[tokens.flatten()]
        x = bsf8.gemm(h, *self.qkv).squeeze(1)
        q, k, v = (t.unflatten(1, (-1, D)) for t in x.split([HQ * D, HKV * D, HKV * D], 1))
        req = torch.arange(B, device="cuda", dtype=torch.int32).repeat_interleave(T)
        node = torch.arange(T, device="cuda", dtype=torch.int32)
        q = bsf8.qkv_append(q, k, v, cache, table, req, (ctx[:, None] + node).flatten(), pos=(ctx[:, None] + depth).flatten(),
                            cos_sin=self.cos_sin, q_norm=self.norm[0], k_norm=self.norm[1])
        o = bsf8.tree_attention(q.view(B, T, HQ, D), cache, table, ctx, mask=mask)
        h = h + bsf8.gemm(o.view(B * T, HQ * D), *self.out).squeeze(1)
        return self.logits(h).view(B, T, VOCAB)


def start(model, prompts):
    """A cache with the prompts' tokens but the last, which becomes each tree's node 0."""
    B, most = len(prompts), max(len(p) for p in prompts)
    pages = -(-(most + 1024) // PAGE)
    cache = bsf8.KVCache.empty(B * pages, HKV, D, PAGE)
    table = torch.randperm(B * pages, device="cuda").to(torch.int32).view(B, pages)
    for b, prompt in enumerate(prompts):
        n, zero = len(prompt) - 1, torch.zeros(1, dtype=torch.int32, device="cuda")
        for i in range(0, n, 256):  # a chain of up to 256 tokens a pass
            part = prompt[i:min(n, i + 256)]
            model.forward(part[None], cache, table[b:b + 1], zero + i, torch.arange(len(part), device="cuda", dtype=torch.int32))
    return cache, table, torch.tensor([len(p) - 1 for p in prompts], dtype=torch.int32, device="cuda")


def shortfall(model, prompt, tokens):
    """How far each token's logit is below the best one's in a plain pass over the request (a chain on a
    fresh cache), in units of the logits' standard deviation."""
    cache, table, ctx = start(model, [prompt])
    told = torch.tensor(tokens, device="cuda")
    chain = torch.cat([prompt[-1:], told[:-1]])[None]
    node = torch.arange(chain.shape[1], device="cuda", dtype=torch.int32)
    logits = model.forward(chain, cache, table, ctx, node)[0]
    return ((logits.amax(-1) - logits.gather(1, told[:, None])[:, 0]) / logits.std(-1)).tolist()


def speculative(model, prompts, steps, sample=False, seed=1):
    """Returns each request's tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, T = len(prompts), len(PARENT)
    cache, table, ctx = start(model, prompts)
    parent = torch.tensor(PARENT, dtype=torch.int32, device="cuda").expand(B, T).contiguous()
    depth, see = [0] * T, torch.eye(T, dtype=torch.bool)
    for i, j in enumerate(PARENT[1:], 1):
        depth[i] = depth[j] + 1
        see[i] |= see[j]
    word = sum(see[:, j].to(torch.int32) << j for j in range(T))
    mask = word[None, :, None].expand(B, T, 1).to(torch.int32).contiguous().cuda()
    depth = torch.tensor(depth, dtype=torch.int32, device="cuda")

    got = [[] for _ in range(B)]
    last = torch.stack([p[-1] for p in prompts])
    for _ in range(steps):
        tokens = torch.empty((B, T), dtype=torch.int64, device="cuda")
        q = torch.zeros((B, T, VOCAB), device="cuda")
        tokens[:, 0] = last
        for i in range(T):  # a node's children: drawn from the draft, or its best ones
            kids = [j for j in range(T) if PARENT[j] == i]
            q[:, i] = model.draft(tokens[:, i])
            if kids:
                tokens[:, kids] = (torch.multinomial(q[:, i], len(kids), replacement=True, generator=g) if sample
                                   else q[:, i].topk(len(kids)).indices)
        logits = model.forward(tokens, cache, table, ctx, depth, mask)
        if sample:
            p = torch.softmax(logits, -1)
        else:
            p = torch.nn.functional.one_hot(logits.argmax(-1), VOCAB).float()
        u = torch.rand((B, T), generator=g, device="cuda")
        path, count, token = bsf8.verify_tree(p, tokens.to(torch.int32), parent, u, q=q if sample else None)
        bsf8.kv_commit(cache, table, ctx, path, count)
        ctx += count
        for b in range(B):  # what the kept nodes after node 0 stand for, then the drawn token
            keep = path[b, 1:count[b]].long()
            got[b] += tokens[b, keep].tolist() + [int(token[b])]
        last = token.long()
    return got


def prompts(seed=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randint(0, VOCAB, (n,), generator=g, device="cuda") for n in (700, 33)]


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--steps", type=int, default=16)
    a.add_argument("--sample", action="store_true")
    args = a.parse_args()
    model = Model()
    got = speculative(model, prompts(), args.steps, args.sample)
    for b, t in enumerate(got):
        print(f"request {b}: {len(t)} tokens in {args.steps} steps: {t[:12]} ...")
    if not args.sample:
        for b, t in enumerate(got):
            d = shortfall(model, prompts()[b], t)
            print(f"request {b}: {sum(x == 0 for x in d)} of {len(t)} tokens are a plain pass's best; furthest off: "
                  f"{max(d):.4f} standard deviations of the logits")
    print("device status", bsf8.device_status())


if __name__ == "__main__":
    main()
