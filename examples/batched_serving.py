"""Continuous batching over long contexts with the package's operators: two layers with random weights, requests
that come, are read in chunks, answer a token a step and leave.

    python examples/batched_serving.py [--requests 6] [--keep 8]

Each step

    kv_plan            pages of requests that left go back, new tokens get pages, requests and slots
    per layer:
      residual_norm    the block before, added to the residual, normed for this one
      gemm -> qkv_append -> kv_bounds
      select_pages -> sparse_attention   over the pages that promise most (or all of them)
      gemm
    residual_norm, gemm (head), sample_tokens

Chunks of prompts and single tokens share a step: a request's new tokens are the nodes of a chain.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp8_weight_gb300 as bsf8  # noqa: E402

HIDDEN, HQ, HKV, D, ROT, VOCAB, PAGE, LAYERS = 1024, 8, 2, 128, 64, 8192, 32, 2
ROWS, CHUNK, LONGEST, POOL = 4, 64, 2048, 160  # requests at a time, new tokens of one a step, tokens of one, pages


def twin(N, K, g):
    """A random [N, K] weight in its e4m3 + ue8m0 form, of about 1 / sqrt(K)."""
    w8 = torch.randint(0, 256, (1, N, K), generator=g, device="cuda").to(torch.uint8)
    w8 = (w8 & 0x80) | (w8 & 0x7F).clamp_(max=0x48)  # up to 4
    return w8, torch.full((1, N // 32, K // 32), 127 - (K.bit_length() - 1) // 2, dtype=torch.uint8, device="cuda")


class Layer:
    def __init__(self, g):
        self.qkv, self.out = twin((HQ + 2 * HKV) * D, HIDDEN, g), twin(HIDDEN, HQ * D, g)
        vec = lambda n: (1 + 0.1 * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
        self.norm, self.post, self.gate, self.q_norm, self.k_norm = vec(HIDDEN), vec(HIDDEN), vec(HIDDEN), vec(D), vec(D)


class Model:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.emb = torch.randn((VOCAB, HIDDEN), generator=g, device="cuda").to(torch.bfloat16)
        self.layers = [Layer(g) for _ in range(LAYERS)]
        self.norm = (1 + 0.1 * torch.randn(HIDDEN, generator=g, device="cuda")).to(torch.bfloat16)
        self.head = twin(VOCAB, HIDDEN, g)
        a = torch.arange(LONGEST, device="cuda")[:, None] * 10000.0 ** (-torch.arange(ROT // 2, device="cuda") / (ROT // 2))
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float()


class Server:
    """The state of a batch: page books, a cache and its pages' bounds a layer, each row's tokens."""

    def __init__(self, model, keep):
        self.model, self.keep = model, keep
        self.book = bsf8.PageBook.empty(ROWS, LONGEST // PAGE, POOL)
        self.caches = [bsf8.KVCache.empty(POOL, HKV, D, PAGE) for _ in range(LAYERS)]
        self.bounds = [bsf8.PageBounds.empty(c) for c in self.caches]
        self.lens = torch.zeros(ROWS, dtype=torch.int32, device="cuda")

    def step(self, new, done, u):
        """new: each row's tokens to read (a list, empty for a free row); done: rows whose request has left.
        Returns how many tokens each row got in, and the token drawn after each row's last one."""
        m, lens = self.model, self.lens
        add = torch.tensor([len(t) for t in new], dtype=torch.int32, device="cuda")
        gone = torch.tensor(done, device="cuda")
        lens.masked_fill_(gone, 0)
        N = sum(len(t) for t in new)
        req, slot, start, granted = bsf8.kv_plan(self.book, lens, add, page_size=PAGE, tokens=N, done=gone.to(torch.int32))
        table, ends = self.book.table, lens + granted
        # the granted tokens, one request's after another's, as the plan has them; and their places in [ROWS, CHUNK]
        got = granted.tolist()
        x = [t for row, n in zip(new, got) for t in row[:n]]
        h = m.emb[torch.tensor(x + [0] * (N - len(x)), device="cuda")]
        node = (slot - lens[req.long()]).clamp(min=0).long()
        at = torch.where(slot < 0, ROWS * CHUNK, req.long() * CHUNK + node)
        r, f = h.clone(), None
        for layer, cache, bounds in zip(m.layers, self.caches, self.bounds):
            if f is None:
                h, _ = bsf8.residual_norm(h, None, layer.norm)
            else:
                h, r = bsf8.residual_norm(f, r, layer.norm, post_weight=before.post, gate=before.gate, scale=0.5)
            q, k, v = (t.unflatten(1, (-1, D)) for t in bsf8.gemm(h, *layer.qkv).squeeze(1).split([HQ * D, HKV * D, HKV * D], 1))
            q = bsf8.qkv_append(q, k, v, cache, table, req, slot, pos=slot.clamp(min=0), cos_sin=m.cos_sin, q_norm=layer.q_norm,
                                k_norm=layer.k_norm)
            tree = q.new_zeros((ROWS * CHUNK + 1, HQ, D)).index_copy_(0, at, q)[:-1].view(ROWS, CHUNK, HQ, D)
            if self.keep:
                pages, kept = bsf8.select_pages(tree, bounds, table, lens, self.keep, nodes=granted, sink=1, recent=1)
                o = bsf8.sparse_attention(tree, cache, pages, kept, nodes=granted)
            else:
                o = bsf8.tree_attention(tree, cache, table, lens, nodes=granted)
            # the pages that these tokens filled
            bsf8.kv_bounds(cache, bounds, table, ends, start=lens)
            o = o.view(ROWS * CHUNK, HQ * D)[at.clamp(max=ROWS * CHUNK - 1)]
            f, before = bsf8.gemm(o, *layer.out).squeeze(1), layer
        h, _ = bsf8.residual_norm(f, r, m.norm, post_weight=before.post, gate=before.gate, scale=0.5)
        last = (start[1:] - 1).clamp(min=0).long()
        self.logits = bsf8.gemm_f32(h[last], *m.head).squeeze(1)
        token, _ = bsf8.sample_tokens(self.logits, u, temperature=torch.full((ROWS,), self.temperature, device="cuda"),
                                      top_k=torch.full((ROWS,), 40, dtype=torch.int32, device="cuda"))
        self.lens = ends
        return got, token.tolist()

    temperature = 0.0


def serve(model, prompts, answer, keep, temperature=0.0, seed=3):
    """Each prompt's `answer` tokens, in order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    server = Server(model, keep)
    server.temperature = temperature
    waiting, rows, out, done = list(range(len(prompts))), [None] * ROWS, [[] for _ in prompts], [False] * ROWS
    todo = [[] for _ in range(ROWS)]  # tokens not read yet
    while waiting or any(r is not None for r in rows):
        for i in range(ROWS):
            if rows[i] is None and waiting:
                rows[i] = waiting.pop(0)
                todo[i] = list(prompts[rows[i]])
        u = torch.rand(ROWS, generator=g, device="cuda")
        got, token = server.step([t[:CHUNK] for t in todo], done, u)
        done = [False] * ROWS
        for i, n in enumerate(got):
            if rows[i] is None or n == 0:
                continue
            todo[i] = todo[i][n:]
            if not todo[i]:  # all is read: the drawn token is the answer's next
                out[rows[i]].append(token[i])
                todo[i] = [token[i]]
                if len(out[rows[i]]) == answer:
                    rows[i], todo[i], done[i] = None, [], True
    return out


def prompts(n, seed=2):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(0, VOCAB, (int(k),), generator=g).tolist() for k in torch.randint(1, 1200, (n,), generator=g)]


def main():
    a = argparse.ArgumentParser()
    a.add_argument("--requests", type=int, default=6)
    a.add_argument("--keep", type=int, default=8, help="pages kept by score; 0: attention over all of them")
    a.add_argument("--temperature", type=float, default=0.0)
    args = a.parse_args()
    model, asked = Model(), prompts(args.requests)
    for p, t in zip(asked, serve(model, asked, 8, args.keep, args.temperature)):
        print(f"{len(p)} tokens in: {t}")
    print("device status", bsf8.device_status())


if __name__ == "__main__":
    main()
