"""Binding of the decode operators (include/bsf8.h, "decode operators"): the paged block-scaled
fp8 cache of keys and values, attention of a drafted token tree over it, and the verification
of the drafts.  Like the rest of the binding it only checks and marshals arguments -- here through
the extension _bsf8_torch (csrc/bsf8_torch.cpp), as a decode step's operators take the GPU less
time than a ctypes call of this many arguments takes the host; every computation runs in the
library's kernels on the current stream of the tensors' device.

One step of speculative decoding, per layer and then once:

    q = qkv_append(q, k, v, cache, table, req, slot, pos=pos, cos_sin=cos_sin, q_norm=..., k_norm=...)
    o = tree_attention(q.view(B, T, Hq, D), cache, table, ctx, nodes=nodes, mask=mask)
    ...
    path, count, token = verify_tree(p, tokens, parent, u, q=draft_p, nodes=nodes)
    kv_commit(cache, table, ctx, path, count)          # per layer; then ctx += count

A token tree's node 0 is the last token kept before (its keys and values are not cached yet);
node i sits at slot ctx + i of its request, its position is ctx plus its depth.
"""
from __future__ import annotations

import ctypes

from . import _check, _torch, load
from . import build as _build


class _Unloaded:
    """Stands for the extension until a call needs it: torch is imported and what is missing built then."""

    def __getattr__(self, name):
        global _ext
        load()
        _ext = _build.load_extension()
        return getattr(_ext, name)


_ext = _Unloaded()

MAX_NODES = 256


class _CacheStruct(ctypes.Structure):
    """bsf8_kv_cache."""
    _fields_ = [("k8", ctypes.c_void_p), ("kexp", ctypes.c_void_p), ("v8", ctypes.c_void_p),
                ("vexp", ctypes.c_void_p), ("pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("heads", ctypes.c_int), ("dim", ctypes.c_int)]


class KVCache:
    """A layer's cache: codes k8, v8 uint8 [pages, heads, page_size, dim] and exponent bytes
    kexp, vexp uint8 [pages, heads, page_size, dim / 32], contiguous CUDA tensors that the
    caller owns (KVCache.empty allocates them)."""

    __slots__ = ("k8", "kexp", "v8", "vexp")

    def __init__(self, k8, kexp, v8, vexp):
        self.k8, self.kexp, self.v8, self.vexp = k8, kexp, v8, vexp

    @classmethod
    def empty(cls, pages: int, heads: int, dim: int, page_size: int = 64, device="cuda"):
        """A new cache; its contents are undefined until tokens are appended."""
        torch = _torch()
        code = lambda: torch.empty((pages, heads, page_size, dim), dtype=torch.uint8, device=device)  # noqa: E731
        byte = lambda: torch.empty((pages, heads, page_size, dim // 32), dtype=torch.uint8, device=device)  # noqa: E731
        return cls(code(), byte(), code(), byte())

    @property
    def heads(self):
        return self.k8.shape[1]

    @property
    def page_size(self):
        return self.k8.shape[2]

    @property
    def dim(self):
        return self.k8.shape[3]

    def _struct(self):
        """bsf8_kv_cache, for calls of the C ABI; checks the tensors' shapes."""
        pages, heads, size, dim = self.k8.shape
        for name, t, want in (("kexp", self.kexp, (pages, heads, size, dim // 32)), ("v8", self.v8, self.k8.shape),
                              ("vexp", self.vexp, (pages, heads, size, dim // 32))):
            if tuple(t.shape) != tuple(want):
                raise ValueError(f"{name} must have shape {tuple(want)}, got {tuple(t.shape)}")
        return _CacheStruct(self.k8.data_ptr(), self.kexp.data_ptr(), self.v8.data_ptr(), self.vexp.data_ptr(),
                            pages, size, heads, dim)


def qkv_append(q, k, v, cache: KVCache, table, req, slot, *, pos=None, cos_sin=None, q_norm=None,
               k_norm=None, eps: float = 1e-6, interleaved: bool = False, out=None):
    """Norm, rotate and append in one pass: q [N, Hq, D], k and v [N, Hkv, D] (bf16; rows may be
    views of one projection's output), token n into slot[n] of request req[n] (int32 [N]).
    q_norm, k_norm: bf16 [D] weights of the per-head RMS norm; cos_sin: fp32 [positions, rot],
    cosines then sines, with pos int32 [N].  Returns the queries, bf16 [N, Hq, D] (q None: only
    keys and values, returns None)."""
    r = _ext.qkv_append(cache.k8, cache.kexp, cache.v8, cache.vexp, q, k, v, table, req, slot, pos, cos_sin, q_norm,
                        k_norm, eps, interleaved, out)
    if type(r) is int:
        _check(r, "bsf8_qkv_append")
    return r


def kv_read(cache: KVCache, table, req, slot, *, k_out=None, v_out=None):
    """Cached tokens as bf16: (k, v), each [N, Hkv, D], of slot[n] of request req[n]."""
    r = _ext.kv_read(cache.k8, cache.kexp, cache.v8, cache.vexp, table, req, slot, k_out, v_out)
    if type(r) is int:
        _check(r, "bsf8_kv_read")
    return r


def tree_attention_workspace_bytes(B: int, T: int, Hq: int, heads: int, dim: int) -> int:
    return int(load().bsf8_tree_attention_workspace_bytes(B, T, Hq, heads, dim))


def tree_attention(q, cache: KVCache, table, ctx, *, nodes=None, mask=None, scale=None, max_len=None,
                   out=None, lse=None, workspace=None):
    """Attention of token trees over the cache: q bf16 [B, T, Hq, D] (row t of request b is node t, at
    slot ctx[b] + t; the batch stride must be T row strides), ctx and nodes int32 [B] (nodes None: all
    T), mask int32 [B, T, ceil(T / 32)] with bit j of row t set where node t sees node j (None: a
    chain, j <= t).  scale defaults to 1 / sqrt(D); max_len bounds a request's cached tokens with its
    nodes (at most 2^30; default: the table's capacity).  Returns bf16 [B, T, Hq, D]; lse, where given (fp32
    [B, T, Hq]), receives the log of the softmax sums."""
    r = _ext.tree_attention(cache.k8, cache.kexp, cache.v8, cache.vexp, q, table, ctx, nodes, mask, scale, max_len,
                            out, lse, workspace)
    if type(r) is int:
        _check(r, "bsf8_tree_attention")
    return r


def verify_tree(p, tokens, parent, u, *, q=None, nodes=None):
    """Which drafted nodes are kept: p fp32 [B, T, V], the target's distribution after each node; q
    likewise the draft's (None: drafts that were not drawn at random); tokens and parent int32
    [B, T]; u fp32 [B, T] uniform numbers (u[b, 0] draws the next token); nodes int32 [B].
    Returns (path int32 [B, T]: the kept nodes, then -1; count int32 [B]; token int32 [B])."""
    r = _ext.verify_tree(p, tokens, parent, u, q, nodes)
    if type(r) is int:
        _check(r, "bsf8_verify_tree")
    return r


def kv_commit(cache: KVCache, table, ctx, path, count):
    """Moves the kept nodes together, in place: slot ctx[b] + path[b][i] -> ctx[b] + i for
    i < count[b] (path and count as verify_tree returns them)."""
    r = _ext.kv_commit(cache.k8, cache.kexp, cache.v8, cache.vexp, table, ctx, path, count)
    if r is not None:
        _check(r, "bsf8_kv_commit")
