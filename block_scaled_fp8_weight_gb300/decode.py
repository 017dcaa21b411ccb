"""Binding of the decode operators (include/bsf8.h, "decode operators"): the paged block-scaled
fp8 cache of keys and values, attention of a drafted token tree over it, and the verification
of the drafts.  Like the rest of the binding it only checks and marshals arguments; every
computation runs in the library's kernels on the current stream of the tensors' device.

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
from dataclasses import dataclass

from . import _check, _dev, _stream, _torch, load

MAX_NODES = 256


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k8", ctypes.c_void_p), ("kexp", ctypes.c_void_p), ("v8", ctypes.c_void_p),
                ("vexp", ctypes.c_void_p), ("pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("heads", ctypes.c_int), ("dim", ctypes.c_int)]


@dataclass
class KVCache:
    """A layer's cache: codes k8, v8 uint8 [pages, heads, page_size, dim] and exponent bytes
    kexp, vexp uint8 [pages, heads, page_size, dim / 32], contiguous CUDA tensors that the
    caller owns (KVCache.empty allocates them)."""

    k8: object
    kexp: object
    v8: object
    vexp: object

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
        torch = _torch()
        if self.k8.dim() != 4:
            raise ValueError("k8 must be [pages, heads, page_size, dim]")
        pages, heads, size, dim = self.k8.shape
        for name, shape in (("k8", (pages, heads, size, dim)), ("kexp", (pages, heads, size, dim // 32)),
                            ("v8", (pages, heads, size, dim)), ("vexp", (pages, heads, size, dim // 32))):
            t = getattr(self, name)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            if t.device != self.k8.device:
                raise ValueError("the cache's tensors must be on one device")
        ptr = [_dev(getattr(self, n), torch.uint8, n) for n in ("k8", "kexp", "v8", "vexp")]
        return _CacheStruct(*ptr, pages, size, heads, dim)


def _int32(t, name, shape, device):
    """A contiguous int32 tensor of the given shape on the given device, as a pointer."""
    torch = _torch()
    p = _dev(t, torch.int32, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the cache on {device}")
    return p


def _table(table, device):
    if table.dim() != 2:
        raise ValueError("table must be [requests, table_pages]")
    return _int32(table, "table", table.shape, device)


def _same(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, the call on {device}")


def _rows(t, name, heads, dim):
    """[N, heads, dim] bf16 rows whose heads lie one after another; their row stride."""
    torch = _torch()
    p = _dev(t, torch.bfloat16, name)
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name} must be [N, {heads}, {dim}], got {tuple(t.shape)}")
    if t.numel() and (t.stride(2) != 1 or (heads > 1 and t.stride(1) != dim)):
        raise ValueError(f"{name}'s heads must lie one after another (strides (*, {dim}, 1))")
    return p, (t.stride(0) if t.shape[0] > 1 else heads * dim)


def _out(t, name, shape, dtype, device):
    """An output the caller gave, checked, or a new one."""
    torch = _torch()
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _dev(t, dtype, name)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {tuple(shape)}")
    _same(device, **{name: t})
    return t


def qkv_append(q, k, v, cache: KVCache, table, req, slot, *, pos=None, cos_sin=None, q_norm=None,
               k_norm=None, eps: float = 1e-6, interleaved: bool = False, out=None):
    """Norm, rotate and append in one pass: q [N, Hq, D], k and v [N, Hkv, D] (bf16; rows may be
    views of one projection's output), token n into slot[n] of request req[n] (int32 [N]).
    q_norm, k_norm: bf16 [D] weights of the per-head RMS norm; cos_sin: fp32 [positions, rot],
    cosines then sines, with pos int32 [N].  Returns the queries, bf16 [N, Hq, D] (q None: only
    keys and values, returns None)."""
    torch = _torch()
    lib = load()
    st = cache._struct()
    dev, D = cache.k8.device, cache.dim
    N = k.shape[0]
    kp, ldk = _rows(k, "k", cache.heads, D)
    vp, ldv = _rows(v, "v", cache.heads, D)
    if v.shape[0] != N:
        raise ValueError("k and v must have the same tokens")
    Hq, qp, ldq, op = 0, None, 0, None
    if q is not None:
        if q.dim() != 3 or q.shape[0] != N:
            raise ValueError(f"q must be [{N}, Hq, {D}]")
        Hq = q.shape[1]
        qp, ldq = _rows(q, "q", Hq, D)
        out = _out(out, "out", (N, Hq, D), torch.bfloat16, dev)
        op = _dev(out, torch.bfloat16, "out")
    _same(dev, q=q, k=k, v=v, q_norm=q_norm, k_norm=k_norm, cos_sin=cos_sin)
    rot, positions, cp, pp = 0, 0, None, None
    if cos_sin is not None:
        if cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be contiguous [positions, rot]")
        if pos is None:
            raise ValueError("a rotation needs pos")
        positions, rot = cos_sin.shape
        cp, pp = _dev(cos_sin, torch.float32, "cos_sin"), _int32(pos, "pos", (N,), dev)
    norms = []
    for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
        if w is not None and (tuple(w.shape) != (D,) or not w.is_contiguous()):
            raise ValueError(f"{name} must be contiguous [{D}]")
        norms.append(None if w is None else _dev(w, torch.bfloat16, name))
    _check(lib.bsf8_qkv_append(qp, kp, vp, ldq, ldk, ldv, op, ctypes.byref(st), _table(table, dev),
                               table.shape[0], table.shape[1], _int32(req, "req", (N,), dev),
                               _int32(slot, "slot", (N,), dev), pp, cp, positions, rot, int(interleaved),
                               norms[0], norms[1], eps, N, Hq, _stream(k)), "bsf8_qkv_append")
    return out if q is not None else None


def kv_read(cache: KVCache, table, req, slot, *, k_out=None, v_out=None):
    """Cached tokens as bf16: (k, v), each [N, Hkv, D], of slot[n] of request req[n]."""
    torch = _torch()
    lib = load()
    st = cache._struct()
    dev, N = cache.k8.device, req.shape[0]
    shape = (N, cache.heads, cache.dim)
    k_out = _out(k_out, "k_out", shape, torch.bfloat16, dev)
    v_out = _out(v_out, "v_out", shape, torch.bfloat16, dev)
    _check(lib.bsf8_kv_read(ctypes.byref(st), _table(table, dev), table.shape[0], table.shape[1],
                            _int32(req, "req", (N,), dev), _int32(slot, "slot", (N,), dev),
                            _dev(k_out, torch.bfloat16, "k_out"), _dev(v_out, torch.bfloat16, "v_out"), N,
                            _stream(cache.k8)), "bsf8_kv_read")
    return k_out, v_out


def tree_attention_workspace_bytes(B: int, T: int, Hq: int, heads: int, dim: int) -> int:
    return int(load().bsf8_tree_attention_workspace_bytes(B, T, Hq, heads, dim))


def tree_attention(q, cache: KVCache, table, ctx, *, nodes=None, mask=None, scale=None, max_len=None,
                   out=None, lse=None, workspace=None):
    """Attention of token trees over the cache: q bf16 [B, T, Hq, D] (row t of request b is node t, at
    slot ctx[b] + t; the batch stride must be T row strides), ctx and nodes int32 [B] (nodes None: all
    T), mask int32 [B, T, ceil(T / 32)] with bit j of row t set where node t sees node j (None: a
    chain, j <= t).  scale defaults to 1 / sqrt(D); max_len bounds a request's cached tokens with its
    nodes (default: the table's capacity).  Returns bf16 [B, T, Hq, D]; lse, where given (fp32
    [B, T, Hq]), receives the log of the softmax sums."""
    torch = _torch()
    lib = load()
    st = cache._struct()
    dev, D = cache.k8.device, cache.dim
    qp = _dev(q, torch.bfloat16, "q")
    if q.dim() != 4 or q.shape[3] != D:
        raise ValueError(f"q must be [B, T, Hq, {D}]")
    B, T, Hq, _ = q.shape
    ldq = q.stride(1) if T > 1 else (q.stride(0) if B > 1 else Hq * D)
    if q.stride(3) != 1 or (Hq > 1 and q.stride(2) != D) or (B > 1 and q.stride(0) != T * ldq):
        raise ValueError(f"q must have strides (T * ld, ld, {D}, 1)")
    if table.shape[0] != B:
        raise ValueError("table must have a row for each request")
    out = _out(out, "out", (B, T, Hq, D), torch.bfloat16, dev)
    if lse is not None:
        lse = _out(lse, "lse", (B, T, Hq), torch.float32, dev)
    _same(dev, q=q)
    if scale is None:
        scale = D ** -0.5
    if max_len is None:
        max_len = table.shape[1] * cache.page_size
    need = int(lib.bsf8_tree_attention_workspace_bytes(B, T, Hq, cache.heads, D))
    ws_ptr, ws_bytes = None, 0
    if need:
        if workspace is None:
            workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
        _same(dev, workspace=workspace)
        ws_ptr, ws_bytes = _dev(workspace, torch.uint8, "workspace"), workspace.numel()
    _check(lib.bsf8_tree_attention(
        qp, ldq, ctypes.byref(st), _table(table, dev), table.shape[1], _int32(ctx, "ctx", (B,), dev),
        None if nodes is None else _int32(nodes, "nodes", (B,), dev),
        None if mask is None else _int32(mask, "mask", (B, T, (T + 31) // 32), dev), scale, max_len,
        _dev(out, torch.bfloat16, "out"), None if lse is None else _dev(lse, torch.float32, "lse"),
        B, T, Hq, ws_ptr, ws_bytes, _stream(q)), "bsf8_tree_attention")
    return out


def verify_tree(p, tokens, parent, u, *, q=None, nodes=None):
    """Which drafted nodes are kept: p fp32 [B, T, V], the target's distribution after each node; q
    likewise the draft's (None: drafts that were not drawn at random); tokens and parent int32
    [B, T]; u fp32 [B, T] uniform numbers (u[b, 0] draws the next token); nodes int32 [B].
    Returns (path int32 [B, T]: the kept nodes, then -1; count int32 [B]; token int32 [B])."""
    torch = _torch()
    lib = load()
    pp = _dev(p, torch.float32, "p")
    if p.dim() != 3:
        raise ValueError("p must be [B, T, V]")
    B, T, V = p.shape
    dev = p.device
    ld = p.stride(1) if T > 1 else (p.stride(0) if B > 1 else V)
    for name, t in (("p", p), ("q", q)):
        if t is None:
            continue
        if tuple(t.shape) != (B, T, V) or (V > 1 and t.stride(2) != 1) or (T > 1 and t.stride(1) != ld) or \
                (B > 1 and t.stride(0) != T * ld):
            raise ValueError(f"{name} must be [B, T, V] with strides (T * ld, ld, 1), p's and q's ld the same")
    _dev(u, torch.float32, "u")
    if tuple(u.shape) != (B, T) or not u.is_contiguous():
        raise ValueError(f"u must be contiguous [{B}, {T}]")
    _same(dev, q=q, u=u)
    path = torch.empty((B, T), dtype=torch.int32, device=dev)
    count = torch.empty((B,), dtype=torch.int32, device=dev)
    token = torch.empty((B,), dtype=torch.int32, device=dev)
    _check(lib.bsf8_verify_tree(
        pp, None if q is None else _dev(q, torch.float32, "q"), ld, _int32(tokens, "tokens", (B, T), dev),
        _int32(parent, "parent", (B, T), dev), _dev(u, torch.float32, "u"),
        None if nodes is None else _int32(nodes, "nodes", (B,), dev), _dev(path, torch.int32, "path"),
        _dev(count, torch.int32, "count"), _dev(token, torch.int32, "token"), B, T, V, _stream(p)),
        "bsf8_verify_tree")
    return path, count, token


def kv_commit(cache: KVCache, table, ctx, path, count):
    """Moves the kept nodes together, in place: slot ctx[b] + path[b][i] -> ctx[b] + i for
    i < count[b] (path and count as verify_tree returns them)."""
    lib = load()
    st = cache._struct()
    dev = cache.k8.device
    if path.dim() != 2:
        raise ValueError("path must be [B, T]")
    B, T = path.shape
    if table.shape[0] != B:
        raise ValueError("table must have a row for each request")
    _check(lib.bsf8_kv_commit(ctypes.byref(st), _table(table, dev), table.shape[1], _int32(ctx, "ctx", (B,), dev),
                              _int32(path, "path", (B, T), dev), _int32(count, "count", (B,), dev), B, T,
                              _stream(cache.k8)), "bsf8_kv_commit")
