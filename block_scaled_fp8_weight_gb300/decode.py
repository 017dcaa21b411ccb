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
import struct

import torch

from . import _check, load

MAX_NODES = 256

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_empty = torch.empty
_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream of a device, as an address


class _CacheStruct(ctypes.Structure):
    """bsf8_kv_cache."""
    _fields_ = [("k8", ctypes.c_void_p), ("kexp", ctypes.c_void_p), ("v8", ctypes.c_void_p),
                ("vexp", ctypes.c_void_p), ("pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("heads", ctypes.c_int), ("dim", ctypes.c_int)]


_pack_cache = struct.Struct("@4P4i").pack  # the same bytes, in a fraction of the time
assert struct.calcsize("@4P4i") == ctypes.sizeof(_CacheStruct)


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
        code = lambda: _empty((pages, heads, page_size, dim), dtype=_U8, device=device)  # noqa: E731
        byte = lambda: _empty((pages, heads, page_size, dim // 32), dtype=_U8, device=device)  # noqa: E731
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
        """bsf8_kv_cache as a ctypes structure."""
        return _CacheStruct.from_buffer_copy(self._view()[2])

    def _view(self):
        """(device index, (pages, heads, page_size, dim), bsf8_kv_cache as bytes)"""
        k8 = self.k8
        if k8.dim() != 4:
            raise ValueError("k8 must be [pages, heads, page_size, dim]")
        di, shape = k8.get_device(), k8.shape
        pages, heads, size, dim = shape
        small = (pages, heads, size, dim // 32)
        for name, t, want in (("kexp", self.kexp, small), ("v8", self.v8, shape), ("vexp", self.vexp, small)):
            if t.shape != want:
                raise ValueError(f"{name} must have shape {tuple(want)}, got {tuple(t.shape)}")
        return di, shape, _pack_cache(_arg(k8, _U8, shape, di, "k8"), _arg(self.kexp, _U8, small, di, "kexp"),
                                      _arg(self.v8, _U8, shape, di, "v8"), _arg(self.vexp, _U8, small, di, "vexp"),
                                      pages, size, heads, dim)


def _arg(t, dtype, shape, di, name):
    """The address of a contiguous tensor of the given type and shape on device index di."""
    if t.dtype is not dtype or t.get_device() != di or di < 0 or t.shape != shape or not t.is_contiguous():
        _refuse(t, dtype, shape, di, name)
    return t.data_ptr()


def _refuse(t, dtype, shape, di, name):
    """Says what is wrong with an argument."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libbsf8 has no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if di < 0:
        raise ValueError("the call's other tensors must be CUDA tensors (libbsf8 has no CPU path)")
    if t.get_device() != di:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the call on cuda:{di}")
    raise ValueError(f"{name} must be contiguous")


def _table(table, di):
    """(address, requests, pages a request) of a block table."""
    if table.dim() != 2:
        raise ValueError("table must be [requests, table_pages]")
    shape = table.shape
    return _arg(table, _I32, shape, di, "table"), shape[0], shape[1]


def _rows(t, name, heads, dim, di):
    """(address, row stride) of [N, heads, dim] bf16 rows whose heads lie one after another."""
    if t.dtype is not _BF16 or t.get_device() != di:
        _refuse(t, _BF16, None, di, name)
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name} must be [N, {heads}, {dim}], got {tuple(t.shape)}")
    ld, hs, cs = t.stride()
    if (cs != 1 or (heads > 1 and hs != dim)) and t.numel():
        raise ValueError(f"{name}'s heads must lie one after another (strides (*, {dim}, 1))")
    return t.data_ptr(), (ld if t.shape[0] > 1 else heads * dim)


def qkv_append(q, k, v, cache: KVCache, table, req, slot, *, pos=None, cos_sin=None, q_norm=None,
               k_norm=None, eps: float = 1e-6, interleaved: bool = False, out=None):
    """Norm, rotate and append in one pass: q [N, Hq, D], k and v [N, Hkv, D] (bf16; rows may be
    views of one projection's output), token n into slot[n] of request req[n] (int32 [N]).
    q_norm, k_norm: bf16 [D] weights of the per-head RMS norm; cos_sin: fp32 [positions, rot],
    cosines then sines, with pos int32 [N].  Returns the queries, bf16 [N, Hq, D] (q None: only
    keys and values, returns None)."""
    di, (_, heads, _, D), st = cache._view()
    N = k.shape[0]
    kp, ldk = _rows(k, "k", heads, D, di)
    vp, ldv = _rows(v, "v", heads, D, di)
    if v.shape[0] != N:
        raise ValueError("k and v must have the same tokens")
    Hq, qp, ldq, op = 0, None, 0, None
    if q is not None:
        if q.dim() != 3 or q.shape[0] != N:
            raise ValueError(f"q must be [{N}, Hq, {D}]")
        Hq = q.shape[1]
        qp, ldq = _rows(q, "q", Hq, D, di)
        if out is None:
            out = _empty((N, Hq, D), dtype=_BF16, device=q.device)
            op = out.data_ptr()
        else:
            op = _arg(out, _BF16, (N, Hq, D), di, "out")
    rot, positions, cp, pp = 0, 0, None, None
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [positions, rot]")
        if pos is None:
            raise ValueError("a rotation needs pos")
        positions, rot = cos_sin.shape
        cp = _arg(cos_sin, _F32, cos_sin.shape, di, "cos_sin")
        pp = _arg(pos, _I32, (N,), di, "pos")
    qn = None if q_norm is None else _arg(q_norm, _BF16, (D,), di, "q_norm")
    kn = None if k_norm is None else _arg(k_norm, _BF16, (D,), di, "k_norm")
    tp, requests, pages = _table(table, di)
    status = load().bsf8_qkv_append(qp, kp, vp, ldq, ldk, ldv, op, st, tp, requests, pages,
                                    _arg(req, _I32, (N,), di, "req"), _arg(slot, _I32, (N,), di, "slot"), pp, cp,
                                    positions, rot, 1 if interleaved else 0, qn, kn, eps, N, Hq, _raw_stream(di))
    if status:
        _check(status, "bsf8_qkv_append")
    return out if q is not None else None


def kv_read(cache: KVCache, table, req, slot, *, k_out=None, v_out=None):
    """Cached tokens as bf16: (k, v), each [N, Hkv, D], of slot[n] of request req[n]."""
    di, (_, heads, _, D), st = cache._view()
    N = req.shape[0]
    shape = (N, heads, D)
    if k_out is None:
        k_out = _empty(shape, dtype=_BF16, device=req.device)
    if v_out is None:
        v_out = _empty(shape, dtype=_BF16, device=req.device)
    tp, requests, pages = _table(table, di)
    status = load().bsf8_kv_read(st, tp, requests, pages, _arg(req, _I32, (N,), di, "req"),
                                 _arg(slot, _I32, (N,), di, "slot"), _arg(k_out, _BF16, shape, di, "k_out"),
                                 _arg(v_out, _BF16, shape, di, "v_out"), N, _raw_stream(di))
    if status:
        _check(status, "bsf8_kv_read")
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
    lib = load()
    di, (_, heads, size, D), st = cache._view()
    if q.dtype is not _BF16 or q.get_device() != di:
        _refuse(q, _BF16, None, di, "q")
    if q.dim() != 4 or q.shape[3] != D:
        raise ValueError(f"q must be [B, T, Hq, {D}]")
    B, T, Hq, _ = shape = q.shape
    sb, ldq, sh, sc = q.stride()
    if T == 1:
        ldq = sb if B > 1 else Hq * D
    if sc != 1 or (Hq > 1 and sh != D) or (B > 1 and sb != T * ldq):
        raise ValueError(f"q must have strides (T * ld, ld, {D}, 1)")
    tp, requests, pages = _table(table, di)
    if requests != B:
        raise ValueError("table must have a row for each request")
    if out is None:
        out = _empty(shape, dtype=_BF16, device=q.device)
    need = lib.bsf8_tree_attention_workspace_bytes(B, T, Hq, heads, D)
    ws, ws_bytes = None, 0
    if need:
        if workspace is None:
            workspace = _empty((need,), dtype=_U8, device=q.device)
        ws, ws_bytes = _arg(workspace, _U8, workspace.shape, di, "workspace"), workspace.numel()
    status = lib.bsf8_tree_attention(
        q.data_ptr(), ldq, st, tp, pages, _arg(ctx, _I32, (B,), di, "ctx"),
        None if nodes is None else _arg(nodes, _I32, (B,), di, "nodes"),
        None if mask is None else _arg(mask, _I32, (B, T, (T + 31) // 32), di, "mask"),
        D ** -0.5 if scale is None else scale, pages * size if max_len is None else max_len,
        _arg(out, _BF16, shape, di, "out"), None if lse is None else _arg(lse, _F32, (B, T, Hq), di, "lse"),
        B, T, Hq, ws, ws_bytes, _raw_stream(di))
    if status:
        _check(status, "bsf8_tree_attention")
    return out


def verify_tree(p, tokens, parent, u, *, q=None, nodes=None):
    """Which drafted nodes are kept: p fp32 [B, T, V], the target's distribution after each node; q
    likewise the draft's (None: drafts that were not drawn at random); tokens and parent int32
    [B, T]; u fp32 [B, T] uniform numbers (u[b, 0] draws the next token); nodes int32 [B].
    Returns (path int32 [B, T]: the kept nodes, then -1; count int32 [B]; token int32 [B])."""
    if p.dim() != 3:
        raise ValueError("p must be [B, T, V]")
    di = p.get_device()
    B, T, V = shape = p.shape
    sb, st, _ = p.stride()
    ld = st if T > 1 else (sb if B > 1 else V)
    for name, t in (("p", p), ("q", q)):
        if t is None:
            continue
        if t.dtype is not _F32 or t.get_device() != di or di < 0:
            _refuse(t, _F32, None, di, name)
        tb, tt, tv = t.stride()
        if t.shape != shape or (V > 1 and tv != 1) or (T > 1 and tt != ld) or (B > 1 and tb != T * ld):
            raise ValueError(f"{name} must be [B, T, V] with strides (T * ld, ld, 1), p's and q's ld the same")
    # the three outputs in one allocation
    buf = _empty((B * T + 2 * B,), dtype=_I32, device=p.device)
    path, count, token = buf[:B * T].view(B, T), buf[B * T:B * T + B], buf[B * T + B:]
    at = buf.data_ptr()
    status = load().bsf8_verify_tree(
        p.data_ptr(), None if q is None else q.data_ptr(), ld, _arg(tokens, _I32, (B, T), di, "tokens"),
        _arg(parent, _I32, (B, T), di, "parent"), _arg(u, _F32, (B, T), di, "u"),
        None if nodes is None else _arg(nodes, _I32, (B,), di, "nodes"), at, at + 4 * B * T, at + 4 * (B * T + B),
        B, T, V, _raw_stream(di))
    if status:
        _check(status, "bsf8_verify_tree")
    return path, count, token


def kv_commit(cache: KVCache, table, ctx, path, count):
    """Moves the kept nodes together, in place: slot ctx[b] + path[b][i] -> ctx[b] + i for
    i < count[b] (path and count as verify_tree returns them)."""
    di, _, st = cache._view()
    if path.dim() != 2:
        raise ValueError("path must be [B, T]")
    B, T = path.shape
    tp, requests, pages = _table(table, di)
    if requests != B:
        raise ValueError("table must have a row for each request")
    status = load().bsf8_kv_commit(st, tp, pages, _arg(ctx, _I32, (B,), di, "ctx"), _arg(path, _I32, (B, T), di, "path"),
                                   _arg(count, _I32, (B,), di, "count"), B, T, _raw_stream(di))
    if status:
        _check(status, "bsf8_kv_commit")
