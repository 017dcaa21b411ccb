"""GPU: the residual between two blocks against 64 bits."""
import numpy as np
import pytest
import torch

import _step_ref as ref
import block_scaled_fp8_weight_gb300 as bsf8

pytestmark = pytest.mark.gpu

EPS = 1e-5


def bf16(r, *shape, scale=1.0):
    return torch.from_numpy((r.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16).cuda()


def f64(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def compare(h, r, x, res, w, post, gate, scale):
    """r: fp32 arithmetic of three products and a sum, 2^-20 of what goes into it (the mean's sum of n terms, added
    in at most 12 + n / 1024 steps a thread and tree, its root and the product included: below 16 roundings of
    2^-24), then its rounding; h: the same through k * weight, and its own roundings."""
    zero = np.zeros(x.shape) if res is None else f64(res)
    wh, wr, mass, k = ref.norm(f64(x), zero, 1.0 if w is None else f64(w), f64(post), f64(gate), float(np.float32(scale)), EPS)
    if r is not None:
        step = 2.0 ** -8 if r.dtype == torch.bfloat16 else 2.0 ** -24
        assert np.all(np.abs(f64(r) - wr) <= np.abs(wr) * step * (1 + 2.0 ** -8) + mass * 2.0 ** -19 + 2.0 ** -133)
    if h is not None:
        assert np.all(np.abs(f64(h) - wh) <= np.abs(wh) * (2.0 ** -8 + 2.0 ** -18) * (1 + 2.0 ** -8) + k * mass * 2.0 ** -19 + 2.0 ** -133)


@pytest.mark.parametrize("M,H", [(1, 8), (3, 64), (6, 5120), (17, 248), (65, 2056), (130, 1024), (1, 8192), (5, 8200), (40, 16384),
                                 (3, 16392), (2, 32768), (1300, 256), (2500, 5120),
                                 (7000, 264), (1300, 8192), (700, 12296)])
@pytest.mark.parametrize("fp32,post,gate", [(False, False, None), (True, True, "channel"), (False, True, "token"), (True, False, "full")])
def test_norm(bsf8_lib, M, H, fp32, post, gate):
    r = np.random.default_rng(M + H)
    x, res, w = bf16(r, M, H, scale=3.0), bf16(r, M, H, scale=2.0), bf16(r, H)
    if fp32:
        res = res.float() + 0.01
    p = bf16(r, H) if post else None
    g = {None: None, "channel": bf16(r, H), "token": bf16(r, M, 1), "full": bf16(r, M, H)}[gate]
    h, o = bsf8.residual_norm(x, res, w, post_weight=p, gate=g, scale=0.7, eps=EPS)
    assert h.dtype == torch.bfloat16 and o.dtype == res.dtype and h.shape == o.shape == x.shape
    compare(h, o, x, res, w, p, g, 0.7)


@pytest.mark.parametrize("fp32", [False, True])
def test_strides_outputs_in_place_and_parts(bsf8_lib, fp32):
    r = np.random.default_rng(5)
    M, H = 37, 520
    big = bf16(r, M, 3 * H)
    x, g = big[:, H:2 * H], big[:, 2 * H:]
    gt = big[:, 7:8]  # a token gate that is a column of something
    wide = bf16(r, M, H + 16)
    res = (wide.float() if fp32 else wide)[:, 8:8 + H]
    w, p = bf16(r, H), bf16(r, H)
    h, o = bsf8.residual_norm(x, res, w, post_weight=p, gate=g, scale=-1.25, eps=EPS)
    compare(h, o, x, res, w, p, g, -1.25)
    h, o = bsf8.residual_norm(x, res, w, gate=gt, eps=EPS)
    compare(h, o, x, res, w, None, gt, 1.0)
    # the residual in place, h into x's own memory
    x1, r1 = x.contiguous(), res.contiguous()
    x0, r0 = x1.clone(), r1.clone()
    h, o = bsf8.residual_norm(x1, r1, w, post_weight=p, out=x1, residual_out=r1, eps=EPS)
    assert h is x1 and o is r1
    compare(h, o, x0, r0, w, p, None, 1.0)
    # without a weight only the sum, without a residual only the norm
    h, o = bsf8.residual_norm(x, res, None, post_weight=p, eps=EPS)
    assert h is None
    compare(None, o, x, res, None, p, None, 1.0)
    h, o = bsf8.residual_norm(x, None, w, eps=EPS)
    assert o is None
    compare(h, None, x, None, w, None, None, 1.0)
    keep = torch.empty(M, H, device="cuda", dtype=torch.float32)
    h, o = bsf8.residual_norm(x, None, w, post_weight=p, residual_out=keep, eps=EPS)
    compare(h, o, x, None, w, p, None, 1.0)
    h, o = bsf8.residual_norm(x[:0], res[:0], w)
    assert h.shape == o.shape == (0, H)


def test_values_at_the_ends(bsf8_lib):
    """Zeros, a row of one large channel, infinities and NaN: only their own rows are touched."""
    M, H = 6, 768
    x = torch.zeros(M, H, device="cuda", dtype=torch.bfloat16)
    res = torch.zeros_like(x)
    x[1, 5], res[2, 700], res[3, 3], x[4, 9] = 2.0 ** 60, 1e-30, float("inf"), float("nan")
    x[5], res[5] = 1.0, 1.0
    w = torch.ones(H, device="cuda", dtype=torch.bfloat16)
    h, o = bsf8.residual_norm(x, res, w, post_weight=w, eps=EPS)
    assert not h[0].any() and not o[0].any()
    compare(h[[0, 1, 2, 5]], o[[0, 1, 2, 5]], x[[0, 1, 2, 5]], res[[0, 1, 2, 5]], w, w, None, 1.0)
    assert torch.isinf(o[3, 3]) and torch.isnan(h[3, 3]) and not h[3, :3].any()  # 1 / inf is 0
    assert torch.isnan(h[4]).all() and torch.isnan(o[4]).all()


def test_same_bits_whatever_else_is_in_the_call(bsf8_lib):
    """A row's result depends on the row alone."""
    r = np.random.default_rng(9)
    x, res, w = bf16(r, 700, 5120), bf16(r, 700, 5120).float(), bf16(r, 5120)
    h, o = bsf8.residual_norm(x, res, w, post_weight=w)
    for i in (0, 1, 333, 699):
        a, b = bsf8.residual_norm(x[i:i + 1], res[i:i + 1], w, post_weight=w)
        assert torch.equal(a[0], h[i]) and torch.equal(b[0], o[i])


@pytest.mark.parametrize("H", [200, 1000, 2056, 5120, 7168, 8192, 12288, 16392])
@pytest.mark.parametrize("fp32", [False, True])
def test_same_bits_in_calls_of_every_size(bsf8_lib, H, fp32):
    """The kernels for few and for many rows add up a row's squares in one order."""
    r = np.random.default_rng(H)
    M = 2600 if H < 8000 else 700
    x, res, w, g = bf16(r, M, H, scale=3.0), bf16(r, M, H), bf16(r, H), bf16(r, M, H)
    if fp32:
        res = res.float() * 1.001
    for post in (None, w):
        for gate in (None, g):
            h, o = bsf8.residual_norm(x, res, w, post_weight=post, gate=gate)
            for n in (1, 9, 150, 450, 1300):
                a, b = bsf8.residual_norm(x[-n:], res[-n:], w, post_weight=post, gate=None if gate is None else g[-n:])
                assert torch.equal(a, h[-n:]) and torch.equal(b, o[-n:])


def test_refused_tensors(bsf8_lib):
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    f = bsf8.residual_norm
    for bad in (lambda: f(x.float(), x, w), lambda: f(x, x.half(), w), lambda: f(x, x, w.float()), lambda: f(x, x, w, gate=w.float())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: f(x, x[:3], w), lambda: f(x, x, w[:32]), lambda: f(x, x, w, gate=x[:, :2]), lambda: f(x, x, w, gate=x[None]),
                lambda: f(x[0], x, w), lambda: f(x.T, x.T, w[:4]), lambda: f(x, x, w, out=x[:2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(bsf8.Bsf8Error):
        f(x, None, None)  # nothing to write
    with pytest.raises(bsf8.Bsf8Error):
        f(x[:, 1:57], x[:, 8:], w[:56])  # not 16-byte aligned


def test_an_output_that_nothing_writes_is_refused(bsf8_lib):
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    out = torch.full_like(x, 3.0)
    for residual, residual_out in ((x, None), (None, torch.empty_like(x)), (None, None)):
        with pytest.raises(ValueError, match="out needs weight"):
            bsf8.residual_norm(x, residual, None, out=out, residual_out=residual_out)
    assert (out == 3).all()


@pytest.mark.parametrize("M,H", [(3000, 5120), (1500, 7168)])  # one row ahead, and two
def test_a_wait_that_runs_out_is_reported(bsf8_lib, M, H):
    """No loads are issued (a test-only option): the kernel for many rows gives up its waits and says so."""
    x = torch.ones(M, H, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(H, device="cuda", dtype=torch.bfloat16)
    res = x.float()
    h = torch.full_like(x, 7.0)
    try:
        bsf8.set_option(bsf8.OPT_DEBUG_SKIP_LOADS, 1)
        bsf8.set_option(bsf8.OPT_WAIT_TIMEOUT_NS, 1000000)
        bsf8.residual_norm(x, res, w, post_weight=w, out=h)
        assert bsf8.device_status() == 7 and (h == 7).all()
    finally:
        bsf8.set_option(bsf8.OPT_DEBUG_SKIP_LOADS, 0)
        bsf8.set_option(bsf8.OPT_WAIT_TIMEOUT_NS, 2000000000)
    bsf8.residual_norm(x, res, w, post_weight=w, out=h)
    assert bsf8.device_status() == 0 and (h == 1).all()
