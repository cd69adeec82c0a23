"""sbl_norm and sbl_norm_backward on the GPU against the formulas in 64 bits.

Bounds.  u = 2^-24.  A row's sums run over at most D = 40 + K / 4096 additions
in sequence (8 columns in a thread, 5 + 5 shuffle steps, the groups of a long
row), so |mean - mean*| <= E = (D + 3) u max|x|, which also covers the
subtraction's rounding.  rstd then has a relative error of at most
E rstd + (D / 2 + 6) u, and xhat one of X = E rstd + |xhat| (E rstd + (D / 2 + 6) u).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def sbl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_linear_layers_b200 as m
    return m


def _inputs(T, K, dtype, seed, offset=0.3):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, K, generator=g) + offset).to(dtype)
    dy = torch.randn(T, K, generator=g).to(dtype)
    w = 1 + 0.2 * torch.randn(K, generator=g)
    b = 0.3 * torch.randn(K, generator=g)
    return x, dy, w, b


def _stats(x, kind, eps):
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros(x.shape[0], 1, dtype=torch.float64)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    return mean, rstd


def _xhat_bound(x, kind, eps):
    """xhat, its bound X and the depth D."""
    K = x.shape[1]
    mean, rstd = _stats(x, kind, eps)
    xh = (x - mean) * rstd
    D = 40 + K / 4096
    E = (D + 3) * U * x.abs().amax(1, keepdim=True)
    return xh, E * rstd + xh.abs() * (E * rstd + (D / 2 + 6) * U), D


def _check(name, got, ref, bound):
    got = got.double().cpu()
    assert got.shape == ref.shape
    bad = (got - ref).abs() > bound
    assert not bad.any(), (name, int(bad.sum()), float(((got - ref).abs() / bound.clamp(min=1e-300)).max()))


def _forward_bound(x, w, b, kind, eps, dtype):
    xh, X, _ = _xhat_bound(x, kind, eps)
    y = xh * w + (b if b is not None else 0.0)
    out = torch.finfo(dtype).eps / 2  # the output's rounding
    return y, w.abs() * (X + 2 * U * xh.abs()) * (1 + 2 * out) + (out + U) * y.abs()


def _backward_refs(x, dy, w, kind, eps, dtype):
    T, K = x.shape
    xh, X, D = _xhat_bound(x, kind, eps)
    _, rstd = _stats(x, kind, eps)
    q = dy * w
    m1 = (q * xh).mean(1, keepdim=True)
    m0 = q.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(m1)
    dx = rstd * (q - m0 - xh * m1)
    m1_err = (q.abs() * X).mean(1, keepdim=True) + (D + 3) * U * (q * xh).abs().mean(1, keepdim=True)
    m0_err = (D + 3) * U * q.abs().mean(1, keepdim=True) if kind == "layer" else 0.0
    size = q.abs() + m0.abs() + (xh * m1).abs()
    out = torch.finfo(dtype).eps / 2
    # rstd itself is one rounding of the exact value here
    dx_bound = rstd * (m0_err + xh.abs() * m1_err + X * (m1.abs() + m1_err) + 6 * U * size) * (1 + 2 * out) \
        + out * dx.abs()
    dw, db = (dy * xh).sum(0), dy.sum(0)
    # at most T + 96 additions in sequence
    dw_bound = (dy.abs() * X).sum(0) + (T + 99) * U * (dy * xh).abs().sum(0)
    db_bound = (T + 99) * U * dy.abs().sum(0)
    return (dx, dx_bound), (dw, dw_bound), (db, db_bound)


SHAPES = [(1, 16), (1, 2048), (3, 48), (7, 256), (5, 272), (33, 896), (130, 2048), (9, 4864), (4, 5136), (6, 8192),
          (3, 8208), (35, 16400), (2500, 64), (1500, 896),
          # many rows: the streaming kernels, with a ragged last tile, each number of
          # columns per thread and, in fp32, tiles of one row
          (10001, 16), (9601, 272), (2503, 1040), (1301, 2064), (901, 5120), (601, 5136), (701, 10240), (100001, 16),
          (7003, 400)]


@pytest.mark.parametrize("T,K", SHAPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_forward_and_backward(sbl, T, K, kind, dtype):
    eps = 1e-5
    x, dy, w, b = _inputs(T, K, dtype, seed=T + K)
    xd, dyd, wd = x.double(), dy.double(), w.double()
    use_b = kind == "layer" or K % 32 == 0
    c = lambda t: t.cuda()
    y, mean, rstd = sbl.sbl_norm(c(x), c(w), c(b) if use_b else None, kind=kind, eps=eps, with_stats=True)
    ref, bound = _forward_bound(xd, wd, b.double() if use_b else None, kind, eps, dtype)
    assert y.dtype == dtype
    _check("y", y, ref, bound)
    assert (mean is None) == (kind == "rms")
    m64, r64 = _stats(xd, kind, eps)
    _, X, D = _xhat_bound(xd, kind, eps)
    E = (D + 3) * U * xd.abs().amax(1)
    _check("rstd", rstd, r64[:, 0], r64[:, 0] * (E * r64[:, 0] + (D / 2 + 6) * U))
    if kind == "layer":
        _check("mean", mean, m64[:, 0], E)
    # backward on the exact statistics rounded once
    st = [None if kind == "rms" else m64[:, 0].float().cuda(), r64[:, 0].float().cuda()]
    refs = _backward_refs(xd, dyd, wd, kind, eps, dtype)
    got = sbl.sbl_norm_backward(c(dy), c(x), c(w), *st, kind=kind)
    for name, t, (r, bd) in zip(("dx", "dw", "db"), got, refs):
        _check(name, t, r, bd)
    assert got[0].dtype == dtype and got[1].dtype == got[2].dtype == torch.float32
    # each gradient alone gives the same bits, and so does a second call
    for i, need in enumerate(((True, False, False), (False, True, False), (False, False, True))):
        one = sbl.sbl_norm_backward(c(dy), c(x), c(w), *st, kind=kind, need_dx=need[0], need_dw=need[1],
                                    need_db=need[2])
        assert [o is not None for o in one] == list(need)
        assert torch.equal(one[i], got[i])


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_gradient_against_differences(sbl, kind):
    """Central differences of the 64-bit loss sum(dy * y): with a step h the
    difference is off by at most h^2 / 6 max|f'''| (below 1e-9 here) and its
    rounding (1e-16 / h), both far below the kernel's own bound."""
    T, K, eps, h = 3, 32, 1e-3, 1e-5
    x, dy, w, b = _inputs(T, K, torch.float32, seed=4)
    xd, dyd, wd = x.double(), dy.double(), w.double()

    def loss(xv, wv):
        mean, rstd = _stats(xv, kind, eps)
        return (dyd * ((xv - mean) * rstd * wv)).sum()

    _, mean, rstd = sbl.sbl_norm(x.cuda(), w.cuda(), None, kind=kind, eps=eps, with_stats=True)
    dx, dw, _ = sbl.sbl_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd, kind=kind)
    (_, dxb), (_, dwb), _ = _backward_refs(xd, dyd, wd, kind, eps, torch.float32)
    for t, k in ((0, 0), (1, 7), (2, 31), (0, 16)):
        p, q = xd.clone(), xd.clone()
        p[t, k] += h
        q[t, k] -= h
        num = (loss(p, wd) - loss(q, wd)) / (2 * h)
        # the kernel's own statistics add their error once more
        assert abs(float(dx[t, k]) - float(num)) <= 2 * float(dxb[t, k]) + 1e-8
    for k in (0, 5, 31):
        p, q = wd.clone(), wd.clone()
        p[k] += h
        q[k] -= h
        num = (loss(xd, p) - loss(xd, q)) / (2 * h)
        assert abs(float(dw[k]) - float(num)) <= 2 * float(dwb[k]) + 1e-8


def test_far_from_zero_mean(sbl):
    """A row whose offset is 1000 times its spread: the variance comes from
    differences, so the bound with E = (D + 3) u max|x| holds."""
    x, _, w, b = _inputs(4, 896, torch.float32, seed=9, offset=1000.0)
    y = sbl.sbl_norm(x.cuda(), w.cuda(), b.cuda(), kind="layer", eps=0.0)
    ref, bound = _forward_bound(x.double(), w.double(), b.double(), "layer", 0.0, torch.float32)
    _check("y", y, ref, bound)


def test_empty_and_constant_rows(sbl):
    w = torch.ones(64, device="cuda")
    e = torch.empty((0, 64), device="cuda")
    y, mean, rstd = sbl.sbl_norm(e, w, kind="layer", with_stats=True)
    assert y.shape == (0, 64) and mean.shape == rstd.shape == (0,)
    dx, dw, db = sbl.sbl_norm_backward(e, e, w, mean, rstd, kind="layer")
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    # a constant row has no spread: layer norm gives the bias, whatever eps > 0
    x = torch.full((2, 64), 3.0, device="cuda")
    b = torch.arange(64.0, device="cuda")
    assert torch.equal(sbl.sbl_norm(x, w, b, kind="layer", eps=1e-5)[1], b)


def test_nonfinite_rows_stay_alone(sbl):
    x, dy, w, b = (t.cuda() for t in _inputs(6, 512, torch.float32, seed=3))
    good = sbl.sbl_norm(x, w, b, kind="layer")
    x2 = x.clone()
    x2[2, 5] = float("nan")
    x2[4, 9] = float("inf")
    y = sbl.sbl_norm(x2, w, b, kind="layer")
    keep = [0, 1, 3, 5]
    assert torch.equal(y[keep], good[keep])
    assert torch.isnan(y[2]).all() and torch.isnan(y[4]).any()


def test_other_stream_and_graph(sbl):
    x, dy, w, b = (t.cuda() for t in _inputs(300, 896, torch.bfloat16, seed=5))

    def both(xv, dyv, stream=None):
        y, mean, rstd = sbl.sbl_norm(xv, w, b, kind="layer", with_stats=True, stream=stream)
        return (y, *sbl.sbl_norm_backward(dyv, xv, w, mean, rstd, kind="layer", stream=stream))

    ref = both(x, dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = both(x, dy, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, r in zip(got, ref):
        assert torch.equal(a, r)
    sx, sdy = x.clone(), dy.clone()
    both(sx, sdy)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = both(sx, sdy)
    x2, dy2 = (t.cuda() for t in _inputs(300, 896, torch.bfloat16, seed=6)[:2])
    sx.copy_(x2)
    sdy.copy_(dy2)
    g.replay()
    g.replay()
    for a, r in zip(cap, both(x2, dy2)):
        assert torch.equal(a, r)
