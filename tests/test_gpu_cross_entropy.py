"""sbl_linear_cross_entropy and its backward on the GPU against the formulas in
64 bits.

Bounds.  u = 2^-24.  A logit is a sum of D exact products in fp32: tensor-core
sums over segments of 1024 terms, rounded towards zero 64 times (each at most
2 u of the running sum), and the segments added to nearest: |z - z*| <= e =
(128 + D / 1024 + 2) u A, A = max_v sum_d |x W|.  Each exponential adds a relative
2^-22 (the special function unit's) and (|z - m| + 2) u of its argument's
rounding, and V of them are added in groups (at most 128 / 4 + 12 in sequence, then
V / (128 * 32) + 32 parts), the logarithm an absolute 2 u |lse| + 2^-22:
|lse - lse*| <= e + L with L = 2^-21 + (44 + V / 4096 + 40 + 100) u + 3 u |lse*|
(exponents below -100 contribute nothing), and the loss' difference adds its own
rounding: 2 e + L + u |loss*|.

G = (p - [v == target]) d with d = dloss / c, c = max |dloss|: p has a relative
error of eps_p = expm1(e + e2 + L) + 2^-20, where e2 = (2 D / 16 + 2) u A is the
error of the backward's own logits, summed by the tensor cores without segments;
G is rounded to bf16 (half a step: finfo(bfloat16).eps / 2 = 2^-8, as 8
significand bits space values 2^-7 apart just above 1), d and the product to
fp32.  A sum of n terms on the tensor cores has n / 16 roundings towards zero of
2 u; dX adds its pieces to nearest.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16 = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module")
def sbl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_linear_layers_b200 as m
    return m


def _inputs(T, D, V, seed, scale=1.5):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(V, D, generator=g) * (scale / D ** 0.5)
    t = torch.randint(0, V, (T,), generator=g)
    x = torch.randn(T, D, generator=g) + 4.0 * (torch.rand(T, 1, generator=g) < 0.4) * w[t]
    t = torch.where(torch.rand(T, generator=g) < 0.15, -100, t)
    return x.bfloat16(), w.bfloat16(), t


def _refs(x, w, t, d, ignore=-100):
    x, w, d = x.double(), w.double(), d.double()
    T, V = x.shape[0], w.shape[0]
    z = x @ w.T
    lse = torch.logsumexp(z, 1)
    live = t != ignore
    col = torch.where(live, t, 0)
    loss = torch.where(live, lse - z.gather(1, col[:, None])[:, 0], 0.0)
    p = torch.softmax(z, 1)
    hot = torch.zeros_like(p)
    hot[live.nonzero()[:, 0], col[live]] = 1.0
    d = torch.where(live, d, 0.0)[:, None]
    return z, lse, loss, p, hot, d


def _bounds(x, w, z, lse, loss):
    T, D = x.shape
    V = w.shape[0]
    A = (x.double().abs() @ w.double().abs().T).amax(1)
    e = (128 + D / 1024 + 2) * U * A
    e2 = (2 * D / 16 + 2) * U * A
    L = 2.0 ** -21 + (184 + V / 4096) * U + 3 * U * lse.abs()
    return e, e2, L


def _grad_bounds(x, w, p, hot, d, e, e2, L):
    """Element bounds of dX and dW: |G| bf16-rounded relative to c, p off by eps."""
    xa, wa = x.double().abs(), w.double().abs()
    eps = (torch.expm1(e + e2 + L) + 2.0 ** -20)[:, None]
    G = (p - hot) * d
    # p's error before the subtraction, then the bf16 rounding and two fp32 ones
    # up to 128 tokens G goes as two bf16 parts, which keep all but 2^-16 of it
    T, V = p.shape
    dG = (p * eps * d.abs()) * (1 + BF16) + G.abs() * ((BF16 if T > 128 else BF16 ** 2) + 4 * U)
    Ga = G.abs() + dG
    ref = G @ w.double(), G.T @ x.double()
    n = 2 if T > 128 else 4  # units of 2^-24 per 16 terms: one or two MMAs
    bx = dG @ wa + (n * V / 16 + 64) * U * (Ga @ wa)
    bw = dG.T @ xa + (n * T / 16 + 8) * U * (Ga.T @ xa)
    out = BF16  # the results' own rounding
    tiny = 1e-30
    return (ref[0], bx * (1 + 2 * out) + out * ref[0].abs() + tiny), (ref[1], bw * (1 + 2 * out) + out * ref[1].abs() + tiny)


def _check(name, got, ref, bound):
    got = got.double().to(ref.device)
    assert got.shape == ref.shape
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(((got - ref).abs() / bound.clamp(min=1e-300)).max()))


SHAPES = [(1, 16, 1), (1, 896, 3000), (128, 64, 700), (1, 32, 7), (2, 64, 128), (3, 48, 129), (65, 80, 257), (129, 128, 300), (256, 64, 256),
          (257, 96, 1000), (40, 896, 2500), (333, 144, 5001), (30, 2048, 513), (700, 272, 1111),
          # 512-row tiles in every product, a ragged tail of each, dX in several parts
          (1000, 272, 20011), (3000, 1040, 1500),
          # few tokens: turned tiles of 64 and 128 tokens, words that end inside a warp's 32, dX in many parts
          (32, 16, 33), (33, 48, 95), (63, 272, 20011), (64, 64, 385), (97, 112, 255), (117, 32, 9000), (128, 1040, 2049)]


@pytest.mark.parametrize("T,D,V", SHAPES)
@pytest.mark.parametrize("weights", ["mean", "random"])
def test_loss_and_gradients(sbl, T, D, V, weights):
    x, w, t = _inputs(T, D, V, seed=T + D + V)
    g = torch.Generator().manual_seed(1)
    d = torch.full((T,), 1.0 / T) if weights == "mean" else torch.randn(T, generator=g)
    z, lse, loss, p, hot, dd = _refs(x, w, t, d)
    e, e2, L = _bounds(x, w, z, lse, loss)
    c = lambda v: v.cuda()
    got_loss, got_lse = sbl.sbl_linear_cross_entropy(c(x), c(w), c(t))
    _check("lse", got_lse, lse, e + L)
    _check("loss", got_loss, loss, 2 * e + L + 2 * U * loss.abs())
    assert not got_loss[c(t) == -100].any()
    (dx, bx), (dw, bw) = _grad_bounds(x, w, p, hot, dd, e, e2, L)
    got = sbl.sbl_linear_cross_entropy_backward(c(d), c(x), c(w), c(t), got_lse)
    _check("dx", got[0], dx, bx)
    _check("dw", got[1], dw, bw)
    assert not got[0][c(t) == -100].any()
    for need in ((True, False), (False, True)):
        one = sbl.sbl_linear_cross_entropy_backward(c(d), c(x), c(w), c(t), got_lse, need_dx=need[0], need_dw=need[1])
        for o, r, n in zip(one, got, need):
            assert (o is not None) == n and (o is None or torch.equal(o, r))
    assert sbl.sbl_device_status() == 0


@pytest.mark.parametrize("T,D,V", [(2100, 64, 131001), (3, 16, 1100001)])
def test_several_pieces_of_the_vocabulary(sbl, T, D, V):
    """More logits than one piece of the backward holds (2^28, or 2^20 words of a
    few tokens), the last piece ragged; the 64-bit reference runs on the device."""
    if T > 128:
        assert sbl.sbl_linear_cross_entropy_backward_workspace_bytes(T, D, V, False) < 2 * T * V
    x, w, t = (v.cuda() for v in _inputs(T, D, V, seed=2))
    t[0], t[1] = V - 1, 0
    d = (torch.rand(T, generator=torch.Generator().manual_seed(3)) + 0.5).cuda()
    z, lse, loss, p, hot, dd = _refs(x, w, t, d)
    e, e2, L = _bounds(x, w, z, lse, loss)
    del z
    got_loss, got_lse = sbl.sbl_linear_cross_entropy(x, w, t)
    _check("lse", got_lse, lse, e + L)
    _check("loss", got_loss, loss, 2 * e + L + 2 * U * loss.abs())
    (dx, bx), (dw, bw) = _grad_bounds(x, w, p, hot, dd, e, e2, L)
    got = sbl.sbl_linear_cross_entropy_backward(d, x, w, t, got_lse)
    _check("dx", got[0], dx, bx)
    _check("dw", got[1], dw, bw)


def test_gradient_against_differences(sbl):
    """Central differences of the 64-bit loss; their own error (h^2 times third
    derivatives of order 1) is far below the bf16 bound."""
    T, D, V, h = 5, 32, 50, 1e-4
    x, w, t = _inputs(T, D, V, seed=8)
    t[0] = 3
    d = torch.full((T,), 0.25)
    z, lse, loss, p, hot, dd = _refs(x, w, t, d)
    (_, bx), (_, bw) = _grad_bounds(x, w, p, hot, dd, *_bounds(x, w, z, lse, loss))
    total = lambda a, b: float((dd[:, 0] * _refs(a, b, t, d)[2]).sum())
    _, got_lse = sbl.sbl_linear_cross_entropy(x.cuda(), w.cuda(), t.cuda())
    dx, dw = (v.cpu().double() for v in sbl.sbl_linear_cross_entropy_backward(d.cuda(), x.cuda(), w.cuda(), t.cuda(), got_lse))
    xd, wd = x.double(), w.double()
    for i, k in ((0, 0), (2, 31), (4, 7)):
        a, b = xd.clone(), xd.clone()
        a[i, k] += h
        b[i, k] -= h
        assert abs(float(dx[i, k]) - (total(a, wd) - total(b, wd)) / (2 * h)) <= float(bx[i, k]) + 1e-7
    for v, k in ((3, 0), (49, 5), (20, 30)):
        a, b = wd.clone(), wd.clone()
        a[v, k] += h
        b[v, k] -= h
        assert abs(float(dw[v, k]) - (total(xd, a) - total(xd, b)) / (2 * h)) <= float(bw[v, k]) + 1e-7


def test_large_logits_do_not_overflow(sbl):
    """Logits of some hundreds: the maximum is taken out before exp."""
    x, w, t = _inputs(20, 64, 500, seed=5, scale=200.0)
    z, lse, loss, *_ = _refs(x, w, t, torch.ones(20))
    assert lse.max() > 300
    e, _, L = _bounds(x, w, z, lse, loss)
    got_loss, got_lse = sbl.sbl_linear_cross_entropy(x.cuda(), w.cuda(), t.cuda())
    _check("lse", got_lse, lse, e + L)
    _check("loss", got_loss, loss, 2 * e + L + 2 * U * loss.abs())


def test_likely_words(sbl):
    """Targets of probability close to 1: the loss is far smaller than lse and the
    target's logit.  dloss/dz = p - onehot sums to 2 (1 - p_target) in magnitude, so
    the logits' error e moves the loss by 2 e (1 - p); the exponentials' 2^-21
    acts on the other words only, and at most 100 additions round at a sum near 1."""
    g = torch.Generator().manual_seed(4)
    T, D, V = 300, 256, 3000
    w = torch.randn(V, D, generator=g) / 16
    t = torch.randint(0, V, (T,), generator=g)
    x = (torch.randn(T, D, generator=g) + torch.linspace(8, 30, T)[:, None] * w[t]).bfloat16()
    w = w.bfloat16()
    z, lse, loss, p, *_ = _refs(x, w, t, torch.ones(T))
    assert loss.min() < 1e-6 and loss.max() > 1e-2
    e, _, _ = _bounds(x, w, z, lse, loss)
    rest = 1 - torch.exp(-loss)
    for n in (T, 200):   # more and fewer than 256 tokens
        got, _ = sbl.sbl_linear_cross_entropy(x[:n].cuda().contiguous(), w.cuda(), t[:n].cuda())
        _check("loss", got, loss[:n], ((2 * e + 2.0 ** -21) * rest + 100 * U)[:n])


def test_empty_all_ignored_and_bad_targets(sbl):
    w = torch.randn(100, 32, device="cuda").bfloat16()
    x = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")
    t = torch.empty((0,), dtype=torch.int64, device="cuda")
    loss, lse = sbl.sbl_linear_cross_entropy(x, w, t)
    assert loss.shape == lse.shape == (0,)
    dx, dw = sbl.sbl_linear_cross_entropy_backward(loss, x, w, t, lse)
    assert dx.shape == (0, 32) and dw.shape == (100, 32) and not dw.any()
    x = torch.randn(9, 32, device="cuda").bfloat16()
    t = torch.full((9,), 7, device="cuda")
    loss, lse = sbl.sbl_linear_cross_entropy(x, w, t, ignore_index=7)
    assert not loss.any() and torch.isfinite(lse).all()
    dx, dw = sbl.sbl_linear_cross_entropy_backward(torch.ones(9, device="cuda"), x, w, t, lse, ignore_index=7)
    assert not dx.any() and not dw.any()
    # zero weights of the losses
    dx, dw = sbl.sbl_linear_cross_entropy_backward(torch.zeros(9, device="cuda"), x, w, t, lse)
    assert not dx.any() and not dw.any()
    assert sbl.sbl_device_status() == 0
    for wrong in (100, -1, 1 << 40):
        t2 = t.clone()
        t2[4] = wrong
        loss, lse = sbl.sbl_linear_cross_entropy(x, w, t2)
        assert sbl.sbl_device_status() == 1     # SBL_ERR_INVALID_ARG
        assert torch.isnan(loss[4]) and torch.isfinite(loss[[0, 1, 2, 3, 5, 6, 7, 8]]).all()
        dx, dw = sbl.sbl_linear_cross_entropy_backward(torch.ones(9, device="cuda"), x, w, t2, lse)
        assert not dx[4].any() and torch.isfinite(dw).all()


@pytest.mark.parametrize("T", [9, 300])
def test_nonfinite_ignored_rows(sbl, T):
    """NaN, Inf and overflowing logits in the rows of ignored tokens (padding that
    nothing ever wrote) change nothing of the other tokens, and their own loss
    and dx are 0."""
    x, w, t = [v.cuda() for v in _inputs(T, 64, 700, seed=21)]
    t[torch.tensor([1, 4, 6])] = -100
    d = torch.full((T,), 0.5, device="cuda")
    run = lambda xv: (lambda loss, lse: (loss, sbl.sbl_linear_cross_entropy_backward(d, xv, w, t, lse, need_dw=False)[0]))(
        *sbl.sbl_linear_cross_entropy(xv, w, t))
    loss, dx = run(x)
    bad = x.clone()
    bad[1] = float("nan")
    bad[4, 3] = float("inf")
    bad[6] = 3e38
    got_loss, got_dx = run(bad)
    assert torch.equal(got_loss, loss) and torch.equal(got_dx, dx)
    assert not got_loss[[1, 4, 6]].any() and not got_dx[[1, 4, 6]].any()


def test_other_stream_and_graph(sbl):
    c = lambda vs: [v.cuda() for v in vs]
    x, w, t = c(_inputs(300, 96, 3000, seed=11))
    d = torch.full((300,), 1 / 300, device="cuda")

    def step(xv, tv, stream=None):
        loss, lse = sbl.sbl_linear_cross_entropy(xv, w, tv, stream=stream)
        return (loss, lse, *sbl.sbl_linear_cross_entropy_backward(d, xv, w, tv, lse, stream=stream))

    ref = step(x, t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(x, t, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, r in zip(got, ref):
        assert torch.equal(a, r)
    sx, sti = x.clone(), t.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = step(sx, sti)
    x2, _, t2 = c(_inputs(300, 96, 3000, seed=12))
    sx.copy_(x2)
    sti.copy_(t2)
    g.replay()
    g.replay()
    for a, r in zip(cap, step(x2, t2)):
        assert torch.equal(a, r)
