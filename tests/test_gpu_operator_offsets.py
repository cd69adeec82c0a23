"""Norms, the gated feed-forward block and the cross entropy on matrices of more
than 2^31 elements: the far rows against the same 64-bit references and bounds as
the small cases."""
import pytest
import torch

import test_gpu_cross_entropy as ce
import test_gpu_norm as nm
from test_gpu_ffn_gated import Case

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def sbl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.get_device_properties(0).total_memory < 120 << 30:
        pytest.skip("needs 60 GB on the device")
    import sparse_linear_layers_b200 as m
    yield m
    torch.cuda.empty_cache()


def test_norm(sbl):
    """Zero rows, then a few at the end: only those have gradients."""
    T, K, n = 270001, 8192, 40
    assert T * K > 2 ** 31
    g = torch.Generator().manual_seed(1)
    far, far_dy = torch.randn(n, K, generator=g).bfloat16(), torch.randn(n, K, generator=g).bfloat16()
    w, b = torch.rand(K, generator=g) + 0.5, torch.randn(K, generator=g)
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros_like(x)
    x[-n:], dy[-n:] = far.cuda(), far_dy.cuda()
    y, mean, rstd = sbl.sbl_norm(x, w.cuda(), b.cuda(), kind="layer", with_stats=True)
    eps = sbl.RMSNORM_EPS_F32
    nm._check("y", y[-n:], *nm._forward_bound(far.double(), w.double(), b.double(), "layer", eps, torch.bfloat16))
    assert torch.equal(y[0], b.cuda().bfloat16()) and torch.equal(y[T - n - 1], y[0])
    dx, dw, db = sbl.sbl_norm_backward(dy, x, w.cuda(), mean, rstd, kind="layer")
    refs = nm._backward_refs(far.double(), far_dy.double(), w.double(), "layer", eps, torch.bfloat16)
    # on the forward's own fp32 statistics: twice the bound; the zero rows add exact zeros
    for name, got, (ref, bound) in zip(("dx", "dw", "db"), (dx[-n:], dw, db), refs):
        nm._check(name, got, ref, 2 * bound)
    assert not dx[:1000].any() and not dx[-n - 1000:-n].any()


@pytest.mark.parametrize("T", [5, 200])
def test_cross_entropy(sbl, T):
    """A vocabulary whose last words lie past 2^31 elements, two of them targets."""
    D, V = 2048, 1100001
    assert D * V > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.empty(V, D, dtype=torch.bfloat16, device="cuda").normal_(std=0.03, generator=g)
    x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    t = torch.randint(0, V, (T,), device="cuda", generator=g)
    t[0], t[1] = V - 1, V - 2
    d = torch.rand(T, device="cuda", generator=g) + 0.5
    xd, pieces = x.double(), range(0, V, 100000)
    z = torch.cat([xd @ w[i:i + 100000].double().T for i in pieces], 1)
    A = torch.stack([(xd.abs() @ w[i:i + 100000].double().abs().T).amax(1) for i in pieces]).amax(0)
    lse, e, e2 = torch.logsumexp(z, 1), (128 + D / 1024 + 2) * U * A, (2 * D / 16 + 2) * U * A  # _bounds, piece by piece
    L = 2.0 ** -21 + (184 + V / 4096) * U + 3 * U * lse.abs()
    loss = lse - z.gather(1, t[:, None])[:, 0]
    got_loss, got_lse = sbl.sbl_linear_cross_entropy(x, w, t)
    ce._check("lse", got_lse, lse, e + L)
    ce._check("loss", got_loss, loss, 2 * e + L + 2 * U * loss.abs())
    dx, dw = sbl.sbl_linear_cross_entropy_backward(d, x, w, t, got_lse)
    p = torch.exp(z - lse[:, None])
    del z
    hot = torch.zeros_like(p).scatter_(1, t[:, None], 1.0)
    dd = d.double()[:, None]
    ref, bound, sized = 0.0, 0.0, 0.0
    for i in pieces:
        s = slice(i, i + 100000)
        G = (p[:, s] - hot[:, s]) * dd
        eps = (torch.expm1(e + e2 + L) + 2.0 ** -20)[:, None]
        dG = p[:, s] * eps * dd * (1 + ce.BF16) + G.abs() * ((ce.BF16 if T > 128 else ce.BF16 ** 2) + 4 * U)
        wd = w[s].double()
        ref, bound, sized = ref + G @ wd, bound + dG @ wd.abs(), sized + (G.abs() + dG) @ wd.abs()
    bound = bound + ((2 if T > 128 else 4) * V / 16 + 64) * U * sized
    ce._check("dx", dx, ref, bound * (1 + 2 * ce.BF16) + ce.BF16 * ref.abs() + 1e-30)
    for s in (slice(0, 500), slice(V - 500, V)):
        _, (dw_ref, dw_bound) = ce._grad_bounds(x, w[s], p[:, s], hot[:, s], dd, e, e2, L)
        ce._check("dw", dw[s], dw_ref, dw_bound)


def test_feed_forward(sbl):
    """Zero tokens, then a few at the end: h, dh and v past 2^31 elements."""
    T, n, K, F = 540011, 150, 64, 4096
    assert T * F > 2 ** 31
    c = Case(sbl, n, K, F, seed=6)
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    x[-n:] = c.x
    h = sbl.sbl_ffn_gated(x, c.gate, c.up)
    nm._check("h", h[-n:], c.h, c.h_bound(torch.float32))
    assert not h[:1000].any() and not h[-n - 1000:-n].any()
    dh = torch.randn(n, F, generator=torch.Generator().manual_seed(3)) * 0.01
    refs = c.grads(dh)
    big = h.zero_()
    big[-n:] = dh.cuda()
    got = sbl.sbl_ffn_gated_backward(big, x, c.gate, c.up)
    for name, v, (ref, bound) in zip(("dx", "dgate", "dup"), (got[0][-n:], *got[1:]), refs):
        nm._check(name, v, ref, bound)
    assert not got[0][:1000].any()
    assert sbl.sbl_device_status() == 0
