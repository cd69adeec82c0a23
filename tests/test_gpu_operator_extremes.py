"""Norms, the gated feed-forward block, the cross entropy and their modules where
values, sizes or callers lie far apart.

The 64-bit references and bounds are those of the operators' own test files unless
a test states another."""
import pytest
import torch

import test_gpu_cross_entropy as ce
from test_gpu_ffn_gated import Case

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16 = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module")
def sbl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_linear_layers_b200 as m
    return m


_check = ce._check  # an output that holds NaN does not pass


# ---------------------------------------------------------------- the feed-forward block
@pytest.mark.parametrize("T,K,F", [(5, 80, 40), (40, 256, 130), (300, 272, 260), (1500, 896, 150), (3001, 64, 100)])
@pytest.mark.parametrize("act,ternary", [("silu", False), ("relu2", True)])
def test_gradients_of_tokens_far_apart(sbl, T, K, F, act, ternary):
    """Tokens whose gradients differ by up to 2^-75, and hidden units that only the
    small ones reach: the floor of each token is 2^-38 of its own largest v."""
    c = Case(sbl, T, K, F, nm=[(2, 4), (3, 4), (6, 8), (4, 8)][T % 4], act=act, seed=T + F)
    g = torch.Generator().manual_seed(T)
    power = torch.tensor([0, 20, 30, 33, 34, 41, 50, 75])[torch.randint(0, 8, (T, 1), generator=g)]
    power[0], power[-1] = 0, 50
    dh = torch.randn(T, F, generator=g) * 2.0 ** -power.double()
    dh[:, F // 2:] *= power >= 33
    dh[:, F - 7:] *= power >= 50
    dh = dh.float()
    refs = c.grads(dh, ternary)
    got = sbl.sbl_ffn_gated_backward(dh.cuda(), c.x, c.gate, c.up, act=act, dw_ternary=ternary)
    for name, v, (r, b) in zip(("dx", "dgate", "dup"), got, refs):
        # 2^-126 times an activation of at most 127 / s: v itself near fp32's end
        _check(name, v, r, b - 1e-37 + 1e-34)
    for need in ((True, False, False), (False, True, False), (False, False, True)):
        one = sbl.sbl_ffn_gated_backward(dh.cuda(), c.x, c.gate, c.up, act=act, dw_ternary=ternary, need_dx=need[0],
                                         need_dgate=need[1], need_dup=need[2])
        for o, v, n in zip(one, got, need):
            assert (o is not None) == n and (o is None or torch.equal(o, v))
    assert sbl.sbl_device_status() == 0


# ---------------------------------------------------------------- the cross entropy
@pytest.mark.parametrize("T", [9, 128, 200, 300, 1000])
@pytest.mark.parametrize("words", [(0, 32), (128, 192), (0, 128), (290, 300), (480, 513)])
def test_nan_words_reach_every_loss(sbl, T, words):
    """Rows of the vocabulary that hold NaN: every token has such a logit."""
    x, w, t = (v.cuda() for v in ce._inputs(T, 64, 513, seed=7))
    t = torch.where(t == -100, 200, t)
    t[1] = -100
    w[words[0]:words[1]] = float("nan")
    loss, lse = sbl.sbl_linear_cross_entropy(x, w, t)
    assert torch.isnan(lse).all() and loss[1] == 0
    loss[1] = float("nan")
    assert torch.isnan(loss).all()


@pytest.mark.parametrize("T,D", [(9, 4096), (100, 4096), (200, 4096), (300, 4096), (600, 2064)])
def test_gradients_of_likely_words(sbl, T, D):
    """Targets of probability 1 - 1e-3 to 1 - 1e-7, whose G = p - 1 is far below the
    logits.  Logits off by at most e move log p_v by 2 e (1 - p_v), as long as the
    backward's logits are the ones that lse is of; beside that p has a relative error
    of eps = 2^-21 + (100 + |lse| + 12) u: the exponentials of lse and of p, at most 100
    additions near 1, the rounding of lse and of the difference."""
    g = torch.Generator().manual_seed(T + D)
    V = 500
    w = torch.randn(V, D, generator=g) / D ** 0.5
    t = torch.randint(0, V, (T,), generator=g)
    x = 0.5 * torch.randn(T, D, generator=g) + torch.linspace(13, 22, T)[:, None] * w[t]
    x, w = x.bfloat16(), w.bfloat16()
    d = torch.ones(T)
    z, lse, loss, p, hot, dd = ce._refs(x, w, t, d)
    assert loss.min() < 1e-6 and loss.max() > 1e-4
    e, _, _ = ce._bounds(x, w, z, lse, loss)
    eps = (2.0 ** -21 + (112 + lse.abs()) * U)[:, None]
    rest = 1 - p
    rest[hot > 0] = -torch.expm1(-loss)
    G = torch.where(hot > 0, -rest, p)
    dG = p * (torch.expm1(2 * e[:, None] * rest) + eps) * (1 + BF16) + G.abs() * ((BF16 if T > 128 else BF16 ** 2) + 4 * U)
    Ga, wa, xa = G.abs() + dG, w.double().abs(), x.double().abs()
    n = 2 if T > 128 else 4
    dx, dw = G @ w.double(), G.T @ x.double()
    bx = dG @ wa + (n * V / 16 + 64) * U * (Ga @ wa)
    bw = dG.T @ xa + (n * T / 16 + 8) * U * (Ga.T @ xa)
    _, got_lse = sbl.sbl_linear_cross_entropy(x.cuda(), w.cuda(), t.cuda())
    got = sbl.sbl_linear_cross_entropy_backward(d.cuda(), x.cuda(), w.cuda(), t.cuda(), got_lse)
    _check("dx", got[0], dx, bx * (1 + 2 * BF16) + BF16 * dx.abs())
    _check("dw", got[1], dw, bw * (1 + 2 * BF16) + BF16 * dw.abs())
