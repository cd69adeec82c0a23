"""sbl_ffn_gated and its backward on the GPU against the formulas in 64 bits on
the oracle's prepared weights and int8 activations.

Bounds.  u = 2^-24.  The integer products are exact; g and the up product take
three fp32 roundings and a reciprocal's: 4 u each.  ex2.approx and rcp.approx
are documented as off by at most 2 and 1 units in the last place (2^-23), the
exponent g log2 e has a relative error of 2 u, which moves exp by 2 u |g|: the
sigmoid has a relative error of at most delta = (5 + 1.2 |g|) 2^-23.  From these
come the errors of act, act', h and v = (dg | du) * scale / s below.

Backward sums: v enters as two fp16 parts, each rounded by half a step (2^-11):
2^-22 |v|, and no finer than 2^-25 where the token's largest v is at least 2^14:
2^-39 of it.  The tensor cores round towards zero (2 u) for each of the 32 MMAs of
a segment of 256 terms, and n / 256 segments are added to nearest: with the
final multiplications (n / 256 + 64 + 4 + 6) u, below the documented
(n / 128 + 80) u.
"""
import numpy as np
import pytest
import torch

import oracle
from sparse_linear_layers_b200 import synthetic

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def sbl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_linear_layers_b200 as m
    return m


class Case:
    """Inputs on the device, and the 64-bit pieces of the reference."""

    def __init__(self, sbl, T, K, F, nm=(2, 4), act="silu", seed=0, scale=0.02, x=None):
        self.T, self.K, self.F, self.act = T, K, F, act
        n, m = nm
        mats = []
        for tag in ("gate", "up"):
            W = synthetic.latent_weights(F, K, seed=seed, tag=f"ffn{tag}") * np.float32(scale / 0.02)
            packed, sc, _, Wt = oracle.prepare_weights(W, n, m)
            w = sbl.PreparedWeights(torch.from_numpy(packed).cuda(), torch.from_numpy(sc).cuda(), n, m, K)
            mats.append((w, torch.from_numpy(sc).double(), torch.from_numpy(Wt).double()))
        (self.gate, self.sg, self.Wg), (self.up, self.su, self.Wu) = mats
        if x is None:
            bits, _ = synthetic.activations(T, K, seed=seed + 1, tag="ffn", outlier_p=0.01)
            x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
        self.x = x.cuda()
        self.finish(x)

    def finish(self, x):
        """The reference's values on x (bf16, on the host) and the matrices."""
        act = self.act
        xq, s = oracle.quant_act(x.float().numpy())
        self.xq, self.s = torch.from_numpy(xq).double(), torch.from_numpy(s).double()[:, None]
        self.g = (self.xq @ self.Wg.T) * self.sg / self.s
        self.u = (self.xq @ self.Wu.T) * self.su / self.s
        g, u = self.g, self.u
        if act == "silu":
            sig = torch.sigmoid(g)
            self.a, self.da = g * sig, sig * (1 + g * (1 - sig))
            delta = (5 + 1.2 * g.abs()) * 2.0 ** -23
            self.a_err = self.da.abs() * 4 * U * g.abs() * 1.001 + self.a.abs() * (delta + 4 * U) + 1e-35
            inner = (1 + g * (1 - sig)).abs()
            self.da_err = sig * (g.abs() * (delta * sig + 6 * U) + 2 * U * (1 + g.abs())) + inner * sig * (delta + 2 * U) \
                + 4 * U * g.abs()
        else:
            r = torch.relu(g)
            self.a, self.da = r * r, 2 * r
            self.a_err, self.da_err = 10 * U * self.a, 10 * U * self.da
        self.u_err = 4 * U * u.abs()
        self.h = self.a * u

    def h_bound(self, dtype):
        e = self.a_err * (self.u.abs() + self.u_err) + self.a.abs() * self.u_err + 2 * U * self.h.abs()
        out = torch.finfo(dtype).eps / 2
        return e * (1 + 2 * out) + out * self.h.abs() + 1e-38

    def grads(self, dh, ternary=False):
        """((dX, bound), (dW_gate, bound), (dW_up, bound))"""
        d = dh.double()
        dg, du = d * self.u * self.da, d * self.a
        dg_err = d.abs() * (self.u_err * (self.da.abs() + self.da_err) + self.u.abs() * self.da_err) + 8 * U * dg.abs()
        du_err = d.abs() * self.a_err + 8 * U * du.abs()
        sg, su = self.sg, self.su
        floor = torch.maximum((dg.abs() * sg).amax(1), (du.abs() * su).amax(1))[:, None] * 2.0 ** -38  # of v * s
        Wga, Wua = self.Wg.abs(), self.Wu.abs()
        n = 2 * self.F
        dx = (dg * sg) @ self.Wg + (du * su) @ self.Wu
        bx = (dg_err * sg) @ Wga + (du_err * su) @ Wua + (n / 128 + 80) * U * ((dg.abs() * sg) @ Wga + (du.abs() * su) @ Wua) \
            + floor * (Wga.sum(0) + Wua.sum(0))
        xh = self.xq / self.s
        out = [(dx, bx + 1e-37)]
        for q, q_err, sc in ((dg, dg_err, sg), (du, du_err, su)):
            ref = q.T @ xh
            bound = q_err.T @ xh.abs() + (self.T / 128 + 80) * U * (q.abs().T @ xh.abs()) \
                + ((floor / self.s).T @ self.xq.abs()) / sc[:, None]
            mul = sc[:, None] if ternary else 1.0
            out.append((ref * mul, bound * mul + 1e-37))
        return out


def _check(name, got, ref, bound):
    got = got.double().cpu()
    assert got.shape == ref.shape
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(((got - ref).abs() / bound.clamp(min=1e-300)).max()))


NMS = [(2, 4), (3, 4), (6, 8), (4, 8)]
# decode sizes (T <= 16; K of every chunk width and a ragged one), tile sizes with ragged rows, tokens
# and k, K that TMA cannot address (K % 64 != 0), odd F (rows that TMA cannot store)
SHAPES = [(1, 16, 1), (1, 64, 8), (1, 256, 130), (2, 144, 37), (5, 896, 200), (9, 128, 33), (16, 2048, 77), (13, 48, 515),
          (17, 64, 128), (33, 80, 97), (100, 128, 129), (256, 256, 256), (257, 192, 131), (300, 272, 260), (520, 896, 300),
          # both gradients' reductions in parts
          (3001, 64, 100)]


@pytest.mark.parametrize("T,K,F", SHAPES)
@pytest.mark.parametrize("act", ["silu", "relu2"])
def test_forward(sbl, T, K, F, act):
    c = Case(sbl, T, K, F, nm=NMS[(T + F) % 4] if K % 8 == 0 else (2, 4), act=act, seed=T + F)
    for dt in (torch.float32, torch.bfloat16):
        h = sbl.sbl_ffn_gated(c.x, c.gate, c.up, act=act, out_dtype=dt)
        assert h.dtype == dt
        _check(f"h {dt}", h, c.h, c.h_bound(dt))
    assert sbl.sbl_device_status() == 0


def test_forward_of_many_decode_passes(sbl):
    """K so long that a pass holds fewer tokens than the call has, and one that
    leaves the decode kernel altogether."""
    for T, K, F in ((16, 20480, 24), (3, 131072, 9)):
        c = Case(sbl, T, K, F, seed=3, scale=0.005)
        h = sbl.sbl_ffn_gated(c.x, c.gate, c.up)
        _check("h", h, c.h, c.h_bound(torch.float32))


@pytest.mark.parametrize("T,K,F", [s for s in SHAPES if s[0] != 16])
@pytest.mark.parametrize("act,ternary", [("silu", False), ("relu2", True)])
def test_backward(sbl, T, K, F, act, ternary):
    c = Case(sbl, T, K, F, nm=NMS[(T + F + 1) % 4], act=act, seed=T + F)
    dh = torch.randn(T, F, generator=torch.Generator().manual_seed(T)) * 0.01
    dh *= 10.0 ** torch.randint(-3, 1, (T, 1), generator=torch.Generator().manual_seed(F))  # tokens of differing weight
    if T > 4:
        dh[3] = 0.0
    refs = c.grads(dh, ternary)
    got = sbl.sbl_ffn_gated_backward(dh.cuda(), c.x, c.gate, c.up, act=act, dw_ternary=ternary)
    for name, g, (r, b) in zip(("dx", "dgate", "dup"), got, refs):
        _check(name, g, r, b)
    for i in range(3):
        need = [j == i for j in range(3)]
        one = sbl.sbl_ffn_gated_backward(dh.cuda(), c.x, c.gate, c.up, act=act, dw_ternary=ternary, need_dx=need[0],
                                         need_dgate=need[1], need_dup=need[2])
        assert [o is not None for o in one] == need
        assert torch.equal(one[i], got[i])
    assert sbl.sbl_device_status() == 0


def test_backward_against_differences(sbl):
    """Central differences, in 64 bits, of sum(dh * h) over the dequantised
    activations and weights: the straight-through gradient is the gradient of
    that smooth function."""
    c = Case(sbl, 6, 64, 20, seed=5, scale=0.2)
    dh = torch.randn(6, 20, generator=torch.Generator().manual_seed(1))
    (_, bx), (_, bg), (_, bu) = c.grads(dh)
    xh, Wg, Wu = c.xq / c.s, c.Wg * c.sg[:, None], c.Wu * c.su[:, None]

    def total(x, a, b):
        g = x @ a.T
        return float((dh.double() * g * torch.sigmoid(g) * (x @ b.T)).sum())

    dx, dg, du = (v.cpu().double() for v in sbl.sbl_ffn_gated_backward(dh.cuda(), c.x, c.gate, c.up))
    step = 1e-5

    def moved(m, i, j, h):
        m = m.clone()
        m[i, j] += h
        return m

    for i, j in ((0, 0), (5, 63), (3, 17)):
        num = (total(moved(xh, i, j, step), Wg, Wu) - total(moved(xh, i, j, -step), Wg, Wu)) / (2 * step)
        assert abs(float(dx[i, j]) - num) <= float(bx[i, j]) + 1e-7
    for i, j in ((0, 1), (19, 63), (7, 30)):
        num = (total(xh, moved(Wg, i, j, step), Wu) - total(xh, moved(Wg, i, j, -step), Wu)) / (2 * step)
        assert abs(float(dg[i, j]) - num) <= float(bg[i, j]) + 1e-7
        num = (total(xh, Wg, moved(Wu, i, j, step)) - total(xh, Wg, moved(Wu, i, j, -step))) / (2 * step)
        assert abs(float(du[i, j]) - num) <= float(bu[i, j]) + 1e-7


def test_matches_the_grouped_linear(sbl):
    """g and u are sbl_linear_grouped's: with a squared ReLU and an up matrix equal
    to the gate's, h is the cube of max(y, 0)."""
    c = Case(sbl, 200, 256, 192, act="relu2", seed=8)
    y = sbl.sbl_linear(c.x, c.gate).double().clamp(min=0)
    h = sbl.sbl_ffn_gated(c.x, c.gate, c.gate, act="relu2").double()
    assert ((h - y ** 3).abs() <= 20 * U * y ** 3).all()


def test_edges(sbl):
    c = Case(sbl, 4, 64, 16, seed=2)
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert sbl.sbl_ffn_gated(e, c.gate, c.up).shape == (0, 16)
    dx, dg, du = sbl.sbl_ffn_gated_backward(torch.empty((0, 16), device="cuda"), e, c.gate, c.up)
    assert dx.shape == (0, 64) and not dg.any() and not du.any()
    # all-zero tokens and all-zero gradients
    z = torch.zeros((40, 64), dtype=torch.bfloat16, device="cuda")
    for T in (3, 40):
        assert not sbl.sbl_ffn_gated(z[:T].contiguous(), c.gate, c.up).any()
    x = torch.randn(40, 64, device="cuda").bfloat16()
    for t in sbl.sbl_ffn_gated_backward(torch.zeros((40, 16), device="cuda"), x, c.gate, c.up):
        assert not t.any()
    # gradients of 1e-30 and of 1e30: the per-token powers of two
    ref = sbl.sbl_ffn_gated_backward(torch.ones((40, 16), device="cuda"), x, c.gate, c.up)
    for p in (-100, 80):
        got = sbl.sbl_ffn_gated_backward(torch.full((40, 16), 2.0 ** p, device="cuda"), x, c.gate, c.up)
        if p > 0:  # every operation scales exactly by a power of two
            for a, b in zip(got, ref):
                assert torch.equal(a, b * 2.0 ** p)
            continue
        # near 2^-111 the smaller v fall below 2^-126, where fp32 spaces values 2^-149
        # apart: each of v's five products adds at most 2^-150 max(1, |u|), and the fp16 parts
        # 2^-22 of a value below 2^-126; 2^-145 (1 + |u|) covers them for each term
        c40 = Case(sbl, 40, 64, 16, seed=2, x=x.cpu())
        E = 2.0 ** -145 * (1 + float(c40.u.abs().max()))
        (rx, bx), (rg, bg), (ru, bu) = c40.grads(torch.full((40, 16), 2.0 ** p))
        _check("dx", got[0], rx, bx + c40.s * 2 * 16 * E)
        _check("dgate", got[1], rg, bg + 40 * 127 * E / c40.sg[:, None])
        _check("dup", got[2], ru, bu + 40 * 127 * E / c40.su[:, None])
    assert sbl.sbl_device_status() == 0
    for T in (2, 40):
        bad = x[:T].clone()
        bad[1, 3] = float("nan")
        sbl.sbl_ffn_gated(bad, c.gate, c.up)
        assert sbl.sbl_device_status() == 3   # SBL_ERR_NONFINITE


def test_other_stream_graph_and_repeats(sbl):
    c = Case(sbl, 300, 192, 200, seed=4)
    c2 = Case(sbl, 300, 192, 200, seed=40)
    dh = torch.randn(300, 200, device="cuda")

    def both(x, d, stream=None):
        return (sbl.sbl_ffn_gated(x, c.gate, c.up, stream=stream),
                *sbl.sbl_ffn_gated_backward(d, x, c.gate, c.up, stream=stream))

    ref = both(c.x, dh)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = both(c.x, dh, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    sx, sd = c.x.clone(), dh.clone()
    one = c.x[:1].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cap = both(sx, sd)
        tok = sbl.sbl_ffn_gated(one, c.gate, c.up, out_dtype=torch.bfloat16)
    sx.copy_(c2.x)
    sd.mul_(-3.0)
    one.copy_(c2.x[5:6])
    g.replay()
    g.replay()
    for a, b in zip(cap, both(c2.x, dh * -3.0)):
        assert torch.equal(a, b)
    assert torch.equal(tok, sbl.sbl_ffn_gated(c2.x[5:6].contiguous(), c.gate, c.up, out_dtype=torch.bfloat16))
