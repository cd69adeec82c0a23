"""A training step of the operators together: norm, gated feed-forward block (its
down projection a SparseBitLinear), residual sum, layer norm, vocabulary loss.

Each stage is checked against the 64-bit formulas on that stage's own inputs and
output gradient as autograd carried them, so that a code of the int8 quantiser
that a rounding upstream moves does not stand between them."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_cross_entropy import _bounds, _grad_bounds, _refs
from test_gpu_ffn_gated import Case
from test_gpu_norm import _backward_refs, _forward_bound

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16 = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module")
def sbl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_linear_layers_b200 as m
    return m


def _close(name, got, ref, bound):
    got = got.detach().double().cpu()
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(((got - ref).abs() / bound.clamp(min=1e-300)).max()))


@pytest.mark.parametrize("B,S,D,F,V,act", [(2, 75, 192, 272, 1003, "silu"), (1, 1, 128, 96, 50, "relu2")])
def test_block_step(sbl, B, S, D, F, V, act):
    torch.manual_seed(B * S + D)
    T, n, m = B * S, 2, 4
    norm1 = sbl.SparseBitNorm(D, device="cuda")
    ffn = sbl.SparseBitFeedForward(D, F, n, m, act=act, device="cuda")
    norm2 = sbl.SparseBitNorm(D, kind="layer", bias=True, device="cuda")
    head = sbl.LinearCrossEntropy(D, V, device="cuda")
    with torch.no_grad():
        norm1.weight.add_(0.1 * torch.randn_like(norm1.weight))
        norm2.bias.add_(0.1 * torch.randn_like(norm2.bias))
        head.weight.mul_(5.0)
    x = torch.randn(B, S, D, device="cuda", requires_grad=True)
    target = torch.randint(0, V, (B, S), device="cuda")
    if T > 1:
        target[0, ::5] = -100
    a = norm1(x)
    f = ffn(a)
    r = x + f
    z = norm2(r)
    for t in (a, f, r, z):
        t.retain_grad()
    loss = head(z, target)
    loss.backward()
    cpu = lambda t: t.detach().cpu().reshape(T, -1)

    # the head, on z rounded to bf16
    zb, wb, tg = cpu(z).bfloat16(), head.weight.detach().cpu().bfloat16(), target.cpu().reshape(T)
    count = int((tg != -100).sum())
    d = torch.full((T,), 1.0 / count)
    zz, lse, per, p, hot, dd = _refs(zb, wb, tg, d)
    e, e2, L = _bounds(zb, wb, zz, lse, per)
    total = float(per.sum()) / count
    assert abs(loss.item() - total) <= float((2 * e + L).sum()) / count + (T + 4) * U * float(per.sum()) / count
    (dz, bz), (dw, bw) = _grad_bounds(zb, wb, p, hot, dd, e, e2, L)
    _close("z.grad", cpu(z.grad), dz, bz + 2 * U * dz.abs())
    _close("head.weight.grad", head.weight.grad, dw, bw + 2 * U * dw.abs())

    # layer norm (its backward runs on the forward's own fp32 statistics: twice the bound)
    w2, b2 = norm2.weight.detach().cpu().double(), norm2.bias.detach().cpu().double()
    y, by = _forward_bound(cpu(r).double(), w2, b2, "layer", norm2.eps, torch.float32)
    _close("z", cpu(z), y, by)
    refs = _backward_refs(cpu(r).double(), cpu(z.grad).double(), w2, "layer", norm2.eps, torch.float32)
    for name, g, (ref, bound) in zip(("dr", "norm2.weight", "norm2.bias"), (cpu(r.grad), norm2.weight.grad, norm2.bias.grad), refs):
        _close(name, g, ref, 2 * bound)

    # the feed-forward block on a rounded to bf16: gate and up
    c = Case.__new__(Case)
    ab = cpu(a).bfloat16()
    c.__dict__.update(T=T, K=D, F=F, act=act)
    mats = []
    for w in (ffn.gate, ffn.up, ffn.down.weight):
        _, sc, _, Wt = oracle.prepare_weights(w.detach().cpu().numpy(), n, m)
        mats.append((torch.from_numpy(sc).double(), torch.from_numpy(Wt).double()))
    (c.sg, c.Wg), (c.su, c.Wu), (sd, Wd) = mats
    c.finish(ab)
    # h is what the down projection quantised: from the forward, by the library's own call
    gate, up = sbl.sbl_prepare_weights_grouped([ffn.gate.detach(), ffn.up.detach()], n, m)
    h = sbl.sbl_ffn_gated(a.detach().reshape(T, D).bfloat16(), gate, up, act=act)
    _close("h", h, c.h, c.h_bound(torch.float32))
    hq, hs = oracle.quant_act(h.bfloat16().float().cpu().numpy())
    hq, hs = torch.from_numpy(hq).double(), torch.from_numpy(hs).double()[:, None]
    ref = (hq @ Wd.T) * sd / hs
    _close("f", cpu(f), ref, 8 * U * ref.abs() + 1e-37)
    df = cpu(f.grad).double()
    gw = df.T @ (hq / hs)
    _close("down.weight.grad", ffn.down.weight.grad, gw, (T + 4) * U * (df.abs().T @ (hq / hs).abs()) + 1e-37)
    # dh: the down projection's gradient, rounded to bf16 on its way
    dh = (df * sd) @ Wd
    dh_bound = (D + 3) * U * ((df.abs() * sd) @ Wd.abs()) * (1 + 2 * BF16) + BF16 * dh.abs()
    got_dh = sbl.sbl_linear_backward(f.grad.detach().reshape(T, D), torch.from_numpy(hq.numpy().astype(np.int8)).cuda(),
                                     torch.from_numpy(hs[:, 0].numpy().astype(np.float32)).cuda(),
                                     sbl.sbl_prepare_weights(ffn.down.weight.detach(), n, m), need_dw=False)[0].bfloat16()
    _close("dh", got_dh, dh, dh_bound)
    (dx, bx), (dg, bg), (du, bu) = c.grads(got_dh.float().cpu())
    _close("gate.grad", ffn.gate.grad, dg, bg)
    _close("up.grad", ffn.up.grad, du, bu)
    _close("a.grad", cpu(a.grad), dx, bx * (1 + 2 * BF16) + BF16 * dx.abs())

    # RMS norm, and the residual
    w1 = norm1.weight.detach().cpu().double()
    refs = _backward_refs(cpu(x).double(), cpu(a.grad).double(), w1, "rms", norm1.eps, torch.float32)
    _close("norm1.weight.grad", norm1.weight.grad, refs[1][0], 2 * refs[1][1])
    dx_all = refs[0][0] + cpu(r.grad).double()
    _close("x.grad", cpu(x.grad), dx_all, 2 * refs[0][1] + 2 * U * dx_all.abs())


def test_frozen_parts_and_reductions(sbl):
    """Only what asks for a gradient gets one; the reductions agree."""
    torch.manual_seed(3)
    norm = sbl.SparseBitNorm(64, bias=True, device="cuda")
    ffn = sbl.SparseBitFeedForward(64, 96, device="cuda", check_finite=False)
    heads = {r: sbl.LinearCrossEntropy(64, 77, reduction=r, device="cuda") for r in ("mean", "sum", "none")}
    for h in heads.values():
        h.weight.data.copy_(heads["mean"].weight.data)
    norm.bias.requires_grad_(False)
    ffn.up.requires_grad_(False)
    heads["mean"].weight.requires_grad_(False)
    x = torch.randn(20, 64, device="cuda").bfloat16()
    t = torch.randint(0, 77, (20,), device="cuda")
    t[3] = -100
    z = ffn(norm(x))
    loss = heads["mean"](z, t)
    loss.backward()
    assert norm.weight.grad is not None and norm.bias.grad is None
    assert ffn.gate.grad is not None and ffn.up.grad is None and ffn.down.weight.grad is not None
    assert heads["mean"].weight.grad is None
    with torch.no_grad():
        per = heads["none"](z, t)
        assert per[3] == 0 and torch.allclose(heads["sum"](z, t), per.sum()) and torch.allclose(loss, per.sum() / 19)
    with pytest.raises(ValueError):
        heads["mean"](z, t[:5])
    with pytest.raises(ValueError):
        sbl.LinearCrossEntropy(64, 77, reduction="max")
    with pytest.raises(ValueError):
        sbl.SparseBitFeedForward(64, 264)   # the down projection's rows are not whole blocks


def test_norm_of_other_types(sbl):
    """fp16 goes through fp32 and back: half a step of fp16 (2^-11) on top of the
    fp32 result, which is far below it."""
    norm = sbl.SparseBitNorm(64, kind="layer", bias=True, device="cuda")
    x = torch.randn(5, 3, 64, device="cuda").half().requires_grad_()
    y = norm(x)
    y.sum().backward()
    assert y.dtype == x.grad.dtype == torch.float16 and y.shape == x.shape
    want = torch.nn.functional.layer_norm(x.detach().double(), (64,), eps=norm.eps)
    assert ((y.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -18).all()


def test_feed_forward_stops_on_nonfinite_input(sbl):
    ffn = sbl.SparseBitFeedForward(64, 96, device="cuda")
    x = torch.randn(30, 64, device="cuda")
    ffn(x)
    x[4, 5] = float("inf")
    with pytest.raises(FloatingPointError):
        ffn(x)


def test_step_in_a_graph(sbl):
    """The whole step's calls, captured once and replayed on new inputs."""
    torch.manual_seed(5)
    T, D, F, V = 96, 128, 160, 300
    g1, w2, b2 = torch.rand(D, device="cuda") + 0.5, torch.rand(D, device="cuda") + 0.5, torch.randn(D, device="cuda")
    W = [torch.randn(F, D, device="cuda") * 0.1 for _ in range(2)]
    gate, up = sbl.sbl_prepare_weights_grouped(W, 3, 4)
    down = sbl.sbl_prepare_weights(torch.randn(D, F, device="cuda") * 0.1, 3, 4)
    vocab = torch.randn(V, D, device="cuda").bfloat16() * 0.1
    dloss = torch.full((T,), 1 / T, device="cuda")

    def step(x, t):
        a, _, r1 = sbl.sbl_norm(x, g1, with_stats=True)
        h = sbl.sbl_ffn_gated(a, gate, up, out_dtype=torch.bfloat16)
        y = sbl.sbl_linear(h, down, out_dtype=torch.bfloat16)
        z, m2, r2 = sbl.sbl_norm(y, w2, b2, kind="layer", with_stats=True)
        loss, lse = sbl.sbl_linear_cross_entropy(z, vocab, t)
        dz, dv = sbl.sbl_linear_cross_entropy_backward(dloss, z, vocab, t, lse)
        dy, dw2, db2 = sbl.sbl_norm_backward(dz, y, w2, m2, r2, kind="layer")
        hq, hs = sbl.sbl_quant_act(h)
        dh, dd = sbl.sbl_linear_backward(dy.float(), hq, hs, down)
        da, dg, du = sbl.sbl_ffn_gated_backward(dh, a, gate, up)
        dx, dw1, _ = sbl.sbl_norm_backward(da.bfloat16(), x, g1, None, r1, need_db=False)
        return loss, dv, dw2, db2, dd, dg, du, dx, dw1

    def inputs(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return torch.randn(T, D, device="cuda", generator=g).bfloat16(), torch.randint(0, V, (T,), device="cuda", generator=g)

    x, t = inputs(1)
    step(x, t)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(x, t)
    x2, t2 = inputs(2)
    x.copy_(x2)
    t.copy_(t2)
    g.replay()
    g.replay()
    for a, b in zip(out, step(x2, t2)):
        assert torch.equal(a, b)
    assert sbl.sbl_device_status() == 0


def test_modules_in_a_graph(sbl):
    """Forward and backward of the modules captured as a training loop captures them:
    warmed up on a side stream, no eager graph of the same parameters alive."""
    torch.manual_seed(9)
    T, D, F, V = 150, 128, 160, 900
    norm = sbl.SparseBitNorm(D, kind="layer", bias=True, device="cuda")
    ffn = sbl.SparseBitFeedForward(D, F, 3, 4, device="cuda", check_finite=False)
    head = sbl.LinearCrossEntropy(D, V, reduction="sum", device="cuda")
    params = [*norm.parameters(), *ffn.parameters(), *head.parameters()]

    def step(x, t):
        for p in params:
            p.grad = None
        loss = head(x + ffn(norm(x)), t)
        loss.backward()
        return loss.detach()

    new = lambda: (torch.randn(T, D, device="cuda"), torch.randint(0, V, (T,), device="cuda"))
    x, t = new()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(x, t)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss = step(x, t)
    grads = [p.grad for p in params]
    x2, t2 = new()
    x.copy_(x2)
    t.copy_(t2)
    g.replay()
    torch.cuda.synchronize()
    got = [loss.clone(), *(v.clone() for v in grads)]
    want = step(x2, t2)
    for a, b in zip(got, [want, *(p.grad for p in params)]):
        assert torch.equal(a, b)


def test_first_use_inside_a_capture():
    """A process whose very first calls of the operators are captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch, sparse_linear_layers_b200 as sbl
T, D, F, V = 600, 128, 160, 3000
w = torch.ones(D, device="cuda")
x = torch.randn(T, D, device="cuda").bfloat16()
one = x[:1].clone()
packed = torch.full((F, D // 4), 0x21, dtype=torch.uint8, device="cuda")
p = sbl.PreparedWeights(packed, torch.full((F,), 0.05, device="cuda"), 2, 4, D)
vocab = torch.randn(V, D, device="cuda").bfloat16()
t = torch.randint(0, V, (T + 1,), device="cuda")[1:]   # a view at an odd element
dh = torch.randn(T, F, device="cuda")
d = torch.full((T,), 1 / T, device="cuda")
def step():
    y, mean, rstd = sbl.sbl_norm(x, w, w, kind="layer", with_stats=True)
    out = [y, *sbl.sbl_norm_backward(y, x, w, mean, rstd, kind="layer"), sbl.sbl_ffn_gated(one, p, p), sbl.sbl_ffn_gated(x, p, p)]
    out += sbl.sbl_ffn_gated_backward(dh, x, p, p)
    loss, lse = sbl.sbl_linear_cross_entropy(x, vocab, t)
    return out + [loss, lse, *sbl.sbl_linear_cross_entropy_backward(d, x, vocab, t, lse)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = step()
g.replay()
for a, b in zip(out, step()):
    assert torch.equal(a, b)
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_two_streams_at_once(sbl):
    """The same calls on two streams, each with its own workspace, while both run."""
    torch.manual_seed(7)
    T, D, F, V = 700, 256, 320, 5000
    gate, up = sbl.sbl_prepare_weights_grouped([torch.randn(F, D, device="cuda") * 0.1 for _ in range(2)], 2, 4)
    vocab = torch.randn(V, D, device="cuda").bfloat16() * 0.1
    w = torch.rand(D, device="cuda") + 0.5
    d = torch.full((T,), 1 / T, device="cuda")
    xs = [torch.randn(T, D, device="cuda").bfloat16() for _ in range(2)]
    ts = [torch.randint(0, V, (T,), device="cuda") for _ in range(2)]

    def step(i, stream=None):
        y, _, rstd = sbl.sbl_norm(xs[i], w, with_stats=True, stream=stream)
        h = sbl.sbl_ffn_gated(y, gate, up, stream=stream)
        out = [h, *sbl.sbl_ffn_gated_backward(h, y, gate, up, stream=stream)]
        loss, lse = sbl.sbl_linear_cross_entropy(y, vocab, ts[i], stream=stream)
        out += [loss, *sbl.sbl_linear_cross_entropy_backward(d, y, vocab, ts[i], lse, stream=stream)]
        return out + list(sbl.sbl_norm_backward(out[-2], xs[i], w, None, rstd, stream=stream))

    ref = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[step(i, streams[i]) for i in range(2)] for _ in range(3)]
    torch.cuda.synchronize()
    for rep in got:
        for i in range(2):
            for a, b in zip(rep[i], ref[i]):
                assert torch.equal(a, b)
