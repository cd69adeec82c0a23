"""Norms, the gated feed-forward block, the cross entropy and their modules where
values, sizes or callers lie far apart.

The 64-bit references and bounds are those of the operators' own test files unless
a test states another."""
import ctypes
import os
import subprocess

import pytest
import torch

import test_gpu_cross_entropy as ce
import test_gpu_norm as nm
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
@pytest.mark.parametrize("T,K,F", [(5, 80, 40), (40, 256, 130), (300, 272, 260), (1500, 896, 150), (3001, 64, 100),
                                   # more small tokens than the kernel's list of them holds at once
                                   (7003, 144, 40)])
@pytest.mark.parametrize("act,ternary", [("silu", False), ("relu2", True)])
@pytest.mark.parametrize("powers", [(0, 20, 30, 33, 34, 41, 50, 75), (0, 12, 16, 19, 20, 21, 22), (0, 22, 24, 26, 28, 30, 31)])
def test_gradients_of_tokens_far_apart(sbl, T, K, F, act, ternary, powers):
    """Tokens whose gradients differ by up to 2^-75, and hidden units that only the
    small ones reach: the floor of each token is 2^-38 of its own largest v."""
    c = Case(sbl, T, K, F, nm=[(2, 4), (3, 4), (6, 8), (4, 8)][T % 4], act=act, seed=T + F)
    g = torch.Generator().manual_seed(T)
    power = torch.tensor(powers)[torch.randint(0, len(powers), (T, 1), generator=g)]
    power[0], power[-1] = powers[0], powers[-2]
    dh = torch.randn(T, F, generator=g) * 2.0 ** -power.double()
    dh[:, F // 2:] *= power >= powers[len(powers) // 2]
    dh[:, F - 7:] *= power >= powers[-2]
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


@pytest.mark.parametrize("d", [0, 15, 20, 22, 23, 26, 29, 30, 31, 32, 40])
def test_gradients_of_one_small_token_beside_others(sbl, d):
    """A column of dW whose terms are one token's, 2^-d of the largest token (which has
    x = 0 there), and smaller ones of tokens in between: each sum within 90 u of its
    terms.  One weight a row, at column 0 with x = 127, makes s = 1, g = u = 127 scale
    and dup = sum dh g^2 x (squared ReLU)."""
    T, K, F = 16, 16, 128
    packed = torch.zeros(F, K // 4, dtype=torch.uint8)
    packed[:, 0] = 1
    w = sbl.PreparedWeights(packed.cuda(), torch.full((F,), 1 / 128, device="cuda"), 2, 4, K)
    g = torch.Generator().manual_seed(d)
    x, dh = torch.zeros(T, K), torch.zeros(T, F)
    x[:, 0] = 127
    dh[0] = 1.9
    x[1, 1:] = torch.randint(1, 3, (K - 1,), generator=g).float()
    dh[1] = (1 + torch.rand(F, generator=g)) * 2.0 ** -d
    x[2:, 1:] = torch.randint(-9, 10, (T - 2, K - 1), generator=g).float()
    dh[2:] = torch.randn(T - 2, F, generator=g) * 2.0 ** -(d + 8)
    dh[2:, 0] = 2.0 ** -max(d - 9, 0)   # what scales them: their largest
    terms = dh.double() * (127 / 128) ** 2
    _, _, dup = sbl.sbl_ffn_gated_backward(dh.cuda(), x.bfloat16().cuda(), w, w, act="relu2")
    floor = 2.0 ** -38 * 2 * terms.abs().amax(1, keepdim=True)    # the gate's v is twice the up's
    bound = 90 * U * (terms.abs().T @ x.double().abs()) + (floor * x.double().abs()).sum(0)
    _check("dup", dup, terms.T @ x.double(), bound)


@pytest.mark.parametrize("T", [1, 12, 40])
def test_silu_of_enormous_activations(sbl, T):
    """g * u beyond fp32's range where act(g) * u is not.  x = 127 gives x_q = 127 and s = 1
    exactly, so g = 2032 scale_gate and u = 2032 scale_up of the chosen signs, acc * scale
    no larger than u (with s = 127 the layer's own acc * scale / s would pass fp32's range
    for u above 3.4e38 / 127).  The sigmoid has the relative error delta of the ordinary
    cases; below 2^-126, where it counts as 0, an absolute one of 2^-126."""
    K, A, gs = 16, 16 * 127, torch.tensor([-100.0, -80.0, -60.0, -100.0, -86.0, 3.0, 0.5, -88.0])
    us = torch.tensor([4e36, 8e36, 3e37, -4e36, 1e38, 1e37, -2e37, 1e38])
    F = gs.numel()
    rows = lambda v: torch.where(v[:, None] > 0, 0x55, 0xAA).to(torch.uint8).expand(F, K // 4).contiguous()  # all +1 / all -1
    make = lambda v: sbl.PreparedWeights(rows(v).cuda(), (v.abs() / A).cuda(), 2, 4, K)
    gate, up = make(gs), make(us)
    x = torch.full((T, K), 127.0, dtype=torch.bfloat16, device="cuda")
    g, u = gs.sign().double() * (gs.abs() / A).double() * A, us.sign().double() * (us.abs() / A).double() * A
    sig = torch.sigmoid(g)
    delta = (5 + 1.2 * g.abs()) * 2.0 ** -23 + 4 * U * (1 + g.abs())
    h = (g * sig * u).expand(T, F)
    bound = (h.abs() * (delta + 12 * U) + g.abs() * u.abs() * 2.0 ** -126).expand(T, F)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.finfo(dt).eps / 2
        _check("h", sbl.sbl_ffn_gated(x, gate, up, out_dtype=dt), h, bound * (1 + 2 * out) + out * h.abs())
    # dh = 1000: dh * u passes fp32's range before act'(g) brings it back
    keep = gs < 0
    dh = torch.full((T, F), 1000.0) * keep
    du, dg = dh.double() * g * sig, dh.double() * u * sig * (1 + g * (1 - sig))
    du_err = dh.double() * g.abs() * (sig * (delta + 12 * U) + 2.0 ** -126)
    slope = 1 + g.abs()
    dg_err = dh.double() * u.abs() * slope * (sig * (2 * delta + 20 * U) + 2.0 ** -125)
    dx, dwg, dwu = sbl.sbl_ffn_gated_backward(dh.cuda(), x, gate, up)
    # dW: x_hat = 127; the reductions' (T / 128 + 80) u, and 2^-38 of the token's largest v
    sg, su = (gs.abs() / A).double(), (us.abs() / A).double()
    floor = torch.maximum((dg.abs() * sg).amax(1), (du.abs() * su).amax(1))[:, None] * 2.0 ** -38 + 1e-37
    for name, v, q, e, sc in (("dgate", dwg, dg, dg_err, sg), ("dup", dwu, du, du_err, su)):
        ref = 127 * q.sum(0)[:, None].expand(F, K)
        b = 127 * (e.sum(0) + (T / 128 + 90) * U * q.abs().sum(0) + (floor.sum(0) * 1.01 / sc))[:, None].expand(F, K)
        _check(name, v, ref, b)
    ref = ((dg * g.sign() * sg).sum(1) + (du * u.sign() * su).sum(1))[:, None].expand(T, K)
    terms = (dg.abs() * sg).sum(1) + (du.abs() * su).sum(1)
    b = (dg_err * sg).sum(1) + (du_err * su).sum(1) + (2 * F / 128 + 90) * U * terms + 2 * F * floor[:, 0]
    _check("dx", dx, ref, b[:, None].expand(T, K))


CALLERS = r"""
#include <pthread.h>
#include <stdint.h>
#include "sbl.h"
struct call { const void* f; void* x; void* w; void* s; void* h; void* ws; int64_t K; void* stream; int repeats, linear; long refused; };
static void* loop(void* p) {
    struct call* c = p;
    for (int i = 0; i < c->repeats; ++i) {
        sbl_status r = c->linear
            ? ((__typeof__(&sbl_linear_path))c->f)(c->x, c->linear, c->K, c->w, c->s, 8, 2, 4, c->h, SBL_F32, 0, c->ws, 1 << 21, SBL_PATH_DECODE, c->stream)
            : ((__typeof__(&sbl_ffn_gated))c->f)(c->x, 16, c->K, c->w, c->s, c->w, c->s, 8, 2, 4, SBL_ACT_SILU, c->h, SBL_F32, 0, 0, c->stream);
        if (r != SBL_OK) ++c->refused;
    }
    return 0;
}
long two_at_once(struct call* c) {
    pthread_t t[2];
    for (int i = 0; i < 2; ++i) if (pthread_create(&t[i], 0, loop, c + i)) return -1;
    for (int i = 0; i < 2; ++i) pthread_join(t[i], 0);
    return c[0].refused + c[1].refused;
}
"""


@pytest.mark.parametrize("linear", [0, 8, 16])
def test_decode_calls_of_two_threads(sbl, linear, tmp_path):
    """Calls for a few tokens, of different lengths K, from two host threads at once (in C:
    Python's lock would keep them apart): what one asks of the kernel's shared memory
    does not undercut the other's launch.  sbl_ffn_gated, and sbl_linear's decode on the
    CUDA cores (8 tokens, K % 64 != 0) and the warp-level MMA (16)."""
    from sparse_linear_layers_b200._lib import lib
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src, so = tmp_path / "callers.c", tmp_path / "callers.so"
    src.write_text(CALLERS)
    subprocess.run(["gcc", "-O2", "-std=gnu99", "-shared", "-fPIC", "-pthread", f"-I{root}/include", str(src), "-o", str(so)],
                   check=True)
    fields = [(n, ctypes.c_void_p) for n in ("f", "x", "w", "s", "h", "ws")] + [("K", ctypes.c_int64), ("stream", ctypes.c_void_p)] \
        + [("repeats", ctypes.c_int), ("linear", ctypes.c_int), ("refused", ctypes.c_long)]
    Call = type("Call", (ctypes.Structure,), {"_fields_": fields})
    f = ctypes.cast(lib.sbl_linear_path if linear else lib.sbl_ffn_gated, ctypes.c_void_p)
    held, calls, streams = [], (Call * 2)(), [torch.cuda.Stream(), torch.cuda.Stream()]
    for c, K, st in zip(calls, (8208, 16400) if linear == 8 else (4096, 8192), streams):
        x = torch.randn(16, K, device="cuda").bfloat16()
        w = sbl.PreparedWeights(torch.full((8, K // 4), 0x21, dtype=torch.uint8, device="cuda"),
                                torch.full((8,), 0.01, device="cuda"), 2, 4, K)
        ws, h = torch.empty(1 << 21, dtype=torch.uint8, device="cuda"), torch.zeros(linear or 16, 8, device="cuda")
        want = sbl.sbl_linear(x[:linear].contiguous(), w, path="decode") if linear else sbl.sbl_ffn_gated(x, w, w)
        c.f, c.x, c.w, c.s, c.h, c.ws = f, x.data_ptr(), w.packed.data_ptr(), w.row_scale.data_ptr(), h.data_ptr(), ws.data_ptr()
        c.K, c.stream, c.repeats, c.linear = K, st.cuda_stream, 5000, linear
        held.append((x, w, ws, h, want))
    torch.cuda.synchronize()
    run = ctypes.CDLL(str(so)).two_at_once
    run.restype = ctypes.c_long
    assert run(calls) == 0
    torch.cuda.synchronize()
    for *_, h, want in held:
        assert torch.equal(h, want)


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


def test_module_names_its_bad_targets(sbl):
    """A target outside the vocabulary: the module's own error before anything runs;
    without its check, or in a graph, the loss is NaN and no other module's forward
    claims the error as its own."""
    x = torch.randn(20, 64, device="cuda")
    t = torch.randint(0, 77, (20,), device="cuda")
    t[3] = -100
    for wrong in (77, -1, 1 << 40):
        head = sbl.LinearCrossEntropy(64, 77, device="cuda")
        head(x, t)
        bad = t.clone()
        bad[5] = wrong
        with pytest.raises(IndexError, match="LinearCrossEntropy"):
            head(x, bad)
        assert sbl.sbl_device_status() == 0
        free = sbl.LinearCrossEntropy(64, 77, device="cuda", check_targets=False)
        assert torch.isnan(free(x, bad))
        with pytest.raises(sbl.SblError, match="sbl_linear_cross_entropy"):
            sbl.SparseBitFeedForward(64, 96, device="cuda")(x)
        assert sbl.sbl_device_status() == 0
    # a forward in a graph is not checked; the graph's loss is the module's
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad():
        with torch.cuda.graph(graph):
            loss = head(x, t)
    graph.replay()
    assert torch.equal(loss, head(x, t))


# ---------------------------------------------------------------- norms
@pytest.mark.parametrize("T,K", [(33, 896), (1900, 896), (7, 8192), (500, 4864), (9601, 272), (400, 5136), (35, 16400)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward_far_from_zero_mean(sbl, T, K, dtype):
    """Rows whose mean is 1000 times their spread, by the formulas of the very mean and
    rstd given: x - mean is rounded once and so is its product with rstd, X = 2 u
    |xhat|, in every kernel (few rows, many rows, long rows)."""
    g = torch.Generator().manual_seed(K)
    x = (torch.randn(T, K, generator=g) + 1000.0 * torch.sign(torch.randn(T, 1, generator=g))).to(dtype)
    dy, w = torch.randn(T, K, generator=g).to(dtype), 1 + 0.2 * torch.randn(K, generator=g)
    m64, r64 = nm._stats(x.double(), "layer", 1e-5)
    mean, rstd = m64[:, 0].float(), r64[:, 0].float()
    m, r, xd, dyd, wd = mean.double()[:, None], rstd.double()[:, None], x.double(), dy.double(), w.double()
    xh, D = (xd - m) * r, 40 + K / 4096
    X, q = 2.01 * U * xh.abs(), dyd * wd
    m1, m0 = (q * xh).mean(1, keepdim=True), q.mean(1, keepdim=True)
    m1_err = (q.abs() * X).mean(1, keepdim=True) + (D + 3) * U * (q * xh).abs().mean(1, keepdim=True)
    m0_err = (D + 3) * U * q.abs().mean(1, keepdim=True)
    out = torch.finfo(dtype).eps / 2
    dx = r * (q - m0 - xh * m1)
    size = q.abs() + m0.abs() + (xh * m1).abs()
    bx = r * (m0_err + xh.abs() * m1_err + X * (m1.abs() + m1_err) + 6 * U * size) * (1 + 2 * out) + out * dx.abs()
    got = sbl.sbl_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean.cuda(), rstd.cuda(), kind="layer")
    _check("dx", got[0], dx, bx)
    _check("dw", got[1], (dyd * xh).sum(0), (dyd.abs() * X).sum(0) + (T + 99) * U * (dyd * xh).abs().sum(0))
    _check("db", got[2], dyd.sum(0), (T + 99) * U * dyd.abs().sum(0))


@pytest.mark.parametrize("T,K", nm.SHAPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_outputs_are_numbers(sbl, T, K, kind, dtype):
    """Finite rows, a constant one and one of zeros among them, give finite outputs."""
    x, dy, w, b = (v.cuda() for v in nm._inputs(T, K, dtype, seed=T + 2 * K, offset=100.0))
    x[T // 2] = 3.0
    if T > 2:
        x[T - 1] = 0.0
    y, mean, rstd = sbl.sbl_norm(x, w, b, kind=kind, eps=1e-5, with_stats=True)
    outs = [y, rstd, *sbl.sbl_norm_backward(dy, x, w, mean, rstd, kind=kind)] + ([mean] if kind == "layer" else [])
    assert all(torch.isfinite(v).all() for v in outs)
    if kind == "layer":  # with no spread only the bias is left
        assert torch.equal(y[T // 2], b.to(dtype))


def test_far_rows_are_numbers(sbl):
    """Past 2^31 elements: the last rows of a norm and of the block, as numbers."""
    if torch.cuda.get_device_properties(0).total_memory < 120 << 30:
        pytest.skip("needs 60 GB on the device")
    T, K, n = 270001, 8192, 40
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    x[-n:] = torch.randn(n, K, device="cuda").bfloat16()
    w = torch.rand(K, device="cuda") + 0.5
    y, mean, rstd = sbl.sbl_norm(x, w, w, kind="layer", with_stats=True)
    assert torch.isfinite(y[-2 * n:]).all() and torch.isfinite(mean).all() and torch.isfinite(rstd).all()
    dx, dw, db = sbl.sbl_norm_backward(y, x, w, mean, rstd, kind="layer")
    assert torch.isfinite(dx[-2 * n:]).all() and torch.isfinite(dw).all() and torch.isfinite(db).all()
    del x, y, dx
    T, K, F = 540011, 64, 4096
    c = Case(sbl, 150, K, F, seed=6)
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    x[-150:] = c.x
    h = sbl.sbl_ffn_gated(x, c.gate, c.up)
    assert torch.isfinite(h[-300:]).all() and h[-150:].any()
    got = sbl.sbl_ffn_gated_backward(h, x, c.gate, c.up)
    assert torch.isfinite(got[0][-300:]).all() and all(torch.isfinite(v).all() for v in got[1:])
    del x, h, got
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- empty batches
def test_one_gradient_of_an_empty_batch(sbl):
    """No tokens, and only the gradient of the input (or of one weight) wanted."""
    w = torch.ones(64, device="cuda")
    e, s = torch.empty((0, 64), device="cuda"), torch.empty((0,), device="cuda")
    eb = e.bfloat16()
    p = sbl.PreparedWeights(torch.zeros((16, 16), dtype=torch.uint8, device="cuda"), torch.ones(16, device="cuda"), 2, 4, 64)
    W = torch.ones((50, 64), dtype=torch.bfloat16, device="cuda")
    t = torch.empty((0,), dtype=torch.int64, device="cuda")
    calls = [(3, lambda n: sbl.sbl_norm_backward(e, e, w, s, s, kind="layer", need_dx=n[0], need_dw=n[1], need_db=n[2])),
             (3, lambda n: sbl.sbl_ffn_gated_backward(torch.empty((0, 16), device="cuda"), eb, p, p, need_dx=n[0],
                                                      need_dgate=n[1], need_dup=n[2])),
             (2, lambda n: sbl.sbl_linear_cross_entropy_backward(s, eb, W, t, s, need_dx=n[0], need_dw=n[1])),
             (2, lambda n: sbl.sbl_linear_backward(torch.empty((0, 16), device="cuda"), torch.empty((0, 64), dtype=torch.int8, device="cuda"),
                                                   s, p, need_dx=n[0], need_dw=n[1]))]
    for outs, call in calls:
        for i in range(outs):
            got = call([j == i for j in range(outs)])
            assert [v is not None for v in got] == [j == i for j in range(outs)]
            assert not got[i].any() and (i > 0 or got[0].shape == (0, 64))


def test_modules_with_frozen_weights_on_an_empty_batch(sbl):
    x = torch.empty((0, 64), device="cuda", requires_grad=True)
    norm = sbl.SparseBitNorm(64, bias=True, device="cuda").requires_grad_(False)
    ffn = sbl.SparseBitFeedForward(64, 96, device="cuda").requires_grad_(False)
    head = sbl.LinearCrossEntropy(64, 50, reduction="sum", device="cuda").requires_grad_(False)
    loss = head(ffn(norm(x)), torch.empty((0,), dtype=torch.int64, device="cuda"))
    loss.backward()
    assert loss == 0 and x.grad.shape == (0, 64)
