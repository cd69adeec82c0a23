"""The measured cases of three operators around the Sparse-BitLinear layer.

- ``norm``: layer norm and RMS norm of rows, forward and backward (with the
  sums over the rows that give the weight's and the bias' gradients);
- ``ffn``: the gated feed-forward block on prepared N:M ternary weights,
  h = act(gate(x)) * up(x), for serving and with its straight-through backward;
- ``xent``: softmax cross entropy of a vocabulary projection, per token, without
  keeping the logits, with the gradients of its two inputs.

``run`` computes them in elementary torch operations, or, with ``own``, through
the package's entry points.
"""
import math

import torch

own = False

_DEV = "cuda"
_IGNORE = -100


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token through the RMS norm in front of a layer: the latency of a decode step
        dict(name="norm_token", op="norm", kind="rms", dtype="bf16", T=1, K=2048, bias=False, train=False),
        # a 4096-token prompt through a layer norm with weight and bias
        dict(name="norm_prompt", op="norm", kind="layer", dtype="bf16", T=4096, K=2048, bias=True, train=False),
        # a training step's norm of the widest activations: forward, backward, sums over 16384 rows
        dict(name="norm_train", op="norm", kind="layer", dtype="bf16", T=16384, K=4864, bias=True, train=True),
        # a short fp32 training batch with an odd number of rows
        dict(name="norm_train_fp32", op="norm", kind="rms", dtype="fp32", T=1021, K=896, bias=False, train=True),
        # one generated token through the gate and up projections of the hidden-2048 stack
        dict(name="ffn_token", op="ffn", nm="2:4", act="silu", out="bf16", T=1, K=2048, F=7168, train=False),
        # thirteen sequences decoding together, 0.5B-shaped layer
        dict(name="ffn_tokens", op="ffn", nm="3:4", act="silu", out="bf16", T=13, K=896, F=4864, train=False),
        # the prompt phase of the 0.5B-shaped layer
        dict(name="ffn_prompt", op="ffn", nm="3:4", act="silu", out="bf16", T=2048, K=896, F=4864, train=False),
        # a training step of the hidden-2048 stack: forward, and the gradients of x and both matrices
        dict(name="ffn_train", op="ffn", nm="2:4", act="silu", out="fp32", T=4096, K=2048, F=7168, train=True),
        # a ragged training batch, an odd hidden width, the squared ReLU
        dict(name="ffn_train_ragged", op="ffn", nm="6:8", act="relu2", out="fp32", T=1001, K=896, F=2731, train=True),
        # scoring a paragraph: losses only, an odd vocabulary
        dict(name="xent_score", op="xent", T=333, D=896, V=50001, train=False),
        # a training step's loss and gradients
        dict(name="xent_train", op="xent", T=4096, D=2048, V=32000, train=True),
        # the largest: a long batch on a large vocabulary, whose logits would take 4 GB
        dict(name="xent_train_large", op="xent", T=8192, D=896, V=128000, train=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "ffn", "xent"])
    train = rng.random() < 0.6
    if op == "norm":
        K = 16 * _log_int(rng, 1, 512)
        T = _log_int(rng, 1, max(1, min(65536, 16384 * 4864 // (2 * K))))
        return dict(op=op, kind=rng.choice(["layer", "rms"]), dtype=rng.choice(["bf16", "fp32"]), T=T, K=K,
                    bias=rng.random() < 0.5, train=train)
    if op == "ffn":
        return dict(op=op, nm=rng.choice(["2:4", "3:4", "6:8", "4:8"]), act=rng.choice(["silu", "relu2"]),
                    out=rng.choice(["bf16", "fp32"]), T=_log_int(rng, 1, 4096), K=16 * _log_int(rng, 2, 128),
                    F=_log_int(rng, 33, 7168), train=train)
    D = 16 * _log_int(rng, 2, 128)
    V = _log_int(rng, 500, 128000)
    T = _log_int(rng, 1, max(1, min(8192, 8192 * 896 * 128000 // (V * D))))
    return dict(op=op, T=T, D=D, V=V, train=train)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=_DEV, dtype=torch.float32)


def _prepared(g, F, K, n, m):
    """Packed codes and row scales of N(0, 0.02) latent weights: the n largest of
    every m kept, the row's mean over them, 2 bits a weight (01 = +1, 10 = -1)."""
    w = _randn(g, F, K) * 0.02
    groups = w.abs().view(F, K // m, m)
    kept = torch.zeros_like(groups).scatter_(2, groups.topk(n, dim=2).indices, 1.0).view(F, K) > 0
    scale = ((w.abs() * kept).sum(1) / kept.sum(1)).clamp(min=1e-5)
    big = kept & (w.abs() > 0.5 * scale[:, None])
    code = torch.where(big, torch.where(w > 0, 1, 2), 0).to(torch.uint8).view(F, K // 4, 4)
    packed = code[..., 0] | (code[..., 1] << 2) | (code[..., 2] << 4) | (code[..., 3] << 6)
    return packed.contiguous(), scale.contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "norm":
        T, K = case["T"], case["K"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # a residual stream: rows of differing size around a small common offset
        s["x"] = ((_randn(g, T, K) + 0.25) * (0.5 + 2 * torch.rand(T, 1, generator=g, device=_DEV))).to(dt)
        s["weight"] = 1 + 0.1 * _randn(g, K)
        s["bias_t"] = 0.1 * _randn(g, K) if case["bias"] else None
        s["eps"] = 1e-5
        if case["train"]:
            s["dy"] = _randn(g, T, K).to(dt)
    elif case["op"] == "ffn":
        T, K, F = case["T"], case["K"], case["F"]
        n, m = (int(v) for v in case["nm"].split(":"))
        s["gate"] = _prepared(g, F, K, n, m)
        s["up"] = _prepared(g, F, K, n, m)
        x = _randn(g, T, K)
        x = torch.where(torch.rand(T, K, generator=g, device=_DEV) < 0.01, 20 * x, x)  # 1% outliers
        s["x"] = x.to(torch.bfloat16)
        if case["train"]:
            s["dh"] = _randn(g, T, F) * 0.01
    else:
        T, D, V = case["T"], case["D"], case["V"]
        w = _randn(g, V, D) * (1.5 / math.sqrt(D))
        target = torch.randint(0, V, (T,), generator=g, device=_DEV)
        # hidden states that know half of their targets
        sure = 6.0 * (torch.rand(T, 1, generator=g, device=_DEV) < 0.5)
        s["x"] = (_randn(g, T, D) + sure * w[target]).to(torch.bfloat16)
        s["w"] = w.to(torch.bfloat16)
        # a tenth of the positions count for nothing (padding)
        s["target"] = torch.where(torch.rand(T, generator=g, device=_DEV) < 0.1, _IGNORE, target)
        if case["train"]:
            counted = (s["target"] != _IGNORE).sum().clamp(min=1)
            s["dloss"] = (1.0 / counted).expand(T).contiguous().float()  # of the mean over counted positions
    return s


# ---------------------------------------------------------------- plain forms
def _norm_plain(s):
    x, w = s["x"].float(), s["weight"]
    mean = x.mean(1, keepdim=True) if s["kind"] == "layer" else 0.0
    c = x - mean
    rstd = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + s["eps"])
    xhat = c * rstd
    y = xhat * w
    if s["bias"]:
        y = y + s["bias_t"]
    out = {"y": y.to(s["x"].dtype)}
    if s["train"]:
        dy = s["dy"].float()
        dxhat = dy * w
        d = dxhat - xhat * (dxhat * xhat).mean(1, keepdim=True)
        if s["kind"] == "layer":
            d = d - dxhat.mean(1, keepdim=True)
        out["dx"] = (d * rstd).to(s["x"].dtype)
        out["dweight"] = (dy * xhat).sum(0)
        if s["bias"]:
            out["dbias"] = dy.sum(0)
    return out


def _codes(packed):
    c = packed.to(torch.int32)
    c = torch.stack([(c >> (2 * j)) & 3 for j in range(4)], -1).flatten(1)
    return ((c == 1).float() - (c == 2).float())


def _ffn_plain(s):
    x = s["x"].float()
    top = x.abs().amax(1, keepdim=True).clamp(min=1e-5)
    st = torch.full_like(top, 127.0) / top  # one IEEE division (a scalar over a tensor would be a reciprocal and a product)
    xq = torch.round(x * st).clamp(-128, 127)
    wg, wu = _codes(s["gate"][0]), _codes(s["up"][0])
    sg, su = s["gate"][1], s["up"][1]
    g = (xq @ wg.T) * sg / st
    u = (xq @ wu.T) * su / st
    if s["act"] == "silu":
        sig = 1 / (1 + torch.exp(-g))
        a, da = g * sig, sig * (1 + g * (1 - sig))
    else:
        r = g.clamp(min=0)
        a, da = r * r, 2 * r
    out = {"h": (a * u).to(torch.bfloat16 if s["out"] == "bf16" else torch.float32)}
    if s["train"]:
        dg, du = s["dh"] * u * da, s["dh"] * a
        out["dx"] = (dg * sg) @ wg + (du * su) @ wu
        xhat = xq / st
        out["dgate"] = dg.T @ xhat
        out["dup"] = du.T @ xhat
    return out


def _xent_plain(s):
    x, w, t = s["x"].float(), s["w"].float(), s["target"]
    logits = x @ w.T
    counted = t != _IGNORE
    col = torch.where(counted, t, 0)[:, None]
    top = logits.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(logits - top).sum(1, keepdim=True))
    loss = torch.where(counted, (lse - logits.gather(1, col))[:, 0], 0.0)
    out = {"loss": loss, "lse": lse[:, 0]}
    if s["train"]:
        grad = torch.exp(logits - lse)
        grad.scatter_add_(1, col, torch.full_like(lse, -1.0))
        grad *= torch.where(counted, s["dloss"], 0.0)[:, None]
        out["dx"] = (grad @ w).to(torch.bfloat16)
        out["dw"] = (grad.T @ x).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------- the package's entry points
def _norm_own(s):
    import sparse_linear_layers_b200 as sbl
    if not s["train"]:
        return {"y": sbl.sbl_norm(s["x"], s["weight"], s["bias_t"], kind=s["kind"], eps=s["eps"])}
    y, mean, rstd = sbl.sbl_norm(s["x"], s["weight"], s["bias_t"], kind=s["kind"], eps=s["eps"], with_stats=True)
    dx, dw, db = sbl.sbl_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd, kind=s["kind"], need_db=s["bias"])
    out = {"y": y, "dx": dx, "dweight": dw}
    if s["bias"]:
        out["dbias"] = db
    return out


def _ffn_own(s):
    import sparse_linear_layers_b200 as sbl
    n, m = (int(v) for v in s["nm"].split(":"))
    gate = sbl.PreparedWeights(*s["gate"], n, m, s["K"])
    up = sbl.PreparedWeights(*s["up"], n, m, s["K"])
    dt = torch.bfloat16 if s["out"] == "bf16" else torch.float32
    out = {"h": sbl.sbl_ffn_gated(s["x"], gate, up, act=s["act"], out_dtype=dt)}
    if s["train"]:
        out["dx"], out["dgate"], out["dup"] = sbl.sbl_ffn_gated_backward(s["dh"], s["x"], gate, up, act=s["act"])
    return out


def _xent_own(s):
    import sparse_linear_layers_b200 as sbl
    loss, lse = sbl.sbl_linear_cross_entropy(s["x"], s["w"], s["target"], ignore_index=_IGNORE)
    out = {"loss": loss, "lse": lse}
    if s["train"]:
        out["dx"], out["dw"] = sbl.sbl_linear_cross_entropy_backward(s["dloss"], s["x"], s["w"], s["target"], lse,
                                                                     ignore_index=_IGNORE)
    return out


def run(state):
    if own:
        return {"norm": _norm_own, "ffn": _ffn_own, "xent": _xent_own}[state["op"]](state)
    return {"norm": _norm_plain, "ffn": _ffn_plain, "xent": _xent_plain}[state["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "norm":
        T, K = case["T"], case["K"]
        e = 2 if case["dtype"] == "bf16" else 4
        params = 2 if case["bias"] else 1
        if case["train"]:  # x, dy in; y, dx out; the parameters and their gradients
            return {"bytes": 4 * T * K * e + 8 * params * K, "flops": 20 * T * K}
        return {"bytes": 2 * T * K * e + 4 * params * K, "flops": 8 * T * K}
    if case["op"] == "ffn":
        T, K, F = case["T"], case["K"], case["F"]
        b = 2 * T * K + 2 * (F * K // 4 + 4 * F) + T * F * (2 if case["out"] == "bf16" else 4)
        f = 4 * T * F * K
        if case["train"]:  # dh in; the gradients of x and of both matrices out
            b += 4 * T * F + 4 * T * K + 8 * F * K
            f *= 3
        return {"bytes": b, "flops": f}
    T, D, V = case["T"], case["D"], case["V"]
    b, f = 2 * (T + V) * D + 16 * T, 2 * T * V * D
    if case["train"]:
        b += 2 * (T + V) * D + 4 * T
        f *= 3
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------- the definitions in 64 bits
def _norm_exact(s):
    x, w = s["x"].double(), s["weight"].double()
    K = x.shape[1]
    if s["kind"] == "layer":
        x = x - x.sum(1, keepdim=True) / K
    r = (x.square().sum(1, keepdim=True) / K + s["eps"]).rsqrt()
    n = x * r
    out = {"y": n * w + (s["bias_t"].double() if s["bias"] else 0.0)}
    if s["train"]:
        dy = s["dy"].double()
        q = dy * w
        along = (q * n).sum(1, keepdim=True) / K
        q_mean = q.sum(1, keepdim=True) / K if s["kind"] == "layer" else 0.0
        out["dx"] = r * (q - q_mean - n * along)
        out["dweight"] = torch.einsum("tk,tk->k", dy, n)
        if s["bias"]:
            out["dbias"] = dy.sum(0)
    return out


def _ffn_exact(s):
    # the int8 codes are defined by two IEEE float32 operations (s = 127 / max|x|, x * s) and a
    # rounding to even; everything after them is exact or in 64 bits
    x32 = s["x"].to(torch.float32)
    st32 = torch.full_like(x32[:, :1], 127.0) / torch.maximum(x32.abs().max(1, keepdim=True).values,
                                                              torch.full_like(x32[:, :1], 1e-5))
    xq = torch.round(torch.mul(x32, st32)).double()
    st = st32.double()
    mats = []
    for packed, scale in (s["gate"], s["up"]):
        t = torch.zeros(packed.shape[0], 4 * packed.shape[1], dtype=torch.float64, device=packed.device)
        for j in range(4):
            two = packed.bitwise_right_shift(2 * j).bitwise_and(3)
            t[:, j::4] = (two.bitwise_and(1).double() - two.bitwise_right_shift(1).double())
        mats.append(t * scale.double()[:, None])
    xh = xq / st
    g, u = xh @ mats[0].T, xh @ mats[1].T
    if s["act"] == "silu":
        sig = torch.sigmoid(g)
        a, slope = g * sig, sig + g * sig * (1 - sig)
    else:
        a, slope = torch.relu(g) ** 2, 2 * torch.relu(g)
    out = {"h": a * u}
    if s["train"]:
        dh = s["dh"].double()
        dg, du = dh * u * slope, dh * a
        out["dx"] = dg @ mats[0] + du @ mats[1]
        out["dgate"] = dg.T @ xh
        out["dup"] = du.T @ xh
    return out


def _xent_exact(s):
    x, w, t = s["x"].double(), s["w"].double(), s["target"]
    T, V = x.shape[0], w.shape[0]
    loss = torch.zeros(T, dtype=torch.float64, device=x.device)
    lse = torch.zeros_like(loss)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    rows = max(1, (1 << 28) // V)  # so many rows of logits at a time
    for a in range(0, T, rows):
        z = x[a:a + rows] @ w.T
        lse[a:a + rows] = torch.logsumexp(z, 1)
        live = (t[a:a + rows] != _IGNORE).nonzero()[:, 0]
        own_col = t[a:a + rows][live]
        loss[a + live] = lse[a + live] - z[live, own_col]
        if s["train"]:
            z = torch.softmax(z, 1)
            z[live, own_col] -= 1
            weight = torch.zeros(z.shape[0], dtype=torch.float64, device=x.device)
            weight[live] = s["dloss"][a:a + rows][live].double()
            z *= weight[:, None]
            dx[a:a + rows] = z @ w
            dw += z.T @ x[a:a + rows]
    out = {"loss": loss, "lse": lse}
    if s["train"]:
        out["dx"], out["dw"] = dx, dw
    return out


def exact(case, seed):
    return {"norm": _norm_exact, "ffn": _ffn_exact, "xent": _xent_exact}[case["op"]](prepare(case, seed))
