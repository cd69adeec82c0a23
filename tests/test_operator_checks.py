"""Refusals of the norm, gated feed-forward and cross-entropy calls, without a GPU:
the C entry points on fake aligned addresses (validation fails before anything
is enqueued), and the PyTorch calls with the library replaced by a recorder."""
import pytest
import torch

from sparse_linear_layers_b200 import api


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


class _NoLaunch:
    def __init__(self, device, stream):
        pass

    def __enter__(self):
        return 0

    def __exit__(self, *exc):
        pass


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder()
    monkeypatch.setattr(api, "lib", r)
    monkeypatch.setattr(api, "_LaunchOn", _NoLaunch)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: self.device.type == "cpu"))
    return r


def test_norm_rejects_on_host():
    from sparse_linear_layers_b200._lib import lib
    p, q = 4096, 8192
    N = lib.sbl_norm
    assert N(None, 1, 0, 64, 0, None, None, 1e-5, None, None, None, None) == 0   # T == 0
    assert N(p, 1, 4, 40, 0, p, None, 1e-5, q, None, None, None) == 1            # K % 16 != 0
    assert N(p, 1, 4, 1 << 25, 0, p, None, 1e-5, q, None, None, None) == 2       # K too long
    assert N(p, 1, -1, 64, 0, p, None, 1e-5, q, None, None, None) == 1
    assert N(p, 2, 4, 64, 0, p, None, 1e-5, q, None, None, None) == 1            # type
    assert N(p, 1, 4, 64, 2, p, None, 1e-5, q, None, None, None) == 1            # kind
    assert N(p, 1, 4, 64, 0, p, None, -1.0, q, None, None, None) == 1            # eps
    assert N(p, 1, 4, 64, 0, p, None, float("nan"), q, None, None, None) == 1
    assert N(p, 1, 4, 64, 0, None, None, 1e-5, q, None, None, None) == 1         # no weight
    assert N(p, 1, 4, 64, 0, p + 4, None, 1e-5, q, None, None, None) == 1        # unaligned weight
    assert N(p, 1, 4, 64, 0, p, p + 8, 1e-5, q, None, None, None) == 1           # unaligned bias
    assert N(p, 1, 4, 64, 0, p, None, 1e-5, p, None, None, None) == 1            # y is x
    B = lib.sbl_norm_backward
    assert B(p, p, 1, 4, 64, 0, p, None, p, None, None, None, q, 1 << 20, None) == 1        # no output
    assert B(p, p, 1, 4, 64, 1, p, None, p, q, None, None, q, 1 << 20, None) == 1           # layer: no mean
    assert B(p, p, 1, 4, 64, 0, p, None, None, q, None, None, q, 1 << 20, None) == 1        # no rstd
    assert B(p, p, 1, 4, 64, 0, p, None, p, p, None, None, q, 1 << 20, None) == 1           # dx is dy
    assert B(p, q, 1, 4, 64, 0, p, None, p, q, None, None, q, 1 << 20, None) == 1           # dx is x
    assert B(p, p, 1, 4, 64, 0, p, None, p, None, q + 4, None, q, 1 << 20, None) == 1       # unaligned dweight
    assert B(p, p, 1, 4, 64, 0, p, None, p, None, q, None, None, 1 << 20, None) == 6        # no workspace
    assert B(p, p, 1, 4, 64, 0, p, None, p, None, q, None, q + 16, 1 << 20, None) == 6      # unaligned workspace


def test_norm_tensor_checks(rec):
    x, w = torch.zeros(4, 64), torch.ones(64)
    ok = [lambda: api.sbl_norm(x, w), lambda: api.sbl_norm(x.bfloat16(), w, w, kind="layer", with_stats=True)]
    for f in ok:
        f()
    assert rec.calls == ["sbl_norm", "sbl_norm"]
    r = torch.ones(4)
    bad = [lambda: api.sbl_norm(x, w, kind="batch"), lambda: api.sbl_norm(x.half(), w), lambda: api.sbl_norm(x[0], w),
           lambda: api.sbl_norm(x, w[:32]), lambda: api.sbl_norm(x, w.double()), lambda: api.sbl_norm(x, w, w[:16]),
           lambda: api.sbl_norm(x.t(), torch.ones(4)), lambda: api.sbl_norm(x, w, y=torch.zeros(4, 32)),
           lambda: api.sbl_norm(x, w, y=torch.zeros(4, 64).bfloat16()),
           lambda: api.sbl_norm_backward(x[:3], x, w, None, r), lambda: api.sbl_norm_backward(x.bfloat16(), x, w, None, r),
           lambda: api.sbl_norm_backward(x, x, w, None, r[:3]), lambda: api.sbl_norm_backward(x, x, w, None, r, kind="layer"),
           lambda: api.sbl_norm_backward(x, x, w, r.double(), r, kind="layer"),
           lambda: api.sbl_norm_backward(x, x, w, None, r, need_dx=False, need_dw=False, need_db=False),
           lambda: api.sbl_norm_backward(x, x, w, None, r, workspace=torch.zeros(8))]
    for f in bad:
        with pytest.raises(ValueError):
            f()


def test_cross_entropy_rejects_on_host():
    from sparse_linear_layers_b200._lib import lib
    p, big = 4096, 1 << 40
    F = lib.sbl_linear_cross_entropy
    assert F(None, 0, 64, None, 100, None, -100, None, None, None, 0, None) == 0      # T == 0
    assert F(p, 4, 40, p, 100, p, -100, p, p, p, big, None) == 1                      # D % 16 != 0
    assert F(p, -1, 64, p, 100, p, -100, p, p, p, big, None) == 1
    assert F(p, 4, 64, p, 0, p, -100, p, p, p, big, None) == 1                        # no words
    assert F(p, 4, 64, p, 1 << 25, p, -100, p, p, p, big, None) == 2
    assert F(p, 1 << 25, 64, p, 100, p, -100, p, p, p, big, None) == 2
    assert F(p, 4, 64, None, 100, p, -100, p, p, p, big, None) == 1                   # missing W
    assert F(p + 8, 4, 64, p, 100, p, -100, p, p, p, big, None) == 1                  # unaligned x
    assert F(p, 4, 64, p, 100, p + 4, -100, p, p, p, big, None) == 1                  # unaligned target
    assert F(p, 4, 64, p, 100, p + 8, -100, p + 4, p + 4, None, big, None) == 6       # any element will do
    assert F(p, 1 << 24, 64, p, 1 << 24, p, -100, p, p, p, big, None) == 2            # too many tiles
    assert F(p, 4, 64, p, 100, p, -100, p, p, None, big, None) == 6
    assert F(p, 4, 64, p, 100, p, -100, p, p, p + 16, big, None) == 6
    need = lib.sbl_linear_cross_entropy_workspace_bytes(4, 100)
    assert need == 256 + 256 and F(p, 4, 64, p, 100, p, -100, p, p, p, need - 1, None) == 6
    B = lib.sbl_linear_cross_entropy_backward
    assert B(p, p, 4, 64, p, 100, p, -100, p, None, None, p, big, None) == 1          # no output
    assert B(p, p, 4, 64, p, 100, p, -100, p, p + 4, None, p, big, None) == 1         # unaligned dx
    assert B(p, p, 4, 64, p, 100, p, -100, None, p, None, p, big, None) == 1          # no lse
    assert B(None, p, 4, 64, p, 100, p, -100, p, p, None, p, big, None) == 1          # no dloss
    assert B(p, p, 4, 64, p, 100, p, -100, p, p, None, None, big, None) == 6
    assert B(p, p, 4, 64, p, 100, p, -100, p, p, None, p + 16, big, None) == 6
    assert lib.sbl_linear_cross_entropy_backward_workspace_bytes(0, 64, 100, 1) == 0


def test_cross_entropy_tensor_checks(rec):
    x, w, t = torch.zeros(4, 64).bfloat16(), torch.zeros(100, 64).bfloat16(), torch.zeros(4, dtype=torch.int64)
    f = torch.zeros(4)
    rec.sbl_linear_cross_entropy_workspace_bytes = lambda *a: 16
    rec.sbl_linear_cross_entropy_backward_workspace_bytes = lambda *a: 16
    api.sbl_linear_cross_entropy(x, w, t)
    api.sbl_linear_cross_entropy_backward(f, x, w, t, f)
    assert rec.calls == ["sbl_linear_cross_entropy", "sbl_linear_cross_entropy_backward"]
    bad = [lambda: api.sbl_linear_cross_entropy(x.float(), w, t), lambda: api.sbl_linear_cross_entropy(x, w.float(), t),
           lambda: api.sbl_linear_cross_entropy(x, w[:, :32], t), lambda: api.sbl_linear_cross_entropy(x, w, t.int()),
           lambda: api.sbl_linear_cross_entropy(x, w, t[:3]), lambda: api.sbl_linear_cross_entropy(x[0], w, t),
           lambda: api.sbl_linear_cross_entropy(x, w.t().contiguous().t(), t),
           lambda: api.sbl_linear_cross_entropy_backward(f[:3], x, w, t, f),
           lambda: api.sbl_linear_cross_entropy_backward(f.double(), x, w, t, f),
           lambda: api.sbl_linear_cross_entropy_backward(f, x, w, t, f[:2]),
           lambda: api.sbl_linear_cross_entropy_backward(f, x, w, t, f, need_dx=False, need_dw=False)]
    for g in bad:
        with pytest.raises(ValueError):
            g()


def test_ffn_gated_rejects_on_host():
    from sparse_linear_layers_b200._lib import lib
    p, big = 4096, 1 << 40
    F = lib.sbl_ffn_gated
    assert F(None, 0, 64, None, None, None, None, 8, 2, 4, 0, None, 1, None, 0, None) == 0     # T == 0
    assert F(None, 4, 64, None, None, None, None, 0, 2, 4, 0, None, 1, None, 0, None) == 0     # F == 0
    assert F(p, 4, 40, p, p, p, p, 8, 2, 4, 0, p, 1, p, big, None) == 1                        # K % 16 != 0
    assert F(p, 4, 64, p, p, p, p, 8, 1, 4, 0, p, 1, p, big, None) == 2                        # pattern
    assert F(p, 4, 64, p, p, p, p, 8, 2, 4, 2, p, 1, p, big, None) == 1                        # activation
    assert F(p, 4, 64, p, p, p, p, 8, 2, 4, 0, p, 2, p, big, None) == 1                        # output type
    assert F(p, 4, 64, p, p, None, p, 8, 2, 4, 0, p, 1, p, big, None) == 1                     # no up matrix
    assert F(p, 4, 64, p, p, p, p + 4, 8, 2, 4, 0, p, 1, p, big, None) == 1                    # unaligned scale
    assert F(p, 1 << 25, 64, p, p, p, p, 8, 2, 4, 0, p, 1, p, big, None) == 2
    assert F(p, 4, 1 << 18, p, p, p, p, 8, 2, 4, 0, p, 1, p, big, None) == 2
    assert lib.sbl_ffn_gated_workspace_bytes(16, 2048, 7168) == 0
    need = lib.sbl_ffn_gated_workspace_bytes(17, 64, 8)
    assert need == 17 * 64 + 192 + 256                 # x_q rounded to 256, s_tok
    assert F(p, 17, 64, p, p, p, p, 8, 2, 4, 0, p, 1, None, big, None) == 6
    assert F(p, 17, 64, p, p, p, p, 8, 2, 4, 0, p, 1, p + 64, big, None) == 6
    assert F(p, 17, 64, p, p, p, p, 8, 2, 4, 0, p, 1, p, need - 1, None) == 6
    B = lib.sbl_ffn_gated_backward
    assert B(p, p, 4, 64, p, p, p, p, 8, 2, 4, 0, None, None, None, 0, p, big, None) == 1      # no output
    assert B(p, p, 4, 64, p, p, p, p, 8, 2, 4, 0, p, None, None, 2, p, big, None) == 1         # flags
    assert B(None, p, 4, 64, p, p, p, p, 8, 2, 4, 0, p, None, None, 0, p, big, None) == 1      # no dh
    assert B(p, p, 4, 64, p, p, p, p, 8, 2, 4, 0, p, p + 4, None, 0, p, big, None) == 1        # unaligned dW
    need = lib.sbl_ffn_gated_backward_workspace_bytes(4, 64, 8, 1, 0)
    assert need > 0 and B(p, p, 4, 64, p, p, p, p, 8, 2, 4, 0, p, None, None, 0, p, need - 1, None) == 6
    assert B(p, p, 4, 64, p, p, p, p, 8, 2, 4, 0, p, None, None, 0, None, big, None) == 6


def test_ffn_gated_tensor_checks(rec):
    def weights(F=8, K=64, n=2, m=4):
        return api.PreparedWeights(torch.zeros((F, K // 4), dtype=torch.uint8), torch.zeros(F), n, m, K)

    x, g, u, dh = torch.zeros(4, 64).bfloat16(), weights(), weights(), torch.zeros(4, 8)
    rec.sbl_ffn_gated_workspace_bytes = lambda *a: 0
    rec.sbl_ffn_gated_backward_workspace_bytes = lambda *a: 16
    api.sbl_ffn_gated(x, g, u)
    api.sbl_ffn_gated_backward(dh, x, g, u)
    assert rec.calls == ["sbl_ffn_gated", "sbl_ffn_gated_backward"]
    short = api.PreparedWeights(g.packed, torch.zeros(7), 2, 4, 64)
    bad = [lambda: api.sbl_ffn_gated(x.float(), g, u), lambda: api.sbl_ffn_gated(x[0], g, u),
           lambda: api.sbl_ffn_gated(x, g, weights(F=9)), lambda: api.sbl_ffn_gated(x, g, weights(K=128)),
           lambda: api.sbl_ffn_gated(x, g, weights(n=3)), lambda: api.sbl_ffn_gated(x, g, short),
           lambda: api.sbl_ffn_gated(x, g, u, act="gelu"), lambda: api.sbl_ffn_gated(x, g, u, out_dtype=torch.float16),
           lambda: api.sbl_ffn_gated(x, g, u, h=torch.zeros(4, 7)), lambda: api.sbl_ffn_gated(x, g, u, h=torch.zeros(8, 4).t()),
           lambda: api.sbl_ffn_gated_backward(dh[:, :4], x, g, u), lambda: api.sbl_ffn_gated_backward(dh.bfloat16(), x, g, u),
           lambda: api.sbl_ffn_gated_backward(dh, x, g, u, need_dx=False, need_dgate=False, need_dup=False)]
    for f in bad:
        with pytest.raises(ValueError):
            f()


def test_feed_forward_runs_on_the_device_of_its_input(monkeypatch):
    """The module's calls are made with the input's device current."""
    import contextlib

    from sparse_linear_layers_b200 import train

    entered = []

    @contextlib.contextmanager
    def device(d):
        entered.append(d)
        yield

    class OnGpu:
        is_cuda, device = True, torch.device("cuda", 1)

    monkeypatch.setattr(torch.cuda, "device", device)
    with train._on_device_of(OnGpu()):
        assert entered == [torch.device("cuda", 1)]
    with train._on_device_of(torch.zeros(1)):
        assert len(entered) == 1
    ffn = train.SparseBitFeedForward(64, 96)
    with pytest.raises(ValueError):
        ffn(torch.zeros(2, 64))     # not on a GPU
