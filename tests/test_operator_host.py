"""Host-side behaviour of the operators around the layer, without a GPU."""


def test_empty_batches_ask_for_nothing_on_the_host():
    """The gradient of an empty input has no address: alone it is no missing output."""
    from sparse_linear_layers_b200._lib import lib
    p = 4096
    norm = lambda T, kind=0: lib.sbl_norm_backward(None, None, 1, T, 64, kind, p, None, None, None, None, None, None, 0, None)
    assert norm(0) == norm(0, 1) == 0 and norm(4) == 1
    ffn = lambda T, F: lib.sbl_ffn_gated_backward(p, p, T, 64, p, p, p, p, F, 2, 4, 0, None, None, None, 0, p, 1 << 40, None)
    assert ffn(0, 8) == ffn(4, 0) == ffn(0, 0) == 0 and ffn(4, 8) == 1
    ce = lambda T: lib.sbl_linear_cross_entropy_backward(p, p, T, 64, p, 100, p, -100, p, None, None, p, 1 << 40, None)
    assert ce(0) == 0 and ce(4) == 1
    for f, ws in ((lib.sbl_linear_backward, ()), (lib.sbl_linear_backward_ws, (p, 1 << 20))):
        lin = lambda T, O: f(p, T, O, p, p, 64, p, p, None, None, 0, *ws, None)
        assert lin(0, 8) == lin(4, 0) == 0 and lin(4, 8) == 1
    # sizes and types are checked all the same
    assert norm(-1) == 1 and norm(0, 2) == 1 and ffn(-1, 8) == 1 and ce(-1) == 1


PLAN_PROGRAM = r"""
#include <cstdio>
#include "gemm_f16.cuh"
using namespace sbl;
int main() {
    const GemmWork none{0, 1, 0.0, 0.0, 0.0, 1};
    int wrong = 0;
    for (long long tiles = 1; tiles < 700; ++tiles)
        for (long long KB : {1, 3, 14, 37, 250, 2048}) {
            const GemmWork x{tiles, KB, 0.55, 1.0, 1e6, 64};
            const GemmPlan p = gemm_plan(x, none);
            // alone: the rounds of 74 pairs, and no tiles of a second product to begin with
            const double s = p.splits1;
            const double us = (long long)((tiles * p.splits1 + 73) / 74) * ((KB + p.splits1 - 1) / p.splits1 * 0.55 + 1.0) +
                              (s > 1 ? 3.0 + s * 2.0 / 6.0 : 0.0);
            if (p.lead != 0 || p.splits2 != 1 || !(p.us - us < 1e-9 && us - p.us < 1e-9)) {
                if (!wrong++) printf("%lld tiles of %lld: lead %d, splits %d %d, %g us for %g\n", tiles, KB, p.lead, p.splits1, p.splits2, p.us, us);
            }
        }
    printf("%d wrong\n", wrong);
    return wrong != 0;
}
"""


def test_plan_of_one_product_alone(tmp_path):
    """gemm_plan with no second product: a finite plan, without tiles of it to lead with."""
    import subprocess

    from sparse_linear_layers_b200 import build
    src = tmp_path / "plan.cu"
    src.write_text(PLAN_PROGRAM)
    exe = str(tmp_path / "plan")
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", build.INCLUDE, "-I", build.CSRC,
                    str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_bad_targets_are_named_before_anything_runs():
    import pytest
    import torch

    from sparse_linear_layers_b200 import train
    head = train.LinearCrossEntropy(16, 10, ignore_index=99)
    for wrong in (-1, 10, 1 << 40, -100):
        with pytest.raises(IndexError, match="LinearCrossEntropy.*%d " % wrong):
            head(torch.zeros(2, 16), torch.tensor([3, wrong]))
    for ok in (0, 9, 99):
        with pytest.raises(ValueError):       # past the check: x is not on a GPU
            head(torch.zeros(2, 16), torch.tensor([3, ok]))
    head.check_targets = False
    with pytest.raises(ValueError):
        head(torch.zeros(2, 16), torch.tensor([3, 10]))


def test_an_earlier_calls_status_is_not_blamed_on_a_module(monkeypatch):
    import pytest

    from sparse_linear_layers_b200 import _lib, api, train
    monkeypatch.setattr(api, "sbl_device_status", lambda: _lib.SBL_ERR_INVALID_ARG)
    with pytest.raises(_lib.SblError, match="earlier call .sbl_linear_cross_entropy"):
        train._stop_on_nonfinite("SparseBitLinear")
    monkeypatch.setattr(api, "sbl_device_status", lambda: _lib.SBL_ERR_NONFINITE)
    with pytest.raises(FloatingPointError, match="SparseBitLinear"):
        train._stop_on_nonfinite("SparseBitLinear")


def test_outputs_over_inputs_are_refused_on_the_host():
    """One row further on, or the same memory: some kernels read their inputs until
    their last output is written."""
    from sparse_linear_layers_b200._lib import lib
    x, far, big = 1 << 20, 1 << 30, 1 << 40
    norm = lambda y, dt=1: lib.sbl_norm(x, dt, 8, 64, 0, far, None, 1e-5, y, None, None, None)
    for y in (x, x + 128, x - 128, x + 7 * 128):
        assert norm(y) == 1 and norm(y, 0) == 1
    back = lambda dx, dy=far: lib.sbl_norm_backward(dy, x, 1, 8, 64, 0, far, None, far, dx, None, None, None, 0, None)
    for dx in (x + 128, x - 7 * 128, far + 256, far - 128):
        assert back(dx) == 1
    ffn = lambda h, T, F, dt: lib.sbl_ffn_gated(x, T, 64, far, far, far, far, F, 2, 4, 0, h, dt, far, big, None)
    for T in (1, 8, 16):
        assert ffn(x, T, 64, 1) == 1 and ffn(x + 128 * T - 16, T, 16, 0) == 1 and ffn(x - 16, T, 5, 0) == 1
    ce = lambda dx, dw: lib.sbl_linear_cross_entropy_backward(far, x, 8, 64, 2 * x, 100, far, -100, far, dx, dw, far, big, None)
    for p in (x, x + 128, 2 * x, 2 * x + 99 * 128, 2 * x - 128):
        assert ce(None, p) == 1 and ce(far, p) == 1
    if not has_device():    # beside its input: nothing is refused before the missing device
        assert norm(x + 8 * 128) == back(x - 8 * 128) == ffn(x + 8 * 128, 8, 64, 1) == ffn(x - 8 * 4, 8, 1, 0) == 4
        assert ce(x + 8 * 128, 2 * x + 100 * 128) == 4


def has_device():
    import torch
    return torch.cuda.is_available()
