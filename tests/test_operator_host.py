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
