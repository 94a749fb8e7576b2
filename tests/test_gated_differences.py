"""The check of the gated product's gradients against differences passes for the formulas' gradients, rounded where the
kernels round, and fails for wrong ones (no GPU: the mistakes are planted in a plain form)."""
import pytest
import torch

from _gated import SLOPES, activation, check_differences, inputs


def plain(x, wg, wu, dh, act, wrong=None):
    """dx, dw_gate and dw_up with every rounding of the kernels, and a mistake."""
    def half(t):
        return t.half().double()
    X, G, V, D = (t.double() for t in (x, wg, wu, dh))
    z = half(X @ G.t()).requires_grad_()
    up, A = half(X @ V.t()), activation(z, act)
    DA = torch.autograd.grad(A.sum(), z)[0]
    if wrong == "no slope":
        DA = torch.ones_like(DA)
    if wrong == "slope of another":
        DA = torch.autograd.grad(activation(z, "relu" if act != "relu" else "silu").sum(), z)[0]
    dg, du = half(D * DA * up), half(D * A.detach())
    if wrong == "up forgotten":
        dg = half(D * DA)
    dx = half(dg @ G + (0 if wrong == "a term of dx" else du @ V))
    dwg, dwu = dg.t() @ X, du.t() @ X
    if wrong == "swapped":
        dwg, dwu = dwu, dwg
    if wrong in ("dx", "dw_gate", "dw_up"):
        (dx if wrong == "dx" else dwg if wrong == "dw_gate" else dwu).zero_()
    return dx, dwg, dwu


@pytest.mark.parametrize("seed", [3, 4, 5])
@pytest.mark.parametrize("act", SLOPES)
def test_right_gradients_pass(act, seed):
    x, wg, wu, dh = inputs(seed)
    check_differences(plain(x, wg, wu, dh, act), x, wg, wu, dh, act)


@pytest.mark.parametrize("wrong", ["dx", "dw_gate", "dw_up", "no slope", "slope of another", "up forgotten", "a term of dx",
                                   "swapped"])
@pytest.mark.parametrize("act", SLOPES)
def test_wrong_gradients_do_not(act, wrong):
    x, wg, wu, dh = inputs()
    with pytest.raises(AssertionError, match="differences"):
        check_differences(plain(x, wg, wu, dh, act, wrong), x, wg, wu, dh, act)
