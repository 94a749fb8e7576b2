"""The gated product in plain form, in 64 bits, and a check of its gradients against differences of it. torch only."""
import math

import torch

STEP = 2.0 ** -11  # half a step of fp16

# the largest slope of the activation, and of its derivative
SLOPES = {"silu": (1.1, 0.5), "gelu": (1.13, 0.8), "gelu_tanh": (1.13, 0.8), "relu": (1.0, 0.0), "sigmoid": (0.25, 0.1)}


def activation(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1 + torch.erf(g / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    return torch.relu(g) if act == "relu" else 1 / (1 + torch.exp(-g))


def value(x, wg, wu, dh, act):
    """sum of dh * h, whose gradients gated_product_backward gives."""
    return (activation(x @ wg.t(), act) * (x @ wu.t()) * dh).sum()


def inputs(seed=3, m=12, d=40, f=72):
    """x, w_gate, w_up and dh in fp16."""
    g = torch.Generator().manual_seed(seed)
    x, wg, wu, dh = (torch.randn(*s, generator=g) for s in ((m, d), (f, d), (f, d), (m, f)))
    return x.half(), (wg * 0.1).half(), (wu * 0.1).half(), dh.half()


def against_differences(grads, x, wg, wu, dh, act):
    """[(operand, what the gradient says of the slope along a direction, the slope by differences, how far they may be
    apart)] for (dx, dw_gate, dw_up), all on the host. The direction has the signs of the gradient, so that the slope is as
    large as its terms.

    How far: gate and up are kept in fp16, and dgate, dup and dx are rounded to it, each by at most STEP of its value.
    dgate = dh act'(gate) up is then off by three such steps of itself (up's, its own, dx's) and one of gate through act',
    dup = dh act(gate) by two of itself and one of gate through act; fp32 sums and the differences' own error (step^2 times
    third derivatives) are under a hundredth of a step."""
    ops = [t.double().requires_grad_() for t in (x, wg, wu)]
    D = dh.double()
    signs = [g.sign() for g in torch.autograd.grad(value(*ops, D, act), ops)]
    X, G, V = (t.detach() for t in ops)
    Z, U = X @ G.t(), X @ V.t()
    s1, s2 = SLOPES[act]
    A = activation(Z, act).abs()
    z = Z.clone().requires_grad_()
    DA = torch.autograd.grad(activation(z, act).sum(), z)[0].abs()
    eg = STEP * D.abs() * (3.1 * DA * U.abs() + s2 * Z.abs() * U.abs())
    eu = STEP * D.abs() * (2.1 * A + s1 * Z.abs())
    far = (eg @ G.abs() + eu @ V.abs(), eg.t() @ X.abs(), eu.t() @ X.abs())
    out, h = [], 1e-6
    for k, (name, e) in enumerate(zip(("dx", "dw_gate", "dw_up"), signs)):
        up, down = ([t + s * h * e if i == k else t for i, t in enumerate((X, G, V))] for s in (1, -1))
        slope = (value(*up, D, act) - value(*down, D, act)) / (2 * h)
        out.append((name, float((grads[k].double().cpu() * e).sum()), float(slope), float((far[k] * e.abs()).sum())))
    return out


def check_differences(grads, x, wg, wu, dh, act):
    for name, got, slope, far in against_differences(grads, x, wg, wu, dh, act):
        assert abs(got - slope) <= far, f"{act}: {name} says {got}, the differences {slope}, {far} apart at most"
        assert far <= 0.2 * slope, "a bound that lets everything pass"
