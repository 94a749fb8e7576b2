"""The gated product and its backward pass on the GPU against plain forms in 64 bits.

Most cases use small whole numbers, whose products and sums fp32 holds exactly in
any order: there the outputs must be the exact result rounded once, and every
value of every tile, whatever its size and alignment, is checked for equality.
Random values are compared within the error of the fp32 sums, at most
K 2^-23 sum |a b| for a contraction of K terms in any order, truncation included,
carried through the formulas, and half a step of the output's type."""
import math

import numpy as np
import pytest
import torch

import _gated
import zero_dp_partitioned_amd as zdp
from _gpu_helpers import DEV

pytestmark = pytest.mark.gpu

DTS = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
U = 2.0 ** -24
ACTS = list(zdp.ACTIVATIONS)


@pytest.fixture(scope="module")
def ws():
    w = zdp.new_workspace(1)
    w.fill_(0xFF)  # NaN patterns: nothing of it may be read before it is written
    return w


def wide(t, pad):
    """The same values as rows of a wider tensor that start off its beginning."""
    if not pad:
        return t
    big = torch.full((t.shape[0], t.shape[1] + pad + 1), float("nan"), dtype=t.dtype, device=DEV)
    big[:, 1:1 + t.shape[1]] = t
    return big[:, 1:1 + t.shape[1]]


class Blank:
    """An output inside a larger one full of a marker."""

    def __init__(self, rows, cols, dtype, pad):
        self.big = torch.full((rows + 2, cols + 2 * pad), -77.0, dtype=dtype, device=DEV)
        self.t = self.big[1:1 + rows, pad:pad + cols] if pad else self.big[1:1 + rows]

    def check(self):
        mask = torch.ones_like(self.big, dtype=torch.bool)
        r, c = self.t.shape
        off = (self.big.shape[1] - c) // 2
        mask[1:1 + r, off:off + c] = False
        assert (self.big[mask] == -77).all(), "written outside the output"


def whole_numbers(g, rows, cols, dtype, density):
    """-1, 0 and 1, `density` of them not 0."""
    t = torch.randint(0, 2 ** 16, (rows, cols), generator=g, device=DEV)
    return (torch.where(t % 2 == 0, 1.0, -1.0) * (t < density * 2 ** 16)).to(dtype)


def same(got, want, what):
    """got is the exact want rounded to its type."""
    bad = got != want.to(got.dtype)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[0].tolist()}"


# (m, d, f): one, the ends of a slot, of a chunk of 64, of each tile and of the tiles' variants; short and long contractions
SIZES = [(1, 1, 1), (1, 8, 8), (2, 7, 9), (1, 64, 64), (1, 65, 130), (3, 200, 333), (16, 64, 128), (17, 72, 136), (33, 63, 65),
         (64, 128, 64), (65, 129, 127), (63, 136, 64), (1, 1600, 640), (45, 1600, 640), (128, 256, 128), (129, 257, 255),
         (100, 1, 100), (100, 5, 77), (300, 64, 40), (257, 8, 1000), (128, 4096, 64), (5, 16, 4000), (1000, 264, 200),
         (1001, 100, 203), (1500, 136, 1111), (70, 64, 5000), (2100, 72, 130), (256, 2048, 3000), (250, 2043, 2995),
         (2100, 72, 1300), (2100, 2600, 72), (2100, 2603, 70), (72, 1700, 1304), (71, 1703, 1301)]
# many tiles of 256: forward by m x f, dx by m x d, dw by f x d
LARGE = [(2560, 72, 2048), (2500, 67, 2001), (2561, 128, 2056), (4096, 2560, 72), (4000, 2555, 65), (4001, 2568, 136),
         (72, 2560, 2048), (67, 2555, 2043), (130, 2568, 2056), (1300, 1300, 1300)]


def pads(size):
    return 3 if sum(size) % 3 == 0 else 0


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("size", SIZES + LARGE, ids=str)
def test_forward_of_whole_numbers(size, dt):
    m, d, f = size
    g, dtype, pad = torch.Generator(device=DEV).manual_seed(m + d + f), DTS[dt], pads(size)
    p = min(1.0, math.sqrt(200 / d))  # products of a few tens
    x, wg, wu = (whole_numbers(g, r, d, dtype, p) for r in (m, f, f))
    G, U_ = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    x, wg, wu = wide(x, pad), wide(wg, pad), wide(wu, pad)
    outs = [Blank(m, f, dtype, pad) for _ in range(3)]
    zdp.gated_product(x, wg, wu, outs[0].t, "relu", gate=outs[1].t, up=outs[2].t)
    for o, want, what in zip(outs, (G.clamp_min(0) * U_, G, U_), ("h", "gate", "up")):
        same(o.t, want, what)
        o.check()
    h = torch.empty(m, f, dtype=dtype, device=DEV)
    zdp.gated_product(x, wg, wu, h, "relu")  # without the products
    assert torch.equal(h, outs[0].t)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("size", SIZES + LARGE, ids=str)
def test_backward_of_whole_numbers(size, dt, ws):
    m, d, f = size
    g, dtype, pad = torch.Generator(device=DEV).manual_seed(m + d + f + 1), DTS[dt], pads(size)
    x, wg, wu = (whole_numbers(g, r, d, dtype, 0.5) for r in (m, f, f))
    gate, up = (whole_numbers(g, m, f, dtype, 0.9) * 2 for _ in range(2))
    dh = whole_numbers(g, m, f, dtype, min(1.0, math.sqrt(100 / max(m, f))))
    X, WG, WU, GT, UP, DH = (t.double() for t in (x, wg, wu, gate, up, dh))
    DG, DU = DH * (GT > 0) * UP, DH * GT.clamp_min(0)
    DX, DWG, DWU = DG @ WG + DU @ WU, DG.t() @ X, DU.t() @ X
    x, wg, wu, gate, up, dh = (wide(t, pad) for t in (x, wg, wu, gate, up, dh))
    dg, du, dx = Blank(m, f, dtype, pad), Blank(m, f, dtype, pad), Blank(m, d, dtype, pad)
    out = torch.float32 if (m + d) % 2 else dtype
    dwg, dwu = Blank(f, d, out, pad), Blank(f, d, out, pad)
    zdp.gated_product_backward(dh, x, wg, wu, gate, up, dg.t, du.t, ws, dx=dx.t, dw_gate=dwg.t, dw_up=dwu.t, act="relu")
    for o, want, what in zip((dg, du, dx, dwg, dwu), (DG, DU, DX, DWG, DWU), ("dgate", "dup", "dx", "dw_gate", "dw_up")):
        same(o.t, want, what)
        o.check()
    # one at a time, the gradients of the weights added to what they hold, dgate and dup in the place of gate and up
    base = torch.randint(-8, 9, (f, d), generator=g, device=DEV).to(out)
    dwg.t.copy_(base)
    dwu.t.copy_(-base)
    dx2 = torch.empty(m, d, dtype=dtype, device=DEV)
    zdp.gated_product_backward(dh, x, wg, wu, gate, up, dg.t, du.t, ws, dx=dx2, act="relu")
    assert torch.equal(dx2, dx.t)
    zdp.gated_product_backward(dh, x, wg, wu, gate, up, gate, up, ws, dw_gate=dwg.t, dw_up=dwu.t, act="relu", accumulate=True)
    same(dwg.t, DWG + base.double(), "dw_gate added")
    same(dwu.t, DWU - base.double(), "dw_up added")
    assert torch.equal(gate, dg.t) and torch.equal(up, du.t)
    dwg.check()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("size", [(1500, 1600, 640), (1501, 1600, 648), (1500, 1608, 1000), (500, 1600, 6400)], ids=str)
def test_both_products_of_the_backward_pass_in_one_launch(size, dt, ws):
    """Sizes whose dx and dw share a launch, against the two asked for one by one, with and without adding: exact."""
    m, d, f = size
    g, dtype = torch.Generator(device=DEV).manual_seed(m), DTS[dt]
    x, wg, wu = (whole_numbers(g, r, d, dtype, 0.5) for r in (m, f, f))
    gate, up = (whole_numbers(g, m, f, dtype, 0.9) * 2 for _ in range(2))
    dh = whole_numbers(g, m, f, dtype, math.sqrt(100 / max(m, f)))
    out = torch.float32 if m % 2 else dtype
    dg, du = torch.empty_like(gate), torch.empty_like(up)
    base = torch.randint(-8, 9, (f, d), generator=g, device=DEV).to(out)
    dx, a, b = Blank(m, d, dtype, 8), Blank(f, d, out, 8), Blank(f, d, out, 8)
    for accumulate in (False, True):
        for t in (a.t, b.t):
            t.copy_(base)
        zdp.gated_product_backward(dh, x, wg, wu, gate, up, dg, du, ws, dx=dx.t, dw_gate=a.t, dw_up=b.t, act="relu",
                                   accumulate=accumulate)
        G, H = dg.double(), du.double()
        extra = base.double() if accumulate else 0
        same(dx.t, G @ wg.double() + H @ wu.double(), "dx")
        same(a.t, G.t() @ x.double() + extra, "dw_gate")
        same(b.t, H.t() @ x.double() + extra, "dw_up")
        for o in (dx, a, b):
            o.check()


# --------------------------------------------------------------------------
# random values
# --------------------------------------------------------------------------

def act_of(z, act):
    """The activation, its derivative, and a bound of the derivative's own slope (float64)."""
    if act == "relu":
        return z.clamp_min(0), (z > 0).double()
    s = torch.sigmoid(z)
    if act == "sigmoid":
        return s, s * torch.sigmoid(-z)
    if act == "silu":
        return z * s, s + z * s * torch.sigmoid(-z)
    if act == "gelu":
        c = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    a = 2 * math.sqrt(2 / math.pi) * z * (1 + 0.044715 * z * z)
    s = torch.sigmoid(a)
    return z * s, s + z * s * torch.sigmoid(-a) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)


def close(got, want, err, what):
    h, tiny = HALF_STEP[got.dtype], TINY[got.dtype]
    assert got.isfinite().all(), what
    over = (got.double() - want).abs() - (err * (1 + 2 * h) + h * want.abs() + tiny)
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} off, worst by {float(over.max())}"


def act_error(z, a):
    """What the fp32 activation is off by: exp's argument is rounded, which is |argument| u of its value, 1 / x and the
    products add a few u each, and the argument of gelu_tanh grows as 1.6 |z| + 0.08 |z|^3: (2 |z| + 0.1 |z|^3 + 16) u of
    |a|. Where a falls below 2^-60 it is as good as 0 beside the products' own errors."""
    return (2 * z.abs() + 0.1 * z.abs() ** 3 + 16) * U * (a.abs() + 2.0 ** -60)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", [(1, 512, 200), (37, 200, 333), (130, 640, 256), (513, 100, 1000)], ids=str)
def test_forward(size, act, dt):
    m, d, f = size
    g, dtype = torch.Generator(device=DEV).manual_seed(d + f), DTS[dt]
    x = torch.randn(m, d, generator=g, device=DEV).to(dtype)
    wg, wu = ((torch.randn(f, d, generator=g, device=DEV) * 3 / math.sqrt(d)).to(dtype) for _ in range(2))
    h, gate, up = (torch.empty(m, f, dtype=dtype, device=DEV) for _ in range(3))
    zdp.gated_product(x, wg, wu, h, act, gate=gate, up=up)
    G, V = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    eg, ev = (d * 2.0 ** -23 * (x.double().abs() @ w.double().abs().t()) for w in (wg, wu))
    close(gate, G, eg, "gate")
    close(up, V, ev, "up")
    A, _ = act_of(G, act)
    ea = 1.2 * eg + act_error(G, A)  # no activation here is steeper than 1.13
    close(h, A * V, ea * (V.abs() + ev) + A.abs() * ev + 2 * U * (A * V).abs(), "h")


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", [(1, 200, 512), (37, 200, 333), (130, 256, 640), (1000, 100, 130)], ids=str)
def test_backward(size, act, dt, ws):
    m, d, f = size
    g, dtype = torch.Generator(device=DEV).manual_seed(d + f + 7), DTS[dt]

    def rnd(r, c, s=1.0):
        return (torch.randn(r, c, generator=g, device=DEV) * s).to(dtype)
    x, wg, wu, dh = rnd(m, d), rnd(f, d, 0.1), rnd(f, d, 0.1), rnd(m, f)
    gate, up = rnd(m, f, 3.0), rnd(m, f)
    dg, du, dx = torch.empty_like(gate), torch.empty_like(up), torch.empty_like(x)
    dwg, dwu = torch.empty(f, d, device=DEV), torch.empty(f, d, device=DEV)
    zdp.gated_product_backward(dh, x, wg, wu, gate, up, dg, du, ws, dx=dx, dw_gate=dwg, dw_up=dwu, act=act)
    Z, V, D = gate.double(), up.double(), dh.double()
    A, DA = act_of(Z, act)
    # the derivative is a sum of two products that may cancel: its error is relative to their magnitudes, at most 1 + |z| / 2
    eda = act_error(Z, 1 + Z.abs() / 2) if act != "relu" else torch.zeros_like(Z)
    close(dg, D * DA * V, (D * V).abs() * (eda + 3 * U * DA.abs()), "dgate")
    close(du, D * A, D.abs() * (act_error(Z, A) + 2 * U * A.abs()), "dup")
    G, H = dg.double(), du.double()  # the products are those of the rounded values
    k = 2.0 ** -23
    close(dx, G @ wg.double() + H @ wu.double(), 2 * f * k * (G.abs() @ wg.double().abs() + H.abs() @ wu.double().abs()), "dx")
    close(dwg, G.t() @ x.double(), m * k * (G.abs().t() @ x.double().abs()), "dw_gate")
    close(dwu, H.t() @ x.double(), m * k * (H.abs().t() @ x.double().abs()), "dw_up")


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act, ws):
    """The gradients are the forward pass's slopes: differences of its 64-bit form in a random direction."""
    m, d, f = 12, 40, 72
    g = torch.Generator(device=DEV).manual_seed(3)
    x, wg, wu, dh = (torch.randn(*s, generator=g, device=DEV).half() for s in ((m, d), (f, d), (f, d), (m, f)))
    wg, wu = wg * 0.1, wu * 0.1
    h, gate, up, dg, du = (torch.empty(m, f, dtype=x.dtype, device=DEV) for _ in range(5))
    zdp.gated_product(x, wg, wu, h, act, gate=gate, up=up)
    dx, dwg, dwu = torch.empty_like(x), torch.empty(f, d, device=DEV), torch.empty(f, d, device=DEV)
    zdp.gated_product_backward(dh, x, wg, wu, gate, up, dg, du, ws, dx=dx, dw_gate=dwg, dw_up=dwu, act=act)
    e = [torch.randn(t.shape, generator=g, device=DEV, dtype=torch.float64) for t in (x, wg, wu)]
    step = 1e-6

    def value(s):
        X, G, V = (t.double() + s * step * q for t, q in zip((x, wg, wu), e))
        return ((act_of(X @ G.t(), act)[0] * (X @ V.t())) * dh.double()).sum()
    slope = (value(1) - value(-1)) / (2 * step)
    parts = [(t.double() * q) for t, q in zip((dx, dwg, dwu), e)]
    got = sum(p.sum() for p in parts)
    # gate, up, dgate, dup and dx are rounded to fp16, half a step of 2^-11 each; the sums of the magnitudes bound all five
    D, Z, V = dh.double(), gate.double(), up.double()
    A, DA = act_of(Z, act)
    size = (D * DA * V).abs() + (D * A).abs() + (D * V).abs() * Z.abs() * 1.2 + (D * DA * V).abs()
    reach = (size @ wg.double().abs() + size @ wu.double().abs()) * e[0].abs()
    reach2 = (size.t() @ x.double().abs()) * (e[1].abs() + e[2].abs())
    assert (got - slope).abs() <= 2.0 ** -11 * 2 * (reach.sum() + reach2.sum())


def test_no_rows_columns_or_contraction(ws):
    t = DTS["bf16"]

    def ones(*s):
        return torch.ones(*s, dtype=t, device=DEV)
    x, w = ones(5, 16), ones(9, 16)
    zdp.gated_product(x[:0], w, w, ones(0, 9), gate=ones(0, 9), up=ones(0, 9))
    zdp.gated_product(x, w[:0], w[:0], ones(5, 0))
    h = ones(5, 9)
    zdp.gated_product(ones(5, 0), ones(9, 0), ones(9, 0), h, "sigmoid")
    assert (h == 0).all()  # sigmoid(0) * 0
    e = ones(0, 9)
    dwg, dwu = torch.full((9, 16), 2.0, device=DEV), torch.full((9, 16), 3.0, device=DEV)
    zdp.gated_product_backward(e, x[:0], w, w, e, e, e.clone(), e.clone(), ws, dx=ones(0, 16), dw_gate=dwg, dw_up=dwu,
                               accumulate=True)
    assert (dwg == 2).all() and (dwu == 3).all()
    zdp.gated_product_backward(e, x[:0], w, w, e, e, e.clone(), e.clone(), ws, dw_gate=dwg, dw_up=dwu)
    assert (dwg == 0).all() and (dwu == 0).all()
    e, dx = ones(5, 0), ones(5, 16)
    zdp.gated_product_backward(e, x, w[:0], w[:0], e, e, e.clone(), e.clone(), ws, dx=dx)
    assert (dx == 0).all()


@pytest.mark.parametrize("m", [3, 200])
def test_one_row_s_trouble_stays_its_own(m, ws):
    """Infinities and NaN of a token, in its own outputs and in the weights' gradients, nowhere else."""
    g = torch.Generator(device=DEV).manual_seed(1)
    d, f = 136, 200
    x, w, dh, gate = (torch.randn(*s, generator=g, device=DEV).bfloat16() for s in ((m, d), (f, d), (m, f), (m, f)))
    x[1, 5] = float("inf")
    dh[1, 7] = float("nan")
    h = torch.empty_like(dh)
    zdp.gated_product(x, w, w, h)
    assert h[0].isfinite().all() and h[2:].isfinite().all() and not h[1].isfinite().any()
    dg, du, dx = torch.empty_like(dh), torch.empty_like(dh), torch.empty_like(x)
    dwg, dwu = torch.empty(f, d, device=DEV), torch.empty(f, d, device=DEV)
    zdp.gated_product_backward(dh, x, w, w, gate, gate, dg, du, ws, dx=dx, dw_gate=dwg, dw_up=dwu)
    assert dx[0].isfinite().all() and dx[2:].isfinite().all() and not dx[1].isfinite().any()
    bad = torch.zeros(f, d, dtype=torch.bool, device=DEV)
    bad[7] = True
    bad[:, 5] = True
    assert torch.equal(~dwg.isfinite(), bad) and torch.equal(~dwu.isfinite(), bad)


@pytest.mark.parametrize("m", [1, 2, 4])
@pytest.mark.parametrize("d", [9, 520, 1029])
def test_infinite_weights_of_single_tokens(m, d):
    """An infinite weight makes its own outputs infinite, with no NaN from the values that lanes past the end load again."""
    x = torch.ones(m, d, dtype=torch.bfloat16, device=DEV)
    wg, wu = torch.ones(20, d, dtype=torch.bfloat16, device=DEV), torch.ones(20, d, dtype=torch.bfloat16, device=DEV)
    wg[3, d - 1] = wg[4, d - 8] = wg[5, 0] = float("inf")
    h, g, u = (torch.empty(m, 20, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    zdp.gated_product(x, wg, wu, h, "relu", gate=g, up=u)
    want = torch.full((m, 20), float(d), device=DEV).bfloat16()
    assert torch.equal(u, want)
    want[:, 3:6] = float("inf")
    assert torch.equal(g, want) and h[:, 3:6].isinf().all() and h[:, 6:].isfinite().all()


def test_results_repeat(ws):
    """No atomics: the same call gives the same bits."""
    g = torch.Generator(device=DEV).manual_seed(5)
    m, d, f = 33, 512, 4096  # dx in splits
    x, w, dh, gate = (torch.randn(*s, generator=g, device=DEV).bfloat16() for s in ((m, d), (f, d), (m, f), (m, f)))
    dg, du = torch.empty_like(dh), torch.empty_like(dh)
    seen = []
    for _ in range(3):
        dx, a, b, h = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w), torch.empty_like(dh)
        zdp.gated_product(x, w, w, h)
        zdp.gated_product_backward(dh, x, w, w, gate, gate, dg, du, ws, dx=dx, dw_gate=a, dw_up=b)
        seen.append((h, dx, a, b))
    assert all(torch.equal(p, q) for s in seen[1:] for p, q in zip(seen[0], s))


def gates(dtype):
    """Finite gates over a type's whole range, both signs."""
    top = torch.finfo(dtype).max
    g = [0.0, 2.0 ** -14, 1.0, 13.3, 30.0, 63.0, 64.0, 65.0, 100.0, 1e4, top] + [1e10, 4e19, 6e19, 1e20, 1e30] * (top > 1e38)
    return torch.tensor([s * v for v in g for s in (1, -1)], dtype=torch.float64).to(dtype)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("act", ACTS)
def test_gradients_at_gates_of_any_size(act, dt, ws):
    """Finite gates give the formulas' finite gradients, however large (with dh = up = 1 dgate is the derivative itself
    and dup the activation). The errors up to |z| = 16 are those of test_backward; past it the smaller of sigmoid(z) and
    sigmoid(-z) is under 2^-23, so that what it is off by is lost beside the few u of the products."""
    dtype = DTS[dt]
    gate = gates(dtype).to(DEV).view(2, -1)
    m, f = gate.shape
    one, x, w = torch.ones_like(gate), torch.zeros(m, 8, dtype=dtype, device=DEV), torch.zeros(f, 8, dtype=dtype, device=DEV)
    dg, du = torch.empty_like(gate), torch.empty_like(gate)
    zdp.gated_product_backward(one, x, w, w, gate, one, dg, du, ws, act=act)
    Z = gate.double().cpu()
    A, _ = act_of(Z, act)
    DA = act_of(Z.clamp(-100, 100), act)[1]  # past that it has reached its limit, to e^-95
    low, eda = Z.abs() <= 16, act_error(Z, 1 + Z.abs() / 2)
    close(dg.cpu(), DA, torch.where(low, eda, 8 * U), "dgate")
    close(du.cpu(), A, torch.where(low, act_error(Z, A), 8 * U * (A.abs() + 1)) + 2 * U * A.abs(), "dup")


@pytest.mark.parametrize("act, lo, hi", [("silu", 60, 104), ("sigmoid", 60, 104), ("gelu", 10, 14), ("gelu_tanh", 8, 11)])
def test_small_values_of_far_gates(act, lo, hi, ws):
    """bf16 reaches down to 2^-133, and so do the activations and their derivatives at far gates. What they are off by,
    relative to the activation: its argument is rounded, |argument| u of the exponential at each rounding of it (silu one,
    gelu_tanh four; gelu's erfc, whose own error is 16 units at most, moves by z^2 of its argument's), and a few u more;
    and what falls below fp32's normal values is rounded at 2^-149."""
    g = torch.linspace(lo, hi, 353, dtype=torch.float64).bfloat16().unique()
    gate = torch.stack([-g, g]).to(DEV)
    m, f = gate.shape
    one, x, w = (torch.ones_like(gate), torch.zeros(m, 8, dtype=gate.dtype, device=DEV),
                 torch.zeros(f, 8, dtype=gate.dtype, device=DEV))
    dg, du = torch.empty_like(gate), torch.empty_like(gate)
    zdp.gated_product_backward(one, x, w, w, gate, one, dg, du, ws, act=act)
    Z = gate.double()
    z = Z.abs()
    A, DA = act_of(Z, act)
    rel = {"silu": 2 * z, "sigmoid": 2 * z, "gelu": 2 * z * z + 32, "gelu_tanh": 4 * (1.6 * z + 0.0714 * z ** 3)}[act] * U + 16 * U
    tail, step = act_of(-z, act)[0].abs(), 2.0 ** -149
    slope = 2 + 0.3 * z * z  # at least that of the argument, and |z|, by which gelu's density exceeds the tail
    ea = rel * tail + 8 * U * A.abs() + step * (1 + z)
    close(du, A, ea, "dup")
    close(dg, DA, rel * tail * slope + 8 * U * DA.abs() + step * (2 + (1 + z) * slope), "dgate")
    assert (tail > 2.0 ** -126).any() and (tail < 2.0 ** -126).any()
    # the forward pass: products of one term, by the kernel of single tokens and by tiles, among gates that are not far
    # and get the same bits without far ones beside them
    near = torch.linspace(-3, 3, f, device=DEV).bfloat16()
    for rows in (1, 5, 300):
        x1, wu = (torch.zeros(r, 8, dtype=gate.dtype, device=DEV) for r in (rows, f))
        x1[:, 0], wu[:, 0] = 1, 1

        def forward(gates):
            w = torch.zeros(f, 8, dtype=gate.dtype, device=DEV)
            w[:, 0] = gates
            h = torch.empty(rows, f, dtype=gate.dtype, device=DEV)
            zdp.gated_product(x1, w, wu, h, act)
            return h
        close(forward(gate[0]), A[:1].expand(rows, f), ea[:1], f"h of {rows} rows")
        odd = torch.arange(f, device=DEV) % 2 == 1
        mixed, alone = forward(torch.where(odd, gate[0], near)), forward(near)
        assert torch.equal(mixed[:, ~odd], alone[:, ~odd])


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("size", [(700, 1280, 5120), (153, 1344, 7920), (1410, 1584, 1504), (451, 776, 976), (4096, 1024, 1024),
                                  (2001, 400, 264)],
                         ids=str)
def test_backward_at_sizes_on_both_sides_of_the_shared_launch(size, dt, ws):
    """Shared launches with dx in splits and with large, middle and small tiles for dw alone; and sizes beside them that
    take two launches (the last two)."""
    test_both_products_of_the_backward_pass_in_one_launch(size, dt, ws)


@pytest.mark.parametrize("seed", [3, 4])
@pytest.mark.parametrize("act", ACTS)
def test_each_gradient_against_differences(act, seed, ws):
    """dx, dw_gate and dw_up one by one, in directions in which none can be missing (tests/_gated.py; its check is tested
    with wrong gradients in test_gated_differences.py)."""
    host = _gated.inputs(seed)
    x, wg, wu, dh = (t.to(DEV) for t in host)
    (m, d), f = x.shape, wg.shape[0]
    h, gate, up, dg, du = (torch.empty(m, f, dtype=x.dtype, device=DEV) for _ in range(5))
    zdp.gated_product(x, wg, wu, h, act, gate=gate, up=up)
    dx, dwg, dwu = torch.empty_like(x), torch.empty(f, d, device=DEV), torch.empty(f, d, device=DEV)
    zdp.gated_product_backward(dh, x, wg, wu, gate, up, dg, du, ws, dx=dx, dw_gate=dwg, dw_up=dwu, act=act)
    _gated.check_differences((dx, dwg, dwu), *host, act)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("size", [(2560, 520, 2048), (2561, 515, 2047), (300, 640, 1300)], ids=str)
def test_forward_in_large_and_middle_tiles(size, dt):
    """Random values through the tiles that test_forward's sizes do not reach."""
    test_forward(size, "silu", dt)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("size", [(4096, 2560, 520), (4099, 2563, 515), (700, 1280, 5120), (520, 2560, 2056), (300, 1288, 1400)],
                         ids=str)
def test_backward_in_large_and_middle_tiles_and_one_launch(size, dt, ws):
    """Random values through the tiles, and the shared launch of dx and dw, that test_backward's sizes do not reach."""
    test_backward(size, "gelu_tanh", dt, ws)


@pytest.mark.parametrize("cap", [1, 3])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("dt", DTS)
def test_backward_under_a_grid_cap(dt, pad, cap, ws):
    """The gate pass's loop over what its grid does not cover, over dense rows (one run) and strided ones, with dgate and
    dup of their own and in the place of gate and up: the bits of the free run."""
    m, d, f = 37, 40, 1601
    g, dtype = torch.Generator(device=DEV).manual_seed(cap), DTS[dt]
    x, wg, wu, dh, gate, up = (torch.randn(*s, generator=g, device=DEV).to(dtype)
                               for s in ((m, d), (f, d), (f, d), (m, f), (m, f), (m, f)))

    def run(own):
        a, b, c = (wide(t.clone(), pad) for t in (dh, gate, up))
        dg, du = (Blank(m, f, dtype, pad), Blank(m, f, dtype, pad)) if own else (None, None)
        dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
        p, q = (dg.t, du.t) if own else (b, c)
        zdp.gated_product_backward(a, x, wg, wu, b, c, p, q, ws, dx=dx, dw_gate=dwg, dw_up=dwu, act="silu")
        if own:
            dg.check()
            du.check()
        return [t.clone() for t in (p, q, dx, dwg, dwu)]
    free = run(True)
    zdp.set_grid_limit(cap)
    try:
        capped, over = run(True), run(False)
    finally:
        zdp.set_grid_limit(0)
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(free, capped, over))
