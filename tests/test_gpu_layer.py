"""Layer norm, dropout and their backward passes on the GPU against plain forms
in 64 bits (tests/_layer.py).

Tolerances. u = 2^-24, half a step of fp32. An fp32 sum of terms t_i by runs that
are then added is off by at most k u sum |t_i| (to first order), where k counts
the sums that a term passes through: a lane's own values, 6 steps over the wave,
the waves of a row. From that follows the error of each result, written at its
check; an output of a smaller type adds half a step of that type (HALF_STEP of
the value, or half its smallest subnormal)."""
import numpy as np
import pytest
import torch

import _layer
import zero_dp_partitioned_amd as zdp
from _gpu_helpers import DEV

pytestmark = pytest.mark.gpu

DTS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
U = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, err, what):
    """|got - want| within `err` (of the fp32 arithmetic) and the rounding to got's type."""
    h, tiny = HALF_STEP[got.dtype], TINY[got.dtype]
    got = f64(got)
    assert np.isfinite(got).all(), what
    bound = err * (1 + 2 * h) + h * np.abs(want) + tiny
    over = np.abs(got - want) - bound
    assert (over <= 0).all(), f"{what}: {(over > 0).sum()} off, worst by {over.max()} of {bound.flat[over.argmax()]}"


def depth(cols, kernel_elems=32):
    """Sums a value of a row passes through: at most 32 of its lane (a long row: its share of 1024 lanes), 6, 16 waves, and 2."""
    return max(kernel_elems, -(-cols // 1024) + 8) + 24


def make(rows, cols, dt, seed, pad=0):
    g = np.random.default_rng(seed)
    x = g.normal(size=(rows, cols)) * np.exp2(g.integers(-3, 4, (rows, 1))) + g.normal(size=(rows, 1))
    if cols > 8:
        x[:, ::7] *= 6
    return wide(x, dt, pad)


def wide(x, dt, pad=0):
    """x as a device tensor of the type; with `pad`, rows of a wider one that start off its beginning."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(DTS[dt])
    if not pad:
        return t.to(DEV)
    big = torch.full((x.shape[0], x.shape[1] + pad + 1), 7.0, dtype=t.dtype)
    big[:, 1:1 + x.shape[1]] = t
    return big.to(DEV)[:, 1:1 + x.shape[1]]


def blank(rows, cols, dt, pad=0):
    """An output full of a marker, and a check that nothing around it was written."""
    big = torch.full((rows, cols + 2 * pad), -77.0, dtype=DTS[dt], device=DEV)
    out = big[:, pad:pad + cols] if pad else big

    def untouched():
        if pad:
            assert (big[:, :pad] == -77).all() and (big[:, pad + cols:] == -77).all()
    return out, untouched


# widths at the ends of a slot (4 or 8 values), of a wave's slots and of each variant, and beyond all of them
WIDTHS = [1, 2, 3, 7, 8, 9, 63, 64, 65, 255, 511, 512, 513, 1000, 1023, 1025, 1600, 2047, 2049, 4095, 4096, 4097, 8191, 8192,
          8200, 16383, 16385, 33000]


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("cols", WIDTHS)
def test_norm(cols, dt):
    rows, eps, pad = 5, 1e-5, 0 if cols % 3 else 3
    x = make(rows, cols, dt, cols, pad)
    w32 = cols % 2 == 0  # fp32 weights beside 16-bit rows
    w, b = (make(1, cols, "f32" if w32 else dt, cols + k)[0] for k in (1, 2))
    bias = None if cols % 5 == 0 else b
    y, untouched = blank(rows, cols, dt, pad)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    zdp.layer_norm(x, w, bias, y, eps, mean=mean, rstd=rstd)
    X, W, B = f64(x), f64(w), 0.0 if bias is None else f64(b)
    Y, M, R = _layer.norm(X, W, B, eps)
    k = depth(cols) + 3
    dmean = (k * U * np.abs(X).mean(1) + U * np.abs(M))[:, None]  # the sum, its division and rounding
    close(mean, M, dmean[:, 0], "mean")
    d = np.abs(X - M[:, None])
    # sum of squares of values that are each off by dmean + U d: relative to var, 2 sqrt(mean of those squares / var)
    shift = np.sqrt(((dmean + U * d) ** 2).mean(1, keepdims=True)) * R[:, None]
    drstd = R[:, None] * ((k / 2 + 4) * U + shift + shift ** 2)
    close(rstd, R, drstd[:, 0], "rstd")
    err = (dmean + 2 * U * d) * R[:, None] + d * drstd
    close(y, Y, np.abs(W) * err + 4 * U * (np.abs(W) * d * R[:, None] + np.abs(B)), "y")
    untouched()
    y2 = torch.empty_like(x)
    zdp.layer_norm(x, w, bias, y2, eps)  # without the statistics: the same values
    assert torch.equal(y2, y)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows, cols", [(3, c) for c in WIDTHS] + [(1, 1600), (2, 4096), (513, 64), (1001, 1600), (4099, 512),
                                                                 (2500, 2048), (1030, 4100), (700, 9000), (150, 17000)])
def test_norm_backward(rows, cols, dt):
    pad = 0 if cols % 3 else 3
    x, dy = make(rows, cols, dt, cols + rows, pad), make(rows, cols, dt, cols + rows + 1, pad)
    res = make(rows, cols, dt, cols + rows + 2) if rows % 2 else None
    w = make(1, cols, "f32" if cols % 2 == 0 else dt, cols + 3)[0]
    X, D, W = f64(x), f64(dy), f64(w)
    _, M, R = _layer.norm(X, W, None, 1e-5)
    mean, rstd = (torch.from_numpy(v.astype(np.float32)).to(DEV) for v in (M, R))
    M, R = f64(mean)[:, None], f64(rstd)[:, None]
    dx, untouched = blank(rows, cols, dt, pad)
    gdt = ("f32", dt)[cols % 2]
    dw, db = (torch.full((cols,), np.nan, dtype=DTS[gdt], device=DEV) for _ in range(2))
    ws = zdp.new_workspace(1)
    ws.fill_(0xFF)  # NaN patterns: nothing of it may be read before it is written
    zdp.layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, workspace=ws, dresidual=res)
    P = None if res is None else f64(res)
    DX, DW, DB = _layer.norm_grad(D, X, W, M[:, 0], R[:, 0], P)
    xhat, v = np.abs((X - M) * R), np.abs(D * W)
    k = depth(cols)
    c1, c2 = v.mean(1, keepdims=True), (v * xhat).mean(1, keepdims=True)
    # v is off by u, xhat by 2u, their product by 4u, the sums by k u and the division by 2u; then three operations
    err = R * ((k + 4) * U * c1 + (k + 8) * U * xhat * c2 + 6 * U * (v + c1 + xhat * c2))
    close(dx, DX, err + 2 * U * np.abs(DX) + (0 if P is None else 2 * U * np.abs(P)), "dx")
    untouched()
    # a value passes through its block's rows, 8 groups, the blocks of a run (16), 32 runs; long rows: runs of 64 or more
    k = rows / 64 + 8 + 16 + 32 + 70
    close(dw, DW, (k + 4) * U * (np.abs(D) * xhat).sum(0), "dweight")
    close(db, DB, k * U * np.abs(D).sum(0), "dbias")
    # each alone, and added to what is there
    dw2, db2, dx2 = dw.clone(), db.clone(), torch.empty_like(dx)
    zdp.layer_norm_backward(dy, x, w, mean, rstd, dx2, dw2, None, workspace=ws, dresidual=res, accumulate=True)
    zdp.layer_norm_backward(dy, x, w, mean, rstd, dx2, None, db2, workspace=ws, dresidual=res, accumulate=True)
    assert torch.equal(dx2, dx)
    close(dw2, DW + f64(dw), (k + 4) * U * (np.abs(D) * xhat).sum(0) + 2 * U * np.abs(f64(dw)), "dweight added")
    close(db2, DB + f64(db), k * U * np.abs(D).sum(0) + 2 * U * np.abs(f64(db)), "dbias added")
    dx3 = torch.empty_like(dx)
    zdp.layer_norm_backward(dy, x, w, mean, rstd, dx3, dresidual=res)  # no column sums, no workspace
    assert torch.equal(dx3, dx)


@pytest.mark.parametrize("cols", [5, 96, 1601, 9000])
def test_norm_gradients_against_differences(cols):
    """The formula's gradient is the slope of the forward pass: differences of its 64-bit form, in a random direction."""
    rows, g = 4, np.random.default_rng(cols)
    x, w, b, dy = (torch.from_numpy(g.normal(size=s)).float().to(DEV) for s in ((rows, cols), cols, cols, (rows, cols)))
    y, dx, mean, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    zdp.layer_norm(x, w, b, y, 1e-5, mean=mean, rstd=rstd)
    zdp.layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, workspace=zdp.new_workspace(1))
    X, W, B, D = f64(x), f64(w), f64(b), f64(dy)
    h, (ex, ew, eb) = 1e-5, (g.normal(size=s) for s in ((rows, cols), cols, cols))
    up, down = (_layer.norm(X + s * h * ex, W + s * h * ew, B + s * h * eb, 1e-5)[0] for s in (1, -1))
    slope = ((up - down) / (2 * h) * D).sum()
    got = (f64(dx) * ex).sum() + (f64(dw) * ew).sum() + (f64(db) * eb).sum()
    # differences: h^2 times third derivatives of order one; gradients: fp32 sums and statistics, k u of their terms
    terms = np.abs(f64(dx) * ex).sum() + np.abs(f64(dw) * ew).sum() + np.abs(f64(db) * eb).sum()
    assert abs(got - slope) <= 1e-8 * terms + 200 * U * terms


def test_norm_rows_without_spread_and_without_numbers():
    x = torch.zeros(6, 40, device=DEV)
    x[1] = 3.25
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    x[4] = torch.arange(40.0)
    x[5] = 1e20  # squares past fp32's range never form: the row has no spread
    w, b = torch.full((40,), 2.0, device=DEV), torch.full((40,), 0.5, device=DEV)
    y, mean, rstd = torch.empty_like(x), torch.empty(6, device=DEV), torch.empty(6, device=DEV)
    zdp.layer_norm(x, w, b, y, 1e-5, mean=mean, rstd=rstd)
    assert (y[0] == 0.5).all() and (y[1] == 0.5).all() and (y[5] == 0.5).all()
    assert y[2].isnan().all() and y[3].isnan().all()  # a row's own trouble ...
    assert y[4].isfinite().all()  # ... and nobody else's
    zdp.layer_norm(x[:1], w, b, y[:1], 0.0)
    assert y[0].isnan().all()  # 0 * 1 / 0, as the formula says


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [7, 13, 1001, 1600])
def test_an_infinite_gradient_at_a_row_s_end(cols, dt):
    """dy infinite in the last column, in a slot that is moved back and so loads values that another one has: with
    xhat = 1 in the row its two means are infinite, as the formula has them, and not NaN; no other row notices."""
    x, dy, w = make(3, cols, dt, 1), make(3, cols, dt, 2), torch.ones(cols, dtype=DTS[dt], device=DEV)
    mean, rstd = torch.zeros(3, device=DEV), torch.ones(3, device=DEV)
    x[1] = 1.0
    dy[1] = 1.0
    dy[1, cols - 1] = float("inf")
    dx, dw, db = torch.empty_like(x), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    zdp.layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, workspace=zdp.new_workspace(1))
    # mean(v) = mean(v xhat) = inf: 1 - inf - inf, and in the last column inf - inf
    assert (dx[1, :cols - 1] == -float("inf")).all() and dx[1, cols - 1].isnan()
    assert dx[0].isfinite().all() and dx[2].isfinite().all()
    assert dw[:cols - 1].isfinite().all() and db[cols - 1] == float("inf")


@pytest.mark.parametrize("eps", [1e-45, 1e-46, 1e-300, 5e-324])
def test_norm_with_an_eps_below_fp32_s_values(eps):
    """It still keeps rows without spread from NaN, and adds nothing to the others."""
    x = torch.zeros(4, 100, device=DEV)
    x[1] = 3.25
    x[2:] = torch.randn(2, 100, device=DEV)
    w, b = torch.full((100,), 2.0, device=DEV), torch.full((100,), 0.5, device=DEV)
    y, plain = torch.empty_like(x), torch.empty_like(x)
    zdp.layer_norm(x, w, b, y, eps)
    zdp.layer_norm(x, w, b, plain, 0.0)
    assert (y[:2] == 0.5).all() and torch.equal(y[2:], plain[2:]) and plain[:2].isnan().all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [3, 5, 64, 1000, 1600, 4096, 9000, 33000])
def test_norm_of_rows_whose_sums_pass_fp32(cols, dt):
    """Rows whose squares, or whose values' sums, pass fp32's range have their statistics like any others. The bounds are
    test_norm's: the sums are then those of values times a power of two."""
    g = np.random.default_rng(cols)
    n = g.normal(size=(8, cols))
    x = np.stack([n[0], n[1] * 1e20, n[2] * 1e30, np.abs(n[3]) * 3e37, 1e38 * (1 + 0.01 * n[4].clip(-5, 5)),
                  1.2e38 * np.sign(n[5]), n[6] * 1e25 + 1e27, n[7]])
    x = wide(x, dt)
    w, b = (make(1, cols, "f32", cols + k)[0] for k in (1, 2))
    y, mean, rstd = torch.empty_like(x), torch.empty(8, device=DEV), torch.empty(8, device=DEV)
    zdp.layer_norm(x, w, b, y, 1e-5, mean=mean, rstd=rstd)
    X, W, B = f64(x), f64(w), f64(b)
    Y, M, R = _layer.norm(X, W, B, 1e-5)
    k = depth(cols) + 3
    dmean = (k * U * np.abs(X).mean(1) + U * np.abs(M))[:, None]
    close(mean, M, dmean[:, 0], "mean")
    d = np.abs(X - M[:, None])
    shift = np.sqrt(((dmean + U * d) ** 2).mean(1, keepdims=True)) * R[:, None]
    drstd = R[:, None] * ((k / 2 + 4) * U + shift + shift ** 2)
    close(rstd, R, drstd[:, 0], "rstd")
    err = (dmean + 2 * U * d) * R[:, None] + d * drstd
    close(y, Y, np.abs(W) * err + 4 * U * (np.abs(W) * d * R[:, None] + np.abs(B)), "y")
    # the backward pass takes such statistics
    dy, dx = make(8, cols, dt, cols + 5), torch.empty_like(x)
    zdp.layer_norm_backward(dy, x, w, mean, rstd, dx)
    M, R, D = f64(mean)[:, None], f64(rstd)[:, None], f64(dy)
    DX = _layer.norm_grad(D, X, W, M[:, 0], R[:, 0])[0]
    xhat, v = np.abs((X - M) * R), np.abs(D * W)
    c1, c2 = v.mean(1, keepdims=True), (v * xhat).mean(1, keepdims=True)
    err = R * ((k + 4) * U * c1 + (k + 8) * U * xhat * c2 + 6 * U * (v + c1 + xhat * c2))
    close(dx, DX, err + 2 * U * np.abs(DX), "dx")


@pytest.mark.parametrize("cols", [5, 100, 1600, 33000])
def test_norm_rows_that_fp32_cannot_hold_are_nan(cols):
    """Infinities, NaN, and distances from the mean past fp32's range; the rows beside them do not notice."""
    x = torch.randn(9, cols, device=DEV)
    x[1, 2], x[3, 2], x[5, 2] = float("inf"), float("nan"), -float("inf")
    x[7] = -3e38
    x[7, 0] = 3e38
    w, y, mean, rstd = torch.ones(cols, device=DEV), torch.empty_like(x), torch.empty(9, device=DEV), torch.empty(9, device=DEV)
    zdp.layer_norm(x, w, w, y, mean=mean, rstd=rstd)
    assert y[1::2].isnan().all() and y[::2].isfinite().all() and rstd[1::2].isnan().all()


def test_norm_of_no_rows():
    w = torch.ones(16, device=DEV)
    x, ws = torch.empty(0, 16, device=DEV), zdp.new_workspace(1)
    none = torch.empty(0, device=DEV)
    zdp.layer_norm(x, w, w, x.clone(), mean=none, rstd=none)
    dw, db = torch.full((16,), 3.0, device=DEV), torch.full((16,), 4.0, device=DEV)
    zdp.layer_norm_backward(x, x, w, none, none, x.clone(), dw, db, workspace=ws, accumulate=True)
    assert (dw == 3).all() and (db == 4).all()
    zdp.layer_norm_backward(x, x, w, none, none, x.clone(), dw, db, workspace=ws)
    assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("cap", [1, 3])
@pytest.mark.parametrize("cols", [100, 1600, 5000, 40000])
def test_norm_under_a_grid_cap(cap, cols):
    """Every loop over rows that a full grid leaves out."""
    rows = 37
    x, dy, w = make(rows, cols, "bf16", 1), make(rows, cols, "bf16", 2), make(1, cols, "bf16", 3)[0]
    ws = zdp.new_workspace(1)

    def both():
        y, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
        m, r = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        zdp.layer_norm(x, w, w, y, mean=m, rstd=r)
        zdp.layer_norm_backward(dy, x, w, m, r, dx, dw, db, workspace=ws)
        return y, m, r, dx, dw, db
    free = both()
    zdp.set_grid_limit(cap)
    try:
        capped = both()
    finally:
        zdp.set_grid_limit(0)
    assert all(torch.equal(a, b) for a, b in zip(free[:4], capped[:4]))
    for a, b, t in zip(free[4:], capped[4:], (f64(dy) * (f64(x) - f64(free[1])[:, None]) * f64(free[2])[:, None], f64(dy))):
        assert (np.abs(f64(a) - f64(b)) <= 2 * (rows + 60) * U * np.abs(t).sum(0)).all()


# --------------------------------------------------------------------------
# dropout
# --------------------------------------------------------------------------

SEED, OFFSET = 0x0123456789ABCDEF, 0xFEDCBA9876543210


def dropped(X, P, p, mask):
    y = np.where(mask, X / (1 - p), 0.0) + (0 if P is None else P)
    return y, 3 * U * np.abs(np.where(mask, X / (1 - p), 0.0)) + U * np.abs(y)  # the scale, the product, the sum


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("first", [0, 1, 2, 3, 5, 2 ** 34 + 7, 2 ** 62 + 2])
@pytest.mark.parametrize("shape", [(1, 1), (1, 3), (1, 4), (1, 9), (5, 1), (7, 8), (9, 13), (3, 4099), (1, 100003)])
def test_dropout(shape, first, dt):
    rows, cols = shape
    p = (0.1, 0.5, 0.9)[(cols + first) % 3]
    for pad in (0, 3):
        x = make(rows, cols, dt, 5, pad)
        x[x == 0] = 1
        res = make(rows, cols, dt, 6, pad) if first % 2 else None
        y, untouched = blank(rows, cols, dt, pad)
        zdp.dropout(x, y, p, SEED, OFFSET, residual=res, first=first)
        mask = _layer.kept(rows * cols, p, SEED, OFFSET, first).reshape(rows, cols)
        P = None if res is None else f64(res)
        Y, err = dropped(f64(x), P, p, mask)
        close(y, Y, err, f"pad {pad}")
        if res is None:
            assert ((f64(y) != 0) == mask).all()
        untouched()


def test_dropout_rates():
    """The share that is kept, within five deviations of its expectation; other seeds and offsets draw other masks."""
    n = 1 << 20
    x = torch.ones(n, device=DEV)
    seen = []
    for p in (0.0, 0.1, 0.5, 0.999):
        for seed, offset in ((1, 0), (2, 0), (1, 1)):
            y = torch.empty_like(x)
            zdp.dropout(x, y, p, seed, offset)
            k = int((y != 0).sum())
            assert abs(k - n * (1 - p)) <= 5 * np.sqrt(n * p * (1 - p)) + n * 2.0 ** -32
            if p == 0.5:
                seen.append(y)
    assert all(not torch.equal(a, b) for i, a in enumerate(seen) for b in seen[:i])


def test_dropout_of_parts_is_the_whole():
    x = make(1, 50_001, "bf16", 3)[0]
    whole = torch.empty_like(x)
    zdp.dropout(x, whole, 0.3, 99, 4)
    parts = torch.empty_like(x)
    for a, b in ((0, 1), (1, 2), (2, 777), (777, 778), (778, 20_003), (20_003, 50_001)):
        zdp.dropout(x[a:b], parts[a:b], 0.3, 99, 4, first=a)
    assert torch.equal(whole, parts)
    rows = torch.empty(3, 16667, dtype=x.dtype, device=DEV)
    zdp.dropout(x.view(3, 16667), rows, 0.3, 99, 4)
    assert torch.equal(rows.view(-1), whole)
    cube = torch.empty(3, 7, 2381, dtype=x.dtype, device=DEV)
    zdp.dropout(x.view(3, 7, 2381), cube, 0.3, 99, 4)
    assert torch.equal(cube.view(-1), whole)


@pytest.mark.parametrize("dt", DTS)
def test_dropout_in_place_and_backward(dt):
    """y over x or over the residual; the same call on dy multiplies by the same mask."""
    x, res, dy = (make(11, 333, dt, k) for k in (1, 2, 3))
    want = torch.empty_like(x)
    zdp.dropout(x, want, 0.4, 7, 8, residual=res)
    a, b = x.clone(), res.clone()
    zdp.dropout(a, a, 0.4, 7, 8, residual=res)
    zdp.dropout(x, b, 0.4, 7, 8, residual=b)
    assert torch.equal(a, want) and torch.equal(b, want)
    dx = torch.empty_like(dy)
    zdp.dropout(dy, dx, 0.4, 7, 8)
    mask = _layer.kept(11 * 333, 0.4, 7, 8).reshape(11, 333)
    Y, err = dropped(f64(dy), None, 0.4, mask)
    close(dx, Y, err, "dx")


def test_dropout_of_infinities_and_nan():
    """A dropped value is 0 whatever it was; a kept one keeps its trouble."""
    x = torch.full((4096,), float("inf"), device=DEV)
    x[1::2] = float("nan")
    y = torch.empty_like(x)
    zdp.dropout(x, y, 0.5, 3)
    mask = torch.from_numpy(_layer.kept(4096, 0.5, 3)).to(DEV)
    assert (y[~mask] == 0).all() and not y[mask].isfinite().any()


def test_dropout_counter_is_read_when_the_kernel_runs():
    """In a captured graph that advances its counter every replay draws its own mask, eager work in between."""
    x = make(64, 320, "bf16", 9)
    y, counter = torch.empty_like(x), torch.zeros(1, dtype=torch.int64, device=DEV)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        zdp.dropout(x, y, 0.2, 11, 100, counter=counter)  # first use outside the capture
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        zdp.dropout(x, y, 0.2, 11, 100, counter=counter)
        counter += 1
    for k in range(4):
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(x)
        zdp.dropout(x, want, 0.2, 11, 100 + k)
        assert torch.equal(y, want)
    counter.fill_(-101)  # the sum wraps: 2^64 - 1
    graph.replay()
    zdp.dropout(x, want, 0.2, 11, -1)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("cap", [1, 2])
def test_dropout_under_a_grid_cap(cap):
    x = make(37, 1601, "f16", 2)
    free, capped = torch.empty_like(x), torch.empty_like(x)
    zdp.dropout(x, free, 0.5, 1)
    zdp.set_grid_limit(cap)
    try:
        zdp.dropout(x, capped, 0.5, 1)
    finally:
        zdp.set_grid_limit(0)
    assert torch.equal(free, capped)
