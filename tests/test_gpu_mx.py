"""The microscaled 4-bit calls on the GPU against plain forms in 64 bits
(tests/_mx.py).

Codes and scales are compared for equality, and so are widened values: they are
exact operations rounded once. Averages perform the fp32 operations of the
16-bit averaging pass, so they are compared bit for bit with those operations
in numpy. A product's terms are exact and its sum has K terms in fp32, so with
any order and with truncation its error is at most K * 2^-23 * sum |a b|; the
output's rounding adds half a step of its type. The rounding of a sum grows with
the root of K in practice: the relative 2-norm of the error is held to 1e-6 for
fp32 outputs as well."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import _mx
import zero_dp_partitioned_amd as zdp
from _gpu_helpers import DEV, assert_bits_equal, down32, up32

pytestmark = pytest.mark.gpu

DTS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}  # the smallest subnormal


def _up(a):
    return torch.from_numpy(np.ascontiguousarray(a).copy()).to(DEV)


def _down(t):
    return t.detach().cpu().numpy().copy()


def _f64(t):
    return t.detach().double().cpu().numpy()


def _inputs(rows, cols, dt, seed, rare=True):
    """Values over many exponents, with ties, zero blocks and, if `rare`, the
    edges of the type; as a device tensor of the type."""
    g = np.random.default_rng(seed)
    x = g.normal(size=(rows, cols)) * np.exp2(g.integers(-9, 6, (rows, 1)))
    flat = x.reshape(-1)
    n = flat.size
    k = g.integers(0, n, max(1, n // 50))
    flat[k] = g.integers(-64, 65, k.size) / 8.0  # ties and exact codes
    if rows > 2:
        x[1] = 0.0
    if rare:
        for value in (np.inf, -np.inf, np.nan, float(torch.finfo(DTS[dt]).max), float(torch.finfo(DTS[dt]).tiny),
                      TINY[dt], -0.0):
            flat[g.integers(0, n)] = value
    return torch.from_numpy(x).to(DTS[dt]).to(DEV)


def _mx_dev(rows, cols, ld=None, fill=0xA5):
    """Outputs of `ld` blocks a row in buffers filled with a mark."""
    kb = _mx.blocks(cols)
    ld = kb if ld is None else ld
    c = torch.full((max(rows, 1), 16 * ld), fill, dtype=torch.uint8, device=DEV)
    s = torch.full((max(rows, 1), ld), fill, dtype=torch.uint8, device=DEV)
    return c, s, c[:rows, :16 * kb], s[:rows, :kb]


def _check_mx(got_c, got_s, want, what):
    np.testing.assert_array_equal(_down(got_s), want[1], err_msg=f"{what}: scales")
    np.testing.assert_array_equal(_down(got_c), want[0], err_msg=f"{what}: codes")


SHAPES = [(1, 1), (1, 31), (1, 32), (1, 33), (1, 4096), (1, 5003), (3, 64), (5, 97), (33, 8), (64, 128), (127, 129),
          (130, 260), (257, 1600), (1001, 333), (32, 1), (1, 128), (2050, 70)]


@pytest.mark.parametrize("dt", list(DTS))
@pytest.mark.parametrize("rows, cols", SHAPES)
def test_quantize(rows, cols, dt):
    x = _inputs(rows, cols, dt, rows * 7 + cols)
    want, want_t = _mx.quantize(_f64(x)), _mx.quantize(_f64(x).T)
    c, s = zdp.mx_empty(rows, cols)
    ct, st = zdp.mx_empty(cols, rows)
    zdp.mx_quantize(x, c, s)
    _check_mx(c, s, want, "rows")
    zdp.mx_quantize(x, codes_t=ct, scales_t=st)
    _check_mx(ct, st, want_t, "columns")
    for t in (c, s, ct, st):
        t.fill_(0x5A)
    zdp.mx_quantize(x, c, s, ct, st)
    _check_mx(c, s, want, "both, rows")
    _check_mx(ct, st, want_t, "both, columns")


@pytest.mark.parametrize("dt", list(DTS))
@pytest.mark.parametrize("rows, cols, off, ld", [(5, 97, 1, 6), (130, 200, 3, 9), (64, 128, 4, 4), (1, 700, 5, 30),
                                                 (300, 33, 7, 2), (129, 256, 2, 8)])
def test_quantize_strided(rows, cols, off, ld, dt):
    """A column slice at an odd offset; outputs inside wider ones, whose other blocks stay as they were."""
    base = _inputs(rows, cols + off + 6, dt, 5, rare=False)
    x = base[:, off:off + cols]
    tld = _mx.blocks(rows) + 3
    c_all, s_all, c, s = _mx_dev(rows, cols, ld)
    ct_all, st_all, ct, st = _mx_dev(cols, rows, tld)
    zdp.mx_quantize(x, c, s, ct, st)
    _check_mx(c, s, _mx.quantize(_f64(x)), "rows")
    _check_mx(ct, st, _mx.quantize(_f64(x).T), "columns")
    kb, kt = _mx.blocks(cols), _mx.blocks(rows)
    for t, used in ((c_all, 16 * kb), (s_all, kb), (ct_all, 16 * kt), (st_all, kt)):
        assert (t[:, used:] == 0xA5).all(), "blocks past a row's last one were written"


def _ordinary(rows, cols, dt, seed, special=None):
    """Values without zero blocks, some of them ties; `special` stands in the first value only."""
    g = np.random.default_rng(seed)
    x = g.normal(size=(rows, cols)) * np.exp2(g.integers(-9, 6, (rows, 1)))
    x.reshape(-1)[g.integers(0, x.size, x.size // 8)] = g.choice([-2.5, 0.25, 0.75, 1.75, 3.5, -5.0])
    if special is not None:
        x[0, 0] = special
    return torch.from_numpy(x).to(DTS[dt])


def _codes_where(want, nan):
    """The expected blocks are NaN blocks where `nan` says so, and every other one, a partial one too, has codes."""
    codes, scales = want
    np.testing.assert_array_equal(scales == 255, nan)
    np.testing.assert_array_equal((codes.reshape(*scales.shape, 16) & 0x77).any(-1), ~nan)


FILLED = SHAPES + [(1, 2), (1, 7), (1, 63), (1, 65), (31, 1), (33, 1), (31, 33), (65, 2)]
FILLED = [(r, c, None) for r, c in FILLED] + [(r, c, v) for r, c in FILLED if r > 32 < c for v in (np.inf, np.nan)]


@pytest.mark.parametrize("dt", list(DTS))
@pytest.mark.parametrize("rows, cols, special", FILLED)
def test_quantize_with_codes_in_every_block(rows, cols, special, dt):
    """Ragged sizes with something to get wrong in each block: one special value at most, where there are more blocks."""
    x = _ordinary(rows, cols, dt, rows * 5 + cols, special)
    want, want_t = _mx.quantize(x.double().numpy()), _mx.quantize(x.double().numpy().T)
    nan = [np.zeros(w[1].shape, bool) for w in (want, want_t)]
    if special is not None:
        nan[0][0, 0] = nan[1][0, 0] = True
    _codes_where(want, nan[0])
    _codes_where(want_t, nan[1])
    x = x.to(DEV)
    c, s = zdp.mx_empty(rows, cols)
    zdp.mx_quantize(x, c, s)
    _check_mx(c, s, want, "rows")
    ct, st = zdp.mx_empty(cols, rows)
    zdp.mx_quantize(x, codes_t=ct, scales_t=st)
    _check_mx(ct, st, want_t, "columns")
    for t in (c, s, ct, st):
        t.fill_(0x5A)
    zdp.mx_quantize(x, c, s, ct, st)
    _check_mx(c, s, want, "both, rows")
    _check_mx(ct, st, want_t, "both, columns")


@pytest.mark.parametrize("n", [1, 2, 3, 5, 7, 31, 32, 33, 34, 63, 64, 65, 1023, 1025, 4095, 4097])
@pytest.mark.parametrize("shift", [0, 1, 2, 3])
def test_cast_writeback_with_codes_in_every_block(n, shift):
    """Short slices from masters at every 4-byte alignment, written and widened again."""
    x = _ordinary(1, n + shift, "f32", n)[0, shift:]
    want = _mx.quantize(x.double().numpy()[None])
    _codes_where(want, np.zeros(want[1].shape, bool))
    b0, b = 2, _mx.blocks(n)
    c = torch.full((16 * (b0 + b),), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full((b0 + b,), 0xA5, dtype=torch.uint8, device=DEV)
    base = torch.full((n + 8,), float("nan"), device=DEV)  # what stands around the master is not read into it
    master = base[shift:shift + n]
    master.copy_(x)
    zdp.mx_cast_writeback(master, c, s, 32 * b0)
    np.testing.assert_array_equal(_down(s)[b0:], want[1][0])
    np.testing.assert_array_equal(_down(c)[16 * b0:], want[0][0])
    assert (c[:16 * b0] == 0xA5).all() and (s[:b0] == 0xA5).all()
    for dt in DTS:
        out = torch.empty(n, dtype=DTS[dt], device=DEV)
        zdp.mx_dequantize(c, s, out, offset=32 * b0)
        v = torch.from_numpy(_mx.decode(*want)[0, :n]).to(DTS[dt])
        assert torch.equal(out.cpu(), v) and torch.isfinite(v).all()


# Scale bytes that the largest magnitudes of each type reach, subnormal values included (byte 0 also stands for all below).
BYTES = {"f32": range(0, 253), "f16": range(101, 139), "bf16": range(0, 253)}


def _every_scale(dt):
    """[rows, 64] values of the type: for every scale byte eight rows whose blocks' largest magnitude is 4 to 8 times the
    scale, in sixteenths of it (ties and saturation among them); rows below byte 0; and rows of the smallest subnormal."""
    g = np.random.default_rng(21)
    e = np.repeat(np.arange(BYTES[dt][0] - (24 if BYTES[dt][0] == 0 else 0), BYTES[dt][-1] + 1), 8) - 127
    x = g.integers(-127, 128, (e.size, 64)) / 16.0
    for block in (0, 32):
        x[np.arange(e.size), block + g.integers(0, 32, e.size)] = g.integers(64, 128, e.size) / 16.0
    x = np.concatenate([np.ldexp(x, e[:, None]), g.choice([-TINY[dt], 0.0, TINY[dt]], (4, 64))])
    return torch.from_numpy(x).to(DTS[dt])


@pytest.mark.parametrize("dt", list(DTS))
def test_quantize_under_every_scale(dt):
    """Every scale byte with codes of every magnitude, from subnormal inputs to the type's largest, in each kernel."""
    x = _every_scale(dt)
    assert torch.isfinite(x).all()
    want = _mx.quantize(x.double().numpy())
    assert set(want[1].reshape(-1)) == set(BYTES[dt])
    for byte in BYTES[dt][4 if dt == "f16" else 0:]:  # fp16's smallest values are too coarse for every code
        codes = want[0].reshape(-1, 16)[want[1].reshape(-1) == byte]
        assert len(set(np.concatenate([codes & 15, codes >> 4]).reshape(-1)) - {0, 8}) == 14, f"codes at byte {byte}"
    rows = x.shape[0]
    for buf in (x.to(DEV), torch.cat([x, x], 1).to(DEV)[:, :64]):  # dense; rows inside a wider array
        c, s = zdp.mx_empty(rows, 64)
        zdp.mx_quantize(buf, c, s)
        _check_mx(c, s, want, "rows")
    for both in (False, True):
        ct, st = zdp.mx_empty(rows, 64)
        other = zdp.mx_empty(64, rows) if both else (None, None)
        zdp.mx_quantize(x.t().contiguous().to(DEV), *other, ct, st)
        _check_mx(ct, st, want, "columns")
    if dt == "f32":
        fc, fs = (t.view(-1) for t in zdp.mx_empty(1, x.numel()))
        zdp.mx_cast_writeback(x.view(-1).to(DEV), fc, fs)
        _check_mx(fc, fs, (want[0].reshape(-1), want[1].reshape(-1)), "flat")


@pytest.mark.parametrize("n", [1, 7, 31, 32, 33, 4095, 8192, 8193, 196_899, 1_048_577])
@pytest.mark.parametrize("shift", [0, 1])
def test_cast_writeback(n, shift):
    """A slice of a flat vector, from masters at any 4-byte alignment; what is around it stays."""
    x = _inputs(1, n + shift, "f32", n)[0, shift:]
    b0, b = 3, _mx.blocks(n)
    c = torch.full((16 * (b0 + b),), 0xA5, dtype=torch.uint8, device=DEV)
    s = torch.full((b0 + b,), 0xA5, dtype=torch.uint8, device=DEV)
    zdp.mx_cast_writeback(x, c, s, 32 * b0)
    want = _mx.quantize(_f64(x)[None])
    np.testing.assert_array_equal(_down(s)[b0:], want[1][0])
    np.testing.assert_array_equal(_down(c)[16 * b0:], want[0][0])
    assert (c[:16 * b0] == 0xA5).all() and (s[:b0] == 0xA5).all()
    for dt in DTS:
        out = torch.empty(n, dtype=DTS[dt], device=DEV)
        zdp.mx_dequantize(c, s, out, offset=32 * b0)
        with np.errstate(over="ignore"):
            v = torch.from_numpy(_mx.decode(*want)[0, :n]).float().to(DTS[dt])
        torch.testing.assert_close(out.cpu(), v, rtol=0, atol=0, equal_nan=True)


def test_offsets_past_32_bits():
    """A slice that begins past element 2^32, and codes past byte 2^32."""
    n, offset = 70_001, 2 ** 33 + 32 * 5
    b = offset // 32 + _mx.blocks(n)
    c, s = torch.empty(16 * b, dtype=torch.uint8, device=DEV), torch.empty(b, dtype=torch.uint8, device=DEV)
    c[:1 << 20] = 0xA5
    c[-16 * _mx.blocks(n) - 4096:] = 0xA5
    x = _inputs(1, n, "f32", 3)[0]
    zdp.mx_cast_writeback(x, c, s, offset)
    want = _mx.quantize(_f64(x)[None])
    np.testing.assert_array_equal(_down(c[offset // 2:]), want[0][0])
    np.testing.assert_array_equal(_down(s[offset // 32:]), want[1][0])
    assert (c[:1 << 20] == 0xA5).all() and (c[offset // 2 - 4096:offset // 2] == 0xA5).all()
    out = torch.empty(n, device=DEV)
    zdp.mx_dequantize(c, s, out, offset=offset)
    np.testing.assert_array_equal(_f64(out), _mx.decode(*want)[0, :n])


@pytest.mark.parametrize("dt", list(DTS))
def test_dequantize_every_code_under_every_scale(dt):
    """All 256 pairs of codes under all 256 scale bytes."""
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(1, 16, 16), (256, 1, 1)).reshape(256, 256)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    out = torch.empty(256, 512, dtype=DTS[dt], device=DEV)
    zdp.mx_dequantize(_up(codes), _up(scales), out)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(_mx.decode(codes, scales)).float().to(DTS[dt])  # fp32 holds the values exactly
    torch.testing.assert_close(out.cpu(), want, rtol=0, atol=0, equal_nan=True)
    nan = out[255].view(torch.int32 if dt == "f32" else torch.int16).cpu()
    assert (nan == {"f32": 0x7FC00000, "f16": 0x7E00, "bf16": 0x7FC0}[dt]).all()


@pytest.mark.parametrize("dt", list(DTS))
@pytest.mark.parametrize("rows, cols, ld, out_ld, off", [(1, 1, 1, 1, 0), (7, 97, 5, 101, 1), (130, 64, 2, 64, 0),
                                                         (33, 200, 9, 211, 3), (3, 8, 1, 8, 0), (64, 1001, 32, 1001, 0)])
def test_dequantize_strided(rows, cols, ld, out_ld, off, dt):
    g = np.random.default_rng(rows)
    codes, scales = _mx.random_mx(g, rows, ld)
    kb = _mx.blocks(cols)
    buf = torch.full((rows * out_ld + off + 8,), 7.0, dtype=DTS[dt], device=DEV)
    out = buf[off:off + rows * out_ld].view(rows, out_ld)[:, :cols]
    zdp.mx_dequantize(_up(codes)[:, :16 * kb], _up(scales)[:, :kb], out)
    want = torch.from_numpy(_mx.decode(codes, scales)[:, :cols]).to(DTS[dt])
    torch.testing.assert_close(out.cpu(), want, rtol=0, atol=0)
    mark = buf.clone()
    mark[off:off + rows * out_ld].view(rows, out_ld)[:, :cols] = 7.0
    assert (mark == 7.0).all(), "values outside the matrix were written"


@pytest.mark.parametrize("blocks", [1, 3])
def test_grid_stride_rounds(blocks):
    """The streaming loops under a capped grid: the same outputs."""
    x = _inputs(300, 1100, "bf16", 11)
    flat = _inputs(1, 100_003, "f32", 12)[0]
    zdp.set_grid_limit(blocks)
    try:
        c, s = zdp.mx_empty(300, 1100)
        ct, st = zdp.mx_empty(1100, 300)
        zdp.mx_quantize(x, c, s, ct, st)
        out = torch.empty_like(x)
        zdp.mx_dequantize(c, s, out)
        fc, fs = zdp.mx_empty(1, 100_003)
        zdp.mx_cast_writeback(flat, fc.view(-1), fs.view(-1))
        fout = torch.empty_like(flat)
        zdp.mx_dequantize(fc.view(-1), fs.view(-1), fout)
        st8, ws = zdp.new_state(1.0), zdp.new_workspace(1)
        avg = torch.empty_like(flat)
        zdp.mx_reduce_grad_segment([fc.view(-1)] * 2, [fs.view(-1)] * 2, avg, ws, 0, st8)
        y = torch.empty(300, 300, device=DEV)
        zdp.mx_product(c, s, c, s, y)
        torch.cuda.synchronize()
    finally:
        zdp.set_grid_limit(0)
    want = _mx.quantize(_f64(x))
    _check_mx(c, s, want, "rows")
    _check_mx(ct, st, _mx.quantize(_f64(x).T), "columns")
    np.testing.assert_array_equal(_f64(out), _mx.decode(*want)[:, :1100])
    fw = _mx.decode(*_mx.quantize(_f64(flat)[None]))[0, :100_003]
    np.testing.assert_array_equal(_f64(fout), fw)
    with np.errstate(over="ignore"):  # the largest fp32 value plus itself
        np.testing.assert_array_equal(down32(avg), _plain_average([_down(fc[0])] * 2, [_down(fs[0])] * 2, 100_003))
    _check_product(y, (_down(c), _down(s)), (_down(c), _down(s)), "f32")


# --------------------------------------------------------------------------
# average of the copies
# --------------------------------------------------------------------------

def _plain_average(codes, scales, n):
    acc = np.zeros(n, np.float32)
    for c, s in zip(codes, scales):
        acc = acc + _mx.decode(c, s)[:n].astype(np.float32)
    return acc if len(codes) == 1 else acc / np.float32(len(codes))


@pytest.mark.parametrize("n", [0, 1, 31, 32, 33, 2049, 196_993, 1_048_577])
@pytest.mark.parametrize("n_d", [1, 2, 3, 8])
def test_average(n, n_d):
    _average_case(n, n_d, spaced=False)


@pytest.mark.parametrize("n_d", [7, 9, 16, 63, 64, 65, 100])
def test_average_of_many_copies(n_d):
    _average_case(5003, n_d, spaced=True)


def _average_case(n, n_d, spaced, scale=512.0):
    g = np.random.default_rng(n * 100 + n_d)
    kb = _mx.blocks(n)
    codes, scales = _mx.random_mx(g, n_d, kb, 115, 125)
    if spaced:
        cd, sd = _up(codes), _up(scales)
        cl, sl = list(cd.unbind(0)), list(sd.unbind(0))
    else:
        cl, sl = [_up(c) for c in codes], [_up(s) for s in scales]
    buf = torch.full((n + 9,), -3.0, device=DEV)
    avg = buf[1:n + 1]  # any 4-byte alignment
    st, ws = zdp.new_state(scale), zdp.new_workspace(1)
    zdp.mx_reduce_grad_segment(cl, sl, avg, ws, 0, st)
    zdp.grad_norm_overflow(None, ws, 1, st)
    want = _plain_average(codes, scales, n)
    assert_bits_equal(down32(avg), want, "average")
    assert (buf[:1] == -3.0).all() and (buf[n + 1:] == -3.0).all()
    r = zdp.read_state(st)
    norm2 = float(np.sum((want * np.float32(1.0 / scale)).astype(np.float64) ** 2))
    assert r["overflow"] == 0
    assert abs(r["grad_norm_sq"] - norm2) <= 1e-10 * norm2  # the same squares, grouped otherwise


@pytest.mark.parametrize("n, n_d, at", [(100, 2, (1, 3)), (1_200_003, 3, (0, 0)), (64, 1, (0, 1)), (33, 4, (3, 1))])
def test_a_nan_block_sets_the_flag(n, n_d, at):
    g = np.random.default_rng(n)
    codes, scales = _mx.random_mx(g, n_d, _mx.blocks(n), 115, 125)
    scales[at] = 255
    avg = torch.empty(n, device=DEV)
    st, ws = zdp.new_state(1.0), zdp.new_workspace(2)
    zdp.mx_reduce_grad_segment([_up(c) for c in codes], [_up(s) for s in scales], avg, ws, 1, st)
    clean = torch.zeros(64, device=DEV)
    zc, zs = _up(np.zeros(32, np.uint8)), _up(np.full(2, 127, np.uint8))
    zdp.mx_reduce_grad_segment([zc], [zs], clean, ws, 0, st)
    zdp.grad_norm_overflow(None, ws, 2, st, zdp.policy(skip_on_overflow=True))
    r = zdp.read_state(st)
    assert r["overflow"] == 1 and r["skipped"] == 1 and np.isnan(r["grad_norm"])
    lo, hi = 32 * at[1], min(n, 32 * at[1] + 32)
    got = down32(avg)
    assert np.isnan(got[lo:hi]).all() and np.isfinite(np.delete(got, np.s_[lo:hi])).all()


def test_codes_past_the_end_do_not_count():
    """The unused codes of a short last block are not the shard's: neither the norm nor the flag sees them."""
    codes = np.full((1, 32), 0x77, np.uint8)
    scales = np.array([[127, 127]], np.uint8)
    avg = torch.empty(33, device=DEV)
    st, ws = zdp.new_state(1.0), zdp.new_workspace(1)
    zdp.mx_reduce_grad_segment([_up(codes[0])], [_up(scales[0])], avg, ws, 0, st)
    zdp.grad_norm_overflow(None, ws, 1, st)
    assert zdp.read_state(st)["grad_norm_sq"] == 33 * 36.0


@pytest.mark.parametrize("n_d", [1, 4, 8])
def test_average_is_the_16_bit_average_of_the_widened_copies(n_d):
    """bf16 holds the format's values exactly, so both averaging passes add the same numbers."""
    n = 300_007
    g = np.random.default_rng(n_d)
    codes, scales = _mx.random_mx(g, n_d, _mx.blocks(n), 100, 130)
    cl, sl = [_up(c) for c in codes], [_up(s) for s in scales]
    wide = []
    for c, s in zip(cl, sl):
        out = torch.empty(n, dtype=torch.bfloat16, device=DEV)
        zdp.mx_dequantize(c, s, out)
        wide.append(out)
    got = []
    for f in (lambda a, w, st: zdp.mx_reduce_grad_segment(cl, sl, a, w, 0, st),
              lambda a, w, st: zdp.reduce_grad_segment(wide, a, w, 0, st)):
        avg, st, ws = torch.empty(n, device=DEV), zdp.new_state(64.0), zdp.new_workspace(1)
        f(avg, ws, st)
        zdp.grad_norm_overflow(None, ws, 1, st)
        got.append((down32(avg), zdp.read_state(st)))
    assert_bits_equal(got[0][0], got[1][0], "average")
    a, b = got[0][1]["grad_norm_sq"], got[1][1]["grad_norm_sq"]
    assert abs(a - b) <= 1e-12 * b


# --------------------------------------------------------------------------
# product
# --------------------------------------------------------------------------

def _check_product(out, a, b, dt, what=""):
    ref, size = _mx.product(*a, *b)
    got = _f64(out)
    k = 32 * a[1].shape[1]
    nan = np.isnan(ref)
    np.testing.assert_array_equal(np.isnan(got), nan, err_msg=f"{what}: NaN")
    got, ref, size = got[~nan], ref[~nan], size[~nan]
    bound = k * 2.0 ** -23 * size
    # a value rounds to infinity from half a step above the type's largest on, (2 - eps / 2) * 2^emax
    top = float(torch.finfo(DTS[dt]).max)
    limit = top * (2 - HALF_STEP[dt]) / (2 - 2 * HALF_STEP[dt])
    inf = np.isinf(got)
    assert inf[np.abs(ref) - bound >= limit].all(), f"{what}: finite where the sum overflows"
    assert (np.abs(ref) + bound >= limit)[inf].all(), f"{what}: infinite where the sum does not overflow"
    assert (np.signbit(got) == np.signbit(ref))[inf].all()
    bound = bound + HALF_STEP[dt] * (np.abs(ref) + bound) + TINY[dt]
    err, bound = np.abs(got - ref)[~inf], bound[~inf]
    bad = err > bound
    assert not bad.any(), (f"{what}: {bad.sum()} of {err.size} outputs outside the bound, worst "
                           f"{np.max(err / np.maximum(bound, 1e-300))} times")
    if dt == "f32" and err.size and np.linalg.norm(ref) > 0 and not inf.any():
        assert np.linalg.norm(err) <= 1e-6 * np.linalg.norm(size), what


PRODUCTS = [(1, 1, 1), (1, 33, 2), (2, 5, 7), (31, 32, 3), (32, 64, 8), (33, 65, 9), (1, 1000, 128), (3, 4096, 33),
            (45, 1600, 50), (64, 130, 16), (65, 257, 17), (128, 128, 24), (129, 300, 31), (200, 77, 130),
            (256, 256, 8), (257, 511, 40), (500, 1030, 20), (1030, 140, 12), (2048, 16, 9), (17, 3000, 64),
            (512, 768, 90), (1100, 2100, 7), (300, 4500, 200)]


@pytest.mark.parametrize("dt", list(DTS))
@pytest.mark.parametrize("m, n, kb", PRODUCTS)
def test_product(m, n, kb, dt):
    g = np.random.default_rng(m * 31 + n * 7 + kb)
    a, b = _mx.random_mx(g, m, kb, 118, 126), _mx.random_mx(g, n, kb, 118, 126)
    out = torch.full((m, n), 9.0, dtype=DTS[dt], device=DEV)
    args = [_up(t) for t in (*a, *b)]
    zdp.mx_product(*args, out)
    _check_product(out, a, b, dt)
    again = torch.empty_like(out)
    zdp.mx_product(*args, again)
    assert torch.equal(out, again), "another run gave other bits"


@pytest.mark.parametrize("dt", list(DTS))
@pytest.mark.parametrize("m, n, kb, extra", [(5, 40, 3, 1), (70, 100, 9, 3), (300, 260, 18, 5), (260, 1000, 50, 2)])
def test_product_strided(m, n, kb, extra, dt):
    """Operands and output inside wider arrays: odd block strides, scales at odd addresses."""
    g = np.random.default_rng(m)
    a, b = _mx.random_mx(g, m, kb + extra), _mx.random_mx(g, n, kb + extra)
    a[1][:, kb:] = 255  # what lies past the operand is not read into the sum
    b[1][:, :extra] = 255
    ca, sa, cb, sb = (_up(t) for t in (*a, *b))
    buf = torch.full((m, n + 3), 5.0, dtype=DTS[dt], device=DEV)
    out = buf[:, 1:n + 1]
    zdp.mx_product(ca[:, :16 * kb], sa[:, :kb], cb[:, 16 * extra:], sb[:, extra:], out)
    _check_product(out, (a[0][:, :16 * kb], a[1][:, :kb]), (b[0][:, 16 * extra:], b[1][:, extra:]), dt)
    assert (buf[:, 0] == 5.0).all() and (buf[:, n + 1:] == 5.0).all()


def _check_large(out, a, b, dt):
    """_check_product's bound with the 64-bit products on the device."""
    a64, b64 = (torch.from_numpy(_mx.decode(*t)).to(DEV) for t in (a, b))
    ref, size = a64 @ b64.t(), a64.abs() @ b64.abs().t()
    got, nan = out.double(), torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan)
    got, ref, size = got[~nan], ref[~nan], size[~nan]
    bound = a64.shape[1] * 2.0 ** -23 * size
    bound = bound + HALF_STEP[dt] * (ref.abs() + bound) + TINY[dt]
    err = (got - ref).abs()
    assert torch.isfinite(got).all() and (err <= bound).all(), f"worst {float((err / bound).max())} of the bound"
    if dt == "f32":
        assert float(err.norm()) <= 1e-6 * float(size.norm())


# Whole and partial chunks of 8 blocks, whole and partial groups of 4 chunks, on both sides of each.
TILE_BLOCKS = [8, 9, 15, 16, 23, 24, 31, 32, 33, 40, 41, 50, 63, 64, 65, 71, 100]


@pytest.mark.parametrize("kb", TILE_BLOCKS)
@pytest.mark.parametrize("m, n", [(1700, 1600), (1665, 1603), (3300, 3328), (3311, 3331)])
def test_product_of_many_tiles(m, n, kb):
    """Enough output for the tiles of 128 and 256, ragged and whole, rows of outputs on and off 16 bytes; operands
    dense and inside wider arrays at odd strides."""
    g = np.random.default_rng(m + kb)
    dt = list(DTS)[(kb + m) % 3]
    extra = (kb * 7 + n) % 4
    a, b = _mx.random_mx(g, m, kb + extra, 118, 126), _mx.random_mx(g, n, kb + extra, 118, 126)
    a[1][:, kb:] = 255
    b[1][:, kb:] = 255
    a[1][m // 3, kb - 1] = 255  # one row of NaN
    args = [_up(t) for t in (*a, *b)]
    args = [t[:, :kb * (16 if q % 2 == 0 else 1)] for q, t in enumerate(args)]
    out = torch.full((m, n), 9.0, dtype=DTS[dt], device=DEV)
    zdp.mx_product(*args, out)
    cut = tuple((c[:, :16 * kb], s[:, :kb]) for c, s in (a, b))
    _check_large(out, *cut, dt)
    again = torch.empty_like(out)
    zdp.mx_product(*args, again)
    assert torch.equal(out.view(torch.int32 if dt == "f32" else torch.int16),
                       again.view(torch.int32 if dt == "f32" else torch.int16)), "another run gave other bits"


@pytest.mark.parametrize("m, n", [(1700, 1600), (3300, 3331)])
def test_product_of_many_tiles_inside_a_wider_output(m, n):
    g = np.random.default_rng(n)
    a, b = _mx.random_mx(g, m, 18, 118, 126), _mx.random_mx(g, n, 18, 118, 126)
    for dt in DTS:
        buf = torch.full((m, n + 5), 5.0, dtype=DTS[dt], device=DEV)
        out = buf[:, 3:n + 3]
        zdp.mx_product(*(_up(t) for t in (*a, *b)), out)
        _check_large(out, a, b, dt)
        assert (buf[:, :3] == 5.0).all() and (buf[:, n + 3:] == 5.0).all()


def test_captured_without_a_call_before():
    """The first call of a kernel with more LDS than the default may be a captured one."""
    a, b = (torch.randint(0, 256, (r, 16 * 20), dtype=torch.uint8, device=DEV) for r in (1800, 1900))
    sa, sb = (torch.randint(118, 126, (r, 20), dtype=torch.uint8, device=DEV) for r in (1800, 1900))
    out, want = (torch.empty(1800, 1900, dtype=torch.float16, device=DEV) for _ in range(2))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zdp.mx_product(a, sa, b, sb, out)
    zdp.mx_product(a, sa, b, sb, want)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_first_calls_of_a_process_are_captured():
    """Every variant, in a process where no call came before the capture."""
    script = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_mx_first_capture.py")
    r = subprocess.run([sys.executable, script], capture_output=True, text=True, timeout=110)
    assert r.returncode == 0 and "first calls captured: ok" in r.stdout, r.stdout[-1000:] + r.stderr[-3000:]


@pytest.mark.parametrize("m, n, kb", [(3, 40, 5), (70, 90, 20), (300, 520, 33)])
def test_product_nan_blocks_and_extreme_scales(m, n, kb):
    g = np.random.default_rng(kb)
    a, b = _mx.random_mx(g, m, kb, 0, 60), _mx.random_mx(g, n, kb, 150, 254)  # products stay inside fp32
    a[1][m // 2, kb // 2] = 255
    b[1][n - 1, kb - 1] = 255
    a[0][0] = 0  # a row of zeros
    out = torch.empty(m, n, device=DEV)
    zdp.mx_product(*(_up(t) for t in (*a, *b)), out)
    _check_product(out, a, b, "f32")
    assert torch.isnan(out[m // 2]).all() and torch.isnan(out[:, n - 1]).all()


def test_product_overflow_to_infinity():
    a, b = np.full((40, 16), 0x77, np.uint8), np.full((40, 16), 0x77, np.uint8)
    s = np.full((40, 1), 200, np.uint8)
    out = torch.empty(40, 40, device=DEV)
    zdp.mx_product(_up(a), _up(s), _up(b), _up(s), out)
    assert torch.isposinf(out).all()
    s = np.full((40, 1), 134, np.uint8)  # 32 * 36 * 2^14 is past fp16's largest
    half = torch.empty(40, 40, dtype=torch.float16, device=DEV)
    zdp.mx_product(_up(a), _up(s), _up(b), _up(s), half)
    assert torch.isposinf(half).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("low", [-166, -158, -150, -142, -134, -126])
@pytest.mark.parametrize("m, n, kb", [(3, 40, 5), (70, 90, 20), (300, 520, 33), (1700, 1600, 9), (3300, 3328, 11)])
def test_product_terms_around_the_smallest_fp32_values(m, n, kb, low, dt):
    """Terms whose scales multiply to 2^low to 2^(low + 6): below fp32's smallest value, among its subnormals, above.

    To the bound of other products come up to 2^-149 for each term (what of it lies below fp32's smallest step) and as
    much again for each of at most as many additions (a subnormal sum rounded or cut)."""
    g = np.random.default_rng(m - low)
    lo = (254 + low) // 2
    a, b = _mx.random_mx(g, m, kb, lo, lo + 4), _mx.random_mx(g, n, kb, 254 + low - lo, 254 + low - lo + 4)
    out = torch.full((m, n), 9.0, dtype=DTS[dt], device=DEV)
    zdp.mx_product(*(_up(t) for t in (*a, *b)), out)
    a64, b64 = (torch.from_numpy(_mx.decode(*t)).to(DEV) for t in (a, b))
    ref, size, k = a64 @ b64.t(), a64.abs() @ b64.abs().t(), 32 * kb
    bound = k * 2.0 ** -23 * size + 2 * k * 2.0 ** -149
    bound = bound + HALF_STEP[dt] * (ref.abs() + bound) + TINY[dt]
    err = (out.double() - ref).abs()
    assert (err <= bound).all(), f"worst {float((err / bound).max())} of the bound"
    if low >= (-142 if dt == "f32" else -134):  # most outputs lie well above the smallest step of their type
        assert float(((out.double() - ref).abs() < ref.abs()).double().mean()) > 0.9
    if low <= -150:
        assert float(out.double().abs().max()) < 2.0 ** -126, "no subnormal sums"


def test_product_of_the_smallest_scales_is_zero():
    c, s = np.full((40, 32), 0x77, np.uint8), np.zeros((40, 2), np.uint8)
    out = torch.full((40, 40), 9.0, device=DEV)
    zdp.mx_product(_up(c), _up(s), _up(c), _up(s), out)
    assert (out == 0.0).all()  # 64 * 36 * 2^-254


@pytest.mark.parametrize("m, n, kb", [(0, 5, 2), (5, 0, 2), (4, 6, 0), (300, 300, 0)])
def test_empty_products(m, n, kb):
    out = torch.full((m, n), 3.0, device=DEV)
    z = lambda r: (torch.zeros(r, 16 * kb, dtype=torch.uint8, device=DEV),  # noqa: E731
                   torch.zeros(r, kb, dtype=torch.uint8, device=DEV))
    zdp.mx_product(*z(m), *z(n), out)
    assert (out == 0.0).all()  # an empty sum


def test_product_of_a_tensor_in_the_flat_vector():
    """The weights straight out of the flat vector that the writeback filled."""
    n, k, off = 200, 160, 32 * 7
    master = up32(np.random.default_rng(2).normal(size=off + n * k + 17) * 0.02)
    c, s = zdp.mx_empty(1, master.numel())
    c, s = c.view(-1), s.view(-1)
    zdp.mx_cast_writeback(master, c, s)
    wc, wsc = zdp.mx_view(c, s, off, n, k)
    x = _inputs(30, k, "bf16", 4, rare=False)
    xc, xs = zdp.mx_empty(30, k)
    zdp.mx_quantize(x, xc, xs)
    out = torch.empty(30, n, dtype=torch.bfloat16, device=DEV)
    zdp.mx_product(xc, xs, wc, wsc, out)
    w = _mx.quantize(_f64(master)[off:off + n * k].reshape(n, k))
    _check_product(out, _mx.quantize(_f64(x)), w, "bf16")


# --------------------------------------------------------------------------
# together, as a training step uses them
# --------------------------------------------------------------------------

def _grid_matrix(g, rows, cols):
    """Values the format holds exactly along either way under the scale 2^-3: magnitudes of the grid with a 6 in every
    block of 32 along the rows and along the columns, so that every block gets the same scale."""
    v = g.choice(np.concatenate([_mx.GRID, -_mx.GRID]), (rows, cols)) / 8
    for i in range(0, rows, 32):
        for j in range(0, cols, 32):
            for t in range(32):
                v[i + t, j + t] = 6 / 8
    return v.astype(np.float32)


def test_gradients_of_a_layer():
    """y = x W^T with operands the format holds: y, dx and dW are the formula's, and a step in one weight changes
    sum(dy * y) by its gradient times the step (exactly: all of it is small integers over 256)."""
    g = np.random.default_rng(8)
    t, o, i = 64, 96, 160
    x, w, dy = _grid_matrix(g, t, i), _grid_matrix(g, o, i), _grid_matrix(g, t, o)

    def both(v):
        c, s = zdp.mx_empty(*v.shape)
        ct, st = zdp.mx_empty(v.shape[1], v.shape[0])
        zdp.mx_quantize(up32(v), c, s, ct, st)
        return c, s, ct, st

    X, W, D = both(x), both(w), both(dy)
    y, dx, dw = (torch.empty(s, device=DEV) for s in ((t, o), (t, i), (o, i)))
    zdp.mx_product(*X[:2], *W[:2], y)
    zdp.mx_product(*D[:2], *W[2:], dx)
    zdp.mx_product(*D[2:], *X[2:], dw)
    x64, w64, d64 = (v.astype(np.float64) for v in (x, w, dy))
    np.testing.assert_array_equal(_f64(y), x64 @ w64.T)
    np.testing.assert_array_equal(_f64(dx), d64 @ w64)
    np.testing.assert_array_equal(_f64(dw), d64.T @ x64)
    for a, b in ((3, 50), (90, 7)):
        moved = w.copy()
        old = moved[a, b]
        moved[a, b] = 0.25 if old != 0.25 else 0.5
        M = both(moved)
        y2 = torch.empty_like(y)
        zdp.mx_product(*X[:2], *M[:2], y2)
        diff = float((_f64(y2) * d64).sum() - (_f64(y) * d64).sum())
        assert diff == float(dw[a, b]) * float(moved[a, b] - old)


def test_a_step_in_4_bits():
    """Two ranks' gradient copies in 4 bits, their average, an AdamW step, the writeback in 4 bits, and the products
    of the next forward and backward; each stage against its plain form on the stage's own inputs."""
    t, o, i, n_d = 96, 200, 160, 2
    n = o * i
    g = np.random.default_rng(5)
    master0 = (g.normal(size=n) * 0.02).astype(np.float32)
    master, m, v = up32(master0), torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    c, s = (f.view(-1) for f in zdp.mx_empty(1, n))
    scale = 256.0
    st, ws = zdp.new_state(scale), zdp.new_workspace(1)
    pol = zdp.policy(skip_on_overflow=True)
    plain_step = _AdamW(master0)
    zdp.mx_cast_writeback(master, c, s)
    for step in range(3):
        copies = []
        for r in range(n_d):
            x = torch.from_numpy(g.normal(size=(t, i))).to(torch.bfloat16).to(DEV)
            dy = torch.from_numpy(g.normal(size=(t, o)) * 1e-3 * scale).to(torch.bfloat16).to(DEV)
            if step == 1 and r == 1:
                dy[5, 9] = float("inf")
            wc, wsc = zdp.mx_view(c, s, 0, o, i)
            w16 = torch.empty(o, i, dtype=torch.bfloat16, device=DEV)
            zdp.mx_dequantize(wc, wsc, w16)
            X, D, WT = (*zdp.mx_empty(t, i), *zdp.mx_empty(i, t)), (*zdp.mx_empty(t, o), *zdp.mx_empty(o, t)), zdp.mx_empty(i, o)
            zdp.mx_quantize(x, *X)
            zdp.mx_quantize(dy, *D)
            zdp.mx_quantize(w16, codes_t=WT[0], scales_t=WT[1])
            y, dx = torch.empty(t, o, dtype=torch.bfloat16, device=DEV), torch.empty(t, i, dtype=torch.bfloat16, device=DEV)
            dw = torch.empty(o, i, device=DEV)
            zdp.mx_product(*X[:2], wc, wsc, y)
            zdp.mx_product(*D[:2], *WT, dx)
            zdp.mx_product(*D[2:], *X[2:], dw)
            xq, dq, xt, dt_ = _mx.quantize(_f64(x)), _mx.quantize(_f64(dy)), _mx.quantize(_f64(x).T), _mx.quantize(_f64(dy).T)
            w64 = _f64(w16)
            _check_product(y, xq, _mx.quantize(w64), "bf16", "y")
            _check_product(dx, dq, _mx.quantize(w64.T), "bf16", "dx")
            _check_product(dw, dt_, xt, "f32", "dW")
            gc, gs = (f.view(-1) for f in zdp.mx_empty(1, n))
            zdp.mx_cast_writeback(dw.view(-1), gc, gs)
            want = _mx.quantize(_f64(dw).reshape(1, -1))
            _check_mx(gc, gs, (want[0][0], want[1][0]), "gradient copy")
            copies.append((gc, gs))
        avg = torch.empty(n, device=DEV)
        zdp.mx_reduce_grad_segment([p[0] for p in copies], [p[1] for p in copies], avg, ws, 0, st)
        zdp.grad_norm_overflow(None, ws, 1, st, pol)
        zdp.adam_step([zdp.Group(master, m, v, avg=avg, lr=1e-3, weight_decay=0.1)], ws, st, pol)
        zdp.mx_cast_writeback(master, c, s)
        plain = _plain_average([_down(p[0]) for p in copies], [_down(p[1]) for p in copies], n)
        r = zdp.read_state(st)
        assert r["skipped"] == int(step == 1) and r["step"] == (1, 1, 2)[step]
        if step != 1:
            assert_bits_equal(down32(avg), plain, "average")
            plain_step(plain, scale if step == 0 else scale / 2)
        assert_bits_equal(down32(master), plain_step.master, f"master after call {step}")
        want = _mx.quantize(plain_step.master[None].astype(np.float64))
        _check_mx(c, s, (want[0][0], want[1][0]), "written parameters")


class _AdamW:
    """AdamW (lr 1e-3, decay 0.1) from an fp32 average, every operation in fp32, as the step defines it."""

    def __init__(self, master):
        self.master, self.m, self.v = master.copy(), np.zeros_like(master), np.zeros_like(master)
        self.p1 = self.p2 = 1.0

    def __call__(self, avg, scale):
        f = np.float32
        self.p1, self.p2 = self.p1 * 0.9, self.p2 * 0.999
        g = avg * f(1.0 / scale)
        th = self.master * f(1.0 - 1e-3 * 0.1)
        self.m = f(0.9) * self.m + f(1.0 - 0.9) * g
        self.v = f(0.999) * self.v + f(1.0 - 0.999) * (g * g)
        den = np.sqrt(self.v / f(1.0 - self.p2)) + f(1e-8)
        self.master = th - f(1e-3) * ((self.m / f(1.0 - self.p1)) / den)


# --------------------------------------------------------------------------
# streams, graphs, two calls at once
# --------------------------------------------------------------------------

def _chain(x, w, X, W, y, out):
    zdp.mx_quantize(x, *X)
    zdp.mx_quantize(w, *W)
    zdp.mx_product(X[0], X[1], W[0], W[1], y)
    zdp.mx_dequantize(X[0], X[1], out)


def test_captured_and_replayed():
    """The calls in a graph, replayed with new inputs and eager work between the replays, against the eager calls;
    the average with its norm as well."""
    t, o, i, n, n_d = 70, 300, 256, 40_003, 3
    x, w = torch.empty(t, i, dtype=torch.bfloat16, device=DEV), torch.empty(o, i, dtype=torch.bfloat16, device=DEV)
    X, W = (*zdp.mx_empty(t, i), *zdp.mx_empty(i, t)), (*zdp.mx_empty(o, i), *zdp.mx_empty(i, o))
    y, out = torch.empty(t, o, device=DEV), torch.empty(t, i, dtype=torch.float16, device=DEV)
    copies = [zdp.mx_empty(1, n) for _ in range(n_d)]
    cl, sl = [c.view(-1) for c, _ in copies], [s.view(-1) for _, s in copies]
    src, avg = torch.empty(n_d, n, device=DEV), torch.empty(n, device=DEV)
    st, ws = zdp.new_state(8.0), zdp.new_workspace(1)

    def calls():
        _chain(x, w, X, W, y, out)
        for r in range(n_d):
            zdp.mx_cast_writeback(src[r], cl[r], sl[r])
        zdp.mx_reduce_grad_segment(cl, sl, avg, ws, 0, st)
        zdp.grad_norm_overflow(None, ws, 1, st)

    def fill(seed):
        torch.manual_seed(seed)
        x.normal_()
        w.normal_(std=0.02)
        src.normal_(std=1e-3)

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    held = (X[0], X[1], X[2], X[3], W[0], W[1], y, out, avg, st)
    for seed in (1, 2, 3, 4):
        fill(seed)
        for b in held[:-1]:
            b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [b.clone() for b in held]
        for b in held[:-1]:
            b.zero_()
        calls()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, held)):
            assert torch.equal(a, b), f"replay {seed}: buffer {k} differs from the eager calls"


def test_two_streams_at_once():
    """Independent calls on two streams, each with its own buffers."""
    sets, want = [], []
    for k, (t, o, i) in enumerate(((300, 700, 512), (64, 900, 1024))):
        torch.manual_seed(k)
        x, w = torch.randn(t, i, device=DEV), torch.randn(o, i, device=DEV)
        sets.append((x, w, (*zdp.mx_empty(t, i), *zdp.mx_empty(i, t)), (*zdp.mx_empty(o, i), *zdp.mx_empty(i, o)),
                     torch.empty(t, o, device=DEV), torch.empty(t, i, device=DEV)))
        _chain(*sets[-1])
        want.append((sets[-1][4].clone(), sets[-1][5].clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for q in sets:
            q[4].zero_()
            q[5].zero_()
        torch.cuda.synchronize()
        for stream, q in zip(streams, sets):
            with torch.cuda.stream(stream):
                _chain(*q)
        torch.cuda.synchronize()
        for q, (y, out) in zip(sets, want):
            assert torch.equal(q[4], y) and torch.equal(q[5], out)


def test_a_named_stream():
    x = torch.randn(40, 64, device=DEV)
    c, s = zdp.mx_empty(40, 64)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    zdp.mx_quantize(x, c, s, stream=side)
    side.synchronize()
    _check_mx(c, s, _mx.quantize(_f64(x)), "rows")


def test_refusals_on_the_device():
    x = torch.zeros(4, 64, device=DEV)
    c, s = zdp.mx_empty(4, 64)
    flat_c, flat_s = c.view(-1), s.view(-1)
    with pytest.raises(ValueError):
        zdp.mx_quantize(x)
    with pytest.raises(ValueError):
        zdp.mx_quantize(x, c)
    with pytest.raises(ValueError):
        zdp.mx_quantize(x, c.cpu(), s)
    with pytest.raises(ValueError):
        zdp.mx_quantize(x, codes_t=c, scales_t=s)
    with pytest.raises(TypeError):
        zdp.mx_quantize(x.double(), c, s)
    with pytest.raises(ValueError, match="dense"):
        zdp.mx_quantize(x.t(), c, s)
    with pytest.raises(ValueError):
        zdp.mx_cast_writeback(x.view(-1)[:40], flat_c, flat_s, 0)  # ends inside a block that is not the last
    with pytest.raises(ValueError):
        zdp.mx_cast_writeback(x.view(-1)[:40], flat_c, flat_s, 16)
    with pytest.raises(ValueError):
        zdp.mx_dequantize(flat_c, flat_s, torch.empty(257, device=DEV))
    with pytest.raises(ValueError):
        zdp.mx_product(c, s, c[:, :16], s[:, :1], torch.empty(4, 4, device=DEV))
    with pytest.raises(ValueError):
        zdp.mx_product(c, s, c, s, torch.empty(4, 5, device=DEV))
    with pytest.raises(zdp.ZeroError):  # codes that do not start on a block
        odd = torch.zeros(4 * 32 + 16, dtype=torch.uint8, device=DEV)[8:8 + 128].view(4, 32)
        zdp.mx_quantize(x, odd, s)
    st, ws = zdp.new_state(), zdp.new_workspace(1)
    with pytest.raises(ValueError):
        zdp.mx_reduce_grad_segment([flat_c], [], torch.empty(8, device=DEV), ws, 0, st)
    with pytest.raises(ValueError):
        zdp.mx_reduce_grad_segment([flat_c], [flat_s], torch.empty(300, device=DEV), ws, 0, st)


def test_a_matrix_in_the_place_of_a_flat_vector_is_refused():
    """Rows of 40 values are padded to 64: none of the flat calls reads or writes them as 1,280 values in a row."""
    c, s = zdp.mx_empty(32, 40)
    marked = [t.fill_(0xA5) for t in (c, s)]
    out = torch.full((1280,), 3.0, device=DEV)
    st, ws = zdp.new_state(), zdp.new_workspace(1)
    for codes, scales in ((c, s), (c.view(-1), s), (c, s.view(-1))):
        with pytest.raises(ValueError, match="dimensions"):
            zdp.mx_dequantize(codes, scales, out)
        with pytest.raises(ValueError, match="dimensions"):
            zdp.mx_cast_writeback(torch.zeros(1280, device=DEV), codes, scales)
        with pytest.raises(ValueError, match="dimensions"):
            zdp.mx_reduce_grad_segment([codes], [scales], out, ws, 0, st)
    assert (out == 3.0).all() and all((t == 0xA5).all() for t in marked)
